"""Refusals and workspace sizes of the calls that record attention weights and
of the eviction, through the C ABI without a GPU; the allocator's side of it."""

import ctypes

import numpy as np
import pytest

P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
X = P(1 << 20)  # a 16-byte aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib(cuda_lib_path):
    lib = ctypes.CDLL(cuda_lib_path)
    lib.pkv_last_error.restype = ctypes.c_char_p
    for name, n in (("pkv_decode_weights_workspace_bytes", 7), ("pkv_evict_workspace_bytes", 5), ("pkv_decode_workspace_bytes", 7)):
        getattr(lib, name).restype = sz
        getattr(lib, name).argtypes = [i32] * n
    lib.pkv_prefill_weights_workspace_bytes.restype = sz
    lib.pkv_prefill_weights_workspace_bytes.argtypes = [i32, i64] + [i32] * 6
    return lib


def prefill(lib, Tq=10, Hq=4, Hkv=2, D=64, NB=8, bs=16, B=2, MBS=4, max_q=5, window=0, weights=X, ws=X, ws_bytes=1 << 30, scale=0.1):
    return lib.pkv_paged_prefill_weights(X, X, X, X, MBS, X, X, B, i64(Tq), max_q, Hq, Hkv, D, i64(NB), bs, f32(scale), X,
                                         weights, window, ws, sz(ws_bytes), None, None)


Y = P(1 << 21)


def evict(lib, k=X, v=Y, w=X, tables=X, MBS=4, lens=X, B=2, Hkv=2, D=64, eb=2, NB=8, bs=16, budget=20, recent=5, out=X, ws=X, ws_bytes=1 << 30):
    return lib.pkv_evict_kvcache(k, v, w, tables, MBS, lens, B, Hkv, D, eb, i64(NB), bs, budget, recent, out, ws,
                                 sz(ws_bytes), None, None)


def test_workspace_sizes(lib):
    up = lambda n: n + -n % 256
    base = lib.pkv_decode_workspace_bytes(4, 4, 2, 64, 19, 16, 0)
    boxes = 4 * 2 * 19
    want = up(up(up(base) + 4 * 4 * 4) + boxes * 16) + boxes * 16 * 2 * 4
    assert lib.pkv_decode_weights_workspace_bytes(4, 4, 2, 64, 19, 16, 0) == want
    assert lib.pkv_decode_weights_workspace_bytes(0, 4, 2, 64, 19, 16, 0) == 0
    assert lib.pkv_decode_weights_workspace_bytes(4, 6, 4, 64, 19, 16, 0) == 0
    f = lib.pkv_prefill_weights_workspace_bytes
    # log-sum-exps and a counter (a few tokens need no partial sums of weights); 1 pair of query tiles x 2 KV heads x 3 sequences are 6 items
    base = up(100 * 4 * 4 + 4)
    assert f(3, 100, 40, 4, 2, 64, 4, 16) == base  # contexts too short to split
    # 8192 tokens are 64 tiles, 16 splits of 4: a log-sum-exp and 64 outputs per split and row
    assert f(3, 100, 40, 4, 2, 64, 512, 16) == base + up(16 * 400 * 4) + 16 * 400 * 64 * 4
    assert f(3, 100, 40, 4, 2, 64, 1 << 16, 16) == base + up(51 * 400 * 4) + 51 * 400 * 64 * 4  # 304 items in all
    assert f(3, 100, 40, 4, 2, 64, 4, 16) == f(3, 100, 1000, 4, 2, 64, 4, 16) - up(152 * 8 * 4) - 152 * 16 * 256 * 4
    assert f(76, 1 << 20, 20, 4, 2, 64, 512, 16) == up((1 << 22) * 4 + 4)  # 152 items: none split
    assert f(0, 100, 4, 4, 2, 64, 4, 16) == 0 and f(3, 0, 4, 4, 2, 64, 4, 16) == 0 and f(3, 10, 4, 5, 2, 64, 4, 16) == 0
    # per (sequence, KV head) the range that moves, and where the kept tokens come from
    assert lib.pkv_evict_workspace_bytes(3, 2, 4, 16, 20) == up(3 * 2 * 8) + 3 * 2 * 20 * 4
    # a budget above what the tables can name needs no more than that
    assert lib.pkv_evict_workspace_bytes(3, 2, 4, 16, 1 << 30) == lib.pkv_evict_workspace_bytes(3, 2, 4, 16, 64)
    assert lib.pkv_evict_workspace_bytes(0, 2, 4, 16, 20) == 0
    assert lib.pkv_evict_workspace_bytes(3, 2, 4, 16, 0) == 0


@pytest.mark.parametrize("kw,status,text", [
    (dict(window=-1), INVALID, b"window"),
    (dict(weights=None), INVALID, b"weights"),
    (dict(weights=P((1 << 20) + 8)), INVALID, b"weights"),
    (dict(ws=None), WORKSPACE, b"workspace"),
    (dict(ws_bytes=159), WORKSPACE, b"workspace"),
    (dict(MBS=4096, ws_bytes=256), WORKSPACE, b"workspace"),
    (dict(max_q=1000, ws_bytes=256), WORKSPACE, b"workspace"),
    (dict(ws=P((1 << 20) + 4)), WORKSPACE, b"workspace"),
    (dict(Hq=3), INVALID, b"multiple"),
    (dict(Hq=6, Hkv=2), UNSUPPORTED, b"Hq/Hkv"),
    (dict(D=96), UNSUPPORTED, b"head_dim"),
    (dict(bs=24), UNSUPPORTED, b"block_size"),
    (dict(scale=float("inf")), INVALID, b"scale"),
    (dict(Hq=1 << 20, Hkv=1 << 20, B=2048), UNSUPPORTED, b"2^31"),
])
def test_prefill_weights_refusals(lib, kw, status, text):
    assert prefill(lib, **kw) == status
    assert text in lib.pkv_last_error()


@pytest.mark.parametrize("kw", [dict(B=0), dict(Tq=0), dict(max_q=0)])
def test_prefill_weights_nothing_to_do(lib, kw):
    assert prefill(lib, weights=None, ws=None, ws_bytes=0, **kw) == OK


@pytest.mark.parametrize("kw,status,text", [
    (dict(budget=0), INVALID, b"budget"),
    (dict(recent=-1), INVALID, b"recent"),
    (dict(recent=21), INVALID, b"recent"),
    (dict(B=-1), INVALID, b"sizes"),
    (dict(MBS=0), INVALID, b"sizes"),
    (dict(NB=0), INVALID, b"sizes"),
    (dict(D=32), UNSUPPORTED, b"head_dim"),
    (dict(eb=4), UNSUPPORTED, b"element"),
    (dict(bs=20), UNSUPPORTED, b"block_size"),
    (dict(NB=1 << 27), INVALID, b"2^31"),
    (dict(MBS=1 << 27), INVALID, b"2^31"),
    (dict(B=65536), UNSUPPORTED, b"65535"),
    (dict(Hkv=65536), UNSUPPORTED, b"65535"),
    (dict(k=None), INVALID, b"null"), (dict(v=None), INVALID, b"null"), (dict(w=None), INVALID, b"null"),
    (dict(tables=None), INVALID, b"null"), (dict(lens=None), INVALID, b"null"), (dict(out=None), INVALID, b"null"),
    (dict(k=P((1 << 20) + 8)), INVALID, b"misaligned"), (dict(w=P((1 << 20) + 4)), INVALID, b"misaligned"),
    (dict(out=P((1 << 20) + 2)), INVALID, b"misaligned"),
    (dict(v=X), INVALID, b"same memory"),
    (dict(ws=None), WORKSPACE, b"workspace"),
    (dict(ws_bytes=64), WORKSPACE, b"workspace"),
])
def test_evict_refusals(lib, kw, status, text):
    assert evict(lib, **kw) == status
    assert text in lib.pkv_last_error()


def test_evict_of_no_sequences(lib):
    assert evict(lib, B=0, ws=None, ws_bytes=0) == OK


def test_decode_weights_refuses_sizes(lib):
    for name, scales in (("pkv_paged_attn_decode_weights", []), ("pkv_paged_attn_decode_weights_fp8", [f32(1), f32(1)])):
        f = getattr(lib, name)
        call = lambda Hq=4, Hkv=2, D=64, bs=16, B=2, s=scales: f(X, X, X, X, 4, X, B, Hq, Hkv, D, i64(8), bs, f32(0.1), *s, X, X,
                                                                 X, sz(1 << 30), 0, None, None)
        assert call(Hq=3) == INVALID
        assert call(D=96) == UNSUPPORTED
        assert call(bs=24) == UNSUPPORTED
        assert call(B=0) == OK
        if scales:
            assert call(s=[f32(0), f32(1)]) == INVALID


# --------------------------------------------------------- the allocator's side


@pytest.fixture
def bm(cuda_lib_path):
    from paged_kv_cache_85_gb300.block_manager import BlockManager

    return BlockManager(16, 4)


def test_evict_gives_blocks_back_and_appends_go_on(bm):
    bm.allocate(1, np.arange(18))
    table = bm.block_table(1)
    assert len(table) == 5 and bm.num_free_blocks == 11
    bm.evict(1, 100)  # not above its budget
    assert bm.seq_len(1) == 18 and bm.num_free_blocks == 11
    assert bm.can_evict(1)
    bm.evict(1, 6)
    assert bm.seq_len(1) == 6 and bm.num_free_blocks == 14
    np.testing.assert_array_equal(bm.block_table(1), table[:2])
    assert bm.append(1, 7) == int(table[1]) * 4 + 2
    assert bm.append(1, 7) == int(table[1]) * 4 + 3
    slot = bm.append(1, 7)  # a new block, from the pool's front
    assert slot % 4 == 0 and bm.seq_len(1) == 9 and len(bm.block_table(1)) == 3


def test_evicted_blocks_are_not_reused_as_prefixes(bm):
    bm.allocate(1, np.arange(16))
    bm.evict(1, 8)
    assert bm.allocate(2, np.arange(16)) == 0
    for t in range(8):  # full blocks of a trimmed sequence are not registered either
        bm.append(1, t)
    bm.deallocate(2)
    assert bm.allocate(3, np.concatenate([np.arange(8), np.arange(8)])) == 8  # sequence 2's blocks
    bm.deallocate(1)
    bm.deallocate(3)
    assert bm.num_free_blocks == 16


def test_evict_keeps_another_owner_of_the_same_hash(bm):
    """Dropping a trimmed block's hash leaves another block with the same content registered."""
    bm.allocate(1, np.arange(8))
    bm.evict(1, 4)
    assert bm.allocate(2, np.arange(8)) == 0
    bm.evict(1, 2)
    assert bm.allocate(3, np.arange(8)) == 8
    assert not bm.can_evict(2) and not bm.can_evict(3)


def test_evict_refuses_shared_and_unknown(bm):
    from paged_kv_cache_85_gb300 import PkvError

    bm.allocate(1, np.arange(12))
    bm.allocate(2, np.arange(12))
    assert not bm.can_evict(1) and not bm.can_evict(9)
    with pytest.raises(PkvError, match="shares"):
        bm.evict(1, 4)
    assert bm.seq_len(1) == 12 and bm.num_free_blocks == 13
    bm.deallocate(2)
    assert bm.can_evict(1)
    for seq, budget in ((9, 4), (1, 0)):
        with pytest.raises(PkvError):
            bm.evict(seq, budget)
