"""Refusals and workspace sizes of the calls on E4M3 caches with block scales and of
the copies of blocks, through the C ABI without a GPU; the allocator's side of it."""

import ctypes

import numpy as np
import pytest

P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
X, Y, Z, W = (P(n << 20) for n in (1, 2, 3, 4))  # 16-byte aligned addresses that no refused call reads
BENT = P((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib(cuda_lib_path):
    lib = ctypes.CDLL(cuda_lib_path)
    lib.pkv_last_error.restype = ctypes.c_char_p
    lib.pkv_prefill_scaled_workspace_bytes.restype = sz
    lib.pkv_prefill_scaled_workspace_bytes.argtypes = [i32, i64] + [i32] * 6
    return lib


def store(lib, k=X, v=X, kc=X, vc=Y, ks=Z, vs=W, slots=X, N=4, Hkv=2, D=64, NB=8, bs=16):
    return lib.pkv_store_kvcache_scaled(k, v, kc, vc, ks, vs, slots, i64(N), Hkv, D, i64(NB), bs, None, None)


def decode(lib, q=X, kc=X, ks=X, vs=X, tables=X, MBS=4, lens=X, B=2, Hq=4, Hkv=2, D=64, NB=8, bs=16, scale=0.1, out=X, ws=X,
           ws_bytes=1 << 30, max_ctas=0):
    return lib.pkv_paged_attn_decode_scaled(q, kc, X, ks, vs, tables, MBS, lens, B, Hq, Hkv, D, i64(NB), bs, f32(scale), out,
                                            ws, sz(ws_bytes), max_ctas, None, None)


def prefill(lib, q=X, kc=X, ks=X, vs=X, tables=X, MBS=4, B=2, Tq=10, max_q=5, Hq=4, Hkv=2, D=64, NB=8, bs=16, scale=0.1, out=X,
            ws=X, ws_bytes=1 << 30):
    return lib.pkv_paged_prefill_scaled(q, kc, X, ks, vs, tables, MBS, X, X, B, i64(Tq), max_q, Hq, Hkv, D, i64(NB), bs,
                                        f32(scale), out, ws, sz(ws_bytes), None, None)


def copy(lib, tensors=(X, Y), sizes=(64, 4), m=None, pairs=X, n=2, NB=8):
    t = None if tensors is None else (P * len(tensors))(*tensors)
    s = None if sizes is None else (i64 * len(sizes))(*sizes)
    return lib.pkv_copy_blocks(t, s, len(tensors or ()) if m is None else m, pairs, n, i64(NB), None, None)


def refused(lib, status, got, text):
    assert got == status, lib.pkv_last_error()
    assert text in lib.pkv_last_error()


@pytest.mark.parametrize("kw,status,text", [
    (dict(N=-1), INVALID, b"sizes"), (dict(N=1 << 31), UNSUPPORTED, b"N must"), (dict(Hkv=0), INVALID, b"sizes"),
    (dict(Hkv=65536), UNSUPPORTED, b"Hkv"), (dict(D=96), UNSUPPORTED, b"head_dim"), (dict(bs=24), UNSUPPORTED, b"block_size"),
    (dict(bs=0), INVALID, b"sizes"), (dict(NB=0), INVALID, b"sizes"), (dict(NB=1 << 27), INVALID, b"2^31"),
    (dict(NB=1 << 62), INVALID, b"2^31"), (dict(k=None), INVALID, b"null"), (dict(ks=None), INVALID, b"null"),
    (dict(vs=None), INVALID, b"null"), (dict(slots=None), INVALID, b"null"), (dict(vc=X), INVALID, b"share"),
    (dict(vs=Z), INVALID, b"share"), (dict(k=BENT), INVALID, b"aligned"), (dict(ks=BENT), INVALID, b"aligned"),
    (dict(slots=P((1 << 20) + 4)), INVALID, b"aligned")])
def test_store_refuses(lib, kw, status, text):
    refused(lib, status, store(lib, **kw), b"store_kvcache_scaled")
    assert text in lib.pkv_last_error()


def test_empty_calls_do_nothing(lib):
    assert store(lib, N=0, k=None) == OK
    assert decode(lib, B=0) == OK
    for kw in (dict(B=0), dict(Tq=0), dict(max_q=0)):
        assert prefill(lib, **kw) == OK
    assert copy(lib, n=0) == OK and copy(lib, m=0) == OK


@pytest.mark.parametrize("kw,status,text", [
    (dict(ks=None), INVALID, b"scales"), (dict(vs=BENT), INVALID, b"scales"), (dict(q=None), INVALID, b"null"),
    (dict(Hq=3), INVALID, b"multiple"), (dict(Hq=6), UNSUPPORTED, b"Hq/Hkv"), (dict(D=96), UNSUPPORTED, b"head_dim"),
    (dict(bs=24), UNSUPPORTED, b"block_size"), (dict(scale=float("nan")), INVALID, b"scale"), (dict(B=-1), INVALID, b"sizes"),
    (dict(NB=1 << 27), INVALID, b"2^31"), (dict(max_ctas=-1), INVALID, b"max_ctas")])
def test_decode_refuses(lib, kw, status, text):
    got = decode(lib, **kw)
    if got == 4:  # without a GPU the plan ends before the pointers are looked at
        pytest.skip("needs a device")
    refused(lib, status, got, text)


@pytest.mark.parametrize("kw,status,text", [
    (dict(ks=None), INVALID, b"scales"), (dict(vs=BENT), INVALID, b"scales"), (dict(q=None), INVALID, b"null"),
    (dict(Hq=3), INVALID, b"multiple"), (dict(Hq=6), UNSUPPORTED, b"Hq/Hkv"), (dict(D=96), UNSUPPORTED, b"head_dim"),
    (dict(bs=24), UNSUPPORTED, b"block_size"), (dict(scale=float("inf")), INVALID, b"scale"), (dict(max_q=-1), INVALID, b"sizes"),
    (dict(MBS=4096, ws=None), WORKSPACE, b"workspace"), (dict(MBS=4096, ws_bytes=100), WORKSPACE, b"workspace"),
    (dict(MBS=4096, ws=BENT), WORKSPACE, b"workspace"), (dict(Hq=1 << 20, Hkv=1 << 20, B=2048), UNSUPPORTED, b"2^31")])
def test_prefill_refuses(lib, kw, status, text):
    refused(lib, status, prefill(lib, **kw), text)


def test_prefill_workspace(lib):
    f, up = lib.pkv_prefill_scaled_workspace_bytes, lambda n: n + -n % 256
    assert f(3, 100, 40, 4, 2, 64, 4, 16) == 0  # contexts too short to split
    assert f(3, 100, 40, 4, 2, 64, 512, 16) == up(16 * 400 * 4) + 16 * 400 * 64 * 4  # 64 tiles in splits of 4
    assert f(76, 1 << 20, 20, 4, 2, 64, 512, 16) == 0  # 152 items
    for args in ((0, 1, 1, 4, 2, 64, 4, 16), (1, 0, 1, 4, 2, 64, 4, 16), (1, 1, 1, 5, 2, 64, 4, 16), (1, 1, -1, 4, 2, 64, 4, 16)):
        assert f(*args) == 0


@pytest.mark.parametrize("kw,text", [
    (dict(m=-1), b"sizes"), (dict(n=-1), b"sizes"), (dict(NB=0), b"sizes"), (dict(NB=1 << 31), b"sizes"),
    (dict(tensors=None, m=2), b"null"), (dict(sizes=None), b"null"), (dict(pairs=None), b"null"),
    (dict(pairs=P((1 << 20) + 4)), b"aligned"), (dict(tensors=(X, None)), b"null"), (dict(tensors=(X, X)), b"same memory"),
    (dict(sizes=(64, 0)), b"bytes per block"), (dict(sizes=(1 << 31, 4)), b"bytes per block"),
    (dict(sizes=(64, -4)), b"bytes per block")])
def test_copy_refuses(lib, kw, text):
    refused(lib, INVALID, copy(lib, **kw), text)


# ---------------------------------------------------------------- the allocator


@pytest.fixture(scope="module")
def Manager(cuda_lib_path):
    from paged_kv_cache_85_gb300.block_manager import BlockManager

    return BlockManager


class Pool:
    """What the blocks hold, token ids in place of K/V rows."""

    def __init__(self, bm):
        self.bm, self.rows, self.tokens = bm, np.full((bm.num_blocks, bm.block_size), -1), {}

    def allocate(self, s, tokens):
        self.bm.allocate(s, tokens)
        self.tokens[s] = list(tokens)
        self.rows.reshape(-1)[self.bm.slots(s, 0, len(tokens))] = tokens

    def append(self, s, token):
        self.rows.reshape(-1)[self.bm.append(s, token)] = token
        self.tokens[s].append(token)

    def copy(self, pairs):
        assert pairs.dtype == np.int32 and pairs.shape[1] == 2
        assert len(np.unique(pairs[:, 1])) == len(pairs) and not np.intersect1d(pairs[:, 0], pairs[:, 1]).size
        for a, b in pairs:
            self.rows[b] = self.rows[a]

    def fork(self, a, b):
        pairs = self.bm.fork(a, b)
        self.tokens[b] = list(self.tokens[a])
        self.copy(pairs)
        return pairs

    def drop(self, s):
        self.bm.deallocate(s)
        del self.tokens[s]

    def check(self):
        refs = np.zeros(self.bm.num_blocks, int)
        for s, t in self.tokens.items():
            table = self.bm.block_table(s)
            np.add.at(refs, table, 1)
            assert self.bm.seq_len(s) == len(t)
            assert self.rows[table].reshape(-1)[: len(t)].tolist() == t
        assert [self.bm.ref_count(i) for i in range(self.bm.num_blocks)] == refs.tolist()
        assert self.bm.num_free_blocks == int((refs == 0).sum())
        return refs


def test_fork(Manager):
    p = Pool(Manager(20, 4))
    p.allocate(1, range(10))
    pairs = p.fork(1, 2)
    assert pairs.tolist() == [[p.bm.block_table(1)[2], p.bm.block_table(2)[2]]]
    assert p.bm.block_table(1)[:2].tolist() == p.bm.block_table(2)[:2].tolist()
    p.check()
    for i in range(6):
        p.append(1, 100 + i)
        p.append(2, 200 + i)
        p.check()
    assert p.bm.seq_len(1) == 16
    assert p.fork(1, 3).shape == (0, 2)  # nothing but full blocks
    p.append(3, 7)
    p.append(1, 8)
    p.check()
    # the blocks that the child filled are offered for prefixes
    assert p.bm.allocate(9, list(range(10)) + [200, 201, 202, 203, 204, 205, 1]) == 16
    p.bm.deallocate(9)
    for s in (1, 2, 3):
        p.drop(s)
    assert (p.check() == 0).all()


def test_fork_refuses(Manager):
    from paged_kv_cache_85_gb300 import PkvError

    p = Pool(Manager(3, 4))
    p.allocate(1, range(9))
    for a, b, status in ((7, 8, INVALID), (1, 1, INVALID), (1, 2, WORKSPACE)):
        with pytest.raises(PkvError) as e:
            p.bm.fork(a, b)
        assert e.value.status == status
        p.check()
    p.bm.deallocate(1)


def test_evicted_sequences_fork(Manager):
    bm = Manager(20, 4)
    bm.allocate(1, range(18))
    bm.evict(1, 10)
    assert len(bm.fork(1, 2)) == 1
    assert not bm.can_evict(1) and bm.seq_len(2) == 10
    for i in range(2):  # fills the block: never offered as a prefix
        bm.append(2, i)
    assert bm.allocate(3, list(range(10)) + [0, 1, 5]) == 0


def test_compact(Manager):
    rng = np.random.default_rng(0)
    p = Pool(Manager(64, 4))
    prompt = list(range(1000, 1011))
    for s in range(12):
        p.allocate(s, prompt[: int(rng.integers(1, 12))] + rng.integers(0, 5, int(rng.integers(1, 9))).tolist())
    for s in (0, 3, 4, 8, 9):
        p.drop(s)
    p.fork(5, 20)
    used = int((p.check() > 0).sum())
    pairs = p.bm.compact()
    assert len(pairs) > 0 and (pairs[:, 0] >= used).all() and (pairs[:, 1] < used).all()
    p.copy(pairs)
    refs = p.check()
    assert (refs[:used] > 0).all() and (refs[used:] == 0).all()
    assert len(p.bm.compact()) == 0
    # prefixes are found where they are now, and only there
    q = next(s for s in p.tokens if len(p.tokens[s]) >= 8 and p.tokens[s][:8] == prompt[:8])
    assert p.bm.allocate(50, p.tokens[q][:8] + [77]) == 8
    assert p.bm.block_table(50)[:2].tolist() == p.bm.block_table(q)[:2].tolist()
    p.bm.deallocate(50)
    for _ in range(30):  # a pool in use: everything at once
        s = int(rng.integers(0, 40))
        if s in p.tokens:
            if rng.random() < 0.5:
                p.drop(s)
            elif p.bm.can_append(s):
                p.append(s, int(rng.integers(0, 5)))
        elif p.tokens and rng.random() < 0.5 and p.bm.num_free_blocks:
            p.fork(int(rng.choice(list(p.tokens))), s)
        elif p.bm.can_allocate(12):
            p.allocate(s, rng.integers(0, 2, int(rng.integers(1, 13))).tolist())
        p.check()
        if rng.random() < 0.3:
            p.copy(p.bm.compact())
            used = int((p.check() > 0).sum())
            assert all(p.bm.ref_count(i) > 0 for i in range(used))


def test_compact_with_a_short_list(Manager):
    p = Pool(Manager(10, 4))
    for s in range(4):
        p.allocate(s, range(10 * s, 10 * s + 5))
    p.drop(0)
    p.drop(1)
    lib, n = p.bm._lib, i64()
    short = np.empty((3, 2), np.int32)
    assert lib.pkv_bm_compact(p.bm._h, short.ctypes.data_as(P), 3, ctypes.byref(n)) == WORKSPACE and n.value == 4
    p.check()
    assert len(p.bm.compact()) == 4
    assert lib.pkv_bm_compact(None, None, 0, ctypes.byref(n)) == INVALID
    assert lib.pkv_bm_compact(p.bm._h, None, 1, ctypes.byref(n)) == INVALID
    assert lib.pkv_bm_fork(None, 1, 2, None) == INVALID
