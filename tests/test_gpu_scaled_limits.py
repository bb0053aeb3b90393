"""The calls on scaled caches at the ends of their ranges: many sequences, large caches, odd addresses, zero scales."""

import numpy as np
import pytest

import scaled_reference as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv(cuda_lib_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_85_gb300 as m

    m.load_library()
    return m


def dev(x, offset=0):
    """On the GPU; offset: elements by which it lies behind an aligned address."""
    x = np.ascontiguousarray(x)
    t = torch.from_numpy(x.view(np.int16)).view(torch.bfloat16) if x.dtype == np.uint16 else torch.from_numpy(x)
    if not offset:
        return t.cuda()
    big = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
    big[offset:] = t.cuda().reshape(-1)
    return big[offset:].view(t.shape)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def ends(n):
    return dev(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))


@pytest.mark.parametrize("B", [33, 152, 153, 256, 257, 700])
def test_prefill_of_many_sequences(pkv, B):
    """The ranked schedule's chunks, and beyond them; the sequences that the join can look through."""
    rng = np.random.default_rng(B)
    q_lens = rng.integers(0, 9, B)
    q_lens[B // 2] = 70
    c = ref.Cache(q_lens + rng.integers(0, 60, B), 16, 1, 64, seed=B)
    q = ref.bf16(rng.standard_normal((int(q_lens.sum()), 2, 64)))
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.paged_prefill_scaled(dev(q), dev(c.k), dev(c.v), dev(c.ks), dev(c.vs), dev(c.tables), ends(q_lens), ends(c.lens), 70, 0.1,
                             out, err_flag=err)
    assert int(err.item()) == 0
    want, mag = ref.prefill(q, c, q_lens, 0.1)
    ref.check(host(out), want, mag)


def test_caches_beyond_4_gb(pkv):
    """Blocks whose bytes lie past 32 bits: stored, read by decode and prefill, copied."""
    rng = np.random.default_rng(0)
    bs, Hkv, D = 32, 8, 128
    NB = (5 << 30) // (bs * Hkv * D)
    lens = np.array([100, 33], np.int32)
    c = ref.Cache(lens, bs, Hkv, D, seed=1)
    first = NB - c.NB  # the small pool is the end of the large one
    big = [torch.empty((NB, bs, Hkv, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((NB, Hkv), float("nan"), device="cuda") for _ in range(2)]
    for t, x in zip(big + scales, (c.k, c.v, c.ks, c.vs)):
        t[first:] = dev(x)
    tables = np.where(c.tables >= 0, c.tables + first, -1).astype(np.int32)
    # the last tokens of both contexts anew, seven and one
    at = np.concatenate([c.slots(0)[-7:], c.slots(1)[-1:]])
    k, v = (ref.bf16(4 * rng.standard_normal((8, Hkv, D))) for _ in range(2))
    pkv.store_kvcache_scaled(dev(k), dev(v), *big, *scales, dev(at + first * bs))
    for x, cc, s in ((k, c.k, c.ks), (v, c.v, c.vs)):
        ref.store(x, cc, s, at)
    for t, x in zip(big, (c.k, c.v)):
        got = t[first:].cpu().numpy()
        nan = (x & 0x7F) == 0x7F
        np.testing.assert_array_equal(got[~nan], x[~nan])
    q = ref.bf16(0.3 * rng.standard_normal((2, 16, D)))
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    want, mag = ref.decode(q, c, 0.08)
    pkv.paged_attn_decode_scaled(dev(q), *big, *scales, dev(tables), dev(lens), 0.08, out)
    ref.check(host(out), want, mag)
    out.zero_()
    pkv.paged_prefill_scaled(dev(q), *big, *scales, dev(tables), ends([1, 1]), ends(lens), 1, 0.08, out)
    ref.check(host(out), want, mag)
    # to the front and decoded there
    used = tables[tables >= 0]
    pairs = np.stack([used, np.arange(len(used))], 1).astype(np.int32)
    pkv.copy_blocks(big + scales, dev(pairs))
    front = np.full_like(tables, -1)
    front[tables >= 0] = pairs[:, 1]
    out.zero_()
    pkv.paged_attn_decode_scaled(dev(q), *big, *scales, dev(front), dev(lens), 0.08, out)
    ref.check(host(out), want, mag)


@pytest.mark.parametrize("D", [64, 128])
def test_addresses_that_16_bytes_divide_and_32_do_not(pkv, D):
    rng = np.random.default_rng(D)
    Hkv, bs = 2, 16
    c = ref.Cache([300, 5000, 17], bs, Hkv, D, seed=2)
    new = [(0, 40), (1, 600), (2, 1)]
    at = np.concatenate([c.slots(b)[-n:] for b, n in new])
    k, v = (ref.bf16(0.3 * rng.standard_normal((len(at), Hkv, D))) for _ in range(2))
    t = [dev(c.k, 16), dev(c.v, 48), dev(c.ks, 4), dev(c.vs, 12)]
    for x in t:
        assert x.data_ptr() % 16 == 0 and x.data_ptr() % 32 == 16
    pkv.store_kvcache_scaled(dev(k, 8), dev(v, 24), *t, dev(at, 1))
    for x, cc, s in ((k, c.k, c.ks), (v, c.v, c.vs)):
        ref.store(x, cc, s, at)
    for x, want in zip(t[:2], (c.k, c.v)):
        nan = (want & 0x7F) == 0x7F
        np.testing.assert_array_equal(x.cpu().numpy()[~nan], want[~nan])
    for q_lens in ([40, 600, 1], [1, 1, 1]):  # whole items, and items split over the keys
        q = ref.bf16(rng.standard_normal((sum(q_lens), 4, D)))
        out = dev(np.zeros(q.shape, np.uint16), 8)
        want, mag = ref.prefill(q, c, q_lens, 0.1)
        need = pkv.prefill_scaled_workspace_bytes(3, sum(q_lens), max(q_lens), 4, 2, D, c.MBS, bs)
        ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")[16:] if need else None
        pkv.paged_prefill_scaled(dev(q, 8), *t, dev(c.tables, 1), ends(q_lens), ends(c.lens), max(q_lens), 0.1, out, workspace=ws)
        ref.check(host(out), want, mag)
    q = ref.bf16(rng.standard_normal((3, 4, D)))
    out = dev(np.zeros(q.shape, np.uint16), 8)
    pkv.paged_attn_decode_scaled(dev(q, 8), *t, dev(c.tables, 1), dev(c.lens, 3), 0.1, out)
    want, mag = ref.decode(q, c, 0.1)
    ref.check(host(out), want, mag)


def test_scales_of_zero(pkv):
    """Blocks whose values are all zero, beside others, in K and in V; all of them in one context."""
    rng = np.random.default_rng(3)
    c = ref.Cache([200, 70], 16, 1, 64, seed=5)
    c.ks[c.tables[0, [0, 3, 12]]] = 0
    c.vs[c.tables[0, [0, 5, 11]]] = 0
    c.ks[c.tables[1, :5]] = 0
    c.vs[c.tables[1, :5]] = 0
    t = [dev(x) for x in (c.k, c.v, c.ks, c.vs, c.tables)]
    q = ref.bf16(rng.standard_normal((2, 4, 64)))
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    pkv.paged_attn_decode_scaled(dev(q), *t, dev(c.lens), 0.1, out)
    want, mag = ref.decode(q, c, 0.1)
    ref.check(host(out), want, mag)
    q_lens = [150, 70]
    q = ref.bf16(rng.standard_normal((220, 4, 64)))
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    pkv.paged_prefill_scaled(dev(q), *t, ends(q_lens), ends(c.lens), 150, 0.1, out)
    want, mag = ref.prefill(q, c, q_lens, 0.1)
    ref.check(host(out), want, mag)


@pytest.mark.parametrize("N", [511, 512, 513, 640])
def test_store_where_its_windows_change(pkv, N):
    rng = np.random.default_rng(N)
    NB, bs, Hkv, D = 60, 32, 2, 128
    c = [rng.integers(0, 256, (NB, bs, Hkv, D)).astype(np.uint8) for _ in range(2)]
    s = [np.full((NB, Hkv), 2.0 ** -6, np.float32) for _ in range(2)]
    t = [dev(x) for x in (*c, *s)]
    slots = np.concatenate([rng.permutation(NB)[:18][:, None] * bs + np.arange(5, 32)[None]], 0).reshape(-1)
    slots = np.concatenate([slots, np.full(N, -1)])[:N]
    k, v = (ref.bf16(rng.standard_normal((N, Hkv, D)) * 2.0 ** (3 * rng.standard_normal((N, 1, 1)))) for _ in range(2))
    pkv.store_kvcache_scaled(dev(k), dev(v), *t, dev(slots))
    for x, cc, ss in zip((k, v), c, s):
        ref.store(x, cc, ss, slots)
    for got, want in zip(t[2:], s):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    for got, want in zip(t[:2], c):
        nan = (want & 0x7F) == 0x7F
        np.testing.assert_array_equal(got.cpu().numpy()[~nan], want[~nan])


@pytest.mark.parametrize("N,Hkv,D,bs,runs", [
    (5120, 8, 128, 16, "long"), (5121, 8, 128, 16, "long"), (5121, 8, 64, 256, "long"), (5300, 8, 128, 1024, "long"),
    (2561, 16, 64, 48, "long"), (41000, 1, 128, 2048, "long"), (5633, 8, 128, 16, "one"), (5121, 8, 128, 32, "short"),
])
def test_store_of_many_tokens(pkv, N, Hkv, D, bs, runs):
    """Both sides of 40960 rows of a head, where windows become larger: blocks that go on over several windows, that
    start in each place of one, that are full, begun or continued; a block for every token; padding between."""
    rng = np.random.default_rng(N + bs)
    slots, blk = [], 0
    while len(slots) < N:
        first = int(rng.integers(0, bs)) if runs != "one" and rng.random() < 0.5 else 0
        n = {"long": bs - first, "short": int(rng.integers(1, bs - first + 1)), "one": 1}[runs]
        slots += list(range(blk * bs + first, blk * bs + first + n))
        blk += 1
        if rng.random() < 0.1:
            slots += [-1] * int(rng.integers(1, 40))
    slots = np.asarray(slots[:N])
    order = rng.permutation(blk)
    slots = np.where(slots >= 0, order[slots // bs] * bs + slots % bs, -1)
    c = [rng.integers(0, 0x7F, (blk, bs, Hkv, D)).astype(np.uint8) for _ in range(2)]
    s = [np.full((blk, Hkv), 2.0 ** -6, np.float32) for _ in range(2)]
    t = [dev(x) for x in (*c, *s)]
    k, v = (ref.bf16(rng.standard_normal((N, Hkv, D)) * 2.0 ** (3 * rng.standard_normal((N, Hkv, 1)))) for _ in range(2))
    pkv.store_kvcache_scaled(dev(k), dev(v), *t, dev(slots))
    for x, cc, ss in zip((k, v), c, s):
        ref.store(x, cc, ss, slots)
    for got, want in zip(t, c + s):
        np.testing.assert_array_equal(got.cpu().numpy(), want)


def test_queries_of_all_sizes(pkv):
    """Elements far below their row's largest, rows of zeros, of tiny and of huge numbers."""
    rng = np.random.default_rng(7)
    c = ref.Cache([130, 300], 32, 1, 128, seed=3)
    t = [dev(x) for x in (c.k, c.v, c.ks, c.vs, c.tables)]
    x = rng.standard_normal((20, 2, 128)) * 2.0 ** -rng.integers(0, 25, (20, 2, 128))
    x[0] = 0
    x[1] *= 1e-30
    x[2] = 1e-39
    x[3, 0] = 0
    x[3, 0, 5] = 3.0
    for i, e in enumerate((1e30, 1e-20, 100.0)):
        x[4 + i] *= e
    q = ref.bf16(x)
    for rows, size in ((slice(0, 4), 0.1), (slice(4, 5), 1e-31), (slice(5, 6), 1e18), (slice(6, 7), 1e-3), (slice(7, 20), 0.1)):
        n = rows.stop - rows.start
        part = q[rows]
        out = torch.empty(part.shape, dtype=torch.bfloat16, device="cuda")
        pkv.paged_prefill_scaled(dev(part), *t, ends([0, n]), ends(c.lens), n, size, out)
        want, mag = ref.prefill(part, c, [0, n], size)
        ref.check(host(out), want, mag, f"rows {rows}")
