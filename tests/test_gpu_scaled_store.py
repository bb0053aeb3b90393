"""The quantising store into E4M3 caches with a scale per block and KV head: bit for bit the 64-bit form."""

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


def dev(x):
    x = np.ascontiguousarray(x)
    return torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).cuda() if x.dtype == np.uint16 else torch.from_numpy(x).cuda()


class Pool:
    """Both caches on both sides; rows start as junk, NaN codes among them, scales as what `scales` gives."""

    def __init__(self, NB, bs, Hkv, D, seed=0, scales=None):
        rng = np.random.default_rng(seed)
        self.shape = (NB, bs, Hkv, D)
        self.c = [rng.integers(0, 256, self.shape).astype(np.uint8) for _ in range(2)]
        self.s = [(2.0 ** rng.integers(-8, 3, (NB, Hkv)) if scales is None else scales(rng, (NB, Hkv))).astype(np.float32)
                  for _ in range(2)]
        self.dc, self.ds = [dev(c) for c in self.c], [dev(s) for s in self.s]
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(self, pkv, k, v, slots, bad=0):
        slots = np.asarray(slots, dtype=np.int64)
        pkv.store_kvcache_scaled(dev(k), dev(v), *self.dc, *self.ds, dev(slots), err_flag=self.err)
        for x, c, s in zip((k, v), self.c, self.s):
            assert ref.store(x, c, s, slots) == bad
        self.check()

    def check(self):
        for name, got, want in zip(("k", "v"), self.ds, self.s):
            got = got.cpu().numpy()
            np.testing.assert_array_equal(got.view(np.uint32), want.view(np.uint32), err_msg=name + " scales")
        for name, got, want in zip(("k", "v"), self.dc, self.c):
            got = got.cpu().numpy()
            nan = (want & 0x7F) == 0x7F  # a NaN's sign carries nothing
            np.testing.assert_array_equal(got[~nan], want[~nan], err_msg=name)
            assert ((got[nan] & 0x7F) == 0x7F).all()


def draw(rng, N, Hkv, D, spread=2.0):
    x = rng.standard_normal((N, Hkv, D)) * 2.0 ** (spread * rng.standard_normal((N, Hkv, 1)))
    return ref.bf16(x)


def sequence_slots(rng, NB, bs, spans):
    """Slots of spans (first position, tokens), each a sequence of its own blocks."""
    perm = rng.permutation(NB)
    at, out = 0, []
    for first, n in spans:
        blocks = perm[at: at + (first + n + bs - 1) // bs]
        at += len(blocks)
        t = np.arange(first, first + n)
        out.append(blocks[t // bs] * bs + t % bs)
    return np.concatenate(out) if out else np.zeros(0, np.int64)


@pytest.mark.parametrize("Hkv,D,bs", [(1, 64, 16), (2, 128, 16), (3, 64, 48), (8, 128, 256), (4, 128, 32)])
def test_prompts_then_steps(pkv, Hkv, D, bs):
    """Prompts of all lengths, then token by token: scales grow, old rows are recoded, new blocks begin."""
    rng = np.random.default_rng(bs + Hkv)
    lens = [1, 2, 15, 16, 17, 40, 3 * bs, bs - 1, 0, 1]
    NB = sum((n + 40 + bs - 1) // bs for n in lens) + 3
    p = Pool(NB, bs, Hkv, D)
    perm = rng.permutation(NB)
    tables, at = [], 0
    for n in lens:
        m = (n + 40 + bs - 1) // bs
        tables.append(perm[at: at + m])
        at += m
    slot = lambda b, t: tables[b][t // bs] * bs + t % bs
    slots = [slot(b, t) for b, n in enumerate(lens) for t in range(n)]
    p.step(pkv, draw(rng, len(slots), Hkv, D), draw(rng, len(slots), Hkv, D), slots)
    for i in range(20):
        slots = [slot(b, n + i) for b, n in enumerate(lens)] + [-1] * (i % 3)
        p.step(pkv, draw(rng, len(slots), Hkv, D), draw(rng, len(slots), Hkv, D), slots)
    assert int(p.err.item()) == 0


@pytest.mark.parametrize("N,bs,Hkv,D", [(2048, 16, 2, 128), (5000, 256, 1, 64), (2100, 512, 1, 128), (3001, 48, 1, 128),
                                        (4096, 1024, 1, 64), (2500, 128, 2, 64)])
def test_many_tokens(pkv, N, bs, Hkv, D):
    """Runs that cross the kernel's windows, that begin anywhere in them, and that are longer than what it keeps."""
    rng = np.random.default_rng(N)
    spans, left = [], N
    while left:
        n = min(left, int(rng.integers(1, 3 * bs + 200)))
        spans.append((int(rng.integers(0, 2 * bs)), n))
        left -= n
    NB = sum((f + n + bs - 1) // bs for f, n in spans) + 1
    slots = sequence_slots(rng, NB, bs, spans)
    p = Pool(NB, bs, Hkv, D)
    p.step(pkv, draw(rng, N, Hkv, D), draw(rng, N, Hkv, D), slots)
    assert int(p.err.item()) == 0


def test_a_long_chunk_in_short_calls(pkv):
    """Fewer tokens than the large windows take, in blocks larger than the small ones."""
    rng = np.random.default_rng(5)
    p = Pool(12, 256, 2, 128)
    for first, n in ((0, 300), (300, 17), (317, 600), (917, 1), (918, 500)):
        t = np.arange(first, first + n)
        slots = np.array([7, 2, 9, 0, 11, 4])[t // 256] * 256 + t % 256
        p.step(pkv, draw(rng, n, 2, 128), draw(rng, n, 2, 128), slots)


def test_padding_and_bad_slots(pkv):
    rng = np.random.default_rng(1)
    p = Pool(4, 16, 2, 64)
    p.step(pkv, draw(rng, 5, 2, 64), draw(rng, 5, 2, 64), [-1] * 5)
    assert int(p.err.item()) == 0
    p.step(pkv, draw(rng, 0, 2, 64), draw(rng, 0, 2, 64), [])
    p.step(pkv, draw(rng, 7, 2, 64), draw(rng, 7, 2, 64), [-1, 33, -1, 1, 2, -1, 63])
    assert int(p.err.item()) == 0
    p.step(pkv, draw(rng, 6, 2, 64), draw(rng, 6, 2, 64), [64, 5, -2, 18, 1 << 40, -(1 << 40)], bad=4)
    assert int(p.err.item()) == pkv.FLAG_BAD_SLOT
    # many tokens, padding between sequences and windows of nothing but padding
    p = Pool(300, 16, 1, 64)
    slots = np.full(4000, -1, np.int64)
    for i in range(0, 4000, 500):
        slots[i + 3: i + 83] = np.arange(80) + 16 * (i // 100)
    p.step(pkv, draw(rng, 4000, 1, 64), draw(rng, 4000, 1, 64), slots)


@pytest.mark.parametrize("N", [40, 2400])
def test_values_of_all_sizes(pkv, N):
    """Zeros, subnormals, the largest numbers, infinities and NaN; magnitudes at the scales' borders."""
    rng = np.random.default_rng(N)
    special = ref.bf16([0, -0.0, 1e-40, 448, 449, 450, 452, 224, 3.4e38, -3.4e38, 448 * 2.0 ** 40, 2.0 ** -32, 1e-15, 464, 480,
                        2.0 ** -9, 2.0 ** -10, 1.75, 1.7578125])
    inf = np.array([0x7F80, 0xFF80, 0x7FC0, 0xFFC1, 0x7F81], np.uint16)
    NB = N // 8 + 40
    p = Pool(NB, 16, 2, 64)
    for round_ in range(3):
        k, v = draw(rng, N, 2, 64, 8.0), draw(rng, N, 2, 64, 0.5)
        k[rng.random(k.shape) < 0.02] = 0
        for x in (k, v):
            at = rng.random(x.shape) < 0.003
            x[at] = rng.choice(np.concatenate([special, inf]), at.sum())
        k[0], v[1] = 0, inf[0]  # rows of nothing but zeros, and without a finite value
        v[2], k[3] = 0x7FC0, special[8]
        k[4:9, :, :] = special[3:8, None, None]
        first = [0, 5, 16][round_]
        slots = sequence_slots(rng, NB, 16, [(first + i, 1) for i in range(9)] + [(first, N - 9)])
        p.step(pkv, k, v, slots)


def test_scales_that_stand_there(pkv):
    """Scales that are no powers of two grow and recode; those that are no positive number begin anew."""
    def odd(rng, shape):
        s = rng.uniform(1e-4, 0.1, shape)
        s.flat[::5] = rng.choice([0.0, -1.0, np.nan, np.inf, -0.0, -np.inf], s.flat[::5].shape)
        return s
    rng = np.random.default_rng(3)
    p = Pool(40, 32, 3, 128, scales=odd)
    for i in range(3):
        slots = rng.permutation(40)[:30] * 32 + rng.integers(0, 32, 30)
        p.step(pkv, draw(rng, 30, 3, 128), draw(rng, 30, 3, 128), slots)


def test_tokens_of_a_block_in_any_order(pkv):
    rng = np.random.default_rng(9)
    p = Pool(6, 64, 1, 64)
    slots = np.concatenate([b * 64 + rng.permutation(64)[: n] for b, n in ((3, 64), (0, 10), (5, 33), (1, 1))])
    p.step(pkv, draw(rng, len(slots), 1, 64), draw(rng, len(slots), 1, 64), slots)


def test_one_slot_for_many_tokens(pkv):
    """A dummy slot that takes every padded token (all alike, so that the row is defined)."""
    rng = np.random.default_rng(2)
    for N in (100, 3000):
        p = Pool(200, 16, 2, 64)
        k, v = draw(rng, N, 2, 64), draw(rng, N, 2, 64)
        k[30:], v[30:] = k[30], v[30]
        p.step(pkv, k, v, np.concatenate([np.arange(30) + 32, np.full(N - 30, 5 * 16 + 7)]))


def test_captured_and_on_another_stream(pkv):
    rng = np.random.default_rng(4)
    p = Pool(8, 16, 2, 64)
    k, v, slots = dev(draw(rng, 12, 2, 64)), dev(draw(rng, 12, 2, 64)), torch.full((12,), -1, dtype=torch.int64, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pkv.store_kvcache_scaled(k, v, *p.dc, *p.ds, slots)
    for i in range(4):
        kh, vh = draw(rng, 12, 2, 64), draw(rng, 12, 2, 64)
        sh = np.concatenate([np.arange(5) + 16 * i + i, [-1], np.arange(5) + 70 + 5 * i, [-1]])
        with torch.cuda.stream(s):
            k.copy_(dev(kh))
            v.copy_(dev(vh))
            slots.copy_(dev(sh))
            g.replay()
        s.synchronize()
        for x, c, sc in zip((kh, vh), p.c, p.s):
            ref.store(x, c, sc, sh)
        p.check()
