"""Decode and prefill over E4M3 caches with a scale per block and KV head, against the 64-bit form."""

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


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def queries(rng, rows, Hq, D, size=1.0):
    return ref.bf16(size * rng.standard_normal((rows, Hq, D)))


def run_decode(pkv, c, q, scale, flag=0, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    got = pkv.paged_attn_decode_scaled(dev(q), dev(c.k), dev(c.v), dev(c.ks), dev(c.vs), dev(c.tables), dev(c.lens), scale,
                                       out, err_flag=err, **kw)
    assert got is out
    assert int(err.item()) == flag
    return out


def run_prefill(pkv, c, q, q_lens, scale, flag=0, cu_q=None, cu_k=None, max_q=None, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ends = lambda n: np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    got = pkv.paged_prefill_scaled(dev(q), dev(c.k), dev(c.v), dev(c.ks), dev(c.vs), dev(c.tables),
                                   dev(ends(q_lens) if cu_q is None else cu_q), dev(ends(c.lens) if cu_k is None else cu_k),
                                   max(q_lens) if max_q is None else max_q, scale, out, err_flag=err, **kw)
    assert got is out
    assert int(err.item()) == flag
    return out


@pytest.mark.parametrize("Hkv,G,D,bs,spread,pow2", [
    (2, 2, 64, 16, 1.0, True), (1, 1, 64, 48, 0.0, True), (3, 4, 128, 16, 3.0, True), (8, 2, 128, 256, 1.0, True),
    (2, 8, 128, 32, 1.0, True), (4, 8, 64, 64, 6.0, True), (2, 4, 128, 16, 1.0, False), (1, 2, 64, 32, 9.0, False),
    (1, 1, 128, 128, 2.0, True)])
def test_decode(pkv, Hkv, G, D, bs, spread, pow2):
    rng = np.random.default_rng(Hkv * 100 + G)
    lens = [0, 1, 2, 15, 16, 17, 31, 33, 100, 257, 0, 1025, 700]
    c = ref.Cache(lens, bs, Hkv, D, seed=G, spread=spread, pow2=pow2, mbs_extra=1)
    q = queries(rng, len(lens), Hkv * G, D)
    want, mag = ref.decode(q, c, D ** -0.5)
    out = run_decode(pkv, c, q, D ** -0.5)
    ref.check(host(out), want, mag)
    for max_ctas in (1, 7):
        ref.check(host(run_decode(pkv, c, q, D ** -0.5, max_ctas=max_ctas)), want, mag)


@pytest.mark.parametrize("B,G,D,bs", [(1500, 8, 128, 32), (3000, 1, 128, 16), (700, 8, 64, 32), (4000, 2, 64, 64)])
def test_decode_large_batches(pkv, B, G, D, bs):
    """Where the CTAs hold fewer stages: boxes of 32 tokens, eight workers."""
    rng = np.random.default_rng(B)
    c = ref.Cache(rng.integers(0, 90, B), bs, 1, D, seed=1)
    q = queries(rng, B, G, D)
    want, mag = ref.decode(q, c, 0.1)
    ref.check(host(run_decode(pkv, c, q, 0.1)), want, mag)


def test_decode_scales_far_apart(pkv):
    """V scales that rise and fall by more than the weights' range along a context, zeros among them; K's alike with a
    softmax scale that keeps the scores small."""
    rng = np.random.default_rng(0)
    c = ref.Cache([16 * 40, 16 * 33 + 5], 16, 2, 64, seed=3)
    n = (c.tables >= 0).sum(1)
    for b in range(2):
        for h in range(2):
            c.vs[c.tables[b, : n[b]], h] = 2.0 ** rng.integers(-30, 30, n[b])
            c.ks[c.tables[b, : n[b]], h] = 2.0 ** -rng.integers(7, 30, n[b])
    q = queries(rng, 2, 8, 64)
    want, mag = ref.decode(q, c, 0.1)
    ref.check(host(run_decode(pkv, c, q, 0.1)), want, mag)
    # every weight on one block of small scale: nothing of its precision is lost to the others' larger ones
    t = c.tables[0, 20]
    c.vs[c.tables[0, : n[0]], 0] = 2.0
    c.vs[t, 0] = 2.0 ** -25
    c.k[:, :, 0] = 0
    c.k[t, :, 0, 0] = 0x7E  # 448
    c.ks[:, 0] = 1.0
    q[0, :, :] = 0
    q[0, :, 0] = ref.bf16(1.0)
    want, mag = ref.decode(q, c, 1.0)
    ref.check(host(run_decode(pkv, c, q, 1.0)), want, mag)
    # a scale of zero makes its block zero
    c.vs[c.tables[1, 3], 1] = 0
    c.vs[c.tables[1, 0], 1] = 0
    want, mag = ref.decode(q, c, 0.1)
    got = host(run_decode(pkv, c, q, 0.1))
    ref.check(got[1], want[1], mag[1])


def test_decode_bad_blocks_and_lengths(pkv):
    rng = np.random.default_rng(5)
    c = ref.Cache([100, 64, 40, 33], 16, 2, 64, seed=2, mbs_extra=2)
    q = queries(rng, 4, 4, 64)
    skip = {0: np.zeros(128, bool), 1: np.ones(64, bool)}
    skip[0][32:48] = True
    want, mag = ref.decode(q, c, 0.125, skip)
    c.tables[0, 2] = c.NB
    c.tables[1, :] = -5
    ref.check(host(run_decode(pkv, c, q, 0.125, flag=pkv.FLAG_BAD_BLOCK)), want, mag)
    c = ref.Cache([100, 64], 16, 2, 64, seed=2)
    q = queries(rng, 2, 4, 64)
    c.lens[1] = -3
    out = host(run_decode(pkv, c, q, 0.125, flag=pkv.FLAG_BAD_CONTEXT_LEN))
    assert (out[1] == 0).all()
    want, mag = ref.decode(q[:1], c, 0.125)
    ref.check(out[:1], want, mag)


def test_nan_and_infinities(pkv):
    """A NaN scale, code or query element, or an infinite one, makes its own rows NaN and no other."""
    rng = np.random.default_rng(6)
    c = ref.Cache([50, 200, 70], 16, 2, 128, seed=4)
    q = queries(rng, 3, 4, 128)
    q_lens = [5, 7, 3]
    qp = queries(rng, 15, 4, 128)
    clean, clean_p = run_decode(pkv, c, q, 0.1), run_prefill(pkv, c, qp, q_lens, 0.1)
    for name in ("vs", "ks"):
        d = ref.Cache([50, 200, 70], 16, 2, 128, seed=4)
        getattr(d, name)[d.tables[1, 2], 1] = np.nan
        got, got_p = run_decode(pkv, d, q, 0.1), run_prefill(pkv, d, qp, q_lens, 0.1)
        assert got[1, 2:].isnan().all() and got_p[5:12, 2:].isnan().all()
        for x, y in ((got, clean), (got_p, clean_p)):
            there = ~x.isnan()
            assert torch.equal(x[there], y[there])
        assert int(got.isnan().sum()) == 2 * 128 and int(got_p.isnan().sum()) == 7 * 2 * 128
    for bits in (0x7F80, 0xFF80, 0x7FC0):
        q2, qp2 = q.copy(), qp.copy()
        q2[2, 1, 9], qp2[6, 3, 100] = bits, bits
        got, got_p = run_decode(pkv, c, q2, 0.1), run_prefill(pkv, c, qp2, q_lens, 0.1)
        assert got[2, 1].isnan().all() and int(got.isnan().sum()) == 128
        assert got_p[6, 3].isnan().all() and int(got_p.isnan().sum()) == 128


@pytest.mark.parametrize("Hkv,G,D,bs,spread,pow2", [
    (2, 2, 64, 16, 1.0, True), (1, 1, 64, 48, 0.0, True), (2, 4, 128, 16, 3.0, True), (2, 2, 128, 256, 1.0, True),
    (1, 8, 128, 32, 1.0, True), (2, 8, 64, 64, 2.0, True), (2, 4, 128, 16, 1.0, False), (1, 2, 64, 128, 1.0, False),
    (1, 1, 128, 128, 0.0, True)])
def test_prefill(pkv, Hkv, G, D, bs, spread, pow2):
    rng = np.random.default_rng(Hkv * 10 + G)
    q_lens = [1, 3, 0, 130, 17, 300, 64, 2]
    prefix = [0, 200, 40, 0, 16, 127, 0, 1]
    c = ref.Cache(np.add(q_lens, prefix), bs, Hkv, D, seed=G, spread=spread, pow2=pow2, mbs_extra=1)
    q = queries(rng, sum(q_lens), Hkv * G, D)
    for scale in (D ** -0.5, -0.05, 0.0):
        want, mag = ref.prefill(q, c, q_lens, scale)
        ref.check(host(run_prefill(pkv, c, q, q_lens, scale)), want, mag, f"scale {scale}")
    want, mag = ref.prefill(q, c, q_lens, 0.1)
    ref.check(host(run_prefill(pkv, c, q, q_lens, 0.1, max_q=1000)), want, mag, "a loose bound")


@pytest.mark.parametrize("q_lens,prefix,Hkv,G,D,bs", [
    ([5], [6000], 1, 4, 128, 256),   # one item, split over many CTAs
    ([40, 1], [3000, 5], 2, 2, 64, 16),
    ([2000], [9000], 1, 16 // 2, 64, 64),
    ([1300], [5000], 8, 4, 64, 16)])  # 168 items: those of the last round
def test_prefill_split_over_the_keys(pkv, q_lens, prefix, Hkv, G, D, bs):
    rng = np.random.default_rng(1)
    c = ref.Cache(np.add(q_lens, prefix), bs, Hkv, D, seed=7)
    Tq = sum(q_lens)
    assert pkv.prefill_scaled_workspace_bytes(len(q_lens), Tq, max(q_lens), Hkv * G, Hkv, D, c.MBS, bs) > 0
    q = queries(rng, Tq, Hkv * G, D)
    want, mag = ref.prefill(q, c, q_lens, 0.1)
    ref.check(host(run_prefill(pkv, c, q, q_lens, 0.1)), want, mag)


def test_prefill_scales_far_apart(pkv):
    rng = np.random.default_rng(0)
    for bs, D in ((16, 64), (32, 128), (128, 128), (256, 64)):
        c = ref.Cache([1500, 400], bs, 1, D, seed=3)
        n = (c.tables >= 0).sum(1)
        for b in range(2):
            # within a tile of 128 tokens at most 2^10 apart, from tile to tile anything
            per = max(1, 128 // bs)
            tile = np.repeat(rng.integers(-20, 20, n[b] // per + 1), per)[: n[b]]
            c.vs[c.tables[b, : n[b]], 0] = 2.0 ** (tile + rng.integers(-5, 5, n[b]))
            c.ks[c.tables[b, : n[b]], 0] = 2.0 ** -rng.integers(7, 30, n[b])
        q_lens = [300, 400]
        q = queries(rng, 700, 2, D)
        want, mag = ref.prefill(q, c, q_lens, 0.1)
        ref.check(host(run_prefill(pkv, c, q, q_lens, 0.1)), want, mag, f"bs {bs}")


def test_prefill_bad_blocks_lengths_and_rows_behind(pkv):
    rng = np.random.default_rng(5)
    q_lens = [20, 150, 30]
    c = ref.Cache([120, 150, 60], 16, 2, 64, seed=2)
    q = queries(rng, 210, 4, 64)  # ten rows behind the sequences' own
    want, mag = ref.prefill(q, c, q_lens, 0.125)
    out = run_prefill(pkv, c, q, q_lens, 0.125)
    ref.check(host(out)[:200], want[:200], mag[:200])
    assert (out[200:] == 7).all()
    # a block that is not there: its tokens are left out (the reference: no weight for them)
    d = ref.Cache([120, 150, 60], 16, 2, 64, seed=2)
    d.tables[1, 3] = d.NB + 5
    out = host(run_prefill(pkv, d, q, q_lens, 0.125, flag=pkv.FLAG_BAD_BLOCK))
    ref.check(out[:20], want[:20], mag[:20])
    ref.check(out[170:200], want[170:200], mag[170:200])
    K, V = np.delete(c.rows(1, "k"), np.s_[48:64], 0), np.delete(c.rows(1, "v"), np.s_[48:64], 0)
    for i in (0, 47, 50, 63, 64, 149):
        seen = i + 1 if i < 48 else max(48, i + 1 - 16)
        for h in range(4):
            w, m = ref.attend(ref.from_bf16(q[20 + i: 21 + i, h]), K[:seen, h // 2], V[:seen, h // 2], 0.125)
            ref.check(out[20 + i, h], w[0], m[0])
    # lengths that cannot be: the sequence is skipped
    cu_k = np.array([0, 120, 125, 185], np.int32)
    out = run_prefill(pkv, c, q, q_lens, 0.125, flag=pkv.FLAG_BAD_CONTEXT_LEN, cu_k=cu_k)
    assert (out[20:170] == 7).all()
    ref.check(host(out)[:20], want[:20], mag[:20])


def test_the_same_codes_as_one_scale_per_tensor(pkv):
    """With all scales equal the calls agree with the per-tensor ones."""
    rng = np.random.default_rng(8)
    c = ref.Cache([500, 33, 1], 16, 2, 128, seed=1)
    c.ks[:], c.vs[:] = 2.0 ** -7, 2.0 ** -6
    q = queries(rng, 3, 8, 128)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    pkv.paged_attn_decode_fp8(dev(q), dev(c.k), dev(c.v), dev(c.tables), dev(c.lens), 0.1, 2.0 ** -7, 2.0 ** -6, out)
    want, mag = ref.decode(q, c, 0.1)
    got = host(run_decode(pkv, c, q, 0.1))
    ref.check(got, want, mag)
    assert (np.abs(got - host(out)) <= 2.0 ** -7 * np.abs(want) + 2.0 ** -10 * mag).all()


def test_captured_with_two_graphs(pkv):
    """Two graphs captured without a workspace, replayed side by side on changed inputs."""
    rng = np.random.default_rng(3)
    jobs = []
    s = torch.cuda.Stream()
    for seed in (1, 2):
        c = ref.Cache([3000, 40, 700], 32, 1, 64, seed=seed)
        q, qp = queries(rng, 3, 4, 64), queries(rng, 60, 4, 64)
        t = [dev(x) for x in (c.k, c.v, c.ks, c.vs, c.tables)]
        cu_q, cu_k = dev(np.array([0, 50, 55, 60], np.int32)), dev(np.array([0, 3000, 3040, 3740], np.int32))
        x, xp, lens = dev(q), dev(qp), dev(c.lens)
        out, outp = torch.empty_like(x), torch.empty_like(xp)
        call = lambda x=x, xp=xp, t=t, lens=lens, cu_q=cu_q, cu_k=cu_k, out=out, outp=outp: (
            pkv.paged_attn_decode_scaled(x, *t, lens, 0.1, out), pkv.paged_prefill_scaled(xp, *t, cu_q, cu_k, 50, 0.1, outp))
        call()
        torch.cuda.synchronize()
        want = out.clone(), outp.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
        out.zero_(), outp.zero_()
        w, m = ref.decode(q, c, 0.1)
        ref.check(host(want[0]), w, m)
        w, m = ref.prefill(qp, c, [50, 5, 5], 0.1)
        ref.check(host(want[1]), w, m)
        jobs.append((g, (out, outp), want, call))  # (call keeps the inputs)
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(10):
        for (g, *_), t in zip(jobs, streams):
            with torch.cuda.stream(t):
                g.replay()
    torch.cuda.synchronize()
    for _, outs, wants, _ in jobs:
        for a, b in zip(outs, wants):
            assert torch.equal(a, b)


def test_output_in_pinned_memory(pkv):
    rng = np.random.default_rng(2)
    c = ref.Cache([90, 5], 16, 2, 64, seed=1)
    q, qp = queries(rng, 2, 4, 64), queries(rng, 25, 4, 64)
    t = [dev(x) for x in (c.k, c.v, c.ks, c.vs, c.tables)]
    out, outp = (torch.zeros(x.shape, dtype=torch.bfloat16, pin_memory=True) for x in (q, qp))
    pkv.paged_attn_decode_scaled(dev(q), *t, dev(c.lens), 0.1, out)
    pkv.paged_prefill_scaled(dev(qp), *t, dev(np.array([0, 20, 25], np.int32)), dev(np.array([0, 90, 95], np.int32)), 20, 0.1, outp)
    torch.cuda.synchronize()
    w, m = ref.decode(q, c, 0.1)
    ref.check(host(out), w, m)
    w, m = ref.prefill(qp, c, [20, 5], 0.1)
    ref.check(host(outp), w, m)
