"""The budget calls as an engine uses them: prompt, decode steps, eviction, more
decode steps, with the block allocator; streams, graphs and arguments."""

import numpy as np
import pytest

import budget_reference as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv(cuda_lib_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_85_gb300 as m

    m.load_library()
    return m


def bf(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def rows(rng, *shape):
    return ref.to_bf16(rng.standard_normal(shape, dtype=np.float32))


class Model:
    """What the engine should hold: per sequence and KV head, the kept tokens' K, V and weights."""

    def __init__(self, Hkv, G, D, scale):
        self.Hkv, self.G, self.D, self.scale = Hkv, G, D, scale
        self.seqs = {}

    def step(self, s, q, k, v, window=0):
        """New tokens k, v [n, Hkv, D] with queries q [n, Hq, D] (bf16 bits); returns out in 64 bits."""
        old = self.seqs.get(s, [(np.zeros((0, self.D)), np.zeros((0, self.D)), np.zeros(0))] * self.Hkv)
        q, k, v = ref.from_bf16(q), ref.from_bf16(k), ref.from_bf16(v)
        n, out, new = len(q), np.zeros(q.shape), []
        for h in range(self.Hkv):
            K, V = np.concatenate([old[h][0], k[:, h]]), np.concatenate([old[h][1], v[:, h]])
            w, base = np.concatenate([old[h][2], np.zeros(n)]), len(old[h][2])
            for i in range(n):
                m = base + i + 1
                for g in range(self.G):
                    sc = K[:m] @ q[i, h * self.G + g] * self.scale
                    p = np.exp(sc - sc.max())
                    p /= p.sum()
                    out[i, h * self.G + g] = p @ V[:m]
                    if not window or i >= n - window:
                        w[:m] += p
            new.append((K, V, w))
        self.seqs[s] = new
        return out

    def trim(self, s, budget, recent):
        new = []
        for K, V, w in self.seqs[s]:
            n = len(w)
            if n > budget:
                old = n - recent
                heavy = sorted(sorted(range(old), key=lambda t: (-w[t], t))[: budget - recent])
                at = heavy + list(range(old, n))
                K, V, w = K[at], V[at], w[at]
            new.append((K, V, w))
        self.seqs[s] = new


@pytest.mark.parametrize("window", [0, 8])
def test_prompt_decode_evict_decode(pkv, window):
    """Three sequences through a prompt, decode steps, an eviction and more decode steps.

    The eviction goes by weights the GPU formed in fp32 and the model in 64
    bits; they must agree on every token that stays, which the check below
    makes sure of (the border weights differ by far more than their errors)."""
    from paged_kv_cache_85_gb300.block_manager import BlockManager

    Hkv, G, D, bs, NB, MBS = 2, 4, 64, 16, 64, 20
    budget, recent = 60, 12
    scale = D ** -0.5
    rng = np.random.default_rng(11)
    bm, model = BlockManager(NB, bs), Model(Hkv, G, D, scale)
    kc = torch.full((NB, bs, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    w = torch.full((NB, Hkv, bs), float("nan"), dtype=torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, lens = [1, 2, 3], [100, 37, 150]

    def check(out, want):
        got = out.float().cpu().numpy().astype(np.float64)
        # the framework's bar for its attention outputs
        assert (np.abs(got - want) <= 1e-2 + 2.0 ** -8 * np.abs(want)).all()

    # prompt
    for s, n in zip(ids, lens):
        assert bm.allocate(s, rng.integers(0, 1000, n)) == 0
    q, k, v = (rows(rng, sum(lens), h, D) for h in (Hkv * G, Hkv, Hkv))
    slots = torch.from_numpy(np.concatenate([bm.slots(s, 0, n) for s, n in zip(ids, lens)])).cuda()
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    tables, ctx, _ = bm.decode_batch(ids, MBS)
    t, cud = torch.from_numpy(tables).cuda(), torch.from_numpy(cu).cuda()
    qd = bf(q)
    pkv.store_kvcache(bf(k), bf(v), kc, vc, slots, err_flag=err)
    out = pkv.paged_prefill_weights(qd, kc, vc, t, cud, cud, max(lens), scale, torch.empty_like(qd), w, window=window, err_flag=err)
    check(out, np.concatenate([model.step(s, q[a:b], k[a:b], v[a:b], window) for s, a, b in zip(ids, cu, cu[1:])]))

    def decode(steps):
        for _ in range(steps):
            slot = torch.from_numpy(bm.append_batch(ids, [5] * 3)).cuda()
            tables, ctx, _ = bm.decode_batch(ids, MBS)
            q, k, v = (rows(rng, 3, h, D) for h in (Hkv * G, Hkv, Hkv))
            qd = bf(q)
            pkv.store_kvcache(bf(k), bf(v), kc, vc, slot, err_flag=err)
            out = pkv.paged_attn_decode_weights(qd, kc, vc, torch.from_numpy(tables).cuda(), torch.from_numpy(ctx).cuda(), scale,
                                                torch.empty_like(qd), w, err_flag=err)
            check(out, np.concatenate([model.step(s, q[i: i + 1], k[i: i + 1], v[i: i + 1]) for i, s in enumerate(ids)]))

    def weights():
        tables, ctx, _ = bm.decode_batch(ids, MBS)
        flat = w.cpu().numpy()
        for i, s in enumerate(ids):
            at = np.arange(ctx[i])
            got = flat[tables[i, at // bs], :, at % bs]  # [n, Hkv]
            for h in range(Hkv):
                want = model.seqs[s][h][2]
                # some 170 additions of G weights per token, each within weight_tolerance (|score| sums below 40)
                assert np.abs(got[:, h] - want).max() <= ref.weight_tolerance(D, 40) * want.max() + 200 * 2.0 ** -24 * want.max()
                yield s, h, want

    decode(4)
    for s, h, want in weights():
        if len(want) > budget:  # the border is clear of the errors
            x = np.sort(want[: len(want) - recent])[::-1]
            assert x[budget - recent - 1] - x[budget - recent] > 1e-4 * x[budget - recent], "an unlucky draw: choose another seed"

    # eviction: tables first, then the allocator, then the GPU
    tables, ctx, _ = bm.decode_batch(ids, MBS)
    free = bm.num_free_blocks
    ctxd = torch.from_numpy(ctx).cuda()
    for s in ids:
        assert bm.can_evict(s)
        bm.evict(s, budget)
        model.trim(s, budget, recent)
    pkv.evict_kvcache(kc, vc, w, torch.from_numpy(tables).cuda(), ctxd, budget, recent, ctxd, err_flag=err)
    assert ctxd.tolist() == [bm.seq_len(s) for s in ids] == [60, 41, 60]
    assert bm.num_free_blocks == free + (7 - 4) + (10 - 4)
    list(weights())
    decode(20)
    list(weights())

    # a chunk of new tokens on top of trimmed contexts
    n = 9
    q, k, v = (rows(rng, 3 * n, h, D) for h in (Hkv * G, Hkv, Hkv))
    slots = np.concatenate([[bm.append(s, 3) for _ in range(n)] for s in ids])
    tables, ctx, _ = bm.decode_batch(ids, MBS)
    cq = torch.arange(0, 3 * n + 1, n, dtype=torch.int32, device="cuda")
    ck = torch.from_numpy(np.concatenate([[0], np.cumsum(ctx)]).astype(np.int32)).cuda()
    qd = bf(q)
    pkv.store_kvcache(bf(k), bf(v), kc, vc, torch.from_numpy(slots).cuda(), err_flag=err)
    out = pkv.paged_prefill_weights(qd, kc, vc, torch.from_numpy(tables).cuda(), cq, ck, n, scale, torch.empty_like(qd), w,
                                    window=window, err_flag=err)
    check(out, np.concatenate([model.step(s, q[i * n: i * n + n], k[i * n: i * n + n], v[i * n: i * n + n], window) for i, s in enumerate(ids)]))
    list(weights())
    assert int(err.item()) == 0


def three_calls(pkv, c, fp8=False, window=0):
    """(run, outputs): a decode, a prefill (bf16) and an eviction over the same cache."""
    Hkv, D = c.Hkv, c.D
    k, v = (torch.from_numpy(c.k).cuda(), torch.from_numpy(c.v).cuda()) if fp8 else (bf(c.k), bf(c.v))
    w = torch.from_numpy(c.w.copy()).cuda()
    t, n = torch.from_numpy(c.tables).cuda(), torch.from_numpy(c.lens).cuda()
    B = len(c.lens)
    q = bf(ref.to_bf16(np.random.default_rng(1).standard_normal((B, 2 * Hkv, D), dtype=np.float32)))
    ql = np.minimum(c.lens, 20)
    cq = torch.from_numpy(np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)).cuda()
    ck = torch.from_numpy(np.concatenate([[0], np.cumsum(c.lens)]).astype(np.int32)).cuda()
    qp = bf(ref.to_bf16(np.random.default_rng(2).standard_normal((int(ql.sum()), 2 * Hkv, D), dtype=np.float32)))
    o1, o2, o3 = torch.zeros_like(q), torch.zeros_like(qp), torch.zeros_like(n)

    def run():
        if fp8:
            pkv.paged_attn_decode_weights_fp8(q, k, v, t, n, 0.1, c.k_scale, c.v_scale, o1, w)
        else:
            pkv.paged_attn_decode_weights(q, k, v, t, n, 0.1, o1, w)
            pkv.paged_prefill_weights(qp, k, v, t, cq, ck, 20, 0.1, o2, w, window=window)
        pkv.evict_kvcache(k, v, w, t, n, 50, 10, o3)

    return run, (o1, o2, o3, k, v, w)


def bits(tensors):
    return [x.cpu().view(torch.uint8) if x.numel() else x.cpu() for x in tensors]


@pytest.mark.parametrize("fp8", [False, True])
def test_graph_replay_matches_eager(pkv, fp8):
    """Captured once and replayed, each call over its own buffers; an eager call of the same sizes runs in between."""
    c = ref.Cache([70, 1, 200, 333], 16, 2, 64, fp8=fp8, seed=3)
    run, got = three_calls(pkv, c, fp8)
    eager, want = three_calls(pkv, c, fp8)
    for r in (run, eager):  # set-up outside the capture
        r()
    start = [x.clone() for x in want]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            run()
    torch.cuda.current_stream().wait_stream(s)
    for x, y in zip(got, start):
        x.copy_(y)
    for step in range(3):
        graph.replay()
        eager()
        torch.cuda.synchronize()
        for x, y in zip(bits(got), bits(want)):
            assert torch.equal(x, y), f"replay {step}"


def test_two_graphs_do_not_share_scratch(pkv):
    """Two graphs of different sizes, replayed at once on two streams, give what they give alone."""
    big = ref.Cache(np.random.default_rng(0).integers(50, 900, size=40), 16, 4, 128, seed=1)
    small = ref.Cache([300, 20], 32, 2, 64, seed=2)
    graphs, outs, alone = [], [], []
    for c in (big, small):
        run, got = three_calls(pkv, c, window=4)
        start = [x.clone() for x in got]
        run()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                run()
        torch.cuda.synchronize()
        for x, y in zip(got, start):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        alone.append(bits(got))
        for x, y in zip(got, start):
            x.copy_(y)
        graphs.append((g, s, run))  # run holds the captured inputs
        outs.append(got)
    torch.cuda.synchronize()
    for g, s, _ in graphs:
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for got, want in zip(outs, alone):
        for x, y in zip(bits(got), want):
            assert torch.equal(x, y)


def test_calls_on_two_streams_at_once(pkv):
    c = ref.Cache(np.random.default_rng(0).integers(50, 900, size=30), 16, 4, 64, seed=1)
    run, want = three_calls(pkv, c)
    for _ in range(3):
        run()
    torch.cuda.synchronize()
    pair = [three_calls(pkv, c) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for (run, _), s in zip(pair, streams):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for _, got in pair:
        for x, y in zip(bits(got), bits(want)):
            assert torch.equal(x, y)


def test_workspace_given_by_the_caller(pkv):
    """A workspace of exactly the reported size, full of NaN, gives the same results; a smaller one is refused."""
    c = ref.Cache([70, 1, 200], 16, 2, 64, seed=3)
    q = bf(ref.to_bf16(np.random.default_rng(1).standard_normal((3, 4, 64), dtype=np.float32)))
    k, v = bf(c.k), bf(c.v)
    t, n = torch.from_numpy(c.tables).cuda(), torch.from_numpy(c.lens).cuda()
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    ck = torch.from_numpy(np.concatenate([[0], np.cumsum(c.lens)]).astype(np.int32)).cuda()
    MBS = c.MBS
    calls = [
        (pkv.decode_weights_workspace_bytes(3, 4, 2, 64, MBS, 16),
         lambda w, ws: pkv.paged_attn_decode_weights(q, k, v, t, n, 0.1, torch.empty_like(q), w, workspace=ws)),
        (pkv.prefill_weights_workspace_bytes(3, 3, 1, 4, 2, 64, MBS, 16),
         lambda w, ws: pkv.paged_prefill_weights(q, k, v, t, cu, ck, 1, 0.1, torch.empty_like(q), w, workspace=ws)),
        (pkv.evict_workspace_bytes(3, 2, MBS, 16, 50),
         lambda w, ws: pkv.evict_kvcache(k.clone(), v.clone(), w, t, n, 50, 10, torch.empty_like(n), workspace=ws)),
    ]
    for need, call in calls:
        assert need > 0
        res = []
        for ws in (None, torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")):
            w = torch.from_numpy(c.w.copy()).cuda()
            res += [(call(w, ws), w)]
        torch.cuda.synchronize()
        for x, y in zip(*res):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        w = torch.from_numpy(c.w.copy()).cuda()
        with pytest.raises(pkv.PkvError, match="WORKSPACE"):
            call(w, torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
        with pytest.raises(ValueError, match="contiguous"):
            call(w, torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2])
        with pytest.raises(ValueError, match="workspace"):
            call(w, torch.empty(need, dtype=torch.uint8))
        torch.cuda.synchronize()
        assert np.array_equal(w.cpu().numpy(), c.w, equal_nan=True), "a refused call wrote"


def test_output_in_pinned_host_memory(pkv):
    c = ref.Cache([70, 1, 200], 16, 2, 64, seed=3)
    q = bf(ref.to_bf16(np.random.default_rng(1).standard_normal((3, 4, 64), dtype=np.float32)))
    k, v, t, n = bf(c.k), bf(c.v), torch.from_numpy(c.tables).cuda(), torch.from_numpy(c.lens).cuda()
    got = []
    for out in (torch.empty_like(q), torch.empty(q.shape, dtype=q.dtype).pin_memory()):
        w = torch.from_numpy(c.w.copy()).cuda()
        pkv.paged_attn_decode_weights(q, k, v, t, n, 0.1, out, w)
        torch.cuda.synchronize()
        got.append(out.cpu().view(torch.int16))
    assert torch.equal(*got)
    # a prefill step: whole items, and items split over the keys
    for lens in ([70, 1, 200], [3000, 5, 2000]):
        c = ref.Cache(lens, 16, 2, 64, seed=3)
        k, v, t = bf(c.k), bf(c.v), torch.from_numpy(c.tables).cuda()
        cq = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
        ck = torch.from_numpy(np.concatenate([[0], np.cumsum(c.lens)]).astype(np.int32)).cuda()
        got = []
        for out in (torch.empty_like(q), torch.empty(q.shape, dtype=q.dtype).pin_memory()):
            w = torch.from_numpy(c.w.copy()).cuda()
            pkv.paged_prefill_weights(q, k, v, t, cq, ck, 1, 0.1, out, w)
            torch.cuda.synchronize()
            got.append(out.cpu().view(torch.int16))
        assert torch.equal(*got)


def test_arguments_are_checked(pkv):
    c = ref.Cache([70, 1, 200], 16, 2, 64, seed=3)
    q = bf(ref.to_bf16(np.random.default_rng(1).standard_normal((3, 4, 64), dtype=np.float32)))
    k, v, t, n = bf(c.k), bf(c.v), torch.from_numpy(c.tables).cuda(), torch.from_numpy(c.lens).cuda()
    w, out = torch.from_numpy(c.w.copy()).cuda(), torch.empty_like(q)
    dec = lambda **kw: pkv.paged_attn_decode_weights(*[kw.get(x, y) for x, y in dict(
        q=q, k=k, v=v, t=t, n=n, s=0.1, out=out, w=w).items()], **{x: kw[x] for x in ("err_flag",) if x in kw})
    for kw, what in ((dict(w=w.half()), "weights"), (dict(w=w[:-1]), "weights"), (dict(w=w.transpose(1, 2)), "weights"),
                     (dict(w=w.cpu()), "weights"), (dict(q=q.float()), "q"), (dict(k=k.half()), "k_cache"), (dict(v=v[:-1]), "shapes"),
                     (dict(t=t.long()), "block_tables"), (dict(t=t[:2]), "batch"), (dict(n=n[:2]), "batch"), (dict(n=n.cpu()), "context_lens"),
                     (dict(out=out[:2]), "out"), (dict(out=out.cpu()), "out"), (dict(q=q[:, :, :32].contiguous()), "head_dim"),
                     (dict(err_flag=torch.zeros(0, dtype=torch.int32, device="cuda")), "err_flag"),
                     (dict(err_flag=torch.zeros(1, device="cuda")), "err_flag")):
        with pytest.raises((ValueError, TypeError), match=what):
            dec(**kw)
    ev = lambda **kw: pkv.evict_kvcache(*[kw.get(x, y) for x, y in dict(k=k, v=v, w=w, t=t, n=n, budget=20, recent=4, o=n.clone()).items()])
    for kw in (dict(w=w[:-1]), dict(o=n[:2]), dict(o=n.long()), dict(t=t[:2]), dict(v=v.half()), dict(k=k.float())):
        with pytest.raises((ValueError, TypeError)):
            ev(**kw)
    for kw in (dict(budget=0), dict(recent=21), dict(recent=-1)):
        with pytest.raises(pkv.PkvError):
            ev(**kw)
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    with pytest.raises(pkv.PkvError, match="window"):
        pkv.paged_prefill_weights(q, k, v, t, cu, cu, 1, 0.1, out, w, window=-1)
    torch.cuda.synchronize()
    assert np.array_equal(w.cpu().numpy(), c.w, equal_nan=True)


def test_nothing_to_do(pkv):
    """No sequences, no new tokens."""
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(4, 2, 16, device="cuda")
    e = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt, device="cuda")
    q = e(0, 4, 64, dt=torch.bfloat16)
    pkv.paged_attn_decode_weights(q, k, k.clone(), e(0, 1), e(0), 0.1, q.clone(), w)
    pkv.paged_prefill_weights(q, k, k.clone(), e(0, 1), e(1), e(1), 0, 0.1, q.clone(), w)
    pkv.paged_prefill_weights(q, k, k.clone(), e(2, 1), e(3), e(3), 0, 0.1, q.clone(), w)
    pkv.evict_kvcache(k, k.clone(), w, e(0, 1), e(0), 4, 2, e(0))
    torch.cuda.synchronize()
    assert not w.any()
