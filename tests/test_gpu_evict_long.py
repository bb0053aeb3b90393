"""The eviction where a CTA of its selection holds more keys than fit its shared
memory, where clusters of eight share a context, and the budget calls from two
threads at once."""

import threading

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


def dev(x):
    x = np.ascontiguousarray(x)
    return torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).cuda() if x.dtype == np.uint16 else torch.from_numpy(x).cuda()


def host(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy()


def check(pkv, c, budget, recent):
    k, v, w, t, n = dev(c.k), dev(c.v), dev(c.w.copy()), dev(c.tables), dev(c.lens)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pkv.evict_kvcache(k, v, w, t, n, budget, recent, torch.empty_like(n), err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for got, want in zip((k, v, w, out), ref.evict(c, budget, recent)):
        np.testing.assert_array_equal(host(got), want)


def few_values(c, seed):
    """Ties by the thousand, so that the border value's tokens lie in every CTA's part."""
    c.w = np.random.default_rng(seed).integers(0, 3, c.w.shape).astype(np.float32)


@pytest.mark.parametrize("budget,recent", [(100, 10), (12600, 700), (20000, 0), (13000, 13000)])
@pytest.mark.parametrize("ties", [False, True])
def test_keys_beyond_shared_memory(pkv, budget, recent, ties):
    """Many (sequence, KV head) pairs, so one CTA each, with contexts above the 12288 keys that it holds."""
    lens = np.random.default_rng(0).integers(0, 40, size=320)
    lens[[3, 100, 319]] = [25000, 12289, 13001]
    c = ref.Cache(lens, 16, 1, 64, fp8=True, seed=1)
    if ties:
        few_values(c, 2)
    check(pkv, c, budget, recent)


@pytest.mark.parametrize("lens,bs", [([40000, 17001], 16), ([130001], 64)])
@pytest.mark.parametrize("part,recent", [(8, 0.1), (2, 0.5), (1.001, 0.0)])
@pytest.mark.parametrize("ties", [False, True])
def test_clusters_of_eight(pkv, lens, bs, part, recent, ties):
    """Few pairs of long contexts, the longest with more keys than eight CTAs hold."""
    c = ref.Cache(lens, bs, 1, 64, fp8=len(lens) == 1, seed=3)
    if ties:
        few_values(c, 4)
    budget = int(max(lens) / part)
    check(pkv, c, budget, int(budget * recent))


@pytest.mark.parametrize("own_stream", [False, True])
def test_two_threads_at_once(pkv, own_stream):
    """Each thread keeps workspaces of its own, also where both use one stream."""
    rng = np.random.default_rng(5)
    caches = [ref.Cache(rng.integers(200, 900, size=20), 16, 2, 64, seed=s) for s in (1, 2)]

    def inputs(c):
        r = np.random.default_rng(int(c.lens.sum()))
        B, ql = len(c.lens), np.minimum(c.lens, 150)
        cu = lambda x: dev(np.concatenate([[0], np.cumsum(x)]).astype(np.int32))
        q = dev(ref.to_bf16(r.standard_normal((B, 8, 64), dtype=np.float32)))
        qp = dev(ref.to_bf16(r.standard_normal((int(ql.sum()), 8, 64), dtype=np.float32)))
        return dev(c.k), dev(c.v), dev(c.w.copy()), dev(c.tables), dev(c.lens), q, qp, cu(ql), cu(c.lens)

    def steps(x, n=6):
        k, v, w, t, ctx, q, qp, cq, ck = x
        outs = []
        for _ in range(n):
            outs.append(pkv.paged_prefill_weights(qp, k, v, t, cq, ck, 150, 0.125, torch.empty_like(qp), w))
            outs.append(pkv.paged_attn_decode_weights(q, k, v, t, ctx, 0.125, torch.empty_like(q), w))
            pkv.evict_kvcache(k, v, w, t, ctx, 150, 20, torch.empty_like(ctx))
        return outs + [k, v, w]

    want = [steps(inputs(c)) for c in caches]
    torch.cuda.synchronize()
    got, start = [None, None], threading.Barrier(2)
    states = [inputs(c) for c in caches]
    streams = [torch.cuda.Stream() if own_stream else torch.cuda.current_stream() for _ in caches]
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(streams[i]):
            start.wait()
            got[i] = steps(states[i])
            streams[i].synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
