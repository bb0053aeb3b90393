"""Decode steps captured without a workspace of the caller's."""

import numpy as np
import pytest

import budget_reference as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def dev(x):
    x = np.ascontiguousarray(x)
    return torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).cuda() if x.dtype == np.uint16 else torch.from_numpy(x).cuda()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_graph_keeps_its_workspace(cuda_lib_path, fp8):
    """After the capture the stream's own workspace is outgrown and its memory given to others: the graph writes none of
    it and replays, also beside another graph of the same stream, what the eager call gives."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_85_gb300 as pkv

    def inputs(lens, Hkv, seed):
        c = ref.Cache(lens, 32, Hkv, 64, fp8=fp8, seed=seed)
        q = dev(ref.to_bf16(np.random.default_rng(seed).standard_normal((len(lens), 4 * Hkv, 64), dtype=np.float32)))
        return q, dev(c.k), dev(c.v), dev(c.tables), dev(c.lens)

    def call(x, out):
        if fp8:
            return pkv.paged_attn_decode_fp8(*x, 0.1, 1.0, 1.0, out)
        return pkv.paged_attn_decode(*x, 0.1, out)

    small, other = inputs([3000, 40, 700], 1, 1), inputs([900, 2500], 1, 2)
    big = inputs(np.random.default_rng(3).integers(1, 2000, size=60), 4, 3)
    want = [call(x, torch.empty_like(x[0])) for x in (small, other)]
    s = torch.cuda.Stream()
    graphs, outs = [], []
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for x in (small, other):
            call(x, torch.empty_like(x[0]))
            out, g = torch.empty_like(x[0]), torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g, stream=s):
                call(x, out)
            graphs.append(g)
            outs.append(out)
        call(big, torch.empty_like(big[0]))
        torch.cuda.synchronize()
        # whatever was freed is someone else's now
        others = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in (1 << 20, 1 << 21, 1 << 22, 1 << 16) * 8]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for g, t in zip(graphs, streams):
            with torch.cuda.stream(t):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert all(bool((o == 0x5A).all()) for o in others)
