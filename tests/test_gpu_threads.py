"""Calls from a thread that has made no CUDA call of its own yet."""

import threading

import numpy as np
import pytest

import budget_reference as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def dev(x):
    x = np.ascontiguousarray(x)
    return torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).cuda() if x.dtype == np.uint16 else torch.from_numpy(x).cuda()


@pytest.mark.parametrize("name", ["decode", "decode fp8", "prefill", "decode weights", "decode weights fp8", "prefill weights", "evict"])
def test_first_call_of_a_thread(cuda_lib_path, name):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_85_gb300 as pkv

    fp8 = name.endswith("fp8")
    c = ref.Cache([70, 1, 200], 16, 2, 64, fp8=fp8, seed=3)
    k, v, t, n = dev(c.k), dev(c.v), dev(c.tables), dev(c.lens)
    q = dev(ref.to_bf16(np.random.default_rng(1).standard_normal((3, 4, 64), dtype=np.float32)))
    cq = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    ck = dev(np.concatenate([[0], np.cumsum(c.lens)]).astype(np.int32))

    def call(out, w, k, v, lens, ws):
        # every tensor is there already, so that nothing of the caller's touches the GPU first
        if name == "decode":
            pkv.paged_attn_decode(q, k, v, t, n, 0.1, out, workspace=ws)
        elif name == "decode fp8":
            pkv.paged_attn_decode_fp8(q, k, v, t, n, 0.1, 1.0, 1.0, out, workspace=ws)
        elif name == "prefill":
            pkv.paged_prefill(q, k, v, t, cq, ck, 1, 0.1, out)
        elif name == "decode weights":
            pkv.paged_attn_decode_weights(q, k, v, t, n, 0.1, out, w, workspace=ws)
        elif name == "decode weights fp8":
            pkv.paged_attn_decode_weights_fp8(q, k, v, t, n, 0.1, 1.0, 1.0, out, w, workspace=ws)
        elif name == "prefill weights":
            pkv.paged_prefill_weights(q, k, v, t, cq, ck, 1, 0.1, out, w, workspace=ws)
        else:
            pkv.evict_kvcache(k, v, w, t, n, 50, 10, lens, workspace=ws)

    states = [[torch.zeros_like(q), dev(c.w.copy()), k.clone(), v.clone(), torch.zeros_like(n),
               torch.empty(4 << 20, dtype=torch.uint8, device="cuda")] for _ in range(2)]
    call(*states[0])
    torch.cuda.synchronize()
    failed = []

    def work():
        try:
            call(*states[1])
        except Exception as e:
            failed.append(e)

    x = threading.Thread(target=work)
    x.start()
    x.join()
    assert not failed, failed
    torch.cuda.synchronize()
    for a, b in zip(states[0][:5], states[1][:5]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
