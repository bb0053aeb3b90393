"""Contexts whose positions, times the query heads of a group, pass 32 bits."""

import numpy as np
import pytest

import budget_reference as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_prompt_weights_of_a_context_beyond_2_to_the_28(cuda_lib_path):
    """Three new tokens of eight heads on 3 * 2^27 cached ones.  The table names one block of 65536 tokens again and
    again, so that the cache is small and every slot gathers the weights of its 6144 copies: with C copies of the
    scores s and the last block's own scores r,  w = sum over rows of C e^s / (C sum e^s + sum e^r)."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_85_gb300 as pkv

    pkv.load_library()
    bs, D, G, q_len, tail, copies = 1 << 16, 64, 8, 3, 40, 6144
    n, base = copies * bs + tail, copies * bs + tail - 3
    rng = np.random.default_rng(7)
    kb = ref.to_bf16(0.5 * rng.standard_normal((2, bs, 1, D), dtype=np.float32))
    vb = ref.to_bf16(rng.standard_normal((2, bs, 1, D), dtype=np.float32))
    qb = ref.to_bf16(rng.standard_normal((q_len, G, D), dtype=np.float32))
    dev = lambda x: torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    q, k, v = dev(qb), dev(kb), dev(vb)
    table = torch.zeros(1, copies + 1, dtype=torch.int32, device="cuda")
    table[0, copies] = 1
    w = torch.zeros(2, 1, bs, device="cuda")
    w[1, 0, tail - 3:tail] = float("nan")  # the new tokens'
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pkv.paged_prefill_weights(q, k, v, table, i32([0, q_len]), i32([0, n]), q_len, 0.125, torch.empty_like(q), w, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0

    K, V, Q = (ref.from_bf16(x) for x in (kb[:, :, 0], vb[:, :, 0], qb))
    want, want_out = np.zeros((2, bs)), np.zeros(qb.shape)
    for i in range(q_len):
        own = base - copies * bs + i + 1  # tokens of the last block that row i sees
        for g in range(G):
            e, r = np.exp(K[0] @ Q[i, g] * 0.125), np.exp(K[1, :own] @ Q[i, g] * 0.125)
            z = copies * e.sum() + r.sum()
            want[0] += copies * e / z
            want[1, :own] += r / z
            want_out[i, g] = (copies * e @ V[0] + r @ V[1, :own]) / z
    got = w.double().cpu().numpy()[:, 0]
    big = 0.125 * float(np.abs(Q).max()) * float(np.abs(K).sum(-1).max())
    # beyond one softmax weight's own error: a slot's additions, one per copy, and a row's sum, which a thread
    # gathers over the 1/304 of the context that is a split's share, 64 keys at a time, each by fp32 additions
    # of positive terms (off by at most 2^-24 of the sum each)
    tol = ref.weight_tolerance(D, big) + (copies + n / 304 / 128 + 128 + 304) * 2.0 ** -24
    off = np.abs(got - want)
    assert (off <= tol * want + 1e-37).all(), float((off / np.maximum(want, 1e-37)).max() / tol)
    assert np.abs(out.double().cpu().numpy() - want_out).max() <= 1e-2  # the framework's bar for its attention outputs
