"""Calls that follow each other on a stream without the host in between, where
one writes the lengths that the next one reads."""

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


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("store", [False, True])
@pytest.mark.parametrize("record", [False, True])
@pytest.mark.parametrize("lens", [[300, 20, 1000, 77], "many"])
def test_decode_right_after_an_eviction_in_place(pkv, fp8, store, record, lens):
    """evict(lens -> lens), [store,] decode, again and again, enqueued at once: bit for bit what they give one by one."""
    if lens == "many":
        lens = np.random.default_rng(4).integers(1, 700, size=600)
    Hkv, D, bs = 2, 64, 16
    c = ref.Cache(lens, bs, Hkv, D, fp8=fp8, seed=3)
    B, rng = len(c.lens), np.random.default_rng(1)
    q = dev(ref.to_bf16(rng.standard_normal((B, 2 * Hkv, D), dtype=np.float32)))
    new = [dev(ref.to_bf16(rng.standard_normal((B, Hkv, D), dtype=np.float32))) for _ in range(2)]
    t, first = dev(c.tables), dev(c.lens)
    budgets = (60, 200, 33, 500, 16, 100)
    # the newest token's slot under each budget
    kept = [np.minimum(c.lens, b) - 1 for b in budgets]
    slots = [dev(c.tables[np.arange(B), n // bs].astype(np.int64) * bs + n % bs) for n in kept]

    def steps(wait):
        k, v, w = dev(c.k), dev(c.v), dev(c.w.copy())
        ctx, outs = first.clone(), []
        torch.cuda.synchronize()
        for i, budget in enumerate(budgets):
            if i % 2 == 0:
                ctx.copy_(first)
            wait()
            pkv.evict_kvcache(k, v, w, t, ctx, budget, budget // 4, ctx)
            wait()
            if store:
                if fp8:
                    pkv.store_kvcache_fp8(*new, k, v, slots[i], c.k_scale, c.v_scale)
                else:
                    pkv.store_kvcache(*new, k, v, slots[i])
                wait()
            scales = (c.k_scale, c.v_scale) if fp8 else ()
            name = "paged_attn_decode" + ("_weights" if record else "") + ("_fp8" if fp8 else "")
            outs.append(getattr(pkv, name)(q, k, v, t, ctx, 0.125, *scales, torch.empty_like(q), *([w] if record else [])))
            outs.append(ctx.clone())
        torch.cuda.synchronize()
        return outs + [k, v, w]

    want = steps(torch.cuda.synchronize)
    # an odd step trims what the even one left: lengths above its budget only
    np.testing.assert_array_equal(want[1].cpu().numpy(), np.minimum(c.lens, 60))
    np.testing.assert_array_equal(want[3].cpu().numpy(), np.minimum(c.lens, 60))
    np.testing.assert_array_equal(want[5].cpu().numpy(), np.minimum(c.lens, 33))
    for _ in range(10):
        for x, y in zip(steps(lambda: None), want):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_right_after_lengths_written_on_the_gpu(pkv, fp8):
    """Lengths that the caller's own kernel has just written: longer, shorter, empty, out of range and back."""
    c = ref.Cache([700, 20, 1000, 77, 0, 1], 32, 2, 128, fp8=fp8, seed=3)
    q = dev(ref.to_bf16(np.random.default_rng(1).standard_normal((6, 4, 128), dtype=np.float32)))
    k, v, t, full = dev(c.k), dev(c.v), dev(c.tables), dev(c.lens)
    scales = (c.k_scale, c.v_scale) if fp8 else ()
    call = pkv.paged_attn_decode_fp8 if fp8 else pkv.paged_attn_decode
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    plans = [full, full // 2, torch.zeros_like(full), full, full // 3 + 1, full]
    plans[4] = torch.minimum(plans[4], full)
    want = [call(q, k, v, t, n, 0.09, *scales, torch.empty_like(q), err_flag=err) for n in plans]
    torch.cuda.synchronize()
    ctx = torch.zeros_like(full)
    got = []
    for _ in range(20):
        for n in plans:
            torch.add(n, 0, out=ctx)
            got.append(call(q, k, v, t, ctx, 0.09, *scales, torch.empty_like(q), err_flag=err))
            torch.sub(ctx, 10 ** 6, out=ctx)  # out of range between the steps
    for i, out in enumerate(got):
        assert torch.equal(out.view(torch.int16), want[i % 6].view(torch.int16))
    # lengths are judged as they are when the step's turn comes: none was out of range then
    assert int(err.item()) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("slot", [-1, 10 ** 6])
def test_a_store_of_nothing_between_two_calls(pkv, fp8, slot):
    """Calls that share a kept workspace, with a store between them that has only padding (or slots out of range): the
    second call starts once the first has ended, not once the store has."""
    rng = np.random.default_rng(2)
    c = ref.Cache(rng.integers(300, 900, size=12), 16, 2, 64, seed=3)
    B, G = 12, 8
    k, v, t, ctx = dev(c.k), dev(c.v), dev(c.tables), dev(c.lens)
    ql = rng.integers(100, 290, size=B)
    cq, ck = (dev(np.concatenate([[0], np.cumsum(x)]).astype(np.int32)) for x in (ql, c.lens))
    qp = dev(ref.to_bf16(rng.standard_normal((int(ql.sum()), 2 * G, 64), dtype=np.float32)))
    q = dev(ref.to_bf16(rng.standard_normal((B, 2 * G, 64), dtype=np.float32)))
    new = dev(ref.to_bf16(rng.standard_normal((B, 2, 64), dtype=np.float32)))
    codes = torch.zeros((2, *c.k.shape), dtype=torch.uint8, device="cuda")
    slots = torch.full((B,), slot, dtype=torch.int64, device="cuda")

    def steps(wait):
        w = dev(c.w.copy())
        torch.cuda.synchronize()
        for _ in range(4):
            pkv.paged_prefill_weights(qp, k, v, t, cq, ck, int(ql.max()), 0.125, torch.empty_like(qp), w)
            wait()
            if fp8:
                pkv.store_kvcache_fp8(new, new, codes[0], codes[1], slots, 1.0, 1.0)
            else:
                pkv.store_kvcache(new, new, k, v, slots)
            wait()
            pkv.paged_attn_decode_weights(q, k, v, t, ctx, 0.125, torch.empty_like(q), w)
            wait()
        torch.cuda.synchronize()
        return w

    want = steps(torch.cuda.synchronize)
    for _ in range(10):
        assert torch.equal(steps(lambda: None).view(torch.int32), want.view(torch.int32))
