"""Recording prefill steps whose block tables are wider than their contexts: how
the work is split goes by the widths and, per item, by the contexts."""

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


def reference(c, q, cu, G, scale):
    """(out, weights added per slot, largest sum |q_d k_d| scale) in 64 bits, by plain torch operations."""
    k, v = (dev(x).double().view(-1, c.Hkv, c.D) for x in (c.k, c.v))
    q = q.double()
    out, add, big = torch.zeros_like(q), torch.zeros(c.NB * c.bs, c.Hkv, dtype=torch.float64, device="cuda"), 0.0
    for b, n in enumerate(c.lens.tolist()):
        ql = int(cu[b + 1] - cu[b])
        s = torch.from_numpy(c.slots(b)).cuda()
        i = torch.arange(ql, device="cuda").repeat_interleave(G)
        hidden = torch.arange(n, device="cuda")[None] > (n - ql + i)[:, None]
        for h in range(c.Hkv):
            x = q[cu[b]: cu[b + 1], h * G: (h + 1) * G].reshape(ql * G, c.D)
            big = max(big, float((x.abs() @ k[s, h].abs().T).max()) * scale)
            p = torch.softmax((x @ k[s, h].T * scale).masked_fill(hidden, -torch.inf), -1)
            out[cu[b]: cu[b + 1], h * G: (h + 1) * G] = (p @ v[s, h]).view(ql, G, c.D)
            add[s, h] += p.sum(0)
    return out, add.view(c.NB, c.bs, c.Hkv).permute(0, 2, 1).cpu().numpy(), big


@pytest.mark.parametrize("G,Hkv,q_lens,contexts,width", [
    (4, 8, [1300], [4000], 4032),                    # 168 items, 16 of them in a last round of long ones
    (4, 8, [1300], [4000], 40960),
    (2, 8, [1024] * 4, [1024, 1500, 1024, 1030], 40960),  # 256 items, none long enough to be split
    (4, 8, [1024, 600, 300], [1024, 20000, 300], 20032),  # 384 at most, long and short ones in the last round
    (8, 10, [512], [9000], 40960),                   # 160
    (8, 2, [5, 30, 1], [60, 3000, 200], 40960),      # few items: those of short contexts are single pieces
])
@pytest.mark.parametrize("D", [64, 128])
def test_tables_wider_than_the_contexts(pkv, D, G, Hkv, q_lens, contexts, width):
    c = ref.Cache(contexts, 64, Hkv, D, seed=G)
    more = width // 64 - c.tables.shape[1]
    c.tables = np.concatenate([c.tables, np.full((len(contexts), more), -1, c.tables.dtype)], axis=1)
    scale = D ** -0.5
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = dev(ref.to_bf16(np.random.default_rng(1).standard_normal((int(cu[-1]), Hkv * G, D), dtype=np.float32)))
    want_out, add, big = reference(c, q, cu, G, scale)
    want = c.w.astype(np.float64)
    for b in range(len(contexts)):
        s = c.slots(b)[contexts[b] - q_lens[b]:]
        want[s // 64, :, s % 64] = 0.0
    want += add
    k, v, w, t = dev(c.k), dev(c.v), dev(c.w.copy()), dev(c.tables)
    cq, ck = dev(cu), dev(np.concatenate([[0], np.cumsum(c.lens)]).astype(np.int32))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pkv.paged_prefill_weights(q, k, v, t, cq, ck, max(q_lens), scale, torch.empty_like(q), w, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    # the framework's bar for its attention outputs
    assert ((out.double() - want_out).abs() <= 1e-2 + 2.0 ** -8 * want_out.abs()).all()
    ref.check_weights(w.cpu().numpy(), want, add, ref.weight_tolerance(D, big), "wide tables")
