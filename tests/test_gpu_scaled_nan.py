"""Prefill over scaled caches in which a block that some rows do not see holds NaN: those rows are as if it did not."""

import numpy as np
import pytest

import scaled_reference as ref
from test_gpu_scaled_attention import dev, host, pkv, queries, run_decode, run_prefill  # noqa: F401 (pkv: fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_lens,prefix,Hkv,G,D,bs,seq,token", [
    ([200], [0], 1, 2, 128, 16, 0, 112),             # inside the first tile
    ([200], [0], 2, 4, 64, 16, 0, 128),              # the first block of the second
    ([30, 300, 5], [7, 90, 0], 2, 1, 64, 32, 1, 320),
    ([700, 40], [100, 0], 1, 8, 128, 64, 0, 448),    # items before and after it
    ([260, 300], [0, 20], 1, 1, 128, 16, 1, 304),    # the last block: the last rows alone see it
    ([300], [6000], 1, 4, 64, 16, 0, 6144),          # items split over the keys
    ([260], [4000], 2, 2, 128, 32, 0, 4096)])
@pytest.mark.parametrize("which", ["ks", "vs", "both"])
def test_a_nan_scale_reaches_the_rows_that_see_its_block(pkv, q_lens, prefix, Hkv, G, D, bs, seq, token, which):
    rng = np.random.default_rng(token)
    c = ref.Cache(np.add(q_lens, prefix), bs, Hkv, D, seed=3)
    q = queries(rng, sum(q_lens), Hkv * G, D)
    want, mag = ref.prefill(q, c, q_lens, 0.1)
    head = Hkv - 1
    for name in ("ks", "vs"):
        if which in (name, "both"):
            getattr(c, name)[c.tables[seq, token // bs], head] = np.nan
    got = host(run_prefill(pkv, c, q, q_lens, 0.1))
    first = sum(q_lens[:seq]) + token // bs * bs - prefix[seq]  # the first row that sees the block
    rows = np.zeros(got.shape, bool)
    rows[first: sum(q_lens[: seq + 1]), head * G: (head + 1) * G] = True
    assert np.isnan(got[rows]).all() and not np.isnan(got[~rows]).any()
    got[rows], want[rows] = 0, 0
    ref.check(got, want, mag)


CODES = [
    ([200], [0], 1, 2, 128, 16, [(0, 119)]),              # inside the first tile
    ([200], [0], 2, 4, 64, 16, [(0, 128), (0, 199)]),     # the first token of the second, and the last of all
    ([30, 300, 5], [7, 90, 0], 2, 1, 64, 32, [(1, 320), (1, 17), (0, 36)]),
    ([700, 400], [100, 0], 1, 8, 128, 64, [(0, 449), (1, 130)]),
    ([2300, 2300], [0, 300], 8, 1, 64, 256, [(0, 1400), (1, 2222)]),
    ([400] * 6, [0, 30] * 3, 4, 8, 64, 32, [(b, t) for b in range(6) for t in (17 * b, 390)]),  # items follow on a CTA
    ([400] * 12, [0] * 12, 2, 8, 128, 16, [(5, 0), (11, 399)]),
    ([300], [6000], 1, 4, 64, 16, [(0, 6150), (0, 6290)]),            # items split over the keys
    ([260], [4000], 2, 2, 128, 32, [(0, 2000)]),
]


@pytest.mark.parametrize("q_lens,prefix,Hkv,G,D,bs,tokens", CODES)
def test_a_nan_in_v_reaches_its_column_of_the_rows_that_see_it(pkv, q_lens, prefix, Hkv, G, D, bs, tokens):
    """A token's V may hold NaN codes (the store keeps NaN): rows from that token on are NaN in those columns, other
    columns and earlier rows are not touched.  Codes of either sign."""
    rng = np.random.default_rng(len(tokens))
    c = ref.Cache(np.add(q_lens, prefix), bs, Hkv, D, seed=3)
    q = queries(rng, sum(q_lens), Hkv * G, D)
    want, mag = ref.prefill(q, c, q_lens, 0.1)
    bad = np.zeros(want.shape, bool)
    for i, (b, t) in enumerate(tokens):
        head, cols = int(rng.integers(0, Hkv)), [int(rng.integers(0, D // 2)), int(rng.integers(D // 2, D)), D - 1][i % 2:]
        slot = c.slots(b)[t]
        c.v[slot // bs, slot % bs, head, cols] = 0x7F if i % 2 == 0 else 0xFF
        start = sum(q_lens[:b])
        rows = np.arange(start + max(0, t - prefix[b]), start + q_lens[b])
        bad[np.ix_(rows, range(head * G, (head + 1) * G), cols)] = True
    got = host(run_prefill(pkv, c, q, q_lens, 0.1))
    assert np.isnan(got[bad]).all()
    assert not np.isnan(got[~bad]).any(), f"{np.argwhere(np.isnan(got) & ~bad)[:5]}"
    got[bad], want[bad] = 0, 0
    ref.check(got, want, mag)


@pytest.mark.parametrize("D,bs", [(128, 16), (64, 256)])
def test_a_nan_that_came_through_the_store(pkv, D, bs):
    """A prompt one of whose tokens has NaN in K, another in V, stored and attended; then a decode step."""
    rng = np.random.default_rng(D)
    n, Hkv, G, in_k, in_v = 290, 2, 2, 250, 70
    NB = -(-n // bs) + 1
    k, v = (ref.bf16(rng.standard_normal((n, Hkv, D))) for _ in range(2))
    v[in_v, 1, [3, D - 2]] = 0x7FC0
    k[in_k, 0, 5] = 0xFFC1
    t = [torch.zeros(NB, bs, Hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    t += [torch.zeros(NB, Hkv, device="cuda") for _ in range(2)]
    tables = rng.permutation(NB)[None, : -(-n // bs)].astype(np.int32)
    at = tables[0, np.arange(n) // bs].astype(np.int64) * bs + np.arange(n) % bs
    pkv.store_kvcache_scaled(dev(k), dev(v), *t, dev(at))
    q = queries(rng, n, Hkv * G, D, 0.3)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    cu = dev(np.array([0, n], np.int32))
    pkv.paged_prefill_scaled(dev(q), *t, dev(tables), cu, cu, n, 0.1, out)
    got = host(out)
    bad = np.zeros(got.shape, bool)
    bad[in_k:, :G] = True
    bad[in_v:, G:, 3] = bad[in_v:, G:, D - 2] = True
    assert np.isnan(got[bad]).all() and not np.isnan(got[~bad]).any()
    # what the cache stands for, NaN taken out, gives the other elements
    x = [s.cpu().numpy()[:, None, :, None] * ref.E4M3[a.cpu().numpy()] for a, s in zip(t[:2], t[2:])]
    K, V = (np.nan_to_num(y.reshape(NB * bs, Hkv, D)[at]) for y in x)
    qf = ref.from_bf16(q)
    for h in range(Hkv):
        for g in range(G):
            w, m = ref.attend(qf[:, h * G + g], K[:, h], V[:, h], 0.1, first=0)
            there = ~bad[:, h * G + g]
            ref.check(got[:, h * G + g][there], w[there], m[there])
    one = torch.empty(1, Hkv * G, D, dtype=torch.bfloat16, device="cuda")
    pkv.paged_attn_decode_scaled(dev(q[-1:]), *t, dev(tables), dev(np.array([n], np.int32)), 0.1, one)
    np.testing.assert_array_equal(np.isnan(host(one)[0]), bad[-1])
