"""Scaled caches with everything at once: V scales over the whole range, zeros and NaN among them, NaN codes in K and V,
blocks that are not there, on ragged batches, whole and split."""

import numpy as np
import pytest

import scaled_reference as ref
from test_gpu_scaled_attention import host, pkv, queries, run_decode, run_prefill  # noqa: F401 (pkv: fixture)

pytestmark = pytest.mark.gpu


def spoil(c, rng, far):
    """Per sequence a few of each, at blocks and tokens of their own.  Returns the tables as given to the call."""
    tables = c.tables.copy()
    blocks = -(-c.lens // c.bs)
    for b in range(len(c.lens)):
        n = int(blocks[b])
        if far:
            c.vs[c.tables[b, :n]] = 2.0 ** rng.integers(-40, 41, (n, c.Hkv))
        for scales, value, share in ((c.vs, 0, 0.1), (c.ks, 0, 0.1), (c.vs, np.nan, 0.02), (c.ks, np.nan, 0.02)):
            hit = rng.random((n, c.Hkv)) < share
            own = scales[c.tables[b, :n]]
            own[hit] = value
            scales[c.tables[b, :n]] = own
        at = c.slots(b)
        for codes in (c.k, c.v):
            if rng.random() < 0.5 and len(at):
                s = at[int(rng.integers(len(at)))]
                codes[s // c.bs, s % c.bs, int(rng.integers(c.Hkv)), int(rng.integers(c.D))] = 0xFF
        if n and rng.random() < 0.5:
            tables[b, int(rng.integers(n))] = c.NB + 3  # not there: its tokens are left out
    return tables


def expected(c, tables, q, q_lens, scale):
    """(out, weighted |V|, NaN or not), the elements that are NaN set to 0."""
    Hq = q.shape[1]
    G = Hq // c.Hkv
    out, mag, nan = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape, bool)
    qf = ref.from_bf16(q)
    at = 0
    for b, n in enumerate(q_lens):
        m = int(c.lens[b])
        there = (tables[b, np.arange(m) // c.bs] < c.NB)
        pos = np.arange(m)[there]
        K, V = c.rows(b, "k")[there], c.rows(b, "v")[there]
        blk = c.slots(b)[there] // c.bs
        for i in range(n):
            seen = pos <= m - n + i
            if not seen.any():
                continue
            for h in range(c.Hkv):
                k, v = K[seen, h], V[seen, h]
                rows = slice(h * G, (h + 1) * G)
                if np.isnan(k).any() or np.isnan(c.vs[blk[seen], h]).any():
                    nan[at + i, rows] = True
                    continue
                cols = np.isnan(v).any(0)
                nan[at + i, rows] = cols
                o, w = ref.attend(qf[at + i, rows], k, np.nan_to_num(v), scale)
                out[at + i, rows], mag[at + i, rows] = np.where(cols, 0, o), w
        at += n
    return out, mag, nan


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("q_lens,prefix,Hkv,G,D,bs", [
    ([90, 1, 150, 33], [0, 200, 60, 7], 2, 2, 64, 16),
    ([260, 40, 5], [10, 300, 120], 1, 4, 128, 32),
    ([60, 17], [2600, 1900], 2, 1, 128, 16),  # split over the keys
    ([130, 140, 20], [0, 128, 500], 1, 8, 64, 128)])
@pytest.mark.parametrize("seed", range(4))
def test_everything_at_once(pkv, q_lens, prefix, Hkv, G, D, bs, far, seed):
    rng = np.random.default_rng(seed)
    c = ref.Cache(np.add(q_lens, prefix), bs, Hkv, D, seed=seed)
    tables = spoil(c, rng, far)
    scale = 0.1 if seed % 2 else -0.1
    q = queries(rng, sum(q_lens) + 2, Hkv * G, D)
    want, mag, nan = expected(c, tables, q, q_lens, scale)
    missing = (tables >= c.NB).any()
    c.tables = tables
    out = run_prefill(pkv, c, q, q_lens, scale, flag=pkv.FLAG_BAD_BLOCK if missing else 0)
    n = sum(q_lens)
    assert (out[n:] == 7).all()
    got = host(out)[:n]
    np.testing.assert_array_equal(np.isnan(got), nan[:n])
    got[nan[:n]] = 0
    want[nan], mag[nan] = 0, 0
    ref.check(got, want[:n], mag[:n])


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("Hkv,G,D,bs", [(2, 2, 64, 16), (1, 4, 128, 32), (3, 1, 128, 16), (1, 8, 64, 128)])
@pytest.mark.parametrize("seed", range(3))
def test_a_decode_step_over_them(pkv, Hkv, G, D, bs, far, seed):
    rng = np.random.default_rng(seed)
    lens = [90, 1, 300, 33, 2600, 17, 128, 1025]
    c = ref.Cache(lens, bs, Hkv, D, seed=seed)
    tables = spoil(c, rng, far)
    q = queries(rng, len(lens), Hkv * G, D)
    want, mag, nan = expected(c, tables, q, [1] * len(lens), 0.1)
    missing = (tables >= c.NB).any()
    c.tables = tables
    for max_ctas in (0, 3):
        got = host(run_decode(pkv, c, q, 0.1, flag=pkv.FLAG_BAD_BLOCK if missing else 0, max_ctas=max_ctas))
        np.testing.assert_array_equal(np.isnan(got), nan)
        got[nan] = 0
        ref.check(got, np.where(nan, 0, want), np.where(nan, 0, mag))
