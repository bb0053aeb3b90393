"""Prefill over scaled caches in which a block that some rows do not see holds NaN: those rows are as if it did not."""

import numpy as np
import pytest

import scaled_reference as ref
from test_gpu_scaled_attention import host, pkv, queries, run_prefill  # noqa: F401 (pkv: fixture)

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
