"""Which items of a scaled prefill are split over the keys, and that they are right where some of a call are and some
are not."""

import numpy as np
import pytest

import scaled_reference as ref
from test_gpu_scaled_attention import host, pkv, queries, run_prefill  # noqa: F401 (pkv: fixture)


@pytest.fixture(scope="module")
def lib(cuda_lib_path):
    import paged_kv_cache_85_gb300 as m

    m.load_library()
    return m


def pieces(m, B, q, ctx, Hq=32, Hkv=8, D=128, bs=16):
    """Of the call's longest items, by the size of their outputs."""
    n = m.prefill_scaled_workspace_bytes(B, B * q, q, Hq, Hkv, D, -(-ctx // bs), bs)
    rows = B * q * Hq
    if n == 0:
        return 1
    s = n // (rows * (D + 1) * 4)
    assert n == -(-(s * rows * 4) // 256) * 256 + s * rows * D * 4
    return s


@pytest.mark.parametrize("B,q,prefix,want", [
    # fewer items than SMs: 128 items, then 88, 64, 40 and 8 of them
    (1, 1000, 1000, 1), (1, 1000, 16000, 1), (1, 700, 4000, 1), (1, 700, 20000, 3), (1, 512, 512, 1), (1, 512, 1024, 1),
    (1, 512, 2048, 1), (1, 512, 8192, 2), (2, 200, 3000, 2), (1, 300, 8192, 3), (1, 64, 1024, 1), (1, 64, 4096, 8),
    (1, 64, 30000, 19), (1, 1, 40960, 19), (4, 100, 1000, 1),
    # a few rounds of long items
    (1, 1300, 1024, 1), (1, 1300, 28672, 4), (1, 2048, 8192, 1), (1, 2048, 28672, 4), (1, 4096, 16384, 2)])
def test_the_choice(lib, B, q, prefix, want):
    assert pieces(lib, B, q, prefix + q) == want


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens,prefix,Hkv,G,D,bs,mbs_extra", [
    ([40, 40, 40, 40], [0, 900, 2500, 6000], 2, 4, 64, 16, 0),   # long contexts split, short ones not
    ([40, 7, 1], [5000, 30, 5120], 1, 8, 128, 32, 200),           # tables far wider than the contexts
    ([300], [300], 2, 2, 64, 16, 600),                            # ... which are too short
    ([520], [3000], 4, 4, 128, 64, 10),                           # the rows' items differ in length
    ([1, 1, 1, 1, 1], [5000, 4, 4000, 0, 2047], 1, 1, 64, 256, 0)])
def test_some_items_split_and_some_not(pkv, q_lens, prefix, Hkv, G, D, bs, mbs_extra):
    rng = np.random.default_rng(len(q_lens))
    c = ref.Cache(np.add(q_lens, prefix), bs, Hkv, D, seed=5, mbs_extra=mbs_extra)
    assert pkv.prefill_scaled_workspace_bytes(len(q_lens), sum(q_lens), max(q_lens), Hkv * G, Hkv, D, c.MBS, bs) > 0
    q = queries(rng, sum(q_lens) + 3, Hkv * G, D)
    want, mag = ref.prefill(q, c, q_lens, 0.1)
    out = run_prefill(pkv, c, q, q_lens, 0.1)
    n = sum(q_lens)
    ref.check(host(out)[:n], want[:n], mag[:n])
    assert (out[n:] == 7).all()
