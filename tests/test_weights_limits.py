"""Sizes at the limits of the calls that record attention weights and of the
eviction, without a GPU."""

import ctypes

import pytest

i32, i64, sz = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t


def test_prefill_weights_workspace_of_nearly_a_round_of_items(cuda_lib_path):
    """102 to 151 items of 256 rows over long contexts are three splits each (152 are not split): the
    largest workspace of an unsplit round is what the header says."""
    f = ctypes.CDLL(cuda_lib_path).pkv_prefill_weights_workspace_bytes
    f.restype, f.argtypes = sz, [i32, i64] + [i32] * 6
    up = lambda n: n + -n % 256
    for items in range(102, 152):
        rows, D = 256 * items, 128  # one sequence of 256 new tokens, a KV head per item
        want = up(rows * 4 + 4) + up(3 * rows * 4) + 3 * rows * D * 4  # (256 rows per head: no partial sums of weights)
        got = f(1, 256, 256, items, items, D, 4096, 16)
        assert got == want and got <= 4 * (D + 2) * 3 * rows
    assert 59e6 < got < 61e6
    assert f(1, 256, 256, 152, 152, 128, 4096, 16) == up(256 * 152 * 4 + 4)
    # rows of q behind the sequences' own are counted too
    assert f(1, 512, 256, 151, 151, 128, 4096, 16) > 118e6


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1, 10 ** 20])
def test_numbers_beyond_a_c_int_are_refused(value):
    """Not cut to their lower 32 bits: an eviction to a budget of 2^32 + 5 would trim to 5 tokens."""
    import paged_kv_cache_85_gb300 as pkv

    with pytest.raises(ValueError, match="budget"):
        pkv.evict_kvcache(None, None, None, None, None, value, 0, None)
    with pytest.raises(ValueError, match="recent"):
        pkv.evict_kvcache(None, None, None, None, None, 10, value, None)
    with pytest.raises(ValueError, match="window"):
        pkv.paged_prefill_weights(None, None, None, None, None, None, 1, 0.1, None, None, window=value)
    with pytest.raises(ValueError, match="max_seqlen_q"):
        pkv.paged_prefill_weights(None, None, None, None, None, None, value, 0.1, None, None)
    for call, scales in ((pkv.paged_attn_decode_weights, ()), (pkv.paged_attn_decode_weights_fp8, (1.0, 1.0))):
        with pytest.raises(ValueError, match="max_ctas"):
            call(None, None, None, None, None, 0.1, *scales, None, None, max_ctas=value)
