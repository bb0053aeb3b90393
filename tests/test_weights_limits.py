"""Sizes at the limits of the calls that record attention weights and of the
eviction, without a GPU."""

import ctypes

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
