"""Prefill over caches whose blocks' V scales lie far apart inside one tile of keys: a row keeps the values of the
blocks that its weight lies on, whatever the scales of others, seen or not."""

import numpy as np
import pytest

import scaled_reference as ref
from test_gpu_scaled_attention import dev, host, pkv, queries, run_decode, run_prefill  # noqa: F401 (pkv: fixture)

pytestmark = pytest.mark.gpu


def one_block_per_row(q_len, prefix, bs, D, seed):
    """Row i's weight lies on one block of the prefix: K is 448 in dimension i % D of that block and 0 elsewhere, the
    row is 1 in that dimension, so that every other weight is exp(-448).  Returns the cache, the rows and which
    block each looks at."""
    rng = np.random.default_rng(seed)
    c = ref.Cache([prefix + q_len], bs, 1, D, seed=seed)
    n = prefix // bs
    at = rng.permutation(n)[: min(n, D)]  # the block of each dimension
    c.k[:] = 0
    c.ks[:] = 1.0
    for d, blk in enumerate(at):
        c.k[c.tables[0, blk], :, 0, d] = 0x7E  # 448
    dims = np.arange(q_len) % len(at)
    q = np.zeros((q_len, 1, D), np.uint16)
    q[np.arange(q_len), 0, dims] = ref.bf16(1.0)
    return c, q, at[dims], rng


@pytest.mark.parametrize("q_len,prefix,bs,D", [
    (40, 640, 16, 64), (64, 1024, 16, 128), (33, 1500, 32, 128), (300, 2000, 64, 64), (200, 5000, 16, 128)])
@pytest.mark.parametrize("gap,factor", [(12, 1.0), (17, 1.0), (25, 1.0), (26, 1.3), (40, 1.0), (70, 0.7)])
def test_all_weight_on_a_block_of_small_scale(pkv, q_len, prefix, bs, D, gap, factor):
    """Every second block's scale is 2^gap below the others'."""
    c, q, look, _ = one_block_per_row(q_len, prefix, bs, D, seed=gap)
    high = min(gap // 2, 35)
    blocks = c.tables[0, : -(-int(c.lens[0]) // bs)]
    c.vs[blocks, 0] = 2.0 ** high
    c.vs[blocks[1::2], 0] = factor * 2.0 ** (high - gap)
    want, mag = ref.prefill(q, c, [q_len], 1.0)
    assert (np.abs(want[look % 2 == 1]).max(-1) > 0).all()
    ref.check(host(run_prefill(pkv, c, q, [q_len], 1.0)), want, mag)
    # and what decode gives for the last row
    c.lens[0] = prefix + q_len
    last, mag = ref.decode(q[-1:], c, 1.0)
    ref.check(host(run_decode(pkv, c, q[-1:], 1.0)), last, mag)


@pytest.mark.parametrize("bs,D", [(16, 64), (16, 128), (32, 128), (64, 64)])
@pytest.mark.parametrize("seed", range(3))
def test_scales_over_the_whole_range(pkv, bs, D, seed):
    """Any scale in [2^-40, 2^40] beside any other, a tenth of them zero."""
    c, q, _, rng = one_block_per_row(100, 3000, bs, D, seed=seed)
    c.vs[:, 0] = 2.0 ** rng.integers(-40, 41, c.NB) * rng.choice([1.0, 1.0, 0.83], c.NB)
    c.vs[rng.random(c.NB) < 0.1, 0] = 0
    want, mag = ref.prefill(q, c, [100], 1.0)
    # rows that look at a block of zeros: what is left, exp(-448) of other blocks, is below bf16's least number, 2^-133
    assert (np.abs(want[np.abs(want) < 2.0 ** -133]) < 2.0 ** -500).all()
    want[np.abs(want) < 2.0 ** -133] = 0
    ref.check(host(run_prefill(pkv, c, q, [100], 1.0)), want, mag)


@pytest.mark.parametrize("bs,D,G", [(16, 64, 1), (16, 128, 4), (32, 128, 2), (64, 64, 8)])
@pytest.mark.parametrize("low,high", [(-20, 3), (-20, 25), (-40, 40), (0, 20)])
def test_later_blocks_of_large_scale(pkv, bs, D, G, low, high):
    """Blocks that a row does not see are of scales far above all that it does, in its tile and behind earlier ones."""
    rng = np.random.default_rng(bs)
    q_lens, prefix = [128, 120, 300], [0, 128, 16]
    c = ref.Cache(np.add(q_lens, prefix), bs, 1, D, seed=3)
    first = (64, 192, 192)  # tokens from here on are large: inside the first, second and second tile
    for b in range(3):
        t = c.tables[b, : -(-int(c.lens[b]) // bs)]
        c.vs[t, 0] = 2.0 ** (low + rng.integers(0, 3, len(t)))
        c.vs[t[first[b] // bs:], 0] = 2.0 ** (high - rng.integers(0, 3, len(t) - first[b] // bs))
    q = queries(rng, sum(q_lens), G, D)
    want, mag = ref.prefill(q, c, q_lens, 0.1)
    ref.check(host(run_prefill(pkv, c, q, q_lens, 0.1)), want, mag)


@pytest.mark.parametrize("bs,D", [(16, 128), (32, 64)])
@pytest.mark.parametrize("gap", [5, 9, 13])
def test_columns_that_only_blocks_of_small_scale_fill(pkv, bs, D, gap):
    """Equal weights; in half of the columns the blocks of large scale are zero.  Within 2^13 a small block's weights
    keep 2^-24 of the largest weight, so each column holds against its own sum."""
    rng = np.random.default_rng(gap)
    q_lens, prefix = [90, 5], [700, 100]
    c = ref.Cache(np.add(q_lens, prefix), bs, 1, D, seed=gap)
    for b in range(2):
        t = c.tables[b, : -(-int(c.lens[b]) // bs)]
        tile = 2.0 ** np.repeat(rng.integers(-12, 12, len(t)), 128 // bs)[: len(t)]
        large = rng.random(len(t)) < 0.5
        c.vs[t, 0] = tile * np.where(large, 1.0, 2.0 ** -gap)
        own = c.v[t[large]]
        own[..., : D // 2] = 0
        c.v[t[large]] = own
    q = queries(rng, 95, 2, D)
    want, mag = ref.prefill(q, c, q_lens, 0.05)
    got = host(run_prefill(pkv, c, q, q_lens, 0.05))
    at = 0
    for n in q_lens:
        ref.check(got[at: at + n], want[at: at + n], mag[at: at + n])
        at += n
