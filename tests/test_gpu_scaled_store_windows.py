"""The store on both sides of the sizes where its windows change: rows of a head (tokens times heads), tokens, block
size."""

import numpy as np
import pytest

import scaled_reference as ref
from test_gpu_scaled_attention import dev, pkv  # noqa: F401 (pkv: fixture)

pytestmark = pytest.mark.gpu


def mixed_slots(rng, N, bs, runs):
    """One token in each block, whole blocks, or pieces that begin and end inside their blocks, padding between."""
    slots, blk = [], 0
    while len(slots) < N:
        first = 0 if runs == "whole" else int(rng.integers(0, bs))
        n = {"one": 1, "whole": bs, "pieces": int(rng.integers(1, bs - first + 1))}[runs]
        slots += range(blk * bs + first, blk * bs + first + n)
        blk += 1
        if runs == "pieces" and rng.random() < 0.1:
            slots += [-1] * int(rng.integers(1, 20))
    slots = np.asarray(slots[:N])
    order = rng.permutation(blk)
    return np.where(slots >= 0, order[slots // bs] * bs + slots % bs, -1), blk


@pytest.mark.parametrize("N,Hkv,bs", [
    (4096, 1, 16), (4097, 1, 16), (2048, 2, 32), (2049, 2, 32), (1365, 3, 16), (1366, 3, 16), (512, 8, 16), (513, 8, 16),
    (256, 16, 32), (257, 16, 32), (512, 1, 48), (513, 1, 48), (512, 8, 256), (512, 9, 256), (600, 2, 256)])
@pytest.mark.parametrize("runs", ["one", "whole", "pieces"])
def test_where_the_windows_change(pkv, N, Hkv, bs, runs):
    rng = np.random.default_rng(N)
    D = 64
    slots, blocks = mixed_slots(rng, N, bs, runs)
    c = [rng.integers(0, 0x7F, (blocks, bs, Hkv, D)).astype(np.uint8) for _ in range(2)]
    s = [np.full((blocks, Hkv), 2.0 ** -6, np.float32) for _ in range(2)]
    t = [dev(x) for x in (*c, *s)]
    k, v = (ref.bf16(rng.standard_normal((N, Hkv, D)) * 2.0 ** (3 * rng.standard_normal((N, Hkv, 1)))) for _ in range(2))
    pkv.store_kvcache_scaled(dev(k), dev(v), *t, dev(slots))
    for x, cc, ss in zip((k, v), c, s):
        ref.store(x, cc, ss, slots)
    for got, want in zip(t, c + s):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
