"""Copies of blocks in every tensor under their ids, byte for byte."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv(cuda_lib_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_85_gb300 as m

    m.load_library()
    return m


def tensors(NB, kind, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    make = lambda shape, dtype: torch.randint(-(2 ** 31), 2 ** 31 - 1, (NB, -(-int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size() // 4)),
                                              generator=g, device="cuda", dtype=torch.int32).view(torch.uint8)[:, : int(np.prod(shape)) * torch.empty(
                                                  0, dtype=dtype).element_size()].contiguous().view(dtype).view(NB, *shape)
    return [make(s, d) for s, d in {
        "scaled": [((16, 8, 128), torch.uint8)] * 2 + [((8,), torch.float32)] * 2,
        "one head": [((32, 1, 64), torch.uint8)] * 2 + [((1,), torch.float32)] * 2,
        "bf16": [((48, 3, 64), torch.bfloat16)] * 2,
        "weights": [((256, 2, 128), torch.bfloat16)] * 2 + [((2, 256), torch.float32)],
        "odd": [((3,), torch.bfloat16), ((5,), torch.uint8), ((1237,), torch.uint8), ((7, 3), torch.float32), ((4099,), torch.bfloat16)],
        "layers": [((16, 2, 64), torch.uint8)] * 100 + [((2,), torch.float32)] * 51,
    }[kind]]


@pytest.mark.parametrize("kind", ["scaled", "one head", "bf16", "weights", "odd", "layers"])
@pytest.mark.parametrize("n", [1, 9, 60])
def test_copies(pkv, kind, n):
    NB = 2 * n + 5
    rng = np.random.default_rng(n)
    ts = tensors(NB, kind)
    perm = rng.permutation(NB)
    src = perm[n + rng.integers(0, n, n)]  # several destinations of one source
    pairs = np.stack([src, perm[:n]], 1)
    pairs = np.concatenate([pairs, [[-1, -1], [perm[-1], perm[-1]], [-1, -1]]])[rng.permutation(n + 3)].astype(np.int32)
    want = [t.clone() for t in ts]
    for a, b in pairs.tolist():
        if a >= 0:
            for t in want:
                t[b] = t[a]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.copy_blocks(ts, torch.from_numpy(pairs).cuda(), err_flag=err)
    assert int(err.item()) == 0
    for t, w in zip(ts, want):
        assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))


def test_bad_ids_are_skipped(pkv):
    for bad in ([-1, 3], [3, -1], [20, 1], [1, 20], [-2, -2], [2 ** 31 - 1, 0]):
        ts = tensors(20, "scaled", 3)
        want = [t.clone() for t in ts]
        for t in want:
            t[5] = t[4]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkv.copy_blocks(ts, torch.tensor([bad, [4, 5]], dtype=torch.int32, device="cuda"), err_flag=err)
        assert int(err.item()) == pkv.FLAG_BAD_BLOCK
        for t, w in zip(ts, want):
            assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))


def test_nothing_to_copy_and_refusals(pkv):
    ts = tensors(4, "scaled")
    none = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    pair = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    pkv.copy_blocks(ts, none)
    with pytest.raises(ValueError, match="no tensors"):
        pkv.copy_blocks([], pair)
    with pytest.raises(TypeError):
        pkv.copy_blocks([ts[0], 3], pair)
    with pytest.raises(ValueError, match="blocks"):
        pkv.copy_blocks([ts[0], ts[1][:2]], pair)
    with pytest.raises(ValueError, match="contiguous"):
        pkv.copy_blocks([ts[0][:, ::2]], pair)
    with pytest.raises(ValueError, match="pairs"):
        pkv.copy_blocks(ts, pair.long())
    with pytest.raises(ValueError, match="pairs"):
        pkv.copy_blocks(ts, torch.zeros((1, 3), dtype=torch.int32, device="cuda"))
    with pytest.raises(pkv.PkvError, match="same memory"):
        pkv.copy_blocks([ts[0], ts[0]], pair)


def test_blocks_beyond_4_gb(pkv):
    """Offsets past 32 bits."""
    big = torch.empty((9, 600 << 20), dtype=torch.uint8, device="cuda")
    big[1], big[8] = 7, 3
    big[1, -5:] = 9
    pkv.copy_blocks([big], torch.tensor([[1, 8], [8, 0]][:1], dtype=torch.int32, device="cuda"))
    assert torch.equal(big[8], big[1])


def test_captured(pkv):
    ts = tensors(12, "scaled", 5)
    pairs = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pkv.copy_blocks(ts, pairs)
    want = [t.clone() for t in ts]
    torch.cuda.synchronize()
    for a, b in ((3, 4), (4, 9), (0, 11)):
        with torch.cuda.stream(s):
            pairs[1] = torch.tensor([a, b], dtype=torch.int32, device="cuda")
            g.replay()
        for t in want:
            t[b] = t[a]
    torch.cuda.synchronize()
    for t, w in zip(ts, want):
        assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))
