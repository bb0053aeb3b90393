"""Blocks that are new to one sequence of a recording call and already part of
another one's context in the same call: their weights start from zero and
receive every sequence's addition, whatever the order of the sequences."""

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


def fill(c, seed, stale=None):
    """Every slot of the cache finite (sequences share blocks whose tails only some of them use)."""
    rng = np.random.default_rng(seed)
    c.k, c.v = (c._draw(rng, c.k.shape) for _ in range(2))
    c.w = rng.exponential(size=c.w.shape).astype(np.float32)
    if stale is not None:
        for b, first in stale:
            s = c.slots(b)[first:]
            c.w[s // c.bs, :, s % c.bs] = np.nan


def expected(c, add, new):
    """Weights after a call that adds `add`: the slots of the new tokens, (sequence, first new position), start from 0."""
    w = c.w.astype(np.float64)
    for b, first in new:
        s = c.slots(b)[first:]
        w[s // c.bs, :, s % c.bs] = 0.0
    return w + add


def check_prompt(pkv, c, q_lens, G, window, new, repeats=3):
    Tq, cu = int(np.sum(q_lens)), np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    scale = c.D ** -0.5
    qb = ref.to_bf16(1.5 * np.random.default_rng(5).standard_normal((Tq, c.Hkv * G, c.D), dtype=np.float32))
    want_out, _, add, big = ref.prompt(c, ref.from_bf16(qb), cu, scale, window)
    want = expected(c, add, new)
    q, k, v, t = dev(qb), dev(c.k), dev(c.v), dev(c.tables)
    cq, ck = dev(cu), dev(np.concatenate([[0], np.cumsum(c.lens)]).astype(np.int32))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(repeats):
        w, out = dev(c.w.copy()), torch.empty_like(q)
        pkv.paged_prefill_weights(q, k, v, t, cq, ck, int(max(q_lens)), scale, out, w, window=window, err_flag=err)
        got = out.float().cpu().numpy().astype(np.float64)
        # the framework's bar for its attention outputs
        assert (np.abs(got - want_out) <= 1e-2 + 2.0 ** -8 * np.abs(want_out)).all()
        ref.check_weights(w.cpu().numpy(), want, add, ref.weight_tolerance(c.D, big), "shared prefix")
    assert int(err.item()) == 0


@pytest.mark.parametrize("order", [(0, 1, 2, 3), (3, 2, 1, 0), (1, 0, 3, 2)])
@pytest.mark.parametrize("window", [0, 5])
@pytest.mark.parametrize("D,G", [(64, 2), (128, 8)])
@pytest.mark.parametrize("stale", [False, True])
def test_prompts_with_a_common_prefix_in_one_step(pkv, order, window, D, G, stale):
    """The allocator lets a prompt reuse the full blocks of one that is stored in the same step."""
    from paged_kv_cache_85_gb300.block_manager import BlockManager

    bs, Hkv = 16, 2
    rng = np.random.default_rng(1)
    base = rng.integers(0, 1000, 150)
    prompts = [base[:70], np.concatenate([base[:64], rng.integers(1000, 2000, 41)]), rng.integers(2000, 3000, 33), base]
    bm = BlockManager(40, bs)
    cached = [bm.allocate(i, p) for i, p in enumerate(prompts)]
    assert cached == [0, 64, 0, 64]
    lens = np.array([len(prompts[i]) for i in order])
    q_lens = [len(prompts[i]) - cached[i] for i in order]
    c = ref.Cache(lens, bs, Hkv, D, extra_blocks=40)
    c.tables, ctx, _ = bm.decode_batch(list(order), c.MBS)
    np.testing.assert_array_equal(ctx, c.lens)
    new = [(b, int(lens[b]) - q_lens[b]) for b in range(4)]
    fill(c, 3, stale=new if stale else None)
    check_prompt(pkv, c, q_lens, G, window, new)


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("window", [0, 200])
def test_long_common_prefix_in_one_step(pkv, first, window):
    """The owner's prompt is long enough that its query tiles, and the sharers' keys, are split over CTAs."""
    c = ref.Cache([1100, 1107, 1100, 1300], 32, 1, 64, seed=4)
    c.tables[1, :34] = c.tables[0, :34]
    c.tables[2] = c.tables[0]                # every block: its last token is new to both
    c.tables[3, :20] = c.tables[0, :20]
    q_lens = [1100, 19, 1, 5]
    if first:
        c.tables, c.lens, q_lens = c.tables[::-1].copy(), c.lens[::-1].copy(), q_lens[::-1]
    new = [(b, int(c.lens[b]) - q_lens[b]) for b in range(4)]
    fill(c, 6, stale=new)
    check_prompt(pkv, c, q_lens, 8, window, new)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("backwards", [False, True])
@pytest.mark.parametrize("D,G,bs,lens", [(64, 2, 16, [50, 50, 130, 40, 51]), (128, 4, 32, [3001, 3001, 3400, 97, 3002]), (64, 8, 48, [48, 48, 49, 1, 97])])
def test_decode_of_a_sequence_whose_newest_token_another_one_sees(pkv, fp8, backwards, D, G, bs, lens):
    """A step that holds a sequence twice, and sequences that go on from its newest token: each adds to the shared
    blocks, the newest token's included, over stale NaN weights."""
    c = ref.Cache(lens, bs, 2, D, fp8=fp8, seed=2)
    n = -(-lens[0] // bs)
    for b in (1, 2, 4):
        c.tables[b, :n] = c.tables[0, :n]
    if backwards:
        c.tables, c.lens = c.tables[::-1].copy(), c.lens[::-1].copy()
    new = [(b, int(c.lens[b]) - 1) for b in range(5)]
    fill(c, 8, stale=new)
    scale = D ** -0.5
    qb = ref.to_bf16(1.5 * np.random.default_rng(5).standard_normal((5, 2 * G, D), dtype=np.float32))
    _, _, add, big = ref.decode(c, ref.from_bf16(qb), scale)
    want = expected(c, add, new)
    q, k, v, t, ctx = dev(qb), dev(c.k), dev(c.v), dev(c.tables), dev(c.lens)
    scales = (c.k_scale, c.v_scale) if fp8 else ()
    call = pkv.paged_attn_decode_weights_fp8 if fp8 else pkv.paged_attn_decode_weights
    plain = pkv.paged_attn_decode_fp8 if fp8 else pkv.paged_attn_decode
    for _ in range(3):
        w = dev(c.w.copy())
        out = call(q, k, v, t, ctx, scale, *scales, torch.empty_like(q), w)
        assert torch.equal(out, plain(q, k, v, t, ctx, scale, *scales, torch.empty_like(q)))
        ref.check_weights(w.cpu().numpy(), want, add, ref.weight_tolerance(D, big), "shared blocks")
