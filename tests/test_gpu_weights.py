"""Attention that records the weight every cached token received, and the
eviction by it, against plain 64-bit forms (budget_reference.py)."""

import numpy as np
import pytest

import budget_reference as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

FLAG_BAD_BLOCK, FLAG_BAD_CONTEXT_LEN = 0x2, 0x4


@pytest.fixture(scope="module")
def pkv(cuda_lib_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_85_gb300 as m

    m.load_library()
    return m


def bf(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def dev_cache(x):
    return bf(x) if x.dtype == np.uint16 else torch.from_numpy(x).cuda()


def host_cache(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy()


class Dev:
    """A Cache on the GPU."""

    def __init__(self, c):
        self.c = c
        self.k, self.v = dev_cache(c.k), dev_cache(c.v)
        self.w = torch.from_numpy(c.w.copy()).cuda()
        self.tables = torch.from_numpy(c.tables).cuda()
        self.lens = torch.from_numpy(c.lens).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def decode(self, pkv, q, scale, out, **kw):
        if self.c.fp8:
            return pkv.paged_attn_decode_weights_fp8(q, self.k, self.v, self.tables, self.lens, scale, self.c.k_scale,
                                                     self.c.v_scale, out, self.w, err_flag=self.err, **kw)
        return pkv.paged_attn_decode_weights(q, self.k, self.v, self.tables, self.lens, scale, out, self.w,
                                             err_flag=self.err, **kw)

    def plain(self, pkv, q, scale, out, **kw):
        if self.c.fp8:
            return pkv.paged_attn_decode_fp8(q, self.k, self.v, self.tables, self.lens, scale, self.c.k_scale,
                                             self.c.v_scale, out, **kw)
        return pkv.paged_attn_decode(q, self.k, self.v, self.tables, self.lens, scale, out, **kw)


def queries(n, Hq, D, seed, gain=1.5):
    return ref.to_bf16(gain * np.random.default_rng(seed).standard_normal((n, Hq, D), dtype=np.float32))


def check_decode(pkv, c, G, seed=0, max_ctas=0, scale=None, expect=0):
    scale = 1 / np.sqrt(c.D) if scale is None else scale
    qb = queries(len(c.lens), c.Hkv * G, c.D, seed)
    q, d = bf(qb), Dev(c)
    out, plain = torch.empty_like(q), torch.empty_like(q)
    d.decode(pkv, q, scale, out, max_ctas=max_ctas)
    d.plain(pkv, q, scale, plain, max_ctas=max_ctas)
    torch.cuda.synchronize()
    assert int(d.err.item()) == expect
    assert torch.equal(out, plain), "recording changed the attention's output"
    want, w, add, big = ref.decode(c, ref.from_bf16(qb), scale)
    got = out.float().cpu().numpy().astype(np.float64)
    # the framework's bar for its attention outputs, relative for FP8 values above 1
    assert (np.abs(got - want) <= 1e-2 + 2.0 ** -8 * np.abs(want)).all()
    ref.check_weights(d.w.cpu().numpy(), w, add, ref.weight_tolerance(c.D, big), "decode")
    return d


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_decode_weights_shapes(pkv, fp8, D, G):
    """Lengths of zero, one, around a box, a 32-token box and a block; every group size."""
    for bs in (16, 32, 48):
        c = ref.Cache([0, 1, 15, 16, 17, 31, 33, 47, 49, 95, 96, 97, 300], bs, 3, D, fp8=fp8, seed=bs + G, mbs_extra=1)
        check_decode(pkv, c, G, seed=G)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("max_ctas", [0, 1, 3, 40])
def test_decode_weights_long_contexts_split_over_workers(pkv, fp8, max_ctas):
    c = ref.Cache([5000, 1, 333, 0, 2049], 256, 2, 128, fp8=fp8, seed=max_ctas)
    check_decode(pkv, c, 4, max_ctas=max_ctas)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_weights_large_batch(pkv, fp8):
    """Many sequences: larger shared-memory layouts, 32-token boxes for FP8."""
    lens = np.random.default_rng(1).integers(0, 70, size=900)
    check_decode(pkv, ref.Cache(lens, 32, 2, 64, fp8=fp8, seed=7), 2)
    check_decode(pkv, ref.Cache(lens[:300], 32, 1, 128, fp8=fp8, seed=8), 8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0])
def test_decode_weights_scales(pkv, fp8, scale):
    """All weights equal, a negative scale, and a scale that leaves one heavy token."""
    check_decode(pkv, ref.Cache([1, 40, 500], 16, 2, 128, fp8=fp8, seed=3), 2, scale=scale)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_weights_all_empty(pkv, fp8):
    c = ref.Cache([0, 0, 0], 16, 2, 64, fp8=fp8, seed=0, mbs_extra=2)
    d = check_decode(pkv, c, 2)
    assert np.array_equal(d.w.cpu().numpy(), c.w, equal_nan=True)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_weights_bad_block_gets_none(pkv, fp8):
    c = ref.Cache([200, 64, 100], 32, 2, 128, fp8=fp8, seed=5)
    c.tables[0, 2] = c.NB + 3   # in the middle
    c.tables[1, 1] = -1         # the newest token's block
    check_decode(pkv, c, 2, expect=FLAG_BAD_BLOCK)


def test_decode_weights_bad_length_is_clamped(pkv):
    c = ref.Cache([64, 64], 32, 2, 64, seed=5)
    d = Dev(c)
    d.lens[1] = 1000
    qb = queries(2, 4, 64, 0)
    q = bf(qb)
    d.decode(pkv, q, 0.125, torch.empty_like(q))
    assert int(d.err.item()) == FLAG_BAD_CONTEXT_LEN
    _, w, add, big = ref.decode(c, ref.from_bf16(qb), 0.125)  # 64 = the table's 2 blocks of 32
    ref.check_weights(d.w.cpu().numpy(), w, add, ref.weight_tolerance(64, big))


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_weights_shared_prefix_blocks(pkv, fp8):
    """Sequences that share prefix blocks all add to them."""
    c = ref.Cache([300] * 6, 32, 2, 128, fp8=fp8, seed=9)
    c.tables[:, :4] = c.tables[0, :4]
    check_decode(pkv, c, 4)


def test_decode_weights_accumulate_over_steps(pkv):
    """Two steps on the same slots: the second adds, except on the newest token."""
    c = ref.Cache([50, 260], 16, 2, 64, seed=2)
    d = Dev(c)
    for step in range(2):
        qb = queries(2, 4, 64, step)
        q = bf(qb)
        d.decode(pkv, q, 0.125, torch.empty_like(q))
        _, w, add, big = ref.decode(c, ref.from_bf16(qb), 0.125)
        got = d.w.cpu().numpy()
        ref.check_weights(got, w, add, ref.weight_tolerance(64, big), f"step {step}")
        c.w = got


def test_decode_weights_repeat_bit_for_bit(pkv):
    c = ref.Cache(np.random.default_rng(0).integers(1, 3000, size=40), 16, 8, 128, seed=4)
    q = bf(queries(40, 16, 128, 1))
    got = []
    for _ in range(3):
        d = Dev(c)
        d.decode(pkv, q, 0.09, torch.empty_like(q))
        got.append(d.w.view(torch.int32))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [20, 3000])
def test_decode_weights_nan_key_stays_with_its_sequence_and_head(pkv, fp8, n):
    """A NaN among a sequence's keys makes the weights of that sequence and KV head NaN, and no others (with the
    context read by one worker, and split over many)."""
    c = ref.Cache([n, 40], 16, 2, 64, fp8=fp8, seed=1)
    qb = queries(2, 4, 64, 0)
    _, w, add, big = ref.decode(c, ref.from_bf16(qb), 0.125)
    s = c.slots(0)
    c.k.reshape(-1, 2, 64)[s[n // 2], 1, 3] = 0x7F if fp8 else 0x7FC0
    d, q = Dev(c), bf(qb)
    d.decode(pkv, q, 0.125, torch.empty_like(q))
    got = d.w.cpu().numpy()
    assert np.isnan(got[s // 16, 1, s % 16]).all()
    got[s // 16, 1, s % 16], w[s // 16, 1, s % 16] = 0, 0
    add[s // 16, 1, s % 16] = 0
    ref.check_weights(got, w, add, ref.weight_tolerance(64, big))


# ------------------------------------------------------------------ prefill


def check_prompt(pkv, c, q_lens, G, window=0, seed=0, scale=None, expect=0, pad_rows=0, max_q=None):
    scale = 1 / np.sqrt(c.D) if scale is None else scale
    cu_q = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    cu_k = np.concatenate([[0], np.cumsum(c.lens)]).astype(np.int32)
    qb = queries(int(cu_q[-1]) + pad_rows, c.Hkv * G, c.D, seed)
    q, d = bf(qb), Dev(c)
    if pad_rows:
        q[-pad_rows:] = float("nan")
    out = torch.full_like(q, 7.0)
    cq, ck = torch.from_numpy(cu_q).cuda(), torch.from_numpy(cu_k).cuda()
    most = int(max(q_lens)) if max_q is None else max_q
    pkv.paged_prefill_weights(q, d.k, d.v, d.tables, cq, ck, most, scale, out, d.w, window=window, err_flag=d.err)
    torch.cuda.synchronize()
    assert int(d.err.item()) == expect
    want, w, add, big = ref.prompt(c, ref.from_bf16(qb), cu_q, scale, window)
    if pad_rows:
        assert (out[-pad_rows:] == 7.0).all(), "rows behind the last sequence were written"
        out, want = out[:-pad_rows], want[:-pad_rows]
    got = out.float().cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= 1e-2 + 2.0 ** -8 * np.abs(want)).all()
    ref.check_weights(d.w.cpu().numpy(), w, add, ref.weight_tolerance(c.D, big), "prefill")
    return d


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("window", [0, 1, 5, 64])
def test_prompt_weights_shapes(pkv, D, G, window):
    """Chunks of 1 to 150 tokens after prefixes of none to 200, odd lengths, small blocks."""
    q_lens = [1, 7, 16, 65, 150, 3, 130]
    prefix = [0, 33, 128, 1, 0, 200, 127]
    for bs in (16, 48, 64):
        c = ref.Cache(np.add(q_lens, prefix), bs, 2, D, seed=bs + G, mbs_extra=1)
        check_prompt(pkv, c, q_lens, G, window, seed=G, pad_rows=3)


def test_prompt_weights_long(pkv):
    """More than one tile of everything: long prefix, long chunk."""
    check_prompt(pkv, ref.Cache([1500, 700], 256, 2, 128, seed=1), [600, 700], 2)
    check_prompt(pkv, ref.Cache([1500, 700], 16, 1, 64, seed=2), [600, 700], 8, window=33)


def test_prompt_weights_empty_sequences_and_loose_bound(pkv):
    c = ref.Cache([40, 64, 0, 90], 16, 2, 64, seed=3)
    check_prompt(pkv, c, [5, 0, 0, 90], 2, max_q=500)


@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0])
def test_prompt_weights_scales(pkv, scale):
    check_prompt(pkv, ref.Cache([100, 260], 16, 2, 128, seed=3), [50, 200], 2, scale=scale)


def test_prompt_weights_bad_block_gets_none(pkv):
    c = ref.Cache([200, 64, 100], 32, 2, 128, seed=5)
    c.tables[0, 2] = c.NB + 3
    c.tables[1, 0] = -1      # the first tokens: their queries see nothing at all
    check_prompt(pkv, c, [100, 64, 100], 2, expect=FLAG_BAD_BLOCK)


def test_prompt_weights_bad_lengths_record_nothing(pkv):
    """A sequence with more new tokens than context is skipped, the others are not."""
    c = ref.Cache([50, 60, 70], 16, 2, 64, seed=6)
    d = Dev(c)
    cu_q = torch.tensor([0, 20, 100, 130], dtype=torch.int32, device="cuda")  # 80 new tokens > 60
    cu_k = torch.tensor([0, 50, 110, 180], dtype=torch.int32, device="cuda")
    qb = queries(130, 4, 64, 0)
    q = bf(qb)
    pkv.paged_prefill_weights(q, d.k, d.v, d.tables, cu_q, cu_k, 100, 0.125, torch.zeros_like(q), d.w, err_flag=d.err)
    assert int(d.err.item()) == FLAG_BAD_CONTEXT_LEN
    ok = ref.Cache([50, 60, 70], 16, 2, 64, seed=6)
    ok.lens = np.array([50, 0, 70], dtype=np.int32)
    qs = np.concatenate([ref.from_bf16(qb)[:20], ref.from_bf16(qb)[100:]])
    _, w, add, big = ref.prompt(ok, qs, np.array([0, 20, 20, 50]), 0.125)
    ref.check_weights(d.w.cpu().numpy(), w, add, ref.weight_tolerance(64, big))


def test_prompt_weights_neighbour_nan_stays_out(pkv):
    """NaN queries of one sequence do not reach the weights of its neighbours."""
    c = ref.Cache([30, 45, 77], 16, 2, 64, seed=8)
    d = Dev(c)
    cu = torch.tensor([0, 30, 75, 152], dtype=torch.int32, device="cuda")
    qb = queries(152, 4, 64, 0)
    q = bf(qb)
    q[30:75] = float("nan")
    pkv.paged_prefill_weights(q, d.k, d.v, d.tables, cu, cu, 77, 0.125, torch.zeros_like(q), d.w, err_flag=d.err)
    got = d.w.cpu().numpy()
    _, w, add, big = ref.prompt(c, ref.from_bf16(qb), cu.cpu().numpy(), 0.125)
    for b in (0, 2):
        s = c.slots(b)
        pick = np.zeros_like(c.w, dtype=bool)
        pick[s // 16, :, s % 16] = True
        ref.check_weights(np.where(pick, got, 0), np.where(pick, w, 0), np.where(pick, add, 0),
                          ref.weight_tolerance(64, big), f"sequence {b}")


@pytest.mark.parametrize("D,G,Hkv", [(64, 1, 1), (128, 4, 2), (64, 8, 1)])
@pytest.mark.parametrize("q_lens,contexts", [([1], [5000]), ([1, 3, 5], [3000, 700, 4100]), ([0, 40, 2, 130], [600, 40, 2049, 3000]),
                                             ([33], [512]), ([300, 1], [2500, 1])])
def test_prompt_weights_few_rows_over_long_contexts(pkv, D, G, Hkv, q_lens, contexts):
    """Fewer items than SMs: the keys of an item are split over CTAs and the pieces joined."""
    for bs, window in ((256, 0), (16, 2)):
        c = ref.Cache(contexts, bs, Hkv, D, seed=sum(q_lens) + bs, mbs_extra=2)
        check_prompt(pkv, c, q_lens, G, window, seed=G, pad_rows=2)


@pytest.mark.parametrize("D,G,Hkv,q_lens,contexts", [
    (64, 8, 4, [640, 1, 513], [4200, 1, 700]),    # 240 items at most, 148 with work
    (128, 4, 8, [1300], [2500]),                  # 168
    (64, 2, 8, [1300, 1290], [1900, 6200]),       # 176: the second sequence's are the longer ones
    (128, 8, 10, [512], [3500]),                  # 160
])
def test_prompt_weights_last_round_split(pkv, D, G, Hkv, q_lens, contexts):
    """A few more items than SMs: those of the last round are split over the keys, the others are not."""
    c = ref.Cache(contexts, 64, Hkv, D, seed=G, mbs_extra=1)
    c.tables = np.concatenate([c.tables, np.full((len(contexts), 70), -1, c.tables.dtype)], axis=1)
    check_prompt(pkv, c, q_lens, G, 16, seed=G, pad_rows=5)


def test_prompt_weights_split_with_unreadable_pieces(pkv):
    """A split none of whose blocks can be read, and a sequence without any, join to the rest and to zeros."""
    c = ref.Cache([4096, 2048], 64, 2, 64, seed=5)
    c.tables[0, 8:40] = -1
    c.tables[1, :] = c.NB
    check_prompt(pkv, c, [3, 2], 2, expect=FLAG_BAD_BLOCK)


@pytest.mark.parametrize("D,G,Hkv,window", [(64, 8, 1, 0), (128, 4, 2, 0), (64, 8, 1, 700), (64, 1, 3, 0)])
def test_prompt_weights_few_units_split_over_queries(pkv, D, G, Hkv, window):
    """Long prompts of few KV heads: the weights' query tiles are split over CTAs, with the same bits in every run."""
    q_lens, contexts = [1300, 1, 700], [1300, 300, 1100]
    c = ref.Cache(contexts, 32, Hkv, D, seed=G)
    first = check_prompt(pkv, c, q_lens, G, window, seed=G).w.view(torch.int32)
    for _ in range(3):
        d = Dev(c)
        cq = torch.tensor([0, 1300, 1301, 2001], dtype=torch.int32, device="cuda")
        ck = torch.tensor([0, 1300, 1600, 2700], dtype=torch.int32, device="cuda")
        q = bf(queries(2001, Hkv * G, D, G))
        pkv.paged_prefill_weights(q, d.k, d.v, d.tables, cq, ck, 1300, 1 / np.sqrt(D), torch.empty_like(q), d.w, window=window)
        assert torch.equal(d.w.view(torch.int32), first)


@pytest.mark.parametrize("B", [40, 300])
def test_prompt_weights_many_sequences(pkv, B):
    """More sequences than one warp scans at once, and than the longest-first schedule ranks."""
    r = np.random.default_rng(B)
    q_lens = r.integers(0, 12, size=B)
    check_prompt(pkv, ref.Cache(q_lens + r.integers(0, 20, size=B), 16, 1, 64, seed=B), q_lens, 4, window=6, max_q=12)


def test_prompt_weights_tiny_and_large_values(pkv):
    """V is rounded to f16 for P.V: beyond its range it is clamped and flagged, far below it becomes subnormal."""
    c = ref.Cache([70, 200], 16, 2, 64, seed=4)
    v = np.where(np.isnan(ref.from_bf16(c.v)), np.nan, ref.from_bf16(c.v) * 2.0 ** -20)
    c.v = ref.to_bf16(v.astype(np.float32))
    d = check_prompt(pkv, c, [30, 200], 2)
    c = ref.Cache([70, 200], 16, 2, 64, seed=4)
    s = c.slots(1)[:5]
    c.v.reshape(-1, 2, 64)[s] = ref.to_bf16(np.full((5, 2, 64), 65280, dtype=np.float32))  # the last that fits
    d = Dev(c)
    cu = torch.tensor([0, 70, 270], dtype=torch.int32, device="cuda")
    q = bf(queries(270, 4, 64, 0))
    run = lambda out: pkv.paged_prefill_weights(q, d.k, d.v, d.tables, cu, cu, 200, 0.125, out, d.w, err_flag=d.err)
    run(torch.empty_like(q))
    assert int(d.err.item()) == 0
    d.v.view(-1, 2, 64)[torch.from_numpy(s).cuda()] = 1e6
    assert torch.isfinite(run(torch.empty_like(q))).all()
    assert int(d.err.item()) == 0x10  # FLAG_V_RANGE


@pytest.mark.parametrize("idx", [1, 2, 3])
def test_prompt_weights_full_size_steps(pkv, idx):
    """The 16k-token steps: out against the oracle over every row, and the weights against what every softmax
    adds up to: each sequence and KV head receives G per recorded query in all.  Five runs give the same bits
    where no block is shared (shared prefixes receive their additions in any order)."""
    import oracle
    from paged_kv_cache_85_gb300 import workload as wl

    p = wl.prefill_config_workload(idx)
    kc, vc, bad = oracle.store_kvcache(p.k_new, p.v_new, p.k_cache, p.v_cache, p.slot_mapping)
    want = oracle.paged_prefill(p.q, kc, vc, p.block_tables, p.cu_seqlens_q, p.cu_seqlens_k, p.scale, threads=oracle.host_cores())
    q, k, v = bf(p.q), bf(kc), bf(vc)
    t, cq, ck = (torch.from_numpy(x).cuda() for x in (p.block_tables, p.cu_seqlens_q, p.cu_seqlens_k))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = None
    for run in range(5):
        w = torch.zeros(p.NB, p.Hkv, p.bs, device="cuda")
        out = pkv.paged_prefill_weights(q, k, v, t, cq, ck, p.max_seqlen_q, p.scale, torch.empty_like(q), w, err_flag=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        if first is None:
            first = (out, w)
        assert torch.equal(out, first[0])
        if idx != 3:
            assert torch.equal(w, first[1])
    off = np.abs(out.float().cpu().numpy() - want)
    assert off.max() <= 1e-2 and off.mean() <= 1e-3, (off.max(), off.mean())
    # each row's softmax sums to 1 within weight_tolerance (|score| sums below 40 for N(0, 1) inputs), and so do
    # their sums; the fp32 weights themselves are summed in 64 bits
    total = float(first[1].double().sum())
    rows = float(p.Tq) * p.Hq
    assert abs(total - rows) <= ref.weight_tolerance(p.D, 40) * rows
    if idx != 3:
        flat = first[1].double().sum(1).cpu().numpy().reshape(p.NB, p.bs)  # over KV heads
        for b in range(p.B):
            n = int(p.k_lens[b])
            s = np.arange(n)
            got = flat[p.block_tables[b, s // p.bs], s % p.bs].sum()
            assert abs(got - p.q_lens[b] * p.Hq) <= ref.weight_tolerance(p.D, 40) * p.q_lens[b] * p.Hq


def test_prompt_weights_nan_key_reaches_only_its_readers(pkv):
    """A NaN key makes the rows that see it NaN, and with them the weights of the tokens those rows see; earlier
    rows, the other KV head and the other sequences are as without it."""
    c = ref.Cache([300, 90], 16, 2, 64, seed=1)
    cu = torch.tensor([0, 300, 390], dtype=torch.int32, device="cuda")
    qb = queries(390, 4, 64, 0)
    _, w, add, big = ref.prompt(c, ref.from_bf16(qb), cu.cpu().numpy(), 0.125)
    s = c.slots(0)
    c.k.reshape(-1, 2, 64)[s[200], 1, 3] = 0x7FC0
    d, q = Dev(c), bf(qb)
    out = pkv.paged_prefill_weights(q, d.k, d.v, d.tables, cu, cu, 300, 0.125, torch.empty_like(q), d.w, err_flag=d.err)
    got = d.w.cpu().numpy()
    assert torch.isfinite(out[:200]).all() and torch.isfinite(out[300:]).all() and torch.isfinite(out[:, :2]).all()
    assert np.isnan(got[s // 16, 1, s % 16]).all()  # every token is seen by row 200 or a later one
    got[s // 16, 1, s % 16], w[s // 16, 1, s % 16], add[s // 16, 1, s % 16] = 0, 0, 0
    ref.check_weights(got, w, add, ref.weight_tolerance(64, big))


# ------------------------------------------------------------------ eviction


def check_evict(pkv, c, budget, recent, in_place=False, expect=0, want=None):
    d = Dev(c)
    out = d.lens if in_place else torch.full_like(d.lens, -5)
    pkv.evict_kvcache(d.k, d.v, d.w, d.tables, d.lens, budget, recent, out, err_flag=d.err)
    torch.cuda.synchronize()
    assert int(d.err.item()) == expect
    k, v, w, lens = want or ref.evict(c, budget, recent)
    np.testing.assert_array_equal(out.cpu().numpy(), lens)
    np.testing.assert_array_equal(host_cache(d.k), k)
    np.testing.assert_array_equal(host_cache(d.v), v)
    np.testing.assert_array_equal(d.w.cpu().numpy(), w)
    return d


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (17, 5), (64, 64), (64, 0), (100, 99), (299, 32), (5000, 7)])
def test_evict_shapes(pkv, fp8, D, budget, recent):
    for bs, Hkv in ((16, 3), (48, 1)):
        c = ref.Cache([0, 1, 2, 16, 17, 18, 63, 64, 65, 100, 300], bs, Hkv, D, fp8=fp8, seed=budget, mbs_extra=1)
        check_evict(pkv, c, budget, recent, in_place=bs == 16)


@pytest.mark.parametrize("budget,recent", [(1000, 100), (2500, 0), (4999, 2000)])
def test_evict_long(pkv, budget, recent):
    check_evict(pkv, ref.Cache([5000, 3001, 1024, 1025], 256, 2, 128, seed=1), budget, recent)


def test_evict_many_sequences(pkv):
    lens = np.random.default_rng(1).integers(0, 200, size=400)
    check_evict(pkv, ref.Cache(lens, 16, 4, 64, fp8=True, seed=2), 60, 20)


def fill(c, b, h, x):
    s = c.slots(b)
    c.w[s // c.bs, h, s % c.bs] = x


@pytest.mark.parametrize("kind", ["equal", "zeros", "few values", "negative", "infinite", "nan", "signed zero", "subnormal", "ascending", "descending"])
def test_evict_weights_of_every_kind(pkv, kind):
    c = ref.Cache([2300, 700], 64, 2, 64, seed=4)
    r = np.random.default_rng(5)
    for b in range(2):
        n = int(c.lens[b])
        for h in range(2):
            x = {"equal": lambda: np.full(n, 0.25), "zeros": lambda: np.zeros(n), "few values": lambda: r.integers(0, 4, n) * 0.5,
                 "negative": lambda: r.standard_normal(n), "infinite": lambda: r.choice([np.inf, -np.inf, 1.0, 2.0], n),
                 "nan": lambda: r.choice([np.nan, -np.nan, 1.0, np.inf, 0.0], n), "signed zero": lambda: r.choice([-0.0, 0.0], n),
                 "subnormal": lambda: r.integers(0, 50, n) * 1e-45, "ascending": lambda: np.arange(n) * 0.1,
                 "descending": lambda: n - np.arange(n) * 0.1}[kind]()
            fill(c, b, h, x.astype(np.float32))
    check_evict(pkv, c, 300, 30)
    check_evict(pkv, c, 300, 300)


def test_evict_bad_sequences_are_left_alone(pkv):
    c = ref.Cache([200, 150, 100], 32, 2, 64, seed=3)
    good = ref.evict(c, 40, 8)
    k, v, w, lens = (x.copy() for x in good)
    s = c.slots(1)
    for x, y in ((k, c.k), (v, c.v)):
        x.reshape(-1, 2, 64)[s] = y.reshape(-1, 2, 64)[s]
    w[s // 32, :, s % 32] = c.w[s // 32, :, s % 32]
    lens[1] = 150
    c.tables[1, 4] = c.NB
    check_evict(pkv, c, 40, 8, expect=FLAG_BAD_BLOCK, want=(k, v, w, lens))


def test_evict_bad_length_is_left_alone(pkv):
    c = ref.Cache([100, 64], 32, 2, 64, seed=3)
    k, v, w, lens = ref.evict(c, 70, 8)
    c.lens = np.array([100, 129], dtype=np.int32)  # the table holds 4 blocks of 32
    lens[1] = 129
    check_evict(pkv, c, 70, 8, expect=FLAG_BAD_CONTEXT_LEN, want=(k, v, w, lens))
    c.lens = np.array([100, -1], dtype=np.int32)
    lens[1] = -1
    check_evict(pkv, c, 70, 8, expect=FLAG_BAD_CONTEXT_LEN, want=(k, v, w, lens))


def test_evict_lengths_may_overlap(pkv):
    """out_lens may be any view of the lengths' memory."""
    c = ref.Cache([100, 20, 70, 64], 16, 2, 64, seed=3)
    *_, lens = ref.evict(c, 60, 8)
    d = Dev(c)
    both = torch.empty(5, dtype=torch.int32, device="cuda")
    both[:4] = d.lens
    pkv.evict_kvcache(d.k, d.v, d.w, d.tables, both[:4], 60, 8, both[1:])
    assert both[1:].tolist() == lens.tolist()
