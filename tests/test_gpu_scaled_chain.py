"""The calls on scaled caches together, as an engine uses them: prompts with cached prefixes and in chunks, decode steps,
forks, compaction, graphs, threads and streams."""

import threading

import numpy as np
import pytest

import scaled_reference as ref

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


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


class Engine:
    """A pool on the GPU and its 64-bit mirror, driven by the allocator."""

    def __init__(self, pkv, NB, bs, Hkv, G, D, seed=0):
        from paged_kv_cache_85_gb300.block_manager import BlockManager

        self.pkv, self.bm = pkv, BlockManager(NB, bs)
        self.bs, self.Hkv, self.G, self.D = bs, Hkv, G, D
        self.rng = np.random.default_rng(seed)
        shape = (NB, bs, Hkv, D)
        # a pool is not cleared before its first use
        self.c = [self.rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2)]
        self.s = [np.full((NB, Hkv), np.nan, np.float32) for _ in range(2)]
        self.dc, self.ds = [dev(x) for x in self.c], [dev(x) for x in self.s]
        self.scale = D ** -0.5

    def rows(self, n):
        # keys small enough for mild scores, values of all sizes
        k = self.rng.standard_normal((n, self.Hkv, self.D))
        v = self.rng.standard_normal((n, self.Hkv, self.D)) * 2.0 ** (2 * self.rng.standard_normal((n, self.Hkv, 1)))
        return ref.bf16(k), ref.bf16(v)

    def store(self, slots):
        k, v = self.rows(len(slots))
        slots = np.asarray(slots, np.int64)
        self.pkv.store_kvcache_scaled(dev(k), dev(v), *self.dc, *self.ds, dev(slots))
        for x, c, s in zip((k, v), self.c, self.s):
            ref.store(x, c, s, slots)

    def mirror(self, ids):
        """What the 64-bit forms read: a Cache over the mirror with these sequences' tables."""
        m = ref.Cache.__new__(ref.Cache)
        MBS = max(len(self.bm.block_table(i)) for i in ids) + 1
        m.tables, m.lens, _ = self.bm.decode_batch(ids, MBS)
        m.bs, m.Hkv, m.D = self.bs, self.Hkv, self.D
        m.k, m.v, m.ks, m.vs = *self.c, *self.s
        return m

    def prompt(self, jobs):
        """One prefill step: (sequence, tokens that it holds before, tokens to run) each."""
        ids = [i for i, _, _ in jobs]
        self.store(np.concatenate([self.bm.slots(i, a, a + n) for i, a, n in jobs]))
        m = self.mirror(ids)
        m.lens = np.array([a + n for _, a, n in jobs], np.int32)
        q_lens = [n for _, _, n in jobs]
        q = ref.bf16(self.rng.standard_normal((sum(q_lens), self.Hkv * self.G, self.D)))
        ends = lambda x: dev(np.concatenate([[0], np.cumsum(x)]).astype(np.int32))
        out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        self.pkv.paged_prefill_scaled(dev(q), *self.dc, *self.ds, dev(m.tables), ends(q_lens), ends(m.lens), max(q_lens),
                                      self.scale, out)
        want, mag = ref.prefill(q, m, q_lens, self.scale)
        ref.check(host(out), want, mag, "prompt")

    def step(self, ids):
        """One decode step."""
        self.store(self.bm.append_batch(ids, self.rng.integers(0, 1000, len(ids)).astype(np.int32)))
        m = self.mirror(ids)
        q = ref.bf16(self.rng.standard_normal((len(ids), self.Hkv * self.G, self.D)))
        out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        self.pkv.paged_attn_decode_scaled(dev(q), *self.dc, *self.ds, dev(m.tables), dev(m.lens), self.scale, out)
        want, mag = ref.decode(q, m, self.scale)
        ref.check(host(out), want, mag, "step")

    def copy(self, pairs):
        self.pkv.copy_blocks([*self.dc, *self.ds], dev(pairs))
        for t in (*self.c, *self.s):
            t[pairs[:, 1]] = t[pairs[:, 0]]

    def check(self):
        for got, want in zip(self.ds, self.s):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        for got, want in zip(self.dc, self.c):
            got = got.cpu().numpy()
            nan = (want & 0x7F) == 0x7F
            np.testing.assert_array_equal(got[~nan], want[~nan])
            assert ((got[nan] & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("bs,Hkv,G,D", [(16, 2, 4, 64), (32, 3, 2, 128), (256, 1, 8, 128)])
def test_an_engine(pkv, bs, Hkv, G, D):
    e = Engine(pkv, 90 if bs < 256 else 14, bs, Hkv, G, D, seed=bs)
    common = list(range(2 * bs))
    # a prompt; then two that share its first blocks, one of them run in chunks
    e.bm.allocate(1, common + [7] * 11)
    e.prompt([(1, 0, 2 * bs + 11)])
    a = e.bm.allocate(2, common + [9] * (bs // 2 + 3))
    b = e.bm.allocate(3, list(range(bs)) + [3] * (bs + 5))
    assert (a, b) == (2 * bs, bs)
    e.prompt([(2, a, bs // 2 + 3), (3, b, 9)])
    e.prompt([(3, b + 9, bs - 4)])
    for _ in range(4):
        e.step([1, 2, 3])
    # two samples go on from sequence 3
    for child in (4, 5):
        e.copy(e.bm.fork(3, child))
    e.check()
    for _ in range(5):
        e.step([3, 4, 5, 1])
    # one ends, another comes, the pool is compacted
    e.bm.deallocate(1)
    e.bm.deallocate(3)
    e.bm.allocate(6, [5] * (bs + 1))
    e.prompt([(6, 0, bs + 1)])
    moves = e.bm.compact()
    assert len(moves)
    e.copy(moves)
    e.check()
    for _ in range(3):
        e.step([2, 4, 5, 6])
    e.check()


def test_the_graph_runner(pkv):
    """Padded replays of a step over a scaled cache give what the eager calls give."""
    from paged_kv_cache_85_gb300.graph_runner import DecodeGraphRunner

    rng = np.random.default_rng(0)
    c = ref.Cache([100, 17, 33, 64, 250], 16, 2, 64, seed=1, mbs_extra=1)
    t = [dev(x) for x in (c.k, c.v, c.ks, c.vs)]
    with pytest.raises(ValueError):
        DecodeGraphRunner(t[0], t[1], 8, 8, c.MBS, 0.1, k_scales=t[2])
    r = DecodeGraphRunner(t[0], t[1], 8, 8, c.MBS, 0.1, k_scales=t[2], v_scales=t[3])
    eager = [x.clone() for x in t]
    for n in (5, 3, 1):
        q, k, v = (dev(ref.bf16(rng.standard_normal((n, h, 64)))) for h in (8, 2, 2))
        slots = dev(np.array([c.slots(b)[-1] for b in range(n)]))
        tables, lens = dev(c.tables[:n]), dev(c.lens[:n])
        got = r.step(q, k, v, slots, tables, lens).clone()
        want = torch.empty_like(q)
        pkv.store_kvcache_scaled(k, v, *eager, slots)
        pkv.paged_attn_decode_scaled(q, *eager, tables, lens, 0.1, want)
        # (another batch is another split of the contexts)
        assert (got.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
        for x, y in zip(t, eager):
            assert torch.equal(x.nan_to_num() if x.is_floating_point() else x, y.nan_to_num() if y.is_floating_point() else y)


def test_two_threads_and_streams(pkv):
    """Two threads with a stream each, the calls behind each other without a wait."""
    errors = []

    def work(seed):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                rng = np.random.default_rng(seed)
                c = ref.Cache([1000, 40, 333], 32, 2, 128, seed=seed)
                t = [dev(x) for x in (c.k, c.v, c.ks, c.vs)]
                tables, lens = dev(c.tables), dev(c.lens)
                qh = ref.bf16(rng.standard_normal((3, 8, 128)))
                spare = int(np.setdiff1d(np.arange(c.NB), c.tables)[0])
                pairs = dev(np.array([[c.tables[0, 0], spare]], np.int32))
                kh, vh = (ref.bf16(rng.standard_normal((3, 2, 128))) for _ in range(2))
                slots = np.array([c.slots(b)[-1] for b in range(3)])
                q, k, v, sl = dev(qh), dev(kh), dev(vh), dev(slots)
                for x, cc, s in ((kh, c.k, c.ks), (vh, c.v, c.vs)):
                    ref.store(x, cc, s, slots)
                want, mag = ref.decode(qh, c, 0.08)
                outs = [torch.empty_like(q) for _ in range(20)]
                cu_q, cu_k = dev(np.arange(4, dtype=np.int32)), dev(np.array([0, 1000, 1040, 1373], np.int32))
                torch.cuda.current_stream().synchronize()
                for i, out in enumerate(outs):
                    pkv.store_kvcache_scaled(k, v, *t, sl)
                    if i % 2:
                        pkv.paged_attn_decode_scaled(q, *t, tables, lens, 0.08, out)
                    else:  # the newest token as a chunk of one
                        pkv.paged_prefill_scaled(q, *t, tables, cu_q, cu_k, 1, 0.08, out)
                    pkv.copy_blocks(t, pairs)
                torch.cuda.current_stream().synchronize()
                for out in outs:
                    ref.check(host(out), want, mag)
                assert torch.equal(t[0][spare], t[0][int(c.tables[0, 0])])
        except BaseException as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    if errors:
        raise errors[0]


def test_refusals(pkv):
    c = ref.Cache([40, 20], 16, 2, 64, seed=1)
    t = dict(k_cache=dev(c.k), v_cache=dev(c.v), k_scales=dev(np.nan_to_num(c.ks)), v_scales=dev(np.nan_to_num(c.vs)))
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    tables, lens = dev(c.tables), dev(c.lens)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    calls = [lambda **kw: pkv.store_kvcache_scaled(**(dict(k=k, v=k, slot_mapping=slots) | t | kw)),
             lambda **kw: pkv.paged_attn_decode_scaled(**(dict(q=q, block_tables=tables, context_lens=lens, scale=0.1, out=q.clone()) | t | kw)),
             lambda **kw: pkv.paged_prefill_scaled(**(dict(q=q, block_tables=tables, cu_seqlens_q=cu, cu_seqlens_k=cu, max_seqlen_q=1,
                                                           scale=0.1, out=q.clone()) | t | kw))]
    for call in calls:
        call()
        for name in t:
            with pytest.raises((ValueError, TypeError), match=name):
                call(**{name: t[name].cpu()})
            with pytest.raises((ValueError, TypeError)):
                call(**{name: None})
        with pytest.raises(ValueError, match="shapes differ"):
            call(v_cache=t["v_cache"][1:])
        with pytest.raises(ValueError, match="k_scales must be"):
            call(k_scales=t["k_scales"][1:])
        with pytest.raises(ValueError, match="v_scales"):
            call(v_scales=t["v_scales"].double())
        with pytest.raises(ValueError, match="k_cache"):
            call(k_cache=t["k_cache"].to(torch.int8))
        with pytest.raises(ValueError, match="k_cache"):
            call(k_cache=t["k_cache"].transpose(1, 2))
        with pytest.raises(ValueError, match="err_flag"):
            call(err_flag=torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError, match="slot_mapping"):
        calls[0](slot_mapping=slots[:1])
    with pytest.raises(ValueError, match="slot_mapping"):
        calls[0](slot_mapping=slots.int())
    with pytest.raises(ValueError, match="k and v"):
        calls[0](k=k[:, :1].contiguous())
    with pytest.raises(ValueError, match="k must be"):
        calls[0](k=k.float())
    with pytest.raises(pkv.PkvError, match="share"):
        calls[0](v_cache=t["k_cache"])
    for call in calls[1:]:
        with pytest.raises(ValueError, match="head_dim"):
            call(q=torch.zeros((2, 4, 128), dtype=torch.bfloat16, device="cuda"))
        with pytest.raises(ValueError, match="out"):
            call(out=q[:1])
        with pytest.raises(ValueError, match="out"):
            call(out=q.float())
        with pytest.raises(ValueError, match="out"):
            call(out=torch.zeros((2, 4, 64), dtype=torch.bfloat16))  # pageable host memory
        with pytest.raises(ValueError, match="batch"):
            call(block_tables=tables[:1])
        with pytest.raises(pkv.PkvError, match="multiple"):
            call(q=q[:, :3].contiguous(), out=q[:, :3].contiguous())
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=torch.zeros(10))
    with pytest.raises(pkv.PkvError, match="workspace"):
        calls[1](workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="32 bits"):
        calls[1](max_ctas=2 ** 32 + 1)
    with pytest.raises(ValueError, match="32 bits"):
        calls[2](max_seqlen_q=2 ** 32 + 1)
    with pytest.raises(pkv.PkvError, match="scale"):
        calls[1](scale=float("nan"))
    # nothing to do
    empty = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    calls[0](k=k[:0], v=k[:0], slot_mapping=slots[:0])
    calls[1](q=empty, out=empty, block_tables=tables[:0], context_lens=lens[:0])
    calls[2](q=empty, out=empty)
    calls[2](q=empty, out=empty, block_tables=tables[:0], cu_seqlens_q=cu[:1], cu_seqlens_k=cu[:1], max_seqlen_q=0)
