"""Captured calls over scaled caches, replayed on inputs that change from replay to replay: every replay against the
64-bit form of what it read."""

import numpy as np
import pytest

import scaled_reference as ref
from test_gpu_scaled_attention import dev, host, pkv, queries  # noqa: F401 (pkv: fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ends = lambda n: np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


class Job:
    """A decode and a prefill (one long context, split over the keys, beside short ones), captured without a workspace."""

    max_q, rows = 50, 60

    def __init__(self, pkv, seed, stream):
        self.rng = np.random.default_rng(seed)
        # four pools of blocks to draw contexts from: the tables change, the caches stay
        self.c = ref.Cache([3000, 40, 700, 1500], 32, 1, 64, seed=seed)
        self.caches = [dev(x) for x in (self.c.k, self.c.v, self.c.ks, self.c.vs)]
        self.args = {"q": np.zeros((3, 4, 64), np.uint16), "qp": np.zeros((self.rows, 4, 64), np.uint16),
                     "tables": np.zeros((3, self.c.MBS), np.int32), "lens": np.ones(3, np.int32),
                     "cu_q": ends([1, 1, 1]), "cu_k": ends([1, 1, 1])}
        self.args = {n: dev(x) for n, x in self.args.items()}
        self.out = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
        self.outp = torch.zeros(self.rows, 4, 64, dtype=torch.bfloat16, device="cuda")
        a = self.args

        def call():
            pkv.paged_attn_decode_scaled(a["q"], *self.caches, a["tables"], a["lens"], 0.1, self.out)
            pkv.paged_prefill_scaled(a["qp"], *self.caches, a["tables"], a["cu_q"], a["cu_k"], self.max_q, 0.1, self.outp)

        self.put()
        call()
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=stream):
            call()

    def put(self):
        """New sequences, lengths and queries into the captured tensors; outputs cleared."""
        rng, c = self.rng, self.c
        pick = rng.permutation(4)[:3]
        self.v = v = ref.Cache.__new__(ref.Cache)
        v.bs, v.Hkv, v.D, v.k, v.v, v.ks, v.vs, v.tables = c.bs, c.Hkv, c.D, c.k, c.v, c.ks, c.vs, c.tables[pick]
        v.lens = np.array([int(rng.integers(1, c.lens[i] + 1)) for i in pick], np.int32)
        self.q_lens = [int(min(n, rng.integers(1, m))) for n, m in zip(v.lens, (self.max_q, 5, 5))]
        self.q, self.qp = queries(rng, 3, 4, 64), queries(rng, self.rows, 4, 64)
        new = {"q": self.q, "qp": self.qp, "tables": v.tables, "lens": v.lens, "cu_q": ends(self.q_lens), "cu_k": ends(v.lens)}
        for n, x in new.items():
            self.args[n].copy_(dev(x))
        self.out.fill_(7), self.outp.fill_(7)

    def check(self, what):
        n = sum(self.q_lens)
        want, mag = ref.decode(self.q, self.v, 0.1)
        ref.check(host(self.out), want, mag, f"{what}: decode")
        want, mag = ref.prefill(self.qp[:n], self.v, self.q_lens, 0.1)
        ref.check(host(self.outp[:n]), want, mag, f"{what}: prefill")
        assert (self.outp[n:] == 7).all(), what


def test_two_graphs_on_inputs_that_change(pkv):
    s = torch.cuda.Stream()
    jobs = [Job(pkv, seed, s) for seed in (1, 2)]
    assert pkv.prefill_scaled_workspace_bytes(3, Job.rows, Job.max_q, 4, 1, 64, jobs[0].c.MBS, 32) > 0
    streams = [torch.cuda.Stream() for _ in jobs]
    for i in range(12):
        for job in jobs:
            job.put()
        torch.cuda.synchronize()
        for job, t in zip(jobs, streams):  # side by side
            with torch.cuda.stream(t):
                job.graph.replay()
        torch.cuda.synchronize()
        for j, job in enumerate(jobs):
            job.check(f"graph {j}, replay {i}")


def test_one_of_two_graphs_alone(pkv):
    """A replay writes its own outputs and leaves the other graph's."""
    s = torch.cuda.Stream()
    jobs = [Job(pkv, seed, s) for seed in (3, 4)]
    for i in range(4):
        for job in jobs:
            job.put()
        torch.cuda.synchronize()
        one, other = jobs[i % 2], jobs[1 - i % 2]
        one.graph.replay()
        torch.cuda.synchronize()
        one.check(f"replay {i}")
        assert (other.out == 7).all() and (other.outp == 7).all()
