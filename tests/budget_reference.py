"""Plain 64-bit forms (numpy) of the calls that record attention weights and of
the eviction, and the inputs of their tests.  No code of the library is used."""

import numpy as np

# E4M3 code -> value: 1 sign, 4 exponent bits (bias 7), 3 mantissa bits; no infinities
_codes = np.arange(256)
_e, _m = (_codes >> 3) & 15, _codes & 7
E4M3 = np.where(_e == 0, _m * 2.0 ** -9, (8 + _m) * 2.0 ** (_e - 10.0)) * np.where(_codes >> 7, -1.0, 1.0)
E4M3[[0x7F, 0xFF]] = np.nan


def to_bf16(x):
    """fp32 array -> bf16 bits (nearest even)."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def from_bf16(b):
    return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def values(cache, scale=None):
    """A cache's values: bf16 bits, or E4M3 codes times the scale."""
    return from_bf16(cache) if cache.dtype == np.uint16 else E4M3[cache] * scale


class Cache:
    """A paged cache with its block tables; every slot no sequence uses is NaN."""

    def __init__(self, lens, bs, Hkv, D, fp8=False, seed=0, extra_blocks=2, mbs_extra=0):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, dtype=np.int32)
        self.bs, self.Hkv, self.D, self.fp8 = bs, Hkv, D, fp8
        B = len(self.lens)
        nblk = -(-self.lens.astype(np.int64) // bs)
        self.NB = int(nblk.sum()) + extra_blocks
        self.MBS = int(nblk.max()) + mbs_extra if B else 1
        self.MBS = max(self.MBS, 1)
        perm = rng.permutation(self.NB).astype(np.int32)
        self.tables = np.full((B, self.MBS), -1, dtype=np.int32)
        cur = 0
        for b in range(B):
            self.tables[b, : nblk[b]] = perm[cur: cur + nblk[b]]
            cur += int(nblk[b])
        shape = (self.NB, bs, Hkv, D)
        self.k, self.v = (self._draw(rng, shape) for _ in range(2))
        self.w = rng.exponential(size=(self.NB, Hkv, bs)).astype(np.float32)
        used = np.zeros((self.NB, bs), dtype=bool)
        for b in range(B):
            s = self.slots(b)
            used[s // bs, s % bs] = True
        nan = 0x7F if fp8 else 0x7FC0
        self.k[~used] = nan
        self.v[~used] = nan
        self.w[np.broadcast_to(~used[:, None, :], self.w.shape)] = np.nan
        self.k_scale, self.v_scale = (0.03, 0.021) if fp8 else (1.0, 1.0)

    def _draw(self, rng, shape):
        if self.fp8:
            c = rng.integers(0, 256, size=shape, dtype=np.uint8)
            c[(c & 0x7F) == 0x7F] = 0  # no NaN
            return np.where((c & 0x78) > 0x60, c & 0x9F, c).astype(np.uint8)  # magnitudes below 32
        return to_bf16(rng.standard_normal(shape, dtype=np.float32))

    def slots(self, b, n=None):
        """Flat slots of the first n tokens of sequence b (bad entries give negative slots)."""
        t = np.arange(self.lens[b] if n is None else n)
        return self.tables[b, t // self.bs].astype(np.int64) * self.bs + t % self.bs

    def flat(self, x):
        return x.reshape(self.NB * self.bs, self.Hkv, self.D)


def decode(c, q, scale):
    """(out [B, Hq, D], weights, weight added per slot [NB, Hkv, bs], largest |score| sum)."""
    B, Hq, D = q.shape
    G = Hq // c.Hkv
    out, w, big = np.zeros(q.shape), c.w.astype(np.float64), 0.0
    add = np.zeros_like(w)
    k, v = values(c.flat(c.k), c.k_scale), values(c.flat(c.v), c.v_scale)
    for b in range(B):
        n = int(c.lens[b])
        s = c.slots(b)
        ok = (s >= 0) & (s < c.NB * c.bs)
        if n == 0 or not ok.any():
            continue
        r = s[ok]
        qq = q[b].reshape(c.Hkv, G, D)
        sc = np.einsum("hgd,thd->hgt", qq, k[r]) * scale
        big = max(big, float((np.einsum("hgd,thd->hgt", np.abs(qq), np.abs(k[r])) * abs(scale)).max()))
        p = np.exp(sc - sc.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        out[b] = np.einsum("hgt,thd->hgd", p, v[r]).reshape(Hq, D)
        got = p.sum(1)  # [Hkv, t]
        last = s[n - 1]
        if ok[n - 1]:
            w[last // c.bs, :, last % c.bs] = 0.0
        for h in range(c.Hkv):
            np.add.at(w, (r // c.bs, h, r % c.bs), got[h])
            np.add.at(add, (r // c.bs, h, r % c.bs), got[h])
    return out, w, add, big


def prompt(c, q, cu_q, scale, window=0):
    """The same for a prefill step: q [Tq, Hq, D], new tokens cu_q, contexts c.lens."""
    Hq, D = q.shape[1:]
    G = Hq // c.Hkv
    out, w, big = np.full(q.shape, np.nan), c.w.astype(np.float64), 0.0
    add = np.zeros_like(w)
    k, v = values(c.flat(c.k)), values(c.flat(c.v))
    for b in range(len(c.lens)):
        n, ql = int(c.lens[b]), int(cu_q[b + 1] - cu_q[b])
        if ql == 0:
            continue
        s, base = c.slots(b), n - ql
        ok = (s >= 0) & (s < c.NB * c.bs)
        new = s[base:][ok[base:]]
        w[new // c.bs, :, new % c.bs] = 0.0
        for i in range(ql):
            see = np.nonzero(ok[: base + i + 1])[0]
            if not len(see):
                out[cu_q[b] + i] = 0.0
                continue
            r = s[see]
            qq = q[cu_q[b] + i].reshape(c.Hkv, G, D)
            sc = np.einsum("hgd,thd->hgt", qq, k[r]) * scale
            big = max(big, float((np.einsum("hgd,thd->hgt", np.abs(qq), np.abs(k[r])) * abs(scale)).max()))
            p = np.exp(sc - sc.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            out[cu_q[b] + i] = np.einsum("hgt,thd->hgd", p, v[r]).reshape(Hq, D)
            if window and i < ql - window:
                continue
            for h in range(c.Hkv):
                np.add.at(w, (r // c.bs, h, r % c.bs), p.sum(1)[h])
                np.add.at(add, (r // c.bs, h, r % c.bs), p.sum(1)[h])
    return out, w, add, big


def weight_tolerance(D, big):
    """Relative error of one softmax weight formed in fp32.

    The tensor cores sum exact products in fp32, D / 16 steps of which each may
    lose 2 units of 2^-23 of the largest partial sum (they truncate), at most
    `big` = scale * sum |q_d k_d|; scaling, the log-sum-exp (as large as a score
    in magnitude, plus log2 of the length) and the subtraction round once each:
    4 more such units.  An absolute error e of the exponent (natural units) is a
    relative error e of the weight; 2^x itself, the sum behind the log-sum-exp
    and the sum over heads stay below 2^-19 in all."""
    return (D / 16 * 2 + 4) * 2.0 ** -23 * (big + 16) + 2.0 ** -19


def check_weights(got, want, add, tol, what=""):
    """`got` fp32 against `want`: off by tol of what was added and by the rounding of the addition."""
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    fine = ~np.isnan(want)
    # one rounding per addition of the call to the slot (at most 64 sequences share one here)
    bound = tol * add + 2.0 ** -24 * 4 * np.abs(want) + 1e-37
    off = np.abs(got.astype(np.float64) - want)
    bad = fine & (off > bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} weights off, worst {np.max((off / bound)[fine]):.3g} bounds"


def evict(c, budget, recent):
    """(k, v, w, lens) after the eviction, from copies."""
    k, v, w = c.flat(c.k.copy()), c.flat(c.v.copy()), c.w.copy()
    lens = c.lens.copy()
    for b, n in enumerate(c.lens.tolist()):
        if n <= budget:
            continue
        s, old = c.slots(b), n - recent
        for h in range(c.Hkv):
            x = w[s // c.bs, h, s % c.bs]
            order = sorted(range(old), key=lambda t: (0 if np.isnan(x[t]) else 1, 0.0 if np.isnan(x[t]) else -x[t], t))
            kept = sorted(order[: budget - recent]) + list(range(old, n))
            src, dst = s[kept], s[:budget]
            k[dst, h], v[dst, h] = k[src, h].copy(), v[src, h].copy()
            w[dst // c.bs, h, dst % c.bs] = x[kept]
        lens[b] = budget
    return k.reshape(c.k.shape), v.reshape(c.v.shape), w, lens
