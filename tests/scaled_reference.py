"""Plain 64-bit forms (numpy) of the calls on E4M3 caches with a scale per block
and KV head, and the inputs of their tests.  No code of the library is used."""

import numpy as np

from budget_reference import E4M3, from_bf16, to_bf16

NAN_CODE = 0x7F


def encode(x):
    """fp64 -> E4M3 codes: nearest, ties to even, saturating at 448, NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0, x)), 448.0)
    grid = E4M3[:127]  # ascending magnitudes, code = index
    hi = np.searchsorted(grid, a)  # grid[hi - 1] < a <= grid[hi]
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = code | (np.signbit(x).astype(np.int64) << 7)
    return np.where(np.isnan(x), NAN_CODE, code).astype(np.uint8)


def scale_for(a):
    """The least 2^e, e in [-40, 40], with a <= 448 * 2^e."""
    e = -40
    while e < 40 and a > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def store(x, cache, scales, slots):
    """One of K and V: x [N, Hkv, D] bf16 bits; updates cache [NB, bs, Hkv, D] and scales [NB, Hkv] in place.
    Returns how many slots were bad."""
    NB, bs, Hkv, D = cache.shape
    v = from_bf16(x)
    bad, of = 0, {}
    for i, s in enumerate(slots):
        if 0 <= s < NB * bs:
            of.setdefault(int(s) // bs, []).append(i)
        elif s != -1:
            bad += 1
    for b, tokens in of.items():
        off = slots[tokens] % bs
        rows = v[tokens]
        for h in range(Hkv):
            r = np.abs(rows[:, h])
            r = r[np.isfinite(r)]
            want = scale_for(r.max() if r.size else 0.0)
            had = float(scales[b, h])
            if (off == 0).any() or not (np.isfinite(had) and had > 0):
                now = want
            else:
                now = max(had, want)
                if now > had:
                    f = np.float64(np.float32(had) / np.float32(now))
                    # products in fp32, as the definition has it
                    prod = (E4M3[cache[b, :, h]].astype(np.float32) * np.float32(f)).astype(np.float64)
                    cache[b, :, h] = encode(prod)
            scales[b, h] = now
            inv = np.float32(1) / np.float32(now)
            with np.errstate(over="ignore", invalid="ignore"):
                cache[b, off, h] = encode((rows[:, h].astype(np.float32) * inv).astype(np.float64))
    return bad


def values(cache, scales):
    """fp64 [NB, bs, Hkv, D]."""
    return E4M3[cache] * scales.astype(np.float64)[:, None, :, None]


def attend(q, K, V, scale, first=None):
    """softmax(scale q K^T) V of one KV head: q [n, D], K, V [T, D]; query i sees tokens < first + i + 1 where given.
    Returns (out, sum of weight times |V|)."""
    s = scale * (q @ K.T)
    if first is not None:
        s = np.where(np.arange(K.shape[0])[None] <= first + np.arange(q.shape[0])[:, None], s, -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    return p @ V, p @ np.abs(V)


class Cache:
    """A filled scaled cache with its block tables.  Slots that no sequence uses hold NaN codes, blocks that none
    uses NaN scales.  `spread`: blocks' and heads' magnitudes are 2^(spread * normal)."""

    def __init__(self, lens, bs, Hkv, D, seed=0, spread=1.0, extra_blocks=2, mbs_extra=0, pow2=True):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, dtype=np.int32)
        self.bs, self.Hkv, self.D = bs, Hkv, D
        B = len(self.lens)
        nblk = -(-self.lens.astype(np.int64) // bs)
        self.NB = int(nblk.sum()) + extra_blocks
        self.MBS = max(1, (int(nblk.max()) if B else 1) + mbs_extra)
        perm = rng.permutation(self.NB).astype(np.int32)
        self.tables = np.full((B, self.MBS), -1, dtype=np.int32)
        cur = 0
        for b in range(B):
            self.tables[b, : nblk[b]] = perm[cur: cur + nblk[b]]
            cur += int(nblk[b])
        self.k, self.ks = self._draw(rng, spread, pow2)
        self.ks = np.minimum(self.ks, np.float32(1 / 64))  # scores stay small
        self.v, self.vs = self._draw(rng, spread, pow2)
        used = np.zeros((self.NB, bs), dtype=bool)
        for b in range(B):
            s = self.slots(b)
            used[s // bs, s % bs] = True
        for c, s in ((self.k, self.ks), (self.v, self.vs)):
            c[~used] = NAN_CODE
            s[~used.any(1)] = np.nan

    def _draw(self, rng, spread, pow2):
        shape = (self.NB, self.bs, self.Hkv, self.D)
        x = rng.standard_normal(shape)
        s = 2.0 ** np.round(spread * rng.standard_normal((self.NB, self.Hkv))) / 128
        if not pow2:
            s = s * rng.uniform(0.6, 1.0, s.shape)
        return encode(x * 100), s.astype(np.float32)

    def slots(self, b):
        t = np.arange(self.lens[b])
        return self.tables[b, t // self.bs].astype(np.int64) * self.bs + t % self.bs

    def rows(self, b, which):
        c, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        at = self.slots(b)
        return E4M3[c.reshape(-1, self.Hkv, self.D)[at]] * s[at // self.bs].astype(np.float64)[..., None]


def decode(q, c, scale, skip=None):
    """q bf16 bits [B, Hq, D] -> (out, weighted |V|), fp64.  skip[b]: mask of tokens left out."""
    B, Hq, D = q.shape
    G = Hq // c.Hkv
    out, mag = np.zeros((2, B, Hq, D))
    qf = from_bf16(q)
    for b in range(B):
        if c.lens[b] == 0:
            continue
        K, V = c.rows(b, "k"), c.rows(b, "v")
        if skip is not None and skip.get(b) is not None:
            keep = ~skip[b][: len(K)]
            if not keep.any():
                continue
            K, V = K[keep], V[keep]
        for h in range(c.Hkv):
            at = slice(h * G, (h + 1) * G)
            out[b, at], mag[b, at] = attend(qf[b, at], K[:, h], V[:, h], scale)
    return out, mag


def prefill(q, c, q_lens, scale):
    """q bf16 bits [Tq, Hq, D], the last q_lens[b] tokens of each context being new."""
    Hq, D = q.shape[1:]
    G = Hq // c.Hkv
    out, mag = np.zeros((2, *q.shape))
    qf = from_bf16(q)
    at = 0
    for b, n in enumerate(q_lens):
        if n == 0:
            continue
        K, V = c.rows(b, "k"), c.rows(b, "v")
        for h in range(c.Hkv):
            for g in range(G):
                rows = slice(at, at + n)
                out[rows, h * G + g], mag[rows, h * G + g] = attend(
                    qf[rows, h * G + g], K[:, h], V[:, h], scale, first=int(c.lens[b]) - n)
        at += n
    return out, mag


def check(got, ref, mag, what=""):
    """A bf16 output's rounding is 2^-8 of it.  Weights: P and V are rounded to f16 (2^-11 each), and a score that
    is off by d moves weights by 2d of the sum of weight times |V|; scores of up to 16 from products kept to 2^-13 of
    the largest are off by 2^-9 at most.  Together below 2^-7 of that sum."""
    got = np.asarray(got, dtype=np.float64)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    err, bound = np.abs(got - ref), 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * mag
    worst = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), f"{what}: off by {err[worst]:.3e} > {bound[worst]:.3e} at {worst}"
    return float((err / np.maximum(mag, 1e-300)).max())


def bf16(x):
    return to_bf16(np.asarray(x, dtype=np.float32))
