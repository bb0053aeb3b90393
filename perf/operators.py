"""Operators of a KV cache with a budget: what is measured of them.

Three operators work together when contexts outgrow the memory for their cache:

  decode   one decode step of paged attention that also adds, to every cached
           token, the attention weight it received (bf16 and E4M3 caches);
  prompt   causal attention of a chunk of new tokens over a paged cache that
           does the same, over all of the chunk's queries or the last `window`;
  evict    per sequence and KV head, keep the `recent` last tokens and, of the
           others, those with the largest accumulated weight, `budget` in all,
           moved in order to the front of the sequence's blocks.

Layouts are the package's: caches [NB, bs, Hkv, D], block tables [B, MBS]; the
weights are fp32 [NB, Hkv, bs] under the same block ids.
"""

import math
import random

import torch

own = False


# ------------------------------------------------------------------ the cases


def listed():
    return [
        # the package's tiny decode step: four short contexts, latency counts
        dict(name="decode tiny", op="decode", f8=False, B=4, Hq=4, Hkv=2, D=64, bs=16, lo=1, hi=300, spread="uniform"),
        # a model with 16 query and 8 KV heads serving 64 sequences up to its 4096 limit
        dict(name="decode 64 seqs", op="decode", f8=False, B=64, Hq=16, Hkv=8, D=128, bs=256, lo=128, hi=4096, spread="uniform"),
        # an 8-billion-parameter model's heads, 256 sequences in 16-token blocks
        dict(name="decode bs16", op="decode", f8=False, B=256, Hq=32, Hkv=8, D=128, bs=16, lo=1, hi=2048, spread="uniform"),
        # the largest batch the engine runs, over an E4M3 cache
        dict(name="decode fp8 512 seqs", op="decode", f8=True, B=512, Hq=16, Hkv=8, D=128, bs=256, lo=16, hi=4096, spread="log"),
        # four prompts of a few tokens: the smallest prefill step
        dict(name="prompt tiny", op="prompt", B=4, Hq=4, Hkv=2, D=64, bs=16, qlo=1, qhi=40, clo=0, chi=32, window=0),
        # a full 16k-token prefill step, every query recorded, cached prefixes on half of it
        dict(name="prompt 16k", op="prompt", B=8, Hq=16, Hkv=8, D=128, bs=256, qlo=2048, qhi=2048, clo=0, chi=2048, window=0),
        # ragged prompts with prefix hits in 16-token blocks, the last 32 queries observe
        dict(name="prompt ragged window", op="prompt", B=32, Hq=32, Hkv=8, D=128, bs=16, qlo=1, qhi=1023, clo=0, chi=1024, window=32),
        # one chunk of a long prompt (chunked prefill), observed by its last 64 queries
        dict(name="prompt long chunk", op="prompt", B=1, Hq=32, Hkv=8, D=128, bs=256, qlo=2048, qhi=2048, clo=28672, chi=28672, window=64),
        # a handful of short contexts trimmed
        dict(name="evict tiny", op="evict", f8=False, B=4, Hkv=2, D=64, bs=16, lo=1, hi=300, spread="uniform", budget=100, recent=32),
        # 64 sequences trimmed to a quarter of the model's limit
        dict(name="evict 64 seqs", op="evict", f8=False, B=64, Hkv=8, D=128, bs=256, lo=128, hi=4096, spread="uniform", budget=1024, recent=256),
        # long contexts cut to an eighth
        dict(name="evict long", op="evict", f8=False, B=8, Hkv=8, D=128, bs=256, lo=32768, hi=32768, spread="uniform", budget=4096, recent=512),
        # many short contexts over an E4M3 cache in 16-token blocks
        dict(name="evict fp8 bs16", op="evict", f8=True, B=256, Hkv=8, D=128, bs=16, lo=1, hi=2048, spread="uniform", budget=511, recent=65),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["decode", "prompt", "evict"])
    D, bs = rng.choice([64, 128]), rng.choice([16, 32, 48, 64, 128, 256])
    Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 8])
    if op == "prompt":
        B = _log_int(rng, 1, 32)
        # new tokens x context at most those of the 16k step
        qhi = _log_int(rng, 1, max(2, 16384 // B))
        most = max(0, min(30000, (40_000_000 // (B * qhi) - qhi) // max(1, Hkv * G // 16)))
        chi = rng.choice([0, rng.randint(0, most)])
        window = rng.choice([0, _log_int(rng, 1, 2 * qhi + 1)])
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, bs=bs, qlo=rng.randint(1, qhi), qhi=qhi, clo=0, chi=chi, window=window)
    B = _log_int(rng, 1, 512)
    hi = _log_int(rng, 1, min(40000, 500_000 // B))
    lo = rng.randint(1, hi)
    case = dict(op=op, f8=rng.random() < 0.4, B=B, Hkv=Hkv, D=D, bs=bs, lo=lo, hi=hi, spread=rng.choice(["uniform", "log"]))
    if op == "decode":
        return case | dict(Hq=Hkv * G)
    budget = rng.randint(1, hi)
    return case | dict(budget=budget, recent=rng.randint(0, budget))


# ----------------------------------------------------------------- the inputs


def _lengths(case):
    """Host lengths of a case (the engine knows them; the operators read them on the GPU): new
    tokens (prompts only) and contexts, the same for every seed, so that all inputs of a case
    have one shape and one amount of work."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] == "prompt":
        bs = case["bs"]
        q = [r.randint(case["qlo"], case["qhi"]) for _ in range(case["B"])]
        # cached prefixes are whole blocks
        c = [r.randint(case["clo"] // bs, case["chi"] // bs) * bs for _ in range(case["B"])]
        return torch.tensor(q), torch.tensor(q) + torch.tensor(c)
    lo, hi = case["lo"], case["hi"]
    if case["spread"] == "log":
        return None, torch.tensor([_log_int(r, lo, hi) for _ in range(case["B"])])
    return None, torch.tensor([r.randint(lo, hi) for _ in range(case["B"])])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    B, Hkv, D, bs, op = case["B"], case["Hkv"], case["D"], case["bs"], case["op"]
    q_lens, n = _lengths(case)
    blocks = (n + bs - 1) // bs
    MBS, need = int(blocks.max()), int(blocks.sum())
    NB = need + need // 8 + 1
    # blocks scattered over the pool, as a running engine leaves them
    perm = torch.randperm(NB, generator=g, device=dev, dtype=torch.int32)
    ends = blocks.cumsum(0)
    j = torch.arange(MBS)
    used = j[None] < blocks[:, None]
    at = (ends - blocks)[:, None] + j[None]
    tables = torch.where(used.to(dev), perm[at.clamp(max=NB - 1).to(dev)], torch.full((), -1, dtype=torch.int32, device=dev))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    s = dict(op=op, bs=bs, D=D, Hkv=Hkv, scale=1.0 / math.sqrt(D), tables=tables.contiguous())
    k, v = randn(NB, bs, Hkv, D), randn(NB, bs, Hkv, D)
    if case.get("f8"):
        # codes of x / s with one scale per tensor: amax / 448, as the store writes them
        s["k_scale"], s["v_scale"] = 6.0 / 448, 6.0 / 448
        k = (k.float() / s["k_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v.float() / s["v_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s["f8"], s["k_cache"], s["v_cache"] = bool(case.get("f8")), k, v
    # weight gathered so far: a few heavy tokens, many light ones, some that never got any
    w = torch.exp(2 * torch.randn(NB, Hkv, bs, generator=g, device=dev)) * 0.002
    s["weights"] = torch.where(torch.rand(NB, Hkv, bs, generator=g, device=dev) < 0.03, torch.zeros((), device=dev), w)
    if op == "prompt":
        s["cu_q"] = torch.cat([torch.zeros(1, dtype=torch.long), q_lens.cumsum(0)]).to(dev, torch.int32)
        s["cu_k"] = torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)]).to(dev, torch.int32)
        s["max_q"], s["window"] = int(q_lens.max()), case["window"]
        s["q"] = 2 * randn(int(q_lens.sum()), case["Hq"], D)
        s["out"] = torch.empty_like(s["q"])
    else:
        s["lens"] = n.to(dev, torch.int32)
        if op == "decode":
            s["q"] = 2 * randn(B, case["Hq"], D)
            s["out"] = torch.empty_like(s["q"])
        else:
            s["budget"], s["recent"] = case["budget"], case["recent"]
            s["out_lens"] = torch.empty(B, dtype=torch.int32, device=dev)
    return s


# --------------------------------------------------------------- the one pass


def run(s):
    if own:
        return _run_own(s)
    return {"decode": _decode, "prompt": _prompt, "evict": _evict}[s["op"]](s)


def _run_own(s):
    import paged_kv_cache_85_gb300 as pkv

    if s["op"] == "decode":
        if s["f8"]:
            pkv.paged_attn_decode_weights_fp8(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"],
                                              s["k_scale"], s["v_scale"], s["out"], s["weights"])
        else:
            pkv.paged_attn_decode_weights(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"],
                                          s["out"], s["weights"])
        return [s["out"], s["weights"]]
    if s["op"] == "prompt":
        pkv.paged_prefill_weights(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["cu_q"], s["cu_k"], s["max_q"],
                                  s["scale"], s["out"], s["weights"], window=s["window"])
        return [s["out"], s["weights"]]
    pkv.evict_kvcache(s["k_cache"], s["v_cache"], s["weights"], s["tables"], s["lens"], s["budget"], s["recent"], s["out_lens"])
    return [_values(s, "k_cache"), _values(s, "v_cache"), s["weights"], s["out_lens"]]


def _values(s, name):
    return s[name].view(torch.float8_e4m3fn) if s["f8"] else s[name]


def _gathered(s, name, blk, off, scale):
    """[B, T, Hkv, D] fp32 values of every sequence's tokens (padding included)."""
    x = _values(s, name)[blk, off].float()
    return x * scale if s["f8"] else x


def _where(s, T):
    """Block and offset of token t of every sequence, t < T ([B, T]; padding points at block 0)."""
    t = torch.arange(T, device=s["tables"].device)
    blk = s["tables"][:, torch.div(t, s["bs"], rounding_mode="floor").clamp(max=s["tables"].shape[1] - 1)]
    return blk.clamp(min=0).long(), (t % s["bs"])[None].expand(blk.shape[0], T)


def _decode(s):
    q, lens = s["q"].float(), s["lens"].long()
    B, Hq, D = q.shape
    Hkv = s["Hkv"]
    G = Hq // Hkv
    T = s["tables"].shape[1] * s["bs"]
    blk, off = _where(s, T)
    t = torch.arange(T, device=q.device)
    there = t[None] < lens[:, None]
    k = _gathered(s, "k_cache", blk, off, s.get("k_scale", 1.0))
    sc = torch.matmul(q.view(B, Hkv, G, D), k.permute(0, 2, 3, 1)) * s["scale"]
    del k
    sc = sc.masked_fill(~there[:, None, None], -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    v = _gathered(s, "v_cache", blk, off, s.get("v_scale", 1.0))
    v = v.masked_fill(~there[:, :, None, None], 0)
    s["out"].copy_(torch.matmul(p, v.permute(0, 2, 1, 3)).reshape(B, Hq, D))
    had = s["weights"][blk, :, off]  # [B, T, Hkv]
    had = had * (t[None] != lens[:, None] - 1)[:, :, None]
    new = had + p.sum(2).permute(0, 2, 1)
    s["weights"][blk[there], :, off[there]] = new[there]
    return [s["out"], s["weights"]]


def _prompt(s):
    dev = s["q"].device
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    ql, kl = cu_q.diff(), cu_k.diff()
    B, Hkv, D = ql.shape[0], s["Hkv"], s["D"]
    G = s["q"].shape[1] // Hkv
    Q, T = s["max_q"], s["tables"].shape[1] * s["bs"]
    i, t = torch.arange(Q, device=dev), torch.arange(T, device=dev)
    real = i[None] < ql[:, None]  # [B, Q]
    row = (cu_q[:-1, None] + i[None]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(B, Q, Hkv, G, D)
    blk, off = _where(s, T)
    k = _gathered(s, "k_cache", blk, off, 1.0)
    pos = (kl - ql)[:, None] + i[None]
    sees = (t[None, None] <= pos[:, :, None]) & real[:, :, None]  # [B, Q, T]
    sc = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, D), k.permute(0, 2, 3, 1))
    del k
    sc = (sc * s["scale"]).view(B, Hkv, G, Q, T).masked_fill_(~sees[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = sc.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    p = p.div_(p.sum(-1, keepdim=True).clamp(min=1e-30))
    v = _gathered(s, "v_cache", blk, off, 1.0)
    there = t[None] < kl[:, None]
    v = v.masked_fill(~there[:, :, None, None], 0)
    o = torch.matmul(p.view(B, Hkv, G * Q, T), v.permute(0, 2, 1, 3)).view(B, Hkv, G, Q, D)
    s["out"][row[real]] = o.permute(0, 3, 1, 2, 4).reshape(B, Q, Hkv * G, D)[real].to(s["out"].dtype)
    observing = real & (i[None] >= (ql - s["window"])[:, None]) if s["window"] else real
    got = torch.matmul(observing[:, None, None, :].float().expand(B, Hkv, G, Q).reshape(B, Hkv, 1, G * Q), p.view(B, Hkv, G * Q, T))
    had = s["weights"][blk, :, off] * (t[None] < (kl - ql)[:, None])[:, :, None]
    new = had + got[:, :, 0].permute(0, 2, 1)
    s["weights"][blk[there], :, off[there]] = new[there]
    return [s["out"], s["weights"]]


def _evict(s):
    lens = s["lens"].long()
    Hkv, budget, recent = s["Hkv"], s["budget"], s["recent"]
    T = s["tables"].shape[1] * s["bs"]
    blk, off = _where(s, T)
    t = torch.arange(T, device=lens.device)
    w = s["weights"][blk, :, off].permute(0, 2, 1)  # [B, Hkv, T]
    # the recent tokens before all others, padding behind all; a stable sort keeps the lowest index on ties
    rank = w.masked_fill((t[None] >= (lens - recent)[:, None])[:, None], math.inf)
    rank = rank.masked_fill((t[None] >= lens[:, None])[:, None], -math.inf)
    keep = min(budget, T)
    kept = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep].sort(dim=-1).values  # [B, Hkv, keep]
    cut = (lens > budget)[:, None, None].expand_as(kept)
    b = torch.arange(lens.shape[0], device=lens.device)[:, None, None].expand_as(kept)
    h = torch.arange(Hkv, device=lens.device)[None, :, None].expand_as(kept)
    to = torch.arange(keep, device=lens.device)[None, None].expand_as(kept)
    b, h, to, kept = b[cut], h[cut], to[cut], kept[cut]
    for name in ("k_cache", "v_cache"):
        s[name][blk[b, to], off[b, to], h] = s[name][blk[b, kept], off[b, kept], h]
    s["weights"][blk[b, to], h, off[b, to]] = s["weights"][blk[b, kept], h, off[b, kept]]
    s["out_lens"].copy_(lens.clamp(max=budget))
    return [_values(s, "k_cache"), _values(s, "v_cache"), s["weights"], s["out_lens"]]


# ------------------------------------------------------------------- the work


def work(case):
    """Bytes and operations one pass cannot do without."""
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    if case["op"] == "prompt":
        ql, kl = (x.double() for x in _lengths(case))
        pairs = float((ql * (kl - ql) + ql * (ql + 1) / 2).sum())
        tokens, new = float(kl.sum()), float(ql.sum())
        seen = float((kl - ql).sum())
        byte = tokens * Hkv * (2 * D * 2 + 4) + seen * Hkv * 4 + 2 * new * case["Hq"] * D * 2
        return {"bytes": byte, "flops": 4.0 * D * case["Hq"] * pairs}
    n = _lengths(case)[1].double()
    tokens, e = float(n.sum()), 1 if case["f8"] else 2
    if case["op"] == "decode":
        return {"bytes": tokens * Hkv * (2 * D * e + 8) + 4.0 * B * case["Hq"] * D, "flops": 4.0 * tokens * case["Hq"] * D}
    # weights of the sequences that are cut are read, and what is kept moves (all but a short run at the front)
    cut = n[n > case["budget"]]
    moved = float(cut.numel()) * case["budget"] * Hkv
    return {"bytes": float(cut.sum()) * Hkv * 4 + moved * (2 * 2 * D * e + 4) + 8.0 * B, "flops": 0.0}


# ------------------------------------------------------- the definition, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    bs, Hkv, D = s["bs"], s["Hkv"], s["D"]
    tables = s["tables"].cpu()
    wt = s["weights"].double()

    def slots(b, n):
        t = torch.arange(n)
        return (tables[b, t // bs].long() * bs + t % bs).cuda()

    kv = {}
    for name in ("k", "v"):
        x = s[name + "_cache"]
        kv[name] = (x.view(torch.float8_e4m3fn) if s["f8"] else x).reshape(-1, Hkv, D)
    flat = wt.permute(0, 2, 1).reshape(-1, Hkv).contiguous()  # [slot, Hkv]

    def back():
        return flat.view(-1, bs, Hkv).permute(0, 2, 1).contiguous()

    if case["op"] == "evict":
        if sum(_lengths(case)[1].tolist()) * Hkv * D > 1 << 31:
            return None
        k, v = kv["k"].double(), kv["v"].double()
        lens = s["lens"].tolist()
        for b, n in enumerate(lens):
            if n <= case["budget"]:
                continue
            at, old = slots(b, n), n - case["recent"]
            for h in range(Hkv):
                heavy = torch.argsort(-flat[at[:old], h], stable=True)[: case["budget"] - case["recent"]]
                kept = torch.cat([heavy.sort().values, torch.arange(old, n, device="cuda")])
                src, dst = at[kept], at[: case["budget"]]
                k[dst, h], v[dst, h], flat[dst, h] = k[src, h], v[src, h], flat[src, h]
        shape = s["k_cache"].shape
        return [k.view(shape), v.view(shape), back(), torch.tensor([min(n, case["budget"]) for n in lens], dtype=torch.int32)]

    G = case["Hq"] // Hkv
    ks, vs = s.get("k_scale", 1.0), s.get("v_scale", 1.0)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "decode":
        for b, n in enumerate(s["lens"].tolist()):
            at = slots(b, n)
            K, V = kv["k"][at].double() * ks, kv["v"][at].double() * vs
            q = s["q"][b].double().view(Hkv, G, D)
            p = torch.softmax(torch.einsum("hgd,thd->hgt", q, K) * s["scale"], -1)
            out[b] = torch.einsum("hgt,thd->hgd", p, V).reshape(-1, D)
            flat[at[n - 1]] = 0
            flat[at] += p.sum(1).T
        return [out, back()]
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(case["B"]):
        ql, kl = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        at, base = slots(b, kl), kl - ql
        flat[at[base:]] = 0
        K, V = kv["k"][at].double(), kv["v"][at].double()
        i0 = max(0, ql - case["window"]) if case["window"] else 0
        for h in range(Hkv):
            for r in range(0, ql, 1024):
                q = s["q"][cq[b] + r: cq[b] + min(ql, r + 1024), h * G: (h + 1) * G].double()
                i = torch.arange(r, r + q.shape[0], device="cuda")
                sc = torch.einsum("igd,td->igt", q, K[:, h]) * s["scale"]
                sc.masked_fill_(torch.arange(kl, device="cuda")[None, None] > (base + i)[:, None, None], -math.inf)
                p = torch.softmax(sc, -1)
                out[cq[b] + r: cq[b] + r + q.shape[0], h * G: (h + 1) * G] = torch.einsum("igt,td->igd", p, V[:, h])
                flat[at, h] += p[i >= i0].sum((0, 1))
    return [out, back()]
