"""Workloads of the 8-bit KV cache: writing it, reading it back, and attention over it.

The cache holds e4m3 codes with a scale for each block of tokens and KV head: key (page, row, h) is
code * scale[page, row // block, h].  Each case is one call, as a serving loop makes it: new keys and
values quantised into the paged cache, rotated on the way (``fl_kv_append_fp8``), tokens of the cache
read back (``fl_kv_read_fp8``), and attention of the new tokens over it (``fl_attn_chunk_fp8``).
``run`` computes it with elementary torch operations, or with the library's kernels where ``own`` is
true; ``exact`` gives the definition in 64 bits.

The head shapes are those of the repository's workloads (32 query heads over 8 KV heads of 64, 16 over
2, 16 over 16) and a few generic ones.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEVICE = "cuda"
FP8 = torch.float8_e4m3fn
TOP = 448.0   # the largest e4m3 value
LEAST = -100  # log2 of the smallest scale

# ------------------------------------------------------------------ cases


def listed():
    return [
        # new keys of a decode step: 64 requests, a token each, somewhere in a block of 16
        dict(name="append_step", op="append", B=64, long=0, chunk=1, kv_hi=8192, page=256, block=16, Hq=32,
             Hk=8, D=64, rot=64, layout="half", base=500000.0, lens=3, pad=0),
        # a step of long prompts, a scale for each page
        dict(name="append_prompts", op="append", B=24, long=12, chunk=1500, kv_hi=6000, page=64, block=64,
             Hq=16, Hk=2, D=128, rot=128, layout="half", base=10000.0, lens=4, pad=100),
        # a cached prompt of one conversation read back for a check in fp32
        dict(name="read_one", op="read", B=1, kv_hi=777, page=16, block=16, Hk=8, D=64, dtype="fp32", lens=5,
             pad=0),
        # the caches of a batch read back to bf16
        dict(name="read_batch", op="read", B=40, kv_hi=4000, page=128, block=32, Hk=8, D=64, dtype="bf16",
             lens=6, pad=33),
        # the smallest call: one token of one conversation
        dict(name="chunk_one", op="chunk", B=1, long=0, chunk=1, kv_lo=777, kv_hi=777, page=16, block=16,
             Hq=32, Hk=8, D=64, softcap=0.0, causal=True, window=0, lens=5, pad=0),
        # a decode step: the repository's serving workload (64 requests, 512 to 8192 keys)
        dict(name="chunk_tokens", op="chunk", B=64, long=0, chunk=1, kv_lo=512, kv_hi=8192, page=256,
             block=16, Hq=32, Hk=8, D=64, softcap=0.0, causal=True, window=0, lens=6, pad=0),
        # a decode step of wide heads, two drafted tokens for some requests
        dict(name="chunk_drafts_wide", op="chunk", B=48, long=16, chunk=2, kv_lo=4096, kv_hi=8192, page=64,
             block=64, Hq=16, Hk=2, D=128, softcap=0.0, causal=True, window=0, lens=10, pad=0),
        # prompts among decoding requests, softcapped, an idle request and padding rows
        dict(name="chunk_mixed", op="chunk", B=33, long=3, chunk=500, kv_lo=1, kv_hi=4096, page=64, block=32,
             Hq=32, Hk=8, D=64, softcap=20.0, causal=True, window=0, lens=7, pad=64),
        # the last chunk of a long prompt
        dict(name="chunk_long", op="chunk", B=1, long=1, chunk=4096, kv_lo=16384, kv_hi=16384, page=128,
             block=128, Hq=32, Hk=8, D=64, softcap=0.0, causal=True, window=0, lens=8, pad=0),
        # sliding-window layers of wide heads
        dict(name="chunk_window_wide", op="chunk", B=4, long=4, chunk=1400, kv_lo=1400, kv_hi=6000, page=32,
             block=16, Hq=16, Hk=2, D=128, softcap=0.0, causal=True, window=1024, lens=9, pad=0),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((32, 8), (16, 2), (16, 16), (8, 8), (6, 2), (14, 2), (12, 12), (5, 1))
PAGES = (16, 32, 64, 128, 256)


def draw(rng):
    op = rng.choice(("append", "read", "chunk", "chunk"))
    lens = rng.randrange(1 << 20)
    Hq, Hk = rng.choice(HEADS)
    D = rng.choice((64, 128))
    page = rng.choice(PAGES)
    block = rng.choice([b for b in PAGES if b <= page])
    same = dict(op=op, page=page, block=block, Hk=Hk, D=D, lens=lens)
    if op == "read":
        return dict(same, B=_spread(rng, 1, 40), kv_hi=_spread(rng, 1, 4000), dtype=rng.choice(("bf16", "fp32")),
                    Hk=min(Hk, 8), pad=rng.choice((0, 5)))
    if op == "append":
        B = _spread(rng, 1, 64)
        return dict(same, B=B, long=rng.randrange(0, min(B, 12) + 1), chunk=_spread(rng, 1, 1500),
                    kv_hi=_spread(rng, 1600, 6000), Hq=min(Hq, 16), rot=rng.choice((0, D, D // 2)),
                    layout=rng.choice(("half", "interleaved")), base=10000.0, pad=rng.choice((0, 33)))
    B = _spread(rng, 1, 48)
    kv_hi = _spread(rng, 16, 8192)
    chunk = min(_spread(rng, 1, 1500), kv_hi, max(1, int(3e8 / (B * Hq * kv_hi))))
    causal = rng.random() < 0.8
    return dict(same, B=B, long=rng.randrange(0, min(B, 8) + 1), chunk=chunk, kv_lo=max(1, kv_hi // 8),
                kv_hi=kv_hi, Hq=Hq, softcap=rng.choice((0.0, 0.0, 20.0)), causal=causal,
                window=rng.choice((0, 0, 100, 1024)) if causal else 0, pad=rng.choice((0, 5)))


# ------------------------------------------------------------------ request lengths


def _lengths(case):
    """(new tokens, cached tokens before the step) of each request: the first `long` bring up to
    `chunk` tokens, the others one; request B // 2 of a batch of at least 3 with `pad` is idle."""
    r = random.Random("lengths/%d" % case["lens"])
    q, kv = [], []
    for b in range(case["B"]):
        n = 1
        if b < case.get("long", 0):
            n = case["chunk"] if b == 0 else r.randint(max(1, case["chunk"] // 3), case["chunk"])
        total = r.randint(case.get("kv_lo", 1), case["kv_hi"])
        if case["op"] == "read":
            n = 0
            total = case["kv_hi"] if b == 0 else total
        if case["pad"] and case["B"] >= 3 and b == case["B"] // 2:
            n = 0
        q.append(n)
        kv.append(max(0, total - n))
    return q, kv


# ------------------------------------------------------------------ state


def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32).to(dtype)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEVICE)


def _paged(case, gen):
    """The block table of a batch over a shuffled pool (three spare pages)."""
    q, kv = _lengths(case)
    page = case["page"]
    need = [-(-(k + n) // page) for n, k in zip(q, kv)]
    total = sum(need) + 3
    perm = torch.randperm(total, generator=gen, device=DEVICE).to(torch.int32)
    have = _ints(need)
    start = torch.cumsum(have, 0) - have
    col = torch.arange(max(need) + 1, device=DEVICE)
    at = (start[:, None] + col[None]).clamp(max=total - 1).long()
    table = torch.where(col[None] < have[:, None], perm[at], torch.full_like(perm[at], -1))
    return q, kv, table.contiguous(), total


def _scale_of(a):
    """The smallest power of two (from 2^LEAST on) that 448 times it is at least a."""
    m, e = torch.frexp(a.double() / TOP)
    e = torch.where(m == 0.5, e - 1, e).clamp(min=LEAST)
    return torch.ldexp(torch.ones_like(m), torch.where(a > 0, e, torch.full_like(e, LEAST))).float()


def _pool(shape, block, gen):
    """A cache of normal values, heads of different sizes: (codes, scales)."""
    pages, page, heads, D = shape
    size = torch.exp2(torch.randint(-3, 4, (heads, 1), generator=gen, device=DEVICE).float() / 2)
    x = (_normal(shape, gen, torch.float32) * size).view(pages, page // block, block, heads, D)
    scale = _scale_of(x.abs().amax((2, 4)))
    return (x / scale[:, :, None, :, None]).to(FP8).view(shape), scale


def _slots(q, kv, table, page, pad):
    """Slots and positions of tokens kv[b] .. kv[b] + q[b] - 1 of each request, padded with -1."""
    n, before = _ints(q, torch.int64), _ints(kv, torch.int64)
    seq = torch.repeat_interleave(torch.arange(len(q), device=DEVICE), n)
    first = torch.cumsum(n, 0) - n
    pos = torch.arange(sum(q), device=DEVICE) - first[seq] + before[seq]
    slots = table[seq, pos // page].long() * page + pos % page
    tail = torch.full((pad,), -1, dtype=torch.int64, device=DEVICE)
    return torch.cat((slots, tail)), torch.cat((pos, tail)).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    s = dict(case=case)
    op, page, block, Hk, D = (case[n] for n in ("op", "page", "block", "Hk", "D"))
    q, kv, s["table"], pages = _paged(case, gen)
    (s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"]) = (_pool((pages, page, Hk, D), block, gen)
                                                                 for _ in "kv")
    if op == "read":
        s["slots"], _ = _slots(kv, [0] * case["B"], s["table"], page, case["pad"])
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["k_out"], s["v_out"] = (torch.zeros((s["slots"].numel(), Hk, D), dtype=dtype, device=DEVICE)
                                  for _ in "kv")
        return s
    T = sum(q) + case["pad"]
    s["q"] = _normal((T, case["Hq"], D), gen)
    if op == "append":
        s["k"], s["v"] = (_normal((T, Hk, D), gen) for _ in "kv")
        s["q_out"] = torch.zeros_like(s["q"])
        s["slots"], s["positions"] = _slots(q, kv, s["table"], page, case["pad"])
    else:
        cu = [0]
        for n in q:
            cu.append(cu[-1] + n)
        s["cu_q"], s["kv_lens"] = _ints(cu), _ints([k + n for n, k in zip(q, kv)])
        s["max_kv"] = max(k + n for n, k in zip(q, kv))
        s["max_q"] = max(q)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((case["Hq"], T), device=DEVICE)
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program that uses the library sets up once: tables, descs and workspaces."""
    import attention_variant_gb300 as fa
    case = s["case"]
    if case["op"] == "append":
        s["rope"] = fa.make_rope_table(case["rot"], base=case["base"], layout=case["layout"]) if case["rot"] else None
    else:
        s["desc"] = fa.make_chunk_desc(s["cu_q"], s["kv_lens"], s["table"], s["max_kv"],
                                       score_mod="softcap" if case["softcap"] else "none",
                                       softcap=case["softcap"], causal=case["causal"],
                                       window=case["window"])
        s["ws"] = torch.empty(fa.fl_attn_chunk_fp8_workspace_size(s["q"], s["k_cache"], s["desc"]),
                              dtype=torch.uint8, device=DEVICE)


# ------------------------------------------------------------------ one pass

APPENDED = ("q_out", "k_cache", "v_cache", "k_scale", "v_scale")


def run(s):
    op = s["case"]["op"]
    if own:
        import attention_variant_gb300 as fa
        cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        if op == "append":
            fa.fl_kv_append_fp8(s["q"], s["k"], s["v"], s["q_out"], *cache, s["slots"], rope=s["rope"],
                                positions=s["positions"])
            return {n: s[n] for n in APPENDED}
        if op == "read":
            fa.fl_kv_read_fp8(*cache, s["slots"], s["k_out"], s["v_out"])
            return {"k": s["k_out"], "v": s["v_out"]}
        fa.fl_attn_chunk_fp8(s["q"], *cache, s["out"], s["lse"], s["desc"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    return {"append": _append, "read": _read, "chunk": _chunk}[op](s)


def _rotate(x, pos, case):
    """Rotary positions of x [n, H, D] at pos [n], in 32 bits on angles taken in 64."""
    rot = case["rot"]
    x = x.float()
    if not rot:
        return x
    f = torch.exp(-math.log(case["base"]) * torch.arange(0, rot, 2, dtype=torch.float64, device=DEVICE) / rot)
    angle = (pos.double()[:, None] * f)[:, None, :]
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    if case["layout"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        return torch.cat((a * c - b * s, a * s + b * c, x[..., rot:]), -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    y = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _quantise(cache, scale, x, at, block):
    """x [n, Hk, D] into rows `at` of a cache: a block that gets its first row starts a scale of its
    own, another's scale may grow, and then the rows that it holds are coded anew."""
    Hk, D = x.shape[1:]
    codes, scales = cache.view(-1, block, Hk, D), scale.view(-1, Hk)
    blocks, of = torch.unique(at // block, return_inverse=True)
    size = torch.zeros((blocks.numel(), Hk), device=DEVICE).index_reduce_(
        0, of, torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1), "amax")
    fresh = torch.zeros(blocks.numel(), device=DEVICE).index_reduce_(0, of, (at % block == 0).float(), "amax") > 0
    old = torch.where(fresh[:, None], 0.0, scales[blocks])
    new = torch.maximum(old, _scale_of(size))
    ratio = torch.where(old > 0, old / new, torch.ones_like(new))
    codes[blocks] = (codes[blocks].float() * ratio[:, None, :, None]).to(FP8)
    scales[blocks] = new
    cache.view(-1, Hk, D)[at] = (x / new[of][..., None]).to(FP8)


def _append(s):
    case = s["case"]
    live = s["slots"] >= 0
    at, pos = s["slots"][live], s["positions"][live]
    _quantise(s["k_cache"], s["k_scale"], _rotate(s["k"][live], pos, case), at, case["block"])
    _quantise(s["v_cache"], s["v_scale"], s["v"][live].float(), at, case["block"])
    s["q_out"][live] = _rotate(s["q"][live], pos, case).to(torch.bfloat16)
    return {n: s[n] for n in APPENDED}


def _read(s):
    case = s["case"]
    live = s["slots"] >= 0
    at = s["slots"][live]
    for n in "kv":
        codes, scales = s[n + "_cache"].view(-1, case["Hk"], case["D"]), s[n + "_scale"].view(-1, case["Hk"])
        s[n + "_out"][live] = (codes[at].float() * scales[at // case["block"]][..., None]).to(s[n + "_out"].dtype)
    return {"k": s["k_out"], "v": s["v_out"]}


def _chunk(s):
    case = s["case"]
    B, Hq, Hk, D, N = case["B"], case["Hq"], case["Hk"], case["D"], s["max_q"]
    cu, L = s["cu_q"].long(), s["kv_lens"].long()
    n = cu[1:] - cu[:-1]
    keys = -(-s["max_kv"] // case["page"]) * case["page"]
    pages = s["table"][:, : keys // case["page"]].clamp(min=0).long()
    j = torch.arange(keys, device=DEVICE)
    held = j < L[:, None]
    k, v = ((c[pages].float() * f[pages].repeat_interleave(case["block"], 2)[..., None]).view(B, keys, Hk, D)
            .transpose(1, 2) for c, f in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
    # the requests' rows, padded to the longest chunk: [B, Hk, group * N, D]
    r = torch.arange(N, device=DEVICE)
    row = (cu[:-1, None] + r).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(B, N, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D)
    z = torch.matmul(q, k.transpose(2, 3)).view(B, Hk, Hq // Hk, N, keys)
    z = z / math.sqrt(D)
    if case["softcap"]:
        z = case["softcap"] * torch.tanh(z / case["softcap"])
    pos = (L - n)[:, None] + r
    allowed = held[:, None, :].expand(B, N, keys)
    if case["causal"]:
        allowed = allowed & (j <= pos[..., None])
    if case["window"]:
        allowed = allowed & (pos[..., None] - j < case["window"])
    z = z.masked_fill(~allowed[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(m), 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hk, -1, keys), v).view(B, Hq, N, D)
    o = o / torch.where(l == 0, 1.0, l).view(B, Hq, N, 1)
    lse = (m + torch.log(l)).view(B, Hq, N)
    # back to the ragged rows; rows of no request stay as they were
    b = torch.repeat_interleave(torch.arange(B, device=DEVICE), n)
    t = torch.arange(b.numel(), device=DEVICE)
    at = t - cu[b]
    s["out"][: b.numel()] = o[b, :, at].to(torch.bfloat16)
    s["lse"][:, : b.numel()] = lse[b, :, at].t()
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ floors


def work(case):
    op, Hk, D = case["op"], case["Hk"], case["D"]
    q, kv = _lengths(case)
    if op == "read":
        x = sum(kv) * Hk
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * x * (D * (1 + size) + 4.0 / case["block"]) + 8 * (sum(kv) + case["pad"]),
                "flops": 2 * x * D}
    T = sum(q)
    if op == "append":
        blocks = sum(-(-(k + n) // case["block"]) - k // case["block"] for n, k in zip(q, kv) if n)
        return {"bytes": T * (4 * case["Hq"] + 6 * Hk) * D + 16 * blocks * Hk + 12 * (T + case["pad"]),
                "flops": T * (3 * case["Hq"] + 7 * Hk) * D}
    keys = pairs = 0
    for n, k in zip(q, kv):
        if not n:
            continue
        if not case["causal"]:
            keys, pairs = keys + k + n, pairs + n * (k + n)
            continue
        W = case["window"] or k + n
        keys += k + n - max(0, k + 1 - W)
        full = max(0, min(n, W - k - 1))  # rows that see every key before them
        pairs += full * k + full * (full + 1) // 2 + (n - full) * W
    return {"bytes": 2 * keys * Hk * (D + 4.0 / case["block"]) + T * case["Hq"] * (4 * D + 4)
            + 4 * (keys // case["page"]), "flops": 4 * D * case["Hq"] * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits


def _turned(x, pos, case):
    """x [N, H, D] rotated at pos [N]: each pair as a complex number times e^(i pos f)."""
    rot = case["rot"]
    y = x.double().clone()
    for i in range(rot // 2):
        ia, ib = (i, i + rot // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
        t = pos.double() * case["base"] ** (-2.0 * i / rot)
        z = torch.complex(x[..., ia].double(), x[..., ib].double()) * torch.polar(torch.ones_like(t), t)[:, None]
        y[..., ia], y[..., ib] = z.real, z.imag
    return y


def _coded(cache, scale, x, at, case):
    """The codes before their rounding, and the scales, after x went into rows `at`."""
    page, block, Hk = case["page"], case["block"], case["Hk"]
    codes, scales = cache.double(), scale.double().cpu()
    sizes, fresh = {}, set()
    for slot, size in zip(at.tolist(), x.abs().amax(-1).cpu()):
        b = slot // block
        sizes[b] = torch.maximum(sizes[b], size) if b in sizes else size
        if slot % block == 0:
            fresh.add(b)
    for b, size in sizes.items():
        p, i = divmod(b, page // block)
        for h in range(Hk):
            e = LEAST
            if size[h] > 0:
                e = max(LEAST, math.floor(math.log2(float(size[h]) / TOP)) - 1)
                while TOP * 2.0 ** e < float(size[h]):
                    e += 1
            s = 2.0 ** e
            if b not in fresh and float(scales[p, i, h]) > 0:
                old = float(scales[p, i, h])
                s = max(s, old)
                if s != old:
                    codes[p, i * block:(i + 1) * block, h] *= old / s
            scales[p, i, h] = s
    scales = scales.to(DEVICE)
    codes[at // page, at % page] = x / scales[at // page, at % page // block][..., None]
    return codes, scales


def exact(case, seed):
    s = prepare(case, seed)
    op, page, block = case["op"], case["page"], case["block"]
    values = lambda n, p, r: s[n + "_cache"][p, r].double() * s[n + "_scale"][p, r // block].double()[..., None]  # noqa: E731
    if op == "read":
        live = torch.nonzero(s["slots"] >= 0)[:, 0]
        got = {}
        for n in "kv":
            got[n] = s[n + "_out"].double()
            got[n][live] = values(n, s["slots"][live] // page, s["slots"][live] % page)
        return got
    if op == "append":
        live = torch.nonzero(s["slots"] >= 0)[:, 0]
        at, pos = s["slots"][live], s["positions"][live]
        got = {"q_out": s["q_out"].double()}
        got["q_out"][live] = _turned(s["q"][live], pos, case)
        for n, x in (("k", _turned(s["k"][live], pos, case)), ("v", s["v"][live].double())):
            got[n + "_cache"], got[n + "_scale"] = _coded(s[n + "_cache"], s[n + "_scale"], x, at, case)
        return got
    cu, L = s["cu_q"].tolist(), s["kv_lens"].tolist()
    G = case["Hq"] // case["Hk"]
    out, lse = s["out"].double(), s["lse"].double()
    for b in range(case["B"]):
        t0, n = cu[b], cu[b + 1] - cu[b]
        if not n:
            continue
        keys = torch.arange(L[b], device=DEVICE)
        where = s["table"][b, keys // page].long()
        k, v = values("k", where, keys % page), values("v", where, keys % page)
        for r0 in range(0, n, 1024):
            r1 = min(n, r0 + 1024)
            at = torch.arange(r0, r1, device=DEVICE) + L[b] - n
            gone = torch.zeros((r1 - r0, L[b]), dtype=torch.bool, device=DEVICE)
            if case["causal"]:
                gone |= keys[None] > at[:, None]
            if case["window"]:
                gone |= keys[None] <= at[:, None] - case["window"]
            for h in range(case["Hq"]):
                z = s["q"][t0 + r0: t0 + r1, h].double() @ k[:, h // G].T * case["D"] ** -0.5
                if case["softcap"]:
                    z = torch.tanh(z / case["softcap"]) * case["softcap"]
                z[gone] = -math.inf
                lse[h, t0 + r0: t0 + r1] = torch.logsumexp(z, -1)
                out[t0 + r0: t0 + r1, h] = torch.nan_to_num(torch.softmax(z, -1)) @ v[:, h // G]
    return {"out": out, "lse": lse}
