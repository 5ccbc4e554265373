"""Workloads of the serving and rotary-position operators.

Each case is one call of one operator, as a serving loop or a training step makes it: rotary
positions (``fl_rope``), the step's block tables and slot maps (``fl_kv_plan``), new keys and values
into the paged cache (``fl_kv_append``) and attention of the new tokens over that cache
(``fl_attn_chunk``).  ``run`` computes it with elementary torch operations, or with the library's
kernels where ``own`` is true; ``exact`` gives the definition in 64 bits.

The head shapes are those of the repository's workloads (32 query heads over 8 KV heads of 64, 16 over
2, 16 over 16) and a few generic ones.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEVICE = "cuda"

# ------------------------------------------------------------------ cases


def listed():
    return [
        # one step of a serving loop: 64 requests, a new token each, far into long contexts
        dict(name="rope_step", op="rope", B=1, S=64, Hq=32, Hk=8, D=64, rot=64, layout="half",
             dtype="bf16", base=500000.0, scaling="bands", factor=32.0, context=8192, far=131072,
             explicit=True, backward=False),
        # q and k of a training step (the MHA sweep's S = 2048)
        dict(name="rope_train", op="rope", B=8, S=2048, Hq=16, Hk=16, D=64, rot=64, layout="half",
             dtype="bf16", base=10000.0, scaling="none", factor=1.0, context=2048, far=0,
             explicit=False, backward=False),
        # the backward of a quarter-rotated, interleaved, long-context layer kept in fp32
        dict(name="rope_grad_fp32", op="rope", B=4, S=4095, Hq=16, Hk=2, D=128, rot=32,
             layout="interleaved", dtype="fp32", base=10000.0, scaling="ramp", factor=16.0,
             context=4096, far=1000000, explicit=True, backward=True),
        # the book-keeping of a decode step: a token for each of 256 requests
        dict(name="plan_step", op="plan", B=256, long=0, chunk=1, kv_hi=8192, page=256, lens=1, pad=0),
        # the same for a large batch with many prompts in it, padded for a captured graph
        dict(name="plan_prompts", op="plan", B=2000, long=200, chunk=600, kv_hi=4000, page=16, lens=2,
             pad=777),
        # new keys of a decode step, rotated on their way into the cache
        dict(name="append_step", op="append", B=64, long=0, chunk=1, kv_hi=8192, page=256, Hq=32, Hk=8,
             D=64, rot=64, layout="half", base=500000.0, scaling="bands", factor=32.0, context=8192,
             lens=3, pad=0),
        # a step of long prompts
        dict(name="append_prompts", op="append", B=24, long=12, chunk=1500, kv_hi=6000, page=64, Hq=16,
             Hk=2, D=128, rot=128, layout="half", base=10000.0, scaling="none", factor=1.0,
             context=8192, lens=4, pad=100),
        # the smallest call: one token of one conversation
        dict(name="chunk_one", op="chunk", B=1, long=0, chunk=1, kv_lo=777, kv_hi=777, page=16, Hq=32,
             Hk=8, D=64, softcap=0.0, causal=True, window=0, lens=5, pad=0),
        # a decode step: the repository's serving workload (64 requests, 512 to 8192 keys)
        dict(name="chunk_tokens", op="chunk", B=64, long=0, chunk=1, kv_lo=512, kv_hi=8192, page=256,
             Hq=32, Hk=8, D=64, softcap=0.0, causal=True, window=0, lens=6, pad=0),
        # prompts among decoding requests, softcapped, an idle request and padding rows
        dict(name="chunk_mixed", op="chunk", B=33, long=3, chunk=500, kv_lo=1, kv_hi=4096, page=64,
             Hq=32, Hk=8, D=64, softcap=20.0, causal=True, window=0, lens=7, pad=64),
        # the last chunk of a long prompt
        dict(name="chunk_long", op="chunk", B=1, long=1, chunk=4096, kv_lo=16384, kv_hi=16384, page=128,
             Hq=32, Hk=8, D=64, softcap=0.0, causal=True, window=0, lens=8, pad=0),
        # sliding-window layers of wide heads
        dict(name="chunk_window_wide", op="chunk", B=4, long=4, chunk=1400, kv_lo=1400, kv_hi=6000,
             page=32, Hq=16, Hk=2, D=128, softcap=0.0, causal=True, window=1024, lens=9, pad=0),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((32, 8), (16, 2), (16, 16), (8, 8), (6, 2), (14, 2), (12, 12), (5, 1))


def draw(rng):
    op = rng.choice(("rope", "plan", "append", "chunk", "chunk"))
    lens = rng.randrange(1 << 20)
    Hq, Hk = rng.choice(HEADS)
    if op == "rope":
        D = rng.choice((32, 64, 80, 128))
        S = _spread(rng, 1, 4096)
        B = min(rng.choice((1, 2, 3, 8)), max(1, 16384 // S))
        scaling = rng.choice(("none", "linear", "base", "bands", "ramp"))
        return dict(op=op, B=B, S=S, Hq=min(Hq, 16), Hk=min(Hk, 16), D=D,
                    rot=rng.choice((D, D // 2, D // 2 + 4)), layout=rng.choice(("half", "interleaved")),
                    dtype=rng.choice(("bf16", "fp32")), base=rng.choice((10000.0, 500000.0)),
                    scaling=scaling, factor=1.0 if scaling == "none" else rng.choice((4.0, 8.0, 32.0)),
                    context=rng.choice((2048, 8192)), far=_spread(rng, 1, 1000000),
                    explicit=rng.random() < 0.5, backward=rng.random() < 0.5)
    if op == "plan":
        B = _spread(rng, 1, 2000)
        long = rng.randrange(0, min(B, 200) + 1)
        return dict(op=op, B=B, long=long, chunk=_spread(rng, 1, 600), kv_hi=_spread(rng, 700, 8000),
                    page=rng.choice((16, 32, 64, 128, 256)), lens=lens, pad=rng.choice((0, 1, 500)))
    if op == "append":
        B = _spread(rng, 1, 64)
        D = rng.choice((64, 128))
        return dict(op=op, B=B, long=rng.randrange(0, min(B, 12) + 1), chunk=_spread(rng, 1, 1500),
                    kv_hi=_spread(rng, 1600, 6000), page=rng.choice((16, 32, 64, 128, 256)),
                    Hq=min(Hq, 16), Hk=min(Hk, 16), D=D, rot=rng.choice((0, D, D // 2)),
                    layout=rng.choice(("half", "interleaved")), base=10000.0, scaling="linear",
                    factor=4.0, context=4096, lens=lens, pad=rng.choice((0, 33)))
    B = _spread(rng, 1, 48)
    kv_hi = _spread(rng, 16, 8192)
    chunk = min(_spread(rng, 1, 1500), kv_hi, max(1, int(3e8 / (B * Hq * kv_hi))))
    causal = rng.random() < 0.8
    return dict(op="chunk", B=B, long=rng.randrange(0, min(B, 8) + 1), chunk=chunk,
                kv_lo=max(1, kv_hi // 8), kv_hi=kv_hi, page=rng.choice((16, 32, 64, 128, 256)), Hq=Hq,
                Hk=Hk, D=rng.choice((64, 128)), softcap=rng.choice((0.0, 0.0, 20.0)), causal=causal,
                window=rng.choice((0, 0, 100, 1024)) if causal else 0, lens=lens,
                pad=rng.choice((0, 5)))


# ------------------------------------------------------------------ request lengths


def _lengths(case):
    """(new tokens, cached tokens before the step) of each request: the first `long` bring up to
    `chunk` tokens, the others one; request B // 2 of a batch of at least 3 with `pad` is idle."""
    r = random.Random("lengths/%d" % case["lens"])
    q, kv = [], []
    for b in range(case["B"]):
        n = 1
        if b < case["long"]:
            n = case["chunk"] if b == 0 else r.randint(max(1, case["chunk"] // 3), case["chunk"])
        total = r.randint(case.get("kv_lo", 1), case["kv_hi"])
        if case["pad"] and case["B"] >= 3 and b == case["B"] // 2:
            n = 0
        q.append(n)
        kv.append(max(0, total - n))
    return q, kv


def _scaled(case):
    """What make_rope_table takes."""
    return dict(base=case["base"], layout=case["layout"], scaling=case["scaling"],
                factor=case["factor"], context=case["context"])


# ------------------------------------------------------------------ state


def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32).to(dtype)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEVICE)


def _paged(case, gen, with_new):
    """The block table of a batch over a shuffled pool (three spare pages), with the pages of the
    new tokens in it or still on the free list."""
    q, kv = _lengths(case)
    page = case["page"]
    old = [-(-k // page) for k in kv]
    new = [-(-(k + n) // page) for n, k in zip(q, kv)]
    width = max(new) + 1
    total = sum(new) + 3
    perm = torch.randperm(total, generator=gen, device=DEVICE).to(torch.int32)
    have = _ints(new if with_new else old)
    start = torch.cumsum(have, 0) - have
    col = torch.arange(width, device=DEVICE)
    at = (start[:, None] + col[None]).clamp(max=total - 1).long()
    table = torch.where(col[None] < have[:, None], perm[at], torch.full_like(perm[at], -1))
    return q, kv, table.contiguous(), perm[int(sum(new if with_new else old)):].contiguous(), total


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "rope":
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["q"] = _normal((case["B"], case["S"], case["Hq"], case["D"]), gen, dtype)
        s["k"] = _normal((case["B"], case["S"], case["Hk"], case["D"]), gen, dtype)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        if case["explicit"]:
            s["positions"] = torch.randint(0, max(1, case["far"]), (case["B"], case["S"]), generator=gen,
                                           device=DEVICE, dtype=torch.int32)
        else:
            s["positions"] = None
    elif op == "plan":
        q, kv, s["table"], s["free"], s["pages"] = _paged(case, gen, False)
        s["q_lens"], s["kv_lens"] = _ints(q), _ints(kv)
        s["T"] = sum(q) + case["pad"]
        s["free_head"] = _ints([0])
        for name, n, t in (("kv_out", case["B"], torch.int32), ("cu_q", case["B"] + 1, torch.int32),
                           ("positions", s["T"], torch.int32), ("slots", s["T"], torch.int64),
                           ("head_out", 1, torch.int32)):
            s[name] = torch.zeros(n, dtype=t, device=DEVICE)
    else:
        q, kv, s["table"], _, pages = _paged(case, gen, True)
        T = sum(q) + case["pad"]
        pool = (pages, case["page"], case["Hk"], case["D"])
        s["q"] = _normal((T, case["Hq"], case["D"]), gen)
        s["k_cache"], s["v_cache"] = _normal(pool, gen), _normal(pool, gen)
        cu = [0]
        for n in q:
            cu.append(cu[-1] + n)
        if op == "append":
            s["k"], s["v"] = (_normal((T, case["Hk"], case["D"]), gen) for _ in "kv")
            s["q_out"] = torch.zeros_like(s["q"])
            n, before = _ints(q, torch.int64), _ints(kv, torch.int64)
            seq = torch.repeat_interleave(torch.arange(case["B"], device=DEVICE), n)
            pos = torch.arange(cu[-1], device=DEVICE) - _ints(cu[:-1], torch.int64)[seq] + before[seq]
            slots = s["table"][seq, pos // case["page"]].long() * case["page"] + pos % case["page"]
            tail = torch.full((case["pad"],), -1, dtype=torch.int64, device=DEVICE)
            s["positions"] = torch.cat((pos, tail)).to(torch.int32)
            s["slots"] = torch.cat((slots, tail))
        else:
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
    if case["op"] in ("rope", "append"):
        s["rope"] = fa.make_rope_table(case["rot"], **_scaled(case)) if case["rot"] else None
    elif case["op"] == "plan":
        s["desc"] = fa.make_kv_plan_desc(s["q_lens"], s["kv_lens"], s["free"], s["free_head"], s["table"],
                                         s["kv_out"], s["cu_q"], s["positions"], s["slots"],
                                         s["head_out"], page_size=case["page"])
    else:
        s["desc"] = fa.make_chunk_desc(s["cu_q"], s["kv_lens"], s["table"], s["max_kv"],
                                       score_mod="softcap" if case["softcap"] else "none",
                                       softcap=case["softcap"], causal=case["causal"],
                                       window=case["window"])
        s["ws"] = torch.empty(fa.fl_attn_chunk_workspace_size(s["q"], s["k_cache"], s["desc"]),
                              dtype=torch.uint8, device=DEVICE)


# ------------------------------------------------------------------ one pass


def run(s):
    op = s["case"]["op"]
    if own:
        import attention_variant_gb300 as fa
        if op == "rope":
            fa.fl_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["rope"], positions=s["positions"],
                       backward=s["case"]["backward"])
            return {"q": s["q_out"], "k": s["k_out"]}
        if op == "plan":
            fa.fl_kv_plan(s["desc"])
            return {n: s[n] for n in ("kv_out", "cu_q", "positions", "slots", "head_out", "table")}
        if op == "append":
            fa.fl_kv_append(s["q"], s["k"], s["v"], s["q_out"], s["k_cache"], s["v_cache"], s["slots"],
                            rope=s["rope"], positions=s["positions"])
            return {n: s[n] for n in ("q_out", "k_cache", "v_cache")}
        fa.fl_attn_chunk(s["q"], s["k_cache"], s["v_cache"], s["out"], s["lse"], s["desc"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    return {"rope": _rope, "plan": _plan, "append": _append, "chunk": _chunk}[op](s)


def _frequencies(case):
    """(radians a position of each rotated pair, factor on cos and sin) of a case's scaling."""
    rot, base, factor, context = case["rot"], case["base"], case["factor"], case["context"]
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=DEVICE)
    kind, magnitude = case["scaling"], 1.0
    if kind == "base":
        base = base * factor ** (rot / (rot - 2))
    f = torch.exp(-math.log(base) * i / rot)
    if kind == "linear":
        f = f / factor
    elif kind == "bands":  # long waves slowed down, short ones kept, a blend between 1 and 4 turns
        turns = context * f / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = keep * f + (1 - keep) * f / factor
    elif kind == "ramp":  # the same by the pair's index, between 32 turns and 1 turn in `context`
        at = [rot * math.log(context / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        slow = ((i / 2 - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = (1 - slow) * f + slow * f / factor
        magnitude = 0.1 * math.log(factor) + 1.0
    return f, magnitude


def _rotate(x, pos, case, backward):
    """Rotary positions of x [..., H, D] at pos [...], in 32 bits on angles taken in 64."""
    rot = case["rot"]
    x = x.float()
    if not rot:
        return x
    f, magnitude = _frequencies(case)
    angle = (pos.double()[..., None] * f)[..., None, :]
    c, s = (torch.cos(angle) * magnitude).float(), (torch.sin(angle) * magnitude).float()
    if backward:
        s = -s
    if case["layout"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        return torch.cat((a * c - b * s, a * s + b * c, x[..., rot:]), -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    y = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _rope(s):
    case = s["case"]
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(case["S"], device=DEVICE).expand(case["B"], case["S"])
    for n in "qk":
        s[n + "_out"].copy_(_rotate(s[n], pos, case, case["backward"]))
    return {"q": s["q_out"], "k": s["k_out"]}


def _plan(s):
    page, T, B = s["case"]["page"], s["T"], s["case"]["B"]
    n, kv = s["q_lens"].long(), s["kv_lens"].long()
    end = torch.cumsum(n, 0)
    have, need = (kv + page - 1) // page, (kv + n + page - 1) // page
    fresh = need - have
    first = torch.cumsum(fresh, 0) - fresh + s["free_head"].long()
    col = torch.arange(s["table"].shape[1], device=DEVICE)[None]
    at = (first[:, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    taken = (col >= have[:, None]) & (col < need[:, None])
    s["table"].copy_(torch.where(taken, s["free"][at], s["table"]))
    t = torch.arange(T, device=DEVICE)
    b = torch.searchsorted(end, t, right=True).clamp(max=B - 1)
    live = t < end[-1]
    pos = torch.where(live, t - (end - n)[b] + kv[b], torch.full_like(t, -1))
    p = s["table"][b, (pos.clamp(min=0) // page).clamp(max=s["table"].shape[1] - 1)].long()
    s["kv_out"].copy_(kv + n)
    s["cu_q"][1:].copy_(end)
    s["positions"].copy_(pos)
    s["slots"].copy_(torch.where(live, p * page + pos % page, pos))
    s["head_out"].copy_(s["free_head"] + fresh.sum())
    return {n: s[n] for n in ("kv_out", "cu_q", "positions", "slots", "head_out", "table")}


def _append(s):
    case = s["case"]
    live = s["slots"] >= 0
    at, pos = s["slots"][live], s["positions"][live]
    rows = lambda cache: cache.view(-1, case["Hk"], case["D"])  # noqa: E731
    rows(s["k_cache"])[at] = _rotate(s["k"][live], pos, case, False).to(torch.bfloat16)
    rows(s["v_cache"])[at] = s["v"][live]
    s["q_out"][live] = _rotate(s["q"][live], pos, case, False).to(torch.bfloat16)
    return {n: s[n] for n in ("q_out", "k_cache", "v_cache")}


def _chunk(s):
    case = s["case"]
    B, Hq, Hk, D, N = case["B"], case["Hq"], case["Hk"], case["D"], s["max_q"]
    cu, L = s["cu_q"].long(), s["kv_lens"].long()
    n = cu[1:] - cu[:-1]
    keys = -(-s["max_kv"] // case["page"]) * case["page"]
    pages = s["table"][:, : keys // case["page"]].clamp(min=0).long()
    j = torch.arange(keys, device=DEVICE)
    held = j < L[:, None]
    k, v = (torch.where(held[..., None, None], c[pages].view(B, keys, Hk, D), 0).float().transpose(1, 2)
            for c in (s["k_cache"], s["v_cache"]))
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
    op = case["op"]
    if op == "rope":
        size = 2 if case["dtype"] == "bf16" else 4
        tokens = case["B"] * case["S"]
        x = tokens * (case["Hq"] + case["Hk"]) * case["D"]
        return {"bytes": 2 * x * size + (4 * tokens if case["explicit"] else 0), "flops": 3 * x}
    q, kv = _lengths(case)
    T, B = sum(q), case["B"]
    if op == "plan":
        fresh = sum(-(-(k + n) // case["page"]) - -(-k // case["page"]) for n, k in zip(q, kv))
        return {"bytes": 16 * B + 8 * fresh + 12 * (T + case["pad"]) + 4 * B, "flops": 0}
    if op == "append":
        x = T * (case["Hq"] + 2 * case["Hk"]) * case["D"]
        return {"bytes": 4 * x + 12 * (T + case["pad"]), "flops": 3 * x}
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
    return {"bytes": 4 * keys * case["Hk"] * case["D"] + T * case["Hq"] * (4 * case["D"] + 4)
            + 4 * (keys // case["page"]), "flops": 4 * case["D"] * case["Hq"] * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits


def _turned(x, pos, case, backward):
    """x [N, H, D] rotated at pos [N]: each pair as a complex number times m e^(i pos f)."""
    rot = case["rot"]
    y = x.double().clone()
    for i in range(rot // 2):
        base = case["base"]
        if case["scaling"] == "base":
            base *= case["factor"] ** (rot / (rot - 2.0))
        f, m = base ** (-2.0 * i / rot), 1.0
        slow = f / case["factor"]
        if case["scaling"] == "linear":
            f = slow
        if case["scaling"] == "bands":
            wave = 2 * math.pi / f
            if wave > case["context"] / 1.0:
                f = slow
            elif wave >= case["context"] / 4.0:
                w = (case["context"] / wave - 1.0) / 3.0
                f = (1 - w) * slow + w * f
        if case["scaling"] == "ramp":
            dim = lambda turns: rot * math.log(case["context"] / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(dim(32)), 0), min(math.ceil(dim(1)), rot - 1)
            w = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f * (1 - w) + slow * w
            m = 0.1 * math.log(case["factor"]) + 1.0
        ia, ib = (i, i + rot // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
        t = pos.double() * f * (-1 if backward else 1)
        z = torch.complex(x[..., ia].double(), x[..., ib].double()) * (m * torch.polar(torch.ones_like(t), t))[:, None]
        y[..., ia], y[..., ib] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None
    if op == "rope":
        pos = s["positions"]
        if pos is None:
            pos = torch.arange(case["S"], device=DEVICE).repeat(case["B"])
        return {n: _turned(s[n].flatten(0, 1), pos.reshape(-1), case, case["backward"]).view(s[n].shape)
                for n in "qk"}
    if op == "append":
        live = torch.nonzero(s["slots"] >= 0)[:, 0]
        page, row = s["slots"][live] // case["page"], s["slots"][live] % case["page"]
        got = {n: s[n].double() for n in ("q_out", "k_cache", "v_cache")}
        got["q_out"][live] = _turned(s["q"][live], s["positions"][live], case, False)
        got["k_cache"][page, row] = _turned(s["k"][live], s["positions"][live], case, False)
        got["v_cache"][page, row] = s["v"][live].double()
        return got
    cu, L = s["cu_q"].tolist(), s["kv_lens"].tolist()
    G, page = case["Hq"] // case["Hk"], case["page"]
    out, lse = s["out"].double(), s["lse"].double()
    for b in range(case["B"]):
        t0, n = cu[b], cu[b + 1] - cu[b]
        if not n:
            continue
        keys = torch.arange(L[b], device=DEVICE)
        where = s["table"][b, keys // page].long()
        k, v = (c[where, keys % page].double() for c in (s["k_cache"], s["v_cache"]))
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
