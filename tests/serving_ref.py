"""Plain float64 definitions of rotary positions, of a serving step's
book-keeping and of attention over a cache, for the tests (CPU torch, none of
the library's code)."""
from __future__ import annotations

import math

import torch


def frequencies(rot, *, base=10000.0, scaling="none", factor=1.0, context=8192, low=0.0, high=0.0,
                magnitude=0.0):
    """([rot / 2] radians a position, magnitude)."""
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    if not low and not high:
        low, high = 1.0, 32.0 if scaling == "ramp" else 4.0
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "bands":
            n = context * f / (2 * math.pi)
            if n <= low:
                f /= factor
            elif n < high:
                w = (n - low) / (high - low)
                f = w * f + (1 - w) * f / factor
        elif scaling == "ramp":
            at = [rot * math.log(context / (2 * math.pi * n)) / (2 * math.log(base)) for n in (high, low)]
            a, z = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
            w = 1 - min(1.0, max(0.0, (i - a) / max(z - a, 0.001)))
            f = w * f + (1 - w) * f / factor
        out.append(f)
    if not magnitude:
        magnitude = 0.1 * math.log(factor) + 1.0 if scaling == "ramp" else 1.0
    return torch.tensor(out, dtype=torch.float64), magnitude


def rope(x, pos, rot, layout, *, backward=False, **scaling):
    """x [..., H, D] at pos [...] -> (float64 result, bound on its fp32 error).

    The bound per element of a pair is (|x_a| + |x_b|) m times: 2^-24 each for
    the sine's own error and its scaled argument's, for its product with m, for
    the product with x and for the sum (5 roundings, 8 allowed), and 2^-50
    |pos f| for the frequency's own roundings in 64 bits on both sides."""
    f, m = frequencies(rot, **scaling)
    x = x.double()
    t = pos.double()[..., None, None] * f
    c, s = m * torch.cos(t), m * torch.sin(t) * (-1 if backward else 1)
    if layout == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    size = (a.abs() + b.abs()) * m * (8 * 2.0 ** -24 + t.abs() * 2.0 ** -50)
    y, e = x.clone(), torch.zeros_like(x)
    for out, (u, v) in ((y, (a * c - b * s, a * s + b * c)), (e, (size, size))):
        if layout == "half":
            out[..., : rot // 2], out[..., rot // 2: rot] = u, v
        else:
            out[..., 0:rot:2], out[..., 1:rot:2] = u, v
    return y, e


def plan(q_lens, kv_lens, table, free, head, page, max_tokens):
    """The lists fl_kv_plan writes (table is copied)."""
    table = [list(r) for r in table]
    kv_out, cu, positions, slots, short = [], [0], [], [], False
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        n, kv = max(n, 0), max(kv, 0)
        for p in range(-(-kv // page), -(-(kv + n) // page)):
            got = free[head] if head < len(free) else -1
            head += 1
            if p < len(table[b]):
                table[b][p] = got
        for pos in range(kv, kv + n):
            got = table[b][pos // page] if pos // page < len(table[b]) else -1
            short |= got < 0
            positions.append(pos)
            slots.append(got * page + pos % page if got >= 0 else -1)
        kv_out.append(kv + n)
        cu.append(cu[-1] + n)
    tail = [-1] * max(0, max_tokens - len(positions))
    return dict(table=table, kv_out=kv_out, cu_q=cu, head=head, positions=(positions + tail)[:max_tokens],
                slots=(slots + tail)[:max_tokens], short=short)


def chunk_rows(q, k, v, n_pos, *, causal=True, window=0, softcap=0.0, scale=None):
    """One request: q [n, Hq, D], keys and values [L, Hk, D] (all cached keys;
    rows that no query sees are not touched) -> float64 O [n, Hq, D], LSE
    [Hq, n] and a bound on the error of a bf16 O.

    The bound: each weight is rounded to bf16 (half a step, 2^-8 of it) and the
    weights are normalised by their rounded sum, so O moves by at most
    2^-8 sum_j w_j |v_j - O| <= 2^-8 sqrt(sum_j w_j v_j^2 - O^2) (to first
    order; 2% on top for the second), and its own rounding adds 2^-8 |O|.
    2e-5 covers the fp32 scores."""
    n, Hq, D = q.shape
    L, Hk = k.shape[0], k.shape[1]
    G = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(n, Hq, D, dtype=torch.float64)
    tol = torch.full((n, Hq, D), 2e-5, dtype=torch.float64)
    lse = torch.full((Hq, n), -math.inf, dtype=torch.float64)
    for s in range(n):
        pos = L - n + s if n_pos is None else n_pos[s]
        hi = min(L, pos + 1) if causal else L
        lo = max(0, pos - window + 1) if window else 0
        if hi <= lo:
            continue
        for h in range(Hk):
            kk, vv = k[lo:hi, h].double(), v[lo:hi, h].double()
            z = q[s, h * G:(h + 1) * G].double() @ kk.T * scale
            if softcap:
                z = softcap * torch.tanh(z / softcap)
            w = torch.softmax(z, -1)
            o = w @ vv
            out[s, h * G:(h + 1) * G] = o
            spread = (w @ vv ** 2 - o ** 2).clamp(min=0).sqrt()
            tol[s, h * G:(h + 1) * G] += 2.0 ** -8 * (o.abs() + 1.02 * spread)
            lse[h * G:(h + 1) * G, s] = torch.logsumexp(z, -1)
    return out, lse, tol
