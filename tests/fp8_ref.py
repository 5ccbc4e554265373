"""Plain definitions of the 8-bit KV cache for the tests (CPU torch, none of the library's code)."""
from __future__ import annotations

import math

import torch

FP8 = torch.float8_e4m3fn
NAN_CODE = 0x7F


def need(size):
    """The smallest power of two s >= 2^-100 with 448 s >= size."""
    e = -100
    if size > 448.0 * 2.0 ** e:
        e = math.frexp(float(size) / 448.0)[1] - 2
        while 448.0 * 2.0 ** e < size:
            e += 1
    return 2.0 ** e


def code(x, s):
    """x / s rounded to e4m3; what is not finite is NaN."""
    y = (x.double() / s).float()  # s is a power of two (exact), or any for a double's worth
    return torch.where(torch.isfinite(x), y, torch.full_like(y, math.nan)).clamp(-448, 448).to(FP8)


def append(cache, scale, x, slots):
    """x [T, Hk, D] (finite or not) into copies of cache [P, page, Hk, D] and scale [P, page / block, Hk]."""
    P, page, Hk, D = cache.shape
    block = page // scale.shape[1]
    codes, scales = cache.clone().view(-1, block, Hk, D), scale.clone().view(-1, Hk)
    by_block = {}
    for t, slot in enumerate(slots.tolist()):
        if 0 <= slot < P * page:
            by_block.setdefault(slot // block, []).append((t, slot % block))
    for b, rows in by_block.items():
        for h in range(Hk):
            v = x[[t for t, _ in rows], h]
            fine = v[torch.isfinite(v)].abs()
            s = need(fine.max().item() if fine.numel() else 0.0)
            old = float(scales[b, h])
            if any(r == 0 for _, r in rows) or not (0 < old < math.inf):
                old = 0.0
            if old:
                if s > old:
                    codes[b, :, h] = (codes[b, :, h].double() * (old / s)).float().to(FP8)
                s = max(s, old)
            scales[b, h] = s
            for t, r in rows:
                codes[b, r, h] = code(x[t, h], s)
    return codes.view(cache.shape), scales.view(scale.shape)


def values(cache, scale):
    """float64 values of a cache."""
    block = cache.shape[1] // scale.shape[1]
    return cache.double() * scale.double().repeat_interleave(block, 1)[..., None]
