"""GPU parity of the 8-bit KV cache with its plain definitions: the quantising append
(fl_kv_append_fp8), reading back (fl_kv_read_fp8), attention of ragged chunks over it
(fl_attn_chunk_fp8), and serving steps of all of them."""
from __future__ import annotations

import math
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import attention_variant_gb300 as fa  # noqa: E402
from tests import fp8_ref as ref8  # noqa: E402
from tests import serving_ref as ref  # noqa: E402
from tests.fp8_ref import FP8  # noqa: E402

NAN = float("nan")


def _rand(shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _bits(x):
    return x.cpu().view(torch.uint8)


def _pool(P, page, block, Hk, D, seed):
    """A cache of random codes (no NaN) and scales."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (P, page, Hk, D), generator=g, dtype=torch.int32)
    codes[(codes & 0x7F) == 0x7F] = 0x13
    scale = torch.exp2(torch.randint(-9, 3, (P, page // block, Hk), generator=g).float())
    return codes.to(torch.uint8).view(FP8), scale


# ------------------------------------------------------------------ reading back


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
def test_read_every_code(D, dtype):
    # every code at scales from one end to the other, NaN among them
    page, Hk = 32, 3
    codes = (torch.arange(2 * page * Hk * D) % 256).to(torch.uint8).view(2, page, Hk, D)
    codes = codes.roll(7, -1).contiguous().view(FP8)
    scale = torch.exp2(torch.tensor([-100, 100, 0, -3, 8, 7, 6, 64, -64, 1, 2, 3]).float()).view(2, 2, Hk)
    out = [torch.full((2 * page, Hk, D), 7.0, dtype=dtype, device="cuda") for _ in "kv"]
    slots = torch.arange(2 * page - 1, -1, -1)
    fa.fl_kv_read_fp8(codes.cuda(), codes.flip(0).cuda(), scale.cuda(), scale.flip(0).cuda(), slots.cuda(), *out)
    want = ref8.values(codes, scale).to(dtype).view(-1, Hk, D)
    for got, w in zip(out, (want.flip(0), want.view(2, page, Hk, D).flip(0).reshape(-1, Hk, D).flip(0))):
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(w))
        assert torch.equal(got.cpu().nan_to_num(), w.nan_to_num())


@pytest.mark.parametrize("T,Hk,D,page,block", [(1, 1, 64, 16, 16), (7, 5, 128, 256, 64), (3000, 2, 64, 32, 32),
                                               (20000, 3, 64, 256, 256), (333, 8, 128, 48, 16)])
def test_read_slots_and_strides(T, Hk, D, page, block):
    P = 9
    kc, ks = _pool(P, page, block, Hk, D, 1)
    vc, vs = _pool(P, page, block, Hk, D, 2)
    g = torch.Generator().manual_seed(T)
    slots = torch.randint(0, P * page, (T,), generator=g)  # some of them twice
    if T > 3:
        slots[1], slots[T // 2], slots[-1] = -1, P * page, -(1 << 40)
    live = (slots >= 0) & (slots < P * page)
    for dtype in (torch.bfloat16, torch.float32):
        wide = torch.full((T, 2, Hk + 1, D), 7.0, dtype=dtype, device="cuda")
        fa.fl_kv_read_fp8(kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), slots.cuda(), wide[:, 0, :Hk], wide[:, 1, :Hk])
        want = torch.full((T, 2, Hk + 1, D), 7.0, dtype=dtype)
        for i, (c, s) in enumerate(((kc, ks), (vc, vs))):
            want[live, i, :Hk] = ref8.values(c, s).view(-1, Hk, D)[slots[live]].to(dtype)
        assert torch.equal(wide.cpu(), want)


# ------------------------------------------------------------------ append


def _append(k, v, slots, kc, vc, ks, vs, **kw):
    t = [x.cuda() for x in (kc, vc, ks, vs)]
    fa.fl_kv_append_fp8(None, k.cuda(), v.cuda(), None, *t, slots.cuda(), **kw)
    return [x.cpu() for x in t]


def _check_append(x_k, x_v, slots, P, page, block, seed=0):
    Hk, D = x_k.shape[1:]
    (kc, ks), (vc, vs) = _pool(P, page, block, Hk, D, seed + 1), _pool(P, page, block, Hk, D, seed + 2)
    got = _append(x_k, x_v, slots, kc, vc, ks, vs)
    for i, (c, s, x) in enumerate(((kc, ks, x_k), (vc, vs, x_v))):
        want_c, want_s = ref8.append(c, s, x, slots)
        assert torch.equal(got[2 + i], want_s)
        nan = torch.isnan(want_c.float())
        assert torch.equal(torch.isnan(got[i].float()), nan)
        assert torch.equal(_bits(got[i])[~nan], _bits(want_c)[~nan])
    return got


def _runs(rng, P, page, block, T, whole=0.3):
    """Slots of T tokens: runs in blocks of their own, some from the block's first row, some out of order."""
    blocks = list(range(P * page // block))
    rng.shuffle(blocks)
    slots = []
    while len(slots) < T and blocks:
        b = blocks.pop()
        if rng.random() < whole:
            rows = list(range(block))
        else:
            a = rng.randrange(block)
            rows = list(range(a, rng.randint(a + 1, block)))
        if rng.random() < 0.3:
            rng.shuffle(rows)
        slots += [b * block + r for r in rows]
        if rng.random() < 0.2:
            slots.append(rng.choice((-1, P * page, -(1 << 40), 1 << 40)))
    return torch.tensor(slots[:T])


@pytest.mark.parametrize("Hk,D,page,block", [(1, 64, 16, 16), (8, 64, 64, 16), (2, 128, 64, 64), (3, 128, 256, 256),
                                             (5, 64, 256, 256), (16, 64, 128, 32), (17, 128, 128, 128), (4, 64, 48, 16)])
@pytest.mark.parametrize("T", [1, 45, 700])
def test_append_codes_and_scales(T, Hk, D, page, block):
    rng = random.Random(T + Hk)
    P = max(3, 3 * T // page)
    slots = _runs(rng, P, page, block, T)
    T = slots.numel()
    loud = torch.exp2(torch.randint(-12, 9, (T, Hk, 1), generator=torch.Generator().manual_seed(T)).float())
    x = [(_rand((T, Hk, D), s, torch.float32) * loud).to(torch.bfloat16) for s in (3, 4)]
    _check_append(*x, slots, P, page, block)


@pytest.mark.parametrize("D", [64, 128])
def test_append_many_tokens(D):
    # more runs than thread blocks, prompts and single tokens, in fresh blocks and held ones
    rng = random.Random(5)
    slots = torch.cat([_runs(rng, 200, 128, 16, 20000, 0.9), ])
    x = [_rand((slots.numel(), 2, D), s) for s in (1, 2)]
    _check_append(*x, slots, 200, 128, 16)


def test_append_borders_of_scales():
    # sizes at 448 2^k and just past it, zeros, the smallest and largest numbers
    page, D = 16, 64
    sizes = [448.0, 450.0, 1.75, 1.7578125, 0.0, 2.0 ** -120, 448 * 2.0 ** -100, 450 * 2.0 ** -100, 3e38, 2.0 ** -133,
             896.0, 1.0]
    x = torch.zeros((len(sizes), 1, D))
    x[:, 0, 5] = torch.tensor(sizes)
    x[:, 0, 6] = -torch.tensor(sizes) / 3
    x[:, 0, 7] = torch.tensor(sizes) * 2.0 ** -9
    x = x.to(torch.bfloat16)
    slots = torch.arange(len(sizes)) * page  # each starts a block
    _check_append(x, x.roll(1, 0), slots, len(sizes), page, page)
    _check_append(x, x.roll(1, 0), slots + 3, len(sizes), page, page)  # and into held ones


def test_append_values_that_are_not_finite():
    page, D, Hk = 32, 128, 3
    x = _rand((40, Hk, D), 1)
    x[3, 0, 7], x[4, 1, 100], x[20, 2, 0], x[39, 0, 64] = math.inf, NAN, -math.inf, NAN
    x[10, 1] = NAN
    slots = torch.arange(10, 50)
    got = _check_append(x, x.flip(0), slots, 3, page, 32)
    assert bool(torch.isfinite(got[2]).all())
    assert int(torch.isnan(got[0].float()).sum()) == 4 + D


def test_append_into_scales_of_nothing():
    # scales that are 0, negative, NaN or infinite count as none
    page, D = 16, 64
    x = _rand((5, 1, D), 1)
    codes, _ = _pool(5, page, page, 1, D, 3)
    scale = torch.tensor([0.0, -1.0, NAN, math.inf, 0.25]).view(5, 1, 1)
    slots = torch.arange(5) * page + 7
    got = _append(x, x, slots, codes, codes, scale, scale)
    want_c, want_s = ref8.append(codes, scale, x, slots)
    assert torch.equal(got[2], want_s) and torch.equal(got[3], want_s)
    assert torch.equal(_bits(got[0]), _bits(want_c)) and torch.equal(_bits(got[1]), _bits(want_c))


def test_append_scales_do_not_depend_on_the_split():
    # a block filled token by token, in two parts or at once: the same scales, and codes
    # but for subnormals, which a growing scale rounds once more
    Hk, D, page, block = 4, 64, 64, 32
    x = (_rand((2 * block, Hk, D), 1, torch.float32) * torch.exp2(torch.arange(64) / 8.0 - 4)[:, None, None]).to(
        torch.bfloat16)
    got = []
    for parts in ([64], [40, 24], [1] * 64, [5, 27, 1, 31]):
        (kc, ks), (vc, vs) = _pool(1, page, block, Hk, D, 1), _pool(1, page, block, Hk, D, 2)
        t = [c.cuda() for c in (kc, vc, ks, vs)]
        at = 0
        for n in parts:
            fa.fl_kv_append_fp8(None, x[at:at + n].cuda(), x[at:at + n].cuda(), None, *t,
                                torch.arange(at, at + n, device="cuda"))
            at += n
        got.append([c.cpu() for c in t])
    for g in got[1:]:
        for i in (0, 1):
            assert torch.equal(g[2 + i], got[0][2 + i])
            s = got[0][2 + i].repeat_interleave(block, 1)[..., None].double()
            off = (g[i].double() - got[0][i].double()).abs()
            normal = x.double().view(1, page, Hk, D).abs() >= s * 2.0 ** -6
            assert not bool((off * normal).any())
            assert float(off.max()) <= 2.0 ** -9  # a step of the subnormals


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot,Hq,Hk,page,block", [(64, 64, 8, 2, 16, 16), (128, 64, 4, 4, 64, 32), (64, 20, 5, 1, 48, 16),
                                                    (128, 128, 3, 3, 256, 256), (64, 6, 2, 2, 32, 32),
                                                    (128, 48, 1, 1, 16, 16)])
def test_append_rotated(layout, D, rot, Hq, Hk, page, block):
    T, P = 300, 20
    slots = _runs(random.Random(D + rot), P, page, block, T, 0.5)
    T = slots.numel()
    pos = torch.randint(0, 100000, (T,), generator=torch.Generator().manual_seed(1))
    q, k, v = _rand((T, Hq, D), 1), _rand((T, Hk, D), 2), _rand((T, Hk, D), 3)
    (kc, ks), (vc, vs) = _pool(P, page, block, Hk, D, 1), _pool(P, page, block, Hk, D, 2)
    t = [x.cuda() for x in (kc, vc, ks, vs)]
    qo = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.fl_kv_append_fp8(q.cuda(), k.cuda(), v.cuda(), qo, *t, slots.cuda(),
                        rope=fa.make_rope_table(rot, layout=layout), positions=pos.to(torch.int32).cuda())
    got_kc, got_vc, got_ks, got_vs = (x.cpu() for x in t)
    want_v = ref8.append(vc, vs, v, slots)
    assert torch.equal(got_vs, want_v[1]) and torch.equal(_bits(got_vc), _bits(want_v[0]))
    live = (slots >= 0) & (slots < P * page)
    assert bool((qo.cpu()[~live] == 7).all())
    want, bound = ref.rope(q[live], pos[live], rot, layout)
    assert bool(((qo.cpu()[live].double() - want).abs() <= bound * 1.01 + 2.0 ** -8 * want.abs()).all())
    # k: a size within its fp32 error of 448 2^k may take either scale; a value is off by
    # that error and half an e4m3 step, of itself or of the smallest normal number
    want, bound = ref.rope(k[live], pos[live], rot, layout)
    full, err = torch.zeros(T, Hk, D, dtype=torch.float64), torch.zeros(T, Hk, D, dtype=torch.float64)
    full[live], err[live] = want, bound * 1.01
    lo = ref8.append(kc, ks, full.abs() - err, slots)[1]
    hi = ref8.append(kc, ks, full.abs() + err, slots)[1]
    assert bool(((got_ks == lo) | (got_ks == hi)).all())
    at = slots[live]
    s = got_ks.double()[at // page, at % page // block][..., None]
    got = got_kc.double().view(-1, Hk, D)[at] * s
    assert bool(((got - want).abs() <= err[live] + torch.maximum(2.0 ** -4 * (want.abs() + err[live]), s * 2.0 ** -10)).all())
    kept = torch.ones(P * page, dtype=torch.bool)
    kept[at] = False
    same = got_ks == ref8.append(kc, ks, full, slots)[1]
    want_c = ref8.append(kc, ks, full, slots)[0]
    rows = same.repeat_interleave(block, 1).view(-1, Hk) & kept[:, None]
    assert torch.equal(_bits(got_kc).view(-1, Hk, D)[rows], _bits(want_c).view(-1, Hk, D)[rows])


def test_append_into_strided_caches():
    # head-major pages, K and V interleaved in one pool, scales too
    T, P, page, block, Hk, D = 50, 4, 32, 16, 2, 64
    pool = torch.zeros((P, 2, Hk, page, D), dtype=torch.uint8, device="cuda")
    scales = torch.full((P, 3, 2, Hk + 1), 0.5, device="cuda")
    kc, vc = (pool[:, i].transpose(1, 2).view(FP8) for i in (0, 1))
    ks, vs = (scales[:, :2, i, :Hk] for i in (0, 1))
    wide = _rand((T, 2, Hk, 2 * D), 1)
    k, v = wide[:, 0, :, :D], wide[:, 1, :, D:]
    slots = torch.arange(7, 57)
    fa.fl_kv_append_fp8(None, *(wide.cuda()[:, i, :, i * D:(i + 1) * D] for i in (0, 1)), None, kc, vc, ks, vs, slots.cuda())
    zero, half = torch.zeros((P, page, Hk, D), dtype=torch.uint8).view(FP8), torch.full((P, 2, Hk), 0.5)
    for c, s, x in ((kc, ks, k), (vc, vs, v)):
        want_c, want_s = ref8.append(zero, half, x, slots)
        assert torch.equal(s.cpu(), want_s)
        assert torch.equal(c.cpu().contiguous().view(torch.uint8), want_c.view(torch.uint8))
    assert bool((scales[:, 2] == 0.5).all()) and bool((scales[..., Hk] == 0.5).all())


# ------------------------------------------------------------------ chunks


def _problem(q_lens, kv_lens, Hq, Hk, D, page, block, *, seed=0, pad=0, width_extra=1, window=0, loud=1.0, v_range=(0, 1)):
    """A ragged batch over a shuffled pool (contiguous cache: page 0).  Codes of keys that no row
    sees are NaN, as are scales of blocks of nothing else, and every page of no request."""
    g = torch.Generator().manual_seed(seed)
    T, B = sum(q_lens) + pad, len(q_lens)
    q = (loud * torch.randn((T, Hq, D), generator=g)).to(torch.bfloat16)
    if page:
        per = [-(-L // page) for L in kv_lens]
        P = sum(per) + 2
        ids = torch.randperm(P, generator=g).to(torch.int32)
        table = torch.full((B, max(per) + width_extra), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            table[b, : per[b]] = ids[at: at + per[b]]
            at += per[b]
        rows = page
    else:
        rows = -(-(max(kv_lens) + 3) // block) * block
        P, table = B, None
    seen = torch.zeros((P, rows), dtype=torch.bool)
    for b, L in enumerate(kv_lens):
        lo = max(0, L - q_lens[b] - window + 1) if window and q_lens[b] else 0
        for j in range(lo, L):
            p, r = (int(table[b, j // page]), j % page) if page else (b, j)
            seen[p, r] = True
    held = seen.view(P, -1, block).any(-1)
    out = {}
    for n in "kv":
        codes = (torch.randn((P, rows, Hk, D), generator=g) * 64).clamp(-448, 448).to(FP8)
        lo, hi = (-1, 2) if n == "k" else v_range
        scale = torch.exp2(torch.randint(lo, hi, (P, rows // block, Hk), generator=g).float() - 6)
        out["values_" + n] = ref8.values(codes, scale)
        codes.view(torch.uint8)[~seen] = ref8.NAN_CODE
        scale[~held] = NAN
        out[n + "c"], out[n + "s"] = codes, scale
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    for n in "kv":
        out[n] = []
        for b, L in enumerate(kv_lens):
            j = torch.arange(max(L, 1))
            x = out["values_" + n][table[b, j // page].long(), j % page] if page and L else out["values_" + n][b % P, :max(L, 1)]
            out[n].append(x)
    return dict(out, q=q, table=table, cu=cu, q_lens=q_lens, kv_lens=kv_lens, T=T)


def _expected(p, **mask):
    T, Hq, D = p["q"].shape
    out, tol = torch.full((T, Hq, D), 7.0, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    lse = torch.full((Hq, T), 7.0, dtype=torch.float64)
    for b, n in enumerate(p["q_lens"]):
        a, z, L = p["cu"][b], p["cu"][b + 1], p["kv_lens"][b]
        out[a:z], lse[:, a:z], tol[a:z] = ref.chunk_rows(p["q"][a:z], p["k"][b][:L], p["v"][b][:L], None, **mask)
    return out, lse, tol


def _desc(p, max_kv=None, error_word=None, **mask):
    if mask.get("softcap"):
        mask["score_mod"] = "softcap"
    else:
        mask.pop("softcap", None)
    return fa.make_chunk_desc(_ints(p["cu"]), _ints(p["kv_lens"]), p["table"].cuda() if p["table"] is not None else None,
                              max_kv or max(p["kv_lens"] + [1]), error_word=error_word, **mask)


def _launch(p, *, calls=1, max_kv=None, lse=True, **mask):
    err = _ints([0])
    d = _desc(p, max_kv, err, **mask)
    q, kc, vc, ks, vs = (p[n].cuda() for n in ("q", "kc", "vc", "ks", "vs"))
    ws = torch.full((fa.fl_attn_chunk_fp8_workspace_size(q, kc, d),), 0xFF, dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(calls):
        out = torch.full_like(q, 7.0)
        ls = torch.full((q.shape[1], q.shape[0]), 7.0, device="cuda") if lse else None
        fa.fl_attn_chunk_fp8(q, kc, vc, ks, vs, out, ls, d, ws)
        got.append((out, ls))
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return got


def _compare(got, want, what, lse_tol=2e-4, extra=0.0):
    out, lse, tol = want
    o = got[0].double().cpu()
    assert bool(torch.isfinite(o).all()), f"{what}: not finite"
    worst = ((o - out).abs() - tol - extra).max().item()
    assert worst <= 0, f"{what}: O {worst:.3e} past its bound"
    if got[1] is not None:
        l = got[1].double().cpu()
        live = torch.isfinite(lse)
        assert torch.equal(live, torch.isfinite(l)), f"{what}: rows without keys"
        # as for a cache in bf16: the scores' sums in fp32, exp and log
        assert (l - lse)[live].abs().max() <= lse_tol, f"{what}: LSE {(l - lse)[live].abs().max():.3e}"


def _case(q_lens, kv_lens, Hq=8, Hk=2, D=64, page=16, block=16, *, calls=1, **kw):
    mask = {k: kw.pop(k) for k in ("causal", "window", "softcap", "scale") if k in kw}
    p = _problem(q_lens, kv_lens, Hq, Hk, D, page, block, window=mask.get("window", 0), **kw)
    want = _expected(p, **mask)
    got = _launch(p, calls=calls, **mask)
    for g in got:
        _compare(g, want, f"q {q_lens} kv {kv_lens} {mask}")
    for g in got[1:]:
        assert torch.equal(g[0], got[0][0]) and torch.equal(g[1], got[0][1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([1], [1]), ([1], [2]), ([1], [127]), ([1], [129]), ([2], [2]), ([33], [33]), ([65], [300]),
    ([130], [130]), ([1, 1, 1], [64, 65, 63]), ([5, 0, 1, 90], [5, 12, 700, 401]), ([0, 3], [0, 9]),
])
def test_chunk_lengths(D, q_lens, kv_lens):
    _case(q_lens, kv_lens, D=D, pad=3, calls=2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,block", [(0, 16), (0, 64), (16, 16), (32, 32), (64, 16), (128, 64), (256, 256), (256, 16)])
def test_chunk_pages_and_blocks(D, page, block):
    _case([70, 1, 9], [517, 258, 9], D=D, page=page, block=block)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (4, 4), (6, 2), (14, 2), (5, 1), (32, 8), (16, 1), (9, 3), (5, 5),
                                   (100, 1), (128, 1)])
def test_chunk_head_groups(Hq, Hk, D):
    _case([19, 1, 40], [150, 77, 260], Hq=Hq, Hk=Hk, D=D, page=32, block=16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 4, 5, 8, 16, 17, 31, 32, 33])
def test_chunk_few_rows(n, D):
    _case([n, n], [700, n], Hq=8, Hk=2, D=D, page=64, block=32)
    _case([n], [301], Hq=3, Hk=3, D=D, page=16, softcap=10.0, window=150)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mask", [dict(causal=False), dict(window=1), dict(window=50), dict(window=200),
                                  dict(window=100000), dict(softcap=20.0), dict(softcap=5.0, window=77),
                                  dict(softcap=20.0, causal=False), dict(scale=0.3)])
def test_chunk_masks_and_mods(D, mask):
    _case([150, 1, 7, 40], [420, 333, 7, 41], D=D, page=64, block=16, **mask)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lo,hi", [(-60, 3), (9, 40), (-100, -97), (60, 61)])
def test_chunk_scales_far_apart(D, lo, hi):
    # values of blocks from 2^lo to 2^hi: every output is right relative to its own weights' values
    p = _problem([1, 60, 3], [400, 300, 130], 8, 2, D, 64, 16, v_range=(lo, hi))
    got, = _launch(p)
    # in units of the largest value of all, so that the bound's 2e-5 for the scores is relative to it
    unit = 2.0 ** math.frexp(max(float(x.abs().max()) for x in p["v"]))[1]
    p["v"] = [x / unit for x in p["v"]]
    _compare((got[0].double() / unit, got[1]), _expected(p), f"scales 2^{lo} .. 2^{hi}")


def test_chunk_scales_that_are_no_powers_of_two():
    p = _problem([1, 70, 4], [200, 150, 300], 4, 2, 64, 32, 16)
    for n in "kv":
        p[n + "s"] *= 1.3
        p[n] = [x * float(torch.tensor(1.3)) for x in p[n]]
    _compare(_launch(p)[0], _expected(p), "scales times 1.3")


@pytest.mark.parametrize("D", [64, 128])
def test_chunk_rows_that_are_not_finite(D):
    # a row of q with an infinity or NaN is NaN, the others are as they were; rows of tiny and
    # of huge elements keep their precision
    p = _problem([1, 2, 50], [300, 40, 90], 8, 2, D, 32, 16, seed=3)
    q = p["q"]
    q[1, 3, 5], q[2, 0, 0], q[10, 7, 9], q[30, 2, 1] = math.inf, NAN, -math.inf, NAN
    bad = [(1, 3), (2, 0), (10, 7), (30, 2)]
    q[0, 1] *= 2.0 ** -90
    q[20, 6] *= 2.0 ** -70
    q[21, 5] = (q[21, 5].float() * torch.exp2(-torch.arange(D) / 4.0)).to(torch.bfloat16)
    clean = dict(p, q=q.clone())
    for t, h in bad:
        clean["q"][t, h] = 0
    want = _expected(clean)
    out, lse = _launch(p)[0]
    for t, h in bad:
        assert bool(torch.isnan(out[t, h]).all())
        out[t, h], lse[h, t] = want[0][t, h].to(out), want[1][h, t].to(lse)
    _compare((out, lse), want, "rows that are not finite")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 3, 130, 256, 300])
def test_chunk_few_rows_at_the_tiles_borders(D, window):
    lens = [255, 256, 257, 511, 512, 513, 16, 17, 271, 273]
    _case([1] * 9 + [3], lens, Hq=5, Hk=5, D=D, page=16, window=window, calls=2)
    _case([2] * 10, lens, Hq=16, Hk=2, D=D, page=0, block=32, window=window)


def test_chunk_lengths_past_their_bound():
    p = _problem([4], [100], 8, 2, 64, 16, 16)
    for strict, want in ((False, 0), (True, fa.FL_DEVERR_LENGTHS)):
        err = _ints([0])
        d = _desc(p, 60, err, strict_lengths=strict)
        q, kc, vc, ks, vs = (p[n].cuda() for n in ("q", "kc", "vc", "ks", "vs"))
        ws = torch.empty(fa.fl_attn_chunk_fp8_workspace_size(q, kc, d), dtype=torch.uint8, device="cuda")
        out, lse = torch.zeros_like(q), torch.zeros((8, 4), device="cuda")
        fa.fl_attn_chunk_fp8(q, kc, vc, ks, vs, out, lse, d, ws)
        torch.cuda.synchronize()
        assert int(err.item()) == want
        cut = dict(p, kv_lens=[60])
        _compare((out, lse), _expected(cut), "cut to 60 keys")


def test_caches_of_more_than_4_gigabytes():
    # codes 2^32 and more into the caches, scales far into theirs
    P, page, block, Hk, D, T = 70000, 256, 16, 4, 64, 40
    dev = "cuda"
    codes = [torch.zeros((P, page, Hk, D), dtype=torch.uint8, device=dev).view(FP8) for _ in "kv"]
    scales = [torch.full((P, page // block, Hk), 2.0 ** -5, device=dev) for _ in "kv"]
    k, v, q = (_rand((T, h, D), i) for i, h in enumerate((Hk, Hk, 8)))
    slots = torch.cat((torch.arange(30) + (P - 1) * page + 100, torch.arange(10) + (P - 3) * page))
    fa.fl_kv_append_fp8(None, k.to(dev), v.to(dev), None, *codes, *scales, slots.to(dev))
    back = [torch.zeros((T, Hk, D), device=dev) for _ in "kv"]
    fa.fl_kv_read_fp8(*codes, *scales, slots.to(dev), *back)
    for x, b, c, s in zip((k, v), back, codes, scales):
        held_c, held_s = ref8.append(c[P - 3:].cpu(), torch.full((3, page // block, Hk), 2.0 ** -5), x, slots - (P - 3) * page)
        assert torch.equal(s[P - 3:].cpu(), held_s)
        assert torch.equal(_bits(c[P - 3:]), _bits(held_c))
        assert torch.equal(b.cpu().double(), ref8.values(held_c, held_s).view(-1, Hk, D)[slots - (P - 3) * page])
    # both kinds of rows over the last page, and over the one before the last but one
    d = fa.make_chunk_desc(_ints([0, 1, 31]), _ints([10, 256]), _ints([[P - 3], [P - 1]]), 256)
    q = q[:31].to(dev)
    out, lse = torch.zeros_like(q), torch.zeros((8, 31), device=dev)
    ws = torch.empty(fa.fl_attn_chunk_fp8_workspace_size(q, codes[0], d), dtype=torch.uint8, device=dev)
    fa.fl_attn_chunk_fp8(q, *codes, *scales, out, lse, d, ws)
    for a, z, page_at, L in ((0, 1, P - 3, 10), (1, 31, P - 1, 256)):
        kk, vv = (ref8.values(c[page_at:page_at + 1].cpu(), s[page_at:page_at + 1].cpu())[0, :L] for c, s in zip(codes, scales))
        want, wl, tol = ref.chunk_rows(q[a:z].cpu(), kk, vv, None)
        _compare((out[a:z], lse[:, a:z]), (want, wl, tol), "far into the cache")


def test_chunk_rows_without_keys():
    p = _problem([9, 4, 3], [4, 0, 3], 8, 2, 64, 16, 16)
    got, = _launch(p)
    out, lse, tol = _expected(p)
    assert bool((out[:5] == 0).all()) and bool(torch.isinf(lse[:, :5]).all())
    _compare(got, (out, lse, tol), "rows before the sequence")
    p = _problem([3], [0], 8, 2, 64, 16, 16)
    for causal in (True, False):
        got, = _launch(p, causal=causal)
        assert not bool(got[0].any()) and bool((got[1] == -math.inf).all())


@pytest.mark.parametrize("D", [64, 128])
def test_chunk_long_keys_few_rows(D):
    _case([1], [9001], D=D, page=64, block=64, calls=3)
    _case([3, 1], [6000, 2500], D=D, page=256, block=32, Hq=16, Hk=2, calls=2, softcap=20.0)


@pytest.mark.parametrize("D,Hq,Hk", [(64, 8, 2), (128, 4, 1), (64, 2, 2)])
def test_chunk_long_prompts(D, Hq, Hk):
    _case([700, 1, 333], [1500, 2000, 333], Hq=Hq, Hk=Hk, D=D, page=128, block=128, calls=2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(4, 2), (3, 3), (6, 1)])
def test_chunk_many_requests(D, Hq, Hk):
    rng = random.Random(4)
    q_lens = [rng.choice((0, 1, 1, 1, 2, 5)) for _ in range(300)]
    kv_lens = [n + rng.randrange(0, 200) for n in q_lens]
    _case(q_lens, kv_lens, Hq=Hq, Hk=Hk, D=D, page=16, pad=9)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk,page,block", [(16, 2, 64, 32), (5, 5, 128, 16), (4, 1, 16, 16)])
def test_chunk_many_long_requests(D, Hq, Hk, page, block):
    rng = random.Random(9)
    kv_lens = [rng.randrange(300, 6000) for _ in range(40)]
    _case([1] * 40, kv_lens, Hq=Hq, Hk=Hk, D=D, page=page, block=block, calls=2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(8, 2), (16, 1), (6, 3), (20, 1)])
@pytest.mark.parametrize("q_lens", [[1] * 37 + [60], [150] + [1] * 20 + [0, 90, 2], [1, 2, 1, 1]])
def test_chunk_both_kinds_of_work(q_lens, Hq, Hk, D):
    rng = random.Random(len(q_lens))
    kv_lens = [n + rng.randrange(0, 400) for n in q_lens]
    p = _problem(q_lens, kv_lens, Hq, Hk, D, 32, 16, width_extra=10000)
    want = _expected(p)
    for max_kv in (max(kv_lens), 300000):
        got = _launch(p, max_kv=max_kv, calls=3)
        for g in got:
            _compare(g, want, f"q {q_lens} max_kv {max_kv}")
            assert torch.equal(g[0], got[0][0]) and torch.equal(g[1], got[0][1])


def test_chunk_loud_scores():
    # logits of several hundred: the maximum moves far between tiles; scores' fp32 sums are
    # off by up to 66 * 2^-24 * 2000 / 8 = 1e-3, and every weight by that much
    p = _problem([40, 1], [500, 400], 8, 2, 64, 32, 16, loud=40.0)
    _compare(_launch(p)[0], _expected(p), "loud", lse_tol=2e-3, extra=2e-2)


def test_chunk_pages_outside_the_cache_read_as_zeros():
    p = _problem([1, 40], [100, 100], 8, 2, 64, 16, 16)
    for b in (0, 1):
        p["table"][b, 2] = (1 << 30, -5)[b]
        for n in "kv":
            p[n][b] = p[n][b].clone()
            p[n][b][32:48] = 0
    _compare(_launch(p)[0], _expected(p), "pages outside")


def test_chunk_without_lse_and_strided():
    p = _problem([3, 40], [50, 90], 8, 2, 64, 16, 16, pad=2)
    want, d = _expected(p), _desc(p)
    q = torch.zeros((p["T"], 3, 8, 64), dtype=torch.bfloat16, device="cuda")
    q[:, 1] = p["q"].cuda()
    out = torch.full((p["T"], 8, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    P, page, Hk, D = p["kc"].shape
    pool = torch.zeros((P, 2, Hk, page, D), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((P, 2, 1, Hk + 2), device="cuda")
    for i, n in enumerate("kv"):
        pool[:, i] = p[n + "c"].view(torch.uint8).cuda().transpose(1, 2)
        scales[:, i, :, :Hk] = p[n + "s"].cuda()
    kc, vc = (pool[:, i].transpose(1, 2).view(FP8) for i in (0, 1))
    ws = torch.empty(fa.fl_attn_chunk_fp8_workspace_size(q[:, 1], kc, d), dtype=torch.uint8, device="cuda")
    fa.fl_attn_chunk_fp8(q[:, 1], kc, vc, scales[:, 0, :, :Hk], scales[:, 1, :, :Hk], out[:, :, 1], None, d, ws)
    _compare((out[:, :, 1], None), want, "strided")
    assert bool((out[:, :, 0] == 7).all())


# ------------------------------------------------------------------ steps


def test_serving_steps_in_graphs():
    # prompts, then single tokens: plan, append, attention over the 8-bit cache in a captured
    # step that is replayed, against the definitions on the values that the cache holds; a
    # second graph of the same step on another stream, with a workspace of its own
    Hq, Hk, D, page, block, B, P = 8, 2, 64, 32, 16, 3, 60
    rope = fa.make_rope_table(D)
    dev = "cuda"
    free, head, table = torch.randperm(P, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(dev), _ints([0]), \
        torch.full((B, 20), -1, dtype=torch.int32, device=dev)
    caches = [torch.full((P, page, Hk, D), ref8.NAN_CODE, dtype=torch.uint8, device=dev).view(FP8) for _ in "kv"]
    scales = [torch.full((P, page // block, Hk), NAN, device=dev) for _ in "kv"]
    kv = _ints([0] * B)
    history = [[] for _ in range(B)]
    step = 0
    for q_lens in ([70, 5, 33], [1, 1, 1], [1, 0, 1], [2, 1, 40], [1, 1, 1]):
        T = sum(q_lens) + 4
        q, k, v = (_rand((T, h, D), 100 * step + i).to(dev) for i, h in enumerate((Hq, Hk, Hk)))
        qo, out = torch.zeros_like(q), torch.full_like(q, 7.0)
        out2 = torch.full_like(q, 7.0)
        lens, kv_out, cu = _ints(q_lens), _ints([0] * B), _ints([0] * (B + 1))
        pos, slots, head_out = _ints([0] * T), _ints([0] * T, torch.int64), _ints([0])
        plan = fa.make_kv_plan_desc(lens, kv, free, head, table, kv_out, cu, pos, slots, head_out, page_size=page)
        d = fa.make_chunk_desc(cu, kv_out, table, 600)
        ws = [torch.empty(fa.fl_attn_chunk_fp8_workspace_size(q, caches[0], d), dtype=torch.uint8, device=dev) for _ in "ab"]

        def write():
            fa.fl_kv_plan(plan)
            fa.fl_kv_append_fp8(q, k, v, qo, *caches, *scales, slots, rope=rope, positions=pos)

        torch.cuda.synchronize()
        g, g2, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g):
            write()
            fa.fl_attn_chunk_fp8(qo, *caches, *scales, out, None, d, ws[0])
        with torch.cuda.graph(g2):
            fa.fl_attn_chunk_fp8(qo, *caches, *scales, out2, None, d, ws[1])
        g.replay()
        g.replay()  # the same step again: the same cache
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            g2.replay()
        g.replay()
        torch.cuda.synchronize()
        kc, vc = (ref8.values(c.cpu(), s.cpu()) for c, s in zip(caches, scales))
        at, tab = 0, table.cpu()
        for b, n in enumerate(q_lens):
            history[b] += list(range(at, at + n))
            L = int(kv[b]) + n
            j = torch.arange(L)
            keys, vals = (c[tab[b, j // page].long(), j % page] for c in (kc, vc))
            assert bool(torch.isfinite(keys).all())
            want, _, tol = ref.chunk_rows(qo.cpu()[at:at + n], keys, vals, None)
            for o in (out, out2):
                assert bool(((o.cpu()[at:at + n].double() - want).abs() <= tol).all()), (step, b)
            # what was written stands for k and v: off by half a step of e4m3 at the most
            back = vals[L - n:]
            x = v.cpu()[at:at + n].double()
            s = scales[1].cpu().double()[tab[b, j[L - n:] // page].long(), j[L - n:] % page // block][..., None]
            assert bool(((back - x).abs() <= torch.maximum(2.0 ** -4 * x.abs(), s * 2.0 ** -10)).all())
            at += n
        assert bool((out[at:] == 7).all()) and bool((out2[at:] == 7).all())
        # read back by slots
        ko, vo = (torch.full((T, Hk, D), 7.0, device=dev) for _ in "kv")
        fa.fl_kv_read_fp8(*caches, *scales, slots, ko, vo)
        s_cpu = slots.cpu()
        live = s_cpu >= 0
        assert torch.equal(vo.cpu()[live].double(), vc.view(-1, Hk, D)[s_cpu[live]])
        assert torch.equal(ko.cpu()[live].double(), kc.view(-1, Hk, D)[s_cpu[live]]) and bool((ko.cpu()[~live] == 7).all())
        kv.copy_(kv_out)
        head.copy_(head_out)
        step += 1
