"""Writing and reading the 8-bit KV cache where scales are no powers of two, slots are skipped, or q is long."""
from __future__ import annotations

import math
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import attention_variant_gb300 as fa  # noqa: E402
from tests import fp8_ref as ref8  # noqa: E402
from tests import serving_ref as ref  # noqa: E402
from tests import test_gpu_fp8 as base  # noqa: E402
from tests.fp8_ref import FP8  # noqa: E402


def _rounded(y, bits, least):
    """float64 y rounded once, to `bits` significant bits or the step of 2^least, to nearest even."""
    e = torch.clamp(torch.frexp(y)[1].double() - 1, min=least)
    step = torch.exp2(e - (bits - 1))
    return torch.round(y / step) * step


def _e4m3(y):
    return _rounded(y, 4, -6).clamp(-448, 448).float().to(FP8)


def _odd_scales(shape, seed):
    """Scales that are no powers of two."""
    g = torch.Generator().manual_seed(seed)
    return torch.exp2(16 * torch.rand(shape, generator=g) - 12).float()


# ------------------------------------------------------------------ scales that are no powers of two


@pytest.mark.parametrize("D", [64, 128])
def test_read_rounds_once(D):
    # every code times 4 x 20,000 scales: the product has up to 28 bits, and is rounded to bf16 once
    P, page, Hk = 2500, 32, 4
    codes = (torch.arange(P * page * Hk * D) % 254).to(torch.uint8)
    codes[codes >= 127] += 1  # no NaN
    codes = codes.view(P, page, Hk, D).view(FP8)
    scale = [_odd_scales((P, 2, Hk), i) for i in (1, 2)]
    slots = torch.arange(P * page)
    for dtype, bits in ((torch.bfloat16, 8), (torch.float32, 24)):
        out = [torch.zeros((P * page, Hk, D), dtype=dtype, device="cuda") for _ in "kv"]
        fa.fl_kv_read_fp8(codes.cuda(), codes.cuda(), *(s.cuda() for s in scale), slots.cuda(), *out)
        for got, s in zip(out, scale):
            want = _rounded(ref8.values(codes, s), bits, -126).view(-1, Hk, D)
            assert torch.equal(got.cpu().double(), want)


@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("Hk,D", [(3, 64), (8, 128)])
def test_append_into_blocks_of_such_scales(Hk, D, block):
    # rows after a block's first: a scale that stays, or grows to a power of two
    P, page = 400, 64
    rng = random.Random(Hk)
    slots = torch.tensor([b * block + r for b in range(P * page // block) for r in sorted(rng.sample(range(1, block), 3))])
    T = slots.numel()
    loud = torch.exp2(torch.randint(-6, 7, (T, Hk, 1), generator=torch.Generator().manual_seed(1)).float())
    x = [(base._rand((T, Hk, D), s, torch.float32) * loud).to(torch.bfloat16) for s in (1, 2)]
    codes = [base._pool(P, page, block, Hk, D, s)[0] for s in (3, 4)]
    scale = [_odd_scales((P, page // block, Hk), s) for s in (5, 6)]
    got = base._append(*x, slots, *codes, *scale)
    stays = 0
    for i in (0, 1):
        old = scale[i].double().view(-1, Hk)
        size = x[i].double().abs().amax(-1).view(-1, 3, Hk).amax(1)
        need = torch.tensor([[ref8.need(float(a)) for a in row] for row in size], dtype=torch.float64)
        new = torch.maximum(old, need)
        stays += int((new == old).sum())
        assert torch.equal(got[2 + i].double().view(-1, Hk), new)
        c = codes[i].double().view(-1, block, Hk, D)
        want = torch.where((need > old)[:, None, :, None], _e4m3(c * (old / new)[:, None, :, None]).double(), c)
        want.view(-1, Hk, D)[slots] = _e4m3(x[i].double() / new[slots // block][..., None]).double()
        assert torch.equal(got[i].double().view(want.shape), want)
    assert T // 6 < stays < T // 3 * 2 * Hk


# ------------------------------------------------------------------ skipped slots


def _holes(rng, P, page, block, T, share):
    """Runs of tokens, some of them masked, alone and in stretches of up to 700, before, inside and after the runs."""
    slots = []
    for b in rng.sample(range(P * page // block), P * page // block):
        a = rng.randrange(block)
        for r in range(a, rng.randint(a + 1, block)):
            slots.append(b * block + r)
            if rng.random() < share:
                slots += [rng.choice((-1, P * page, -(1 << 40)))] * rng.choice((1, 1, 1, 2, 31, 32, 33, 300, 700))
    return torch.tensor(slots[:T])


@pytest.mark.parametrize("Hk,D,page,block", [(2, 64, 16, 16), (8, 64, 64, 64), (3, 128, 256, 256), (1, 128, 64, 32)])
@pytest.mark.parametrize("share", [0.02, 0.3])
@pytest.mark.parametrize("T", [9, 300, 6000])
def test_append_around_skipped_slots(T, share, Hk, D, page, block):
    # tokens of a block with skipped ones between them: the tokens of the block that came in earlier
    # calls keep their values, but for a scale that grows
    rng = random.Random(T + block)
    P = max(3, T // page)
    slots = _holes(rng, P, page, block, T, share)
    slots = torch.cat((torch.full((rng.choice((0, 1, 40)),), -1), slots))
    x = [base._rand((slots.numel(), Hk, D), s) * 2 ** (6 * s) for s in (1, 2)]
    base._check_append(*x, slots, P, page, block)


def test_append_of_one_block_with_every_other_slot_skipped():
    P, page, block, Hk, D = 2, 256, 256, 4, 64
    slots = torch.arange(1, 513) // 2
    slots[::2] = -1
    x = [base._rand((512, Hk, D), s) for s in (1, 2)]
    base._check_append(*x, slots, P, page, block)
    base._check_append(x[0].repeat(20, 1, 1), x[1].repeat(20, 1, 1),
                       torch.cat((slots[:300], torch.full((20 * 512 - 512,), -1), slots[300:])), P, page, block)


# ------------------------------------------------------------------ many tokens of q


@pytest.mark.parametrize("layout,D,rot", [("half", 128, 128), ("interleaved", 64, 64), ("half", 64, 0), ("half", 64, 20)])
def test_append_with_more_of_q_than_the_gpu_holds(layout, D, rot):
    # q in a kernel of its own beside K's and V's, also in place and in a captured graph
    Hq, Hk, page, block, T = 16, 2, 64, 64, 11000
    P = T // page + 1
    at = torch.randperm(P * page // block, generator=torch.Generator().manual_seed(1))
    slots = (at[:, None] * block + torch.arange(block)).flatten()[:T]
    slots[4992:5056] = -1  # a whole block
    live = slots >= 0
    pos = torch.randint(0, 100000, (T,), generator=torch.Generator().manual_seed(2))
    q, k, v = base._rand((T, Hq, D), 1), base._rand((T, Hk, D), 2), base._rand((T, Hk, D), 3)
    pools = [base._pool(P, page, block, Hk, D, s) for s in (1, 2)]
    kw = dict(rope=fa.make_rope_table(rot, layout=layout), positions=pos.to(torch.int32).cuda()) if rot else {}
    dev = [x.cuda() for x in (q, k, v, slots)]
    want = [q[live].double(), k[live].double()]
    bound = [torch.zeros_like(x) for x in want]
    if rot:
        want, bound = zip(*(ref.rope(x[live], pos[live], rot, layout) for x in (q, k)))
    results = []
    for graph in (False, True):
        caches = [x.cuda() for x in (pools[0][0], pools[1][0], pools[0][1], pools[1][1])]
        for in_place in (False, True):
            t = [c.clone() for c in caches]
            qi = dev[0].clone()
            qo = qi if in_place else torch.full_like(qi, 7.0)

            def call():
                fa.fl_kv_append_fp8(qi, dev[1], dev[2], qo, *t, dev[3], **kw)

            if graph:
                torch.cuda.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    call()
                g.replay()
            else:
                call()
            # what follows in the stream sees both kernels' work
            results.append([x.cpu() for x in (qo.clone(), *(c.clone() for c in t))])
            if not in_place:
                assert bool((results[-1][0][~live] == 7).all())
    for r in results:
        assert bool(((r[0][live].double() - want[0]).abs() <= bound[0] * 1.01 + 2.0 ** -8 * want[0].abs()).all())
        for i in range(5):
            a, b = (x if i else x[live] for x in (r[i], results[0][i]))
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    _, kc, vc, ks, vs = results[0]
    want_c, want_s = ref8.append(*pools[1], v, slots)
    assert torch.equal(vs, want_s) and torch.equal(vc.view(torch.uint8), want_c.view(torch.uint8))
    at = slots[live]
    s = ks.double()[at // page, at % page // block][..., None]
    got = kc.double().view(-1, Hk, D)[at] * s
    err = bound[1] * 1.01
    assert bool(((got - want[1]).abs() <= err + torch.maximum(2.0 ** -4 * (want[1].abs() + err), s * 2.0 ** -10)).all())
