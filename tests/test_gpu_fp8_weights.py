"""Weights of very different sizes in attention over the 8-bit KV cache: one key that holds most of a
row's weight, blocks of V whose scales are far apart, loud keys that a row does not see.

A result is bounded relative to what its own row sees, sum_j w_j |v_j|: see _expected."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import fp8_ref as ref8  # noqa: E402
from tests import serving_ref as ref  # noqa: E402
from tests import test_gpu_fp8 as base  # noqa: E402
from tests.fp8_ref import FP8  # noqa: E402

# what an f16 weight loses below its smallest step, relative to the largest weight times scale of
# its row: half of 2^-24 where that one is 2^12 (few rows) or 2^6 (row blocks)
FEW, BLOCKS = 2.0 ** -37, 2.0 ** -31


def _scales(x, block):
    """The append's scales of x [L, Hk, D], L a multiple of block: [L / block, Hk]."""
    size = x.abs().view(-1, block, *x.shape[1:]).amax((1, 3))
    return torch.tensor([[ref8.need(float(a)) for a in row] for row in size], dtype=torch.float64)


def _held(q, keys, vals, q_lens, page=64, block=16, seed=0):
    """A problem of requests whose keys and values are given (float64 [L, Hk, D] each), coded as the
    append does, in a pool of pages in any order (page 0: a contiguous cache)."""
    contiguous = not page
    page = page or -(-max(k.shape[0] for k in keys) // block) * block
    kv_lens = [k.shape[0] for k in keys]
    Hk, D = keys[0].shape[1:]
    per = [-(-L // page) for L in kv_lens]
    ids = torch.arange(sum(per)) if contiguous else torch.randperm(sum(per), generator=torch.Generator().manual_seed(seed))
    p = dict(q=q, T=q.shape[0], q_lens=q_lens, kv_lens=kv_lens, cu=[0])
    for n in q_lens:
        p["cu"].append(p["cu"][-1] + n)
    p["table"] = torch.full((len(keys), max(per)), -1, dtype=torch.int32)
    for n, all_x in (("k", keys), ("v", vals)):
        codes = torch.zeros((sum(per), page, Hk, D), dtype=torch.uint8).view(FP8)
        scales = torch.full((sum(per), page // block, Hk), 2.0 ** -100)
        p[n], p[n + "_scale"], at = [], [], 0
        for b, x in enumerate(all_x):
            L = x.shape[0]
            mine = ids[at: at + per[b]]
            at += per[b]
            p["table"][b, : per[b]] = mine.to(torch.int32)
            full = torch.zeros((per[b] * page, Hk, D), dtype=torch.float64)
            full[:L] = x
            s = _scales(full, block)
            by_key = s.repeat_interleave(block, 0)
            c = (full / by_key[..., None]).float().to(FP8)
            codes.view(torch.uint8)[mine] = c.view(torch.uint8).view(per[b], page, Hk, D)
            scales[mine] = s.float().view(per[b], page // block, Hk)
            p[n].append((c.double() * by_key[..., None])[:L])
            p[n + "_scale"].append(by_key[:L])
        p[n + "c"], p[n + "s"] = codes, scales
    if contiguous:
        p["table"] = None
    return p


def _expected(p, floor, *, causal=True, window=0, softcap=0.0):
    """float64 O [T, Hq, D], LSE [Hq, T] and bounds on the errors of both.

    A score is off by dz at the most: its fp32 sum (2^-21 of the sum of the products' sizes), q's second
    term (2^-18 of the row's largest element, times the key's), 2^-16 for the exponent's sums, whose
    terms are below 2^8, and 2^-21 of a softcap, which makes none of the others larger.  A weight is off by 2^-11 of itself in f16, by dz through its score
    and by as much through the sum of all, or by `floor` of the row's largest weight times scale,
    in which it counts a code; the output's rounding adds 2^-8 of O."""
    T, Hq, D = p["q"].shape
    Hk = p["k"][0].shape[1]
    G = Hq // Hk
    out, lse = torch.zeros(T, Hq, D, dtype=torch.float64), torch.full((Hq, T), -math.inf, dtype=torch.float64)
    tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(p["q_lens"]):
        L, a = p["kv_lens"][b], p["cu"][b]
        pos, j = L - n + torch.arange(n), torch.arange(L)
        seen = torch.ones((n, L), dtype=torch.bool)
        if causal:
            seen &= j <= pos[:, None]
        if window:
            seen &= j > pos[:, None] - window
        for h in range(Hq):
            q, k, v = p["q"][a: a + n, h].double(), p["k"][b][:, h // G], p["v"][b][:, h // G]
            s = p["v_scale"][b][:, h // G]
            z = q @ k.T * D ** -0.5
            if softcap:
                z = softcap * torch.tanh(z / softcap)
            z = z.masked_fill(~seen, -math.inf)
            dz = D ** -0.5 * (2.0 ** -21 * (q.abs() @ k.abs().T) + 2.0 ** -18 * q.abs().amax(-1)[:, None] * k.abs().sum(-1))
            dz = 2.0 ** -16 + 2.0 ** -21 * softcap + dz.masked_fill(~seen, 0).amax(-1)
            w = torch.softmax(z, -1)
            o = w @ v
            out[a: a + n, h], lse[h, a: a + n] = o, torch.logsumexp(z, -1)
            codes = seen.double() @ (v.abs() / s[:, None])
            tol[a: a + n, h] = (2.0 ** -8 * o.abs() + (2.0 ** -11 + 2 * dz)[:, None] * (w @ v.abs())
                                + floor * (w * s).amax(-1)[:, None] * codes)
            lse_tol[h, a: a + n] = dz + 2.0 ** -21 * lse[h, a: a + n].abs() + 2.0 ** -18
    return out, lse, tol, lse_tol


def _check(p, floor, what, calls=1, **mask):
    out, lse, tol, lse_tol = _expected(p, floor, **mask)
    for o, l in base._launch(p, calls=calls, **mask):
        o, l = o.cpu().double(), l.cpu().double()
        assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(l).all()), f"{what}: not finite"
        worst = ((l - lse).abs() / lse_tol).max().item()
        assert worst <= 1, f"{what}: LSE {worst:.3g} times its bound"
        # (1e-300: rows whose values are all zero)
        worst = ((o - out).abs() / (tol + 1e-300)).max().item()
        assert worst <= 1, f"{what}: O {worst:.3g} times its bound"
    return out, lse


def _normal(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def _sink_problem(D, n, L, share, Hq=8, Hk=2, seed=1):
    """Requests of n new tokens on L keys, one of which has about `share` of every row's weight: the first
    key, one in the middle, the first of the last tile.  Its V is a twentieth of the others', which have a mean."""
    at = [0, L // 2 + 5, (L - n) // 256 * 256 - 256]
    # scores of the others are N(0, 1): their exponentials sum up to L e^(1/2)
    z = math.log(share / (1 - share) * L) + 0.5
    q = _normal((3 * n, Hq, D), seed)
    q[..., 0] = z * D ** 0.5 / 16
    keys, vals = [], []
    for b, i in enumerate(at):
        k, v = _normal((L, Hk, D), seed + 2 * b + 1), 0.5 + 0.25 * _normal((L, Hk, D), seed + 2 * b + 2)
        k[..., 0] = 0
        k[i] = 0
        k[i, :, 0] = 16
        v[i] /= 20
        keys.append(k)
        vals.append(v)
    return _held(q.to(torch.bfloat16), keys, vals, [n] * 3, page=256)


@pytest.mark.parametrize("share", [0.5, 0.9, 0.99])
@pytest.mark.parametrize("L", [8192, 32768])
@pytest.mark.parametrize("n", [1, 2, 3])
@pytest.mark.parametrize("D", [64, 128])
def test_small_weights_beside_a_large_one(D, n, L, share):
    # tokens of 4, 8 and 12 rows a KV head
    p = _sink_problem(D, n, L, share)
    out, lse = _check(p, FEW, f"{share} on one of {L} keys")
    for b in range(3):  # and inside the bound that weights in bf16 have
        a, z = b * n, (b + 1) * n
        want, _, tol = ref.chunk_rows(p["q"][a:z], p["k"][b], p["v"][b], None)
        assert torch.allclose(want, out[a:z], rtol=1e-12, atol=1e-12)
        got = base._launch(p)[0][0][a:z].cpu().double()
        assert bool(((got - want).abs() <= tol).all())


@pytest.mark.parametrize("D", [64, 128])
def test_small_weights_beside_one_that_is_nearly_all(D):
    # the others together have 2^-14 of the weight, each 2^-27, and the large one's V is 0
    p = _sink_problem(D, 1, 8192, 1 - 2.0 ** -14)
    for b, i in enumerate([0, 8192 // 2 + 5, 8191 // 256 * 256 - 256]):
        page, row = int(p["table"][b, i // 256]), i % 256
        p["vc"].view(torch.uint8)[page, row] = 0
        p["v"][b][i] = 0
    _check(p, FEW, "nearly all")


@pytest.mark.parametrize("share", [0.5, 0.99])
@pytest.mark.parametrize("D", [64, 128])
def test_small_weights_beside_a_large_one_in_row_blocks(D, share):
    _check(_sink_problem(D, 40, 8192, share), BLOCKS, f"{share} in row blocks")


# ------------------------------------------------------------------ scales of V far apart


def _zero_blocks(D, n, L, log_s, Hq=8, Hk=2):
    """Requests whose V is zero in every other 48 keys (scale 2^-100) and has scales near 2^log_s between;
    the last request begins with zeros, the others do not."""
    q = _normal((3 * n, Hq, D), 3).to(torch.bfloat16)
    keys = [_normal((x, Hk, D), 4 + b) for b, x in enumerate((L, L + 33, n + 7))]
    vals = []
    for b, k in enumerate(keys):
        v = _normal(k.shape, 8 + b) * 2.0 ** (log_s + 7)
        j = torch.arange(k.shape[0]) // 48
        v[(j % 2 == (1 if b < 2 else 0)) & (torch.arange(k.shape[0]) < k.shape[0] - 1)] = 0
        vals.append(v)
    return _held(q, keys, vals, [n] * 3, page=16)


@pytest.mark.parametrize("log_s", [-8, 20, 30, 60, 99])
@pytest.mark.parametrize("n,L", [(1, 200), (1, 9000), (2, 3000), (4, 700), (40, 400), (70, 1500)])
@pytest.mark.parametrize("D", [64, 128])
def test_blocks_of_zeros_beside_loud_ones(D, n, L, log_s):
    _check(_zero_blocks(D, n, L, log_s), FEW if 4 * n <= 16 else BLOCKS, f"zeros beside 2^{log_s}", calls=2)


def _loud(D, n, L, at, gain, z=None, Hq=8, Hk=2, page=32):
    """Two requests of n new tokens on L keys, the V of keys `at` 2^gain times the others'; with z, those keys' scores are z."""
    q = _normal((2 * n, Hq, D), 5)
    keys, vals = [_normal((L, Hk, D), 6 + b) for b in (0, 1)], [_normal((L, Hk, D), 9 + b) for b in (0, 1)]
    if z is not None:
        q[..., 0] = 4
    for k, v in zip(keys, vals):
        v[at] *= 2.0 ** gain
        if z is not None:
            k[..., 0] = 0
            k[at] = 0
            k[at, :, 0] = z * D ** 0.5 / 4
    return _held(q.to(torch.bfloat16), keys, vals, [n] * 2, page=page)


@pytest.mark.parametrize("gain", [20, 35, 60, 100])
@pytest.mark.parametrize("n,L", [(3, 290), (4, 4994), (60, 306), (100, 2002), (300, 706)])
@pytest.mark.parametrize("D", [64, 128])
def test_loud_values_that_come_later(D, n, L, gain):
    # the last 2 tokens' V, a block of its own, is 2^gain louder, which the rows before do not see
    _check(_loud(D, n, L, slice(L - 2, L), gain), FEW if 4 * n <= 16 else BLOCKS, f"2^{gain} later", calls=2)


@pytest.mark.parametrize("gain", [35, 60, 100])
@pytest.mark.parametrize("n,window", [(3, 5), (60, 20), (200, 90), (130, 300)])
@pytest.mark.parametrize("D", [64, 128])
def test_loud_values_that_a_window_has_left(D, n, window, gain):
    p = _loud(D, n, 600, slice(600 - n - 10, 600 - n - 6), gain)
    _check(p, FEW if 4 * n <= 16 else BLOCKS, f"2^{gain} left", window=window)


@pytest.mark.parametrize("gain,z", [(40, -60.0), (60, -60.0), (90, -90.0), (-90, 60.0), (60, -20.0), (-60, 20.0)])
@pytest.mark.parametrize("n,L", [(1, 300), (1, 6000), (4, 2000), (60, 300), (150, 1200)])
@pytest.mark.parametrize("D", [64, 128])
def test_loud_values_of_little_weight(D, n, L, gain, z):
    # a block whose scale and weights differ by 2^90 and more from the others', in either order
    p = _loud(D, n, L, slice(32, 48), gain, z)
    _check(p, FEW if 4 * n <= 16 else BLOCKS, f"2^{gain} at {z}", calls=2)


@pytest.mark.parametrize("n,L", [(1, 9000), (2, 300), (4, 700), (40, 400), (300, 700)])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_far_apart_under_a_softcap(D, n, L):
    floor = FEW if 4 * n <= 16 else BLOCKS
    for log_s in (-8, 60):
        _check(_zero_blocks(D, n, L, log_s), floor, f"zeros beside 2^{log_s}", softcap=20.0)
    _check(_loud(D, n, L, slice(L // 16 * 16, L), 60), floor, "later", softcap=5.0)
    _check(_loud(D, n, L, slice(32, 48), 60, -30.0), floor, "of little weight", softcap=40.0)
    _check(_loud(D, n, L, slice(32, 48), -60, 30.0), floor, "of great weight", softcap=40.0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk,page", [(5, 5, 16), (16, 1, 256), (6, 2, 0), (32, 8, 64)])
def test_scales_far_apart_by_head_groups(Hq, Hk, page, D):
    # one slot, sixteen rows of a token, odd groups, a contiguous cache; rows before the sequence
    for n, L in ((1, 1000), (2, 129), (20, 700), (9, 4)):
        p = _loud(D, n, L, slice(L // 32 * 16, L // 32 * 16 + 16), 70, Hq=Hq, Hk=Hk, page=page)
        floor = FEW if n * Hq // Hk <= 16 else BLOCKS
        if L < n:
            out, lse = base._launch(p)[0]
            assert not bool(out.view(2, n, Hq, D)[:, : n - L].any()) and bool((lse.view(Hq, 2, n)[..., : n - L] == -math.inf).all())
        else:
            _check(p, floor, f"{n} on {L}")


@pytest.mark.parametrize("log_s", [-100, 100])
@pytest.mark.parametrize("n,L", [(1, 20000), (4, 9000), (40, 16000), (100, 9000)])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_at_the_ends_of_their_range(D, n, L, log_s):
    # many keys of the largest or smallest scale; scores rise by 5 after the first tiles, less than
    # what moves a reference, so that sums of weights reach 2^20
    q, k = _normal((n, 8, D), 1), _normal((L, 2, D), 2) / 8
    q[..., 0], k[..., 0] = 4, 0
    k[:300, :, 0] = -5 * D ** 0.5 / 4
    v = _normal((L, 2, D), 3).sign() * 400 * 2.0 ** log_s
    v[..., : D // 2] = 448 * 2.0 ** log_s
    _check(_held(q.to(torch.bfloat16), [k], [v], [n], page=256), FEW if 4 * n <= 16 else BLOCKS, f"scales of 2^{log_s}")


# ------------------------------------------------------------------ rows that are not numbers


@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_are_not_finite_have_no_lse(D):
    # an LSE of NaN for a row of q that holds an infinity or a NaN, in both kinds of rows,
    # of one part and of several
    p = base._problem([1, 2, 50, 1], [300, 40, 90, 9000], 8, 2, D, 32, 16, seed=3)
    q = p["q"]
    q[1, 3, 5], q[2, 0, 0], q[10, 7, 9], q[30, 2, 1], q[53, 4, 0] = math.inf, math.nan, -math.inf, math.nan, math.inf
    bad = torch.zeros((8, p["T"]), dtype=torch.bool)
    for t, h in ((1, 3), (2, 0), (10, 7), (30, 2), (53, 4)):
        bad[h, t] = True
    out, lse = base._launch(p)[0]
    assert torch.equal(torch.isnan(lse.cpu()), bad)
    assert torch.equal(torch.isnan(out.cpu()).any(-1), bad.T) and torch.equal(torch.isnan(out.cpu()).all(-1), bad.T)
