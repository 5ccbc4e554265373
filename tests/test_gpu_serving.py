"""GPU parity of a serving step with its plain definitions: the step's
book-keeping (fl_kv_plan), the append of new keys (fl_kv_append), attention of
ragged chunks over the cache (fl_attn_chunk), and several steps of all three
together."""
from __future__ import annotations

import math
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import attention_variant_gb300 as fa  # noqa: E402
from tests import serving_ref as ref  # noqa: E402

NAN = float("nan")


def _rand(shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


# ------------------------------------------------------------------ book-keeping


def _run_plan(q, kv, page, *, width=None, n_free=None, head=0, max_tokens=None, seed=0, slots=True):
    rng = random.Random(seed)
    held = [-(-max(k, 0) // page) for k in kv]
    need = [-(-(max(k, 0) + max(n, 0)) // page) for n, k in zip(q, kv)]
    width = max(need + [1]) + 1 if width is None else width
    ids = list(range(sum(need) + head + 3))
    rng.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append((ids[at:at + h] + [-9] * width)[:width])
        at += h
    free = [1000 + i for i in range(head)] + ids[at:]
    free = free if n_free is None else free[:n_free]
    max_tokens = sum(max(n, 0) for n in q) + 5 if max_tokens is None else max_tokens
    want = ref.plan(q, kv, table, free, head, page, max_tokens)
    B = len(q)
    t = dict(q=_ints(q), kv=_ints(kv), free=_ints(free), head=_ints([head]), table=_ints(table),
             kv_out=_ints([-7] * B), cu=_ints([-7] * (B + 1)), pos=_ints([-7] * max_tokens),
             slots=_ints([-7] * max_tokens, torch.int64), head_out=_ints([-7]), err=_ints([0]))
    d = fa.make_kv_plan_desc(t["q"], t["kv"], t["free"], t["head"], t["table"], t["kv_out"], t["cu"], t["pos"],
                             t["slots"] if slots else None, t["head_out"], page_size=page, error_word=t["err"])
    for _ in range(2):  # a second call on the same buffers gives the same
        fa.fl_kv_plan(d)
    torch.cuda.synchronize()
    assert t["kv_out"].tolist() == want["kv_out"]
    assert t["cu"].tolist() == want["cu_q"]
    assert t["pos"].tolist() == want["positions"]
    if slots:
        assert t["slots"].tolist() == want["slots"]
    assert t["table"].tolist() == want["table"]
    assert t["head_out"].tolist() == [want["head"]]
    err = (fa.FL_DEVERR_PAGES if want["short"] else 0) | \
        (fa.FL_DEVERR_LENGTHS if want["cu_q"][-1] > max_tokens else 0)
    return int(t["err"].item()), err


@pytest.mark.parametrize("q,kv,page", [
    ([1], [0], 16), ([1], [15], 16), ([1], [16], 16), ([17], [16], 16), ([0], [0], 32), ([5], [0], 256),
    ([1, 0, 3, 40], [31, 7, 0, 100], 32), ([-4, 2], [3, -1], 16), ([1000], [77], 64),
])
def test_plan_small(q, kv, page):
    got, want = _run_plan(q, kv, page)
    assert got == want == 0


@pytest.mark.parametrize("B", [1023, 1024, 1025, 2500])
def test_plan_many_requests(B):
    rng = random.Random(B)
    q = [rng.choice((0, 1, 1, 1, 30)) for _ in range(B)]
    kv = [rng.randrange(0, 300) for _ in range(B)]
    got, want = _run_plan(q, kv, 16, head=3, seed=B)
    assert got == want == 0


def test_plan_long_prompts_and_no_slots():
    assert _run_plan([9000, 1, 5000], [10, 200, 0], 128) == (0, 0)
    assert _run_plan([9, 1, 5], [10, 200, 0], 128, slots=False) == (0, 0)


def test_plan_out_of_pages_and_out_of_table():
    got, want = _run_plan([40, 20], [0, 10], 16, n_free=3)
    assert got == want == fa.FL_DEVERR_PAGES
    got, want = _run_plan([40, 1], [0, 3], 16, width=2)
    assert got == want == fa.FL_DEVERR_PAGES


def test_plan_more_tokens_than_stated():
    got, want = _run_plan([40, 20], [0, 10], 16, max_tokens=50)
    assert got & fa.FL_DEVERR_LENGTHS and got == want


def test_plan_nonsense_lengths_stay_inside():
    # lengths that overflow 32 bits: numbers without meaning, but nothing is
    # read or written outside the arrays (guard rows around the table stay)
    big = (1 << 31) - 1
    for q, kv in (([big, 5], [0, 3]), ([7, 2], [big, big - 3]), ([big, big, big, 9], [0, 0, 0, 0])):
        B = len(q)
        table = _ints([[-9] * 4] * (B + 2))
        t = [_ints(q), _ints(kv), _ints([5, 6, 7]), _ints([0]), table[1:-1]]
        out = [_ints([0] * B), _ints([0] * (B + 1)), _ints([0] * 3000), _ints([0] * 3000, torch.int64), _ints([0])]
        fa.fl_kv_plan(fa.make_kv_plan_desc(*t, *out, page_size=16))
        torch.cuda.synchronize()
        assert table[0].tolist() == [-9] * 4 == table[-1].tolist()
        slots = out[3]
        assert bool((slots < 8 * 16).all()) and bool((slots >= -1).all())


# ------------------------------------------------------------------ append


@pytest.mark.parametrize("layout", ["half", "interleaved", None])
@pytest.mark.parametrize("D,rot,Hq,Hk,page", [(64, 64, 8, 2, 16), (128, 64, 4, 4, 64), (64, 20, 5, 1, 48),
                                              (32, 32, 3, 3, 1)])
def test_append(layout, D, rot, Hq, Hk, page):
    T, P = 45, 9 if page > 1 else 70
    g = torch.Generator().manual_seed(D + page)
    slots = torch.randperm(P * page, generator=g)[:T]
    slots[3], slots[10], slots[44] = -1, P * page, -(1 << 40)  # skipped
    pos = torch.randint(0, 100000, (T,), generator=g)
    q, k, v = _rand((T, Hq, D), 1), _rand((T, Hk, D), 2), _rand((T, Hk, D), 3)
    caches = [_rand((P, page, Hk, D), s) for s in (4, 5)]
    qo = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    kc, vc = (c.cuda() for c in caches)
    table = fa.make_rope_table(rot, layout=layout) if layout else None
    fa.fl_kv_append(q.cuda(), k.cuda(), v.cuda(), qo, kc, vc, slots.cuda(), rope=table,
                    positions=pos.to(torch.int32).cuda() if layout else None)
    live = (slots >= 0) & (slots < P * page)
    at = slots[live]
    want_v = caches[1].clone().view(-1, Hk, D)
    want_v[at] = v[live]
    assert torch.equal(vc.cpu().view(-1, Hk, D), want_v)
    got_k, old_k = kc.cpu().view(-1, Hk, D), caches[0].view(-1, Hk, D)
    kept = torch.ones(P * page, dtype=torch.bool)
    kept[at] = False
    assert torch.equal(got_k[kept], old_k[kept])
    assert bool((qo[~live.cuda()] == 7).all())
    for got, x in ((got_k[at], k[live]), (qo.cpu()[live], q[live])):
        if not layout:
            assert torch.equal(got, x)
            continue
        want, bound = ref.rope(x, pos[live], rot, layout)
        err = (got.double() - want).abs()
        assert bool((err <= bound * 1.01 + 2.0 ** -8 * want.abs()).all())


def test_append_without_q_into_strided_caches():
    # head-major pages; K and V interleaved in one pool
    T, P, page, Hk, D = 20, 4, 16, 2, 64
    pool = torch.zeros((P, 2, Hk, page, D), dtype=torch.bfloat16, device="cuda")
    kc, vc = (pool[:, i].transpose(1, 2) for i in (0, 1))
    k, v = _rand((T, Hk, D), 1), _rand((T, Hk, D), 2)
    fa.fl_kv_append(None, k.cuda(), v.cuda(), None, kc, vc, torch.arange(7, 27, device="cuda"))
    for got, x in ((kc, k), (vc, v)):
        flat = got.reshape(-1, Hk, D).cpu()
        assert torch.equal(flat[7:27], x)
        assert not bool(flat[:7].any()) and not bool(flat[27:].any())


# ------------------------------------------------------------------ chunks


def _problem(q_lens, kv_lens, Hq, Hk, D, page, *, seed=0, pad=0, width_extra=1, window=0, causal=True,
             poison=True, loud=1.0):
    """A ragged batch over a shuffled pool (contiguous cache: page 0).  Every
    key that no row sees, and every page of no request, is NaN."""
    g = torch.Generator().manual_seed(seed)
    T = sum(q_lens) + pad
    q = (loud * torch.randn((T, Hq, D), generator=g)).to(torch.bfloat16)
    keys = [torch.randn((max(L, 1), Hk, D), generator=g).to(torch.bfloat16) for L in kv_lens]
    vals = [torch.randn((max(L, 1), Hk, D), generator=g).to(torch.bfloat16) for L in kv_lens]
    fill = NAN if poison else 1.0
    B = len(q_lens)
    if page:
        per = [-(-L // page) for L in kv_lens]
        P = sum(per) + 2
        ids = torch.randperm(P, generator=g).to(torch.int32)
        table = torch.full((B, max(per) + width_extra), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            table[b, : per[b]] = ids[at: at + per[b]]
            at += per[b]
        kc, vc = (torch.full((P, page, Hk, D), fill, dtype=torch.bfloat16) for _ in "kv")
    else:
        S = max(kv_lens) + 3
        table = None
        kc, vc = (torch.full((B, S, Hk, D), fill, dtype=torch.bfloat16) for _ in "kv")
    for b, L in enumerate(kv_lens):
        lo = 0
        if window and q_lens[b]:
            lo = max(0, L - q_lens[b] - window + 1)  # keys before it no row sees
        for j in range(lo, L):
            p, r = (int(table[b, j // page]), j % page) if page else (b, j)
            kc[p, r], vc[p, r] = keys[b][j], vals[b][j]
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    return dict(q=q, k=keys, v=vals, kc=kc, vc=vc, table=table, cu=cu, q_lens=q_lens, kv_lens=kv_lens, T=T)


def _expected(p, **mask):
    T, Hq, D = p["q"].shape
    out, tol = torch.full((T, Hq, D), 7.0, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    lse = torch.full((Hq, T), 7.0, dtype=torch.float64)
    for b, n in enumerate(p["q_lens"]):
        a, z = p["cu"][b], p["cu"][b + 1]
        L = p["kv_lens"][b]
        out[a:z], lse[:, a:z], tol[a:z] = ref.chunk_rows(p["q"][a:z], p["k"][b][:L], p["v"][b][:L], None, **mask)
    return out, lse, tol


def _launch(p, *, calls=1, max_kv=None, lse=True, desc=None, ws=None, stream=None, **mask):
    if mask.get("softcap"):
        mask["score_mod"] = "softcap"
    else:
        mask.pop("softcap", None)
    err = _ints([0])
    d = desc or fa.make_chunk_desc(_ints(p["cu"]), _ints(p["kv_lens"]),
                                   p["table"].cuda() if p["table"] is not None else None,
                                   max_kv or max(p["kv_lens"] + [1]), error_word=err, **mask)
    q, kc, vc = (p[n].cuda() for n in ("q", "kc", "vc"))
    if ws is None:
        ws = torch.full((fa.fl_attn_chunk_workspace_size(q, kc, d),), 0xFF, dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(calls):
        out = torch.full_like(q, 7.0)
        ls = torch.full((q.shape[1], q.shape[0]), 7.0, device="cuda") if lse else None
        fa.fl_attn_chunk(q, kc, vc, out, ls, d, ws, stream=stream)
        got.append((out, ls))
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return got


def _compare(got, want, what):
    out, lse, tol = want
    o = got[0].double().cpu()
    assert bool(torch.isfinite(o).all()), f"{what}: not finite"
    worst = ((o - out).abs() - tol).max().item()
    assert worst <= 0, f"{what}: O {worst:.3e} past its bound"
    if got[1] is not None:
        l = got[1].double().cpu()
        live = torch.isfinite(lse)
        assert torch.equal(live, torch.isfinite(l)), f"{what}: rows without keys"
        # scores: D products summed in fp32 (at most (D + 2) 2^-24 sum |q k| / sqrt(D), 1e-4
        # for these inputs), 2^-21 of a softcapped score, exp and log of 2^-22
        assert (l - lse)[live].abs().max() <= 2e-4, f"{what}: LSE {(l - lse)[live].abs().max():.3e}"


def _case(q_lens, kv_lens, Hq=8, Hk=2, D=64, page=16, *, what="", calls=1, **kw):
    mask = {k: kw.pop(k) for k in ("causal", "window", "softcap", "scale") if k in kw}
    p = _problem(q_lens, kv_lens, Hq, Hk, D, page, causal=mask.get("causal", True),
                 window=mask.get("window", 0), **kw)
    want = _expected(p, **mask)
    got = _launch(p, calls=calls, **mask)
    for g in got:
        _compare(g, want, what or f"q {q_lens} kv {kv_lens} {mask}")
    for g in got[1:]:
        assert torch.equal(g[0], got[0][0]) and torch.equal(g[1], got[0][1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([1], [1]), ([1], [2]), ([1], [111]), ([1], [113]), ([2], [2]), ([33], [33]), ([65], [300]),
    ([130], [130]), ([1, 1, 1], [64, 65, 63]), ([5, 0, 1, 90], [5, 12, 700, 401]), ([0, 3], [0, 9]),
])
def test_chunk_lengths(D, q_lens, kv_lens):
    _case(q_lens, kv_lens, D=D, pad=3, calls=2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [0, 16, 32, 64, 128, 256])
def test_chunk_pages(D, page):
    _case([70, 1, 9], [517, 258, 9], D=D, page=page)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (4, 4), (6, 2), (14, 2), (5, 1), (32, 8), (16, 1), (9, 3), (5, 5),
                                   (100, 1), (128, 1)])
def test_chunk_head_groups(Hq, Hk, D):
    _case([19, 1, 40], [150, 77, 260], Hq=Hq, Hk=Hk, D=D, page=32)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 32, 33])
def test_chunk_few_rows(n, D):
    # every way of filling the row blocks, on both sides of their limits
    _case([n, n], [700, n], Hq=8, Hk=2, D=D, page=64)
    _case([n], [301], Hq=3, Hk=3, D=D, page=16, softcap=10.0, window=150)


@pytest.mark.parametrize("D", [64, 128])
def test_chunk_few_loud_rows(D):
    # the maximum of single tokens' rows moves far between tiles, rows apart
    # from one another; the largest key may come last
    p = _problem([1, 2], [900, 1300], 6, 3, D, 16, loud=1.0)
    for b, n in ((0, 900), (1, 1300)):
        ramp = torch.linspace(0, 30, n)[:, None, None]
        p["k"][b] = (p["k"][b].float() * ramp).to(torch.bfloat16)
        for j in range(n):
            pg, r = int(p["table"][b, j // 16]), j % 16
            p["kc"][pg, r] = p["k"][b][j]
    want = _expected(p)
    got, = _launch(p)
    out, lse, tol = want
    # scores of up to ~150, summed in fp32: off by at most (D + 2) 2^-24 sum |q k| / sqrt(D)
    # < 130 * 2^-24 * 128 * 4 * 120 / 11 = 4e-2 at the very worst, typically 1e-5; a weight by
    # as much, and 2^-22 of the exponent's argument (up to 220): 5e-5
    assert ((got[0].double().cpu() - out).abs() <= tol + 5e-3).all()
    assert (got[1].double().cpu() - lse).abs().max() <= 5e-3


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mask", [dict(causal=False), dict(window=1), dict(window=50), dict(window=200),
                                  dict(window=100000), dict(softcap=20.0), dict(softcap=5.0, window=77),
                                  dict(softcap=20.0, causal=False), dict(scale=0.3)])
def test_chunk_masks_and_mods(D, mask):
    _case([150, 1, 7, 40], [420, 333, 7, 41], D=D, page=64, **mask)


def test_chunk_rows_without_keys():
    # fewer cached keys than rows: the first rows sit before the sequence
    p = _problem([9, 4, 3], [4, 0, 3], 8, 2, 64, 16)
    got, = _launch(p)
    out, lse, tol = _expected(p)
    assert bool((out[:5] == 0).all()) and bool(torch.isinf(lse[:, :5]).all())
    _compare(got, (out, lse, tol), "rows before the sequence")
    p = _problem([3], [0], 8, 2, 64, 16)
    for causal in (True, False):
        got, = _launch(p, causal=causal)
        assert not bool(got[0].any()) and bool((got[1] == -math.inf).all())


@pytest.mark.parametrize("D", [64, 128])
def test_chunk_long_keys_few_rows(D):
    # keys split over the whole GPU and merged, twice with the same bits
    _case([1], [9001], D=D, page=64, calls=3)
    _case([3, 1], [6000, 2500], D=D, page=256, Hq=16, Hk=2, calls=2, softcap=20.0)


@pytest.mark.parametrize("D,Hq,Hk", [(64, 8, 2), (128, 4, 1), (64, 2, 2)])
def test_chunk_long_prompts(D, Hq, Hk):
    _case([700, 1, 333], [1500, 2000, 333], Hq=Hq, Hk=Hk, D=D, page=128, calls=2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(4, 2), (3, 3), (6, 1)])
def test_chunk_many_requests(D, Hq, Hk):
    rng = random.Random(4)
    q_lens = [rng.choice((0, 1, 1, 1, 2, 5)) for _ in range(300)]
    kv_lens = [n + rng.randrange(0, 200) for n in q_lens]
    _case(q_lens, kv_lens, Hq=Hq, Hk=Hk, D=D, page=16, pad=9)


@pytest.mark.parametrize("D", [64, 128])
def test_chunk_thousands_of_requests(D):
    # both lists longer than a round of the planning kernel and than what it keeps at hand
    rng = random.Random(12)
    q_lens = [9] * 1030 + [1] * 1070 + [0] * 50
    rng.shuffle(q_lens)
    kv_lens = [n + rng.randrange(0, 40) for n in q_lens]
    _case(q_lens, kv_lens, Hq=2, Hk=1, D=D, page=16, pad=5, calls=2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk,page", [(16, 2, 64), (5, 5, 128), (4, 1, 16)])
def test_chunk_many_long_requests(D, Hq, Hk, page):
    # tens of key tiles per CTA, of neighbouring heads and across requests, so
    # that the rings of tiles turn many times, at every offset to the heads
    rng = random.Random(9)
    kv_lens = [rng.randrange(300, 6000) for _ in range(40)]
    _case([1] * 40, kv_lens, Hq=Hq, Hk=Hk, D=D, page=page, calls=2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(8, 2), (16, 1), (6, 3), (20, 1)])
@pytest.mark.parametrize("q_lens", [
    [1] * 37 + [60],                # few tokens a request: few rows first, then a row block
    [150] + [1] * 20 + [0, 90, 2],  # row blocks first
    [1, 2, 1, 1],                   # few rows alone (groups of up to 8 heads)
])
def test_chunk_both_kinds_of_work(q_lens, Hq, Hk, D):
    # a cache that may hold far more than it does, so that the loads are taken
    # for many, and the same with a tight bound
    rng = random.Random(len(q_lens))
    kv_lens = [n + rng.randrange(0, 400) for n in q_lens]
    p = _problem(q_lens, kv_lens, Hq, Hk, D, 32, width_extra=10000)
    want = _expected(p)
    for max_kv in (max(kv_lens), 300000):
        got = _launch(p, max_kv=max_kv, calls=3)
        for g in got:
            _compare(g, want, f"q {q_lens} max_kv {max_kv}")
            assert torch.equal(g[0], got[0][0]) and torch.equal(g[1], got[0][1])


def test_chunk_loud_scores():
    # logits of several hundred: the maximum moves far between tiles
    p = _problem([40, 1], [500, 400], 8, 2, 64, 32, loud=40.0)
    want = _expected(p)
    got, = _launch(p)
    out, lse, tol = want
    # scores of up to ~150: their fp32 sums are off by up to (D + 2) 2^-24 sum |q k| / 8
    # < 66 * 2^-24 * 2000 / 8 = 1e-3, and every weight by that much: 2e-3 |v - O|
    assert ((got[0].double().cpu() - out).abs() <= tol + 2e-3 * 10).all()
    assert (got[1].double().cpu() - lse).abs().max() <= 2e-3


def test_chunk_clamped_lengths():
    # entries of kv_lens above max_kv_len count as max_kv_len
    p = _problem([4], [100], 8, 2, 64, 16)
    got, = _launch(p, max_kv=60)
    want, lse, tol = ref.chunk_rows(p["q"], p["k"][0][:60], p["v"][0][:60], None)
    _compare(got, (want, lse, tol), "clamped")


def test_chunk_strided_views():
    # q a slice of a fused projection, head-major pages, out with gaps
    p = _problem([50, 1], [130, 90], 8, 2, 64, 16)
    want = _expected(p)
    T = p["T"]
    big = torch.full((T, 20, 64), NAN, dtype=torch.bfloat16, device="cuda")
    big[:, 4:12] = p["q"].cuda()
    kc, vc = (p[n].cuda().transpose(1, 2).contiguous().transpose(1, 2) for n in ("kc", "vc"))
    out = torch.full((T, 10, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, T + 5), 7.0, device="cuda")
    d = fa.make_chunk_desc(_ints(p["cu"]), _ints(p["kv_lens"]), p["table"].cuda(), 130)
    q = big[:, 4:12]
    ws = torch.empty(fa.fl_attn_chunk_workspace_size(q, kc, d), dtype=torch.uint8, device="cuda")
    fa.fl_attn_chunk(q, kc, vc, out[:, 1:9], lse[:, :T], d, ws)
    torch.cuda.synchronize()
    _compare((out[:, 1:9], lse[:, :T]), want, "strided")
    assert bool((out[:, 0] == 7).all()) and bool((out[:, 9] == 7).all()) and bool((lse[:, T:] == 7).all())


def test_chunk_bad_pages_read_as_zeros():
    # a table entry outside the pool: zero keys and values, no fault
    p = _problem([1], [64], 8, 2, 64, 32)
    p["table"][0, 0] = 1 << 30
    p["k"][0][:32], p["v"][0][:32] = 0, 0
    got, = _launch(p)
    _compare(got, _expected(p), "bad page")
    p["table"][0, 0] = -5
    got, = _launch(p)
    _compare(got, _expected(p), "negative page")


def test_chunk_bad_offsets_stay_inside():
    # cu_q entries outside [0, T] or descending: every row still belongs to at
    # most the tensor, nothing hangs, and sane requests are right
    p = _problem([4, 6], [40, 60], 8, 2, 64, 16)
    want, lse, tol = _expected(p)
    p["cu"] = [-3, 4, 10]
    q, kc, vc = (p[n].cuda() for n in ("q", "kc", "vc"))
    d = fa.make_chunk_desc(_ints([-3, 4, 999]), _ints(p["kv_lens"]), p["table"].cuda(), 60)
    ws = torch.empty(fa.fl_attn_chunk_workspace_size(q, kc, d), dtype=torch.uint8, device="cuda")
    out, ls = torch.full_like(q, 7.0), torch.full((8, 10), 7.0, device="cuda")
    fa.fl_attn_chunk(q, kc, vc, out, ls, d, ws)
    torch.cuda.synchronize()
    _compare((out, ls), (want, lse, tol), "clamped offsets")
    d = fa.make_chunk_desc(_ints([9, 2, 1]), _ints(p["kv_lens"]), p["table"].cuda(), 60)
    fa.fl_attn_chunk(q, kc, vc, out, ls, d, ws)
    torch.cuda.synchronize()


def test_chunk_far_pages():
    # a pool of more than 2^32 elements: page offsets pass 32 bits
    P, page, Hk, D = 33000, 256, 8, 64
    assert P * page * Hk * D > 1 << 32
    pools = [torch.empty((P, page, Hk, D), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    L, pages = 600, [32999, 0, 16500]
    keys, vals = _rand((L, Hk, D), 1), _rand((L, Hk, D), 2)
    q = _rand((2, 32, D), 3)
    # the append puts them there, too
    slots = torch.tensor([pages[j // page] * page + j % page for j in range(L)], device="cuda")
    fa.fl_kv_append(None, keys.cuda(), vals.cuda(), None, pools[0], pools[1], slots)
    d = fa.make_chunk_desc(_ints([0, 2]), _ints([L]), _ints([pages]), L)
    qd = q.cuda()
    ws = torch.empty(fa.fl_attn_chunk_workspace_size(qd, pools[0], d), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(qd), torch.empty((32, 2), device="cuda")
    fa.fl_attn_chunk(qd, pools[0], pools[1], out, lse, d, ws)
    torch.cuda.synchronize()
    _compare((out, lse), ref.chunk_rows(q, keys, vals, None), "far pages")


def test_chunk_without_lse_and_on_another_stream():
    p = _problem([30, 1], [100, 200], 8, 2, 64, 16)
    want = _expected(p)
    got, = _launch(p, lse=False)
    _compare(got, want, "no lse")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, = _launch(p)
    _compare(got, want, "side stream")


def test_chunk_two_calls_at_once():
    # two streams with a workspace each: the calls' kernels share the GPU as they come
    ps = [_problem([300, 1, 1, 7], [1500, 2000, 3, 7], 8, 2, 64, 16, seed=3),
          _problem([1] * 24, [700 + 90 * i for i in range(24)], 8, 2, 64, 64, seed=4)]
    wants = [_expected(p) for p in ps]
    runs = []
    for p in ps:
        t = dict(q=p["q"].cuda(), kc=p["kc"].cuda(), vc=p["vc"].cuda(), cu=_ints(p["cu"]), kv=_ints(p["kv_lens"]),
                 table=p["table"].cuda(), stream=torch.cuda.Stream())
        t["d"] = fa.make_chunk_desc(t["cu"], t["kv"], t["table"], max(p["kv_lens"]))
        t["ws"] = torch.empty(fa.fl_attn_chunk_workspace_size(t["q"], t["kc"], t["d"]), dtype=torch.uint8, device="cuda")
        t["outs"] = [(torch.full_like(t["q"], 7.0), torch.full((8, p["T"]), 7.0, device="cuda")) for _ in range(20)]
        runs.append(t)
    torch.cuda.synchronize()
    for i in range(20):
        for t in runs:
            fa.fl_attn_chunk(t["q"], t["kc"], t["vc"], *t["outs"][i], t["d"], t["ws"], stream=t["stream"])
    torch.cuda.synchronize()
    for t, want in zip(runs, wants):
        for out in t["outs"]:
            _compare(out, want, "beside another call")
            assert torch.equal(out[0], t["outs"][0][0]) and torch.equal(out[1], t["outs"][0][1])


def test_chunk_captured_graphs_share_a_workspace():
    # two captured steps of different shapes replay in turn over one workspace
    ps = [_problem([60, 1], [100, 3000], 8, 2, 64, 16, seed=1), _problem([1, 1, 9], [2000, 5, 9], 8, 2, 64, 16, seed=2)]
    wants = [_expected(p) for p in ps]
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    calls = []
    for p in ps:
        t = dict(q=p["q"].cuda(), kc=p["kc"].cuda(), vc=p["vc"].cuda(), cu=_ints(p["cu"]), kv=_ints(p["kv_lens"]),
                 table=p["table"].cuda())
        d = fa.make_chunk_desc(t["cu"], t["kv"], t["table"], max(p["kv_lens"]))
        assert fa.fl_attn_chunk_workspace_size(t["q"], t["kc"], d) <= ws.numel()
        t["out"], t["lse"], t["d"] = torch.full_like(t["q"], 7.0), torch.full((8, p["T"]), 7.0, device="cuda"), d
        g = torch.cuda.CUDAGraph()
        fa.fl_attn_chunk(t["q"], t["kc"], t["vc"], t["out"], t["lse"], d, ws)
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            fa.fl_attn_chunk(t["q"], t["kc"], t["vc"], t["out"], t["lse"], d, ws)
        calls.append((g, t))
    for _ in range(3):
        for g, t in calls:
            t["out"].fill_(7.0)
            g.replay()
    torch.cuda.synchronize()
    for (_, t), want in zip(calls, wants):
        _compare((t["out"], t["lse"]), want, "captured")


def test_chunk_agrees_with_decode():
    """Single tokens through fl_attn_chunk and fl_attn_decode: the same rows."""
    B, page = 6, 64
    kv_lens = [1, 64, 65, 300, 1000, 2048]
    p = _problem([1] * B, kv_lens, 32, 8, 64, page)
    got, = _launch(p)
    q, kc, vc = p["q"].cuda().unsqueeze(1), p["kc"].cuda(), p["vc"].cuda()
    dd = fa.make_decode_desc(_ints(kv_lens), max(kv_lens), block_table=p["table"].cuda())
    out, lse = torch.empty_like(q), torch.empty((B, 32, 1), device="cuda")
    ws = torch.empty(fa.fl_attn_decode_workspace_size(q, kc, dd), dtype=torch.uint8, device="cuda")
    fa.fl_attn_decode(q, kc, vc, out, lse, dd, ws)
    torch.cuda.synchronize()
    want = _expected(p)
    _compare(got, want, "chunk")
    _compare((out[:, 0], lse[..., 0].t()), want, "decode")


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("captured", [False, True])
def test_steps_of_a_serving_loop(captured):
    """Prompts and tokens of three requests over several steps, all book-keeping
    on the GPU: every step's outputs against attention over the whole history
    so far (rotated keys as the cache holds them, bf16)."""
    Hq, Hk, D, page, T = 8, 2, 64, 16, 64
    steps = [[40, 3, 0], [1, 20, 7], [1, 1, 1], [30, 1, 33], [1, 0, 1]]
    B, P = 3, 40
    ids = torch.randperm(P, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    t = dict(q_lens=_ints([0] * B), kv=_ints([0] * B), kv2=_ints([0] * B), head=_ints([0]), head2=_ints([0]),
             table=_ints([[-1] * 8] * B), cu=_ints([0] * (B + 1)), pos=_ints([0] * T),
             slots=_ints([0] * T, torch.int64), err=_ints([0]))
    x = {n: torch.zeros((T, h, D), dtype=torch.bfloat16, device="cuda")
         for n, h in (("q", Hq), ("k", Hk), ("v", Hk), ("qr", Hq), ("out", Hq))}
    lse = torch.zeros((Hq, T), device="cuda")
    kc, vc = (torch.full((P, page, Hk, D), NAN, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    table = fa.make_rope_table(D, base=500000.0, scaling="bands", factor=32.0)
    plan = fa.make_kv_plan_desc(t["q_lens"], t["kv"], ids, t["head"], t["table"], t["kv2"], t["cu"], t["pos"],
                                t["slots"], t["head2"], page_size=page, error_word=t["err"])
    desc = fa.make_chunk_desc(t["cu"], t["kv2"], t["table"], 8 * page, error_word=t["err"])
    ws = torch.empty(fa.fl_attn_chunk_workspace_size(x["q"], kc, desc), dtype=torch.uint8, device="cuda")

    def step():
        fa.fl_kv_plan(plan)
        fa.fl_kv_append(x["q"], x["k"], x["v"], x["qr"], kc, vc, t["slots"], rope=table, positions=t["pos"])
        fa.fl_attn_chunk(x["qr"], kc, vc, x["out"], lse, desc, ws)
        t["kv"].copy_(t["kv2"])
        t["head"].copy_(t["head2"])

    graph = None
    if captured:
        step()  # once with no tokens, outside the capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    history = [([], []) for _ in range(B)]
    for i, q_lens in enumerate(steps):
        n = sum(q_lens)
        new = {name: _rand((n, h, D), 100 * i + j) for j, (name, h) in enumerate((("q", Hq), ("k", Hk), ("v", Hk)))}
        for name in new:
            x[name][:n] = new[name].cuda()
        t["q_lens"].copy_(torch.tensor(q_lens, dtype=torch.int32))
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        assert int(t["err"].item()) == 0
        at = 0
        for b, m in enumerate(q_lens):
            pos = torch.arange(m) + len(history[b][0])
            turn = lambda y: ref.rope(y, pos, D, "half", base=500000.0, scaling="bands", factor=32.0)[0]  # noqa: E731
            rows = slice(at, at + m)
            history[b][0].extend(turn(new["k"][rows]).to(torch.bfloat16))
            history[b][1].extend(new["v"][rows])
            if m:
                want, wl, tol = ref.chunk_rows(turn(new["q"][rows]).to(torch.bfloat16), torch.stack(history[b][0]),
                                               torch.stack(history[b][1]), None)
                # a rotated bf16 value next to a rounding border may fall to the other
                # side (one step, 2^-7 of one of 64 products): 64 terms of |q k| / 8, a
                # few of them off, moves a score by under 0.02 and a row by 0.02 |v - O|
                err = (x["out"][rows].double().cpu() - want).abs()
                assert bool((err <= 2 * tol + 0.02).all()), f"step {i} request {b}: {(err - tol).max():.3e}"
                assert (lse[:, rows].double().cpu() - wl).abs().max() <= 0.02
            at += m
    assert t["kv"].tolist() == [len(h[0]) for h in history]
    assert int(t["head"].item()) == sum(-(-len(h[0]) // page) for h in history)


def test_refusals_of_the_binding():
    p = _problem([2], [20], 8, 2, 64, 16)
    q, kc, vc = (p[n].cuda() for n in ("q", "kc", "vc"))
    cu, kv, table = _ints(p["cu"]), _ints([20]), p["table"].cuda()
    d = fa.make_chunk_desc(cu, kv, table, 20)
    ws = torch.empty(fa.fl_attn_chunk_workspace_size(q, kc, d), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    with pytest.raises(ValueError, match="current device"):
        fa.fl_attn_chunk(q.cpu(), kc, vc, out, None, d, ws)
    with pytest.raises(fa.FlAttnError, match="needed"):
        fa.fl_attn_chunk(q, kc, vc, out, None, d, ws[:16])
    with pytest.raises(ValueError, match="workspace"):
        fa.fl_attn_chunk(q, kc, vc, out, None, d, ws.cpu())
    with pytest.raises(ValueError, match="error_word"):
        fa.make_chunk_desc(cu, kv, table, 20, error_word=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="desc"):
        # tensors of no GPU stand for those of another
        fa.fl_attn_chunk(q, kc, vc, out, None, fa.make_chunk_desc(cu.cpu(), kv.cpu(), table.cpu(), 20), ws)
    with pytest.raises(TypeError):
        fa.make_chunk_desc(cu.long(), kv, table, 20)
    with pytest.raises(ValueError):
        fa.make_chunk_desc(cu[:1], kv, table, 20)
    with pytest.raises(ValueError, match="contiguous"):
        fa.make_chunk_desc(cu, kv, torch.zeros((1, 8), dtype=torch.int32, device="cuda")[:, ::2], 20)
