"""GPU parity of the serving-step entry points where lengths, offsets and windows
are at the limits of what their documentation allows."""
from __future__ import annotations

import math
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import attention_variant_gb300 as fa  # noqa: E402
from tests.test_gpu_serving import _compare, _expected, _ints, _launch, _problem, _run_plan  # noqa: E402


# ------------------------------------------------------------------ chunks


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_chunk_blocks_without_keys_between_long_ones(D, page, softcap):
    # whole row blocks before the sequence (no key, so nothing to load), each
    # followed in its CTA by items that fill the rings of tiles; several times
    q_lens, kv_lens = [], []
    for i in range(24):
        q_lens += [200, 40, 70]
        kv_lens += [(50, 0, 120, 3)[i % 4], 900 + 37 * i, (0, 5)[i % 2]]
    p = _problem(q_lens, kv_lens, 4, 1, D, page, seed=7)
    want = _expected(p, softcap=softcap)
    got = _launch(p, calls=4, softcap=softcap)
    for g in got:
        _compare(g, want, "blocks without keys")
        assert torch.equal(g[0], got[0][0]) and torch.equal(g[1], got[0][1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 100, 1 << 30])
def test_chunk_windows_as_long_as_an_int_goes(D, window):
    # rows before the sequence and rows with keys in one entry, in row blocks and
    # in few rows: the window hides nothing
    p = _problem([60, 3, 300, 1], [20, 1, 290, 500], 8, 2, D, 16, seed=3)
    want = _expected(p)
    for kw in (dict(window=window), dict()):
        got, = _launch(p, **kw)
        _compare(got, want, f"window {window}")


def _error_of(p, kv_lens, max_kv, **kw):
    err = _ints([0])
    d = fa.make_chunk_desc(_ints(p["cu"]), _ints(kv_lens), p["table"].cuda(), max_kv, error_word=err, **kw)
    q, kc, vc = (p[n].cuda() for n in ("q", "kc", "vc"))
    ws = torch.empty(fa.fl_attn_chunk_workspace_size(q, kc, d), dtype=torch.uint8, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((q.shape[1], q.shape[0]), 7.0, device="cuda")
    fa.fl_attn_chunk(q, kc, vc, out, lse, d, ws)
    torch.cuda.synchronize()
    return int(err.item()), (out, lse)


@pytest.mark.parametrize("n", [1, 40])
def test_chunk_lengths_past_the_bound_are_reported(n):
    # a request that outgrew max_kv_len: its rows are no longer where they were
    # meant to be, and the caller can learn of it; the others are right
    p = _problem([n, 3], [100, 60], 8, 2, 64, 16)
    want, lse, tol = _expected(p)
    for max_kv in (100, 99, 61):
        err, got = _error_of(p, [100, 60], max_kv, strict_lengths=True)
        assert err == (fa.FL_DEVERR_LENGTHS if max_kv < 100 else 0)
        rows = slice(0 if max_kv == 100 else n, n + 3)
        _compare((got[0][rows], got[1][:, rows]), (want[rows], lse[:, rows], tol[rows]), f"bound {max_kv}")
    # lengths below 0 are never right
    for strict in (False, True):
        err, got = _error_of(p, [-5, 60], 100, strict_lengths=strict)
        assert err == fa.FL_DEVERR_LENGTHS
        assert not bool(got[0][:n].any()) and bool((got[1][:, :n] == -math.inf).all())
        _compare((got[0][n:], got[1][:, n:]), (want[n:], lse[:, n:], tol[n:]), "beside a negative length")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [0.25, 1000.0, 16384.0])
def test_chunk_small_and_large_softcaps(D, cap):
    p = _problem([50, 1, 3], [300, 400, 90], 8, 2, D, 32)
    want, lse, tol = _expected(p, softcap=cap)
    (o, l), = _launch(p, softcap=cap)
    # cap (1 - 2 / (1 + 2^x)) in fp32: 2^x, the sum, the reciprocal and the last sum round at
    # the size of 1, each at most 2^-22 (twice their sum allowed): a score is off by d, the
    # LSE by as much, a weight by 2 d, and O by that times |v - O| <= 2 max |v|
    d = 8 * 2.0 ** -22 * cap
    v = max(x.float().abs().max().item() for x in p["v"])
    assert ((o.double().cpu() - want).abs() <= tol + 4 * d * v).all()
    assert (l.double().cpu() - lse).abs().max() <= 2e-4 + d


def test_chunk_workspaces_that_are_not_one_piece():
    # as many elements as are needed, but not as many bytes behind the address
    p = _problem([2], [20], 8, 2, 64, 16)
    q, kc, vc = (p[n].cuda() for n in ("q", "kc", "vc"))
    d = fa.make_chunk_desc(_ints(p["cu"]), _ints([20]), p["table"].cuda(), 20)
    n = fa.fl_attn_chunk_workspace_size(q, kc, d)
    out = torch.full_like(q, 7.0)
    for ws in (torch.empty(1, dtype=torch.uint8, device="cuda").expand(n),
               torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2],
               torch.empty((64, n), dtype=torch.uint8, device="cuda").t()):
        with pytest.raises(ValueError, match="workspace"):
            fa.fl_attn_chunk(q, kc, vc, out, None, d, ws)
    assert bool((out == 7).all())
    ws = torch.empty((2, n // 8 + 1), dtype=torch.float32, device="cuda")
    fa.fl_attn_chunk(q, kc, vc, out, None, d, ws)
    torch.cuda.synchronize()
    _compare((out, None), _expected(p), "workspace of floats")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,first", [(60, "blocks"), (12, "few")])
def test_chunk_replays_follow_the_lengths(T, first, D):
    # one captured call with work of both kinds, whose requests change from replay to
    # replay: each has a plan of its own, in the workspace that held the last one's
    rng = random.Random(T)
    B = 4 if first == "blocks" else 8
    page, Hq, Hk, width = 16, 8, 1, 64
    fixed = dict(cu=_ints([0] * (B + 1)), kv=_ints([1] * B), table=_ints([[0] * width] * B))
    q = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.zeros((B * width + 2, page, Hk, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    out, lse = torch.empty_like(q), torch.empty((Hq, T), device="cuda")
    err = _ints([0])
    d = fa.make_chunk_desc(fixed["cu"], fixed["kv"], fixed["table"], 900, error_word=err)
    n = fa.fl_attn_chunk_workspace_size(q, kc, d)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    fa.fl_attn_chunk(q, kc, vc, out, lse, d, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fl_attn_chunk(q, kc, vc, out, lse, d, ws)
    for i in range(8):
        q_lens = [rng.randrange(0, 2) for _ in range(B - 1)]
        q_lens.insert(rng.randrange(B), T - sum(q_lens) - 3)
        kv_lens = [m + rng.randrange(0, 800) for m in q_lens]
        p = _problem(q_lens, kv_lens, Hq, Hk, D, page, seed=i)
        m = sum(q_lens)
        q[:m].copy_(p["q"])
        for dst, src in ((kc, p["kc"]), (vc, p["vc"])):
            dst[: src.shape[0]].copy_(src)
        fixed["cu"].copy_(torch.tensor(p["cu"], dtype=torch.int32))
        fixed["kv"].copy_(torch.tensor(kv_lens, dtype=torch.int32))
        fixed["table"][:, : p["table"].shape[1]].copy_(p["table"])
        want = _expected(p)
        for _ in range(3):
            out.fill_(7.0)
            lse.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            _compare((out[:m], lse[:, :m]), want, f"replay {i} q {q_lens} kv {kv_lens}")
            assert bool((out[m:] == 7).all()) and bool((lse[:, m:] == 7).all())
    assert int(err.item()) == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,Hq", [(2, 1), (2, 4), (1, 8), (4, 4), (1, 16)])
@pytest.mark.parametrize("L", [4, 5, 7])
def test_chunk_few_rows_keep_both_terms_of_p(n, Hq, D, L):
    # values that cancel: O is what the weights differ by, which one bf16 per
    # weight does not hold
    q, k, v = torch.zeros(n, Hq, D), torch.zeros(L, 1, D), torch.zeros(L, 1, D)
    q[..., :2] = torch.tensor([1.0, 1.5, 0.75, 2.0])[torch.arange(n * Hq) % 4].view(n, Hq, 1)
    k[:, 0, 0], k[:, 0, 1] = -1.25, torch.tensor([(5 * j % 7 - 3) * 2.0 ** -9 for j in range(L)])
    v[:, 0] = torch.tensor([1.0, -1.0, -1.0, 1.0, 0.0, 1.0, -1.0])[:L, None]
    p = _problem([n], [L], Hq, 1, D, 16, causal=False)
    for name, x in (("q", q), ("k", k), ("v", v)):
        x = x.to(torch.bfloat16)
        if name == "q":
            p["q"] = x
            continue
        p[name][0] = x
        p[name + "c"][int(p["table"][0, 0]), :L] = x
    want, lse, _ = _expected(p, causal=False, scale=1.0)
    z = q[..., :1].double() * k[:, 0].double().sum(-1)  # [n, Hq, L]
    w = torch.exp(z)

    def out_of(weights):  # of what the kernel multiplies V by; the sum is of w itself
        return (weights @ v[:, 0, 0].double() / w.sum(-1))[..., None].expand(n, Hq, D)

    first = w.float().to(torch.bfloat16).double()
    rest = w - first
    assert (out_of(w) - want).abs().max() < 1e-12
    # the second term's own rounding (2^-8 of it), the output's (2^-8), and 2^x, the sums and
    # the reciprocal in fp32: 2^-22 of weights that sum to 1, four times
    tol = 2.0 ** -8 * (rest.abs().sum(-1) / w.sum(-1)).max() + 2.0 ** -8 * want.abs() + 4 * 2.0 ** -22
    assert (out_of(first) - want).abs().max() > 8 * tol.max()  # the first term alone
    (o, _), = _launch(p, causal=False, scale=1.0)
    assert ((o.double().cpu() - want).abs() <= tol).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("Hq,Hk", [(14, 2), (40, 1), (6, 2), (8, 2), (5, 1)])
def test_chunk_rows_depend_on_their_own_request(Hq, Hk, D, softcap):
    # groups that do not fill the 128 rows of a block, and blocks that end inside it:
    # what else lies there (rows of loud neighbours, what Q's buffers held before) must
    # not reach a row's bits, not even by the moment at which a warp rescales
    q_lens, kv_lens = [45, 150, 1, 45, 2, 70], [600, 700, 800, 500, 300, 70]
    quiet = _problem(q_lens, kv_lens, Hq, Hk, D, 32, seed=1)
    others = [0, 2, 4, 5]  # the neighbours; 1 and 3 stay
    kw = dict(softcap=softcap)
    want = _expected(quiet, **kw)
    (o0, l0), = _launch(quiet, **kw)
    _compare((o0, l0), want, "quiet")
    for loud in (30.0, 1e4):
        p = dict(quiet, q=quiet["q"].clone())
        for b in others:
            p["q"][p["cu"][b]: p["cu"][b + 1]] *= loud
        for o, l in _launch(p, calls=3, **kw):
            for b in (1, 3):
                rows = slice(p["cu"][b], p["cu"][b + 1])
                assert torch.equal(o[rows], o0[rows]) and torch.equal(l[:, rows], l0[:, rows])
    for o, l in _launch(quiet, calls=3, **kw):  # after the loud ones
        assert torch.equal(o, o0) and torch.equal(l, l0)


# ------------------------------------------------------------------ book-keeping


@pytest.mark.parametrize("max_tokens", [0, 1, 45, 46, 47, 59])
@pytest.mark.parametrize("slots", [True, False])
def test_plan_takes_every_page_whatever_it_lists(max_tokens, slots):
    # pages that begin with a token past max_tokens are in the table all the same
    got, want = _run_plan([40, 20], [0, 10], 16, max_tokens=max_tokens, slots=slots)
    assert got == (want if max_tokens else 0)


@pytest.mark.parametrize("B", [700, 1024, 2300])
@pytest.mark.parametrize("max_tokens", [0, 700, 40000])
def test_plan_takes_every_page_of_many_requests(B, max_tokens):
    # the limit falls into any of the scans, or a request of many pages
    rng = random.Random(B + max_tokens)
    q = [rng.choice((0, 1, 1, 30, 300)) for _ in range(B)]
    q[B // 2] = 30000
    kv = [rng.randrange(0, 300) for _ in range(B)]
    got, want = _run_plan(q, kv, 16, head=3, seed=B, max_tokens=max_tokens)
    assert got == (want if max_tokens else 0)


@pytest.mark.parametrize("max_tokens", [0, 5])
def test_plan_reports_pages_that_unlisted_tokens_lack(max_tokens):
    lengths = fa.FL_DEVERR_LENGTHS if max_tokens else 0
    assert _run_plan([40, 20], [0, 10], 16, n_free=2, max_tokens=max_tokens)[0] == fa.FL_DEVERR_PAGES | lengths
    assert _run_plan([40, 1], [0, 3], 16, width=2, max_tokens=max_tokens)[0] == fa.FL_DEVERR_PAGES | lengths
