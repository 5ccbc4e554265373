"""GPU parity of rotary positions with the float64 definition: both layouts,
part of the head, scaled contexts, far positions, strides, in place, the
backward, and their use in a training step."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import attention_variant_gb300 as fa  # noqa: E402
from tests import serving_ref as ref  # noqa: E402


def _rand(shape, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def _close(got, want, bound, dtype, what):
    # the fp32 result's bound, and half a step of the output type
    half = torch.finfo(dtype).eps / 2
    err = (got.double().cpu() - want).abs()
    tol = bound * (1 + half) + half * want.abs()
    worst = (err - tol).max().item()
    assert worst <= 0, f"{what}: {worst:.3e} past the bound ({err.max():.3e} off)"


def _check(B, S, Hq, Hk, D, rot, layout, dtype, pos, *, backward=False, inplace=False, **scaling):
    q, k = _rand((B, S, Hq, D), 1, dtype), _rand((B, S, Hk, D), 2, dtype)
    table = fa.make_rope_table(rot, layout=layout, **scaling)
    qd, kd = q.cuda(), k.cuda()
    qo, ko = (qd, kd) if inplace else (torch.full_like(qd, float("nan")), torch.full_like(kd, float("nan")))
    fa.fl_rope(qd, kd, qo, ko, table, positions=pos.to(torch.int32).cuda(), backward=backward)
    torch.cuda.synchronize()
    at = pos if pos.dim() == 2 else pos.expand(B, S)
    for got, x, name in ((qo, q, "q"), (ko, k, "k")):
        want, bound = ref.rope(x, at, rot, layout, backward=backward, **scaling)
        _close(got, want, bound, dtype, f"{name} {layout} rot {rot} of {D}")
        assert torch.equal(got[..., rot:].cpu(), x[..., rot:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 32), (80, 44), (64, 2), (256, 256), (48, 24)])
def test_layouts_and_parts(dtype, layout, D, rot):
    _check(2, 37, 6, 2, D, rot, layout, dtype, torch.arange(74).reshape(2, 37) * 13)


@pytest.mark.parametrize("scaling", [dict(scaling="linear", factor=8.0), dict(scaling="base", factor=4.0),
                                     dict(scaling="bands", factor=32.0, base=500000.0),
                                     dict(scaling="ramp", factor=16.0, context=4096),
                                     dict(scaling="ramp", factor=4.0, context=2048, low=2.0, high=16.0,
                                          magnitude=1.25)])
@pytest.mark.parametrize("backward", [False, True])
def test_scaled_contexts(scaling, backward):
    pos = torch.randint(0, 1 << 20, (3, 50), generator=torch.Generator().manual_seed(5))
    _check(3, 50, 4, 4, 64, 64, "half", torch.float32, pos, backward=backward, **scaling)


def test_far_and_negative_positions():
    pos = torch.tensor([0, 1, -1, -77777, 1 << 20, (1 << 31) - 1, -(1 << 31), 123456789])
    for layout in ("half", "interleaved"):
        _check(1, 8, 4, 1, 128, 128, layout, torch.float32, pos)


@pytest.mark.parametrize("B,S,Hq,Hk", [(1, 1, 1, 1), (1, 1, 32, 8), (3, 1, 5, 1), (1, 2049, 16, 2),
                                       (5, 333, 12, 12)])
def test_sizes(B, S, Hq, Hk):
    _check(B, S, Hq, Hk, 64, 64, "half", torch.bfloat16, torch.arange(S) + 100)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place(layout):
    _check(2, 65, 4, 2, 96, 64, layout, torch.bfloat16, torch.arange(65), inplace=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_views_and_offset(dtype):
    # q, k as slices of one projection, stored head-major; rows of no call stay
    B, S, H, D = 2, 21, 3, 64
    x = _rand((B, 3 * H, S, D), 3, dtype).cuda()
    out = torch.full((B, S, 4 * H, D), 7.0, dtype=dtype, device="cuda")
    q, k = x[:, :H].transpose(1, 2), x[:, H:2 * H].transpose(1, 2)
    table = fa.make_rope_table(64)
    fa.fl_rope(q, k, out[:, :, :H], out[:, :, 2 * H:3 * H], table, offset=1000)
    pos = (torch.arange(S) + 1000).expand(B, S)
    for got, src in ((out[:, :, :H], q), (out[:, :, 2 * H:3 * H], k)):
        want, bound = ref.rope(src.cpu(), pos, 64, "half")
        _close(got, want, bound, dtype, "strided")
    assert bool((out[:, :, H:2 * H] == 7).all()) and bool((out[:, :, 3 * H:] == 7).all())


def test_fp32_at_odd_addresses():
    # an fp32 tensor may start at any 4-byte address and have any strides
    base = _rand((5 * 67 + 1,), 4, torch.float32).cuda()
    x = torch.as_strided(base, (1, 5, 1, 64), (5 * 67, 67, 67, 1), 1)
    out = torch.empty_like(x)
    fa.fl_rope(x, None, out, None, fa.make_rope_table(64, layout="interleaved"))
    want, bound = ref.rope(x.cpu(), torch.arange(5)[None], 64, "interleaved")
    _close(out, want, bound, torch.float32, "odd address")


def test_ragged_rows_alone():
    q = _rand((29, 4, 64), 6, torch.bfloat16)
    pos = torch.arange(29) % 7
    out = torch.empty_like(q, device="cuda")
    fa.fl_rope(q.cuda(), None, out, None, fa.make_rope_table(64), positions=pos.to(torch.int32).cuda())
    want, bound = ref.rope(q, pos, 64, "half")
    _close(out, want, bound, torch.bfloat16, "ragged")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_backward_is_the_transposed_map(layout):
    # against differences: the map is linear, so (R(x + h e) - R(x)) / h is its
    # column e up to the roundings of R's fp32 results (2^-24 of values below 8
    # over h = 4: 2^-22 each side)
    D, rot = 12, 8
    table = fa.make_rope_table(rot, layout=layout, scaling="ramp", factor=4.0, context=512)
    x = _rand((1, 1, 1, D), 7, torch.float32).cuda()
    pos = torch.tensor([5], dtype=torch.int32, device="cuda")

    def apply(t, backward=False):
        out = torch.empty_like(t)
        fa.fl_rope(t, None, out, None, table, positions=pos, backward=backward)
        return out.reshape(-1).cpu()

    eye = torch.eye(D).cuda()
    jac = torch.stack([(apply(x + 4 * eye[e]) - apply(x)) / 4 for e in range(D)], 1)
    for e in range(D):
        grad = apply(eye[e].reshape(1, 1, 1, D), backward=True)
        assert (grad - jac[e]).abs().max() <= 4 * 2.0 ** -22


def test_training_step_gradients():
    """rope -> fl_attn_fwd -> fl_attn_bwd -> rope's backward against float64
    autograd of the whole; the attention backward's own tolerance (10 * 2^-9 of
    the gradient's largest value) plus two bf16 roundings through the rotation."""
    B, S, H, Hk, D = 2, 200, 4, 2, 64
    q, k, v, do = (_rand((B, S, h, D), 10 + i, torch.bfloat16) for i, h in enumerate((H, Hk, Hk, H)))
    table = fa.make_rope_table(D, base=500000.0, scaling="bands", factor=32.0)
    qd, kd, vd, dod = (x.cuda() for x in (q, k, v, do))
    qr, kr, out = torch.empty_like(qd), torch.empty_like(kd), torch.empty_like(qd)
    lse = torch.empty(B, H, S, device="cuda")
    desc = fa.make_desc(mask="causal")
    fa.fl_rope(qd, kd, qr, kr, table)
    fa.fl_attn_fwd(qr, kr, vd, out, lse, desc)
    dq, dk, dv = (torch.empty_like(x) for x in (qd, kd, vd))
    ws = torch.empty(fa.fl_attn_bwd_workspace_size(qr, kr, desc), dtype=torch.uint8, device="cuda")
    fa.fl_attn_bwd(qr, kr, vd, out, lse, dod, dq, dk, dv, desc, ws)
    fa.fl_rope(dq, dk, dq, dk, table, backward=True)
    torch.cuda.synchronize()

    x = [t.double().requires_grad_() for t in (q, k, v)]
    f, m = ref.frequencies(D, base=500000.0, scaling="bands", factor=32.0)
    t = torch.arange(S).double()[:, None, None] * f

    def turn(y):
        a, b = y[..., :32], y[..., 32:]
        return m * torch.cat((a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()), -1)

    qq, kk = turn(x[0]).transpose(1, 2), turn(x[1]).transpose(1, 2).repeat_interleave(2, 1)
    z = qq @ kk.transpose(2, 3) / 8
    z = z.masked_fill(torch.ones(S, S, dtype=torch.bool).triu(1), float("-inf"))
    (torch.softmax(z, -1) @ x[2].transpose(1, 2).repeat_interleave(2, 1)).transpose(1, 2).backward(do.double())
    for name, got, want in (("dq", dq, x[0].grad), ("dk", dk, x[1].grad), ("dv", dv, x[2].grad)):
        err = (got.double().cpu() - want).abs().max().item()
        # 10 * 2^-9 from the attention; the rotated bf16 q and k it ran on are off
        # by 2^-8 of a value, which moves z by up to 2 * 2^-8 |z| (|z| < 6) and P
        # and dS by as much
        tol = (10 * 2.0 ** -9 + 2 * 2.0 ** -8 * 6 + 2 * 2.0 ** -8) * want.abs().max().item()
        assert err <= tol, f"{name}: {err:.3e} > {tol:.3e}"


def test_captured_and_on_another_stream():
    x = _rand((2, 64, 8, 64), 8, torch.bfloat16).cuda()
    table = fa.make_rope_table(64)
    want, out = torch.empty_like(x), torch.zeros_like(x)
    fa.fl_rope(x, None, want, None, table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fa.fl_rope(x, None, out, None, table)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    with torch.cuda.stream(side):
        fa.fl_rope(x, None, out, None, table)
    side.synchronize()
    assert torch.equal(out, want)


def test_cpu_tensors_and_wrong_positions_are_refused():
    x = _rand((1, 4, 2, 64), 9, torch.bfloat16).cuda()
    table = fa.make_rope_table(64)
    with pytest.raises(ValueError, match="current device"):
        fa.fl_rope(x, None, x.cpu(), None, table)
    with pytest.raises(TypeError, match="int32"):
        fa.fl_rope(x, None, x, None, table, positions=torch.arange(4, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        fa.fl_rope(x, None, x, None, table, positions=torch.zeros(5, dtype=torch.int32, device="cuda"))
    with pytest.raises(fa.FlAttnError):
        fa.fl_rope(x, x, x, None, table)
    with pytest.raises(fa.FlAttnError):
        fa.fl_rope(x, None, torch.empty(1, 4, 2, 72, dtype=x.dtype, device="cuda"), None, table)
    with pytest.raises(ValueError, match="shape"):
        # rows of a batch have one position each
        fa.fl_rope(x[0], None, x[0], None, table, positions=torch.zeros((4, 2), dtype=torch.int32, device="cuda"))
