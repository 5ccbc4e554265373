"""Rotary tables and the refusals of the rotary and serving-step entry points
(no GPU: every refusal comes before any CUDA call)."""
from __future__ import annotations

import ctypes

import pytest

import attention_variant_gb300 as fa
from attention_variant_gb300 import build as fbuild

torch = pytest.importorskip("torch")
from tests import serving_ref as ref  # noqa: E402

fake_addresses = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses (host-only test)")


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fa.load_library()


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
            dict(scaling="bands", factor=32.0, base=500000.0), dict(scaling="bands", factor=2.0, low=0.5, high=9.0),
            dict(scaling="ramp", factor=16.0, context=4096), dict(scaling="ramp", factor=40.0, magnitude=1.5)]


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("rot", [4, 32, 64, 128, 256])
def test_tables_hold_the_frequencies(lib, kw, rot):
    t = fa.make_rope_table(rot, **kw)
    f, m = ref.frequencies(rot, **kw)
    for i in range(rot // 2):
        want = f[i].item() / 6.283185307179586 % 1.0
        # a few roundings in 64 bits on either side
        assert abs(t.turns[i] / 2.0 ** 64 - want) <= 2.0 ** -48 * max(want, 2.0 ** -12)
    assert t.magnitude == pytest.approx(m, rel=2.0 ** -24)
    assert all(t.turns[i] == 0 for i in range(rot // 2, fa.FL_ROPE_MAX_PAIRS))


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=258), dict(layout=5), dict(scaling=9),
                                dict(base=1.0), dict(base=float("nan")), dict(scaling="linear", factor=0.0),
                                dict(scaling="base", factor=4.0, rot_dim=2), dict(scaling="bands", factor=2.0, context=0),
                                dict(scaling="ramp", factor=2.0, low=4.0, high=2.0), dict(magnitude=-1.0),
                                dict(scaling="base", factor=1e-9)])
def test_tables_refused(lib, kw):
    kw = dict(dict(rot_dim=64), **kw)
    with pytest.raises(fa.FlAttnError) as e:
        fa.make_rope_table(**kw)
    assert e.value.status == fa.FL_ERR_INVALID_ARG


def _t(shape, dtype=fa.FL_BF16, ptr=0x10000, strides=None):
    t = fa.FlTensor()
    t.ptr, t.dtype, t.ndim = ptr, dtype, len(shape)
    acc = 1
    for d in range(len(shape) - 1, -1, -1):
        t.sizes[d] = shape[d]
        t.strides[d] = acc if strides is None else strides[d]
        acc *= shape[d]
    return bytes(t)


def _rope_desc(table, positions=0, stride=0, offset=0, backward=0):
    return fa._ROPE_DESC.pack(ctypes.addressof(table), positions, stride, offset, backward)


@fake_addresses
def test_rope_refusals(lib):
    table = fa.make_rope_table(64)
    d = _rope_desc(table)
    q, k = _t((2, 5, 4, 64)), _t((2, 5, 2, 64))
    bad = lambda status, *a: lib.fl_rope(*a, None) == status  # noqa: E731
    inv = fa.FL_ERR_INVALID_ARG
    assert bad(inv, None, None, q, None, d)
    assert bad(inv, q, None, None, None, d)
    assert bad(inv, q, k, q, None, d)
    assert bad(inv, q, None, _t((2, 5, 4, 64), fa.FL_F32), None, d)
    assert bad(inv, q, None, _t((2, 5, 4, 128)), None, d)
    assert bad(inv, q, _t((2, 6, 2, 64)), q, _t((2, 6, 2, 64)), d)
    assert bad(inv, q, None, q, None, None)
    assert bad(inv, q, None, q, None, _rope_desc(fa.FlRopeTable()))
    assert bad(inv, _t((2, 5, 4, 32)), None, _t((2, 5, 4, 32)), None, d)  # rot_dim > D
    assert bad(inv, _t((5, 64)), None, _t((5, 64)), None, d)
    assert bad(inv, q, None, q, None, _rope_desc(table, stride=-1))
    assert bad(fa.FL_ERR_ALIGNMENT, q, None, q, None, _rope_desc(table, positions=0x1002))
    assert bad(fa.FL_ERR_ALIGNMENT, _t((2, 5, 4, 64), ptr=0x10004), None, q, None, d)
    huge = _t((1 << 16, 1 << 15, 1, 64))
    assert bad(fa.FL_ERR_UNSUPPORTED, huge, None, huge, None, d)


@fake_addresses
def test_append_refusals(lib):
    k, c, q = _t((7, 2, 64)), _t((5, 16, 2, 64)), _t((7, 8, 64))
    table = fa.make_rope_table(64)
    good = _rope_desc(table, positions=0x1000)
    bad = lambda status, *a: lib.fl_kv_append(*a, None) == status  # noqa: E731
    inv = fa.FL_ERR_INVALID_ARG
    assert bad(inv, None, None, k, None, c, c, 0x1000, None)
    assert bad(inv, None, k, _t((8, 2, 64)), None, c, c, 0x1000, None)
    assert bad(inv, None, k, k, None, _t((5, 16, 3, 64)), c, 0x1000, None)
    assert bad(inv, None, k, k, None, c, _t((6, 16, 2, 64)), 0x1000, None)
    assert bad(inv, None, k, k, None, c, c, None, None)
    assert bad(fa.FL_ERR_ALIGNMENT, None, k, k, None, c, c, 0x1004, None)
    assert bad(inv, q, k, k, None, c, c, 0x1000, None)
    assert bad(inv, _t((6, 8, 64)), k, k, _t((6, 8, 64)), c, c, 0x1000, None)
    assert bad(inv, q, k, k, _t((7, 9, 64)), c, c, 0x1000, None)
    assert bad(inv, q, k, k, q, c, c, 0x1000, _rope_desc(table))  # no positions
    assert bad(inv, q, k, k, q, c, c, 0x1000, _rope_desc(table, positions=0x1000, backward=1))
    assert bad(inv, None, _t((7, 2, 32)), _t((7, 2, 32)), None, _t((5, 16, 2, 32)), _t((5, 16, 2, 32)), 0x1000, good)


def _plan_desc(**kw):
    d = fa.FlKvPlanDesc()
    base = dict(batch=4, page_size=16, max_tokens=8, n_free=3, block_table_stride=5, q_lens=0x1000, kv_lens=0x2000,
                free_pages=0x3000, free_head=0x4000, block_table=0x5000, kv_lens_out=0x6000, cu_q=0x7000,
                positions=0x8000, slots=0x9000, free_head_out=0xA000)
    for n, v in dict(base, **kw).items():
        setattr(d, n, v)
    return d


@fake_addresses
def test_plan_refusals(lib):
    inv = fa.FL_ERR_INVALID_ARG
    for status, kw in ((inv, dict(batch=0)), (inv, dict(max_tokens=-1)), (inv, dict(n_free=-1)),
                       (inv, dict(block_table_stride=0)), (fa.FL_ERR_UNSUPPORTED, dict(page_size=48)),
                       (fa.FL_ERR_UNSUPPORTED, dict(page_size=8)), (fa.FL_ERR_UNSUPPORTED, dict(page_size=512)),
                       (inv, dict(q_lens=None)), (inv, dict(kv_lens=None)), (inv, dict(free_pages=None)),
                       (inv, dict(free_head=None)), (inv, dict(block_table=None)), (inv, dict(kv_lens_out=None)),
                       (inv, dict(cu_q=None)), (inv, dict(positions=None)), (inv, dict(free_head_out=None)),
                       (fa.FL_ERR_ALIGNMENT, dict(q_lens=0x1001)), (fa.FL_ERR_ALIGNMENT, dict(slots=0x9004)),
                       (inv, dict(kv_lens_out=0x2000)), (inv, dict(kv_lens_out=0x200C)), (inv, dict(cu_q=0x1000)),
                       (inv, dict(free_head_out=0x4000))):
        assert lib.fl_kv_plan(ctypes.byref(_plan_desc(**kw)), None) == status, kw
    assert lib.fl_kv_plan(None, None) == inv


def _chunk_desc(**kw):
    d = fa.FlChunkDesc()
    base = dict(batch=3, causal=1, cu_q=0x1000, kv_lens=0x2000, max_kv_len=100, block_table=0x3000,
                block_table_stride=7, softcap=20.0)
    for n, v in dict(base, **kw).items():
        setattr(d, n, v)
    return d


@fake_addresses
def test_chunk_refusals(lib):
    q, c = _t((9, 8, 64)), _t((20, 16, 2, 64))
    inv, uns, ali = fa.FL_ERR_INVALID_ARG, fa.FL_ERR_UNSUPPORTED, fa.FL_ERR_ALIGNMENT

    def st(q=q, k=c, v=c, out=None, lse=None, ws=0x100000, nbytes=1 << 40, **kw):
        return lib.fl_attn_chunk(q, k, v, out or q, lse, ctypes.byref(_chunk_desc(**kw)), ws, nbytes, None)

    assert st(q=None, out=q) == inv and st(k=None) == inv and st(v=None) == inv
    assert st(v=_t((21, 16, 2, 64))) == inv
    assert st(out=_t((9, 8, 128))) == inv
    assert st(lse=_t((9, 8), fa.FL_F32)) == inv
    assert st(q=_t((9, 8, 32)), k=_t((20, 16, 2, 32)), v=_t((20, 16, 2, 32))) == uns
    assert st(q=_t((9, 8, 128))) == inv
    assert st(q=_t((9, 7, 64))) == inv
    assert st(q=_t((9, 258, 64))) == uns  # 129 query heads per KV head
    assert st(k=_t((20, 48, 2, 64)), v=_t((20, 48, 2, 64))) == uns
    for status, kw in ((inv, dict(batch=0)), (inv, dict(max_kv_len=0)), (inv, dict(window=-1)),
                       (inv, dict(window=5, causal=0)), (uns, dict(score_mod=fa.FL_MOD_ALIBI)),
                       (inv, dict(score_mod=fa.FL_MOD_SOFTCAP, softcap=0.0)), (inv, dict(scale=-1.0)),
                       (inv, dict(scale=float("inf"))), (inv, dict(block_table_stride=6)),
                       (inv, dict(block_table=None)), (ali, dict(block_table=0x3002)), (inv, dict(cu_q=None)),
                       (inv, dict(kv_lens=None)), (ali, dict(cu_q=0x1002)), (inv, dict(ws=None)),
                       (ali, dict(ws=0x100080)), (inv, dict(nbytes=16))):
        assert st(**kw) == status, kw
    short = _t((3, 99, 2, 64))
    assert st(k=short, v=short, block_table=None) == inv  # max_kv_len > S_max
    n = ctypes.c_size_t()
    assert lib.fl_attn_chunk_workspace_size(q, c, ctypes.byref(_chunk_desc()), None) == inv
    assert lib.fl_attn_chunk_workspace_size(q, c, ctypes.byref(_chunk_desc(batch=0)), ctypes.byref(n)) == inv
