"""The refusals of the 8-bit KV cache's entry points (no GPU: every refusal comes before any CUDA call)."""
from __future__ import annotations

import pytest

import attention_variant_gb300 as fa
from attention_variant_gb300 import build as fbuild
from tests.test_serving_host import _rope_desc, _t

torch = pytest.importorskip("torch")
fake_addresses = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses (host-only test)")

INV, UNS, ALI = fa.FL_ERR_INVALID_ARG, fa.FL_ERR_UNSUPPORTED, fa.FL_ERR_ALIGNMENT


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fa.load_library()


def _cache(P=5, page=32, Hk=2, D=64, **kw):
    return _t((P, page, Hk, D), kw.pop("dtype", fa.FL_E4M3), **kw)


def _scale(P=5, blocks=2, Hk=2, **kw):
    return _t((P, blocks, Hk), kw.pop("dtype", fa.FL_F32), **kw)


# caches and scales that no entry point takes: (status, k_cache, v_cache, k_scale, v_scale)
BAD = [
    (INV, None, _cache(), _scale(), _scale()),
    (INV, _cache(), None, _scale(), _scale()),
    (INV, _cache(), _cache(), None, _scale()),
    (INV, _cache(), _cache(), _scale(), None),
    (INV, _cache(dtype=fa.FL_BF16), _cache(), _scale(), _scale()),
    (INV, _cache(), _cache(dtype=fa.FL_F32), _scale(), _scale()),
    (INV, _cache(), _cache(P=6), _scale(), _scale()),
    (INV, _cache(), _cache(), _scale(dtype=fa.FL_BF16, Hk=8), _scale()),
    (INV, _cache(), _cache(), _scale(P=4), _scale()),
    (INV, _cache(), _cache(), _scale(Hk=3), _scale()),
    (INV, _cache(), _cache(), _scale(blocks=3), _scale()),            # does not divide the page
    (INV, _cache(), _cache(), _scale(), _scale(blocks=1)),            # not the block of K
    (UNS, _cache(), _cache(), _scale(blocks=4), _scale(blocks=4)),    # 8 keys
    (UNS, _cache(page=96), _cache(page=96), _scale(), _scale()),      # 48 keys
    (UNS, _cache(page=512), _cache(page=512), _scale(blocks=1), _scale(blocks=1)),
    (INV, _cache(), _cache(), _scale(strides=(4, 1, 2)), _scale()),   # heads not contiguous
    (ALI, _cache(), _cache(), _scale(ptr=0x10002), _scale()),
    (ALI, _cache(ptr=0x10008), _cache(), _scale(), _scale()),
    (ALI, _cache(strides=(4104, 128, 64, 1)), _cache(), _scale(), _scale()),
]


@fake_addresses
@pytest.mark.parametrize("i", range(len(BAD)))
def test_caches_refused(lib, i):
    status, kc, vc, ks, vs = BAD[i]
    k, q = _t((7, 2, 64)), _t((7, 8, 64))
    assert lib.fl_kv_append_fp8(None, k, k, None, kc, vc, ks, vs, 0x1000, None, None) == status
    assert lib.fl_kv_read_fp8(kc, vc, ks, vs, 0x1000, k, k, None) == status
    d = _desc()
    got = lib.fl_attn_chunk_fp8(q, kc, vc, ks, vs, q, None, d, 0x100000, 1 << 40, None)
    assert got == status or (status == UNS and got == UNS)


def _desc(**kw):
    d = fa.FlChunkDesc()
    base = dict(causal=1, batch=4, cu_q=0x1000, kv_lens=0x2000, max_kv_len=90, block_table=0x3000, block_table_stride=40)
    for n, v in dict(base, **kw).items():
        setattr(d, n, v)
    return d


@fake_addresses
def test_append_refusals(lib):
    k, q = _t((7, 2, 64)), _t((7, 8, 64))
    c = (_cache(), _cache(), _scale(), _scale())
    bad = lambda status, *a: lib.fl_kv_append_fp8(*a, None) == status  # noqa: E731
    table = fa.make_rope_table(64)
    assert bad(INV, None, None, k, None, *c, 0x1000, None)
    assert bad(INV, None, k, None, None, *c, 0x1000, None)
    assert bad(INV, None, k, _t((8, 2, 64)), None, *c, 0x1000, None)
    assert bad(INV, None, _t((7, 3, 64)), _t((7, 3, 64)), None, *c, 0x1000, None)
    assert bad(INV, None, _t((7, 2, 64), fa.FL_F32), k, None, *c, 0x1000, None)
    assert bad(INV, q, k, k, None, *c, 0x1000, None)
    assert bad(INV, _t((6, 8, 64)), k, k, _t((6, 8, 64)), *c, 0x1000, None)
    assert bad(INV, None, k, k, None, *c, None, None)
    assert bad(ALI, None, k, k, None, *c, 0x1004, None)
    assert bad(INV, q, k, k, q, *c, 0x1000, _rope_desc(table))
    assert bad(INV, q, k, k, q, *c, 0x1000, _rope_desc(table, positions=0x1000, backward=1))
    assert bad(INV, None, k, k, None, *c, 0x1000, _rope_desc(fa.make_rope_table(128), positions=0x1000))
    w = _t((7, 2, 32))
    assert bad(UNS, None, w, w, None, _cache(D=32), _cache(D=32), *c[2:], 0x1000, None)
    m = _t((7, 9000, 64))
    assert bad(UNS, None, m, m, None, _cache(Hk=9000), _cache(Hk=9000), _scale(Hk=9000), _scale(Hk=9000), 0x1000, None)
    # and e4m3 is no type of the other append's
    assert lib.fl_kv_append(None, k, k, None, c[0], c[1], 0x1000, None, None) == INV


@fake_addresses
def test_read_refusals(lib):
    k = _t((7, 2, 64))
    c = (_cache(), _cache(), _scale(), _scale())
    bad = lambda status, *a: lib.fl_kv_read_fp8(*a, None) == status  # noqa: E731
    assert bad(INV, *c, None, k, k)
    assert bad(ALI, *c, 0x1004, k, k)
    assert bad(INV, *c, 0x1000, None, k)
    assert bad(INV, *c, 0x1000, k, None)
    assert bad(INV, *c, 0x1000, k, _t((7, 2, 64), fa.FL_F32))
    assert bad(INV, *c, 0x1000, _t((7, 2, 64), fa.FL_E4M3), k)
    assert bad(INV, *c, 0x1000, k, _t((8, 2, 64)))
    assert bad(INV, *c, 0x1000, _t((7, 3, 64)), _t((7, 3, 64)))
    assert bad(UNS, _cache(D=32), _cache(D=32), *c[2:], 0x1000, _t((7, 2, 32)), _t((7, 2, 32)))
    f = _t((7, 2, 64), fa.FL_F32, strides=(130, 64, 1))
    assert bad(ALI, *c, 0x1000, f, f)
    f = _t((7, 2, 64), fa.FL_F32, ptr=0x10004)
    assert bad(ALI, *c, 0x1000, f, f)


@fake_addresses
def test_chunk_refusals(lib):
    q = _t((7, 8, 64))
    c = (_cache(), _cache(), _scale(), _scale())
    run = lambda d, qq=q, o=q, lse=None, ws=0x100000, n=1 << 40, cc=c: lib.fl_attn_chunk_fp8(  # noqa: E731
        qq, *cc, o, lse, d, ws, n, None)
    assert run(None) == INV
    assert run(_desc(batch=0)) == INV
    assert run(_desc(max_kv_len=0)) == INV
    assert run(_desc(window=5, causal=0)) == INV
    assert run(_desc(score_mod=fa.FL_MOD_ALIBI)) == UNS
    assert run(_desc(cu_q=None)) == INV
    assert run(_desc(kv_lens=0x2002)) == ALI
    assert run(_desc(block_table_stride=2)) == INV
    assert run(_desc(block_table=None)) == INV  # a contiguous cache is [batch, ...]
    assert run(_desc(), qq=_t((7, 8, 128))) == INV
    assert run(_desc(), qq=_t((7, 7, 64)), o=_t((7, 7, 64))) == INV
    assert run(_desc(), o=_t((7, 8, 64), fa.FL_F32)) == INV
    assert run(_desc(), lse=_t((7, 8), fa.FL_F32)) == INV
    assert run(_desc(), ws=None) == INV
    assert run(_desc(), ws=0x100010) == ALI
    assert run(_desc(), n=100) == INV
    wide = (_cache(D=32), _cache(D=32), c[2], c[3])
    assert run(_desc(), qq=_t((7, 8, 32)), o=_t((7, 8, 32)), cc=wide) == UNS
    # each cache type has its own call
    plain = _t((5, 32, 2, 64))
    assert run(_desc(), cc=(plain, plain, c[2], c[3])) == INV
    assert lib.fl_attn_chunk(q, c[0], c[1], q, None, _desc(), 0x100000, 1 << 40, None) == INV


def test_workspace_sizes(lib):
    import ctypes
    n8, n16 = ctypes.c_size_t(), ctypes.c_size_t()
    q = _t((7, 8, 64))
    assert lib.fl_attn_chunk_fp8_workspace_size(q, _cache(), ctypes.byref(_desc()), ctypes.byref(n8)) == fa.FL_OK
    assert lib.fl_attn_chunk_workspace_size(q, _t((5, 32, 2, 64)), ctypes.byref(_desc()), ctypes.byref(n16)) == fa.FL_OK
    assert n8.value >= n16.value
    assert lib.fl_attn_chunk_fp8_workspace_size(q, _t((5, 32, 2, 64)), ctypes.byref(_desc()), ctypes.byref(n8)) == INV
    assert lib.fl_attn_chunk_fp8_workspace_size(q, _cache(), ctypes.byref(_desc()), None) == INV
