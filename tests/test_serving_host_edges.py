"""Refusals of the rotary and serving-step entry points at the limits of their
arguments (no GPU: every refusal comes before any CUDA call)."""
from __future__ import annotations

import ctypes
import math
import os
import subprocess

import pytest

import attention_variant_gb300 as fa
from attention_variant_gb300 import build as fbuild

torch = pytest.importorskip("torch")
from tests.test_serving_host import _chunk_desc, _plan_desc, _t, fake_addresses  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fa.load_library()


def _chunk(lib, **kw):
    q, c = _t((9, 8, 64)), _t((20, 16, 2, 64))
    return lib.fl_attn_chunk(q, c, c, q, None, ctypes.byref(_chunk_desc(**kw)), 0x100000, 1 << 40, None)


@fake_addresses
def test_chunk_caches_that_an_int_cannot_count(lib):
    # the end of the tile that holds the last key has to be an int
    for n in (2 ** 31 - 1, 2 ** 31 - 255):
        assert _chunk(lib, max_kv_len=n, block_table_stride=2 ** 31 - 1) == fa.FL_ERR_UNSUPPORTED
    # (taken up to the look for a GPU)
    assert _chunk(lib, max_kv_len=2 ** 31 - 256, block_table_stride=2 ** 31 - 1) == fa.FL_ERR_NO_DEVICE


def test_chunk_desc_is_laid_out_as_in_c(lib, tmp_path):
    src = tmp_path / "size.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "fl_attn.h"\n'
                   'int main(void) { printf("%zu %zu %zu", sizeof(fl_chunk_desc), '
                   'offsetof(fl_chunk_desc, wait_timeout_us), offsetof(fl_chunk_desc, strict_lengths)); return 0; }\n')
    root = os.path.dirname(os.path.dirname(os.path.abspath(fa.__file__)))
    exe = str(tmp_path / "size")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", exe], check=True)
    got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    d = fa.FlChunkDesc
    assert got.split() == [str(n) for n in (ctypes.sizeof(d), d.wait_timeout_us.offset, d.strict_lengths.offset)]


@pytest.mark.parametrize("factor", [1.0, 0.5, 1e-3, 1e-6])
def test_ramp_does_not_shrink_contexts_that_it_does_not_stretch(lib, factor):
    # the default magnitude is 0.1 ln(factor) + 1 above 1, and 1 up to it
    assert fa.make_rope_table(64, scaling="ramp", factor=factor).magnitude == 1.0
    assert fa.make_rope_table(64, scaling="ramp", factor=factor, magnitude=1.25).magnitude == 1.25
    up = fa.make_rope_table(64, scaling="ramp", factor=1.0 / factor).magnitude
    assert up == pytest.approx(1.0 + 0.1 * math.log(1.0 / factor), rel=2.0 ** -24)


@fake_addresses
def test_chunk_softcaps_without_digits_left(lib):
    mod = dict(score_mod=fa.FL_MOD_SOFTCAP)
    for cap in (16385.0, 1e6, 1e30):  # rounding of cap tanh(z / cap) alone: 2^-8 and more of a weight
        assert _chunk(lib, softcap=cap, **mod) == fa.FL_ERR_UNSUPPORTED
    for kw in (dict(softcap=1e-40), dict(softcap=1e-3, scale=3e37)):  # 2 scale / cap is no float
        assert _chunk(lib, **kw, **mod) == fa.FL_ERR_INVALID_ARG
    for cap in (16384.0, 20.0, 1e-30):
        assert _chunk(lib, softcap=cap, **mod) == fa.FL_ERR_NO_DEVICE
    assert _chunk(lib, softcap=1e30) == fa.FL_ERR_NO_DEVICE  # not used


@fake_addresses
def test_error_words_are_aligned(lib):
    # the kernels OR into it: an odd address would be a fault
    for at in (0xB001, 0xB002, 0xB003):
        assert lib.fl_kv_plan(ctypes.byref(_plan_desc(error_word=at)), None) == fa.FL_ERR_ALIGNMENT
        assert _chunk(lib, error_word=at) == fa.FL_ERR_ALIGNMENT
    assert lib.fl_kv_plan(ctypes.byref(_plan_desc(error_word=0xB004)), None) == fa.FL_ERR_NO_DEVICE
    assert _chunk(lib, error_word=0xB004) == fa.FL_ERR_NO_DEVICE


def test_error_words_hold_32_bits(lib):
    # (tensors of no GPU: the descs are built, not used)
    cu, kv, table = (torch.zeros(s, dtype=torch.int32) for s in (2, 1, (1, 4)))
    for word in (torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.int16), torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(ValueError, match="error_word"):
            fa.make_chunk_desc(cu, kv, table, 20, error_word=word)
    for word in (torch.zeros(1, dtype=torch.int32), torch.zeros((), dtype=torch.int32), torch.zeros(2, dtype=torch.int64)):
        assert fa.make_chunk_desc(cu, kv, table, 20, error_word=word).error_word == word.data_ptr()


@fake_addresses
def test_plan_lists_that_an_int_cannot_count(lib):
    # the threads' token numbers run to the end of the last block of 1024
    for n in (2 ** 31 - 1, 2 ** 31 - 1023):
        assert lib.fl_kv_plan(ctypes.byref(_plan_desc(max_tokens=n)), None) == fa.FL_ERR_UNSUPPORTED
    assert lib.fl_kv_plan(ctypes.byref(_plan_desc(max_tokens=2 ** 31 - 1024)), None) == fa.FL_ERR_NO_DEVICE
