"""Python binding of the GB300 fused attention-variant forward (include/fl_attn.h).

Argument marshalling only: every step of the computation runs in the CUDA
library ``_build/libflattn.so``.  There is no CPU fallback -- if the library
is missing, importing the binding's entry points raises.

The names mirror the C ABI: :func:`fl_attn_fwd`, :func:`fl_attn_tile_shape`,
:func:`fl_attn_status_string`, :func:`fl_attn_last_error`,
:func:`fl_attn_version`, :func:`fl_attn_decode_workspace_size`,
:func:`fl_attn_decode`, :func:`fl_attn_decode_static`, :func:`fl_attn_bwd`,
:func:`fl_attn_diff_bwd`, and for rotary positions and serving steps
:func:`fl_rope`, :func:`fl_kv_plan`, :func:`fl_kv_append`, :func:`fl_attn_chunk`, and for a
cache in 8 bits :func:`fl_kv_append_fp8`, :func:`fl_kv_read_fp8`, :func:`fl_attn_chunk_fp8`.
Tensors are torch tensors on the current CUDA device
(PyTorch provides device memory and streams; nothing else).
"""
from __future__ import annotations

import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libflattn.so")

# fl_status
FL_OK = 0
FL_ERR_INVALID_ARG = 1
FL_ERR_UNSUPPORTED = 2
FL_ERR_ALIGNMENT = 3
FL_ERR_CUDA = 4
FL_ERR_DEVICE_TIMEOUT = 5
FL_ERR_NO_DEVICE = 6
# fl_dtype
FL_BF16 = 0
FL_F32 = 1
FL_E4M3 = 2
# fl_kind
FL_KIND_STANDARD = 0
FL_KIND_DIFF = 1
FL_KIND_EVO_ROW = 2
FL_KIND_EVO_COL = 3
# fl_score_mod
FL_MOD_NONE = 0
FL_MOD_ALIBI = 1
FL_MOD_SOFTCAP = 2
FL_MOD_EXPR = 3
# fl_mask
FL_MASK_NONE = 0
FL_MASK_CAUSAL = 1
FL_MASK_WINDOW = 2
FL_MASK_PREFIX = 3
FL_MASK_DOC = 4
# fl_inject
FL_INJECT_NONE = 0
FL_INJECT_DROP_KV_LOAD = 1
FL_DEVERR_TIMEOUT = 0x1
FL_DEVERR_PAGES = 0x2
FL_DEVERR_LENGTHS = 0x4
# fl_rope_layout
FL_ROPE_HALF = 0
FL_ROPE_INTERLEAVED = 1
# fl_rope_scaling
FL_ROPE_SCALE_NONE = 0
FL_ROPE_SCALE_LINEAR = 1
FL_ROPE_SCALE_BASE = 2
FL_ROPE_SCALE_BANDS = 3
FL_ROPE_SCALE_RAMP = 4
FL_ROPE_MAX_PAIRS = 128

MODS = {"none": FL_MOD_NONE, "vanilla": FL_MOD_NONE, "alibi": FL_MOD_ALIBI,
        "softcap": FL_MOD_SOFTCAP, "expr": FL_MOD_EXPR}
MASKS = {"none": FL_MASK_NONE, "causal": FL_MASK_CAUSAL, "window": FL_MASK_WINDOW,
         "prefix": FL_MASK_PREFIX, "doc": FL_MASK_DOC}
KINDS = {"standard": FL_KIND_STANDARD, "diff": FL_KIND_DIFF, "evo_row": FL_KIND_EVO_ROW,
         "evo_col": FL_KIND_EVO_COL}
ROPE_LAYOUTS = {"half": FL_ROPE_HALF, "interleaved": FL_ROPE_INTERLEAVED}
ROPE_SCALINGS = {"none": FL_ROPE_SCALE_NONE, "linear": FL_ROPE_SCALE_LINEAR, "base": FL_ROPE_SCALE_BASE,
                 "bands": FL_ROPE_SCALE_BANDS, "ramp": FL_ROPE_SCALE_RAMP}


class FlTensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("sizes", ctypes.c_int64 * 5), ("strides", ctypes.c_int64 * 5)]


class FlDesc(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32), ("score_mod", ctypes.c_int32), ("softcap", ctypes.c_float),
        ("mask", ctypes.c_int32), ("window", ctypes.c_int32), ("prefix", ctypes.c_int32),
        ("doc_offsets", ctypes.c_void_p), ("doc_stride", ctypes.c_int32),
        ("gqa_group", ctypes.c_int32), ("diff_lambda", ctypes.c_float), ("scale", ctypes.c_float),
        ("alibi_slopes", ctypes.c_void_p), ("debug_tile_counts", ctypes.c_void_p),
        ("error_word", ctypes.c_void_p), ("debug_inject", ctypes.c_int32),
        ("wait_timeout_us", ctypes.c_uint32), ("score_mod_expr", ctypes.c_char_p),
    ]


class FlDecodeDesc(ctypes.Structure):
    _fields_ = [
        ("score_mod", ctypes.c_int32), ("softcap", ctypes.c_float), ("causal", ctypes.c_int32),
        ("scale", ctypes.c_float), ("kv_lens", ctypes.c_void_p), ("max_kv_len", ctypes.c_int32),
        ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int32),
        ("error_word", ctypes.c_void_p), ("wait_timeout_us", ctypes.c_uint32),
    ]


class FlRopeConfig(ctypes.Structure):
    _fields_ = [
        ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
        ("base", ctypes.c_double), ("factor", ctypes.c_double), ("context", ctypes.c_double),
        ("low", ctypes.c_double), ("high", ctypes.c_double), ("magnitude", ctypes.c_double),
    ]


class FlRopeTable(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("magnitude", ctypes.c_float),
                ("valid", ctypes.c_uint32), ("turns", ctypes.c_uint64 * FL_ROPE_MAX_PAIRS)]


class FlKvPlanDesc(ctypes.Structure):
    _device = None  # of the tensors whose addresses it holds
    _fields_ = [
        ("batch", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
        ("n_free", ctypes.c_int32), ("block_table_stride", ctypes.c_int32),
        ("q_lens", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("free_pages", ctypes.c_void_p),
        ("free_head", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
        ("kv_lens_out", ctypes.c_void_p), ("cu_q", ctypes.c_void_p), ("positions", ctypes.c_void_p),
        ("slots", ctypes.c_void_p), ("free_head_out", ctypes.c_void_p), ("error_word", ctypes.c_void_p),
    ]


class FlChunkDesc(ctypes.Structure):
    _device = None  # of the tensors whose addresses it holds
    _fields_ = [
        ("score_mod", ctypes.c_int32), ("softcap", ctypes.c_float), ("causal", ctypes.c_int32),
        ("window", ctypes.c_int32), ("scale", ctypes.c_float), ("batch", ctypes.c_int32),
        ("cu_q", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("max_kv_len", ctypes.c_int32),
        ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int32),
        ("error_word", ctypes.c_void_p), ("wait_timeout_us", ctypes.c_uint32),
        ("strict_lengths", ctypes.c_int32),
    ]


class FlAttnError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{fl_attn_status_string(status)} ({detail})")
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH):
    """Load the CUDA library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise FileNotFoundError(
            f"{path} is missing: build it with `python -m attention_variant_gb300.build` "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    lib.fl_attn_fwd.restype = ctypes.c_int
    lib.fl_attn_fwd.argtypes = [P(FlTensor), P(FlTensor), P(FlTensor), P(FlTensor), P(FlTensor),
                                P(FlDesc), P(FlTensor), P(FlTensor), ctypes.c_void_p]
    lib.fl_attn_tile_shape.restype = ctypes.c_int
    lib.fl_attn_tile_shape.argtypes = [P(FlDesc), ctypes.c_int32, P(ctypes.c_int32),
                                       P(ctypes.c_int32)]
    lib.fl_attn_status_string.restype = ctypes.c_char_p
    lib.fl_attn_status_string.argtypes = [ctypes.c_int]
    lib.fl_attn_last_error.restype = ctypes.c_char_p
    lib.fl_attn_last_error.argtypes = []
    lib.fl_attn_version.restype = ctypes.c_int32
    lib.fl_attn_bwd_workspace_size.restype = ctypes.c_int
    lib.fl_attn_bwd_workspace_size.argtypes = [P(FlTensor), P(FlTensor), P(FlDesc),
                                               P(ctypes.c_size_t)]
    lib.fl_attn_bwd.restype = ctypes.c_int
    lib.fl_attn_bwd.argtypes = [P(FlTensor)] * 9 + [P(FlDesc), ctypes.c_void_p, ctypes.c_size_t,
                                                    ctypes.c_void_p]
    lib.fl_attn_diff_bwd_workspace_size.restype = ctypes.c_int
    lib.fl_attn_diff_bwd_workspace_size.argtypes = [P(FlTensor), P(FlTensor), P(FlTensor), P(FlDesc),
                                                    P(ctypes.c_size_t)]
    lib.fl_attn_diff_bwd.restype = ctypes.c_int
    lib.fl_attn_diff_bwd.argtypes = [P(FlTensor)] * 8 + [P(FlDesc), ctypes.c_void_p, ctypes.c_size_t,
                                                         ctypes.c_void_p]
    lib.fl_attn_evoformer.restype = ctypes.c_int
    lib.fl_attn_evoformer.argtypes = [P(FlTensor), P(FlTensor), P(FlTensor), P(FlTensor), P(FlTensor),
                                      P(FlDesc), P(FlTensor), P(FlTensor), P(FlTensor), ctypes.c_void_p]
    lib.fl_attn_score_expr_check.restype = ctypes.c_int
    lib.fl_attn_score_expr_check.argtypes = [ctypes.c_char_p, ctypes.c_int32]
    lib.fl_attn_decode_workspace_size.restype = ctypes.c_int
    lib.fl_attn_decode_workspace_size.argtypes = [P(FlTensor), P(FlTensor), P(FlDecodeDesc),
                                                  P(ctypes.c_size_t)]
    lib.fl_attn_decode_static.restype = ctypes.c_int
    lib.fl_attn_decode_static.argtypes = [P(FlTensor), P(FlTensor), P(FlTensor), P(FlTensor),
                                          P(FlTensor), P(FlDecodeDesc), ctypes.c_void_p]
    lib.fl_attn_decode.restype = ctypes.c_int
    lib.fl_attn_decode.argtypes = [P(FlTensor), P(FlTensor), P(FlTensor), P(FlTensor), P(FlTensor),
                                   P(FlDecodeDesc), ctypes.c_void_p, ctypes.c_size_t,
                                   ctypes.c_void_p]
    # the rotary and serving-step entry points take their tensors (and the
    # rotary desc) as packed bytes: see _pack
    B = ctypes.c_char_p
    lib.fl_rope_make_table.restype = ctypes.c_int
    lib.fl_rope_make_table.argtypes = [P(FlRopeConfig), P(FlRopeTable)]
    lib.fl_rope.restype = ctypes.c_int
    lib.fl_rope.argtypes = [B] * 5 + [ctypes.c_void_p]
    lib.fl_kv_plan.restype = ctypes.c_int
    lib.fl_kv_plan.argtypes = [P(FlKvPlanDesc), ctypes.c_void_p]
    lib.fl_kv_append.restype = ctypes.c_int
    lib.fl_kv_append.argtypes = [B] * 6 + [ctypes.c_void_p, B, ctypes.c_void_p]
    lib.fl_attn_chunk_workspace_size.restype = ctypes.c_int
    lib.fl_attn_chunk_workspace_size.argtypes = [B, B, P(FlChunkDesc), P(ctypes.c_size_t)]
    lib.fl_attn_chunk.restype = ctypes.c_int
    lib.fl_attn_chunk.argtypes = [B] * 5 + [P(FlChunkDesc), ctypes.c_void_p, ctypes.c_size_t,
                                            ctypes.c_void_p]
    lib.fl_kv_append_fp8.restype = ctypes.c_int
    lib.fl_kv_append_fp8.argtypes = [B] * 8 + [ctypes.c_void_p, B, ctypes.c_void_p]
    lib.fl_kv_read_fp8.restype = ctypes.c_int
    lib.fl_kv_read_fp8.argtypes = [B] * 4 + [ctypes.c_void_p, B, B, ctypes.c_void_p]
    lib.fl_attn_chunk_fp8_workspace_size.restype = ctypes.c_int
    lib.fl_attn_chunk_fp8_workspace_size.argtypes = [B, B, P(FlChunkDesc), P(ctypes.c_size_t)]
    lib.fl_attn_chunk_fp8.restype = ctypes.c_int
    lib.fl_attn_chunk_fp8.argtypes = [B] * 7 + [P(FlChunkDesc), ctypes.c_void_p, ctypes.c_size_t,
                                                ctypes.c_void_p]
    _lib = lib
    return lib


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return FL_BF16
    if t.dtype == torch.float32:
        return FL_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def as_fl_tensor(t) -> FlTensor | None:
    """A torch tensor (or None) -> fl_tensor; no copy, no check."""
    if t is None:
        return None
    ft = FlTensor()
    ft.ptr = t.data_ptr()
    ft.dtype = _dtype_code(t)
    ft.ndim = t.dim()
    for d in range(t.dim()):
        ft.sizes[d] = t.shape[d]
        ft.strides[d] = t.stride(d)
    return ft


def make_desc(kind="standard", score_mod="none", softcap=20.0, mask="none", window=0, prefix=0,
              doc_offsets=None, gqa_group=0, diff_lambda=0.0, scale=0.0, alibi_slopes=None,
              debug_tile_counts=None, error_word=None, debug_inject=0,
              wait_timeout_us=0, score_expr=None) -> FlDesc:
    """Build an fl_attn_variant_desc; tensor arguments are device torch tensors.
    ``score_expr`` (a string in the grammar of include/fl_attn.h) selects
    FL_MOD_EXPR."""
    d = FlDesc()
    if score_expr is not None:
        score_mod = "expr"
        d.score_mod_expr = score_expr.encode()
    d.kind = KINDS[kind] if isinstance(kind, str) else int(kind)
    d.score_mod = MODS[score_mod] if isinstance(score_mod, str) else int(score_mod)
    d.softcap = float(softcap)
    d.mask = MASKS[mask] if isinstance(mask, str) else int(mask)
    d.window = int(window)
    d.prefix = int(prefix)
    if doc_offsets is not None:
        d.doc_offsets = doc_offsets.data_ptr()
        d.doc_stride = int(doc_offsets.shape[-1])
    d.gqa_group = int(gqa_group)
    d.diff_lambda = float(diff_lambda)
    d.scale = float(scale)
    d.alibi_slopes = alibi_slopes.data_ptr() if alibi_slopes is not None else None
    d.debug_tile_counts = debug_tile_counts.data_ptr() if debug_tile_counts is not None else None
    d.error_word = error_word.data_ptr() if error_word is not None else None
    d.debug_inject = int(debug_inject)
    d.wait_timeout_us = int(wait_timeout_us)
    return d


def _ref(x):
    return ctypes.byref(x) if x is not None else None


def fl_attn_bwd_workspace_size(q, k, desc: FlDesc) -> int:
    """Bytes of workspace fl_attn_bwd needs for these shapes."""
    lib = load_library()
    n = ctypes.c_size_t()
    st = lib.fl_attn_bwd_workspace_size(_ref(as_fl_tensor(q)), _ref(as_fl_tensor(k)), ctypes.byref(desc),
                                        ctypes.byref(n))
    if st != FL_OK:
        raise FlAttnError(st, fl_attn_last_error())
    return n.value


def fl_attn_bwd(q, k, v, out, lse, dout, dq, dk, dv, desc: FlDesc, workspace, stream=None) -> None:
    """Enqueue the backward (see include/fl_attn.h); workspace is a device torch
    tensor of at least fl_attn_bwd_workspace_size bytes."""
    lib = load_library()
    if stream is None:
        import torch
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    t = [as_fl_tensor(x) for x in (q, k, v, out, lse, dout, dq, dk, dv)]
    st = lib.fl_attn_bwd(*[_ref(x) for x in t], ctypes.byref(desc),
                         ctypes.c_void_p(workspace.data_ptr()),
                         workspace.numel() * workspace.element_size(), ctypes.c_void_p(stream))
    if st != FL_OK:
        raise FlAttnError(st, fl_attn_last_error())


def fl_attn_diff_bwd_workspace_size(q, k, v, desc: FlDesc) -> int:
    """Bytes of workspace fl_attn_diff_bwd needs for these shapes."""
    lib = load_library()
    n = ctypes.c_size_t()
    st = lib.fl_attn_diff_bwd_workspace_size(_ref(as_fl_tensor(q)), _ref(as_fl_tensor(k)), _ref(as_fl_tensor(v)),
                                             ctypes.byref(desc), ctypes.byref(n))
    if st != FL_OK:
        raise FlAttnError(st, fl_attn_last_error())
    return n.value


def fl_attn_diff_bwd(q, k, v, lse, dout, dq, dk, dv, desc: FlDesc, workspace, stream=None) -> None:
    """Enqueue the differential backward (see include/fl_attn.h); workspace is
    a device torch tensor of at least fl_attn_diff_bwd_workspace_size bytes."""
    lib = load_library()
    if stream is None:
        import torch
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    t = [as_fl_tensor(x) for x in (q, k, v, lse, dout, dq, dk, dv)]
    st = lib.fl_attn_diff_bwd(*[_ref(x) for x in t], ctypes.byref(desc),
                              ctypes.c_void_p(workspace.data_ptr()),
                              workspace.numel() * workspace.element_size(), ctypes.c_void_p(stream))
    if st != FL_OK:
        raise FlAttnError(st, fl_attn_last_error())


def fl_attn_evoformer(q, k, v, out, lse, desc: FlDesc, bias=None, gate=None, msa_mask=None,
                      stream=None) -> None:
    """The Evoformer kinds over a batch of MSA stacks (5-D tensors) with an
    optional MSA mask (see include/fl_attn.h); raises FlAttnError."""
    lib = load_library()
    if stream is None:
        import torch
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    t = [as_fl_tensor(x) if x is not None else None for x in (q, k, v, out, lse, bias, gate, msa_mask)]
    st = lib.fl_attn_evoformer(_ref(t[0]), _ref(t[1]), _ref(t[2]), _ref(t[3]), _ref(t[4]),
                               ctypes.byref(desc), _ref(t[5]), _ref(t[6]), _ref(t[7]),
                               ctypes.c_void_p(stream))
    if st != FL_OK:
        raise FlAttnError(st, fl_attn_last_error())


def fl_attn_score_expr_check(expr: str, compile=False) -> None:
    """Check a score_mod expression against the grammar; with ``compile`` true
    also run the runtime compilation of its forward kernel, with
    ``compile="backward"`` also that of its backward kernels (no GPU needed).
    Raises FlAttnError."""
    lib = load_library()
    level = 2 if compile == "backward" else int(bool(compile))
    st = lib.fl_attn_score_expr_check(expr.encode(), level)
    if st != FL_OK:
        raise FlAttnError(st, fl_attn_last_error())


def fl_attn_fwd(q, k, v, out, lse=None, desc: FlDesc | None = None, bias=None, gate=None,
                stream=None) -> None:
    """Enqueue the fused forward on ``stream`` (default: torch's current stream).

    Raises :class:`FlAttnError` on a non-OK status.  See include/fl_attn.h for
    the layouts of each kind.
    """
    lib = load_library()
    if desc is None:
        desc = make_desc()
    if stream is None:
        import torch
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    tensors = [as_fl_tensor(x) for x in (q, k, v, out, lse, bias, gate)]
    st = lib.fl_attn_fwd(_ref(tensors[0]), _ref(tensors[1]), _ref(tensors[2]), _ref(tensors[3]),
                         _ref(tensors[4]), ctypes.byref(desc), _ref(tensors[5]),
                         _ref(tensors[6]), ctypes.c_void_p(stream))
    if st != FL_OK:
        raise FlAttnError(st, fl_attn_last_error())


def fl_attn_tile_shape(desc: FlDesc, head_dim: int) -> tuple[int, int]:
    lib = load_library()
    bm, bn = ctypes.c_int32(), ctypes.c_int32()
    st = lib.fl_attn_tile_shape(ctypes.byref(desc), int(head_dim), ctypes.byref(bm),
                                ctypes.byref(bn))
    if st != FL_OK:
        raise FlAttnError(st, fl_attn_last_error())
    return bm.value, bn.value


def fl_attn_status_string(status: int) -> str:
    return load_library().fl_attn_status_string(int(status)).decode()


def fl_attn_last_error() -> str:
    return load_library().fl_attn_last_error().decode()


def fl_attn_version() -> int:
    return int(load_library().fl_attn_version())


def make_decode_desc(kv_lens, max_kv_len: int, *, score_mod="none", softcap=20.0, causal=True,
                     scale=0.0, block_table=None, error_word=None,
                     wait_timeout_us=0) -> FlDecodeDesc:
    """Build an fl_decode_desc; kv_lens and block_table are device int32 torch tensors."""
    d = FlDecodeDesc()
    d.score_mod = MODS[score_mod] if isinstance(score_mod, str) else int(score_mod)
    d.softcap = float(softcap)
    d.causal = 1 if causal else 0
    d.scale = float(scale)
    d.kv_lens = kv_lens.data_ptr()
    d.max_kv_len = int(max_kv_len)
    if block_table is not None:
        d.block_table = block_table.data_ptr()
        d.block_table_stride = int(block_table.stride(0))
    d.error_word = error_word.data_ptr() if error_word is not None else None
    d.wait_timeout_us = int(wait_timeout_us)
    d._keep = (kv_lens, block_table, error_word)
    return d


def fl_attn_decode_workspace_size(q, k_cache, desc: FlDecodeDesc) -> int:
    """Bytes of workspace fl_attn_decode needs for these shapes."""
    lib = load_library()
    n = ctypes.c_size_t()
    st = lib.fl_attn_decode_workspace_size(ctypes.byref(as_fl_tensor(q)),
                                           ctypes.byref(as_fl_tensor(k_cache)), ctypes.byref(desc),
                                           ctypes.byref(n))
    if st != FL_OK:
        raise FlAttnError(st, fl_attn_last_error())
    return n.value


def fl_attn_decode(q, k_cache, v_cache, out, lse, desc: FlDecodeDesc, workspace, stream=None) -> None:
    """Enqueue attention against a KV cache (see include/fl_attn.h); workspace is a
    device torch tensor of at least fl_attn_decode_workspace_size bytes."""
    lib = load_library()
    if stream is None:
        import torch
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    tensors = [as_fl_tensor(x) for x in (q, k_cache, v_cache, out, lse)]
    nbytes = workspace.numel() * workspace.element_size()
    st = lib.fl_attn_decode(_ref(tensors[0]), _ref(tensors[1]), _ref(tensors[2]), _ref(tensors[3]),
                            _ref(tensors[4]), ctypes.byref(desc), ctypes.c_void_p(workspace.data_ptr()),
                            nbytes, ctypes.c_void_p(stream))
    if st != FL_OK:
        raise FlAttnError(st, fl_attn_last_error())


def fl_attn_decode_static(q, k_cache, v_cache, out, lse, desc: FlDecodeDesc, stream=None) -> None:
    """fl_attn_decode with the library's own static scratch instead of a
    workspace: for callers that cannot allocate device memory.  Allocates
    nothing; calls that overlap on the GPU race (they share the scratch); the
    first call in a CUDA context (per device, and again after a device reset)
    sets up the scratch address, so make it before any stream capture."""
    lib = load_library()
    if stream is None:
        import torch
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    tensors = [as_fl_tensor(x) for x in (q, k_cache, v_cache, out, lse)]
    st = lib.fl_attn_decode_static(_ref(tensors[0]), _ref(tensors[1]), _ref(tensors[2]),
                                   _ref(tensors[3]), _ref(tensors[4]), ctypes.byref(desc),
                                   ctypes.c_void_p(stream))
    if st != FL_OK:
        raise FlAttnError(st, fl_attn_last_error())


# ---------------------------------------------------------------------------
# Rotary positions and serving steps.  These calls are a few microseconds of
# GPU work, so their marshalling is kept short: a tensor travels as the packed
# bytes of its fl_tensor (one struct.pack; a ctypes structure filled field by
# field takes three times as long), and what is needed of torch is looked up once.

_PACK = [None] + [struct.Struct(f"<Qii{n}q{8 * (5 - n)}x{n}q{8 * (5 - n)}x").pack for n in range(1, 6)]


class _Torch:
    """What these calls use of torch."""

    def __init__(self):
        import torch
        self.codes = {torch.bfloat16: FL_BF16, torch.float32: FL_F32, torch.float8_e4m3fn: FL_E4M3}
        self.types = {"int32": torch.int32, "int64": torch.int64}
        self.int32, self.int64 = torch.int32, torch.int64
        self.device = torch.cuda.current_device
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.stream = raw or (lambda device: torch.cuda.current_stream(device).cuda_stream)


_torch = None


def _tools() -> _Torch:
    global _torch
    if _torch is None:
        _torch = _Torch()
    return _torch


def _pack(t, device: int):
    """A torch tensor (or None) of CUDA device `device` -> the bytes of its fl_tensor."""
    if t is None:
        return None
    shape = t.shape
    n = len(shape)
    code = _torch.codes.get(t.dtype)
    if code is None or t.get_device() != device or not 1 <= n <= 5:
        if t.get_device() != device:
            raise ValueError(f"tensor on {t.device}: the current device is cuda:{device}")
        if code is None:
            raise TypeError(f"unsupported dtype {t.dtype}")
        raise ValueError(f"tensors have 1 to 5 dimensions, got {n}")
    return _PACK[n](t.data_ptr(), code, n, *shape, *t.stride())


def _device() -> int:
    return _tools().device()


def _stream_of(stream, device: int) -> int:
    if stream is None:
        return _torch.stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(st: int) -> None:
    if st != FL_OK:
        raise FlAttnError(st, fl_attn_last_error())


def _index(t, name: str, shape, dtype="int32", device=None) -> int:
    """The address of a contiguous integer tensor of the given shape (None entries: any size)."""
    if t.dtype is not _tools().types[dtype]:
        raise TypeError(f"{name} must be {dtype}, is {t.dtype}")
    if t.shape != shape and (t.dim() != len(shape) or
                             any(s is not None and s != n for s, n in zip(shape, t.shape))):
        raise ValueError(f"{name} must have shape {tuple(shape)}, has {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} on {t.device}: the current device is cuda:{device}")
    return t.data_ptr()


def _error_word(t, device: int):
    if t is None:
        return None
    if t.get_device() != device:
        raise ValueError(f"error_word on {t.device}: the other tensors are on cuda:{device}")
    if t.numel() < 1 or t.element_size() < 4:
        raise ValueError(f"error_word must hold 32 bits, is {tuple(t.shape)} of {t.dtype}")
    return t.data_ptr()


def _check_device(desc, device: int) -> None:
    if desc._device not in (None, device):
        raise ValueError(f"the desc's tensors are on cuda:{desc._device}: the current device is cuda:{device}")


def make_rope_table(rot_dim: int, *, base=10000.0, layout="half", scaling="none", factor=1.0,
                    context=8192, low=0.0, high=0.0, magnitude=0.0) -> FlRopeTable:
    """The frequencies of a model's rotary positions (see include/fl_attn.h);
    made once per model and passed to :func:`fl_rope` and :func:`fl_kv_append`."""
    c = FlRopeConfig()
    c.rot_dim = int(rot_dim)
    c.layout = ROPE_LAYOUTS[layout] if isinstance(layout, str) else int(layout)
    c.scaling = ROPE_SCALINGS[scaling] if isinstance(scaling, str) else int(scaling)
    c.base, c.factor, c.context = float(base), float(factor), float(context)
    c.low, c.high, c.magnitude = float(low), float(high), float(magnitude)
    table = FlRopeTable()
    _check(load_library().fl_rope_make_table(ctypes.byref(c), ctypes.byref(table)))
    return table


_ROPE_DESC = struct.Struct("<QQqii")


def fl_rope(q, k, q_out, k_out, table: FlRopeTable, positions=None, offset=0, backward=False,
            stream=None) -> None:
    """Enqueue rotary positions of q and (unless None) k into q_out and k_out,
    which may be q and k themselves (see include/fl_attn.h).  Tensors are
    [B, S, H, D] with positions (int32) [B, S] or [S], or [T, H, D] with
    positions [T]; without positions, row s of a sequence is at s + offset.
    ``backward`` maps the gradients of the outputs to those of the inputs."""
    lib = load_library()
    dev = _device()
    at = rows = 0
    if positions is not None:
        shape = q.shape
        if positions.dim() == 2 and len(shape) == 4:
            at, rows = _index(positions, "positions", shape[:2], device=dev), shape[1]
        else:
            at = _index(positions, "positions", shape[-3:-2], device=dev)
    desc = _ROPE_DESC.pack(ctypes.addressof(table), at, rows, int(offset), 1 if backward else 0)
    _check(lib.fl_rope(_pack(q, dev), _pack(k, dev), _pack(q_out, dev), _pack(k_out, dev), desc,
                       _stream_of(stream, dev)))


def make_kv_plan_desc(q_lens, kv_lens, free_pages, free_head, block_table, kv_lens_out, cu_q, positions,
                      slots, free_head_out, *, page_size: int, error_word=None) -> FlKvPlanDesc:
    """Build an fl_kv_plan_desc from contiguous device torch tensors, all int32
    but slots (int64); slots and positions set the number of tokens a step may
    have, slots may be None.  A serving loop keeps it: every step reads and
    writes the same buffers."""
    B = q_lens.shape[0]
    dev = q_lens.get_device()
    d = FlKvPlanDesc()
    d.batch, d.page_size, d.max_tokens = B, int(page_size), positions.shape[0]
    d.q_lens = _index(q_lens, "q_lens", (B,), device=dev)
    d.kv_lens = _index(kv_lens, "kv_lens", (B,), device=dev)
    d.n_free = free_pages.shape[0] if free_pages is not None else 0
    d.free_pages = _index(free_pages, "free_pages", (None,), device=dev) if d.n_free else None
    d.free_head = _index(free_head, "free_head", (1,), device=dev)
    d.block_table = _index(block_table, "block_table", (B, None), device=dev)
    d.block_table_stride = block_table.shape[1]
    d.kv_lens_out = _index(kv_lens_out, "kv_lens_out", (B,), device=dev)
    d.cu_q = _index(cu_q, "cu_q", (B + 1,), device=dev)
    d.positions = _index(positions, "positions", (None,), device=dev)
    d.slots = _index(slots, "slots", positions.shape, "int64", device=dev) if slots is not None else None
    d.free_head_out = _index(free_head_out, "free_head_out", (1,), device=dev)
    d.error_word = _error_word(error_word, dev)
    d._device = dev
    d._keep = (q_lens, kv_lens, free_pages, free_head, block_table, kv_lens_out, cu_q, positions, slots,
               free_head_out, error_word)
    return d


def fl_kv_plan(desc: FlKvPlanDesc, stream=None) -> None:
    """Enqueue a serving step's book-keeping (see include/fl_attn.h)."""
    dev = _device()
    _check_device(desc, dev)
    _check(load_library().fl_kv_plan(ctypes.byref(desc), _stream_of(stream, dev)))


def fl_kv_append(q, k, v, q_out, k_cache, v_cache, slots, *, rope: FlRopeTable | None = None,
                 positions=None, stream=None) -> None:
    """Enqueue the write of new keys and values [T, Hk, D] to their slots
    (int64 [T]) of a paged cache, with the rotary positions of q (into q_out)
    and k where ``rope`` is given (then positions, int32 [T], too); q and q_out
    may both be None (see include/fl_attn.h)."""
    lib = load_library()
    dev = _device()
    desc = None
    if rope is not None:
        if positions is None:
            raise ValueError("rope needs positions")
        desc = _ROPE_DESC.pack(ctypes.addressof(rope), _index(positions, "positions", k.shape[:1], device=dev),
                               0, 0, 0)
    _check(lib.fl_kv_append(_pack(q, dev), _pack(k, dev), _pack(v, dev), _pack(q_out, dev),
                            _pack(k_cache, dev), _pack(v_cache, dev),
                            _index(slots, "slots", k.shape[:1], "int64", device=dev), desc,
                            _stream_of(stream, dev)))


def fl_kv_append_fp8(q, k, v, q_out, k_cache, v_cache, k_scale, v_scale, slots, *, rope: FlRopeTable | None = None,
                     positions=None, stream=None) -> None:
    """:func:`fl_kv_append` into a cache of torch.float8_e4m3fn codes with fp32 scales
    [num_pages, page_size / block, Hk], which grow as they have to (see include/fl_attn.h)."""
    lib = load_library()
    dev = _device()
    desc = None
    if rope is not None:
        if positions is None:
            raise ValueError("rope needs positions")
        desc = _ROPE_DESC.pack(ctypes.addressof(rope), _index(positions, "positions", k.shape[:1], device=dev),
                               0, 0, 0)
    _check(lib.fl_kv_append_fp8(_pack(q, dev), _pack(k, dev), _pack(v, dev), _pack(q_out, dev),
                                _pack(k_cache, dev), _pack(v_cache, dev), _pack(k_scale, dev), _pack(v_scale, dev),
                                _index(slots, "slots", k.shape[:1], "int64", device=dev), desc,
                                _stream_of(stream, dev)))


def fl_kv_read_fp8(k_cache, v_cache, k_scale, v_scale, slots, k_out, v_out, stream=None) -> None:
    """Enqueue the read of the tokens at ``slots`` (int64 [T]) of an 8-bit cache into k_out
    and v_out [T, Hk, D], bf16 or fp32 (see include/fl_attn.h)."""
    lib = load_library()
    dev = _device()
    _check(lib.fl_kv_read_fp8(_pack(k_cache, dev), _pack(v_cache, dev), _pack(k_scale, dev), _pack(v_scale, dev),
                              _index(slots, "slots", k_out.shape[:1], "int64", device=dev), _pack(k_out, dev),
                              _pack(v_out, dev), _stream_of(stream, dev)))


def make_chunk_desc(cu_q, kv_lens, block_table, max_kv_len: int, *, score_mod="none", softcap=20.0,
                    causal=True, window=0, scale=0.0, error_word=None, wait_timeout_us=0,
                    strict_lengths=False) -> FlChunkDesc:
    """Build an fl_chunk_desc; cu_q [B + 1], kv_lens [B] and block_table
    [B, pages] (None: contiguous cache) are contiguous device int32 torch tensors.
    A loop whose lengths may outgrow ``max_kv_len`` sets ``strict_lengths``: without it they
    are cut to it, which moves the request's rows to earlier keys, and error_word says nothing."""
    B = kv_lens.shape[0]
    dev = kv_lens.get_device()
    d = FlChunkDesc()
    d.score_mod = MODS[score_mod] if isinstance(score_mod, str) else int(score_mod)
    d.softcap = float(softcap)
    d.causal = 1 if causal else 0
    d.window = int(window)
    d.scale = float(scale)
    d.batch = B
    d.cu_q = _index(cu_q, "cu_q", (B + 1,), device=dev)
    d.kv_lens = _index(kv_lens, "kv_lens", (B,), device=dev)
    d.max_kv_len = int(max_kv_len)
    if block_table is not None:
        d.block_table = _index(block_table, "block_table", (B, None), device=dev)
        d.block_table_stride = block_table.shape[1]
    d.error_word = _error_word(error_word, dev)
    d.wait_timeout_us = int(wait_timeout_us)
    d.strict_lengths = 1 if strict_lengths else 0
    d._device = dev
    d._keep = (cu_q, kv_lens, block_table, error_word)
    return d


def fl_attn_chunk_workspace_size(q, k_cache, desc: FlChunkDesc) -> int:
    """Bytes of workspace fl_attn_chunk needs for these shapes."""
    dev = _device()
    n = ctypes.c_size_t()
    _check(load_library().fl_attn_chunk_workspace_size(_pack(q, dev), _pack(k_cache, dev),
                                                       ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def fl_attn_chunk(q, k_cache, v_cache, out, lse, desc: FlChunkDesc, workspace, stream=None) -> None:
    """Enqueue attention of ragged chunks of new tokens over the cache that
    holds them (see include/fl_attn.h); q and out are [T, Hq, D], lse [Hq, T]
    or None, workspace a contiguous device torch tensor of at least
    fl_attn_chunk_workspace_size bytes."""
    lib = load_library()
    dev = _device()
    _check_device(desc, dev)
    if workspace.get_device() != dev:
        raise ValueError(f"workspace on {workspace.device}: the current device is cuda:{dev}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _check(lib.fl_attn_chunk(_pack(q, dev), _pack(k_cache, dev), _pack(v_cache, dev), _pack(out, dev),
                             _pack(lse, dev), ctypes.byref(desc), workspace.data_ptr(),
                             workspace.numel() * workspace.element_size(), _stream_of(stream, dev)))


def fl_attn_chunk_fp8_workspace_size(q, k_cache, desc: FlChunkDesc) -> int:
    """Bytes of workspace fl_attn_chunk_fp8 needs for these shapes."""
    dev = _device()
    n = ctypes.c_size_t()
    _check(load_library().fl_attn_chunk_fp8_workspace_size(_pack(q, dev), _pack(k_cache, dev),
                                                           ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def fl_attn_chunk_fp8(q, k_cache, v_cache, k_scale, v_scale, out, lse, desc: FlChunkDesc, workspace,
                      stream=None) -> None:
    """:func:`fl_attn_chunk` over a cache in 8 bits (torch.float8_e4m3fn, fp32 scales); the
    workspace holds at least fl_attn_chunk_fp8_workspace_size bytes (see include/fl_attn.h)."""
    lib = load_library()
    dev = _device()
    _check_device(desc, dev)
    if workspace.get_device() != dev:
        raise ValueError(f"workspace on {workspace.device}: the current device is cuda:{dev}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _check(lib.fl_attn_chunk_fp8(_pack(q, dev), _pack(k_cache, dev), _pack(v_cache, dev), _pack(k_scale, dev),
                                 _pack(v_scale, dev), _pack(out, dev), _pack(lse, dev), ctypes.byref(desc),
                                 workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                 _stream_of(stream, dev)))
