"""Python binding of libqll.so, the MI355X (gfx950) scaled_mm library.

The functions here carry the same names as the C entry points declared in
``include/qll.h`` and only marshal arguments: they take torch tensors that
already live on the GPU, allocate outputs (and the Split-K workspace) when the
caller does not pass them, and hand raw device pointers plus the current HIP
stream to the library.  Every step of the computation runs in the library's
HIP kernels; there is no fallback of any kind -- a missing ``libqll.so``
raises.

Operations (see include/qll.h for the full contract):
  quantize_per_token_fp8, quantize_weight_block_fp8,
  gemm_w8a8_int8, gemm_fp8_scaled, gemm_block_fp8, gemm_bf16_batch_invariant,
  linear_fp8_dynamic (per-token quantization + FP8 GEMM in one call),
  gemm_fp8_grouped (per-expert FP8 GEMM over rows sorted by expert),
  quantize_mxfp4, gemm_mxfp4 (MXFP4: E2M1 codes packed two per byte, one
  E8M0 scale byte per 32 elements of a row; tensors as uint8),
  quantize_int4_weights, gemm_w4a16 (INT4 weight-only: int4 codes packed two
  per byte, an fp32 scale per 128-element group, bf16 activations),
  gemm_bf16_epilogue, gemm_fp8_epilogue (bias, activation and residual in the
  epilogue) and gemm_bf16_epilogue_backward,
  gated_bf16, gated_fp8 (act(x Bg^T) * (x Bu^T)) and gated_bf16_backward,
  residual_norm, residual_norm_backward (post-norm, gate, residual stream and
  pre-norm in one pass).
"""
from __future__ import annotations

import ctypes
import json
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqll.so")
TABLE_DIR = os.path.join(HERE, "tables")

QLL_OK = 0
STATUS = {0: "QLL_OK", 1: "QLL_ERR_INVALID_ARG", 2: "QLL_ERR_UNSUPPORTED",
          3: "QLL_ERR_MISALIGNED", 4: "QLL_ERR_WORKSPACE", 5: "QLL_ERR_NO_DEVICE",
          6: "QLL_ERR_TABLE", 7: "QLL_ERR_HIP"}
OUT = {"bf16": 0, "fp32": 1, "int32": 2}
OPS = {"int8": 0, "fp8": 1, "block_fp8": 2, "bf16_bi": 3, "mxfp4": 4, "w4a16": 5,
       "fp8_dynamic": 6}
ACT = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "sigmoid": 5}


class QllError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {STATUS.get(status, status)}")
        self.status = status


class qll_cfg(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("splits", ctypes.c_int32)]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_GEMM_ARGS = [_P, _P, _P, _P, _P, ctypes.c_int, _I64, _I64, _I64, _P,
              ctypes.c_size_t, _P]
_BF16_ARGS = [_P, _P, _P, ctypes.c_int, _I64, _I64, _I64, _P, ctypes.c_size_t, _P]

_lib = None
_table_state = None


def load_library():
    """Load libqll.so (raises when it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is not built; run `python -m "
            "quantized_linear_layer_scaled_amd.build` (needs hipcc)")
    L = ctypes.CDLL(LIB_PATH)
    L.quantize_per_token_fp8.argtypes = [_P, _P, _P, _I64, _I64, _I64, _P]
    L.quantize_weight_block_fp8.argtypes = [_P, _P, _P, _I64, _I64, _P]
    for name in ("gemm_w8a8_int8", "gemm_fp8_scaled", "gemm_block_fp8"):
        getattr(L, name).argtypes = _GEMM_ARGS
        getattr(L, name + "_ex").argtypes = _GEMM_ARGS + [ctypes.POINTER(qll_cfg)]
    L.quantize_mxfp4.argtypes = [_P, _P, _P, _I64, _I64, _P]
    L.quantize_int4_weights.argtypes = [_P, _P, _P, _I64, _I64, _P]
    L.gemm_w4a16.argtypes = _BF16_ARGS[:2] + [_P] + _BF16_ARGS[2:]
    L.gemm_w4a16_ex.argtypes = _BF16_ARGS[:2] + [_P] + _BF16_ARGS[2:] + [ctypes.POINTER(qll_cfg)]
    L.gemm_mxfp4.argtypes = _GEMM_ARGS
    L.gemm_mxfp4_ex.argtypes = _GEMM_ARGS + [ctypes.POINTER(qll_cfg)]
    L.gemm_bf16_batch_invariant.argtypes = _BF16_ARGS
    L.gemm_bf16_batch_invariant_ex.argtypes = _BF16_ARGS + [ctypes.POINTER(qll_cfg)]
    _LIN = [_P, _P, _P, _P, _P, _P, ctypes.c_int, _I64, _I64, _I64, _P, ctypes.c_size_t, _P]
    L.linear_fp8_dynamic.argtypes = _LIN
    L.linear_fp8_dynamic_ex.argtypes = _LIN + [ctypes.POINTER(qll_cfg)]
    _GRP = [_P, _P, _P, _P, _P, _P, ctypes.c_int, _I64, _I64, _I64, _I64, _P]
    L.gemm_fp8_grouped.argtypes = _GRP
    L.gemm_fp8_grouped_ex.argtypes = _GRP + [ctypes.c_char_p]
    L.qll_grouped_select.argtypes = [_I64, _I64, ctypes.c_char_p, ctypes.c_size_t]
    L.qll_init.argtypes = [ctypes.c_char_p]
    L.qll_table_validate.argtypes = [ctypes.c_char_p, ctypes.c_char_p, ctypes.c_int,
                                     ctypes.c_int, ctypes.c_char_p, ctypes.c_char_p,
                                     ctypes.c_size_t]
    L.qll_device_signature.argtypes = [ctypes.c_char_p, ctypes.c_size_t]
    _I, _Z, _F = ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    _MNK = [_I64, _I64, _I64]
    L.gemm_bf16_epilogue.argtypes = [_P] * 4 + [_I, _P, _I] + _MNK + [_P, _Z, _P]
    L.gemm_fp8_epilogue.argtypes = [_P] * 6 + [_I, _P, _I] + _MNK + [_P, _Z, _P]
    L.gemm_bf16_epilogue_backward.argtypes = [_P] * 4 + [_I] + [_P] * 3 + _MNK + [_P, _Z, _P]
    L.gated_bf16.argtypes = [_P] * 3 + [_I, _P, _I] + _MNK + [_P]
    L.gated_fp8.argtypes = [_P] * 6 + [_I, _P, _I] + _MNK + [_P]
    L.gated_bf16_backward.argtypes = [_P] * 4 + [_I] + [_P] * 3 + _MNK + [_P, _Z, _P]
    L.residual_norm.argtypes = [_P, _P, _I] + [_P] * 3 + [_F] * 3 + [_P] * 3 + [_I64, _I64, _P]
    L.residual_norm_backward.argtypes = ([_P, _P, _I] + [_P] * 3 + [_F] * 3 + [_P] * 7 +
                                         [_I64, _I64, _P, _Z, _P])
    L.qll_epilogue_workspace_bytes.argtypes = [_I] + _MNK
    L.qll_epilogue_backward_workspace_bytes.argtypes = [_I, _I] + _MNK
    L.qll_gated_backward_workspace_bytes.argtypes = _MNK
    L.qll_residual_norm_backward_workspace_bytes.argtypes = [_I64, _I64]
    for name in ("epilogue", "epilogue_backward", "gated_backward", "residual_norm_backward"):
        getattr(L, f"qll_{name}_workspace_bytes").restype = _I64
    L.gemm_fp8_scaled_noalloc.argtypes = _GEMM_ARGS[:9] + [_P]
    L.qll_select.argtypes = [ctypes.c_int, _I64, _I64, _I64, ctypes.POINTER(qll_cfg)]
    L.qll_workspace_bytes.argtypes = [ctypes.c_int, _I64, _I64, _I64,
                                      ctypes.POINTER(qll_cfg)]
    L.qll_workspace_bytes.restype = _I64
    L.qll_effective_splits.argtypes = [ctypes.c_int, _I64, ctypes.c_int32]
    L.qll_num_variants.argtypes = [ctypes.c_int]
    L.qll_variant_info.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_char_p,
                                   ctypes.c_size_t]
    L.qll_variant_index.argtypes = [ctypes.c_int, ctypes.c_char_p]
    L.qll_table_entries.argtypes = []
    L.qll_status_str.argtypes = [ctypes.c_int]
    L.qll_status_str.restype = ctypes.c_char_p
    _lib = L
    return L


def _check(fn: str, rc: int):
    if rc != QLL_OK:
        raise QllError(fn, rc)


def default_table() -> str | None:
    """The packaged dispatch table for gfx950 (None if absent)."""
    p = os.path.join(TABLE_DIR, "gfx950.tsv")
    return p if os.path.exists(p) else None


def init(table: str | None = "default") -> int:
    """qll_init: load a dispatch table ("default" = $QLL_TABLE or the packaged
    table, None = heuristic only).  Returns the status (QLL_ERR_TABLE means
    the heuristic stays in force)."""
    global _table_state
    L = load_library()
    if table == "default":
        table = os.environ.get("QLL_TABLE") or default_table()
    rc = L.qll_init(table.encode() if table else None)
    _table_state = (table, rc)
    return rc


def _ensure_init():
    if _table_state is None:
        init()


# --------------------------------------------------------------------------
# marshalling helpers (plumbing only)
# --------------------------------------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dev_ptr(t, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _on(stream):
    """Context in which the binding allocates what it hands to the library:
    the stream the kernels are enqueued on, so that torch's caching allocator
    never gives a temporary (the Split-K workspace) to other work before
    those kernels have used it."""
    import contextlib
    torch = _torch()
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _cfg(op: int, cfg):
    """cfg: None, a qll_cfg, or (variant name or index, splits)."""
    if cfg is None or isinstance(cfg, qll_cfg):
        return cfg
    v, s = cfg
    if isinstance(v, str):
        idx = load_library().qll_variant_index(op, v.encode())
        if idx < 0:
            raise ValueError(f"unknown variant {v!r}")
        v = idx
    return qll_cfg(int(v), int(s))


def _workspace(op, M, N, K, cfg, workspace):
    torch = _torch()
    L = load_library()
    need = L.qll_workspace_bytes(op, M, N, K, ctypes.byref(cfg) if cfg else None)
    if need < 0:
        raise QllError("qll_workspace_bytes", -need)
    if need == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
    nbytes = workspace.numel() * workspace.element_size()
    return workspace, nbytes


def _out(out, M, N, out_dtype, device):
    torch = _torch()
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32, "int32": torch.int32}[out_dtype]
    if out is None:
        out = torch.empty((M, N), dtype=dt, device=device)
    elif out.dtype != dt or tuple(out.shape) != (M, N):
        raise ValueError(f"out must be {dt} of shape {(M, N)}")
    return out


def _bytes8(t, name):
    """fp8 / int8 tensors are passed as bytes."""
    torch = _torch()
    if t.dtype not in (torch.float8_e4m3fn, torch.uint8, torch.int8):
        raise TypeError(f"{name} must be float8_e4m3fn, uint8 or int8")
    return _dev_ptr(t, name)


def _f32(t, name, shape):
    """fp32 scales of the given shape; a vector of length L may also come as
    [L][1] (what the per-token quantizer returns)."""
    torch = _torch()
    ok = t.dtype == torch.float32 and (
        tuple(t.shape) == tuple(shape) or
        (len(shape) == 1 and tuple(t.shape) == (shape[0], 1)))
    if not ok:
        raise ValueError(f"{name} must be float32 of shape {tuple(shape)}")
    return _dev_ptr(t, name)


# --------------------------------------------------------------------------
# quantizers
# --------------------------------------------------------------------------

def quantize_per_token_fp8(x, group: int | None = None, q=None, scales=None,
                           stream=None):
    """bf16 [M][K] -> (e4m3 [M][K], fp32 scales [M][K/group]); group None =
    per token, 128 = per 1x128 group."""
    torch = _torch()
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    M, K = x.shape
    G = K if group in (None, 0, K) else int(group)
    with _on(stream):
        if q is None:
            q = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=x.device)
        if scales is None:
            scales = torch.empty((M, K // G if G else 0), dtype=torch.float32,
                                 device=x.device)
    if tuple(q.shape) != (M, K) or tuple(scales.shape) != (M, K // G):
        raise ValueError("q / scales have the wrong shape")
    rc = load_library().quantize_per_token_fp8(
        _dev_ptr(x, "x"), _bytes8(q, "q"), _dev_ptr(scales, "scales"), M, K,
        0 if G == K else G, _stream(stream))
    _check("quantize_per_token_fp8", rc)
    return q, scales


def quantize_weight_block_fp8(w, q=None, scales=None, stream=None):
    """bf16 [N][K] -> (e4m3 [N][K], fp32 scales [ceil(N/128)][K/128])."""
    torch = _torch()
    if w.dtype != torch.bfloat16 or w.dim() != 2:
        raise ValueError("w must be a 2-D bfloat16 tensor")
    N, K = w.shape
    with _on(stream):
        if q is None:
            q = torch.empty((N, K), dtype=torch.float8_e4m3fn, device=w.device)
        if scales is None:
            scales = torch.empty(((N + 127) // 128, K // 128), dtype=torch.float32,
                                 device=w.device)
    rc = load_library().quantize_weight_block_fp8(
        _dev_ptr(w, "w"), _bytes8(q, "q"), _dev_ptr(scales, "scales"), N, K,
        _stream(stream))
    _check("quantize_weight_block_fp8", rc)
    return q, scales


# --------------------------------------------------------------------------
# GEMMs
# --------------------------------------------------------------------------

def _scaled_gemm(fn, op, A, B, sa, sb, sa_shape, sb_shape, out_dtype, out, cfg,
                 workspace, stream):
    _ensure_init()
    M, K = A.shape
    N, K2 = B.shape
    if K2 != K:
        raise ValueError(f"A is [M][{K}] but B is [N][{K2}]")
    pa, pb = _bytes8(A, "A"), _bytes8(B, "B")
    psa, psb = _f32(sa, "sa", sa_shape(M, N, K)), _f32(sb, "sb", sb_shape(M, N, K))
    c = _cfg(op, cfg)
    with _on(stream):
        out = _out(out, M, N, out_dtype, A.device)
        ws, wsb = _workspace(op, M, N, K, c, workspace)
        L = load_library()
        args = [pa, pb, psa, psb, _dev_ptr(out, "out"), OUT[out_dtype], M, N, K,
                ws.data_ptr() if ws is not None else None, wsb, _stream(stream)]
        rc = getattr(L, fn + "_ex")(*args, ctypes.byref(c)) if c else getattr(L, fn)(*args)
    _check(fn, rc)
    return out


def gemm_w8a8_int8(A, B, sa, sb, out_dtype="bf16", out=None, cfg=None,
                   workspace=None, stream=None):
    """int8 A [M][K] x int8 B [N][K] with fp32 sa [M], sb [N]."""
    return _scaled_gemm("gemm_w8a8_int8", 0, A, B, sa, sb,
                        lambda M, N, K: (M,), lambda M, N, K: (N,), out_dtype,
                        out, cfg, workspace, stream)


def gemm_fp8_scaled(A, B, sa, sb, out_dtype="bf16", out=None, cfg=None,
                    workspace=None, stream=None):
    """e4m3 A [M][K] x e4m3 B [N][K] with fp32 sa [M], sb [N]."""
    return _scaled_gemm("gemm_fp8_scaled", 1, A, B, sa, sb,
                        lambda M, N, K: (M,), lambda M, N, K: (N,), out_dtype,
                        out, cfg, workspace, stream)


def gemm_fp8_scaled_noalloc(A, B, sa, sb, out, out_dtype="bf16", stream=None):
    """gemm_fp8_scaled without a workspace (the library's static Split-K
    scratch array; nothing allocated): the caller passes the output too."""
    _ensure_init()
    M, K = A.shape
    N, K2 = B.shape
    if K2 != K:
        raise ValueError(f"A is [M][{K}] but B is [N][{K2}]")
    if out is None:
        raise ValueError("out must be given (this entry point allocates nothing)")
    out = _out(out, M, N, out_dtype, A.device)
    rc = load_library().gemm_fp8_scaled_noalloc(
        _bytes8(A, "A"), _bytes8(B, "B"), _f32(sa, "sa", (M,)), _f32(sb, "sb", (N,)),
        _dev_ptr(out, "out"), OUT[out_dtype], M, N, K, _stream(stream))
    _check("gemm_fp8_scaled_noalloc", rc)
    return out


def gemm_block_fp8(A, B, sa, sb, out_dtype="bf16", out=None, cfg=None,
                   workspace=None, stream=None):
    """e4m3 A [M][K] x e4m3 B [N][K], sa [M][K/128], sb [ceil(N/128)][K/128]."""
    return _scaled_gemm("gemm_block_fp8", 2, A, B, sa, sb,
                        lambda M, N, K: (M, K // 128),
                        lambda M, N, K: ((N + 127) // 128, K // 128), out_dtype,
                        out, cfg, workspace, stream)


def gemm_bf16_batch_invariant(A, B, out_dtype="bf16", out=None, cfg=None,
                              workspace=None, stream=None):
    """bf16 A [M][K] x bf16 B [N][K]; row m independent of M."""
    torch = _torch()
    _ensure_init()
    if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise TypeError("A and B must be bfloat16")
    M, K = A.shape
    N, K2 = B.shape
    if K2 != K:
        raise ValueError(f"A is [M][{K}] but B is [N][{K2}]")
    c = _cfg(3, cfg)
    with _on(stream):
        out = _out(out, M, N, out_dtype, A.device)
        ws, wsb = _workspace(3, M, N, K, c, workspace)
        L = load_library()
        args = [_dev_ptr(A, "A"), _dev_ptr(B, "B"), _dev_ptr(out, "out"),
                OUT[out_dtype], M, N, K, ws.data_ptr() if ws is not None else None,
                wsb, _stream(stream)]
        if c:
            rc = L.gemm_bf16_batch_invariant_ex(*args, ctypes.byref(c))
        else:
            rc = L.gemm_bf16_batch_invariant(*args)
    _check("gemm_bf16_batch_invariant", rc)
    return out


def _u8(t, name, shape):
    torch = _torch()
    if t.dtype != torch.uint8 or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be uint8 of shape {tuple(shape)}")
    return _dev_ptr(t, name)


def quantize_mxfp4(x, q=None, scales=None, stream=None):
    """bf16 [M][K] -> (packed E2M1 codes uint8 [M][K/2], E8M0 scale bytes
    uint8 [M][K/32]); K % 32 == 0."""
    torch = _torch()
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    M, K = x.shape
    if K % 32:
        raise ValueError("K must be a multiple of 32")
    with _on(stream):
        if q is None:
            q = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
        if scales is None:
            scales = torch.empty((M, K // 32), dtype=torch.uint8, device=x.device)
    rc = load_library().quantize_mxfp4(
        _dev_ptr(x, "x"), _u8(q, "q", (M, K // 2)), _u8(scales, "scales", (M, K // 32)),
        M, K, _stream(stream))
    _check("quantize_mxfp4", rc)
    return q, scales


def gemm_mxfp4(A, B, sa, sb, out_dtype="bf16", out=None, cfg=None, workspace=None,
               stream=None):
    """MXFP4 A [M][K/2] x B [N][K/2] (packed codes, uint8) with E8M0 scale
    bytes sa [M][K/32], sb [N][K/32] (uint8)."""
    _ensure_init()
    M, K2 = A.shape
    N, K2b = B.shape
    if K2b != K2:
        raise ValueError(f"A is [M][{K2}] but B is [N][{K2b}] bytes")
    K = 2 * K2
    pa, pb = _u8(A, "A", (M, K2)), _u8(B, "B", (N, K2))
    psa, psb = _u8(sa, "sa", (M, K // 32)), _u8(sb, "sb", (N, K // 32))
    c = _cfg(4, cfg)
    with _on(stream):
        out = _out(out, M, N, out_dtype, A.device)
        ws, wsb = _workspace(4, M, N, K, c, workspace)
        L = load_library()
        args = [pa, pb, psa, psb, _dev_ptr(out, "out"), OUT[out_dtype], M, N, K,
                ws.data_ptr() if ws is not None else None, wsb, _stream(stream)]
        rc = L.gemm_mxfp4_ex(*args, ctypes.byref(c)) if c else L.gemm_mxfp4(*args)
    _check("gemm_mxfp4", rc)
    return out


def quantize_int4_weights(w, q=None, scales=None, stream=None):
    """bf16 weights [N][K] -> (packed int4 codes uint8 [N][K/2], fp32 scales
    [N][K/128]); K % 128 == 0."""
    torch = _torch()
    if w.dtype != torch.bfloat16 or w.dim() != 2:
        raise ValueError("w must be a 2-D bfloat16 tensor")
    N, K = w.shape
    if K % 128:
        raise ValueError("K must be a multiple of 128")
    with _on(stream):
        if q is None:
            q = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
        if scales is None:
            scales = torch.empty((N, K // 128), dtype=torch.float32, device=w.device)
    rc = load_library().quantize_int4_weights(
        _dev_ptr(w, "w"), _u8(q, "q", (N, K // 2)), _f32(scales, "scales", (N, K // 128)),
        N, K, _stream(stream))
    _check("quantize_int4_weights", rc)
    return q, scales


def gemm_w4a16(A, B, scales, out_dtype="bf16", out=None, cfg=None, workspace=None,
               stream=None):
    """bf16 A [M][K] x packed int4 B [N][K/2] (uint8) with fp32 group scales
    [N][K/128]."""
    torch = _torch()
    _ensure_init()
    if A.dtype != torch.bfloat16 or A.dim() != 2:
        raise TypeError("A must be a 2-D bfloat16 tensor")
    M, K = A.shape
    N = B.shape[0]
    pb = _u8(B, "B", (N, K // 2))
    ps = _f32(scales, "scales", (N, K // 128))
    c = _cfg(5, cfg)
    with _on(stream):
        out = _out(out, M, N, out_dtype, A.device)
        ws, wsb = _workspace(5, M, N, K, c, workspace)
        L = load_library()
        args = [_dev_ptr(A, "A"), pb, ps, _dev_ptr(out, "out"), OUT[out_dtype], M, N, K,
                ws.data_ptr() if ws is not None else None, wsb, _stream(stream)]
        rc = L.gemm_w4a16_ex(*args, ctypes.byref(c)) if c else L.gemm_w4a16(*args)
    _check("gemm_w4a16", rc)
    return out


def linear_fp8_dynamic(x, B, sb, out_dtype="bf16", out=None, q=None, sa=None, cfg=None,
                       workspace=None, stream=None):
    """bf16 x [M][K] -> (out [M][N], q e4m3 [M][K], sa fp32 [M][1]): per-token
    quantization of x and the scaled FP8 GEMM with e4m3 B [N][K], sb [N]."""
    torch = _torch()
    _ensure_init()
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    M, K = x.shape
    N, K2 = B.shape
    if K2 != K:
        raise ValueError(f"x is [M][{K}] but B is [N][{K2}]")
    # the quantizer writes M x K codes into q: its shape is checked before
    # anything is enqueued
    if q is not None and tuple(q.shape) != (M, K):
        raise ValueError(f"q must have shape {(M, K)}")
    c = _cfg(6, cfg)  # the FP8 GEMM variants, then the fused ones
    with _on(stream):
        if q is None:
            q = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=x.device)
        if sa is None:
            sa = torch.empty((M, 1), dtype=torch.float32, device=x.device)
        out = _out(out, M, N, out_dtype, x.device)
        ws, wsb = _workspace(6, M, N, K, c, workspace)
        L = load_library()
        args = [_dev_ptr(x, "x"), _bytes8(B, "B"), _f32(sb, "sb", (N,)), _bytes8(q, "q"),
                _f32(sa, "sa", (M,)), _dev_ptr(out, "out"), OUT[out_dtype], M, N, K,
                ws.data_ptr() if ws is not None else None, wsb, _stream(stream)]
        rc = (L.linear_fp8_dynamic_ex(*args, ctypes.byref(c)) if c
              else L.linear_fp8_dynamic(*args))
    _check("linear_fp8_dynamic", rc)
    return out, q, sa


def gemm_fp8_grouped(A, B, sa, sb, offsets, out_dtype="bf16", out=None, variant=None,
                     stream=None):
    """Grouped (per-expert) FP8 GEMM: A e4m3 [M][K] with rows sorted by
    expert, B e4m3 [E][N][K], sa fp32 [M], sb fp32 [E][N], offsets int32
    [E + 1] on the GPU (rows [offsets[e], offsets[e+1]) use expert e)."""
    torch = _torch()
    _ensure_init()
    M, K = A.shape
    E, N, K2 = B.shape
    if K2 != K:
        raise ValueError(f"A is [M][{K}] but B is [E][N][{K2}]")
    if offsets.dtype != torch.int32 or tuple(offsets.shape) != (E + 1,):
        raise ValueError(f"offsets must be int32 of shape ({E + 1},)")
    with _on(stream):
        out = _out(out, M, N, out_dtype, A.device)
    args = [_bytes8(A, "A"), _bytes8(B, "B"), _f32(sa, "sa", (M,)),
            _f32(sb, "sb", (E, N)), _dev_ptr(offsets, "offsets"), _dev_ptr(out, "out"),
            OUT[out_dtype], M, N, K, E, _stream(stream)]
    L = load_library()
    rc = (L.gemm_fp8_grouped_ex(*args, variant.encode()) if variant
          else L.gemm_fp8_grouped(*args))
    _check("gemm_fp8_grouped", rc)
    return out


def grouped_select(M: int, E: int) -> str:
    """The variant gemm_fp8_grouped picks for M rows over E experts."""
    buf = ctypes.create_string_buffer(64)
    _check("qll_grouped_select", load_library().qll_grouped_select(M, E, buf, 64))
    return buf.value.decode()


# --------------------------------------------------------------------------
# feed-forward operators
# --------------------------------------------------------------------------

# These calls take a few microseconds on the device, so the checks here are
# written for speed: one pass per tensor, and no context manager when the call
# runs on the current stream.  A call with `stream` makes it the current one
# and calls itself, so that what it allocates belongs to that stream too.

def _under(stream, fn, *args, **kw):
    torch = _torch()
    here = torch.cuda.current_device()
    if stream.device.index != here:
        raise ValueError(f"stream is on {stream.device}, the current device is cuda:{here}")
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _place():
    """(current device, its current stream's handle)"""
    torch = _torch()
    here = torch.cuda.current_device()
    return here, torch._C._cuda_getCurrentRawStream(here)


def _refuse(t, name, what, here):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if t.get_device() != here:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{here}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be {what}")


def _need(t, name, dtype, shape, here):
    """Pointer of a contiguous tensor of this type and shape on the current
    device."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == here and
                t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, f"{dtype} of shape {tuple(shape)}", here)


def _arg(t, name, dtype, shape, here):
    """The same, None for None."""
    return None if t is None else _need(t, name, dtype, shape, here)


def _codes(t, name, shape, here):
    """Pointer of e4m3 codes: float8_e4m3fn, or their bytes."""
    torch = _torch()
    dt = getattr(t, "dtype", None)
    if dt is not torch.uint8 and dt is not torch.int8:
        dt = torch.float8_e4m3fn
    return _need(t, name, dt, shape, here)


def _scales(t, name, n, here):
    """Pointer of n fp32 scales, [n] or [n][1]."""
    return _need(t, name, _torch().float32,
                 (n, 1) if getattr(t, "ndim", 1) == 2 else (n,), here)


def _matrix(t, name):
    shape = getattr(t, "shape", None)
    if shape is None:
        raise TypeError(f"{name} must be a torch tensor")
    if len(shape) != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    return shape


def _act(act):
    code = ACT.get(act)
    if code is None:
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACT)}")
    return code


def _float_out(out, M, N, out_dtype, like, here):
    """(output, its pointer, its code), allocated if not given."""
    torch = _torch()
    if out_dtype == "bf16":
        dt, code = torch.bfloat16, 0
    elif out_dtype == "fp32":
        dt, code = torch.float32, 1
    else:
        raise ValueError("out_dtype must be 'bf16' or 'fp32'")
    if out is None:
        out = like.new_empty((M, N), dtype=dt)
        return out, out.data_ptr(), code
    return out, _arg(out, "out", dt, (M, N), here), code


def _scratch(query, need, workspace, like, here):
    """(pointer, bytes, tensor to keep) of at least `need` bytes, allocated if
    not given."""
    if need <= 0:
        if need < 0:
            raise QllError(query, -need)
        return None, 0, None
    torch = _torch()
    if workspace is None:
        workspace = like.new_empty(need, dtype=torch.uint8)
    return (_arg(workspace, "workspace", workspace.dtype, workspace.shape, here),
            workspace.numel() * workspace.element_size(), workspace)


def _epilogue(fp8, A, B, sa, sb, bias, residual, act, out_dtype, out, workspace):
    torch = _torch()
    here, st = _place()
    M, K = _matrix(A, "A")
    N = _matrix(B, "B")[0]
    bf = torch.bfloat16
    L = load_library()
    pb, pr = _arg(bias, "bias", bf, (N,), here), _arg(residual, "residual", bf, (M, N), here)
    code = _act(act)
    if fp8:
        lead = (_codes(A, "A", (M, K), here), _codes(B, "B", (N, K), here),
                _scales(sa, "sa", M, here), _scales(sb, "sb", N, here))
        fn, f = "gemm_fp8_epilogue", L.gemm_fp8_epilogue
    else:
        lead = (_need(A, "A", bf, (M, K), here), _need(B, "B", bf, (N, K), here))
        fn, f = "gemm_bf16_epilogue", L.gemm_bf16_epilogue
    out, po, od = _float_out(out, M, N, out_dtype, A, here)
    ws, wsb, keep = _scratch("qll_epilogue_workspace_bytes",
                             L.qll_epilogue_workspace_bytes(fp8, M, N, K), workspace, A, here)
    rc = f(*lead, pb, pr, code, po, od, M, N, K, ws, wsb, st)
    if rc:
        raise QllError(fn, rc)
    return out


def gemm_bf16_epilogue(A, B, bias=None, residual=None, act="none", out_dtype="bf16", out=None,
                       workspace=None, stream=None):
    """act(A B^T + bias) + residual: bf16 A [M][K], B [N][K], bias [N],
    residual [M][N]."""
    if stream is not None:
        return _under(stream, gemm_bf16_epilogue, A, B, bias, residual, act, out_dtype, out,
                      workspace)
    return _epilogue(0, A, B, None, None, bias, residual, act, out_dtype, out, workspace)


def gemm_fp8_epilogue(A, B, sa, sb, bias=None, residual=None, act="none", out_dtype="bf16",
                      out=None, workspace=None, stream=None):
    """act((A B^T) sa sb + bias) + residual: e4m3 A [M][K], B [N][K], fp32 sa
    [M], sb [N], bf16 bias [N], residual [M][N]."""
    if stream is not None:
        return _under(stream, gemm_fp8_epilogue, A, B, sa, sb, bias, residual, act, out_dtype, out,
                      workspace)
    return _epilogue(1, A, B, sa, sb, bias, residual, act, out_dtype, out, workspace)


def gemm_bf16_epilogue_backward(A, B, dout, bias=None, act="none", need_input=True,
                                need_weight=True, dA=None, dB=None, dbias=None, workspace=None,
                                stream=None):
    """(dA, dB, dbias) of gemm_bf16_epilogue for bf16 dout [M][N] (the
    residual's gradient is dout itself): dA bf16 [M][K], dB bf16 [N][K], dbias
    fp32 [N]; None for what is not needed (dbias without a bias)."""
    if stream is not None:
        return _under(stream, gemm_bf16_epilogue_backward, A, B, dout, bias, act, need_input,
                      need_weight, dA, dB, dbias, workspace)
    torch = _torch()
    here, st = _place()
    M, K = _matrix(A, "A")
    N = _matrix(B, "B")[0]
    code = _act(act)
    if not (need_input or need_weight or bias is not None):
        raise ValueError("nothing to compute")
    L = load_library()
    bf = torch.bfloat16
    pA, pB = _need(A, "A", bf, (M, K), here), _need(B, "B", bf, (N, K), here)
    pd, pb = _need(dout, "dout", bf, (M, N), here), _arg(bias, "bias", bf, (N,), here)
    dA = (torch.empty_like(A) if dA is None else dA) if need_input else None
    dB = (torch.empty_like(B) if dB is None else dB) if need_weight else None
    if bias is None:
        dbias = None
    elif dbias is None:
        dbias = A.new_empty(N, dtype=torch.float32)
    ws, wsb, keep = _scratch(
        "qll_epilogue_backward_workspace_bytes",
        L.qll_epilogue_backward_workspace_bytes(code, bias is not None, M, N, K), workspace, A, here)
    rc = L.gemm_bf16_epilogue_backward(
        pA, pB, pd, pb, code, _arg(dA, "dA", bf, (M, K), here), _arg(dB, "dB", bf, (N, K), here),
        _arg(dbias, "dbias", torch.float32, (N,), here), M, N, K, ws, wsb, st)
    if rc:
        raise QllError("gemm_bf16_epilogue_backward", rc)
    return dA, dB, dbias


def gated_bf16(A, Bg, Bu, act="silu", out_dtype="bf16", out=None, stream=None):
    """act(A Bg^T) * (A Bu^T): bf16 A [M][K], Bg and Bu [N][K]."""
    if stream is not None:
        return _under(stream, gated_bf16, A, Bg, Bu, act, out_dtype, out)
    here, st = _place()
    M, K = _matrix(A, "A")
    N = _matrix(Bg, "Bg")[0]
    bf = _torch().bfloat16
    pA, pg = _need(A, "A", bf, (M, K), here), _need(Bg, "Bg", bf, (N, K), here)
    pu = _need(Bu, "Bu", bf, (N, K), here)
    code = _act(act)
    out, po, od = _float_out(out, M, N, out_dtype, A, here)
    rc = load_library().gated_bf16(pA, pg, pu, code, po, od, M, N, K, st)
    if rc:
        raise QllError("gated_bf16", rc)
    return out


def gated_fp8(A, Bg, Bu, sa, sg, su, act="silu", out_dtype="bf16", out=None, stream=None):
    """act((A Bg^T) sa sg) * ((A Bu^T) sa su): e4m3 A [M][K], Bg and Bu
    [N][K], fp32 sa [M], sg and su [N]."""
    if stream is not None:
        return _under(stream, gated_fp8, A, Bg, Bu, sa, sg, su, act, out_dtype, out)
    here, st = _place()
    M, K = _matrix(A, "A")
    N = _matrix(Bg, "Bg")[0]
    lead = (_codes(A, "A", (M, K), here), _codes(Bg, "Bg", (N, K), here),
            _codes(Bu, "Bu", (N, K), here), _scales(sa, "sa", M, here),
            _scales(sg, "sg", N, here), _scales(su, "su", N, here), _act(act))
    out, po, od = _float_out(out, M, N, out_dtype, A, here)
    rc = load_library().gated_fp8(*lead, po, od, M, N, K, st)
    if rc:
        raise QllError("gated_fp8", rc)
    return out


def gated_bf16_backward(A, Bg, Bu, dout, act="silu", need_input=True, need_weight=True, dA=None,
                        dBg=None, dBu=None, workspace=None, stream=None):
    """(dA, dBg, dBu) of gated_bf16 for bf16 dout [M][N], all bf16; None for
    what is not needed."""
    if stream is not None:
        return _under(stream, gated_bf16_backward, A, Bg, Bu, dout, act, need_input, need_weight,
                      dA, dBg, dBu, workspace)
    here, st = _place()
    M, K = _matrix(A, "A")
    N = _matrix(Bg, "Bg")[0]
    if not (need_input or need_weight):
        raise ValueError("nothing to compute")
    L = load_library()
    torch = _torch()
    bf = torch.bfloat16
    lead = (_need(A, "A", bf, (M, K), here), _need(Bg, "Bg", bf, (N, K), here),
            _need(Bu, "Bu", bf, (N, K), here), _need(dout, "dout", bf, (M, N), here), _act(act))
    dA = (torch.empty_like(A) if dA is None else dA) if need_input else None
    dBg = (torch.empty_like(Bg) if dBg is None else dBg) if need_weight else None
    dBu = (torch.empty_like(Bu) if dBu is None else dBu) if need_weight else None
    ws, wsb, keep = _scratch("qll_gated_backward_workspace_bytes",
                             L.qll_gated_backward_workspace_bytes(M, N, K), workspace, A, here)
    rc = L.gated_bf16_backward(
        *lead, _arg(dA, "dA", bf, (M, K), here), _arg(dBg, "dBg", bf, (N, K), here),
        _arg(dBu, "dBu", bf, (N, K), here), M, N, K, ws, wsb, st)
    if rc:
        raise QllError("gated_bf16_backward", rc)
    return dA, dBg, dBu


def _norm_args(y, r, w_pre, w_post, gate, alpha, beta, eps, here):
    torch = _torch()
    bf = torch.bfloat16
    M, K = _matrix(r, "r")
    dt = r.dtype
    if dt is bf:
        kind = 0
    elif dt is torch.float32:
        kind = 1
    else:
        raise ValueError("r must be bfloat16 or float32")
    if y is None and (w_post is not None or gate is not None or alpha != 1.0):
        raise ValueError("w_post, gate and alpha need a block output y")
    return M, K, dt, (_arg(y, "y", bf, (M, K), here), _need(r, "r", dt, (M, K), here), kind,
                      _arg(w_post, "w_post", bf, (K,), here), _arg(gate, "gate", bf, (K,), here),
                      _need(w_pre, "w_pre", bf, (K,), here), alpha, beta, eps)


def residual_norm(y, r, w_pre, w_post=None, gate=None, alpha=1.0, beta=1.0, eps=1e-6,
                  quantize=False, r_out=None, n_out=None, scales=None, stream=None):
    """Residual stream and pre-norm behind a block: h = alpha r + beta gate *
    (w_post y / rms(y)), n = w_pre h / rms(h).  y bf16 [M][K] (None: h = r), r
    bf16 or fp32 [M][K], vectors bf16 [K].  Returns (h, n) with n bf16, or with
    quantize (h, e4m3 codes, fp32 scales [M][1]).  r_out may be r."""
    if stream is not None:
        return _under(stream, residual_norm, y, r, w_pre, w_post, gate, alpha, beta, eps, quantize,
                      r_out, n_out, scales)
    torch = _torch()
    here, st = _place()
    M, K, dt, lead = _norm_args(y, r, w_pre, w_post, gate, alpha, beta, eps, here)
    ph = None
    if y is None:
        if r_out is not None:
            raise ValueError("without y the stream is r itself")
    elif r_out is None:
        r_out = torch.empty_like(r)
        ph = r_out.data_ptr()
    else:
        ph = _arg(r_out, "r_out", dt, (M, K), here)
    if quantize:
        if n_out is None:
            n_out = torch.empty_like(r, dtype=torch.float8_e4m3fn)
        if scales is None:
            scales = r.new_empty((M, 1), dtype=torch.float32)
        pn, ps = _codes(n_out, "n_out", (M, K), here), _scales(scales, "scales", M, here)
    else:
        if scales is not None:
            raise ValueError("scales need quantize")
        if n_out is None:
            n_out = torch.empty_like(r, dtype=torch.bfloat16)
        pn, ps = _arg(n_out, "n_out", torch.bfloat16, (M, K), here), None
    rc = load_library().residual_norm(*lead, ph, pn, ps, M, K, st)
    if rc:
        raise QllError("residual_norm", rc)
    h = r if y is None else r_out
    return (h, n_out, scales) if quantize else (h, n_out)


def residual_norm_backward(y, r, w_pre, dn, dr_out=None, w_post=None, gate=None, alpha=1.0,
                           beta=1.0, eps=1e-6, dy=None, dr=None, dw_pre=None, dw_post=None,
                           dgate=None, workspace=None, stream=None):
    """(dy, dr, dw_pre, dw_post, dgate) of residual_norm for dn bf16 [M][K]
    and dr_out [M][K] of r's type (None: zero); the vector gradients fp32 [K].
    None for what is not there."""
    if stream is not None:
        return _under(stream, residual_norm_backward, y, r, w_pre, dn, dr_out, w_post, gate, alpha,
                      beta, eps, dy, dr, dw_pre, dw_post, dgate, workspace)
    torch = _torch()
    here, st = _place()
    M, K, dt, lead = _norm_args(y, r, w_pre, w_post, gate, alpha, beta, eps, here)
    L = load_library()
    bf, f32 = torch.bfloat16, torch.float32
    if y is None:
        if dy is not None:
            raise ValueError("without y there is no dy")
    elif dy is None:
        dy = torch.empty_like(y)
    if dr is None:
        dr = torch.empty_like(r)
    vectors = []
    for name, w, dw in (("dw_post", w_post, dw_post), ("dgate", gate, dgate),
                        ("dw_pre", w_pre, dw_pre)):
        if w is None and dw is not None:
            raise ValueError(f"{name} without its vector")
        if w is not None and dw is None:
            dw = r.new_empty(K, dtype=f32)
        vectors.append(dw)
    dw_post, dgate, dw_pre = vectors
    ws, wsb, keep = _scratch("qll_residual_norm_backward_workspace_bytes",
                             L.qll_residual_norm_backward_workspace_bytes(M, K), workspace, r, here)
    rc = L.residual_norm_backward(
        *lead, _need(dn, "dn", bf, (M, K), here), _arg(dr_out, "dr_out", dt, (M, K), here),
        _arg(dy, "dy", bf, (M, K), here), _arg(dr, "dr", dt, (M, K), here),
        _arg(dw_post, "dw_post", f32, (K,), here), _arg(dgate, "dgate", f32, (K,), here),
        _arg(dw_pre, "dw_pre", f32, (K,), here), M, K, ws, wsb, st)
    if rc:
        raise QllError("residual_norm_backward", rc)
    return dy, dr, dw_pre, dw_post, dgate


# --------------------------------------------------------------------------
# registry / dispatch introspection
# --------------------------------------------------------------------------

def variants(op: str | int) -> list[dict]:
    L = load_library()
    o = OPS[op] if isinstance(op, str) else op
    buf = ctypes.create_string_buffer(512)
    out = []
    for i in range(L.qll_num_variants(o)):
        _check("qll_variant_info", L.qll_variant_info(o, i, buf, 512))
        d = json.loads(buf.value.decode())
        d["index"] = i
        out.append(d)
    return out


def select(op: str | int, M: int, N: int, K: int) -> tuple[str, int]:
    """(variant name, requested splits) the entry point would use."""
    _ensure_init()
    L = load_library()
    o = OPS[op] if isinstance(op, str) else op
    c = qll_cfg()
    _check("qll_select", L.qll_select(o, M, N, K, ctypes.byref(c)))
    return variants(o)[c.variant]["name"], c.splits


def effective_splits(op: str | int, K: int, splits: int) -> int:
    o = OPS[op] if isinstance(op, str) else op
    return load_library().qll_effective_splits(o, K, splits)


def workspace_bytes(op: str | int, M: int, N: int, K: int, cfg=None) -> int:
    o = OPS[op] if isinstance(op, str) else op
    c = _cfg(o, cfg)
    n = load_library().qll_workspace_bytes(o, M, N, K, ctypes.byref(c) if c else None)
    if n < 0:
        raise QllError("qll_workspace_bytes", -n)
    return n


def table_entries() -> int:
    return load_library().qll_table_entries()


def parse_signature(sig: str) -> tuple[str, int, int, str]:
    """'<arch> <CUs> <MHz> <name>' -> (arch, cus, mhz, name); the name may be
    empty."""
    parts = sig.strip().split(None, 3)
    if len(parts) < 3:
        raise ValueError(f"bad device signature {sig!r}")
    return parts[0], int(parts[1]), int(parts[2]), (parts[3].strip() if len(parts) > 3 else "")


def table_signature(path: str) -> str | None:
    """The device signature on a table file's device line (None if absent)."""
    with open(path) as f:
        for line in f:
            t = line.strip()
            if t.startswith("device ") or t.startswith("device\t"):
                return t[len("device"):].strip()
    return None


def table_validate(path: str, signature: str):
    """(status, reason) of checking a table file against a device signature
    '<arch> <CUs> <MHz> <name>'."""
    arch, cus, mhz, name = parse_signature(signature)
    buf = ctypes.create_string_buffer(512)
    rc = load_library().qll_table_validate(path.encode(), arch.encode(), cus, mhz,
                                           name.encode(), buf, 512)
    return rc, buf.value.decode()


def device_signature() -> str:
    """The current device's signature, as a table's device line holds it."""
    buf = ctypes.create_string_buffer(512)
    _check("qll_device_signature", load_library().qll_device_signature(buf, 512))
    return buf.value.decode()
