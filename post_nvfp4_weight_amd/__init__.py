"""NVFP4 weight quantization with GPTQ + Schur Replay on AMD Instinct MI355X.

Thin ctypes binding over libnvq.so (C ABI in include/nvq.h).  Every step of
the quantization runs in the library's HIP kernels; this module only checks
tensor metadata, allocates outputs and workspaces with torch, and passes raw
device pointers plus torch's current HIP stream.  There is no CPU fallback:
importing fails if the library is missing.

Method: "Replay the Curvature: Accurate and Scalable NVFP4 Quantization for
Large Language Model Inference" (arXiv 2609.36654), Abstract.
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvq.so")

NVQ_DTYPE_F32 = 0
NVQ_DTYPE_BF16 = 1
NVQ_DTYPE_MXFP4 = 2
FLAG_RTN = 1
FLAG_NO_ERR = 2
FLAG_FP64 = 4
FLAG_INDEP = 8
FLAG_CHECK_FINITE = 16
FLAG_CHOL_FACTOR = 32

EXPORTS = [
    "hessian_workspace_size", "hessian_accumulate",
    "hessian_grouped_workspace_size", "hessian_accumulate_grouped",
    "hessian_host_workspace_size", "hessian_host_staging_size", "hessian_accumulate_host",
    "factor_hinv_workspace_size", "factor_hinv", "factor_hinv_batched",
    "factor_chol_workspace_size", "factor_chol", "factor_chol_batched",
    "nvfp4_global_scale_workspace_size", "nvfp4_global_scale",
    "gptq_nvfp4_workspace_size", "gptq_nvfp4_quantize", "gptq_nvfp4_quantize_batched",
    "nvfp4_dequantize", "nvfp4_gemm_workspace_size", "nvfp4_gemm", "nvfp4_gemm_noalloc", "nvq_check_finite",
    "moe_topk", "moe_topk_backward", "moe_sort_workspace_size", "moe_sort",
    "nvfp4_gemm_grouped", "nvfp4_gemm_grouped_dx", "moe_combine", "moe_combine_backward",
    "mxfp4_quantize", "mxfp4_dequantize", "mxfp4_gemm_workspace_size", "mxfp4_gemm",
    "mxfp4_gemm_dx_workspace_size", "mxfp4_gemm_dx",
    "swiglu", "swiglu_backward", "nvfp4_moe_mlp_workspace_size", "nvfp4_moe_mlp",
    "nvq_status_string", "nvq_last_error",
]


class NvqError(RuntimeError):
    def __init__(self, fn, status, detail):
        super().__init__(f"{fn} failed with status {status}: {detail}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m post_nvfp4_weight_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, SZ, I32, F32, U32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int,
                                 ctypes.c_float, ctypes.c_uint)
    sig = {
        "hessian_workspace_size": (SZ, [I64, I64, I32]),
        "hessian_accumulate": (I32, [P, I32, I64, I64, I64, P, P, SZ, P]),
        "hessian_grouped_workspace_size": (SZ, [P, I64, I64, I32]),
        "hessian_host_workspace_size": (SZ, [I64, I64, I32]),
        "hessian_host_staging_size": (SZ, [I64, I64, I32]),
        "hessian_accumulate_host": (I32, [P, I32, I64, I64, I64, P, I64, P, SZ, P, SZ, P, P]),
        "hessian_accumulate_grouped": (I32, [P, I32, I64, I64, I64, P, P, I64, P, P, SZ, P]),
        "factor_hinv_batched": (I32, [P, I64, I64, I64, F32, P, I64, P, P, P, SZ, P]),
        "gptq_nvfp4_quantize_batched": (I32, [P, I32, I64, I64, I64, I64, I64, P, I64, P, I64, P, I32, U32, P, P,
                                               P, P, P, SZ, P]),
        "factor_hinv_workspace_size": (SZ, [I64]),
        "factor_hinv": (I32, [P, I64, F32, P, P, P, P, SZ, P]),
        "factor_chol_workspace_size": (SZ, [I64]),
        "factor_chol": (I32, [P, I64, F32, P, P, P, P, SZ, P]),
        "factor_chol_batched": (I32, [P, I64, I64, I64, F32, P, I64, P, P, P, SZ, P]),
        "nvfp4_global_scale_workspace_size": (SZ, [I64, I64]),
        "nvfp4_global_scale": (I32, [P, I32, I64, I64, I64, P, P, SZ, P]),
        "gptq_nvfp4_workspace_size": (SZ, [I64, I64, U32]),
        "gptq_nvfp4_quantize": (I32, [P, I32, I64, I64, I64, P, P, P, I32, U32, P, P, P, P, P, SZ, P]),
        "nvfp4_dequantize": (I32, [P, P, P, I64, I64, P, I32, P]),
        "nvfp4_gemm_workspace_size": (SZ, [I64, I64, I64]),
        "nvfp4_gemm": (I32, [P, I32, I64, I64, I64, P, P, P, I64, P, I32, I64, P, SZ, P]),
        "nvfp4_gemm_noalloc": (I32, [P, I32, I64, I64, I64, P, P, P, I64, P, I32, I64, P]),
        "nvq_check_finite": (I32, [P, I32, I64, I64, I64, P, P]),
        "moe_topk": (I32, [P, I32, I64, I64, I64, I32, I32, P, P, P]),
        "moe_topk_backward": (I32, [P, I32, I64, I64, I64, P, P, P, I32, I32, P, I64, P]),
        "moe_sort_workspace_size": (SZ, [I64, I64, I64]),
        "moe_sort": (I32, [P, I64, I64, I64, P, P, P, P, SZ, P]),
        "nvfp4_gemm_grouped": (I32, [P, I32, I64, I64, I64, P, I64, P, I64, P, P, P, I64, P, I32, I64, P]),
        "nvfp4_gemm_grouped_dx": (I32, [P, I32, I64, I64, I64, P, I64, P, P, P, I64, P, I32, I64, P]),
        "moe_combine": (I32, [P, I32, I64, I64, I64, P, P, I64, I64, P, I32, I64, P]),
        "moe_combine_backward": (I32, [P, I32, I64, I64, I64, P, I32, I64, I64, P, P, I64, P, I64, P, P]),
        "mxfp4_quantize": (I32, [P, I32, I64, I64, I64, P, P, P]),
        "mxfp4_dequantize": (I32, [P, P, I64, I64, P, I32, P]),
        "mxfp4_gemm_workspace_size": (SZ, [I32, I64, I64, I64]),
        "mxfp4_gemm": (I32, [P, I32, P, I64, I64, I64, P, P, I64, P, I32, I64, P, SZ, P]),
        "mxfp4_gemm_dx_workspace_size": (SZ, [I64, I64, I64]),
        "mxfp4_gemm_dx": (I32, [P, I32, I64, I64, I64, P, P, I64, P, I32, I64, P, SZ, P]),
        "swiglu": (I32, [P, I32, I64, I64, I64, P, I32, I64, P]),
        "swiglu_backward": (I32, [P, I64, P, I32, I64, I64, I64, P, I64, P]),
        "nvfp4_moe_mlp_workspace_size": (SZ, [I64, I64, I64, I64]),
        "nvfp4_moe_mlp": (I32, [P, I32, I64, I64, I64, P, I32, I64, I64, I64, I32, P, P, P, P, P, I64, P, P, P, I64, P, I32, I64, P, SZ,
                                P]),
        "nvq_status_string": (ctypes.c_char_p, [I32]),
        "nvq_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load()


def _check(fn, status):
    if status != 0:
        raise NvqError(fn, status, lib.nvq_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return NVQ_DTYPE_BF16
    if t.dtype == torch.float32:
        return NVQ_DTYPE_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _workspace(nbytes, device):
    if nbytes == 0:
        return None
    # torch's caching allocator returns 256-byte aligned blocks (checked by the library).
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _rows(t, name):
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a HIP device")
    return t.shape[0], t.shape[1], t.stride(0)


def hessian_accumulate(X, H=None, ws=None):
    """H += X^T X (fp32 [k, k], full symmetric on return).  X: [n, k] bf16 or fp32."""
    n, k, ldx = _rows(X, "X")
    if H is None:
        H = torch.zeros(k, k, dtype=torch.float32, device=X.device)
    need = lib.hessian_workspace_size(n, k, _dtype_code(X))
    if ws is None or ws.numel() < need:
        ws = _workspace(need, X.device)
    _check("hessian_accumulate", lib.hessian_accumulate(_ptr(X), _dtype_code(X), n, k, ldx, _ptr(H), _ptr(ws),
                                                        need, _stream()))
    return H


def nvfp4_gemm(X, codes, scales, g, out_dtype=torch.float32, Y=None):
    """Y = X dequant(W)^T for bf16 activations X [T, k] and NVFP4 weights (codes [m, k/2], scales [m, k/16], g)."""
    T, k, ldx = _rows(X, "X")
    m = codes.shape[0]
    if Y is None:
        Y = torch.empty(T, m, dtype=out_dtype, device=X.device)
    need = lib.nvfp4_gemm_workspace_size(T, k, m)
    ws = _workspace(need, X.device) if need else None
    _check("nvfp4_gemm", lib.nvfp4_gemm(_ptr(X), _dtype_code(X), T, k, ldx, _ptr(codes), _ptr(scales), _ptr(g), m,
                                        _ptr(Y), _dtype_code(Y), Y.stride(0), _ptr(ws), need, _stream()))
    return Y


def nvfp4_gemm_noalloc(X, codes, scales, g, Y):
    """Y = X dequant(W)^T into a preallocated Y [T, m] (fp32 or bf16); the library allocates nothing."""
    T, k, ldx = _rows(X, "X")
    m = codes.shape[0]
    _check("nvfp4_gemm_noalloc", lib.nvfp4_gemm_noalloc(_ptr(X), _dtype_code(X), T, k, ldx, _ptr(codes),
                                                        _ptr(scales), _ptr(g), m, _ptr(Y), _dtype_code(Y),
                                                        Y.stride(0), _stream()))
    return Y


_copy_streams = {}


def hessian_accumulate_host(X, H=None, chunk=32768, staging=True, device="cuda:0"):
    """H += X^T X with X in host memory, streamed to the device in chunks.

    X: a CPU torch tensor (bf16 or fp32, pinned or not) or a NumPy array whose
    rows are contiguous: uint16 holding bf16 bits, or float32 (a np.memmap of
    a file on disk works).  Pageable X goes through pinned staging buffers
    (staging=True); the copies run on a library copy stream of default
    priority, overlapped with the accumulation on the current stream.
    """
    if isinstance(X, torch.Tensor):
        if X.device.type != "cpu" or X.dim() != 2 or X.stride(1) != 1:
            raise ValueError("X must be a 2-D CPU tensor with contiguous rows")
        code = _dtype_code(X)
        ptr, ldx, pinned = X.data_ptr(), X.stride(0), X.is_pinned()
    else:
        import numpy as np
        X = np.asarray(X) if not isinstance(X, np.ndarray) else X
        if X.ndim != 2 or X.strides[1] != X.itemsize:
            raise ValueError("X must be 2-D with contiguous rows")
        if X.dtype == np.uint16:
            code = NVQ_DTYPE_BF16
        elif X.dtype == np.float32:
            code = NVQ_DTYPE_F32
        else:
            raise ValueError("NumPy X must be uint16 (bf16 bits) or float32")
        ptr, ldx, pinned = X.ctypes.data, X.strides[0] // X.itemsize, False
    n, k = X.shape
    dev = torch.device(device)
    if H is None:
        H = torch.zeros(k, k, dtype=torch.float32, device=dev)
    need = lib.hessian_host_workspace_size(chunk, k, code)
    ws = _workspace(need, dev)
    stg, stg_n = None, 0
    if staging and not pinned:
        stg_n = lib.hessian_host_staging_size(chunk, k, code)
        stg = torch.empty(max(1, stg_n), dtype=torch.uint8, pin_memory=True)
    if dev not in _copy_streams:
        _copy_streams[dev] = torch.cuda.Stream(device=dev)
    cs = _copy_streams[dev]
    cur = torch.cuda.current_stream(dev)
    cs.wait_stream(cur)   # H and the workspace are ready before the first copy
    _check("hessian_accumulate_host",
           lib.hessian_accumulate_host(ctypes.c_void_p(ptr), code, n, k, ldx, _ptr(H), chunk, _ptr(ws), need,
                                       _ptr(stg), stg_n, ctypes.c_void_p(cur.cuda_stream),
                                       ctypes.c_void_p(cs.cuda_stream)))
    ws.record_stream(cs)
    return H


def factor_hinv(H, damp_rel=0.01, U=None, ws=None):
    """Returns (U, lam, info) as device tensors: (H + lam I)^-1 = U^T U, lam = damp_rel * mean(diag H)."""
    k = H.shape[0]
    U = torch.empty_like(H) if U is None else U
    lam = torch.empty(1, dtype=torch.float32, device=H.device)
    info = torch.empty(1, dtype=torch.int32, device=H.device)
    need = lib.factor_hinv_workspace_size(k)
    if ws is None or ws.numel() < need:
        ws = _workspace(need, H.device)
    _check("factor_hinv", lib.factor_hinv(_ptr(H), k, float(damp_rel), _ptr(U), _ptr(lam), _ptr(info), _ptr(ws),
                                          need, _stream()))
    return U, lam, info


def nvfp4_global_scale(W):
    """Device fp32 scalar tensor g = fl32(max|W| / 2688) (1 for an all-zero W)."""
    m, k, ldw = _rows(W, "W")
    g = torch.empty(1, dtype=torch.float32, device=W.device)
    need = lib.nvfp4_global_scale_workspace_size(m, k)
    ws = _workspace(need, W.device)
    _check("nvfp4_global_scale", lib.nvfp4_global_scale(_ptr(W), _dtype_code(W), m, k, ldw, _ptr(g), _ptr(ws),
                                                        need, _stream()))
    return g


def gptq_nvfp4_quantize(W, U, H, g, n_cand=16, flags=0, ws=None, out=None):
    """NVFP4 quantization of W [m, k]; returns dict(codes [m, k/2] u8, scales [m, k/16] u8,
    row_err [m] f32 or None, row_loss [m] f32)."""
    m, k, ldw = _rows(W, "W")
    dev = W.device
    if out is None:
        out = {
            "codes": torch.empty(m, k // 2, dtype=torch.uint8, device=dev),
            "scales": torch.empty(m, k // 16, dtype=torch.uint8, device=dev),
            "row_err": None if (flags & FLAG_NO_ERR) else torch.empty(m, dtype=torch.float32, device=dev),
            "row_loss": torch.empty(m, dtype=torch.float32, device=dev),
        }
    need = lib.gptq_nvfp4_workspace_size(m, k, flags)
    if ws is None or ws.numel() < need:
        ws = _workspace(need, dev)
    _check("gptq_nvfp4_quantize", lib.gptq_nvfp4_quantize(
        _ptr(W), _dtype_code(W), m, k, ldw, _ptr(U), _ptr(H), _ptr(g), int(n_cand), int(flags),
        _ptr(out["codes"]), _ptr(out["scales"]), _ptr(out["row_err"]), _ptr(out["row_loss"]), _ptr(ws), need,
        _stream()))
    return out


def nvfp4_dequantize(codes, scales, g, out_dtype=torch.float32):
    m, kh = codes.shape
    k = kh * 2
    out = torch.empty(m, k, dtype=out_dtype, device=codes.device)
    _check("nvfp4_dequantize", lib.nvfp4_dequantize(_ptr(codes), _ptr(scales), _ptr(g), m, k, _ptr(out),
                                                    _dtype_code(out), _stream()))
    return out


def hessian_accumulate_grouped(X, tok_idx, grp_off, H=None):
    """Per-group H[e] += X[idx_e]^T X[idx_e]; tok_idx: device int32 [total], grp_off: host sequence [G+1]."""
    import numpy as np
    n, k, ldx = _rows(X, "X")
    off = np.ascontiguousarray(np.asarray(grp_off, dtype=np.int64))
    G = len(off) - 1
    if H is None:
        H = torch.zeros(G, k, k, dtype=torch.float32, device=X.device)
    offp = off.ctypes.data_as(ctypes.c_void_p)
    need = lib.hessian_grouped_workspace_size(offp, G, k, _dtype_code(X))
    ws = _workspace(need, X.device)
    idx = tok_idx if tok_idx.dtype == torch.int32 else tok_idx.to(torch.int32)
    _check("hessian_accumulate_grouped", lib.hessian_accumulate_grouped(
        _ptr(X), _dtype_code(X), n, k, ldx, _ptr(idx), offp, G, _ptr(H), _ptr(ws), need, _stream()))
    return H


def factor_hinv_batched(H, damp_rel=0.01, max_ws_bytes=8 << 30):
    """H: [B, k, k] -> (U [B, k, k], lam [B], info [B]) as device tensors.

    The workspace holds as many matrices' buffers as fit in max_ws_bytes (at
    least one, at most B): the library factors that many matrices per pass,
    every launch covering all of them."""
    B, k = H.shape[0], H.shape[1]
    U = torch.empty_like(H)
    lam = torch.empty(B, dtype=torch.float32, device=H.device)
    info = torch.empty(B, dtype=torch.int32, device=H.device)
    one = lib.factor_hinv_workspace_size(k)
    need = one * max(1, min(B, max_ws_bytes // one))
    ws = _workspace(need, H.device)
    _check("factor_hinv_batched", lib.factor_hinv_batched(_ptr(H), k, B, H.stride(0), float(damp_rel), _ptr(U),
                                                          U.stride(0), _ptr(lam), _ptr(info), _ptr(ws), need,
                                                          _stream()))
    return U, lam, info


def factor_chol_batched(H, damp_rel=0.01, max_ws_bytes=8 << 30):
    """H: [B, k, k] -> (V [B, k, k], lam [B], info [B]) as device tensors, each V as
    factor_chol gives it (for FLAG_CHOL_FACTOR); passes of as many matrices as
    fit in max_ws_bytes of workspace."""
    B, k = H.shape[0], H.shape[1]
    V = torch.empty_like(H)
    lam = torch.empty(B, dtype=torch.float32, device=H.device)
    info = torch.empty(B, dtype=torch.int32, device=H.device)
    one = lib.factor_chol_workspace_size(k)
    need = one * max(1, min(B, max_ws_bytes // one))
    ws = _workspace(need, H.device)
    _check("factor_chol_batched", lib.factor_chol_batched(_ptr(H), k, B, H.stride(0), float(damp_rel), _ptr(V),
                                                          V.stride(0), _ptr(lam), _ptr(info), _ptr(ws), need,
                                                          _stream()))
    return V, lam, info


def gptq_nvfp4_quantize_batched(W, U, H, g, n_cand=16, flags=0, max_ws_bytes=8 << 30):
    """W: [B, m, k]; U, H: [B, k, k] (or None as the flags allow); g: device fp32 [B].

    The workspace holds as many matrices' working buffers as fit in
    max_ws_bytes (at least one): that many are quantized per pass."""
    B, m, k = W.shape
    dev = W.device
    if W.stride(2) != 1:
        raise ValueError("W must have unit column stride")
    out = {
        "codes": torch.empty(B, m, k // 2, dtype=torch.uint8, device=dev),
        "scales": torch.empty(B, m, k // 16, dtype=torch.uint8, device=dev),
        "row_err": None if (flags & FLAG_NO_ERR) else torch.empty(B, m, dtype=torch.float32, device=dev),
        "row_loss": torch.empty(B, m, dtype=torch.float32, device=dev),
    }
    one = lib.gptq_nvfp4_workspace_size(m, k, flags)
    need = one * max(1, min(B, max_ws_bytes // one))
    ws = _workspace(need, dev)
    _check("gptq_nvfp4_quantize_batched", lib.gptq_nvfp4_quantize_batched(
        _ptr(W), _dtype_code(W), B, m, k, W.stride(1), W.stride(0), _ptr(U), 0 if U is None else U.stride(0),
        _ptr(H), 0 if H is None else H.stride(0), _ptr(g), int(n_cand), int(flags), _ptr(out["codes"]),
        _ptr(out["scales"]), _ptr(out["row_err"]), _ptr(out["row_loss"]), _ptr(ws), need, _stream()))
    return out


def check_finite(A):
    """Device int32 tensor [1]: 0 if every value of A [rows, cols] is finite, else 1 + the first bad row."""
    rows, cols, ld = _rows(A, "A")
    status = torch.empty(1, dtype=torch.int32, device=A.device)
    _check("nvq_check_finite", lib.nvq_check_finite(_ptr(A), _dtype_code(A), rows, cols, ld, _ptr(status), _stream()))
    return status


def factor_chol(H, damp_rel=0.01, V=None, ws=None):
    """Returns (V, lam, info) as device tensors: H + lam I = R R^T with R upper triangular,
    V = -R_ij / R_jj above the diagonal, R_ii on it, 0 below (for FLAG_CHOL_FACTOR)."""
    k = H.shape[0]
    V = torch.empty_like(H) if V is None else V
    lam = torch.empty(1, dtype=torch.float32, device=H.device)
    info = torch.empty(1, dtype=torch.int32, device=H.device)
    need = lib.factor_chol_workspace_size(k)
    if ws is None or ws.numel() < need:
        ws = _workspace(need, H.device)
    _check("factor_chol", lib.factor_chol(_ptr(H), k, float(damp_rel), _ptr(V), _ptr(lam), _ptr(info), _ptr(ws),
                                          need, _stream()))
    return V, lam, info


def quantize_layer(W, X, n_cand=16, damp_rel=0.01, flags=0, chol=False):
    """Whole layer: H = X^T X, the factor (U from factor_hinv, or with chol V from factor_chol and
    FLAG_CHOL_FACTOR), g, the sweep and the weighted error (all on the GPU)."""
    H = hessian_accumulate(X)
    if chol:
        U, lam, info = factor_chol(H, damp_rel)
        flags |= FLAG_CHOL_FACTOR
    else:
        U, lam, info = factor_hinv(H, damp_rel)
    g = nvfp4_global_scale(W)
    res = gptq_nvfp4_quantize(W, U, H, g, n_cand, flags)
    res.update(H=H, U=U, lam=lam, info=info, g=g)
    return res


# ---- mixture of experts -------------------------------------------------------
# moe_topk -> moe_sort -> nvfp4_gemm_grouped -> moe_combine, with the gradients
# of all but the sort.  Tensors of one call must share a device; the work runs
# on that device's current stream.

_F32, _BF16, _I32, _I64, _U8 = torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8
_FLOATS = (_F32, _BF16)
_CODES = {_F32: NVQ_DTYPE_F32, _BF16: NVQ_DTYPE_BF16}


def _want(t, name, dtypes, shape, dev):
    """Raises unless t is a tensor on HIP device number dev (None: any) of one of dtypes and of that shape (None: any size)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a tensor on a HIP device")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, not one of {dtypes}")
    if t.dim() != len(shape) or any(s is not None and s != n for s, n in zip(shape, t.shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")


def _dense(t, name, dtype, shape, dev):
    """t must be a contiguous tensor of that dtype and shape on device number dev."""
    if not (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is dtype and t.shape == shape
            and t.is_contiguous()):
        _want(t, name, (dtype,), shape, dev)
        raise ValueError(f"{name} must be contiguous")


def _matrix(t, name, dtypes, dev=None):
    """(rows, columns, row stride) of a 2-D tensor of unit column stride, of one of dtypes, on device number dev (None: any)."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.dim() == 2
            and (dev is None or t.get_device() == dev)):
        _want(t, name, dtypes, (None, None), dev)
    (rows, cols), (s0, s1) = t.shape, t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows <= 1:
        return rows, cols, cols
    if s0 < cols:
        raise ValueError(f"{name} must not have overlapping rows")
    return rows, cols, s0


def _table(t, name, rows, dev):
    """Columns of a contiguous int32 tensor [rows, *] (rows None: any) on device number dev."""
    if not (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is _I32 and t.dim() == 2
            and (rows is None or t.shape[0] == rows) and t.is_contiguous()):
        _want(t, name, (_I32,), (rows, None), dev)
        raise ValueError(f"{name} must be contiguous")
    return t.shape[1]


def _output(t, name, like, rows, cols, dtype, dev):
    """(t, row stride): the caller's output, checked, or a new one beside `like`."""
    if t is None:
        if dtype not in _FLOATS:
            raise TypeError(f"unsupported dtype {dtype}")
        return like.new_empty((rows, cols), dtype=dtype), cols
    r, c, ld = _matrix(t, name, _FLOATS, dev)
    if r != rows or c != cols:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {(rows, cols)}")
    return t, ld


def _addr(t):
    return None if t is None else t.data_ptr()


_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _call(f, name, dev, *args):
    """The library call on the current stream of device number dev, with that device current."""
    if dev == _current_device():
        status = f(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = f(*args, _raw_stream(dev))
    if status != 0:
        raise NvqError(name, status, lib.nvq_last_error().decode())


def moe_topk(logits, top_k, renorm=True):
    """The router: (ids int32 [T, top_k], weights fp32 [T, top_k]) of logits [T, E] (bf16 or fp32), each token's largest
    logits in falling order (ties: the lower expert) and their softmax weights, over the chosen experts (renorm) or all.
    -inf masks an expert; a slot with no expert left has id -1 and weight 0, a row with a NaN or +inf ids -1 and NaN."""
    T, E, ld = _matrix(logits, "logits", _FLOATS)
    top_k = int(top_k)
    ids = logits.new_empty((T, max(0, top_k)), dtype=_I32)
    weights = logits.new_empty((T, max(0, top_k)), dtype=_F32)
    _call(lib.moe_topk, "moe_topk", logits.get_device(), logits.data_ptr(), _CODES[logits.dtype], T, E, ld, top_k, bool(renorm), ids.data_ptr(),
          weights.data_ptr())
    return ids, weights


def moe_topk_backward(logits, ids, weights, dweights, renorm=True):
    """Gradient of moe_topk's weights with respect to the logits: [T, E] in the logits' dtype."""
    T, E, ld = _matrix(logits, "logits", _FLOATS)
    dev = logits.get_device()
    K = _table(ids, "ids", T, dev)
    _dense(weights, "weights", _F32, (T, K), dev)
    _dense(dweights, "dweights", _F32, (T, K), dev)
    out = logits.new_empty((T, E))
    _call(lib.moe_topk_backward, "moe_topk_backward", dev, logits.data_ptr(), _CODES[logits.dtype], T, E, ld, ids.data_ptr(),
          weights.data_ptr(), dweights.data_ptr(), K, bool(renorm), out.data_ptr(), E)
    return out


def moe_sort(ids, n_experts):
    """Slots sorted by expert: (tok_idx int32 [T*K], grp_off int64 [E+1], pos int32 [T, K]) of ids int32 [T, K].  Row r of
    expert e (grp_off[e] <= r < grp_off[e+1]) is token tok_idx[r]; slot (t, s) is row pos[t, s].  Slots whose id is
    outside [0, n_experts) have pos -1, and tok_idx past the last row is -1.  (hessian_accumulate_grouped takes tok_idx
    and grp_off.tolist().)"""
    if not isinstance(ids, torch.Tensor) or not ids.is_cuda:
        raise ValueError("ids must be a tensor on a HIP device")
    dev = ids.get_device()
    K = _table(ids, "ids", None, dev)
    T = ids.shape[0]
    E = int(n_experts)
    tok_idx = ids.new_empty(T * K)
    grp_off = ids.new_empty(max(0, E) + 1, dtype=_I64)
    pos = ids.new_empty((T, K))
    need = lib.moe_sort_workspace_size(T, K, E)
    ws = _workspace(need, ids.device) if need else None
    _call(lib.moe_sort, "moe_sort", dev, ids.data_ptr(), T, K, E, tok_idx.data_ptr(), grp_off.data_ptr(), pos.data_ptr(), _addr(ws),
          need)
    return tok_idx, grp_off, pos


def _experts(codes, scales, g, grp_off, dev):
    """(G, m, k) of the experts' tensors, checked."""
    _want(codes, "codes", (_U8,), (None, None, None), dev)
    G, m, kh = codes.shape
    _dense(codes, "codes", _U8, (G, m, kh), dev)
    _dense(scales, "scales", _U8, (G, m, kh // 8), dev)
    _dense(g, "g", _F32, (G,), dev)
    _dense(grp_off, "grp_off", _I64, (G + 1,), dev)
    return G, m, 2 * kh


def nvfp4_gemm_grouped(X, codes, scales, g, grp_off, tok_idx=None, out_dtype=torch.float32, Y=None):
    """Y[r] = X[tok_idx[r]] dequant(W_e)^T for the rows r of each expert e (grp_off[e] <= r < grp_off[e+1]).

    X: [n, k] bf16; codes [G, m, k/2], scales [G, m, k/16], g [G] as gptq_nvfp4_quantize_batched gives them; grp_off and
    tok_idx from moe_sort (without tok_idx row r of X is row r).  Rows of Y from grp_off[G] on are not written."""
    n, kx, ldx = _matrix(X, "X", (_BF16,))
    dev = X.get_device()
    G, m, k = _experts(codes, scales, g, grp_off, dev)
    if kx != k:
        raise ValueError(f"X has {kx} columns, the experts {k} inputs")
    rows = n
    if tok_idx is not None:
        if not isinstance(tok_idx, torch.Tensor) or tok_idx.dim() != 1:
            raise ValueError("tok_idx must be a 1-D tensor")
        rows = tok_idx.shape[0]
        _dense(tok_idx, "tok_idx", _I32, (rows,), dev)
    Y, ldy = _output(Y, "Y", X, rows, m, out_dtype, dev)
    _call(lib.nvfp4_gemm_grouped, "nvfp4_gemm_grouped", dev, X.data_ptr(), NVQ_DTYPE_BF16, n, k, ldx, _addr(tok_idx), rows, grp_off.data_ptr(), G,
          codes.data_ptr(), scales.data_ptr(), g.data_ptr(), m, Y.data_ptr(), _CODES[Y.dtype], ldy)
    return Y


def nvfp4_gemm_grouped_dx(dY, codes, scales, g, grp_off, out_dtype=torch.float32, dX=None):
    """Gradient of nvfp4_gemm_grouped with respect to its rows: dX[r] = dY[r] dequant(W_e), dY [rows, m] bf16 (as
    moe_combine_backward gives it for products with out_dtype bf16; their default is fp32).  The tokens'
    gradient is moe_combine(dX, pos).  Rows from grp_off[G] on are not written."""
    rows, my, lddy = _matrix(dY, "dY", (_BF16,))
    dev = dY.get_device()
    G, m, k = _experts(codes, scales, g, grp_off, dev)
    if my != m:
        raise ValueError(f"dY has {my} columns, the experts {m} outputs")
    dX, lddx = _output(dX, "dX", dY, rows, k, out_dtype, dev)
    _call(lib.nvfp4_gemm_grouped_dx, "nvfp4_gemm_grouped_dx", dev, dY.data_ptr(), NVQ_DTYPE_BF16, rows, m, lddy, grp_off.data_ptr(), G,
          codes.data_ptr(), scales.data_ptr(), g.data_ptr(), k, dX.data_ptr(), _CODES[dX.dtype], lddx)
    return dX


def moe_combine(Y, pos, weights=None, out_dtype=None, out=None):
    """out[t] = sum_s weights[t, s] * Y[pos[t, s]] (weights None: all 1), Y [rows, d] bf16 or fp32, pos int32 and weights
    fp32 [T, K].  A pos outside the rows counts as zeros.  out_dtype None: Y's."""
    rows, d, ldy = _matrix(Y, "Y", _FLOATS)
    dev = Y.get_device()
    K = _table(pos, "pos", None, dev)
    T = pos.shape[0]
    if weights is not None:
        _dense(weights, "weights", _F32, (T, K), dev)
    out, ldo = _output(out, "out", Y, T, d, out_dtype or Y.dtype, dev)
    _call(lib.moe_combine, "moe_combine", dev, Y.data_ptr(), _CODES[Y.dtype], rows, d, ldy, pos.data_ptr(), _addr(weights), T, K,
          out.data_ptr(), _CODES[out.dtype], ldo)
    return out


def moe_combine_backward(dout, Y, pos, weights=None, dY=None, need_dY=True, need_dweights=True):
    """Gradients of moe_combine: (dY [rows, d] in Y's dtype, dweights fp32 [T, K]).  Rows of dY that no slot of pos names
    (past moe_sort's last row) are not written; no row may be named twice.  One that is not needed is None: dweights where
    the router is frozen (Y is then not read, and may be None beside a dY of the caller's), dY where the experts and what
    is before them are.  For nvfp4_gemm_grouped_dx, which takes bf16, Y is to be bf16 too."""
    T, d, ldd = _matrix(dout, "dout", _FLOATS)
    dev = dout.get_device()
    if Y is None and (need_dweights or dY is None):
        raise ValueError("Y is required, but beside a dY and without dweights")
    if dY is not None and not need_dY:
        raise ValueError("dY is given, but not needed")
    like = dY if Y is None else Y
    rows, dy, ldy = _matrix(like, "dY" if Y is None else "Y", _FLOATS, dev)
    if dy != d:
        raise ValueError(f"dout has {d} columns, Y {dy}")
    K = _table(pos, "pos", T, dev)
    if weights is not None:
        _dense(weights, "weights", _F32, (T, K), dev)
    if dY is not None and (not isinstance(dY, torch.Tensor) or dY.dtype is not like.dtype):
        raise TypeError("dY must be a tensor of Y's dtype")
    lddy = d
    if need_dY:
        dY, lddy = _output(dY, "dY", like, rows, d, like.dtype, dev)
    dw = dout.new_empty((T, K), dtype=_F32) if need_dweights else None
    _call(lib.moe_combine_backward, "moe_combine_backward", dev, dout.data_ptr(), _CODES[dout.dtype], T, d, ldd, _addr(Y), _CODES[like.dtype],
          rows, ldy, pos.data_ptr(), _addr(weights), K, _addr(dY), lddy, _addr(dw))
    return dY, dw


# ---- MXFP4 and the gated activation ----------------------------------------------
# mxfp4_quantize -> mxfp4_gemm -> swiglu -> mxfp4_gemm is a dense MLP on 4-bit
# activations and weights; swiglu also stands between the experts' products.

def _mxfp4(codes, scales, name, dev):
    """(rows, k) of MXFP4 codes [rows, k/2] and scales [rows, k/32] on device number dev (None: any)."""
    if not (isinstance(codes, torch.Tensor) and codes.is_cuda and codes.dtype is _U8 and codes.dim() == 2
            and (dev is None or codes.get_device() == dev) and codes.is_contiguous()):
        _want(codes, name, (_U8,), (None, None), dev)
        raise ValueError(f"{name} must be contiguous")
    rows, kh = codes.shape
    if kh % 16:
        raise ValueError(f"{name} has {kh} bytes per row, not a multiple of 16 (blocks of 32)")
    if not (isinstance(scales, torch.Tensor) and scales.dtype is _U8 and scales.shape == (rows, kh // 16)
            and scales.get_device() == codes.get_device() and scales.is_contiguous()):
        _dense(scales, f"{name}' scales", _U8, (rows, kh // 16), codes.get_device())
    return rows, 2 * kh


def mxfp4_quantize(X):
    """(codes uint8 [n, k/2], scales uint8 [n, k/32]) of X [n, k] bf16 or fp32: E2M1 elements, 32 of a row under one power of
    two (byte b: 2^(b - 127), 255: NaN).  For gradients the quantization counts as the identity."""
    n, k, ldx = _matrix(X, "X", _FLOATS)
    codes = X.new_empty((n, k // 2), dtype=_U8)
    scales = X.new_empty((n, k // 32), dtype=_U8)
    _call(lib.mxfp4_quantize, "mxfp4_quantize", X.get_device(), X.data_ptr(), _CODES[X.dtype], n, k, ldx, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def mxfp4_dequantize(codes, scales, out_dtype=torch.float32):
    """The values [n, k] of MXFP4 codes and scales, exact in fp32 and in bf16."""
    n, k = _mxfp4(codes, scales, "codes", None)
    if out_dtype not in _FLOATS:
        raise TypeError(f"unsupported dtype {out_dtype}")
    out = codes.new_empty((n, k), dtype=out_dtype)
    _call(lib.mxfp4_dequantize, "mxfp4_dequantize", codes.get_device(), codes.data_ptr(), scales.data_ptr(), n, k, out.data_ptr(),
          _CODES[out_dtype])
    return out


def mxfp4_gemm(X, codes, scales, x_scales=None, out_dtype=torch.float32, Y=None):
    """Y = Q(X) W^T [n, m] on 4-bit operands, W the MXFP4 codes [m, k/2] and scales [m, k/32].

    X: [n, k] bf16 or fp32, quantized within the call as by mxfp4_quantize; or the codes [n, k/2] that mxfp4_quantize gave,
    with their x_scales (one quantization for several products of the same activations)."""
    m, k = _mxfp4(codes, scales, "codes", None)
    dev = codes.get_device()
    if x_scales is not None:
        n, kx = _mxfp4(X, x_scales, "X", dev)
        ldx, code = kx, NVQ_DTYPE_MXFP4
    else:
        n, kx, ldx = _matrix(X, "X", _FLOATS, dev)
        code = _CODES[X.dtype]
    if kx != k:
        raise ValueError(f"X has {kx} columns, the weights {k} inputs")
    Y, ldy = _output(Y, "Y", X, n, m, out_dtype, dev)
    need = lib.mxfp4_gemm_workspace_size(code, n, k, m)
    ws = _workspace(need, X.device) if need else None
    _call(lib.mxfp4_gemm, "mxfp4_gemm", dev, X.data_ptr(), code, _addr(x_scales), n, k, ldx, codes.data_ptr(), scales.data_ptr(), m,
          Y.data_ptr(), _CODES[Y.dtype], ldy, _addr(ws), need)
    return Y


def mxfp4_gemm_dx(dY, codes, scales, out_dtype=torch.float32, dX=None):
    """Gradient of mxfp4_gemm with respect to X (its quantization counts as the identity): dX = dY W, dY [n, m] bf16."""
    m, k = _mxfp4(codes, scales, "codes", None)
    dev = codes.get_device()
    n, my, lddy = _matrix(dY, "dY", (_BF16,), dev)
    if my != m:
        raise ValueError(f"dY has {my} columns, the weights {m} outputs")
    dX, lddx = _output(dX, "dX", dY, n, k, out_dtype, dev)
    need = lib.mxfp4_gemm_dx_workspace_size(n, m, k)
    ws = _workspace(need, dY.device) if need else None
    _call(lib.mxfp4_gemm_dx, "mxfp4_gemm_dx", dev, dY.data_ptr(), NVQ_DTYPE_BF16, n, m, lddy, codes.data_ptr(), scales.data_ptr(), k,
          dX.data_ptr(), _CODES[dX.dtype], lddx, _addr(ws), need)
    return dX


def swiglu(X, out_dtype=None, out=None):
    """silu(gate) * up [n, h] of X = [gate | up] [n, 2h], bf16 or fp32; out_dtype None: X's."""
    n, w, ldx = _matrix(X, "X", _FLOATS)
    if w % 2:
        raise ValueError(f"X has {w} columns, an odd number")
    dev = X.get_device()
    out, ldo = _output(out, "out", X, n, w // 2, out_dtype or X.dtype, dev)
    _call(lib.swiglu, "swiglu", dev, X.data_ptr(), _CODES[X.dtype], n, w // 2, ldx, out.data_ptr(), _CODES[out.dtype], ldo)
    return out


def swiglu_backward(dout, X, dX=None):
    """Gradient of swiglu with respect to X [n, 2h]; dout [n, h] of X's dtype, which dX has too."""
    n, w, ldx = _matrix(X, "X", _FLOATS)
    if w % 2:
        raise ValueError(f"X has {w} columns, an odd number")
    dev = X.get_device()
    nd, h, ldd = _matrix(dout, "dout", (X.dtype,), dev)
    if (nd, 2 * h) != (n, w):
        raise ValueError(f"dout has shape {tuple(dout.shape)}, not {(n, w // 2)}")
    if dX is not None and (not isinstance(dX, torch.Tensor) or dX.dtype is not X.dtype):
        raise TypeError("dX must be a tensor of X's dtype")
    dX, lddx = _output(dX, "dX", X, n, w, X.dtype, dev)
    _call(lib.swiglu_backward, "swiglu_backward", dev, dout.data_ptr(), ldd, X.data_ptr(), _CODES[X.dtype], n, h, ldx, dX.data_ptr(), lddx)
    return dX


def nvfp4_moe_mlp(X, gate_up, down, logits=None, top_k=None, renorm=True, ids=None, weights=None, out_dtype=torch.bfloat16, out=None):
    """A whole mixture-of-experts MLP for at most 64 tokens, X [T, d] bf16: (out [T, m], ids int32 [T, K], weights fp32 [T, K]).

    out[t] = sum_s weights[t, s] D_e (silu(G_e x_t) * (U_e x_t)), e = ids[t, s].  The experts are chosen from logits [T, E]
    (top_k, renorm) as by moe_topk, or given as ids and weights.  gate_up: (codes [E, 2h, d/2], scales [E, 2h, d/16], g [E]),
    each expert's first h rows gate, the others up; down: (codes [E, m, h/2], scales [E, m, h/16], g [E]), as
    gptq_nvfp4_quantize_batched gives them.  For more tokens: moe_topk, moe_sort, nvfp4_gemm_grouped, swiglu,
    nvfp4_gemm_grouped, moe_combine."""
    T, d, ldx = _matrix(X, "X", (_BF16,))
    dev = X.get_device()
    sizes = []
    for layer, name in ((gate_up, "gate_up"), (down, "down")):
        codes, scales, g = layer
        if not (isinstance(codes, torch.Tensor) and codes.is_cuda and codes.get_device() == dev and codes.dtype is _U8
                and codes.dim() == 3 and codes.is_contiguous()):
            _want(codes, f"{name} codes", (_U8,), (None, None, None), dev)
            raise ValueError(f"{name} codes must be contiguous")
        E, rows, kh = codes.shape
        _dense(scales, f"{name} scales", _U8, (E, rows, kh // 8), dev)
        _dense(g, f"{name} g", _F32, (E,), dev)
        sizes.append((E, rows, 2 * kh))
    (E, h2, k), (Ed, m, h) = sizes
    if k != d or Ed != E or h2 != 2 * h:
        raise ValueError(f"X [{T}, {d}], gate_up of {E} experts [{h2}, {k}] and down of {Ed} experts [{m}, {h}] do not fit together")
    if logits is not None:
        if ids is not None or weights is not None or top_k is None:
            raise ValueError("either logits and top_k, or ids and weights")
        t, e, ldl = _matrix(logits, "logits", _FLOATS, dev)
        if (t, e) != (T, E):
            raise ValueError(f"logits has shape {(t, e)}, not {(T, E)}")
        K, code = int(top_k), _CODES[logits.dtype]
        ids = X.new_empty((T, max(0, K)), dtype=_I32)
        weights = X.new_empty((T, max(0, K)), dtype=_F32)
    else:
        if ids is None or weights is None or top_k is not None:
            raise ValueError("either logits and top_k, or ids and weights")
        K, ldl, code = _table(ids, "ids", T, dev), 0, 0
        _dense(weights, "weights", _F32, (T, K), dev)
    out, ldo = _output(out, "out", X, T, m, out_dtype, dev)
    need = lib.nvfp4_moe_mlp_workspace_size(T, E, K, h)
    ws = _workspace(need, X.device) if need else None
    _call(lib.nvfp4_moe_mlp, "nvfp4_moe_mlp", dev, X.data_ptr(), NVQ_DTYPE_BF16, T, d, ldx, _addr(logits), code, E, ldl, K, bool(renorm),
          ids.data_ptr(), weights.data_ptr(), gate_up[0].data_ptr(), gate_up[1].data_ptr(), gate_up[2].data_ptr(), h,
          down[0].data_ptr(), down[1].data_ptr(), down[2].data_ptr(), m, out.data_ptr(), _CODES[out.dtype], ldo, _addr(ws), need)
    return out, ids, weights
