"""Block-scaled (NVFP4 / MXFP4 / MXFP8) quantize + GEMM on MI355X, with the
per-tensor FP8 baseline (format "fp8") for comparison.

Thin Python binding over the C ABI of libbsq.so (include/bsq.h): argument
marshalling only.  PyTorch supplies device memory and the current stream;
every step of the computation runs in the HIP kernels of libbsq.so.  If the
library has not been built (python -m fp8_quantized_gemm_amd._build), every
entry point raises; there is no fallback.
"""

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbsq.so")

BSQ_OK, BSQ_EINVAL, BSQ_EUNSUPPORTED, BSQ_EHIP = 0, 1, 2, 3
FORMATS = {"nvfp4": 0, "mxfp4": 1, "mxfp8": 2, "fp8": 3}
ROUNDING = {"rne": 0, "sr": 1}
GATES = {None: 0, "channel": 1, "row": 2, "full": 3}
SCORING = {"softmax": 0, "sigmoid": 1}
ABI_SYMBOLS = ("nvfp4_quantize", "mx_quantize", "quantize_transpose", "quantize_transpose_amax",
               "fp8_quantize_transpose", "swiglu_amax", "swiglu_backward_amax",
               "master_weight_update", "nvfp4_expand", "bs_gemm", "bs_gemm_noalloc",
               "bs_gemm_nvfp4_bx", "block_norm", "block_norm_backward_workspace",
               "block_norm_backward", "moe_rows", "moe_route_workspace", "moe_route",
               "moe_route_score_bias", "moe_route_backward", "moe_gather", "moe_combine", "moe_combine_backward",
               "bs_gemm_grouped", "bs_gemm_grouped_wgrad", "int8_quantize",
               "int8_quantize_transpose_workspace", "int8_quantize_transpose", "int8_gemm",
               "int8_linear_workspace", "int8_linear", "orthogonalize_workspace", "orthogonalize",
               "muon_update", "bsq_status_string")


class BsqError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed: {msg}")
        self.status = status


_lib = None


def lib():
    """Load libbsq.so (once).  Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m fp8_quantized_gemm_amd._build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I, U64, U32, U16 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                    ctypes.c_uint64, ctypes.c_uint32, ctypes.c_uint16)
        L.nvfp4_quantize.argtypes = [P, I64, I64, I, I, U64, U32, I, U16, P, P, P, P, P]
        L.mx_quantize.argtypes = [P, I64, I64, I, I, U64, U32, P, P, P]
        L.quantize_transpose.argtypes = [P, I64, I64, I, I, I, U64, U32, I, U16,
                                         P, P, P, P, P, P, P]
        L.quantize_transpose_amax.argtypes = [P, I64, I64, I, I, U64, U32, I, U16,
                                              P, P, P, P, P, P, P]
        L.fp8_quantize_transpose.argtypes = [P, I64, I64, P, P, P, P]
        L.swiglu_amax.argtypes = [P, I64, I64, I, U16, P, P, P, P]
        L.swiglu_backward_amax.argtypes = [P, P, I64, I64, I, U16, P, P, P, P]
        L.master_weight_update.argtypes = [P, P, I64, ctypes.c_float, P, P, P]
        L.bs_gemm.argtypes = [I, I64, I64, I64, P, P, P, P, P, P, P, I64, P]
        L.bs_gemm_noalloc.argtypes = [I, I64, I64, I64, P, P, P, P, P, P, P, I64, P]
        L.nvfp4_expand.argtypes = [P, P, I64, I64, P, P]
        L.bs_gemm_nvfp4_bx.argtypes = [I64, I64, I64, P, P, P, P, P, P, I64, P]
        F = ctypes.c_float
        L.block_norm.argtypes = [P, I, P, I64, I64, P, I, P, F, P, F, P, P, P, P, P, P]
        L.block_norm_backward_workspace.argtypes = [I64, I64, P]
        L.block_norm_backward.argtypes = [P, I, P, P, P, I64, I64, P, I, P, F, P, P, P, P, P, P, P, P,
                                          P, I64, P]
        L.moe_rows.argtypes = [I64, I, I, I, P]
        L.moe_route_workspace.argtypes = [I64, I, I, P]
        L.moe_route.argtypes = [P, I, I64, I, I, P, I, I, F, I, I64, P, P, P, P, P, P, I64, P]
        L.moe_route_score_bias.argtypes = L.moe_route.argtypes
        L.moe_route_backward.argtypes = [P, I, I64, I, I, P, P, I, I, F, P, P]
        L.moe_gather.argtypes = [P, I64, I64, I, P, I64, P, P]
        L.moe_combine.argtypes = [P, I64, I64, P, P, I64, I, P, P]
        L.moe_combine_backward.argtypes = [P, P, I64, I64, I, P, P, P, I64, P, P, P]
        L.bs_gemm_grouped.argtypes = [I, I, P, I64, I64, I64, P, P, P, P, P, P, I, P, I64, P]
        L.bs_gemm_grouped_wgrad.argtypes = [I, I, P, I64, I64, I64, P, P, P, P, P, P, P, P]
        L.int8_quantize.argtypes = [P, I64, I64, P, P, P]
        L.int8_quantize_transpose_workspace.argtypes = [I64, I64, P]
        L.int8_quantize_transpose.argtypes = [P, I64, I64, P, P, P, P, P, I64, P]
        L.int8_gemm.argtypes = [I64, I64, I64, P, P, P, P, P, P, I64, P]
        L.int8_linear_workspace.argtypes = [I64, I64, P]
        L.int8_linear.argtypes = [P, I64, I64, I64, P, P, P, P, I64, P, I64, P]
        L.orthogonalize_workspace.argtypes = [I64, I64, I64, P]
        L.orthogonalize.argtypes = [P, I, I64, I64, I64, I, P, F, P, P, I64, P]
        L.muon_update.argtypes = [P, P, P, I64, I64, I64, F, F, I, F, F, I, P, F, P, P, P, I64, P]
        for fn in ABI_SYMBOLS[:-1]:
            getattr(L, fn).restype = I
        L.bsq_status_string.argtypes = [I]
        L.bsq_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(status):
    return lib().bsq_status_string(int(status)).decode()


def _check(fn, status):
    if status != BSQ_OK:
        raise BsqError(fn, status, status_string(status))


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without building a Stream object (0.1 against 2.1 us
# of the 10-20 us that a small call takes on the host).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device):
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _check_device(*tensors, out=None):
    """Every given tensor (None skipped) is a contiguous CUDA tensor on one device,
    and `out` a CUDA matrix with unit column stride (its row stride becomes ldc):
    the library dereferences the raw pointers on the GPU."""
    dev = None
    for t in tensors + ((out,) if out is not None else ()):
        if t is None:
            continue
        ok = isinstance(t, torch.Tensor) and t.is_cuda
        if t is out:
            ok = ok and t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] <= 1)
        else:
            ok = ok and t.is_contiguous()
        if not ok:
            raise ValueError("operands must be contiguous CUDA tensors (out: rows with unit stride)")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("operands must be on one device")


def _check_amax(*amaxes):
    """Each given amax is a float32 tensor of at least one element."""
    for a in amaxes:
        if a is not None and not (isinstance(a, torch.Tensor) and a.dtype == torch.float32
                                  and a.numel() >= 1):
            raise ValueError("amax arguments must be float32 tensors of at least one element")


def _check_operand(what, codes, scales, K, fmt, dim=2):
    """codes (uint8 [rows, K / elements-per-byte]) and scales (uint8 [rows, K /
    block], None for per-tensor FP8) of one K-major GEMM operand (dim 3: of stacked
    ones).  The library takes the row strides from K, so the widths must match
    exactly."""
    per_byte = 1 if fmt in ("mxfp8", "fp8") else 2
    blk = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32, "fp8": None}[fmt]
    if not (isinstance(codes, torch.Tensor) and codes.dtype == torch.uint8 and codes.dim() == dim):
        raise ValueError(f"{what} codes must be a {dim}-D uint8 tensor")
    if K < 0 or K % per_byte or codes.shape[-1] != K // per_byte:
        raise ValueError(f"{what} codes are {list(codes.shape)}; K = {K} needs rows of {K // per_byte}")
    if blk is None:
        return
    if not (isinstance(scales, torch.Tensor) and scales.dtype == torch.uint8 and scales.dim() == dim
            and scales.shape[:-1] == codes.shape[:-1] and scales.shape[-1] == K // blk):
        raise ValueError(f"{what} scales must be uint8 {list(codes.shape[:-1]) + [K // blk]}")


def _check_out(out, M, N, dtype):
    if out.dtype != dtype or tuple(out.shape) != (M, N):
        raise ValueError(f"out must be a {dtype} [{M}, {N}] tensor")


def _row_stride(out):
    """ldc of a checked out [M, N].  Rows that overlap (an expanded tensor) give a stride
    below N, which the library refuses; a single row's stride means nothing."""
    return out.stride(0) if out.shape[0] > 1 else out.shape[1]


def _check_input(x):
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype == torch.bfloat16 and x.dim() == 2):
        raise ValueError("x must be a 2-D bfloat16 CUDA tensor")
    return x.contiguous()


def _u8(shape, device):
    return torch.empty(shape, dtype=torch.uint8, device=device)


def nvfp4_quantize(x, block_rows=1, rnd="rne", seed=0, offset=0, rht=False, rht_signs=0,
                   amax=None):
    """Rowwise NVFP4 of x [R, C] -> (codes uint8 [R, C/2], scales uint8 [R, C/16], amax f32 [1])."""
    x = _check_input(x)
    _check_device(x, amax)
    _check_amax(amax)
    R, C = x.shape
    codes = _u8((R, C // 2), x.device)
    scales = _u8((R, max(C // 16, 0)), x.device)
    amax_out = torch.empty(1, dtype=torch.float32, device=x.device)
    st = lib().nvfp4_quantize(_ptr(x), R, C, int(block_rows), ROUNDING[rnd], int(seed), int(offset),
                              1 if rht else 0, int(rht_signs) & 0xFFFF, _ptr(amax),
                              _ptr(codes), _ptr(scales), _ptr(amax_out), _stream(x.device))
    _check("nvfp4_quantize", st)
    return codes, scales, amax_out


def mx_quantize(x, fmt="mxfp4", rnd="rne", seed=0, offset=0):
    """Rowwise MXFP4 / MXFP8 of x [R, C] -> (codes, scales E8M0 [R, C/32])."""
    x = _check_input(x)
    R, C = x.shape
    codes = _u8((R, C // 2 if fmt == "mxfp4" else C), x.device)
    scales = _u8((R, C // 32), x.device)
    st = lib().mx_quantize(_ptr(x), R, C, FORMATS[fmt], ROUNDING[rnd], int(seed), int(offset),
                           _ptr(codes), _ptr(scales), _stream(x.device))
    _check("mx_quantize", st)
    return codes, scales


def quantize_transpose(x, fmt="nvfp4", block_rows=1, rnd="rne", seed=0, offset=0,
                       rht_col=False, rht_signs=0, row=True, col=True):
    """Row (quantize(x)) and column (quantize(x^T)) outputs from one read of x [R, C].

    Returns a dict with row_codes, row_scales, row_amax, col_codes, col_scales,
    col_amax (entries of a skipped orientation, and amax for MX, are None)."""
    x = _check_input(x)
    R, C = x.shape
    blk = 16 if fmt == "nvfp4" else 32
    w = 1 if fmt == "mxfp8" else 2
    out = dict(row_codes=None, row_scales=None, row_amax=None,
               col_codes=None, col_scales=None, col_amax=None)
    if row:
        out["row_codes"] = _u8((R, C // w), x.device)
        out["row_scales"] = _u8((R, C // blk), x.device)
        if fmt == "nvfp4":
            out["row_amax"] = torch.empty(1, dtype=torch.float32, device=x.device)
    if col:
        out["col_codes"] = _u8((C, R // w), x.device)
        out["col_scales"] = _u8((C, R // blk), x.device)
        if fmt == "nvfp4":
            out["col_amax"] = torch.empty(1, dtype=torch.float32, device=x.device)
    st = lib().quantize_transpose(
        _ptr(x), R, C, FORMATS[fmt], int(block_rows), ROUNDING[rnd], int(seed), int(offset),
        1 if rht_col else 0, int(rht_signs) & 0xFFFF,
        _ptr(out["row_codes"]), _ptr(out["row_scales"]), _ptr(out["row_amax"]),
        _ptr(out["col_codes"]), _ptr(out["col_scales"]), _ptr(out["col_amax"]), _stream(x.device))
    _check("quantize_transpose", st)
    return out


def quantize_transpose_amax(x, amax_row, amax_col, block_rows=1, rnd="rne", seed=0, offset=0,
                            rht_col=False, rht_signs=0, row=True, col=True):
    """NVFP4 row and column outputs of x [R, C] under the given device amaxes
    (f32 [1] each; the one of a skipped side may be None).

    Returns a dict with row_codes, row_scales, col_codes, col_scales (None when skipped)."""
    x = _check_input(x)
    _check_device(x, amax_row, amax_col)
    _check_amax(amax_row, amax_col)
    R, C = x.shape
    out = dict(row_codes=None, row_scales=None, col_codes=None, col_scales=None)
    if row:
        out["row_codes"] = _u8((R, C // 2), x.device)
        out["row_scales"] = _u8((R, C // 16), x.device)
    if col:
        out["col_codes"] = _u8((C, R // 2), x.device)
        out["col_scales"] = _u8((C, R // 16), x.device)
    st = lib().quantize_transpose_amax(
        _ptr(x), R, C, int(block_rows), ROUNDING[rnd], int(seed), int(offset),
        1 if rht_col else 0, int(rht_signs) & 0xFFFF, _ptr(amax_row), _ptr(amax_col),
        _ptr(out["row_codes"]), _ptr(out["row_scales"]), _ptr(out["col_codes"]),
        _ptr(out["col_scales"]), _stream(x.device))
    _check("quantize_transpose_amax", st)
    return out


def swiglu(y_gu, rht_col=False, rht_signs=0, amax=True, out=None):
    """H [T, F] = silu(G) * U of y_gu = [G | U] [T, 2F] (bf16), with amax_row =
    max|H| and amax_col (the column RHT amax with rht_col, else max|H|).

    Returns dict(h, amax_row, amax_col); the amaxes are None with amax=False."""
    y = _check_input(y_gu)
    T, F2 = y.shape
    h = torch.empty((T, F2 // 2), dtype=torch.bfloat16, device=y.device) if out is None else out
    _check_device(y, h)
    if h.dtype != torch.bfloat16 or h.shape != (T, F2 // 2):
        raise ValueError("out must be a bfloat16 [T, F] tensor")
    ar = torch.empty(1, dtype=torch.float32, device=y.device) if amax else None
    ac = torch.empty(1, dtype=torch.float32, device=y.device) if amax else None
    st = lib().swiglu_amax(_ptr(y), T, F2 // 2, 1 if rht_col else 0, int(rht_signs) & 0xFFFF,
                           _ptr(h), _ptr(ar), _ptr(ac), _stream(y.device))
    _check("swiglu_amax", st)
    return dict(h=h, amax_row=ar, amax_col=ac)


def swiglu_backward(y_gu, d_h, rht_col=False, rht_signs=0, amax=True, out=None):
    """dY_gu [T, 2F] = [dG | dU] from y_gu = [G | U] [T, 2F] and d_h [T, F]
    (bf16), with the amaxes of dY_gu as for swiglu.

    Returns dict(d_y_gu, amax_row, amax_col)."""
    y = _check_input(y_gu)
    d = _check_input(d_h)
    T, F2 = y.shape
    if d.shape != (T, F2 // 2):
        raise ValueError("d_h must be [T, F] for y_gu [T, 2F]")
    dy = torch.empty((T, F2), dtype=torch.bfloat16, device=y.device) if out is None else out
    _check_device(y, d, dy)
    if dy.dtype != torch.bfloat16 or dy.shape != (T, F2):
        raise ValueError("out must be a bfloat16 [T, 2F] tensor")
    ar = torch.empty(1, dtype=torch.float32, device=y.device) if amax else None
    ac = torch.empty(1, dtype=torch.float32, device=y.device) if amax else None
    st = lib().swiglu_backward_amax(_ptr(y), _ptr(d), T, F2 // 2, 1 if rht_col else 0,
                                    int(rht_signs) & 0xFFFF, _ptr(dy), _ptr(ar), _ptr(ac),
                                    _stream(y.device))
    _check("swiglu_backward_amax", st)
    return dict(d_y_gu=dy, amax_row=ar, amax_col=ac)


def master_weight_update(w32, grad, lr, w_bf16=None, amax=True):
    """In place w32 <- w32 - lr * grad (FP32 master weight, BF16 gradient of the
    same shape); returns dict(w_bf16, amax) with the BF16 working copy and its
    amax (None with amax=False)."""
    if not (isinstance(w32, torch.Tensor) and w32.is_cuda and w32.dtype == torch.float32
            and w32.is_contiguous()):
        raise ValueError("w32 must be a contiguous float32 CUDA tensor (updated in place)")
    if not (isinstance(grad, torch.Tensor) and grad.is_cuda and grad.dtype == torch.bfloat16
            and grad.shape == w32.shape):
        raise ValueError("grad must be a bfloat16 CUDA tensor shaped like w32")
    g = grad.contiguous()
    wb = torch.empty(w32.shape, dtype=torch.bfloat16, device=w32.device) if w_bf16 is None else w_bf16
    _check_device(w32, g, wb)
    if wb.dtype != torch.bfloat16 or wb.numel() != w32.numel():
        raise ValueError("w_bf16 must be a bfloat16 tensor with w32's element count")
    a = torch.empty(1, dtype=torch.float32, device=w32.device) if amax else None
    st = lib().master_weight_update(_ptr(w32), _ptr(g), w32.numel(), float(lr), _ptr(wb), _ptr(a),
                                    _stream(w32.device))
    _check("master_weight_update", st)
    return dict(w_bf16=wb, amax=a)


def fp8_quantize_transpose(x, row=True, col=True):
    """Per-tensor FP8 (E4M3, s_enc = 448 / amax) of x [R, C] and of x^T.

    Returns a dict with row_codes [R, C], col_codes [C, R] (None when skipped)
    and amax (f32 [1])."""
    x = _check_input(x)
    R, C = x.shape
    rc = _u8((R, C), x.device) if row else None
    cc = _u8((C, R), x.device) if col else None
    amax = torch.empty(1, dtype=torch.float32, device=x.device)
    st = lib().fp8_quantize_transpose(_ptr(x), R, C, _ptr(rc), _ptr(cc), _ptr(amax), _stream(x.device))
    _check("fp8_quantize_transpose", st)
    return dict(row_codes=rc, col_codes=cc, amax=amax)


def bs_gemm(fmt, a_codes, a_scales, b_codes, b_scales, a_amax=None, b_amax=None, K=None, out=None):
    """C [M, N] bf16 = alpha * deq(A) . deq(B)^T with A, B K-major block-scaled operands
    (per-tensor "fp8": scales None, amaxes required)."""
    if fmt not in FORMATS:
        raise ValueError(f"unknown format {fmt!r}")
    if K is None and isinstance(a_codes, torch.Tensor) and a_codes.dim() == 2:
        K = a_codes.shape[1] * (1 if fmt in ("mxfp8", "fp8") else 2)
    K = int(K)
    _check_operand("A", a_codes, a_scales, K, fmt)
    _check_operand("B", b_codes, b_scales, K, fmt)
    if fmt in ("nvfp4", "fp8") and (a_amax is None or b_amax is None):
        raise ValueError(f"{fmt} needs both per-tensor amaxes")
    _check_amax(a_amax, b_amax)
    M, N = a_codes.shape[0], b_codes.shape[0]
    if out is not None:
        _check_out(out, M, N, torch.bfloat16)
    _check_device(a_codes, a_scales, b_codes, b_scales, a_amax, b_amax, out=out)
    dev = a_codes.device
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    ldc = out.stride(0) if out.dim() == 2 else N
    st = lib().bs_gemm(FORMATS[fmt], M, N, int(K), _ptr(a_codes), _ptr(a_scales), _ptr(a_amax),
                       _ptr(b_codes), _ptr(b_scales), _ptr(b_amax), _ptr(out), ldc, _stream(dev))
    _check("bs_gemm", st)
    return out


def bs_gemm_noalloc(fmt, a_codes, a_scales, b_codes, b_scales, a_amax, b_amax, out, K=None):
    """bs_gemm into a caller-provided `out`, through the entry point that
    allocates no device memory (its NVFP4 workspace is the library's static
    per-device array; overlapping calls on one device race)."""
    if fmt not in FORMATS:
        raise ValueError(f"unknown format {fmt!r}")
    if K is None and isinstance(a_codes, torch.Tensor) and a_codes.dim() == 2:
        K = a_codes.shape[1] * (1 if fmt in ("mxfp8", "fp8") else 2)
    K = int(K)
    _check_operand("A", a_codes, a_scales, K, fmt)
    _check_operand("B", b_codes, b_scales, K, fmt)
    if fmt in ("nvfp4", "fp8") and (a_amax is None or b_amax is None):
        raise ValueError(f"{fmt} needs both per-tensor amaxes")
    _check_amax(a_amax, b_amax)
    M, N = a_codes.shape[0], b_codes.shape[0]
    _check_out(out, M, N, torch.bfloat16)
    _check_device(a_codes, a_scales, b_codes, b_scales, a_amax, b_amax, out=out)
    ldc = out.stride(0) if out.dim() == 2 else N
    st = lib().bs_gemm_noalloc(FORMATS[fmt], M, N, K, _ptr(a_codes), _ptr(a_scales), _ptr(a_amax),
                               _ptr(b_codes), _ptr(b_scales), _ptr(b_amax), _ptr(out), ldc,
                               _stream(out.device))
    _check("bs_gemm_noalloc", st)
    return out


# Largest FP16 B operand worth pre-expanding.  Zero: since the register-
# expansion GEMM (K % 256 == 0) expands in the tile faster than the
# pre-expanded-B kernel streams FP16, no Llama MLP GEMM gains from it
# (measured in the 8B step: FPROP_down 1549 against 1345 TF/s, DGRAD_down
# 1437 against 1264).  bs_gemm_nvfp4_bx stays available for callers that keep
# an expanded weight anyway.
BX_MAX_BYTES = 0


def bx_pays(N, K):
    """Whether a GEMM should take its B operand pre-expanded (nvfp4_expand +
    bs_gemm_nvfp4_bx) rather than expand it inside every output tile: when the
    FP16 copy of B is at most BX_MAX_BYTES (see there; currently never)."""
    return N * K * 2 <= BX_MAX_BYTES and K % 128 == 0


def nvfp4_expand(codes, scales, K=None, out=None):
    """FP16 [R, K] expansion v * S * 2^-7 of NVFP4 codes [R, K/2] + scales [R, K/16]."""
    if K is None and isinstance(codes, torch.Tensor) and codes.dim() == 2:
        K = codes.shape[1] * 2
    K = int(K)
    _check_operand("expand", codes, scales, K, "nvfp4")
    R = codes.shape[0]
    if out is not None:
        _check_out(out, R, K, torch.float16)
    _check_device(codes, scales, out)
    if out is None:
        out = torch.empty((R, K), dtype=torch.float16, device=codes.device)
    st = lib().nvfp4_expand(_ptr(codes), _ptr(scales), R, int(K), _ptr(out), _stream(codes.device))
    _check("nvfp4_expand", st)
    return out


def bs_gemm_nvfp4_bx(a_codes, a_scales, a_amax, b_x, b_amax, out=None):
    """C [M, N] bf16 of NVFP4 A (codes, scales, amax) and FP16-expanded B [N, K]."""
    if not (isinstance(b_x, torch.Tensor) and b_x.dtype == torch.float16 and b_x.dim() == 2):
        raise ValueError("b_x must be a 2-D float16 tensor (nvfp4_expand of B)")
    N, K = b_x.shape
    _check_operand("A", a_codes, a_scales, K, "nvfp4")
    if a_amax is None or b_amax is None:
        raise ValueError("nvfp4 needs both per-tensor amaxes")
    _check_amax(a_amax, b_amax)
    M = a_codes.shape[0]
    if out is not None:
        _check_out(out, M, N, torch.bfloat16)
    _check_device(a_codes, a_scales, a_amax, b_x, b_amax, out=out)
    dev = a_codes.device
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    ldc = out.stride(0) if out.dim() == 2 else N
    st = lib().bs_gemm_nvfp4_bx(M, N, int(K), _ptr(a_codes), _ptr(a_scales), _ptr(a_amax), _ptr(b_x),
                                _ptr(b_amax), _ptr(out), ldc, _stream(dev))
    _check("bs_gemm_nvfp4_bx", st)
    return out


# ---------------------------------------------------------------- norms, gate and residual

def _check_stream(x, what="x"):
    """A 2-D bfloat16 or float32 CUDA tensor (a residual stream), made contiguous."""
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dim() == 2
            and x.dtype in (torch.bfloat16, torch.float32)):
        raise ValueError(f"{what} must be a 2-D bfloat16 or float32 CUDA tensor")
    return x.contiguous()


def _check_like(t, what, shape, dtype, device):
    """None, or a contiguous copy of a tensor that must have this shape, type and device."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape
            and t.device == device):
        raise ValueError(f"{what} must be a {dtype} {list(shape)} tensor on {device}")
    return t.contiguous()


def _check_gate(gate, R, C, device):
    """(kind, contiguous gate) of a block_norm gate: float32 [C] per channel, float32
    [R, 1] per row, bfloat16 [R, C] per element."""
    if gate is None:
        return 0, None
    if isinstance(gate, torch.Tensor) and gate.device == device:
        if gate.dtype == torch.float32 and tuple(gate.shape) == (C,):
            return GATES["channel"], gate.contiguous()
        if gate.dtype == torch.float32 and tuple(gate.shape) == (R, 1):
            return GATES["row"], gate.contiguous()
        if gate.dtype == torch.bfloat16 and tuple(gate.shape) == (R, C):
            return GATES["full"], gate.contiguous()
    raise ValueError(f"gate must be float32 [{C}], float32 [{R}, 1] or bfloat16 [{R}, {C}] on {device}")


def block_norm(x, o=None, w_pre=None, w_post=None, gate=None, alpha=1.0, eps=1e-6, amax=False):
    """The step between two blocks: r = alpha * x + gate * norm(o) * w_post and
    h = norm(r) * w_pre, x [R, C] bfloat16 or float32, o [R, C] bfloat16.

    o None: h = norm(x) only.  w_post None: o is not normalised.  w_pre None: no
    h.  gate: None, float32 [C] or [R, 1], or bfloat16 [R, C].  Returns dict(r (x's
    type), h (bfloat16), rstd_post, rstd_pre (float32 [R]), amax (float32 [1],
    max|h|, with amax=True)); entries that do not apply are None."""
    x = _check_stream(x)
    (R, C), dev = x.shape, x.device
    o = _check_like(o, "o", (R, C), torch.bfloat16, dev)
    w_pre = _check_like(w_pre, "w_pre", (C,), torch.float32, dev)
    w_post = _check_like(w_post, "w_post", (C,), torch.float32, dev)
    kind, gate = _check_gate(gate, R, C, dev)
    r = torch.empty_like(x) if o is not None else None
    h = torch.empty(R, C, dtype=torch.bfloat16, device=dev) if w_pre is not None else None
    f32 = lambda n: torch.empty(n, dtype=torch.float32, device=dev)
    if w_post is not None and w_pre is not None and amax:
        rq, rp, am = f32(2 * R + 1).split_with_sizes((R, R, 1))    # one allocation: 1 us less
    else:
        rq = f32(R) if w_post is not None else None
        rp = f32(R) if w_pre is not None else None
        am = f32(1) if amax and w_pre is not None else None
    st = lib().block_norm(_ptr(x), int(x.dtype == torch.float32), _ptr(o), R, C, _ptr(w_post), kind,
                          _ptr(gate), float(alpha), _ptr(w_pre), float(eps), _ptr(r), _ptr(h), _ptr(rq),
                          _ptr(rp), _ptr(am), _stream(dev))
    _check("block_norm", st)
    return dict(r=r, h=h, rstd_post=rq, rstd_pre=rp, amax=am)


def block_norm_backward(r, o=None, d_r=None, d_h=None, w_pre=None, w_post=None, gate=None,
                        rstd_pre=None, rstd_post=None, alpha=1.0):
    """Gradient of block_norm from d_r [R, C] (r's type, or None) and d_h [R, C]
    (bfloat16; with w_pre), given the forward's r (its x when there was no o), o
    and rstd.

    Returns dict(d_x (r's type), d_o (bfloat16), d_gate (the gate's shape and
    type), d_w_pre, d_w_post (float32 [C])); entries that do not apply are None."""
    r = _check_stream(r, "r")
    (R, C), dev = r.shape, r.device
    o = _check_like(o, "o", (R, C), torch.bfloat16, dev)
    d_r = _check_like(d_r, "d_r", (R, C), r.dtype, dev)
    d_h = _check_like(d_h, "d_h", (R, C), torch.bfloat16, dev)
    w_pre = _check_like(w_pre, "w_pre", (C,), torch.float32, dev)
    w_post = _check_like(w_post, "w_post", (C,), torch.float32, dev)
    rstd_pre = _check_like(rstd_pre, "rstd_pre", (R,), torch.float32, dev)
    rstd_post = _check_like(rstd_post, "rstd_post", (R,), torch.float32, dev)
    kind, gate = _check_gate(gate, R, C, dev)
    need = _size("block_norm_backward_workspace", R, C)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    d_x = torch.empty_like(r)
    d_o = torch.empty_like(o) if o is not None else None
    d_g = torch.empty_like(gate) if gate is not None else None
    d_wp = torch.empty_like(w_pre) if w_pre is not None else None
    d_wq = torch.empty_like(w_post) if w_post is not None else None
    st = lib().block_norm_backward(_ptr(r), int(r.dtype == torch.float32), _ptr(o), _ptr(d_r), _ptr(d_h),
                                   R, C, _ptr(w_post), kind, _ptr(gate), float(alpha), _ptr(w_pre),
                                   _ptr(rstd_post), _ptr(rstd_pre), _ptr(d_x), _ptr(d_o), _ptr(d_g),
                                   _ptr(d_wp), _ptr(d_wq), _ptr(ws), need, _stream(dev))
    _check("block_norm_backward", st)
    return dict(d_x=d_x, d_o=d_o, d_gate=d_g, d_w_pre=d_wp, d_w_post=d_wq)


# ---------------------------------------------------------------- expert routing

def _scoring(name):
    if name not in SCORING:
        raise ValueError(f"unknown scoring {name!r}")
    return SCORING[name]


@functools.lru_cache(maxsize=1024)
def _size(fn, *args):
    """The int64 a size query of the library returns for these sizes."""
    n = ctypes.c_int64(0)
    _check(fn, getattr(lib(), fn)(*args, ctypes.byref(n)))
    return n.value


def moe_rows(tokens, experts, k, align=1):
    """Rows of the expert-ordered buffers of moe_route for these sizes."""
    return _size("moe_rows", int(tokens), int(experts), int(k), int(align))


def moe_route(logits, k, bias=None, scoring="softmax", normalize=True, scale=1.0, align=1, score_bias=None):
    """Top-k routing of logits [T, E] (bfloat16 or float32; -inf masks an expert).

    bias, score_bias (float32 [E], one of them): steer the selection and not the
    weights, which goes by logit + bias or by score + score_bias, the score being
    sigmoid(logit) or softmax(logits).  The correction bias of a router balanced
    without an auxiliary loss is a score_bias.

    Returns dict(experts int32 [T, k] (-1: no candidate left), weights float32 [T,
    k], offsets int32 [E + 1] (rows of each expert's padded group), row_of int32
    [T, k] (row of the assignment, -1: none), src int32 [moe_rows] (token * k +
    slot of the row, -1: padding))."""
    logits = _check_stream(logits, "logits")
    (T, E), dev, k = logits.shape, logits.device, int(k)
    if bias is not None and score_bias is not None:
        raise ValueError("bias is added to the logits, score_bias to the scores: give one of them")
    scored = score_bias is not None
    bias = _check_like(score_bias if scored else bias, "score_bias" if scored else "bias", (E,), torch.float32, dev)
    sc, rows = _scoring(scoring), moe_rows(T, E, k, align)
    need = _size("moe_route_workspace", T, E, k)
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device=dev)
    ids, row_of, off, src = i32(2 * T * k + E + 1 + rows).split_with_sizes((T * k, T * k, E + 1, rows))
    ids, row_of = ids.view(T, k), row_of.view(T, k)
    w = torch.empty(T, k, dtype=torch.float32, device=dev)
    ws = i32(need // 4) if need else None
    fn = "moe_route_score_bias" if scored else "moe_route"
    st = getattr(lib(), fn)(_ptr(logits), int(logits.dtype == torch.float32), T, E, k, _ptr(bias), sc,
                            1 if normalize else 0, float(scale), int(align), rows, _ptr(ids), _ptr(w), _ptr(off),
                            _ptr(row_of), _ptr(src), _ptr(ws), need, _stream(dev))
    _check(fn, st)
    return dict(experts=ids, weights=w, offsets=off, row_of=row_of, src=src)


def moe_route_backward(logits, experts, d_weights, scoring="softmax", normalize=True, scale=1.0):
    """d_logits [T, E] (logits' type) from d_weights [T, k] and moe_route's experts."""
    logits = _check_stream(logits, "logits")
    (T, E), dev = logits.shape, logits.device
    if not (isinstance(experts, torch.Tensor) and experts.dim() == 2):
        raise ValueError("experts must be moe_route's int32 [T, k] tensor")
    k = experts.shape[1]
    experts = _check_like(experts, "experts", (T, k), torch.int32, dev)
    if d_weights is None:
        raise ValueError("d_weights is required")
    d_weights = _check_like(d_weights, "d_weights", (T, k), torch.float32, dev)
    d = torch.empty_like(logits)
    st = lib().moe_route_backward(_ptr(logits), int(logits.dtype == torch.float32), T, E, k, _ptr(experts),
                                  _ptr(d_weights), _scoring(scoring), 1 if normalize else 0, float(scale),
                                  _ptr(d), _stream(dev))
    _check("moe_route_backward", st)
    return d


def _check_index(t, what, dim, device):
    if not (isinstance(t, torch.Tensor) and t.dtype == torch.int32 and t.dim() == dim and t.device == device):
        raise ValueError(f"{what} must be a {dim}-D int32 tensor on {device}")
    return t.contiguous()


def moe_gather(x, src, k, out=None):
    """Token rows x [T, C] (bfloat16) in expert order [rows, C]: row p is token src[p]
    // k, zeros where src[p] < 0."""
    x = _check_input(x)
    T, C = x.shape
    src = _check_index(src, "src", 1, x.device)
    if out is None:
        out = torch.empty(src.shape[0], C, dtype=torch.bfloat16, device=x.device)
    else:
        _check_out(out, src.shape[0], C, torch.bfloat16)
    _check_device(x, src, out)
    _check("moe_gather", lib().moe_gather(_ptr(x), T, C, int(k), _ptr(src), src.shape[0], _ptr(out),
                                          _stream(x.device)))
    return out


def moe_combine(y, row_of, weights=None, out=None):
    """[T, C] bfloat16: sum over the slots of weights [T, k] (None: 1) times the rows
    row_of [T, k] of y [rows, C]."""
    y = _check_input(y)
    R, C = y.shape
    row_of = _check_index(row_of, "row_of", 2, y.device)
    T, k = row_of.shape
    weights = _check_like(weights, "weights", (T, k), torch.float32, y.device)
    if out is None:
        out = torch.empty(T, C, dtype=torch.bfloat16, device=y.device)
    else:
        _check_out(out, T, C, torch.bfloat16)
    _check_device(y, row_of, out)
    _check("moe_combine", lib().moe_combine(_ptr(y), R, C, _ptr(row_of), _ptr(weights), T, k, _ptr(out),
                                            _stream(y.device)))
    return out


def moe_combine_backward(d_out, y, src, row_of, weights):
    """(d_y [rows, C] bfloat16, d_weights float32 [T, k]) of moe_combine from d_out [T, C]."""
    d_out, y = _check_input(d_out), _check_input(y)
    (R, C), dev = y.shape, y.device
    row_of = _check_index(row_of, "row_of", 2, dev)
    T, k = row_of.shape
    d_out = _check_like(d_out, "d_out", (T, C), torch.bfloat16, dev)
    src = _check_index(src, "src", 1, dev)
    if src.shape[0] != R:
        raise ValueError(f"src must have y's {R} rows")
    if weights is None:
        raise ValueError("weights are required")
    weights = _check_like(weights, "weights", (T, k), torch.float32, dev)
    d_y = torch.empty_like(y)
    d_w = torch.empty_like(weights)
    _check("moe_combine_backward",
           lib().moe_combine_backward(_ptr(d_out), _ptr(y), T, C, k, _ptr(src), _ptr(row_of), _ptr(weights), R,
                                      _ptr(d_y), _ptr(d_w), _stream(dev)))
    return d_y, d_w


# ---------------------------------------------------------------- expert-grouped products

GROUPED_FORMATS = ("nvfp4", "mxfp4", "mxfp8")


def _check_offsets(offsets):
    if not (isinstance(offsets, torch.Tensor) and offsets.dtype == torch.int32 and offsets.dim() == 1
            and offsets.numel() >= 2):
        raise ValueError("offsets must be a 1-D int32 tensor of experts + 1 elements")
    return offsets.numel() - 1


def bs_gemm_grouped(fmt, a_codes, a_scales, b_codes, b_scales, offsets, a_amax=None, b_amax=None, out=None):
    """C [R, N] bf16: rows offsets[e] .. offsets[e + 1] - 1 of A [R, K] times B[e] [N, K]
    transposed, zeros in the rows of no group.  b_codes [E, N, K / per
    byte], b_scales [E, N, K / block]; nvfp4: a_amax [1], b_amax [1] or [E]."""
    if fmt not in GROUPED_FORMATS:
        raise ValueError(f"unknown grouped format {fmt!r}")
    E = _check_offsets(offsets)
    if not (isinstance(b_codes, torch.Tensor) and b_codes.dim() == 3 and b_codes.shape[0] == E
            and isinstance(b_scales, torch.Tensor) and b_scales.dim() == 3 and b_scales.shape[0] == E
            and isinstance(a_codes, torch.Tensor) and a_codes.dim() == 2):
        raise ValueError(f"A must be [rows, K], B [{E}, N, K] codes and scales")
    _check_device(a_codes, a_scales, b_codes, b_scales, offsets, a_amax, b_amax, out=out)
    K = a_codes.shape[1] * (1 if fmt == "mxfp8" else 2)
    _check_operand("A", a_codes, a_scales, K, fmt)
    _check_operand("B", b_codes, b_scales, K, fmt, 3)
    if fmt == "nvfp4" and (a_amax is None or b_amax is None):
        raise ValueError("nvfp4 needs both per-tensor amaxes")
    _check_amax(a_amax, b_amax)
    bn = 1
    if b_amax is not None and fmt == "nvfp4":
        bn = b_amax.numel()
        if bn not in (1, E):
            raise ValueError(f"b_amax must have 1 or {E} elements")
    M, N = a_codes.shape[0], b_codes.shape[1]
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=a_codes.device)
    else:
        _check_out(out, M, N, torch.bfloat16)
    st = lib().bs_gemm_grouped(FORMATS[fmt], E, _ptr(offsets), M, N, K, _ptr(a_codes), _ptr(a_scales),
                               _ptr(a_amax), _ptr(b_codes), _ptr(b_scales), _ptr(b_amax), bn, _ptr(out),
                               _row_stride(out), _stream(out.device))
    _check("bs_gemm_grouped", st)
    return out


def bs_gemm_grouped_wgrad(fmt, a_codes, a_scales, b_codes, b_scales, offsets, a_amax=None, b_amax=None,
                          out=None):
    """C [E, M, N] bf16: A [M, R] times B [N, R] transposed over the rows of each group
    (codes quantized along the rows, R the expert-ordered rows; offsets multiples
    of the format's scale block)."""
    if fmt not in GROUPED_FORMATS:
        raise ValueError(f"unknown grouped format {fmt!r}")
    E = _check_offsets(offsets)
    if not (isinstance(a_codes, torch.Tensor) and a_codes.dim() == 2
            and isinstance(b_codes, torch.Tensor) and b_codes.dim() == 2):
        raise ValueError("A must be [M, rows], B [N, rows]")
    _check_device(a_codes, a_scales, b_codes, b_scales, offsets, a_amax, b_amax)
    R = a_codes.shape[1] * (1 if fmt == "mxfp8" else 2)
    _check_operand("A", a_codes, a_scales, R, fmt)
    _check_operand("B", b_codes, b_scales, R, fmt)
    if fmt == "nvfp4" and (a_amax is None or b_amax is None):
        raise ValueError("nvfp4 needs both per-tensor amaxes")
    _check_amax(a_amax, b_amax)
    M, N = a_codes.shape[0], b_codes.shape[0]
    if out is None:
        out = torch.empty(E, M, N, dtype=torch.bfloat16, device=a_codes.device)
    elif not (out.dtype == torch.bfloat16 and tuple(out.shape) == (E, M, N)):
        raise ValueError(f"out must be a bfloat16 [{E}, {M}, {N}] tensor")
    _check_device(a_codes, out)
    st = lib().bs_gemm_grouped_wgrad(FORMATS[fmt], E, _ptr(offsets), M, N, R, _ptr(a_codes), _ptr(a_scales),
                                     _ptr(a_amax), _ptr(b_codes), _ptr(b_scales), _ptr(b_amax), _ptr(out),
                                     _stream(out.device))
    _check("bs_gemm_grouped_wgrad", st)
    return out


def _on_device(method):
    """A layer's method with the layer's device (self.dev) current: its calls ask for the
    current device's compute units and set their kernels' LDS there."""
    @functools.wraps(method)
    def run(self, *args, **kwargs):
        if self.dev.index is None or self.dev.index == torch.cuda.current_device():
            return method(self, *args, **kwargs)
        with torch.cuda.device(self.dev):
            return method(self, *args, **kwargs)
    return run


# ---------------------------------------------------------------- 8-bit integers

def _call(fn, dev, *args):
    """The entry point on dev's current stream, with dev current: the library asks for
    the current device's compute units and sets its kernels' LDS there."""
    if dev.index is None or dev.index == torch.cuda.current_device():
        return _check(fn, getattr(lib(), fn)(*args, _stream(dev)))
    with torch.cuda.device(dev):
        return _check(fn, getattr(lib(), fn)(*args, _stream(dev)))


def int8_quantize(x):
    """Codes of the rows of x [R, C] (bfloat16) -> (codes int8 [R, C], scales float32 [R])."""
    x = _check_input(x)
    R, C = x.shape
    codes = torch.empty(R, C, dtype=torch.int8, device=x.device)
    scales = torch.empty(R, dtype=torch.float32, device=x.device)
    _call("int8_quantize", x.device, _ptr(x), R, C, _ptr(codes), _ptr(scales))
    return codes, scales


def int8_quantize_transpose(x, row=True, col=True):
    """int8_quantize of x [R, C] and of x^T.

    Returns dict(row_codes int8 [R, C], row_scales float32 [R], col_codes int8 [C, R],
    col_scales float32 [C]); the entries of a skipped orientation are None."""
    x = _check_input(x)
    if not (row or col):
        raise ValueError("nothing to compute: row and col are both false")
    (R, C), dev = x.shape, x.device
    i8 = lambda on, *s: torch.empty(s, dtype=torch.int8, device=dev) if on else None
    f32 = lambda on, n: torch.empty(n, dtype=torch.float32, device=dev) if on else None
    out = dict(row_codes=i8(row, R, C), row_scales=f32(row, R), col_codes=i8(col, C, R), col_scales=f32(col, C))
    need = _size("int8_quantize_transpose_workspace", R, C)
    ws = _u8(need, dev)
    _call("int8_quantize_transpose", dev, _ptr(x), R, C, _ptr(out["row_codes"]), _ptr(out["row_scales"]),
          _ptr(out["col_codes"]), _ptr(out["col_scales"]), _ptr(ws), need)
    return out


def _check_int8(what, codes, scales, K):
    """(rows) of one int8 operand: codes [rows, K] and scales float32 [rows]."""
    if not (isinstance(codes, torch.Tensor) and codes.dtype == torch.int8 and codes.dim() == 2 and codes.shape[1] == K):
        raise ValueError(f"{what} codes must be an int8 [rows, {K}] tensor")
    if not (isinstance(scales, torch.Tensor) and scales.dtype == torch.float32 and scales.dim() == 1
            and scales.shape[0] == codes.shape[0]):
        raise ValueError(f"{what} scales must be a float32 [{codes.shape[0]}] tensor")
    return codes.shape[0]


def _check_bias(bias, N):
    if bias is not None and not (isinstance(bias, torch.Tensor) and bias.dtype == torch.float32
                                 and tuple(bias.shape) == (N,)):
        raise ValueError(f"bias must be a float32 [{N}] tensor")


def int8_gemm(a_codes, a_scales, b_codes, b_scales, bias=None, out=None):
    """C [M, N] bfloat16 = (A . B^T) * a_scales[:, None] * b_scales + bias of int8 A [M, K]
    and B [N, K] with float32 scales [M] and [N]; bias float32 [N] or None."""
    if not (isinstance(a_codes, torch.Tensor) and a_codes.dim() == 2):
        raise ValueError("A codes must be an int8 [rows, K] tensor")
    K = a_codes.shape[1]
    M, N = _check_int8("A", a_codes, a_scales, K), _check_int8("B", b_codes, b_scales, K)
    _check_bias(bias, N)
    if out is not None:
        _check_out(out, M, N, torch.bfloat16)
    _check_device(a_codes, a_scales, b_codes, b_scales, bias, out=out)
    dev = a_codes.device
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    _call("int8_gemm", dev, M, N, K, _ptr(a_codes), _ptr(a_scales), _ptr(b_codes), _ptr(b_scales), _ptr(bias), _ptr(out),
          _row_stride(out))
    return out


def int8_linear(x, w_codes, w_scales, bias=None, out=None):
    """x [M, K] (bfloat16) quantized by rows, times int8 weights w_codes [N, K] with
    scales [N]: [M, N] bfloat16 (int8_quantize and int8_gemm in one call)."""
    x = _check_input(x)
    M, K = x.shape
    N = _check_int8("weight", w_codes, w_scales, K)
    _check_bias(bias, N)
    if out is not None:
        _check_out(out, M, N, torch.bfloat16)
    _check_device(x, w_codes, w_scales, bias, out=out)
    dev = x.device
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    need = _size("int8_linear_workspace", M, K)
    ws = _u8(need, dev)
    _call("int8_linear", dev, _ptr(x), M, N, K, _ptr(w_codes), _ptr(w_scales), _ptr(bias), _ptr(out),
          _row_stride(out), _ptr(ws), need)
    return out


# ---------------------------------------------------------------- orthogonalised updates

NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)


@functools.lru_cache(maxsize=64)
def _coefs(steps, coefs):
    """(steps, host array of 3 * steps floats) of one triple for every step or one each."""
    try:
        one = [tuple(float(v) for v in c) for c in (coefs if isinstance(coefs[0], tuple) else (coefs,) * steps)]
    except (TypeError, ValueError, IndexError):
        one = []
    if steps < 1 or len(one) != steps or any(len(c) != 3 for c in one):
        raise ValueError(f"coefs must be one triple (a, b, c), or one for each of the {steps} steps")
    return (ctypes.c_float * (3 * steps))(*[v for c in one for v in c])


def _coef_key(coefs):
    """coefs as a triple, or triples, of floats: what _coefs remembers goes by values (a
    tensor's elements, or an array's rows, would be remembered by what they are, and a
    tensor changed in place taken for what it was).  None where they are no numbers."""
    def floats(row):
        row = tuple(row)
        if any(getattr(v, "ndim", 0) for v in row):
            raise ValueError("rows of rows")
        return tuple(float(v) for v in row)

    try:
        c = tuple(coefs)
        nested = c and (isinstance(c[0], (tuple, list)) or getattr(c[0], "ndim", 0))
        return tuple(floats(row) for row in c) if nested else floats(c)
    except (TypeError, ValueError):
        return None


def _check_stack(x, what, dtypes, shape=None):
    """(batch, rows, cols) of a contiguous matrix or stack of matrices."""
    names = " or ".join(str(d) for d in dtypes)
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dim() in (2, 3) and x.dtype in dtypes and x.is_contiguous()
            and (shape is None or x.shape == shape)):
        want = f" {list(shape)}" if shape is not None else " 2-D or 3-D"
        raise ValueError(f"{what} must be a contiguous{want} {names} CUDA tensor")
    return (x.shape if x.dim() == 3 else (1, *x.shape))


def orthogonalize(x, steps=5, coefs=NEWTON_SCHULZ, eps=1e-7, out=None):
    """The matrix x [R, C], or each of a stack [E, R, C] (bfloat16 or float32), moved
    towards the nearest orthogonal one by `steps` Newton-Schulz steps, bfloat16.

    coefs: (a, b, c) of X <- (a I + b A + c A^2) X with A = X X^T, or one triple for
    each step."""
    if isinstance(x, torch.Tensor) and x.is_cuda:
        x = x.contiguous()
    B, R, C = _check_stack(x, "x", (torch.bfloat16, torch.float32))
    host = _coefs(int(steps), _coef_key(coefs))
    dev = x.device
    if out is None:
        out = torch.empty(x.shape, dtype=torch.bfloat16, device=dev)
    else:
        _check_stack(out, "out", (torch.bfloat16,), x.shape)
    _check_device(x, out)
    need = _size("orthogonalize_workspace", B, R, C)
    ws = _u8(need, dev)
    _call("orthogonalize", dev, _ptr(x), int(x.dtype == torch.float32), B, R, C, int(steps), host, float(eps),
          _ptr(out), _ptr(ws), need)
    return out


def muon_update(w32, momentum, grad, lr, mu=0.95, nesterov=True, weight_decay=0.0, scale=None, steps=5,
                coefs=NEWTON_SCHULZ, eps=1e-7, w_bf16=None, amax=True):
    """In place momentum <- mu * momentum + grad and w32 <- (1 - lr * weight_decay) * w32
    - lr * scale * orthogonalize(u), u = grad + mu * momentum (nesterov) or momentum.

    w32, momentum float32 and grad bfloat16, [R, C] or a stack [E, R, C]; scale None:
    0.2 * sqrt(max(R, C)), which gives the update of a weight a root mean square of
    about 0.2.  Returns dict(w_bf16, amax) as master_weight_update does."""
    B, R, C = _check_stack(w32, "w32", (torch.float32,))
    _check_stack(momentum, "momentum", (torch.float32,), w32.shape)
    if not (isinstance(grad, torch.Tensor) and grad.is_cuda and grad.dtype == torch.bfloat16
            and grad.shape == w32.shape):
        raise ValueError("grad must be a bfloat16 CUDA tensor shaped like w32")
    g = grad.contiguous()
    host = _coefs(int(steps), _coef_key(coefs))
    dev = w32.device
    wb = torch.empty(w32.shape, dtype=torch.bfloat16, device=dev) if w_bf16 is None else w_bf16
    _check_stack(wb, "w_bf16", (torch.bfloat16,), w32.shape)
    _check_device(w32, momentum, g, wb)
    a = torch.empty(1, dtype=torch.float32, device=dev) if amax else None
    if scale is None:
        scale = 0.2 * max(R, C) ** 0.5
    need = _size("orthogonalize_workspace", B, R, C)
    ws = _u8(need, dev)
    _call("muon_update", dev, _ptr(w32), _ptr(momentum), _ptr(g), B, R, C, float(lr), float(mu), 1 if nesterov else 0,
          float(weight_decay), float(scale), int(steps), host, float(eps), _ptr(wb), _ptr(a), _ptr(ws), need)
    return dict(w_bf16=wb, amax=a)
