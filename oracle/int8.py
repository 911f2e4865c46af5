"""8-bit integer quantizers and product (definitions in include/bsq.h), in NumPy.

codes = RNE(FP32(x * s_enc)), s_enc = FP32(127 * FP32(1 / amax)) of the row, scale = 1 / s_enc;
C = BF16(FP32(FP32(sum) * FP32(sa * sb)) + bias), every step one FP32 rounding."""

import numpy as np

from . import formats as F

FLT_MAX = np.float32(3.40282346638528859812e+38)


def quantize(bits):
    """(codes int8 [R, C], scales float32 [R]) of BF16 bit patterns [R, C]."""
    x = (bits.astype(np.uint32) << 16).view(np.float32)
    amax = np.abs(x).max(axis=1, initial=0.0).astype(np.float32)
    with np.errstate(divide="ignore", over="ignore"):
        enc = np.where(amax == 0, np.float32(1), np.minimum(np.float32(127) * (np.float32(1) / amax), FLT_MAX)).astype(np.float32)
    codes = np.rint((x * enc[:, None]).astype(np.float32))
    return codes.astype(np.int8), (np.float32(1) / enc).astype(np.float32)


def gemm(a, sa, b, sb, bias=None):
    """The BF16 values [M, N], as float64."""
    acc = (a.astype(np.float64) @ b.astype(np.float64).T).astype(np.float32)   # integers below 2^53: exact
    y = (acc * (sa[:, None] * sb[None, :]).astype(np.float32)).astype(np.float32)
    if bias is not None:
        y = (y + bias[None, :]).astype(np.float32)
    return F.f64_to_bf16_rne(y.astype(np.float64))
