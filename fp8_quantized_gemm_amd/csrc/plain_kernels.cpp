// Runs an 8-bit integer product or an orthogonalisation on a chosen kernel.  Part of
// the measurement library, not of the product ABI: it calls libbsq's own launches, so
// what it runs is what the product runs.
#include "bsq_internal.hpp"

static int code(hipError_t e) { return e == hipErrorInvalidValue ? -1 : (int)e; }

// Operands as for int8_gemm of include/bsq.h, whose checks the caller has made.
// kernel < 0: returns the chosen kernel (bsq::NtKernel) without a launch; else runs
// that one (rest >= 0: its tiles from number `count` on cut for the kernel `rest`) and
// returns 0, -1 where it does not take these operands, or the HIP error.
extern "C" int bsq_int8_on(int kernel, int rest, int count, int64_t M, int64_t N, int64_t K, const uint8_t* a_codes, const float* a_scales,
                           const uint8_t* b_codes, const float* b_scales, const float* bias, void* c, int64_t ldc,
                           void* stream) {
  const bsq::Int8Args a{M, N, K, a_codes, a_scales, b_codes, b_scales, bias, c, ldc};
  if (kernel < 0) return bsq::i8_kernel(a);
  return code(bsq::launch_i8_gemm(a, static_cast<hipStream_t>(stream), kernel, rest, count));
}

// orthogonalize with every product on `kernel` (rest >= 0: half of its tiles on `rest`).
extern "C" int bsq_ortho_on(int kernel, int rest, const void* x, int f32, int64_t batch, int64_t rows, int64_t cols, int steps,
                            const float* coefs, float eps, void* out, void* workspace, void* stream) {
  bsq::OrthoArgs a{};
  a.batch = batch, a.rows = rows, a.cols = cols, a.steps = steps, a.coefs = coefs, a.eps = eps;
  a.workspace = workspace, a.x = x, a.f32 = f32 != 0, a.out = out, a.kernel = kernel, a.rest = rest;
  return code(bsq::launch_ortho(a, static_cast<hipStream_t>(stream)));
}
