// Runs an expert-grouped product on a chosen kernel, and tells which one the
// library chooses.  Part of the measurement library, not of the product ABI: it
// calls libbsq's own launches, so what it runs is what the product runs.
#include "bsq_internal.hpp"

// wgrad, fmt and the operands as for bs_gemm_grouped and bs_gemm_grouped_wgrad of
// include/bsq.h (wgrad: K is the rows, ldc N), whose checks the caller has made.
// kernel < 0: returns the chosen kernel (bsq::GroupedKernel) without a launch; else
// runs that one and returns 0, -1 where it does not take these operands, or the
// HIP error code of the launch.
extern "C" int bsq_grouped_on(int kernel, int wgrad, int fmt, int experts, const int32_t* offsets, int64_t M, int64_t N,
                              int64_t K, const uint8_t* a_codes, const uint8_t* a_scales, const float* a_amax,
                              const uint8_t* b_codes, const uint8_t* b_scales, const float* b_amax, int b_amax_n,
                              void* c, int64_t ldc, void* stream) {
  const bsq::Fmt f = fmt == 0 ? bsq::kNVFP4 : fmt == 1 ? bsq::kMXFP4 : bsq::kMXFP8;
  const bsq::GroupedArgs a{f, experts, offsets, M, N, K, a_codes, a_scales, a_amax,
                           b_codes, b_scales, b_amax, b_amax_n, c, ldc};
  if (kernel < 0) return bsq::grouped_kernel(a, wgrad != 0);
  const hipError_t e = bsq::launch_gemm_grouped_on(a, wgrad != 0, kernel, static_cast<hipStream_t>(stream));
  return e == hipErrorInvalidValue ? -1 : (int)e;
}
