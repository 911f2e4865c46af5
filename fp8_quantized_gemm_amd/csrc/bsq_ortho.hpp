// What the two forms of the orthogonalisation share: the many-kernel one of bsq_ortho.hip
// and the one-workgroup one of bsq_ortho_one.hip.
#pragma once

#include "bsq_nt.hpp"

namespace bsq {

// Power of two of the FP16 forms: entries of X are at most 1.3 with the usual coefficients
// and typically 1 / sqrt(m n) at first; off-diagonal entries of the polynomials at most half
// the product of their leading coefficients.
constexpr float kS = 1024.0f;

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, halfx2{(_Float16)lo, (_Float16)hi});
}
// The same, as the bits that are stored: what is computed from them next goes by these.
// (Otherwise the compiler may round a product or an fma to FP16 in one step where it packs and
// in two where it goes on with the value, which differ next to a tie: the rest of such an
// entry was taken from its other neighbour, a whole FP16 step off.)
__device__ __forceinline__ uint32_t pack_f16x2_stored(float lo, float hi) {
  uint32_t w = pack_f16x2(lo, hi);
  asm("" : "+v"(w));
  return w;
}
__device__ __forceinline__ float f16_lo(uint32_t w) { return (float)__builtin_bit_cast(halfx2, w).x; }
__device__ __forceinline__ float f16_hi(uint32_t w) { return (float)__builtin_bit_cast(halfx2, w).y; }

// What is orthogonalised: a tensor (BF16, FP32) or the moment of an update.
enum NsInput { kNsBf16 = 0, kNsF32 = 1, kNsMoment = 2 };
struct NsSource {
  const void* x;
  float* momentum;
  const uint16_t* grad;
  float mu;
  int nesterov;
};

// What X0 is multiplied by, kS / (||u|| + eps), as frac 2^exp: for a norm and eps below
// kS / FLT_MAX the number itself is no FP32 (a zero matrix under it would become 0 times
// infinity), while each product stays below kS.  sum: of the squares.
struct NsNorm {
  float frac;
  int exp;
};
__device__ __forceinline__ NsNorm ns_norm(double sum, float eps) {
  NsNorm n;
  n.frac = (float)frexp((double)kS / (sqrt(sum) + (double)eps), &n.exp);
  return n;
}
__device__ __forceinline__ float ns_scaled(float x, const NsNorm& n) { return __builtin_ldexpf(x, n.exp) * n.frac; }

__global__ void k_ns_zero(float* p);

// Matrices that one workgroup holds (see bsq_ortho_one.hip).
bool ortho_in_one(int64_t rows, int64_t cols);
hipError_t launch_ortho_one(const OrthoArgs& o, hipStream_t s);

}  // namespace bsq
