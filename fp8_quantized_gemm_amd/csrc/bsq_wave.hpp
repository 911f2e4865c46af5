// Wave-level sums and maxima and BF16 / FP32 row pieces shared by the norm and
// the expert-routing kernels (gfx950, 64 lanes).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bsq_device.hpp"

namespace bsq {

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t dpp_or0(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROW_MASK, 0xF, false);
}

// Sum over the 64 lanes, the same value in every lane, in a fixed order: quad
// pairs, quads, half rows and rows of 16 in place, then the rows' totals
// carried into lane 63.
__device__ __forceinline__ float wave_sum(float v) {
  v += u2f(dpp_or0<0xB1, 0xF>(f2u(v)));    // lane ^ 1
  v += u2f(dpp_or0<0x4E, 0xF>(f2u(v)));    // lane ^ 2
  v += u2f(dpp_or0<0x141, 0xF>(f2u(v)));   // mirror of 8 lanes
  v += u2f(dpp_or0<0x140, 0xF>(f2u(v)));   // mirror of 16 lanes
  v += u2f(dpp_or0<0x142, 0xA>(f2u(v)));   // row 0 -> 1, 2 -> 3
  v += u2f(dpp_or0<0x143, 0xC>(f2u(v)));   // row 1 -> 2, 3
  return u2f((uint32_t)__builtin_amdgcn_readlane((int)f2u(v), 63));
}

// Unsigned maximum over the 64 lanes, in every lane.
__device__ __forceinline__ uint32_t wave_max_dpp(uint32_t v) {
  v = max(v, dpp_or0<0xB1, 0xF>(v));
  v = max(v, dpp_or0<0x4E, 0xF>(v));
  v = max(v, dpp_or0<0x141, 0xF>(v));
  v = max(v, dpp_or0<0x140, 0xF>(v));
  v = max(v, dpp_or0<0x142, 0xA>(v));
  v = max(v, dpp_or0<0x143, 0xC>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Unsigned key with the order of the floats (NaN excluded by the caller): a
// key of 0 is below every float's.
__device__ __forceinline__ uint32_t float_key(float f) {
  const uint32_t b = f2u(f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float float_of_key(uint32_t k) {
  return u2f((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

__device__ __forceinline__ uint16_t bf16_rne(float v) { return (uint16_t)pack_bf16x2(v, 0.0f); }

// Eight BF16 values of a 16-byte piece <-> FP32.
__device__ __forceinline__ void bf16x8_to_f32(const uint4& v, float* y) {
  y[0] = bf16_lo(v.x); y[1] = bf16_hi(v.x);
  y[2] = bf16_lo(v.y); y[3] = bf16_hi(v.y);
  y[4] = bf16_lo(v.z); y[5] = bf16_hi(v.z);
  y[6] = bf16_lo(v.w); y[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 f32_to_bf16x8(const float* y) {
  return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                    pack_bf16x2(y[6], y[7]));
}

}  // namespace bsq
