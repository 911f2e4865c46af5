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

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 16 bytes at an address of 2, 4 or 16-byte alignment.
template <int A>
struct Piece;
template <>
struct Piece<2> { typedef u32x4 type __attribute__((aligned(2))); };
template <>
struct Piece<4> { typedef u32x4 type __attribute__((aligned(4))); };
template <>
struct Piece<16> { typedef u32x4 type; };

// 8 columns of a row as stored: 16 bytes of BF16, 32 of FP32.
template <typename T>
struct Raw {
  u32x4 v[sizeof(T) / 2];
};

// Piece at column col of a row of cols columns, zeros past its end, once
// end_piece has been applied where the piece is used first.  AL: rows are 16-byte
// aligned and cols % 8 == 0; else any element alignment: one unaligned 16-byte
// access per piece, the row's last one shifted back to end with the row, and
// end_piece moves its elements into place.  (Single elements there, loaded in
// turn by one lane, kept the whole row waiting: block_norm on 16,000 x 4,095,
// BF16: 173 against 125 us forward, 350 against 207 us backward.)
template <bool AL, typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* row, int col, int cols) {
  Raw<T> r;
  if (AL || cols < 8) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = u32x4{0u, 0u, 0u, 0u};
  }
  if (AL) {
    if (col < cols) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = reinterpret_cast<const u32x4*>(row + col)[i];
    }
  } else if (cols >= 8) {
    typedef typename Piece<(int)sizeof(T)>::type U;
    const int at = col < cols - 8 ? col : cols - 8;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = reinterpret_cast<const U*>(row + at)[i];
  } else {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (col + j < cols) {
        if constexpr (sizeof(T) == 2) r.v[0][j >> 1] |= (uint32_t)row[col + j] << (16 * (j & 1));
        else r.v[j >> 2][j & 3] = f2u(row[col + j]);
      }
  }
  return r;
}
template <bool AL, typename T>
__device__ __forceinline__ void end_piece(Raw<T>& r, int col, int cols) {
  if (AL || cols < 8 || col <= cols - 8) return;
  const int s = col - (cols - 8);                        // elements of the row before: 1-7, more past the end
  constexpr int D = 2 * sizeof(T);                       // dwords
  uint32_t d[D];
#pragma unroll
  for (int i = 0; i < D; ++i) d[i] = s < 8 ? r.v[i >> 2][i & 3] : 0u;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < D; ++i) d[i] = s & 1 ? __builtin_amdgcn_alignbyte(i + 1 < D ? d[i + 1] : 0u, d[i], 2) : d[i];
  }
#pragma unroll
  for (int b = 1; b < D; b *= 2) {
    const bool on = s & (b * 4 / (int)sizeof(T));
#pragma unroll
    for (int i = 0; i < D; ++i) d[i] = on ? (i + b < D ? d[i + b] : 0u) : d[i];
  }
#pragma unroll
  for (int i = 0; i < D; ++i) r.v[i >> 2][i & 3] = d[i];
}
template <typename T>
__device__ __forceinline__ float raw_at(const Raw<T>& r, int j) {
  if constexpr (sizeof(T) == 2) return (j & 1) ? bf16_hi(r.v[0][j >> 1]) : bf16_lo(r.v[0][j >> 1]);
  else return u2f(r.v[j >> 2][j & 3]);
}
// Makes the compiler forget what it unpacked from r: a piece is unpacked again
// where it is used next, instead of being held as 8 FP32 registers meanwhile.
template <typename T>
__device__ __forceinline__ void forget(Raw<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) asm volatile("" : "+v"(r.v[i]));
}
template <bool AL, typename T>
__device__ __forceinline__ void store_raw(T* row, int col, int cols, const Raw<T>& r) {
  if (AL ? col < cols : col + 8 <= cols) {
    typedef typename Piece<AL ? 16 : (int)sizeof(T)>::type U;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<U*>(row + col)[i] = r.v[i];
  } else if (!AL && col < cols) {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (col + j < cols) {
        if constexpr (sizeof(T) == 2) row[col + j] = (uint16_t)(r.v[0][j >> 1] >> (16 * (j & 1)));
        else row[col + j] = u2f(r.v[j >> 2][j & 3]);
      }
  }
}
// Eight FP32 values rounded to the row's type and stored.
template <bool AL, typename T>
__device__ __forceinline__ void store8(T* row, int col, int cols, const float (&y)[8]) {
  Raw<T> r;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[0][j] = pack_bf16x2(y[2 * j], y[2 * j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.v[j >> 2][j & 3] = f2u(y[j]);
  }
  store_raw<AL>(row, col, cols, r);
}

}  // namespace bsq
