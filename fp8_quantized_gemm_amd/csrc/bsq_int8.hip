// 8-bit integer quantizers and products for gfx950 (contract in include/bsq.h):
//   codes = RNE(x s_enc), s_enc = 127 (1 / amax) of the row (or column)
//   C = BF16(FP32(A . B^T) (sa sb) + bias)
#include "bsq_device.hpp"
#include "bsq_nt.hpp"
#include "bsq_nt_ring.hpp"
#include "bsq_wave.hpp"

namespace bsq {

namespace {

// ---------------------------------------------------------------- encode

// (A reciprocal and a product, as tensor programs compute 127.0 / amax, so that their codes
// are met bit for bit; at most 1.5 2^-24 from the quotient, 4 2^-24 above 2^126, where the
// reciprocal is subnormal.  A comparison, not fminf: a NaN stays one, and the scale is the only
// place that can carry it to the product.  Under an infinity s_enc is 0, the codes too, and the
// scale infinite.)
__device__ __forceinline__ float i8_enc(uint32_t amax_bits) {
  const float amax = u2f(amax_bits), s = 127.0f * (1.0f / amax);
  return amax == 0.0f ? 1.0f : s > kFltMax ? kFltMax : s;
}
// x s rounded to the nearest even integer, in the low byte: adding 1.5 2^23 leaves
// no bits below the unit.  |x s| <= 127.5 by the choice of s, so nothing saturates.
__device__ __forceinline__ uint32_t i8_code(float x, float s) { return f2u(x * s + 12582912.0f); }
__device__ __forceinline__ uint32_t i8_pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0C0C0400u), hi = __builtin_amdgcn_perm(d, c, 0x0C0C0400u);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}
__device__ __forceinline__ uint32_t max_abs(const Raw<uint16_t>& r) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, r.v[0][i] & 0x7FFF7FFFu));
  return (uint32_t)max(m.x, m.y) << 16;
}

// Rows: a group of T threads per row, which stays in registers (P pieces of eight
// columns each) between the maximum and the encoding, so x is read once.  Bound by
// HBM: 2 bytes in, 1 out.
template <bool AL, int T, int P>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_i8_rows(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                             uint8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int WG = T < 256 ? 256 : T, G = WG / T;
  __shared__ uint32_t part[WG / 64];
  const int t = threadIdx.x % T, w = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * G + threadIdx.x / T;
  const bool live = row < rows;                            // G > 1: T is one wave, so a group leaves together
  if (T <= 64 && !live) return;
  const uint16_t* src = x + row * cols;
  Raw<uint16_t> r[P];
#pragma unroll
  for (int p = 0; p < P; ++p) r[p] = load_raw<AL>(src, (p * T + t) * 8, cols);
  uint32_t m = 0;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    end_piece<AL>(r[p], (p * T + t) * 8, cols);
    m = max(m, max_abs(r[p]));
  }
  m = wave_max_dpp(m);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) part[w] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < T / 64; ++i) m = max(m, part[i]);
  }
  const float s = i8_enc(m);
  if (t == 0) scales[row] = 1.0f / s;
  uint8_t* dst = codes + row * cols;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int col = (p * T + t) * 8;
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = i8_code(raw_at(r[p], j), s);
    if (col + 8 <= cols) {
      typedef ntu2 Any __attribute__((aligned(1)));
      const ntu2 v = {i8_pack4(c[0], c[1], c[2], c[3]), i8_pack4(c[4], c[5], c[6], c[7])};
      if (AL) *reinterpret_cast<ntu2*>(dst + col) = v;
      else *reinterpret_cast<Any*>(dst + col) = v;
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (col + j < cols) dst[col + j] = (uint8_t)c[j];
    }
  }
}

// Rows longer than a workgroup's registers hold: two passes, the second mostly from cache.
__global__ __launch_bounds__(1024) void k_i8_rows_long(const uint16_t* __restrict__ x, int64_t cols,
                                                      uint8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ uint32_t part[16];
  const int64_t row = blockIdx.x;
  const uint16_t* src = x + row * cols;
  uint32_t m = 0;
  for (int64_t c = threadIdx.x; c < cols; c += 1024) m = max(m, (uint32_t)(src[c] & 0x7FFF) << 16);
  m = wave_max_dpp(m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, part[i]);
  const float s = i8_enc(m);
  if (threadIdx.x == 0) scales[row] = 1.0f / s;
  for (int64_t c = threadIdx.x; c < cols; c += 1024)
    codes[row * cols + c] = (uint8_t)i8_code(u2f((uint32_t)src[c] << 16), s);
}

template <bool AL, int T, int P>
hipError_t run_rows(const void* x, int64_t rows, int64_t cols, uint8_t* codes, float* scales, hipStream_t s) {
  constexpr int WG = T < 256 ? 256 : T, G = WG / T;
  const int64_t blocks = (rows + G - 1) / G;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_i8_rows<AL, T, P>), dim3((unsigned)blocks), dim3(WG), 0, s, static_cast<const uint16_t*>(x), rows,
                     (int)cols, codes, scales);
  return hipGetLastError();
}
template <bool AL>
hipError_t run_rows_any(const void* x, int64_t rows, int64_t cols, uint8_t* codes, float* scales, hipStream_t s) {
  if (cols <= 512) return run_rows<AL, 64, 1>(x, rows, cols, codes, scales, s);
  if (cols <= 1024) return run_rows<AL, 64, 2>(x, rows, cols, codes, scales, s);
  if (cols <= 2048) return run_rows<AL, 64, 4>(x, rows, cols, codes, scales, s);
  if (cols <= 8192) return run_rows<AL, 256, 4>(x, rows, cols, codes, scales, s);
  if (cols <= 16384) return run_rows<AL, 256, 8>(x, rows, cols, codes, scales, s);
  if (cols <= 65536) return run_rows<AL, 1024, 8>(x, rows, cols, codes, scales, s);
  if (rows > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL(k_i8_rows_long, dim3((unsigned)rows), dim3(1024), 0, s, static_cast<const uint16_t*>(x), cols, codes,
                     scales);
  return hipGetLastError();
}

// ---------------------------------------------------------------- rows and columns

__global__ __launch_bounds__(256) void k_i8_zero(uint32_t* p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0;
}

// Maxima of 256 rows x 512 columns into amax_row [rows] and amax_col [cols] (bits of
// FP32, cleared before; a maximum does not depend on the order of the atomics).
constexpr int kAmaxRows = 256, kAmaxCols = 512;
template <bool AL>
__global__ __launch_bounds__(256) void k_i8_amax(const uint16_t* __restrict__ x, int64_t rows, int64_t cols, int strips,
                                                 uint32_t* amax_row, uint32_t* amax_col) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  __shared__ uint32_t rmax[kAmaxRows];
  __shared__ uint32_t cmax[4][kAmaxCols / 2];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t r0 = (int64_t)(blockIdx.x / strips) * kAmaxRows, c0 = (int64_t)(blockIdx.x % strips) * kAmaxCols;
  const int nr = (int)min((int64_t)kAmaxRows, rows - r0);
  const int64_t col = c0 + lane * 8;
  u16x2 cm[4] = {{0, 0}, {0, 0}, {0, 0}, {0, 0}};
  constexpr int U = 8;
  for (int i0 = w; i0 < kAmaxRows; i0 += 4 * U) {
    ntu4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + 4 * u;
      v[u] = ntu4{0u, 0u, 0u, 0u};
      if (i < nr && col < cols) {
        const uint16_t* src = x + (r0 + i) * cols + col;
        if (AL) {
          v[u] = *reinterpret_cast<const ntu4*>(src);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (col + j < cols) v[u][j >> 1] |= (uint32_t)src[j] << (16 * (j & 1));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      u16x2 rm = {0, 0};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const u16x2 a = __builtin_bit_cast(u16x2, v[u][k] & 0x7FFF7FFFu);
        cm[k] = __builtin_elementwise_max(cm[k], a);
        rm = __builtin_elementwise_max(rm, a);
      }
      const uint32_t m = wave_max_dpp((uint32_t)max(rm.x, rm.y));
      if (lane == 0 && i0 + 4 * u < kAmaxRows) rmax[i0 + 4 * u] = m << 16;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) cmax[w][lane * 4 + k] = __builtin_bit_cast(uint32_t, cm[k]);
  __syncthreads();
  const int t = threadIdx.x;
  if (t < nr) atomicMax(amax_row + r0 + t, rmax[t]);
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, cmax[i][t]));
  const int64_t c = c0 + 2 * t;
  if (c < cols) atomicMax(amax_col + c, (uint32_t)m.x << 16);
  if (c + 1 < cols) atomicMax(amax_col + c + 1, (uint32_t)m.y << 16);
}

// Codes of a 128 x 128 tile under the rows' and the columns' maxima.  A thread owns 8
// rows x 8 columns: the row codes go straight out as 128-byte pieces; the column
// codes, which have scales of their own, are packed along the rows and turned in LDS.
constexpr int kQtT = 128, kQtLd = kQtT + 8;
template <bool AL>
__global__ __launch_bounds__(256) void k_i8_qt(const uint16_t* __restrict__ x, int64_t rows, int64_t cols, int tiles_c,
                                               const uint32_t* __restrict__ amax_row, const uint32_t* __restrict__ amax_col,
                                               uint8_t* __restrict__ codes_row, float* __restrict__ scales_row,
                                               uint8_t* __restrict__ codes_col, float* __restrict__ scales_col) {
  __shared__ __attribute__((aligned(16))) uint8_t tile[kQtT * kQtLd];
  __shared__ float enc[2 * kQtT];
  const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
  const int tr = (int)(blockIdx.x / tiles_c), tc = (int)(blockIdx.x % tiles_c);
  const int64_t r0 = (int64_t)tr * kQtT, c0 = (int64_t)tc * kQtT;
  const int64_t col = c0 + tx * 8;
  ntu4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + ty * 8 + i;
    v[i] = ntu4{0u, 0u, 0u, 0u};
    if (r < rows && col < cols) {
      const uint16_t* src = x + r * cols + col;
      if (AL) {
        v[i] = *reinterpret_cast<const ntu4*>(src);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (col + j < cols) v[i][j >> 1] |= (uint32_t)src[j] << (16 * (j & 1));
      }
    }
  }
  {
    const bool is_row = t < kQtT;
    const int64_t i = is_row ? r0 + t : c0 + t - kQtT, n = is_row ? rows : cols;
    const float s = i < n ? i8_enc(is_row ? amax_row[i] : amax_col[i]) : 0.0f;
    enc[t] = s;
    if (i < n && is_row && tc == 0 && codes_row) scales_row[i] = 1.0f / s;
    if (i < n && !is_row && tr == 0 && codes_col) scales_col[i] = 1.0f / s;
  }
  __syncthreads();
  const auto at = [&](int i, int j) { return (j & 1) ? bf16_hi(v[i][j >> 1]) : bf16_lo(v[i][j >> 1]); };
  if (codes_row) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + ty * 8 + i;
      const float s = enc[ty * 8 + i];
      uint32_t c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = i8_code(at(i, j), s);
      if (r >= rows || col >= cols) continue;
      uint8_t* dst = codes_row + r * cols + col;
      if (AL) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(i8_pack4(c[0], c[1], c[2], c[3]), i8_pack4(c[4], c[5], c[6], c[7]));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (col + j < cols) dst[j] = (uint8_t)c[j];
      }
    }
  }
  if (codes_col) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = enc[kQtT + tx * 8 + j];
      uint32_t c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = i8_code(at(i, j), s);
      *reinterpret_cast<uint2*>(tile + (tx * 8 + j) * kQtLd + ty * 8) =
          make_uint2(i8_pack4(c[0], c[1], c[2], c[3]), i8_pack4(c[4], c[5], c[6], c[7]));
    }
    __syncthreads();
    const bool whole = (rows & 7) == 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int q = i * 16 + ty;                           // the tile's column
      const int64_t c = c0 + q, r = r0 + tx * 8;
      if (c >= cols || r >= rows) continue;
      const uint2 u = *reinterpret_cast<const uint2*>(tile + q * kQtLd + tx * 8);
      uint8_t* dst = codes_col + c * rows + r;
      if (whole) {
        *reinterpret_cast<uint2*>(dst) = u;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (r + j < rows) dst[j] = (uint8_t)((j < 4 ? u.x : u.y) >> (8 * (j & 3)));
      }
    }
  }
}

// ---------------------------------------------------------------- few tokens
//
// int8_linear of at most 64 rows in one launch: a workgroup of eight waves per 16
// columns quantizes all rows into LDS itself, with the weights of its first steps in
// flight meanwhile, then each wave takes an eighth of K, and the parts are added in LDS.
// The rows are quantized by every workgroup again, out of the L2: in at most 128 pieces of
// 512 columns, above which a launch of its own costs less.  Bound by the weights' bytes,
// or by the launch.
// LDS rows are whole 128-byte groups; chunk c of row r sits at slot c ^ (r & 7) of its group.
constexpr int kFewWaves = 8, kFewPieces = 128, kFewRows = 64, kFewAhead = 4;
template <int MI>
constexpr int few_part() { return kFewWaves * 16 * MI * (16 + 4) * 4; }

// PT: pieces of x per wave, at most.
template <int MI, int PT>
__global__ __launch_bounds__(kFewWaves * 64, PT <= 2 ? 4 : 2) void k_i8_linear(const uint16_t* __restrict__ x, int M, int K,
                                                              const uint8_t* __restrict__ w, int64_t N,
                                                              const float* __restrict__ sw,
                                                              const float* __restrict__ bias, uint16_t* __restrict__ c,
                                                              int64_t ldc) {
  constexpr int WK = kFewWaves, NT = 16, MT = 16 * MI, PS = NT + 4, D = kFewAhead;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ uint32_t most[kFewRows];
  const int lane = threadIdx.x & 63, r16 = lane & 15, q4 = lane >> 4;
  const int wk = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * NT;
  const int ks = (K + 127) & ~127;
  const int full = K / 128, steps = ks / 128;
  const int s0 = steps * wk / WK, s1 = steps * (wk + 1) / WK, f1 = min(s1, full);
  // x: pieces wk, wk + 8, ... of the rows' pieces in turn
  const int pr = (K + 511) / 512, pieces = M * pr, rcp = 65536 / pr + 1;   // t / pr = t rcp >> 16 for t < 128
  Raw<uint16_t> v[PT];
#pragma unroll
  for (int i = 0; i < PT; ++i) {
    const int t = wk + WK * i, row = t * rcp >> 16;
    if (t < pieces) v[i] = load_raw<true>(x + (int64_t)row * K, (t - row * pr) * 512 + lane * 8, K);
  }
  // weights: this lane's row (past the matrix: its last row again)
  const uint8_t* b = w + n0 * K;
  const int last_n = (int)min((int64_t)NT - 1, N - n0 - 1);
  const uint32_t ob = (uint32_t)min(r16, last_n) * (uint32_t)K;
  ntu4 fb[D][2];
  const auto load = [&](ntu4 (&f)[2], int s) {
    const uint32_t k = ob + (uint32_t)s * 128u + (uint32_t)q4 * 16u;
    f[0] = *reinterpret_cast<const ntu4*>(b + k);
    f[1] = *reinterpret_cast<const ntu4*>(b + k + 64);
  };
#pragma unroll
  for (int u = 0; u < D; ++u)
    if (s0 + u < f1) load(fb[u], s0 + u);

  if (threadIdx.x < kFewRows) most[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PT; ++i) {
    const int t = wk + WK * i;
    if (t < pieces) {
      const uint32_t m = wave_max_dpp(max_abs(v[i]));
      if (lane == 0) atomicMax(&most[t * rcp >> 16], m);   // a maximum: any order
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PT; ++i) {
    const int t = wk + WK * i, row = t * rcp >> 16, col = (t - row * pr) * 512 + lane * 8;
    if (t < pieces && col < ks) {
      const float s = i8_enc(most[row]);
      uint32_t e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = i8_code(raw_at(v[i], j), s);
      const int ch = col >> 4;
      const bool in = col < K;                             // the group's rest is zero
      *reinterpret_cast<ntu2*>(smem + row * ks + (((ch & ~7) | ((ch ^ row) & 7)) << 4) + (col & 8)) =
          ntu2{in ? i8_pack4(e[0], e[1], e[2], e[3]) : 0u, in ? i8_pack4(e[4], e[5], e[6], e[7]) : 0u};
    }
  }
  __syncthreads();

  nti4 acc[MI];
#pragma unroll
  for (int i = 0; i < MI; ++i) acc[i] = nti4{0, 0, 0, 0};
  const auto multiply = [&](const ntu4 (&f)[2], int s) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int row = min(16 * i + r16, M - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const ntu4 a = *reinterpret_cast<const ntu4*>(smem + row * ks + s * 128 + (((4 * h + q4) ^ (row & 7)) << 4));
        acc[i] = nt_mfma<kNtI8>(f[h], a, acc[i]);
      }
    }
  };
  for (int s = s0; s < f1; s += D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      if (s + u < f1) {
        multiply(fb[u], s + u);
        if (s + u + D < f1) load(fb[u], s + u + D);
      }
    }
  }
  if (s1 > full && s0 < s1) {                              // the partial group at the row's end
#pragma unroll
    for (int h = 0; h < 2; ++h) fb[0][h] = nt_load_end<false>(b + ob, full * 128 + q4 * 16 + 64 * h, K);
    multiply(fb[0], full);
  }
  __syncthreads();                                         // every wave has read the codes
  nti4* part = reinterpret_cast<nti4*>(smem);              // [WK][MT][PS / 4]
#pragma unroll
  for (int i = 0; i < MI; ++i) part[(wk * MT + 16 * i + r16) * PS / 4 + q4] = acc[i];
  __syncthreads();
  for (int q = threadIdx.x; q < M * (NT / 4); q += WK * 64) {
    const int row = q / (NT / 4), col = q % (NT / 4) * 4;
    nti4 v = part[(row * PS + col) / 4];
#pragma unroll
    for (int u = 1; u < WK; ++u) v += part[((u * MT + row) * PS + col) / 4];
    uint16_t* dst = c + row * ldc + n0 + col;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i <= last_n) {
        float y = (float)v[i] * (1.0f / i8_enc(most[row]) * sw[n0 + col + i]);
        if (bias) y = y + bias[n0 + col + i];
        dst[i] = bf16_rne(y);
      }
  }
}

template <int MI, int PT>
hipError_t run_few(const void* x, const Int8Args& a, hipStream_t s) {
  const int codes = (int)(a.M * ((a.K + 127) / 128 * 128)), lds = codes > few_part<MI>() ? codes : few_part<MI>();
  const void* fn = reinterpret_cast<const void*>(&k_i8_linear<MI, PT>);
  constexpr int codes_most = PT * kFewWaves * 512, most = codes_most > few_part<MI>() ? codes_most : few_part<MI>();
  if (lds > most || set_lds_limit(fn, most) != hipSuccess) return hipErrorInvalidConfiguration;
  const int64_t blocks = (a.N + 15) / 16;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_i8_linear<MI, PT>), dim3((unsigned)blocks), dim3(kFewWaves * 64), lds, s,
                     static_cast<const uint16_t*>(x), (int)a.M, (int)a.K, a.bc, a.N, a.bs, a.bias,
                     static_cast<uint16_t*>(a.c), a.ldc);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_i8_rows(const void* x, int64_t rows, int64_t cols, uint8_t* codes, float* scales, hipStream_t s) {
  const bool al = cols % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (reinterpret_cast<uintptr_t>(codes) & 7) == 0;
  return al ? run_rows_any<true>(x, rows, cols, codes, scales, s) : run_rows_any<false>(x, rows, cols, codes, scales, s);
}

bool i8_few_rows(const Int8Args& a) {
  if (a.M > kFewRows || a.K <= 0 || a.K % 16 != 0 || a.K > 8192) return false;
  // few pieces of x cost little beside the weights; more of them pay only where every
  // workgroup runs at once, and there by the launch that the host saves (us on the GPU by this
  // launch / by two: 1 x 28,672 x 4,096 25.6 / 29.8, 1 x 4,096 x 4,096 7.1 / 13.2, 3 x 1,000 x
  // 512 4.3 / 7.9; 48 x 2,048 x 2,048 9.3 / 9.3, 37 x 2,048 x 1,408 11.0 / 8.1 but 11.0 / 13.1
  // a call from Python; 8 x 28,672 x 4,096 45.7 / 30.0)
  const int64_t pieces = a.M * ((a.K + 511) / 512);
  return pieces <= 2 * kFewWaves || (pieces <= kFewPieces && (a.N + 15) / 16 <= 256);
}

hipError_t launch_i8_linear_few(const void* x, const Int8Args& a, hipStream_t s) {
  if (a.M * ((a.K + 511) / 512) <= 2 * kFewWaves) return run_few<1, 2>(x, a, s);   // 16 rows at most
  constexpr int PT = kFewPieces / kFewWaves;
  if (a.M <= 16) return run_few<1, PT>(x, a, s);
  return a.M <= 32 ? run_few<2, PT>(x, a, s) : run_few<4, PT>(x, a, s);
}

hipError_t launch_i8_qt(const void* x, int64_t rows, int64_t cols, uint8_t* codes_row, float* scales_row,
                        uint8_t* codes_col, float* scales_col, uint32_t* amax, hipStream_t s) {
  const int64_t n = rows + cols, strips = (cols + kAmaxCols - 1) / kAmaxCols;
  const int64_t ab = strips * ((rows + kAmaxRows - 1) / kAmaxRows), tiles_c = (cols + kQtT - 1) / kQtT;
  const int64_t qb = tiles_c * ((rows + kQtT - 1) / kQtT);
  if (ab > 0x7FFFFFFF || qb > 0x7FFFFFFF || (n + 255) / 256 > 0x7FFFFFFF) return hipErrorInvalidValue;
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  uint32_t *ar = amax, *ac = amax + rows;
  hipLaunchKernelGGL(k_i8_zero, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, amax, n);
  const bool al = cols % 8 == 0;
  if (al) {
    hipLaunchKernelGGL(k_i8_amax<true>, dim3((unsigned)ab), dim3(256), 0, s, xp, rows, cols, (int)strips, ar, ac);
    hipLaunchKernelGGL(k_i8_qt<true>, dim3((unsigned)qb), dim3(256), 0, s, xp, rows, cols, (int)tiles_c, ar, ac, codes_row,
                       scales_row, codes_col, scales_col);
  } else {
    hipLaunchKernelGGL(k_i8_amax<false>, dim3((unsigned)ab), dim3(256), 0, s, xp, rows, cols, (int)strips, ar, ac);
    hipLaunchKernelGGL(k_i8_qt<false>, dim3((unsigned)qb), dim3(256), 0, s, xp, rows, cols, (int)tiles_c, ar, ac, codes_row,
                       scales_row, codes_col, scales_col);
  }
  return hipGetLastError();
}

namespace {
NtArgs i8_args(const Int8Args& a) { return NtArgs{a.ac, a.bc, a.M, a.N, (uint32_t)a.K, 0, 0, 1, false}; }
}  // namespace

int i8_kernel(const Int8Args& a) {
  const NtArgs g = i8_args(a);
  return nt_choose(g, true, ring_fits(g), false, 0.0f).kernel;
}

hipError_t launch_i8_gemm(const Int8Args& a, hipStream_t s, int kernel, int rest, int count) {
  const NtArgs g = i8_args(a);
  const bool vec = a.ldc % 8 == 0 && (reinterpret_cast<uintptr_t>(a.c) & 15) == 0;
  const EpiI8 e{a.as, a.bs, a.bias, static_cast<uint16_t*>(a.c), a.ldc, a.M, a.N, vec, 0, 0, 0, 0};
  NtChoice c{kernel, rest == kNtChosen ? -1 : count, rest, nt_side(kernel) / nt_side(rest)};
  if (kernel == kNtChosen) c = nt_choose(g, true, ring_fits(g), false, 0.0f);
  if (c.kernel == kNtDirect16x64) return run_nt_direct<kNtI8, 1, 4, 1, 1, 4>(g, e, s);
  if (c.kernel == kNtDirect64x64) return run_nt_direct<kNtI8, 4, 4, 1, 1, 4>(g, e, s);
  return g.kb % 128 == 0 ? run_nt_choice<kNtI8, false>(g, c, e, s) : run_nt_choice<kNtI8, true>(g, c, e, s);
}

}  // namespace bsq
