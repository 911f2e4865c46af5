// Products C = A . B^T of plain operands (8-bit integers or FP16, both K-major)
// for gfx950, shared by the integer products and the Newton-Schulz products:
// which tile a workgroup computes, the kernel that loads operands straight into
// MFMA registers, and how a finished tile reaches its epilogue.
//
// Both element types use the 16 x 16 MFMA that takes 64 bytes of K per row
// (v_mfma_i32_16x16x64_i8, v_mfma_f32_16x16x32_f16): lane l holds row l & 15 and
// the 16 bytes of chunk l >> 4, so the two share every byte of data movement and
// differ in one instruction.  The B tile is the first operand: a lane's accumulator
// holds row l & 15 of the A tile and columns 4 (l >> 4) .. + 3 of the B tile.
#pragma once

#include "bsq_gemm_common.hpp"
#include "bsq_internal.hpp"

namespace bsq {

enum NtElem { kNtI8 = 0, kNtF16 = 1 };

typedef uint32_t ntu4 __attribute__((ext_vector_type(4)));
typedef uint32_t ntu2 __attribute__((ext_vector_type(2)));
typedef int nti4 __attribute__((ext_vector_type(4)));
typedef float ntf4 __attribute__((ext_vector_type(4)));
template <int EL>
struct NtTypes { typedef nti4 acc; };
template <>
struct NtTypes<kNtF16> { typedef ntf4 acc; };

struct NtArgs {
  const uint8_t* a;              // [M rows of kb bytes]
  const uint8_t* b;              // [N rows of kb bytes]
  int64_t M, N;
  uint32_t kb;                   // bytes of K per row, also the row stride
  int64_t stride_a, stride_b;    // bytes from one matrix of a stack to the next
  int batch;
  bool sym;                      // C is symmetric: only the tiles on and below the diagonal
};

// The tiles that a launch computes: `count` of the tiles_m x tiles_n grid of a matrix
// (below the diagonal if symmetric) of each of a stack, from number `first` on in the order
// of nt_tile, each cut into split x split tiles of the launch's own size.
struct NtGrid {
  int first, count, per, tiles_m, tiles_n, split;
};

inline int64_t nt_tiles(const NtArgs& g, int mt, int nt) {
  const int64_t tm = (g.M + mt - 1) / mt, tn = (g.N + nt - 1) / nt;
  return (g.sym ? tm * (tm + 1) / 2 : tm * tn) * g.batch;
}
inline NtGrid nt_grid(const NtArgs& g, int mt, int nt) {
  const int64_t tm = (g.M + mt - 1) / mt, tn = (g.N + nt - 1) / nt, per = g.sym ? tm * (tm + 1) / 2 : tm * tn;
  return NtGrid{0, (int)(per * g.batch), (int)per, (int)tm, (int)tn, 1};
}

// Matrix e and tile (tm, tn) number t: the order sweeps 8 (lower triangle: 4) tile rows at
// a time so that neighbouring tiles share A and B rows.
__device__ __forceinline__ void nt_tile_of(int t, const NtGrid& d, bool sym, int& e, int& tm, int& tn) {
  e = t / d.per;
  t -= e * d.per;
  if (!sym) {
    const int group = 8 * d.tiles_n, first = t / group * 8, gm = min(d.tiles_m - first, 8);
    t %= group;
    tm = first + t % gm;
    tn = t / gm;
    return;
  }
  // rows s .. s + h - 1: the h x s tiles left of the diagonal block in columns of
  // four, then the block's triangle
  int s = 0, h = min(4, d.tiles_m);
  while (t >= h * s + h * (h + 1) / 2) {
    t -= h * s + h * (h + 1) / 2;
    s += 4;
    h = min(4, d.tiles_m - s);
  }
  if (t < h * s) {
    tn = t / (4 * h) * 4;
    t %= 4 * h;
    tm = s + t % h;
    tn += t / h;
  } else {
    t -= h * s;
    int k = 0;
    while (t > k) t -= ++k;
    tm = s + k;
    tn = s + t;
  }
}
// The tile of block `pid`, in scalar registers (the divisions are vector operations).
// Blocks are dealt round-robin to the 8 XCDs; each gets a contiguous run of the order, so
// that its tiles share rows in its L2.
__device__ __forceinline__ void nt_tile(int pid, const NtGrid& d, bool sym, int& e, int& tm, int& tn) {
  const int total = d.count * d.split * d.split, q = total / 8, r = total % 8, x = pid % 8;
  int t = x * q + (x < r ? x : r) + pid / 8, sub = 0;
  if (d.split > 1) {
    sub = t % (d.split * d.split);
    t /= d.split * d.split;
  }
  nt_tile_of(d.first + t, d, sym, e, tm, tn);
  e = __builtin_amdgcn_readfirstlane(e);
  tm = __builtin_amdgcn_readfirstlane(tm * d.split + sub / d.split);
  tn = __builtin_amdgcn_readfirstlane(tn * d.split + sub % d.split);
}

template <int EL>
__device__ __forceinline__ typename NtTypes<EL>::acc nt_mfma(const ntu4& b, const ntu4& a,
                                                            typename NtTypes<EL>::acc c) {
  if constexpr (EL == kNtI8)
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(nti4, b), __builtin_bit_cast(nti4, a), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(halfx8, b), __builtin_bit_cast(halfx8, a), c, 0, 0, 0);
}

// 16 bytes at any alignment.
__device__ __forceinline__ ntu4 nt_load16(const uint8_t* p) {
  typedef ntu4 U __attribute__((aligned(1)));
  return *reinterpret_cast<const U*>(p);
}

// The 16-byte chunk at byte k of a row of kb bytes, for the row's end.  A chunk that
// crosses it is read from kb - 16 on, in both operands alike (the order of K does
// not matter), and its bytes before k, which belong to other chunks, are zeroed in A.
template <bool A>
__device__ __forceinline__ ntu4 nt_load_end(const uint8_t* row, int k, int kb) {
  if (k >= kb) return ntu4{0u, 0u, 0u, 0u};
  if (k + 16 <= kb) return nt_load16(row + k);
  ntu4 v = {0u, 0u, 0u, 0u};
  if (kb >= 16) {
    v = nt_load16(row + kb - 16);
    if (A) {
      const int drop = k + 16 - kb;                        // 1 .. 15 bytes
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = drop - 4 * i;
        v[i] = d <= 0 ? v[i] : d >= 4 ? 0u : v[i] & (0xFFFFFFFFu << (8 * d));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 15; ++i)
      if (i < kb) v[i >> 2] |= (uint32_t)row[i] << (8 * (i & 3));
  }
  return v;
}

// ---------------------------------------------------------------- epilogues
//
// A finished tile becomes 16-bit values in LDS (Epi::pack4, four columns of one row)
// and leaves as whole row pieces of eight (Epi::store), and, with Epi::kTrans, as
// pieces of its transpose (Epi::store_t).  Epi::at moves the epilogue's pointers to a
// wave's part of the tile, whose rows and columns are counted from there; r16 and c4 are
// the lane's row and first column in a 16 x 16 block.  What pack4 needs of the rows of
// block row i (Row), of the columns of block column j (Col) and of what it adds at block
// (i, j) (Add), and store of what it updates (Fetch), is loaded by calls of their own,
// some places ahead.

struct EpiNothing {};

// 8-bit integer products: BF16(FP32(sum) (sa sb) + bias).  The sum is exact, so the
// result does not depend on the kernel that formed it.
struct EpiI8 {
  static constexpr bool kTrans = false;
  const float* sa;
  const float* sb;
  const float* bias;             // null: none
  uint16_t* c;
  int64_t ldc;
  int64_t rows, cols;
  bool vec;                      // c 16-byte aligned and ldc % 8 == 0
  int M, N, r16, c4;             // rows and columns left from the wave's first, negative past the matrix
  struct Row { float s; };
  struct Col { float s[4], b[4]; };
  typedef EpiNothing Add;
  typedef EpiNothing Fetch;
  __device__ __forceinline__ void at(int, int64_t m0, int64_t n0, int r, int c4_) {
    sa += m0;
    sb += n0;
    if (bias) bias += n0;
    c += m0 * ldc + n0;
    M = (int)max((int64_t)-1024, min(rows - m0, (int64_t)1024));
    N = (int)max((int64_t)-1024, min(cols - n0, (int64_t)1024));
    r16 = r;
    c4 = c4_;
  }
  __device__ __forceinline__ Row row_at(int m) const { return Row{sa[min(m, M - 1)]}; }
  __device__ __forceinline__ Col col_at(int n) const {
    Col k;
    const float* b = bias ? bias : sb;                     // loaded either way: no branch around each load
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = min(n + i, N - 1);
      k.s[i] = sb[j];
      k.b[i] = b[j];
    }
    return k;
  }
  __device__ __forceinline__ Row row(int i) const { return row_at(i * 16 + r16); }
  __device__ __forceinline__ Col col(int j) const { return col_at(j * 16 + c4); }
  __device__ __forceinline__ void add(Add&, int, int) const {}
  __device__ __forceinline__ ntu2 pack4(int, int, const Row& r, const Col& k, const Add&, nti4 v) const {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = (float)v[i] * (r.s * k.s[i]);
      y[i] = bias ? y[i] + k.b[i] : y[i];
    }
    return ntu2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
  }
  __device__ __forceinline__ void fetch(Fetch&, int, int) const {}
  __device__ __forceinline__ void store(int m, int n, const ntu4& v, const Fetch&) {
    if (m >= M || n >= N) return;
    uint16_t* dst = c + m * ldc + n;
    if (vec && n + 8 <= N) {
      __builtin_nontemporal_store(v, reinterpret_cast<ntu4*>(dst));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (n + i < N) dst[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
    }
  }
  __device__ __forceinline__ void store_t(int, int, const ntu4&) {}
  __device__ __forceinline__ void finish(uint8_t*) {}
};

// ---------------------------------------------------------------- direct kernel
//
// A workgroup of WM x WN x WK waves per tile of WM MI x WN NI MFMA tiles; the WK
// waves that share a tile split K and add their parts through LDS in wave order.
// Steps of 128 bytes per row, one step ahead of the MFMAs; the four lanes of a row
// read one whole 128-byte line in two instructions.  Any K, any alignment of rows.
template <int MI, int NI, int WM, int WN, int WK>
constexpr int nt_direct_lds() {
  constexpr int MT = WM * MI * 16, NT = WN * NI * 16;
  return WK * MT * (NT + 4) * 4 + MT * (NT + 4) * 2;
}
template <int EL, int MI, int NI, int WM, int WN, int WK, typename Epi>
__global__ __launch_bounds__(WM * WN * WK * 64) void k_nt_direct(NtArgs g, NtGrid d, Epi epi) {
  typedef typename NtTypes<EL>::acc Acc;
  constexpr int MT = WM * MI * 16, NT = WN * NI * 16, T = WM * WN * WK * 64;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & 63, r16 = lane & 15, q4 = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = w / (WM * WN), wm = w % (WM * WN) / WN, wn = w % WN;
  int e, tm, tn;
  nt_tile(blockIdx.x, d, g.sym, e, tm, tn);
  const int64_t m0 = (int64_t)tm * MT, n0 = (int64_t)tn * NT;
  const uint8_t* a = g.a + e * g.stride_a + m0 * g.kb;
  const uint8_t* b = g.b + e * g.stride_b + n0 * g.kb;
  const int last_m = (int)(g.M - m0 < MT ? g.M - m0 - 1 : MT - 1), last_n = (int)(g.N - n0 < NT ? g.N - n0 - 1 : NT - 1);
  uint32_t oa[MI], ob[NI];                                 // this lane's rows; past the operand: its last row again
#pragma unroll
  for (int i = 0; i < MI; ++i) oa[i] = (uint32_t)min((wm * MI + i) * 16 + r16, last_m) * g.kb;
#pragma unroll
  for (int j = 0; j < NI; ++j) ob[j] = (uint32_t)min((wn * NI + j) * 16 + r16, last_n) * g.kb;
  Acc acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = Acc{0, 0, 0, 0};

  const int full = (int)(g.kb / 128), steps = (int)((g.kb + 127) / 128);
  const int s0 = (int)((int64_t)steps * wk / WK), s1 = (int)((int64_t)steps * (wk + 1) / WK), f1 = min(s1, full);
  ntu4 fa[2][MI][2], fb[2][NI][2];
  const auto load = [&](ntu4 (&xa)[MI][2], ntu4 (&xb)[NI][2], int s) {
    const uint32_t k = (uint32_t)s * 128u + (uint32_t)q4 * 16u;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      xb[j][0] = nt_load16(b + ob[j] + k);
      xb[j][1] = nt_load16(b + ob[j] + k + 64);
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      xa[i][0] = nt_load16(a + oa[i] + k);
      xa[i][1] = nt_load16(a + oa[i] + k + 64);
    }
  };
  const auto multiply = [&](const ntu4 (&xa)[MI][2], const ntu4 (&xb)[NI][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[i][j] = nt_mfma<EL>(xb[j][h], xa[i][h], acc[i][j]);
  };
  if (s0 < f1) {
    load(fa[0], fb[0], s0);
    int s = s0;
    for (; s + 2 < f1; s += 2) {
      load(fa[1], fb[1], s + 1);
      multiply(fa[0], fb[0]);
      load(fa[0], fb[0], s + 2);
      multiply(fa[1], fb[1]);
    }
    if (s + 1 < f1) load(fa[1], fb[1], s + 1);
    multiply(fa[0], fb[0]);
    if (s + 1 < f1) multiply(fa[1], fb[1]);
  }
  if (s1 > full && s0 < s1) {                              // the partial step at the row's end
    const int k = full * 128 + q4 * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < NI; ++j) fb[0][j][h] = nt_load_end<false>(b + ob[j], k + 64 * h, (int)g.kb);
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[0][i][h] = nt_load_end<true>(a + oa[i], k + 64 * h, (int)g.kb);
    }
    multiply(fa[0], fb[0]);
  }

  // the waves' parts added, 16-bit tile in rows of NT + 4
  static_assert(!Epi::kTrans, "the direct kernel stores no transpose and adds nothing");
  constexpr int RS = NT + 4, PS = NT + 4;
  uint16_t* E = reinterpret_cast<uint16_t*>(smem + WK * MT * PS * 4);
  epi.at(e, m0, n0, 0, 0);
  Acc* part = reinterpret_cast<Acc*>(smem);                // [WK][MT][PS / 4]
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
      part[((wk * MT + (wm * MI + i) * 16 + r16) * PS + (wn * NI + j) * 16) / 4 + q4] = acc[i][j];
  __syncthreads();
  for (int q = threadIdx.x; q < MT * NT / 4; q += T) {
    const int row = q / (NT / 4), col = q % (NT / 4) * 4;
    Acc v = part[(row * PS + col) / 4];
#pragma unroll
    for (int s = 1; s < WK; ++s) v += part[((s * MT + row) * PS + col) / 4];
    *reinterpret_cast<ntu2*>(E + row * RS + col) = epi.pack4(0, 0, epi.row_at(row), epi.col_at(col), EpiNothing{}, v);
  }
  __syncthreads();
  for (int q = threadIdx.x; q < MT * NT / 8; q += T) {
    const int row = q / (NT / 8), col = q % (NT / 8) * 8;
    const ntu2 x = *reinterpret_cast<const ntu2*>(E + row * RS + col), y = *reinterpret_cast<const ntu2*>(E + row * RS + col + 4);
    epi.store(row, col, ntu4{x[0], x[1], y[0], y[1]}, EpiNothing{});
  }
  epi.finish(smem);
}

template <int EL, int MI, int NI, int WM, int WN, int WK, typename Epi>
hipError_t run_nt_direct(const NtArgs& g, const Epi& epi, hipStream_t s) {
  constexpr int MT = WM * MI * 16, NT = WN * NI * 16, LDS = nt_direct_lds<MI, NI, WM, WN, WK>();
  static_assert(LDS <= 160 * 1024, "LDS plan");
  const int64_t total = nt_tiles(g, MT, NT);
  if (total > 0x7FFFFFFF || (uint64_t)MT * g.kb >= (1ull << 32) || (uint64_t)NT * g.kb >= (1ull << 32))
    return hipErrorInvalidValue;
  const void* fn = reinterpret_cast<const void*>(&k_nt_direct<EL, MI, NI, WM, WN, WK, Epi>);
  if (LDS > 64 * 1024 && set_lds_limit(fn, LDS) != hipSuccess) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_nt_direct<EL, MI, NI, WM, WN, WK, Epi>), dim3((unsigned)total), dim3(WM * WN * WK * 64), LDS, s, g,
                     nt_grid(g, MT, NT), epi);
  return hipGetLastError();
}

}  // namespace bsq
