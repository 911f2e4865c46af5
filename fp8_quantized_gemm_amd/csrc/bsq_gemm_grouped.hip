// Expert-grouped block-scaled GEMMs for gfx950 (contract in include/bsq.h):
//   rows:  C[p, :] = alpha_e A[p, :] . B_e^T for the rows p of group e
//   wgrad: C_e = alpha A[:, group e] . B[:, group e]^T
// with NVFP4, MXFP4 or MXFP8 operands, FP32 accumulation, BF16 out.
//
// k_gemm_grouped: one workgroup per MT x NT output tile, its waves split K and
// add their partial tiles through LDS in wave order.  Operands go from global
// memory straight into MFMA operand registers (no LDS staging): a lane of the
// 16-row MFMA operands owns row lane & 15 and, of each 128-element unit of K,
// 32 elements of lane group g = lane >> 4, so the four lanes of a row read 64
// (FP4) contiguous bytes.  Few rows per group make the product a stream of the
// weights, which this reads once per MT rows.
//  * NVFP4: the 32 codes are expanded to FP16 (dequant8) and feed four
//    16x16x32 FP16 MFMAs; MX: one 16x16x128 scaled MFMA per unit.
//  * FP8 operand bytes 0-15 of lane group g are k = 16 g + i of the unit, bytes
//    16-31 k = 64 + 16 g + i; the scale of the unit's block b (32 elements)
//    comes from lane group b.
// Any K (in whole scale blocks) and any group boundary (wgrad: in whole scale
// blocks): pieces past the range are zero with a unit scale.
#include "bsq_gemm_common.hpp"
#include "bsq_gemm_grouped.hpp"
#include "bsq_internal.hpp"

namespace bsq {

namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// One operand's rows as seen by a lane.
struct GsRow {
  const uint8_t* codes;   // at the first K element of the range
  const uint8_t* scales;
};

// 16 bytes at an address of any alignment.
__device__ __forceinline__ u32x4 load16(const uint8_t* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

template <int FMT>
struct GsFrag {
  u32x4 lo, hi;           // hi: FP8 only
  uint32_t sc;            // MX: scale byte; NVFP4: the two scale bytes of the 32 elements
};

// Unit u (128 elements) of a K range of klen elements: this lane's piece.
template <int FMT>
__device__ __forceinline__ void gs_load(GsFrag<FMT>& f, const GsRow& r, int64_t u, int64_t klen, int g) {
  const u32x4 z = {0u, 0u, 0u, 0u};
  const int64_t k = u * 128 + 32 * g;
  if constexpr (FMT == kMXFP8) {
    const int64_t k0 = u * 128 + 16 * g;
    f.lo = k0 < klen ? load16(r.codes + k0) : z;
    f.hi = k0 + 64 < klen ? load16(r.codes + k0 + 64) : z;
    f.sc = k < klen ? r.scales[k / 32] : 0x7Fu;
  } else if constexpr (FMT == kMXFP4) {
    f.lo = k < klen ? load16(r.codes + k / 2) : z;
    f.sc = k < klen ? r.scales[k / 32] : 0x7Fu;
  } else {
    f.lo = z;
    f.sc = 0;
    if (k + 32 <= klen) {
      f.lo = load16(r.codes + k / 2);
      uint16_t s;
      __builtin_memcpy(&s, r.scales + k / 16, 2);
      f.sc = s;
    } else if (k < klen) {                               // the range ends after 16 elements
      uint32_t h[2];
      __builtin_memcpy(h, r.codes + k / 2, 8);
      f.lo = u32x4{h[0], h[1], 0u, 0u};
      f.sc = r.scales[k / 16];
    }
  }
}

// acc += B tile . A tile^T of one unit: lane holds C row lane & 15 of the A tile
// and columns 4 g + i of the B tile.
template <int FMT>
__device__ __forceinline__ floatx4 gs_mfma_mx(const GsFrag<FMT>& b, const GsFrag<FMT>& a, floatx4 acc) {
  constexpr int T = FMT == kMXFP8 ? 0 : 4;               // operand type
  const u32x4 z = {0u, 0u, 0u, 0u};
  const u32x4 bh = FMT == kMXFP8 ? b.hi : z, ah = FMT == kMXFP8 ? a.hi : z;
  const intx8 bv = __builtin_bit_cast(intx8, __builtin_shufflevector(b.lo, bh, 0, 1, 2, 3, 4, 5, 6, 7));
  const intx8 av = __builtin_bit_cast(intx8, __builtin_shufflevector(a.lo, ah, 0, 1, 2, 3, 4, 5, 6, 7));
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv, av, acc, T, T, 0, (int)b.sc, 0, (int)a.sc);
}

// The four FP16 fragments of an NVFP4 piece (8 elements each).
__device__ __forceinline__ void gs_expand(const GsFrag<kNVFP4>& f, halfx8 (&x)[4]) {
  const halfx2 s0 = nvfp4_scale_pair<0>(f.sc), s1 = nvfp4_scale_pair<1>(f.sc);
  x[0] = dequant8(f.lo[0], s0);
  x[1] = dequant8(f.lo[1], s0);
  x[2] = dequant8(f.lo[2], s1);
  x[3] = dequant8(f.lo[3], s1);
}

template <int FMT, int MI, int NI, int W, bool WGRAD>
__global__ __launch_bounds__(W * 64) void k_gemm_grouped(GroupedArgs a, int tiles_m, int tiles_n, int vec_store) {
  constexpr int MT = MI * 16, NT = NI * 16, RS = NT + 4;
  extern __shared__ __attribute__((aligned(16))) float part[];   // [W][MT][RS]
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  const GroupRef ref{a.offsets, a.experts, a.ba_n};
  int tn;
  constexpr int PB = FMT == kMXFP8 ? 1 : 2, SB = FMT == kNVFP4 ? 16 : 32;   // elements per code / scale byte
  const int64_t code_ld = a.K / PB, scale_ld = a.K / SB;
  int64_t m0, mend, k0 = 0, klen = a.K;
  int e;
  const uint8_t *bc = a.bc, *bs = a.bs;
  uint16_t* c = static_cast<uint16_t*>(a.c);
  if constexpr (WGRAD) {
    int tm, lo, hi;
    e = wgrad_tile(blockIdx.x, tiles_m, tiles_n, tm, tn);
    m0 = (int64_t)tm * MT;
    mend = a.M;
    GroupTile t;
    group_range<SB, SB>(ref, e, a.K, lo, hi, t);
    k0 = t.row0;
    klen = hi;
    c += (int64_t)e * a.M * a.ldc;
  } else {
    GroupTile t;
    if (!group_tile_rows<MT>(ref, a.M, blockIdx.x, tiles_n, t, tn)) return;
    e = t.e;
    m0 = t.row0;
    mend = t.row1;
    if (e < 0) klen = 0;
    else {
      bc += (int64_t)e * a.N * code_ld;
      bs += (int64_t)e * a.N * scale_ld;
    }
  }
  const int64_t n0 = (int64_t)tn * NT;
  GsRow ra[MI], rb[NI];
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    int64_t r = m0 + i * 16 + r16;
    r = r < mend ? r : mend - 1;
    ra[i].codes = a.ac + r * code_ld + k0 / PB;
    ra[i].scales = a.as + r * scale_ld + k0 / SB;
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    int64_t r = n0 + i * 16 + r16;
    r = r < a.N ? r : a.N - 1;
    rb[i].codes = bc + r * code_ld + k0 / PB;
    rb[i].scales = bs + r * scale_ld + k0 / SB;
  }
  floatx4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t units = (klen + 127) / 128;
  const int64_t u0 = units * w / W, u1 = units * (w + 1) / W;
  for (int64_t u = u0; u < u1; ++u) {
    GsFrag<FMT> fa[MI], fb[NI];
#pragma unroll
    for (int j = 0; j < NI; ++j) gs_load<FMT>(fb[j], rb[j], u, klen, g);
#pragma unroll
    for (int i = 0; i < MI; ++i) gs_load<FMT>(fa[i], ra[i], u, klen, g);
    if constexpr (FMT == kNVFP4) {
      halfx8 xa[MI][4];
#pragma unroll
      for (int i = 0; i < MI; ++i) gs_expand(fa[i], xa[i]);
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        halfx8 xb[4];
        gs_expand(fb[j], xb);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int i = 0; i < MI; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xb[s], xa[i][s], acc[i][j], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[i][j] = gs_mfma_mx<FMT>(fb[j], fa[i], acc[i][j]);
    }
  }
  // the waves' partial tiles, added in wave order
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
      *reinterpret_cast<floatx4*>(part + (w * MT + i * 16 + r16) * RS + j * 16 + 4 * g) = acc[i][j];
  __syncthreads();
  float alpha = 1.0f;
  if constexpr (FMT == kNVFP4)
    alpha = nvfp4_s_dec(*a.aa) * nvfp4_s_dec(a.ba[a.ba_n > 1 && e > 0 ? e : 0]) * 16384.0f;
  for (int q = threadIdx.x; q < MT * NT / 8; q += W * 64) {
    const int row = q / (NT / 8), col = q % (NT / 8) * 8;
    const int64_t m = m0 + row, n = n0 + col;
    if (m >= mend || n >= a.N) continue;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
#pragma unroll
    for (int s = 0; s < W; ++s) {
      const floatx4* p = reinterpret_cast<const floatx4*>(part + (s * MT + row) * RS + col);
      const floatx4 x = p[0], y = p[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += x[i], v[4 + i] += y[i];
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(v[2 * i] * alpha, v[2 * i + 1] * alpha);
    uint16_t* dst = c + m * a.ldc + n;
    if (vec_store && n + 7 < a.N) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (n + i < a.N) dst[i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
    }
  }
}

template <int FMT, int MI, int NI, int W, bool WGRAD>
hipError_t run_gs(const GroupedArgs& a, hipStream_t s) {
  constexpr int MT = MI * 16, NT = NI * 16, LDS = W * MT * (NT + 4) * 4;
  static_assert(LDS <= 160 * 1024, "partial tiles fit the LDS");
  const int64_t tn = (a.N + NT - 1) / NT;
  // rows: each group may end inside a tile, and so may the rows past the last
  const int64_t tm = WGRAD ? (a.M + MT - 1) / MT : a.M / MT + a.experts + 1;
  const int64_t blocks = tm * tn * (WGRAD ? a.experts : 1);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  const bool vec = a.ldc % 8 == 0 && (reinterpret_cast<uintptr_t>(a.c) & 15) == 0;
  const void* fn = reinterpret_cast<const void*>(&k_gemm_grouped<FMT, MI, NI, W, WGRAD>);
  if (LDS > 64 * 1024 && set_lds_limit(fn, LDS) != hipSuccess) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_gemm_grouped<FMT, MI, NI, W, WGRAD>), dim3((unsigned)blocks), dim3(W * 64), LDS,
                     s, a, (int)tm, (int)tn, vec ? 1 : 0);
  return hipGetLastError();
}

template <int FMT>
hipError_t pick_rows(const GroupedArgs& a, hipStream_t s) {
  const int64_t per = a.M / a.experts;                   // rows per group, on average
  if (FMT == kNVFP4 && per > 160 && gemm_nvfp4_rx_grouped_fits(a, false))
    return launch_gemm_nvfp4_rx_grouped(a, false, s);
  if (per <= 16) return run_gs<FMT, 1, 4, 4, false>(a, s);
  return run_gs<FMT, 4, 4, 4, false>(a, s);
}

}  // namespace

hipError_t launch_gemm_grouped(const GroupedArgs& a, hipStream_t s) {
  if (a.fmt == kNVFP4) return pick_rows<kNVFP4>(a, s);
  if (a.fmt == kMXFP4) return pick_rows<kMXFP4>(a, s);
  return pick_rows<kMXFP8>(a, s);
}

hipError_t launch_gemm_grouped_wgrad(const GroupedArgs& a, hipStream_t s) {
  if (a.fmt == kNVFP4 && a.K / a.experts > 160 && gemm_nvfp4_rx_grouped_fits(a, true))
    return launch_gemm_nvfp4_rx_grouped(a, true, s);
  if (a.fmt == kNVFP4) return run_gs<kNVFP4, 4, 4, 4, true>(a, s);
  if (a.fmt == kMXFP4) return run_gs<kMXFP4, 4, 4, 4, true>(a, s);
  return run_gs<kMXFP8, 4, 4, 4, true>(a, s);
}

}  // namespace bsq
