// Expert-grouped block-scaled GEMMs for gfx950 (contract in include/bsq.h):
//   rows:  C[p, :] = alpha_e A[p, :] . B_e^T for the rows p of group e
//   wgrad: C_e = alpha A[:, group e] . B[:, group e]^T
// with NVFP4, MXFP4 or MXFP8 operands, FP32 accumulation, BF16 out.
//
// k_gemm_grouped: a workgroup of WM x WN x WK waves per output tile; each wave
// owns MI x NI accumulator tiles of 16 x 16, and the WK waves that share them
// split K and add their parts through LDS in wave order.  Operands go from
// global memory straight into MFMA operand registers (no LDS staging), one K
// step of 128 code bytes per row ahead of the MFMAs: a lane of the 16-row MFMA
// operands owns row lane & 15, and the four lanes of a row read one whole
// 128-byte line in two instructions.  Few rows per group make the product a
// stream of the weights, which a 16-row tile reads once with K split over four
// waves to have enough loads in flight; many rows per group go to the 256 x 256
// kernels.
//  * FP4 (a step is 256 elements of K): lane group g = lane >> 4 owns elements
//    64 g .. 64 g + 63, 32 contiguous code bytes.  NVFP4: expanded to FP16
//    (dequant8) for eight 16x16x32 FP16 MFMAs; MXFP4: two 16x16x128 scaled
//    MFMAs, each lane's 32 elements one block.
//  * MXFP8 (a step is 128 elements): operand bytes 0-15 of lane group g are
//    elements 16 g + i, bytes 16-31 elements 64 + 16 g + i; the scale of block b
//    (32 elements) comes from lane group b.
// A and B use the same map, so the order of K inside a step does not matter.
// Any K (in whole scale blocks) and any group boundary (wgrad: in whole scale
// blocks): pieces past the range are zero with a unit scale.
#include "bsq_gemm_common.hpp"
#include "bsq_gemm_grouped.hpp"
#include "bsq_internal.hpp"

namespace bsq {

namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <int FMT>
constexpr int gs_step() { return FMT == kMXFP8 ? 128 : 256; }          // K elements
template <int FMT>
constexpr int gs_scales() { return FMT == kNVFP4 ? 16 : FMT == kMXFP4 ? 8 : 4; }   // scale bytes per row

// Global memory at a wave-uniform base plus a lane's byte offset.  The base goes
// through an empty statement, so that the compiler keeps it in scalar registers
// and adds the offset inside the load instead of carrying 64-bit addresses (2 rows
// over 8 experts, 4,096 x 14,336, NVFP4: 16 us against 19 us; elsewhere equal).
typedef __attribute__((address_space(1))) const uint8_t* GlobalBytes;
__device__ __forceinline__ GlobalBytes uniform_base(const uint8_t* p) {
  uint64_t v = reinterpret_cast<uint64_t>(p);
  asm volatile("" : "+s"(v));
  return (GlobalBytes)v;
}
// A value of type V at an address of any alignment.
template <typename V>
__device__ __forceinline__ V load_as(GlobalBytes p) {
  typedef V U __attribute__((aligned(1)));
  return *reinterpret_cast<__attribute__((address_space(1))) const U*>(p);
}

// One lane's piece of a step of one 16-row tile.
struct GsFrag {
  u32x4 c[2];
  uint32_t sc;            // NVFP4: 4 scale bytes; MXFP4: 2; MXFP8: 1
};

// Piece at (codes, scales) of the step, lane group g already in the offsets.
template <int FMT>
__device__ __forceinline__ void gs_load(GsFrag& f, GlobalBytes codes, GlobalBytes scales) {
  f.c[0] = load_as<u32x4>(codes);
  f.c[1] = load_as<u32x4>(codes + (FMT == kMXFP8 ? 64 : 16));
  if constexpr (FMT == kNVFP4) f.sc = load_as<uint32_t>(scales);
  else if constexpr (FMT == kMXFP4) f.sc = load_as<uint16_t>(scales);
  else f.sc = *scales;
}

// The same for the last step of a range, of which only rem elements exist.
template <int FMT>
__device__ __forceinline__ void gs_load_part(GsFrag& f, GlobalBytes codes, GlobalBytes scales, int rem, int g) {
  const u32x4 z = {0u, 0u, 0u, 0u};
  if constexpr (FMT == kMXFP8) {
    f.c[0] = 16 * g < rem ? load_as<u32x4>(codes) : z;
    f.c[1] = 16 * g + 64 < rem ? load_as<u32x4>(codes + 64) : z;
    f.sc = 32 * g < rem ? *scales : 0x7Fu;
  } else {
    const int k = 64 * g;
    f.sc = FMT == kMXFP4 ? 0x7F7Fu : 0u;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      f.c[c] = z;
      if (k + 32 * c + 32 <= rem) {
        f.c[c] = load_as<u32x4>(codes + 16 * c);
      } else if (FMT == kNVFP4 && k + 32 * c < rem) {      // ends after 16 elements
        f.c[c] = u32x4{load_as<uint32_t>(codes + 16 * c), load_as<uint32_t>(codes + 16 * c + 4), 0u, 0u};
      }
    }
    constexpr int B = FMT == kNVFP4 ? 16 : 32;
#pragma unroll
    for (int b = 0; b < 64 / B; ++b)
      if (k + b * B < rem) f.sc = (f.sc & ~(0xFFu << (8 * b))) | ((uint32_t)scales[b] << (8 * b));
  }
}

// Scaled MFMA of half H of a step: D = B tile . A tile^T, so a lane holds C row
// lane & 15 of the A tile and columns 4 g + i of the B tile.  With FP8 operands the
// instruction adds eight adjacent products at a time aligned to 2^-13 of the largest
// of them (measured: a product of 2^-14 beside 1 - 1 of the same eight is lost, of
// any other eight kept), everything else in FP32; FP4 products lie within 2^8 of
// each other and add exactly.  It is what the ungrouped MX products use.  On 256 rows
// of K 1,408 it puts 0.9% of the BF16 outputs one step from the nearest (FP32 sums:
// 0.001%) and leaves the error against 64 bits at that of the rounding, 1.654e-3;
// expanding to FP16, whose MFMA adds exactly, would halve the matrix rate.
template <int FMT, int H>
__device__ __forceinline__ floatx4 gs_mfma_mx(const GsFrag& b, const GsFrag& a, floatx4 acc) {
  constexpr int T = FMT == kMXFP8 ? 0 : 4;               // operand type
  const u32x4 z = {0u, 0u, 0u, 0u};
  const u32x4 bh = FMT == kMXFP8 ? b.c[1] : z, ah = FMT == kMXFP8 ? a.c[1] : z;
  const intx8 bv = __builtin_bit_cast(intx8, __builtin_shufflevector(b.c[H], bh, 0, 1, 2, 3, 4, 5, 6, 7));
  const intx8 av = __builtin_bit_cast(intx8, __builtin_shufflevector(a.c[H], ah, 0, 1, 2, 3, 4, 5, 6, 7));
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv, av, acc, T, T, H, (int)b.sc, H, (int)a.sc);
}

// FP16 fragment of eight NVFP4 elements: dword Q (0-7) of the piece, its 16
// elements' scale in half (Q >> 1) & 1 of the pair converted for half Q >> 2.
template <int Q>
__device__ __forceinline__ halfx8 gs_expand(const GsFrag& f) {
  const halfx2 p = nvfp4_scale_pairs2<(Q >> 2)>(f.sc);
  return dequant8(f.c[Q >> 2][Q & 3], (Q & 2) ? halfx2{p.y, p.y} : halfx2{p.x, p.x});
}

template <int MI, int NI, int Q>
__device__ __forceinline__ void gs_nvfp4_steps(const GsFrag (&fa)[MI], const GsFrag (&fb)[NI], floatx4 (&acc)[MI][NI]) {
  if constexpr (Q < 8) {
    halfx8 xa[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) xa[i] = gs_expand<Q>(fa[i]);
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const halfx8 xb = gs_expand<Q>(fb[j]);
#pragma unroll
      for (int i = 0; i < MI; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xb, xa[i], acc[i][j], 0, 0, 0);
    }
    gs_nvfp4_steps<MI, NI, Q + 1>(fa, fb, acc);
  }
}

// All MFMAs of a step.
template <int FMT, int MI, int NI>
__device__ __forceinline__ void gs_multiply(const GsFrag (&fa)[MI], const GsFrag (&fb)[NI], floatx4 (&acc)[MI][NI]) {
  if constexpr (FMT == kNVFP4) {
    gs_nvfp4_steps<MI, NI, 0>(fa, fb, acc);
  } else {
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int i = 0; i < MI; ++i) acc[i][j] = gs_mfma_mx<FMT, 0>(fb[j], fa[i], acc[i][j]);
    if constexpr (FMT == kMXFP4) {
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[i][j] = gs_mfma_mx<FMT, 1>(fb[j], fa[i], acc[i][j]);
    }
  }
}

// Whole pieces of eight columns from LDS to C, which is read by another kernel
// much later: streaming stores (6-8% less time on outputs of 190-270 MB).
__device__ __forceinline__ void gs_store8(uint16_t* dst, const uint32_t (&o)[4], int cols, int vec_store) {
  if (vec_store && cols >= 8) {
    __builtin_nontemporal_store(u32x4{o[0], o[1], o[2], o[3]}, reinterpret_cast<u32x4*>(dst));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cols) dst[i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
  }
}

// The tile through LDS, whole row pieces stored: with K split over WK waves the
// FP32 parts, added in wave order; else the rounded values.  Wave (wk, wm, wn)
// holds MI x NI accumulator tiles; rows and columns past last_m, last_n are not
// stored.
template <int MT, int NT, int WK>
constexpr int gs_store_lds() { return WK > 1 ? WK * MT * (NT + 4) * 4 : MT * (NT + 8) * 2; }
template <int MI, int NI, int WM, int WN, int WK>
__device__ __forceinline__ void gs_store(const floatx4 (&acc)[MI][NI], uint8_t* smem, int wk, int wm, int wn, float alpha,
                                         uint16_t* c, int64_t ldc, int last_m, int last_n, int vec_store) {
  constexpr int MT = WM * MI * 16, NT = WN * NI * 16, T = WM * WN * WK * 64;
  const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
  if constexpr (WK == 1) {
    constexpr int RS = NT + 8;                             // BF16 row stride: 16 bytes of padding
    uint16_t* part = reinterpret_cast<uint16_t*>(smem);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const floatx4 v = acc[i][j];
        *reinterpret_cast<uint2*>(part + ((wm * MI + i) * 16 + r16) * RS + (wn * NI + j) * 16 + 4 * g) =
            make_uint2(pack_bf16x2(v[0] * alpha, v[1] * alpha), pack_bf16x2(v[2] * alpha, v[3] * alpha));
      }
    __syncthreads();
#pragma unroll 4
    for (int q = threadIdx.x; q < MT * NT / 8; q += T) {
      const int row = q / (NT / 8), col = q % (NT / 8) * 8;
      if (row > last_m || col > last_n) continue;
      const u32x4 v = *reinterpret_cast<const u32x4*>(part + row * RS + col);
      const uint32_t o[4] = {v[0], v[1], v[2], v[3]};
      gs_store8(c + (int64_t)row * ldc + col, o, last_n + 1 - col, vec_store);
    }
  } else {
    constexpr int RS = NT + 4;                             // FP32 [WK][MT][RS]
    float* part = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
        *reinterpret_cast<floatx4*>(part + (wk * MT + (wm * MI + i) * 16 + r16) * RS + (wn * NI + j) * 16 + 4 * g) =
            acc[i][j];
    __syncthreads();
#pragma unroll 2
    for (int q = threadIdx.x; q < MT * NT / 8; q += T) {
      const int row = q / (NT / 8), col = q % (NT / 8) * 8;
      if (row > last_m || col > last_n) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
#pragma unroll
      for (int s = 0; s < WK; ++s) {
        const floatx4* p = reinterpret_cast<const floatx4*>(part + (s * MT + row) * RS + col);
        const floatx4 x = p[0], y = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += x[i], v[4 + i] += y[i];
      }
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(v[2 * i] * alpha, v[2 * i + 1] * alpha);
      gs_store8(c + (int64_t)row * ldc + col, o, last_n + 1 - col, vec_store);
    }
  }
}

// alpha of an NVFP4 product with expert e's B (1 for MX).  A tile without a
// reduction (the rows of no group, an empty group) is stored as exact zeros: 0
// whatever the amaxes say, whose decode scales can be infinite or NaN.
template <int FMT>
__device__ __forceinline__ float gs_alpha(const GroupedArgs& a, int e, bool any) {
  if constexpr (FMT != kNVFP4) return 1.0f;
  return any ? nvfp4_s_dec(*a.aa) * nvfp4_s_dec(a.ba[a.ba_n > 1 ? e : 0]) * 16384.0f : 0.0f;
}

// OFF: type of the lanes' byte offsets from the tile's first row (32 bits
// unless a tile's rows span 4 GiB).
template <int FMT, int MI, int NI, int WM, int WN, int WK, bool WGRAD, typename OFF>
__global__ __launch_bounds__(WM * WN * WK * 64) void k_gemm_grouped(GroupedArgs a, int tiles_m, int tiles_n,
                                                                    int vec_store) {
  constexpr int MT = WM * MI * 16, NT = WN * NI * 16, STEP = gs_step<FMT>();
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];   // gs_store
  const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = w / (WM * WN), wm = w % (WM * WN) / WN, wn = w % WN;
  const GroupRef ref{a.offsets, a.experts, a.ba_n};
  constexpr int PB = FMT == kMXFP8 ? 1 : 2, SB = FMT == kNVFP4 ? 16 : 32;   // elements per code / scale byte
  const int64_t code_ld = a.K / PB, scale_ld = a.K / SB;
  int64_t m0, mend, klen = a.K;
  int e, tn;
  const uint8_t *ac = a.ac, *as = a.as, *bc = a.bc, *bs = a.bs;
  uint16_t* c = static_cast<uint16_t*>(a.c);
  if constexpr (WGRAD) {
    int tm, lo, hi;
    e = wgrad_tile(blockIdx.x, tiles_m, tiles_n, tm, tn);
    m0 = (int64_t)tm * MT;
    mend = a.M;
    GroupTile t;
    group_range<SB, SB>(ref, e, a.K, lo, hi, t);
    klen = hi;
    ac += t.row0 / PB;
    as += t.row0 / SB;
    bc += t.row0 / PB;
    bs += t.row0 / SB;
    c += (int64_t)e * a.M * a.ldc;
  } else {
    GroupTile t;
    if (!group_tile_rows<MT>(ref, a.M, blockIdx.x, tiles_n, t, tn)) return;
    e = t.e;
    m0 = t.row0;
    mend = t.row1;
    if (e < 0) {
      klen = 0;                        // rows of no group: zeros
    } else {
      bc += (int64_t)e * a.N * code_ld;
      bs += (int64_t)e * a.N * scale_ld;
    }
  }
  const int64_t n0 = (int64_t)tn * NT;
  ac += m0 * code_ld;
  as += m0 * scale_ld;
  bc += n0 * code_ld;
  bs += n0 * scale_ld;
  // this lane's rows (past the operand: its last row again, never stored)
  OFF oa[MI], sa[MI], ob[NI], sb[NI];
  const int last_m = (int)(mend - m0 < MT ? mend - m0 - 1 : MT - 1);
  const int last_n = (int)(a.N - n0 < NT ? a.N - n0 - 1 : NT - 1);
  const int gc = FMT == kMXFP8 ? 16 * g : 32 * g, gsc = gs_scales<FMT>() / 4 * g;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int r = min((wm * MI + i) * 16 + r16, last_m);
    oa[i] = (OFF)r * (OFF)code_ld + gc;
    sa[i] = (OFF)r * (OFF)scale_ld + gsc;
  }
#pragma unroll
  for (int j = 0; j < NI; ++j) {
    const int r = min((wn * NI + j) * 16 + r16, last_n);
    ob[j] = (OFF)r * (OFF)code_ld + gc;
    sb[j] = (OFF)r * (OFF)scale_ld + gsc;
  }
  floatx4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  const int full = (int)(klen / STEP), rem = (int)(klen - (int64_t)full * STEP);
  const int steps = full + (rem > 0);
  const int s0 = (int)((int64_t)steps * wk / WK), s1 = (int)((int64_t)steps * (wk + 1) / WK);
  const int f1 = min(s1, full);
  // two sets of fragments: a step's loads are in flight during the step before
  GsFrag fa[2][MI], fb[2][NI];
  const auto load = [&](GsFrag (&xa)[MI], GsFrag (&xb)[NI], int s) {
    const int64_t co = (int64_t)s * 128, so = (int64_t)s * gs_scales<FMT>();
    const GlobalBytes pb = uniform_base(bc + co), qb = uniform_base(bs + so);
    const GlobalBytes pa = uniform_base(ac + co), qa = uniform_base(as + so);
#pragma unroll
    for (int j = 0; j < NI; ++j) gs_load<FMT>(xb[j], pb + ob[j], qb + sb[j]);
#pragma unroll
    for (int i = 0; i < MI; ++i) gs_load<FMT>(xa[i], pa + oa[i], qa + sa[i]);
  };
  if (s0 < f1) {
    load(fa[0], fb[0], s0);
    int s = s0;
    for (; s + 2 < f1; s += 2) {
      load(fa[1], fb[1], s + 1);
      gs_multiply<FMT, MI, NI>(fa[0], fb[0], acc);
      load(fa[0], fb[0], s + 2);
      gs_multiply<FMT, MI, NI>(fa[1], fb[1], acc);
    }
    if (s + 1 < f1) load(fa[1], fb[1], s + 1);
    gs_multiply<FMT, MI, NI>(fa[0], fb[0], acc);
    if (s + 1 < f1) gs_multiply<FMT, MI, NI>(fa[1], fb[1], acc);
  }
  if (s1 > full && s0 < s1) {                              // the partial step at the end of the range
    const int64_t co = (int64_t)full * 128, so = (int64_t)full * gs_scales<FMT>();
    const GlobalBytes pb = uniform_base(bc + co), qb = uniform_base(bs + so);
    const GlobalBytes pa = uniform_base(ac + co), qa = uniform_base(as + so);
#pragma unroll
    for (int j = 0; j < NI; ++j) gs_load_part<FMT>(fb[0][j], pb + ob[j], qb + sb[j], rem, g);
#pragma unroll
    for (int i = 0; i < MI; ++i) gs_load_part<FMT>(fa[0][i], pa + oa[i], qa + sa[i], rem, g);
    gs_multiply<FMT, MI, NI>(fa[0], fb[0], acc);
  }

  gs_store<MI, NI, WM, WN, WK>(acc, smem, wk, wm, wn, gs_alpha<FMT>(a, e, klen > 0), c + m0 * a.ldc + n0, a.ldc, last_m,
                               last_n, vec_store);
}

// ---------------------------------------------------------------- LDS-staged kernel
//
// A workgroup of four waves (WM x WN) per output tile of WM MI x WN NI MFMA tiles.
// Steps of 128 code bytes per row reach LDS by global -> LDS direct loads (eight
// lanes per row read one whole line), in NB buffers: with two, a step's loads run
// while the step before is multiplied, one barrier per step.  16-byte chunk c of row r sits at slot c ^ ((r >> 1) & 7), so that 16
// consecutive rows of one chunk fall on distinct banks.  Scales are staged as
// dwords.  Steps start at a multiple of the step in a row; a step that holds K
// elements outside [lo, hi) (the range's ends) is clipped in LDS: the scales there
// become 0 (2^-127 for MX) on both sides, and the codes too where that leaves
// something to add (MXFP4: A's; MXFP8: both), so that the rows of another group
// add exact zeros whatever they hold, NaN included.
constexpr int kGlThreads = 256;
template <int FMT, int MT, int NT>
constexpr int gl_buf() { return (MT + NT) * (128 + gs_scales<FMT>()); }
template <int FMT, int MT, int NT, int NB>
constexpr int gl_lds() {
  constexpr int ring = NB * gl_buf<FMT, MT, NT>(), epi = gs_store_lds<MT, NT, 1>();
  return ring > epi ? ring : epi;
}
__host__ __device__ constexpr int gl_swz(int r) { return (r >> 1) & 7; }

// One operand of a step: R rows, codes into LDS at `lds`, scales at `lds_sc`.
// Rows past `last` and bytes past a row's end are read from the last ones.
template <int FMT, int R>
__device__ __forceinline__ void gl_stage(const uint8_t* codes, const uint8_t* scales, uint32_t code_ld,
                                         uint32_t scale_ld, uint32_t k_code, uint32_t k_scale, int last, uint32_t lds,
                                         uint32_t lds_sc, int w, int lane) {
  constexpr int S = gs_scales<FMT>(), D = S / 4;           // dwords of scales per row
#pragma unroll
  for (int i = 0; i < (R + 31) / 32; ++i) {
    const int base = (i * 4 + w) * 8, r = base + (lane >> 3);
    const uint32_t off = min(k_code + (uint32_t)(((lane & 7) ^ gl_swz(r)) * 16), code_ld - 16);
    const uint32_t to = (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds + (uint32_t)(base * 128)));
    if (R % 32 == 0 || base < R) dma_to_lds<16>(codes, (uint32_t)min(r, last) * code_ld + off, to);
  }
  constexpr int RI = 64 / D, N = (R + RI - 1) / RI;        // rows per load, loads
#pragma unroll
  for (int i = 0; i < (N + 3) / 4; ++i) {
    const int base = (i * 4 + w) * RI, r = base + lane / D;
    const uint32_t off = min(k_scale + (uint32_t)(lane % D * 4), scale_ld - 4);
    const uint32_t to = (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds_sc + (uint32_t)(base * S)));
    if (r < R && (N % 4 == 0 || i * 4 + w < N)) dma_to_lds<4>(scales, (uint32_t)min(r, last) * scale_ld + off, to);
  }
}

template <int FMT, int MI, int NI, int WM, int WN, bool WGRAD, int NB>
__global__ __launch_bounds__(kGlThreads, NB == 1 ? 3 : 2) void k_gemm_grouped_lds(GroupedArgs a, int tiles_m, int tiles_n,
                                                                    int vec_store) {
  constexpr int MT = 16 * WM * MI, NT = 16 * WN * NI, STEP = gs_step<FMT>(), S = gs_scales<FMT>();
  constexpr int BUF = gl_buf<FMT, MT, NT>(), BC = MT * 128, SA = (MT + NT) * 128, SBO = SA + MT * S;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const uint32_t smem_lds = (uint32_t)(size_t)(__attribute__((address_space(3))) uint8_t*)smem;
  const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = w / WN, wn = w % WN;
  const GroupRef ref{a.offsets, a.experts, a.ba_n};
  constexpr int PB = FMT == kMXFP8 ? 1 : 2, SB = FMT == kNVFP4 ? 16 : 32;
  const uint32_t code_ld = (uint32_t)(a.K / PB), scale_ld = (uint32_t)(a.K / SB);
  int64_t m0, mend;
  int e, tn, lo = 0, hi = (int)a.K;
  uint32_t kc = 0, ks = 0;                                 // byte offsets of the first step in a row
  const uint8_t *bc = a.bc, *bs = a.bs;
  uint16_t* c = static_cast<uint16_t*>(a.c);
  GroupTile t;
  if constexpr (WGRAD) {
    int tm;
    e = wgrad_tile(blockIdx.x, tiles_m, tiles_n, tm, tn);
    m0 = (int64_t)tm * MT;
    mend = a.M;
    group_range<SB, STEP>(ref, e, a.K, lo, hi, t);
    // a short range starts at a whole dword of scales instead where that saves a
    // step (32 experts of 125 rows, 2048 x 1408: NVFP4 93 -> 74 us, MXFP4 48 -> 43);
    // a long one keeps whole lines (MXFP4 up to 1.3 times slower without)
    const int cut = lo / (4 * SB) * (4 * SB);
    if (hi <= 3 * STEP && (hi - cut + STEP - 1) / STEP < (hi + STEP - 1) / STEP) {
      t.row0 += cut;
      lo -= cut;
      hi -= cut;
    }
    kc = (uint32_t)(t.row0 / PB);
    ks = (uint32_t)(t.row0 / SB);
    c += (int64_t)e * a.M * a.ldc;
  } else {
    if (!group_tile_rows<MT>(ref, a.M, blockIdx.x, tiles_n, t, tn)) return;
    e = t.e;
    m0 = t.row0;
    mend = t.row1;
    if (e < 0) {
      hi = 0;                          // rows of no group: zeros
    } else {
      bc += (int64_t)e * a.N * code_ld;
      bs += (int64_t)e * a.N * scale_ld;
    }
  }
  const int64_t n0 = (int64_t)tn * NT;
  const uint8_t *ac = a.ac + m0 * code_ld, *as = a.as + m0 * scale_ld;
  bc += n0 * code_ld;
  bs += n0 * scale_ld;
  c += m0 * a.ldc + n0;
  const int last_m = (int)(mend - m0 < MT ? mend - m0 - 1 : MT - 1);
  const int last_n = (int)(a.N - n0 < NT ? a.N - n0 - 1 : NT - 1);
  const int steps = (hi + STEP - 1) / STEP;
  const auto stage = [&](int s) {
    const uint32_t b = smem_lds + (uint32_t)((s & (NB - 1)) * BUF);
    gl_stage<FMT, MT>(ac, as, code_ld, scale_ld, kc + s * 128u, ks + (uint32_t)(s * S), last_m, b, b + SA, w, lane);
    gl_stage<FMT, NT>(bc, bs, code_ld, scale_ld, kc + s * 128u, ks + (uint32_t)(s * S), last_n, b + BC, b + SBO, w, lane);
  };
  floatx4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  if (NB == 2 && steps > 0) stage(0);
  for (int s = 0; s < steps; ++s) {
    if constexpr (NB == 1) {
      if (s > 0) lds_barrier();                            // every wave has read step s - 1
      stage(s);
    }
    // step s has landed for every wave, and (two buffers) every wave has read
    // step s - 1, whose buffer step s + 1 goes into
    wait_vmcnt<0>();
    lds_barrier();
    if (NB == 2 && s + 1 < steps) stage(s + 1);
    uint8_t* b = smem + (s & (NB - 1)) * BUF;
    if (s * STEP < lo || s * STEP + STEP > hi) {
      // codes: MXFP4's A, MXFP8's A and B (whose codes can be NaN); scales: all
      if constexpr (FMT != kNVFP4) {
        for (int q = threadIdx.x; q < (FMT == kMXFP8 ? MT + NT : MT) * 8; q += kGlThreads) {
          const int r = q >> 3, ch = q & 7, k = s * STEP + ch * (STEP / 8);
          if (k < lo || k >= hi) *reinterpret_cast<u32x4*>(b + r * 128 + ((ch ^ gl_swz(r)) << 4)) = u32x4{0u, 0u, 0u, 0u};
        }
      }
      for (int q = threadIdx.x; q < (MT + NT) * S / 4; q += kGlThreads) {
        uint32_t* sc = reinterpret_cast<uint32_t*>(b + SA) + q;
        const int k = s * STEP + q % (S / 4) * 4 * SB;
        uint32_t keep = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (k + i * SB >= lo && k + i * SB < hi) keep |= 0xFFu << (8 * i);
        *sc &= keep;
      }
      lds_barrier();
    }
    GsFrag fa[MI], fb[NI];
    const auto read = [&](GsFrag& f, int row, int codes, int scales) {
      const uint8_t* p = b + codes + row * 128;
      constexpr int c0 = FMT == kMXFP8 ? 1 : 2, c1 = FMT == kMXFP8 ? 4 : 1;
      f.c[0] = *reinterpret_cast<const u32x4*>(p + (((c0 * g) ^ gl_swz(row)) << 4));
      f.c[1] = *reinterpret_cast<const u32x4*>(p + (((c0 * g + c1) ^ gl_swz(row)) << 4));
      const uint8_t* q = b + scales + row * S + S / 4 * g;
      f.sc = S == 16 ? *reinterpret_cast<const uint32_t*>(q) : S == 8 ? *reinterpret_cast<const uint16_t*>(q) : *q;
    };
#pragma unroll
    for (int j = 0; j < NI; ++j) read(fb[j], (wn * NI + j) * 16 + r16, BC, SBO);
#pragma unroll
    for (int i = 0; i < MI; ++i) read(fa[i], (wm * MI + i) * 16 + r16, 0, SA);
    gs_multiply<FMT, MI, NI>(fa, fb, acc);
  }
  lds_barrier();                                           // every wave is done with the buffers
  gs_store<MI, NI, WM, WN, 1>(acc, smem, 0, wm, wn, gs_alpha<FMT>(a, e, steps > 0), c, a.ldc, last_m, last_n, vec_store);
}

// Whole dwords of scales per step and 16-byte aligned code rows; 32-bit offsets
// inside a tile's rows.
template <int FMT>
bool gl_fits(const GroupedArgs& a) {
  const uintptr_t sc = reinterpret_cast<uintptr_t>(a.as) | reinterpret_cast<uintptr_t>(a.bs);
  return a.K > 0 && a.K % (FMT == kNVFP4 ? 64 : 128) == 0 && a.K < ((int64_t)1 << 24) && sc % 4 == 0;
}

template <int FMT, int MI, int NI, int WM, int WN, bool WGRAD, int NB = 2>
hipError_t run_gl(const GroupedArgs& a, hipStream_t s) {
  constexpr int MT = 16 * WM * MI, NT = 16 * WN * NI, LDS = gl_lds<FMT, MT, NT, NB>();
  const int64_t tn = (a.N + NT - 1) / NT;
  const int64_t tm = WGRAD ? (a.M + MT - 1) / MT : max_row_tiles(a.M, a.experts, MT);
  const int64_t blocks = tm * tn * (WGRAD ? a.experts : 1);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  const bool vec = a.ldc % 8 == 0 && (reinterpret_cast<uintptr_t>(a.c) & 15) == 0;
  if (set_lds_limit(reinterpret_cast<const void*>(&k_gemm_grouped_lds<FMT, MI, NI, WM, WN, WGRAD, NB>), LDS) != hipSuccess)
    return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_gemm_grouped_lds<FMT, MI, NI, WM, WN, WGRAD, NB>), dim3((unsigned)blocks), dim3(kGlThreads), LDS, s, a,
                     (int)tm, (int)tn, vec ? 1 : 0);
  return hipGetLastError();
}

template <int FMT, int MI, int NI, int WM, int WN, int WK, bool WGRAD, typename OFF = uint32_t>
hipError_t run_gs(const GroupedArgs& a, hipStream_t s) {
  constexpr int MT = WM * MI * 16, NT = WN * NI * 16, LDS = gs_store_lds<MT, NT, WK>();
  static_assert(LDS <= 160 * 1024, "partial tiles fit the LDS");
  const int64_t tn = (a.N + NT - 1) / NT;
  const int64_t tm = WGRAD ? (a.M + MT - 1) / MT : max_row_tiles(a.M, a.experts, MT);
  const int64_t blocks = tm * tn * (WGRAD ? a.experts : 1);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  const bool vec = a.ldc % 8 == 0 && (reinterpret_cast<uintptr_t>(a.c) & 15) == 0;
  const void* fn = reinterpret_cast<const void*>(&k_gemm_grouped<FMT, MI, NI, WM, WN, WK, WGRAD, OFF>);
  if (LDS > 64 * 1024 && set_lds_limit(fn, LDS) != hipSuccess) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_gemm_grouped<FMT, MI, NI, WM, WN, WK, WGRAD, OFF>), dim3((unsigned)blocks),
                     dim3(WM * WN * WK * 64), LDS, s, a, (int)tm, (int)tn, vec ? 1 : 0);
  return hipGetLastError();
}

// A tile's rows span less than 4 GiB.
bool narrow(const GroupedArgs& a) { return a.K < ((int64_t)1 << 24); }

template <int FMT>
bool rx_fits(const GroupedArgs& a, bool wgrad) {
  return FMT == kNVFP4 ? gemm_nvfp4_rx_grouped_fits(a, wgrad) : gemm_mx_rx_grouped_fits(a, wgrad);
}
template <int FMT>
hipError_t run_rx(const GroupedArgs& a, bool wgrad, hipStream_t s) {
  return FMT == kNVFP4 ? launch_gemm_nvfp4_rx_grouped(a, wgrad, s) : launch_gemm_mx_rx_grouped(a, wgrad, s);
}

template <int FMT, bool WGRAD>
hipError_t run_variant(const GroupedArgs& a, int v, hipStream_t s) {
  if (v == k256x256) return run_rx<FMT>(a, WGRAD, s);
  if (v == kLds64x64) return run_gl<FMT, 2, 2, 2, 2, WGRAD>(a, s);
  if (v == kLds64x128) return run_gl<FMT, 2, 4, 2, 2, WGRAD>(a, s);
  // short reductions (MX): one buffer, so three workgroups instead of two share a
  // compute unit and cover each other's loads and stores (32 experts of 125 rows,
  // 2048 x 1408, MXFP4: 46 us against 57 us); NVFP4's expansion keeps the vector
  // units busy either way and its registers allow only two (106 against 90 us), and
  // a long K is better off with the next step in flight
  if (v == kLds128x128) return run_gl<FMT, 4, 4, 2, 2, WGRAD, WGRAD && FMT != kNVFP4 ? 1 : 2>(a, s);
  if (!narrow(a)) return run_gs<FMT, 1, 4, 1, 1, 4, WGRAD, uint64_t>(a, s);
  if constexpr (!WGRAD) {
    if (v == kLds16x128) return run_gl<FMT, 1, 2, 1, 4, WGRAD>(a, s);
    if (v == kLds32x128) return run_gl<FMT, 2, 2, 1, 4, WGRAD>(a, s);
    if (v == kDirect16x64) return run_gs<FMT, 1, 4, 1, 1, 4, WGRAD>(a, s);
    if (v == kDirect16x32) return run_gs<FMT, 1, 2, 1, 1, 8, WGRAD>(a, s);
  }
  return run_gs<FMT, 4, 4, 1, 1, 4, WGRAD>(a, s);
}

// What a tile costs, in microseconds measured on an MI355X: a K step of 128 code
// bytes per row when the chip is full (per compute unit) and when a workgroup
// runs alone, and a tile besides its steps.
struct TileCost {
  int v, mt, nt, wk;
  float step[3], alone[3], tile;       // [NVFP4, MXFP4, MXFP8]
};
constexpr TileCost kCosts[] = {
    {kDirect16x32, 16, 32, 8, {0.355f, 0.30f, 0.265f}, {1.3f, 1.2f, 1.2f}, 0.3f},
    {kDirect16x64, 16, 64, 4, {0.39f, 0.39f, 0.40f}, {1.4f, 1.3f, 1.2f}, 0.4f},
    {kLds16x128, 16, 128, 1, {0.50f, 0.28f, 0.29f}, {0.75f, 0.50f, 0.50f}, 0.4f},
    {kLds32x128, 32, 128, 1, {0.70f, 0.33f, 0.36f}, {0.87f, 0.55f, 0.50f}, 0.5f},
    {kLds64x64, 64, 64, 1, {0.64f, 0.26f, 0.30f}, {0.87f, 0.50f, 0.45f}, 0.45f},
    {kLds64x128, 64, 128, 1, {1.15f, 0.42f, 0.49f}, {1.44f, 0.65f, 0.60f}, 0.7f},
    {kLds128x128, 128, 128, 1, {1.85f, 0.78f, 0.75f}, {2.1f, 0.90f, 0.75f}, 1.1f},
    {k256x256, 256, 256, 1, {5.4f, 1.8f, 1.66f}, {4.25f, 1.6f, 1.1f}, 6.0f},    // rows
    {k256x256, 256, 256, 1, {4.8f, 1.4f, 1.7f}, {4.8f, 1.4f, 1.7f}, 12.0f},     // wgrad
};

constexpr int kRows256 = 7;
static_assert(kCosts[kRows256].v == k256x256 && kCosts[kRows256 + 1].v == k256x256, "the two 256 x 256 rows");

// The kernel with the least estimated time for `tiles` tiles of `steps` steps:
// the longest of the chip's throughput over all tiles, one workgroup's own way
// through K, and reading B at 5 TB/s (rows; a group's further row tiles find half
// of it in cache), plus 0.3 of the other two, which overlap it only in part.  The
// sizes of the groups are on the device; their average and 0.6 tiles of padding
// each are taken; a 256 x 256 reduction starts and ends at whole 512-element periods
// (MX).  The constants were chosen on 138 row products (K in multiples of 128, N of
// 64) and 72 WGRAD ones.  On shapes that none was chosen by, the choice is within
// 10% of the best kernel in 86 of 90 and 53 of 60 row products of such K and N (36%
// at most), in 51 of 60 WGRAD products of M and N in multiples of 4 (38% at most),
// and in 39 of 60 row products of any other K (twice at most).
// Where scales are not whole dwords (gl_fits) only the direct kernels are to choose
// from, and from 256 rows per expert on the 64 x 64 one takes 1.8 to 5 times as long
// as the neighbouring multiple of 128 (8 experts of 2,048 rows, N 4,096, MXFP4: K
// 2,880 579 us, K 2,944 155 us).  The 128 x 128 tile alone would take 2 to 5 times
// as long for single tokens, the 16 x 128 tile 2 to 4 times for 1,024 rows per
// expert.
template <int FMT>
int pick(const GroupedArgs& a, bool wgrad) {
  if (!gl_fits<FMT>(a)) return !wgrad && a.M / a.experts <= 16 ? kDirect16x64 : kDirect64x64;
  constexpr int f = FMT == kNVFP4 ? 0 : FMT == kMXFP4 ? 1 : 2, STEP = gs_step<FMT>();
  const double cus = device_cus() > 0 ? device_cus() : 256;
  const double rows = (double)(wgrad ? a.K : a.M);
  const double groups = wgrad || rows > a.experts ? a.experts : rows;
  const double row_bytes = (double)a.K * (FMT == kMXFP8 ? 1.0 : 0.5);
  int best = kLds64x64;
  double least = 1e300;
  for (const TileCost& t : kCosts) {
    if (t.v == k256x256 && !rx_fits<FMT>(a, wgrad)) continue;
    if (wgrad ? t.v < kLds64x64 || &t == &kCosts[kRows256] : &t == &kCosts[kRows256 + 1]) continue;
    const double period = t.v == k256x256 && FMT != kNVFP4 ? 512 / STEP : 1;
    const double steps = wgrad ? rows / groups / STEP + 0.5 * period : (double)((a.K + STEP - 1) / STEP);
    const double tn = (double)((a.N + t.nt - 1) / t.nt);
    const double in_group = rows / groups / t.mt + 0.6;
    const double tm = wgrad ? groups * (double)((a.M + t.mt - 1) / t.mt) : groups * (in_group > 1 ? in_group : 1.0);
    double full = tm * tn / cus * (steps * t.step[f] + t.tile);
    const double alone = steps / t.wk * t.alone[f] + t.tile;
    const double read = wgrad ? 0.0 : 0.5 * (groups + tm) * (double)a.N * row_bytes / 5e6;
    // short ranges, clipped at both ends; one buffer for MX (run_variant)
    if (wgrad && t.v == kLds128x128) full *= FMT == kNVFP4 ? 1.15 : 0.85;
    const double most = full > alone ? (full > read ? full : read) : (alone > read ? alone : read);
    const double us = most + 0.3 * (full + alone + read - most);
    if (us < least) {
      least = us;
      best = t.v;
    }
  }
  return best;
}

template <int FMT>
hipError_t run_picked(const GroupedArgs& a, bool wgrad, hipStream_t s) {
  const int v = pick<FMT>(a, wgrad);
  return wgrad ? run_variant<FMT, true>(a, v, s) : run_variant<FMT, false>(a, v, s);
}

hipError_t run_any(const GroupedArgs& a, bool wgrad, hipStream_t s) {
  if (a.fmt == kNVFP4) return run_picked<kNVFP4>(a, wgrad, s);
  if (a.fmt == kMXFP4) return run_picked<kMXFP4>(a, wgrad, s);
  return run_picked<kMXFP8>(a, wgrad, s);
}

// Whether kernel v is one of those that compute this product of these operands.
template <int FMT>
bool takes(const GroupedArgs& a, bool wgrad, int v) {
  if (v < kDirect16x64 || v > k256x256) return false;
  if (wgrad && v < kLds64x64 && v != kDirect64x64) return false;
  if (v == k256x256) return rx_fits<FMT>(a, wgrad);
  return v < kLds16x128 ? narrow(a) : gl_fits<FMT>(a);
}

template <int FMT>
hipError_t run_on(const GroupedArgs& a, bool wgrad, int v, hipStream_t s) {
  if (!takes<FMT>(a, wgrad, v)) return hipErrorInvalidValue;
  return wgrad ? run_variant<FMT, true>(a, v, s) : run_variant<FMT, false>(a, v, s);
}

}  // namespace

int grouped_kernel(const GroupedArgs& a, bool wgrad) {
  if (a.fmt == kNVFP4) return pick<kNVFP4>(a, wgrad);
  return a.fmt == kMXFP4 ? pick<kMXFP4>(a, wgrad) : pick<kMXFP8>(a, wgrad);
}

hipError_t launch_gemm_grouped_on(const GroupedArgs& a, bool wgrad, int kernel, hipStream_t s) {
  if (a.fmt == kNVFP4) return run_on<kNVFP4>(a, wgrad, kernel, s);
  return a.fmt == kMXFP4 ? run_on<kMXFP4>(a, wgrad, kernel, s) : run_on<kMXFP8>(a, wgrad, kernel, s);
}

hipError_t launch_gemm_grouped(const GroupedArgs& a, hipStream_t s) { return run_any(a, false, s); }
hipError_t launch_gemm_grouped_wgrad(const GroupedArgs& a, hipStream_t s) { return run_any(a, true, s); }

}  // namespace bsq
