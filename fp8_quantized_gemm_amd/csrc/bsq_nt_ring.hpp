// The LDS-staged kernel of the plain products (bsq_nt.hpp): C = A . B^T of 8-bit
// integers or FP16 on square tiles of 256, 192, 128, 96 or 64.
//
// A workgroup of four waves (one per SIMD) per tile of 32 NT rows and columns; wave w
// owns the quarter (w >> 1, w & 1) as NT x NT accumulators of 16 x 16, pinned in
// AGPRs by MFMAs written as inline assembly (left to itself the compiler moves them
// between AGPRs and VGPRs).  The 16 x 16 MFMA rather than the 32 x 32 one: the matrix
// pipe is as busy, but draws less power, so the clock holds higher.
//
// Units of 128 bytes of K per row reach LDS by global -> LDS direct loads into a ring
// of NB buffers (the eight lanes of a row read one whole 128-byte line); a unit is two
// steps of 64 bytes, NT^2 MFMAs per wave each.  The fragments of a step are read
// during the step before into the other half of a double-buffered register set.  The
// second step of unit U first waits for unit U + 1, then a barrier makes it visible
// and retires unit U's buffer (whose last reads were issued in the step before), and
// the loads of unit U + NB go into that buffer during the step.  The last NB units are
// peeled, so that every wait count is a constant and a step is one basic block (the
// compiler does not see the MFMAs' operand timing).
//
// LDS rows are 128 bytes; 16-byte chunk c of row r sits at slot c ^ ((r >> 1) & 7):
// 16 lanes (16 consecutive rows, one chunk) are served per cycle by 64 banks, and rows
// of one parity start on the same bank.
//
// Smaller tiles read more bytes per operation (256: 64 KB of LDS fill per 2^23
// multiply-adds of 8-bit integers, per 2^22 of FP16; 192: 1.33, 128: 2 times as much) and
// exist for shapes whose 256 tiles would leave compute units idle.
//
// On tiles of 256 the epilogues of the orthogonalisation's polynomial and product need more
// registers than a wave has: 33 and 71 VGPRs go to scratch memory (136 and 288 bytes a lane),
// the next X of tall matrices 1 VGPR (8 bytes).
#pragma once

#include "bsq_nt.hpp"

namespace bsq {

template <int NT, int NB>
constexpr int ring_lds() {
  const int ring = NB * 2 * 32 * NT * 128, epi = 4 * 16 * NT * (32 * NT + 8);
  return ring > epi ? ring : epi;
}

template <int EL>
__device__ __forceinline__ void ring_mfma(typename NtTypes<EL>::acc& acc, const ntu4& b, const ntu4& a) {
  if constexpr (EL == kNtI8) asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
  else asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}

template <int NT>
struct RingFrag {
  ntu4 a[NT], b[NT];
};

// What a lane needs of the tile: byte offsets of the rows it loads, its chunks of
// even and odd loads, and where it reads fragments.
template <int NT>
struct RingLane {
  const uint8_t* a;
  const uint8_t* b;
  uint32_t va[NT], vb[NT];
  uint32_t ldst;                 // LDS byte of this wave's first load in a buffer
  uint32_t ra, rb;               // byte of this lane's first A / B fragment row in a buffer
  uint32_t c0, c1;               // its chunk's byte in the row, steps 0 and 1
  int lane;
};

// Load Q of a unit (0 .. NT - 1 the A rows, then the B rows) at byte k of the rows.
template <int NT, int Q>
__device__ __forceinline__ void ring_load(const RingLane<NT>& L, uint32_t k, uint32_t buf, uint32_t back_even,
                                          uint32_t back_odd) {
  constexpr int op = Q / NT, q = Q % NT;
  const uint32_t back = (q & 1) ? back_odd : back_even;
  dma_to_lds<16>((op ? L.b : L.a) + k, (op ? L.vb[q] : L.va[q]) - back,
                 buf + L.ldst + (uint32_t)(op * 32 * NT * 128 + q * 1024));
}
template <int NT, int Q = 0>
__device__ __forceinline__ void ring_issue(const RingLane<NT>& L, uint32_t k, uint32_t buf, uint32_t back_even,
                                           uint32_t back_odd) {
  if constexpr (Q < 2 * NT) {
    ring_load<NT, Q>(L, k, buf, back_even, back_odd);
    ring_issue<NT, Q + 1>(L, k, buf, back_even, back_odd);
  }
}

// Fragment Q (0 .. NT - 1 A, then B) of step J of the unit in `buf`.
template <int NT, int J, int Q>
__device__ __forceinline__ void ring_read(RingFrag<NT>& F, const uint8_t* buf, const RingLane<NT>& L) {
  constexpr int op = Q / NT, t = Q % NT;
  const ntu4 v = *reinterpret_cast<const ntu4*>(buf + ((op ? L.rb : L.ra) + (J ? L.c1 : L.c0)) + t * 2048);
  if constexpr (op) F.b[t] = v;
  else F.a[t] = v;
}
template <int NT, int J, int Q = 0>
__device__ __forceinline__ void ring_read_all(RingFrag<NT>& F, const uint8_t* buf, const RingLane<NT>& L) {
  if constexpr (Q < 2 * NT) {
    ring_read<NT, J, Q>(F, buf, L);
    ring_read_all<NT, J, Q + 1>(F, buf, L);
  }
}

// Read q of the next step comes after MFMA ring_rd(q), from MFMA 1 on; load q of n
// after MFMA ring_ld(q, n).
template <int NT>
constexpr int ring_rd(int q) { return 1 + q * (NT * NT * 3 / 4 - 4) / (2 * NT - 1); }
template <int NT>
constexpr int ring_ld(int q) { return q * (NT * NT - 1) / (2 * NT); }

template <int NT, int NJ, int K, int Q = 0>
__device__ __forceinline__ void ring_reads_at(RingFrag<NT>& G, const uint8_t* nbuf, const RingLane<NT>& L) {
  if constexpr (Q < 2 * NT) {
    if constexpr (ring_rd<NT>(Q) == K) ring_read<NT, NJ, Q>(G, nbuf, L);
    ring_reads_at<NT, NJ, K, Q + 1>(G, nbuf, L);
  }
}
template <int NT, int K, int Q = 0>
__device__ __forceinline__ void ring_loads_at(const RingLane<NT>& L, uint32_t k, uint32_t lbuf, uint32_t be, uint32_t bo) {
  if constexpr (Q < 2 * NT) {
    if constexpr (ring_ld<NT>(Q) == K) ring_load<NT, Q>(L, k, lbuf, be, bo);
    ring_loads_at<NT, K, Q + 1>(L, k, lbuf, be, bo);
  }
}

// The MFMAs of a step with the next step's reads (READ, its step NJ from nbuf) and a
// unit's loads (LOAD) between them.
template <int EL, int NT, bool READ, int NJ, bool LOAD, int K = 0>
__device__ __forceinline__ void ring_step(typename NtTypes<EL>::acc (&acc)[NT][NT], const RingFrag<NT>& F,
                                          RingFrag<NT>& G, const uint8_t* nbuf, const RingLane<NT>& L, uint32_t k,
                                          uint32_t lbuf, uint32_t be, uint32_t bo) {
  if constexpr (K < NT * NT) {
    ring_mfma<EL>(acc[K / NT][K % NT], F.b[K % NT], F.a[K / NT]);
    if constexpr (READ) ring_reads_at<NT, NJ, K>(G, nbuf, L);
    if constexpr (LOAD) ring_loads_at<NT, K>(L, k, lbuf, be, bo);
    __builtin_amdgcn_sched_barrier(0);
    ring_step<EL, NT, READ, NJ, LOAD, K + 1>(acc, F, G, nbuf, L, k, lbuf, be, bo);
  }
}

// Chunks of the last unit past the row's end (from chunk `live` on): zero in A.
template <int NT>
__device__ __forceinline__ void ring_clip(uint8_t* buf, int live) {
  for (int r = threadIdx.x; r < 32 * NT; r += 256)
    for (int c = live; c < 8; ++c)
      *reinterpret_cast<ntu4*>(buf + r * 128 + ((c ^ ((r >> 1) & 7)) << 4)) = ntu4{0u, 0u, 0u, 0u};
  lds_barrier();
}

// Unit with REM units from it to the end (REM > NB: more than NB, loads go on).  slot,
// nslot: its buffer and the next unit's.
template <int EL, int NT, int NB, int REM, bool CLIP>
__device__ __forceinline__ void ring_unit(typename NtTypes<EL>::acc (&acc)[NT][NT], RingFrag<NT>& F0, RingFrag<NT>& F1,
                                          uint8_t* smem, uint32_t smem_lds, const RingLane<NT>& L, int slot, int nslot,
                                          uint32_t k_load, uint32_t be, uint32_t bo, int live) {
  constexpr int UNIT = 2 * 32 * NT * 128, LD = 2 * NT;
  constexpr bool more = REM > NB, next = REM > 1;
  constexpr int flying = more ? NB - 1 : REM - 1;          // units in flight behind this one
  uint8_t* buf = smem + slot * UNIT;
  uint8_t* nbuf = smem + nslot * UNIT;
  ring_step<EL, NT, true, 1, false>(acc, F0, F1, buf, L, 0, 0, 0, 0);
  if constexpr (next) {
    wait_vmcnt<(flying - 1) * LD>();
    lds_barrier();
    if (CLIP && REM == 2) ring_clip<NT>(nbuf, live);
    asm volatile("s_nop 4" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }
  ring_step<EL, NT, next, 0, more>(acc, F1, F0, nbuf, L, k_load, smem_lds + (uint32_t)(slot * UNIT), be, bo);
}

template <int EL, int NT, int NB, int REM, bool CLIP>
__device__ __forceinline__ void ring_tail(typename NtTypes<EL>::acc (&acc)[NT][NT], RingFrag<NT>& F0, RingFrag<NT>& F1,
                                          uint8_t* smem, uint32_t smem_lds, const RingLane<NT>& L, int slot, int NU,
                                          int live) {
  if constexpr (REM > 0) {
    int nslot = slot;
    if (REM <= NU) {
      nslot = slot + 1 == NB ? 0 : slot + 1;
      ring_unit<EL, NT, NB, REM, CLIP>(acc, F0, F1, smem, smem_lds, L, slot, nslot, 0, 0, 0, live);
    }
    ring_tail<EL, NT, NB, REM - 1, CLIP>(acc, F0, F1, smem, smem_lds, L, nslot, NU, live);
  }
}

// ---- small tiles: a step is a whole unit.  Its fragments (both halves) are read during
// the unit before, so that the reads' latency, longer than the few MFMAs of half a unit,
// is covered; unit U's buffer is free from the barrier at its start on.  Their MFMAs are
// the compiler's: few accumulators need no pinning, and across the branches of a short
// product it copies them, which assembly MFMAs would have to be guarded against.

template <int NT>
struct RingUnit {
  RingFrag<NT> h[2];
};

template <int NT, int Q>
__device__ __forceinline__ void ring_read2(RingUnit<NT>& G, const uint8_t* nbuf, const RingLane<NT>& L) {
  ring_read<NT, Q / (2 * NT), Q % (2 * NT)>(G.h[Q / (2 * NT)], nbuf, L);
}
template <int NT, int Q = 0>
__device__ __forceinline__ void ring_read2_all(RingUnit<NT>& G, const uint8_t* nbuf, const RingLane<NT>& L) {
  if constexpr (Q < 4 * NT) {
    ring_read2<NT, Q>(G, nbuf, L);
    ring_read2_all<NT, Q + 1>(G, nbuf, L);
  }
}
template <int NT>
constexpr int ring_rd2(int q) { return q * NT / 4; }
template <int NT, int K, int Q = 0>
__device__ __forceinline__ void ring_reads2_at(RingUnit<NT>& G, const uint8_t* nbuf, const RingLane<NT>& L) {
  if constexpr (Q < 4 * NT) {
    if constexpr (ring_rd2<NT>(Q) == K) ring_read2<NT, Q>(G, nbuf, L);
    ring_reads2_at<NT, K, Q + 1>(G, nbuf, L);
  }
}
template <int NT, int K, int Q = 0>
__device__ __forceinline__ void ring_loads2_at(const RingLane<NT>& L, uint32_t k, uint32_t lbuf, uint32_t be, uint32_t bo) {
  if constexpr (Q < 2 * NT) {
    if constexpr (NT * NT + Q * (NT * NT - 1) / (2 * NT) == K) ring_load<NT, Q>(L, k, lbuf, be, bo);
    ring_loads2_at<NT, K, Q + 1>(L, k, lbuf, be, bo);
  }
}
template <int EL, int NT, bool READ, bool LOAD, int K = 0>
__device__ __forceinline__ void ring_step2(typename NtTypes<EL>::acc (&acc)[NT][NT], const RingUnit<NT>& F,
                                           RingUnit<NT>& G, const uint8_t* nbuf, const RingLane<NT>& L, uint32_t k,
                                           uint32_t lbuf, uint32_t be, uint32_t bo) {
  if constexpr (K < 2 * NT * NT) {
    constexpr int h = K / (NT * NT), i = K % (NT * NT) / NT, j = K % NT;
    acc[i][j] = nt_mfma<EL>(F.h[h].b[j], F.h[h].a[i], acc[i][j]);
    if constexpr (LOAD) ring_loads2_at<NT, K>(L, k, lbuf, be, bo);
    if constexpr (READ) ring_reads2_at<NT, K>(G, nbuf, L);
    __builtin_amdgcn_sched_barrier(0);
    ring_step2<EL, NT, READ, LOAD, K + 1>(acc, F, G, nbuf, L, k, lbuf, be, bo);
  }
}
template <int EL, int NT, int NB, int REM, bool CLIP>
__device__ __forceinline__ void ring_unit2(typename NtTypes<EL>::acc (&acc)[NT][NT], const RingUnit<NT>& F,
                                           RingUnit<NT>& G, uint8_t* smem, uint32_t smem_lds, const RingLane<NT>& L,
                                           int& slot, uint32_t k_load, uint32_t be, uint32_t bo, int live) {
  constexpr int UNIT = 2 * 32 * NT * 128, LD = 2 * NT;
  constexpr bool more = REM > NB, next = REM > 1;
  constexpr int flying = more ? NB - 1 : REM - 1;
  const int nslot = slot + 1 == NB ? 0 : slot + 1;
  if constexpr (next) {
    wait_vmcnt<(flying - 1) * LD>();
    lds_barrier();
    if (CLIP && REM == 2) ring_clip<NT>(smem + nslot * UNIT, live);
    __builtin_amdgcn_sched_barrier(0);
  }
  ring_step2<EL, NT, next, more>(acc, F, G, smem + nslot * UNIT, L, k_load, smem_lds + (uint32_t)(slot * UNIT), be, bo);
  slot = nslot;
}
template <int EL, int NT, int NB, int REM, bool CLIP>
__device__ __forceinline__ void ring_tail2(typename NtTypes<EL>::acc (&acc)[NT][NT], RingUnit<NT>& F, RingUnit<NT>& G,
                                           uint8_t* smem, uint32_t smem_lds, const RingLane<NT>& L, int slot, int live) {
  if constexpr (REM > 0) {
    ring_unit2<EL, NT, NB, REM, CLIP>(acc, F, G, smem, smem_lds, L, slot, 0, 0, 0, live);
    ring_tail2<EL, NT, NB, REM - 1, CLIP>(acc, G, F, smem, smem_lds, L, slot, live);
  }
}
// The tail of a product of fewer units than the ring has buffers.
template <int EL, int NT, int NB, int REM, bool CLIP>
__device__ __forceinline__ void ring_short2(typename NtTypes<EL>::acc (&acc)[NT][NT], RingUnit<NT>& F, RingUnit<NT>& G,
                                            uint8_t* smem, uint32_t smem_lds, const RingLane<NT>& L, int NU, int live) {
  if constexpr (REM > 0) {
    if (NU == REM) ring_tail2<EL, NT, NB, REM, CLIP>(acc, F, G, smem, smem_lds, L, 0, live);
    else ring_short2<EL, NT, NB, REM - 1, CLIP>(acc, F, G, smem, smem_lds, L, NU, live);
  }
}

// Whether a step is a whole unit.
constexpr bool ring_whole(int nt, int nb) { return nt <= 3 || (nt == 4 && nb > 2); }

// CLIP: kb is no multiple of 128 (it is one of 16).
template <int EL, int NT, int NB, bool CLIP, typename Epi>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(160 * 1024 / ring_lds<NT, NB>(), 160 * 1024 / ring_lds<NT, NB>())))
void k_nt_ring(NtArgs g, NtGrid d, Epi epi) {
  typedef typename NtTypes<EL>::acc Acc;
  constexpr int MT = 32 * NT, S = 16 * NT, UNIT = 2 * MT * 128, LD = 2 * NT;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const uint32_t smem_lds = (uint32_t)(size_t)(__attribute__((address_space(3))) uint8_t*)smem;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = w >> 1, wn = w & 1;
  int e, tm, tn;
  nt_tile(blockIdx.x, d, g.sym, e, tm, tn);
  const int64_t m0 = (int64_t)tm * MT, n0 = (int64_t)tn * MT;
  // parts of a cut tile above the diagonal, or past the matrix
  if (d.split > 1 && ((g.sym && tn > tm) || m0 >= g.M || n0 >= g.N)) return;
  const int last_m = (int)(g.M - m0 < MT ? g.M - m0 - 1 : MT - 1), last_n = (int)(g.N - n0 < MT ? g.N - n0 - 1 : MT - 1);
  const int NU = (int)((g.kb + 127) / 128);
  RingLane<NT> L;
  L.lane = lane;
  L.a = g.a + e * g.stride_a + m0 * g.kb;
  L.b = g.b + e * g.stride_b + n0 * g.kb;
  // load q of this wave: rows w 8 NT + 8 q + (lane >> 3), slot lane & 7
  const uint32_t ce = (uint32_t)((lane & 7) ^ (((w * 8 * NT + (lane >> 3)) >> 1) & 7)) * 16u;
  const uint32_t co = (uint32_t)((lane & 7) ^ (((w * 8 * NT + 8 + (lane >> 3)) >> 1) & 7)) * 16u;
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int r = w * 8 * NT + 8 * q + (lane >> 3);
    const uint32_t c = (q & 1) ? co : ce;
    L.va[q] = (uint32_t)min(r, last_m) * g.kb + c;
    L.vb[q] = (uint32_t)min(r, last_n) * g.kb + c;
  }
  L.ldst = (uint32_t)(w * 8 * NT * 128);
  const int r16 = lane & 15, q4 = lane >> 4, sw = (r16 >> 1) & 7;
  L.ra = (uint32_t)((wm * S + r16) * 128);
  L.rb = (uint32_t)((MT + wn * S + r16) * 128);
  L.c0 = (uint32_t)((q4 ^ sw) << 4);
  L.c1 = (uint32_t)(((4 + q4) ^ sw) << 4);
  // in the last unit, lanes whose chunk lies past the row's end read its last chunk
  const int live = CLIP ? (int)(g.kb - (uint32_t)(NU - 1) * 128u) / 16 : 8;
  const uint32_t top = (uint32_t)live * 16u;
  const uint32_t be = CLIP && ce >= top ? ce - (top - 16u) : 0u, bo = CLIP && co >= top ? co - (top - 16u) : 0u;

  Acc acc[NT][NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      acc[i][j] = Acc{0, 0, 0, 0};
      if constexpr (!ring_whole(NT, NB)) asm volatile("" : "+a"(acc[i][j]));
    }
  __builtin_amdgcn_sched_barrier(0);

#pragma unroll
  for (int u = 0; u < NB; ++u)
    if (u < NU) {
      const bool end = CLIP && u == NU - 1;
      ring_issue<NT>(L, (uint32_t)u * 128u, smem_lds + (uint32_t)(u * UNIT), end ? be : 0u, end ? bo : 0u);
    }
  if (NU >= NB) wait_vmcnt<(NB - 1) * LD>();
  else wait_vmcnt<0>();
  lds_barrier();
  if (CLIP && NU == 1) ring_clip<NT>(smem, live);
  // what the first rows of accumulators add is loaded before the last units, so that the
  // epilogue does not begin with a wait for memory
  typename Epi::Row row[NT];
  typename Epi::Add add[3][NT];
  const auto ahead = [&]() {
    epi.at(e, m0 + wm * S, n0 + wn * S, r16, 4 * q4);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) epi.add(add[i][j], i, j);
#pragma unroll
    for (int i = 0; i < NT; ++i) row[i] = epi.row(i);
    __builtin_amdgcn_sched_barrier(0);
  };
  int slot = 0;
  if constexpr (ring_whole(NT, NB)) {
    RingUnit<NT> F0, F1;
    ring_read2_all<NT>(F0, smem, L);
    __builtin_amdgcn_sched_barrier(0);
    const auto unit = [&](int U, RingUnit<NT>& F, RingUnit<NT>& G) {
      const bool end = CLIP && U + NB == NU - 1;
      ring_unit2<EL, NT, NB, NB + 1, CLIP>(acc, F, G, smem, smem_lds, L, slot, (uint32_t)(U + NB) * 128u, end ? be : 0u,
                                           end ? bo : 0u, live);
    };
    int U = 0;
    for (; U + NB + 1 < NU; U += 2) {
      unit(U, F0, F1);
      unit(U + 1, F1, F0);
    }
    const bool odd = U + NB < NU;
    if (odd) unit(U, F0, F1);
    ahead();
    if (odd) {
      ring_tail2<EL, NT, NB, NB, CLIP>(acc, F1, F0, smem, smem_lds, L, slot, live);
    } else if (NU >= NB) {
      ring_tail2<EL, NT, NB, NB, CLIP>(acc, F0, F1, smem, smem_lds, L, slot, live);
    } else {
      ring_short2<EL, NT, NB, NB - 1, CLIP>(acc, F0, F1, smem, smem_lds, L, NU, live);
    }
  } else {
    RingFrag<NT> F0, F1;
    ring_read_all<NT, 0>(F0, smem, L);
    __builtin_amdgcn_sched_barrier(0);
    for (int U = 0; U + NB < NU; ++U) {
      const int nslot = slot + 1 == NB ? 0 : slot + 1;
      const bool end = CLIP && U + NB == NU - 1;
      ring_unit<EL, NT, NB, NB + 1, CLIP>(acc, F0, F1, smem, smem_lds, L, slot, nslot, (uint32_t)(U + NB) * 128u,
                                          end ? be : 0u, end ? bo : 0u, live);
      slot = nslot;
    }
    ahead();
    ring_tail<EL, NT, NB, NB, CLIP>(acc, F0, F1, smem, smem_lds, L, slot, NU, live);
  }

  // every wave is done with the ring (the epilogue reuses the LDS; no load is in
  // flight), and the last MFMAs' results have reached the accumulators
  lds_barrier();
  if constexpr (!ring_whole(NT, NB)) {
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) asm volatile("" : "+a"(acc[i][j]));
    __builtin_amdgcn_sched_barrier(0);
  }

  // 16-bit values, four columns of a row per accumulator, staged by rows; what is added
  // to a row of accumulators is loaded two rows ahead (one wave per SIMD: a load that its
  // use waits for waits alone)
  constexpr int RS = S + 4;
  uint16_t* E = reinterpret_cast<uint16_t*>(smem) + w * S * RS;
  ntu2 val[NT][NT];
  {
    typename Epi::Col col[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) col[j] = epi.col(j);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (i + 2 < NT) {
#pragma unroll
        for (int j = 0; j < NT; ++j) epi.add(add[(i + 2) % 3][j], i + 2, j);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        val[i][j] = epi.pack4(i, j, row[i], col[j], add[i % 3][j], acc[i][j]);
        *reinterpret_cast<ntu2*>(E + (i * 16 + r16) * RS + j * 16 + 4 * q4) = val[i][j];
      }
    }
  }
  // a wave stores its own part: whole row pieces, as many rows at a time as its lanes cover
  constexpr int PP = S / 8, RPI = 64 / PP, IT = (S + RPI - 1) / RPI, G = IT < 8 ? IT : 8;
  const int pr = lane / PP, pc = lane % PP * 8;
  const auto piece = [&](int row) {
    const ntu2 x = *reinterpret_cast<const ntu2*>(E + row * RS + pc), y = *reinterpret_cast<const ntu2*>(E + row * RS + pc + 4);
    return ntu4{x[0], x[1], y[0], y[1]};
  };
  const auto row_of = [&](int it) { return it * RPI + pr; };
  const auto mine = [&](int it) { return pr < RPI && it < IT && row_of(it) < S; };
  typename Epi::Fetch f[2][G];
#pragma unroll
  for (int u = 0; u < G; ++u)
    if (mine(u)) epi.fetch(f[0][u], row_of(u), pc);
  __syncthreads();
  // (loops, not unrolled further: the compiler would hold the addresses of all of them)
#pragma unroll 1
  for (int it = 0; it < IT; it += 2 * G) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int u = 0; u < G; ++u)
        if (mine(it + (h + 1) * G + u)) epi.fetch(f[1 - h][u], row_of(it + (h + 1) * G + u), pc);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < G; ++u)
        if (mine(it + h * G + u)) epi.store(row_of(it + h * G + u), pc, piece(row_of(it + h * G + u)), f[h][u]);
    }
  }
  if (Epi::kTrans && !(g.sym && tm == tn)) {
    // staged again by columns: neighbouring lanes (rows m, m + 1) exchange halves, so
    // that the even one writes the pair of columns n and n + 1, the odd one n + 2 and
    // n + 3, as dwords of two rows (read back by 16-bit columns instead, the rows'
    // stride puts four lanes on a bank: 6 us a tile more)
    __syncthreads();
    const bool odd = lane & 1;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint32_t own = odd ? val[i][j][1] : val[i][j][0], give = odd ? val[i][j][0] : val[i][j][1];
        const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)give, 0xB1, 0xF, 0xF, false);   // lane ^ 1
        const uint32_t lo = odd ? got : own, hi = odd ? own : got;        // rows m (even lane's), m + 1
        uint16_t* d = E + (j * 16 + 4 * q4 + (odd ? 2 : 0)) * RS + i * 16 + (r16 & ~1);
        *reinterpret_cast<uint32_t*>(d) = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
        *reinterpret_cast<uint32_t*>(d + RS) = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
      }
    __syncthreads();
#pragma unroll 1
    for (int it = 0; it < IT; it += G) {
#pragma unroll
      for (int u = 0; u < G; ++u)
        if (mine(it + u)) epi.store_t(row_of(it + u), pc, piece(row_of(it + u)));
    }
  }
  epi.finish(smem);
}

// ---------------------------------------------------------------- choice of kernel

// What a tile costs, in microseconds measured on an MI355X with 8-bit integers (a unit of
// FP16 takes 1.2 times as long): a unit of 128 bytes of K when all compute units are busy
// and when few are, a tile besides its units, and what the epilogue of a polynomial of the
// orthogonalisation takes on top (Epi::kWork: how many times that another one takes).
// `per_cu` workgroups share a compute unit at that cost.  On 79 random sizes that none of these
// numbers was fitted to (M 1 to 22,000, N 64 to 32,000, K 128 to 22,000) the call is within 10% of
// the best kernel on 72, at most 18% behind (37 x 21,539 x 14,464), at best 7% ahead, on two
// kernels; profiles/int8_kernel_choice.txt has each.
struct NtCost {
  int kernel, side_m, side_n, per_cu;
  float full, few, tile, work;
};
constexpr NtCost kNtCosts[] = {
    {kNtDirect16x64, 16, 64, 1, 0.29f, 0.22f, 1.9f, 0.0f}, {kNtDirect64x64, 64, 64, 1, 0.52f, 0.50f, 2.0f, 0.0f},
    {kNtRing64, 64, 64, 3, 0.49f, 0.14f, 1.8f, 1.7f},      {kNtRing96, 96, 96, 1, 0.30f, 0.235f, 2.9f, 2.1f},
    {kNtRing128, 128, 128, 2, 0.88f, 0.27f, 3.8f, 5.3f},   {kNtRing128x5, 128, 128, 1, 0.45f, 0.295f, 3.8f, 3.6f},
    {kNtRing192, 192, 192, 1, 0.83f, 0.575f, 5.9f, 6.6f},  {kNtRing256, 256, 256, 1, 1.30f, 0.77f, 9.6f, 12.7f},
};

// Which kernel computes a product: all of it (count of tiles -1), or the first `count`
// tiles, and the rest on `rest`, its tiles cut split x split times.
struct NtChoice {
  int kernel, count, rest, split;
};

inline double nt_cost(const NtCost& c, double tiles, double units, float work, int cus) {
  const double slots = (double)cus * c.per_cu;
  const double rounds = (double)(int64_t)(tiles / slots), last = tiles / slots - rounds;
  const double tile = c.tile + work * c.work;
  return rounds * (units * c.full + tile) + (last > 0 ? units * (c.few + (c.full - c.few) * last) + tile : 0.0);
}

// The choice with the least estimated time: full rounds of workgroups over the compute
// units, and a last round that is cheaper the emptier it is, or is left to smaller tiles
// in a launch of its own (4,096 x 14,336 x 8,192 in 3.5 rounds of 256: 355.8 -> 344.3 us;
// 3,000 x 7,000 x 4,096: 89.6 us on the best single kernel, 83.3 on two).
// direct, ring: which kinds there are to choose from; f16, work: the element type, and
// the epilogue's.
inline NtChoice nt_choose(const NtArgs& g, bool direct, bool ring, bool f16, float work) {
  constexpr double kLaunch = 4.0;
  const int found = device_cus(), cus = found > 0 ? found : 256;
  const double units = (double)((g.kb + 127) / 128) * (f16 ? 1.2 : 1.0);
  const double clip = g.kb % 128 != 0 ? 1.0 : 0.0;         // the last unit clipped in LDS
  NtChoice best{direct ? kNtDirect64x64 : kNtRing64, -1, 0, 1};
  double least = 1e300;
  for (const NtCost& c : kNtCosts) {
    const bool is_direct = c.kernel == kNtDirect16x64 || c.kernel == kNtDirect64x64;
    if (is_direct ? !direct : !ring) continue;
    const int64_t tiles = nt_tiles(g, c.side_m, c.side_n);
    const double us = nt_cost(c, (double)tiles, units, work, cus) + (is_direct ? 0.0 : clip);
    if (us < least) {
      least = us;
      best = NtChoice{c.kernel, -1, 0, 1};
    }
    const int64_t slots = (int64_t)cus * c.per_cu, whole = tiles / slots * slots;
    if (is_direct || whole == 0 || whole == tiles) continue;
    for (const NtCost& r : kNtCosts) {
      const bool small = r.kernel == kNtRing64 || r.kernel == kNtRing96 || r.kernel == kNtRing128 || r.kernel == kNtRing128x5;
      const int k = c.side_m / r.side_m;
      if (!small || k < 2 || k * r.side_m != c.side_m) continue;
      const double both = nt_cost(c, (double)whole, units, work, cus) + nt_cost(r, (double)((tiles - whole) * k * k), units, work, cus) +
                          kLaunch + 2 * clip;
      if (both < least) {
        least = both;
        best = NtChoice{c.kernel, (int)whole, r.kernel, k};
      }
    }
  }
  return best;
}

// kb > 0 and a multiple of 16, rows 16-byte aligned.
inline bool ring_fits(const NtArgs& g) {
  return g.kb > 0 && g.kb % 16 == 0 && g.kb < (1u << 24) &&
         ((reinterpret_cast<uintptr_t>(g.a) | reinterpret_cast<uintptr_t>(g.b)) & 15) == 0;
}

template <int EL, int NT, int NB, bool CLIP, typename Epi>
hipError_t run_nt_ring(const NtArgs& g, const NtGrid& d, const Epi& epi, hipStream_t s) {
  constexpr int LDS = ring_lds<NT, NB>();
  static_assert(LDS <= 160 * 1024, "LDS plan");
  if (!ring_fits(g) || (!CLIP && g.kb % 128 != 0) || (int64_t)d.count * d.split * d.split > 0x7FFFFFFF) return hipErrorInvalidValue;
  const void* fn = reinterpret_cast<const void*>(&k_nt_ring<EL, NT, NB, CLIP, Epi>);
  if (set_lds_limit(fn, LDS) != hipSuccess) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_nt_ring<EL, NT, NB, CLIP, Epi>), dim3((unsigned)(d.count * d.split * d.split)), dim3(256), LDS, s, g, d,
                     epi);
  return hipGetLastError();
}

template <int EL, bool CLIP, typename Epi>
hipError_t run_nt_ring_on(const NtArgs& g, int kernel, const NtGrid& d, const Epi& epi, hipStream_t s) {
  switch (kernel) {
    case kNtRing64: return run_nt_ring<EL, 2, 3, CLIP>(g, d, epi, s);
    case kNtRing96: return run_nt_ring<EL, 3, 6, CLIP>(g, d, epi, s);
    case kNtRing128: return run_nt_ring<EL, 4, 2, CLIP>(g, d, epi, s);
    case kNtRing128x5: return run_nt_ring<EL, 4, 5, CLIP>(g, d, epi, s);
    case kNtRing192: return run_nt_ring<EL, 6, 3, CLIP>(g, d, epi, s);
    case kNtRing256: return run_nt_ring<EL, 8, 2, CLIP>(g, d, epi, s);
    default: return hipErrorInvalidValue;
  }
}
inline int nt_side(int kernel) {
  for (const NtCost& c : kNtCosts)
    if (c.kernel == kernel) return c.side_n;
  return 64;
}

// The product on the ring kernels of a choice.
template <int EL, bool CLIP, typename Epi>
hipError_t run_nt_choice(const NtArgs& g, const NtChoice& c, const Epi& epi, hipStream_t s) {
  const int side = nt_side(c.kernel);
  if (nt_tiles(g, side, side) > 0x7FFFFFFF) return hipErrorInvalidValue;
  NtGrid d = nt_grid(g, side, side);
  const int all = d.count;
  if (c.count >= 0) d.count = c.count;
  const hipError_t e = d.count > 0 ? run_nt_ring_on<EL, CLIP>(g, c.kernel, d, epi, s) : hipSuccess;
  if (e != hipSuccess || d.count == all) return e;
  d.first = d.count;
  d.count = all - d.count;
  d.split = c.split;
  return run_nt_ring_on<EL, CLIP>(g, c.rest, d, epi, s);
}

}  // namespace bsq
