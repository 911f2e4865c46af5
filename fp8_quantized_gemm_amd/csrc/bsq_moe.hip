// Expert routing: the router (top-k selection, weights and the expert-ordered
// row plan), its gradient, and the tokens' way to the experts' rows and back
// (gather, combine, combine's gradient).  The contract is in include/bsq.h.
//
// The plan is deterministic: rows of an expert are in token order, then slot
// order, from counts and ranks (no atomic order is observable: the only atomics
// count integers in LDS).
#include "bsq_internal.hpp"
#include "bsq_wave.hpp"

namespace bsq {

namespace {

__device__ __forceinline__ float logit_at(const void* p, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : u2f((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

// log(sigmoid(l)) = min(l, 0) - log(1 + exp(-|l|)): finite for every finite l.
__device__ __forceinline__ float log_sigmoid(float l) {
  return fminf(l, 0.0f) - log1pf(expf(-fabsf(l)));
}
__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// One token per DPP row of 16 lanes, four tokens per wave: a lane holds NV experts
// (expert 16 j + lane in element j) and, afterwards, slot `lane` of the token
// (k <= 16).  Against one token per wave the exponentials of the k slots and the
// steps of each argmax serve four tokens, and the reductions are four steps
// instead of seven (16,381 tokens over 128 experts: 9 us against 18 us).
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, dpp_or0<0xB1, 0xF>(v));
  v = max(v, dpp_or0<0x4E, 0xF>(v));
  v = max(v, dpp_or0<0x141, 0xF>(v));
  return max(v, dpp_or0<0x140, 0xF>(v));
}
__device__ __forceinline__ uint32_t row_min(uint32_t v) { return ~row_max(~v); }
__device__ __forceinline__ float row_max_f(float v) { return float_of_key(row_max(float_key(v))); }
__device__ __forceinline__ float row_sum(float v) {
  v += u2f(dpp_or0<0xB1, 0xF>(f2u(v)));
  v += u2f(dpp_or0<0x4E, 0xF>(f2u(v)));
  v += u2f(dpp_or0<0x141, 0xF>(f2u(v)));
  return v + u2f(dpp_or0<0x140, 0xF>(f2u(v)));
}

constexpr float kNegInf = -__builtin_inff();

// Softmax over the row's lanes with `on` (0 elsewhere).
__device__ __forceinline__ float row_softmax(float l, bool on) {
  const float m = row_max_f(on ? l : kNegInf);
  const float z = on ? expf(l - m) : 0.0f;
  const float sum = row_sum(z);
  return on ? z / sum : 0.0f;
}

// Max and sum of exp(l - max) over a token's unmasked logits.
template <int NV>
__device__ __forceinline__ void full_softmax_stats(const float (&l)[NV], float& m, float& sum) {
  float lm = kNegInf;
#pragma unroll
  for (int j = 0; j < NV; ++j) lm = fmaxf(lm, l[j]);
  m = row_max_f(lm);
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) s += l[j] > kNegInf ? expf(l[j] - m) : 0.0f;
  sum = row_sum(s);
}

// A token's logits, expert 16 j + lane in element j; masked (past the last
// expert, -inf, NaN) ones as -inf.
template <int NV>
__device__ __forceinline__ void load_logits(const void* logits, bool f32, int64_t t, int experts, int lane,
                                            float (&l)[NV]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = 16 * j + lane;
    const float v = e < experts ? logit_at(logits, f32, t * experts + e) : kNegInf;
    l[j] = v > kNegInf ? v : kNegInf;              // NaN compares false
  }
}

// Selection and weight of token t: lane j < k of the row gets slot j's expert
// (-1: none left) and weight.  SCORED: the bias is added to the score (the FP32
// value the unnormalised weight has), else to the logit.
template <int NV, bool SCORED>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, int lane, const float (&bias)[NV],
                                            int& id, float& w) {
  float l[NV];                                     // read again for the softmax over all: fewer registers
  load_logits<NV>(a.logits, a.f32, t, a.experts, lane, l);
  uint32_t key[NV];
  float m = 0.0f, sum = 1.0f;
  if (SCORED && !a.sigmoid) full_softmax_stats<NV>(l, m, sum);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float s = l[j];                                // masked stays -inf
    if (SCORED && s > kNegInf) s = a.sigmoid ? sigmoid(s) : expf(s - m) / sum;
    s = (s + bias[j]) + 0.0f;                      // -0 counts as +0
    key[j] = s > kNegInf ? float_key(s) : 0u;
  }
  uint32_t mine = ~0u;
  for (int s = 0; s < a.k; ++s) {
    uint32_t best = 0, e = ~0u;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (key[j] > best) best = key[j], e = 16 * j + lane;   // the lowest of equal keys
    const uint32_t m = row_max(best);
    const uint32_t win = row_min(best == m && m != 0 ? e : ~0u);   // ... over the lanes; ~0: nothing left
    if (lane == s) mine = win;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (win == (uint32_t)(16 * j + lane)) key[j] = 0;
  }
  id = (int)mine;                                  // ~0 is -1
  const bool on = id >= 0;
  const float sel = on ? logit_at(a.logits, a.f32, t * a.experts + id) : kNegInf;
  if (a.normalize) {
    w = row_softmax(a.sigmoid && on ? log_sigmoid(sel) : sel, on);
  } else if (a.sigmoid) {
    w = on ? sigmoid(sel) : 0.0f;
  } else {
    if constexpr (!SCORED) {
      load_logits<NV>(a.logits, a.f32, t, a.experts, lane, l);
      full_softmax_stats<NV>(l, m, sum);
    }
    w = on ? expf(sel - m) / sum : 0.0f;
  }
  w = on ? a.scale * w : 0.0f;
}

constexpr int kRouteThreads = 1024, kRouteWaves = kRouteThreads / 64;

// Tokens per workgroup of the two router passes: at most 512 workgroups (each
// of the second pass reads the counts of all), 64 tokens at least.
__host__ __device__ inline int route_span(int64_t tokens) {
  const int64_t s = (tokens + 511) / 512;
  return (int)(s < 64 ? 64 : (s + 63) / 64 * 64);
}

// Selection, weights and per-expert counts of the workgroup's tokens.
template <int NV, bool SCORED>
__device__ __forceinline__ void route_select(const RouteArgs& a, int64_t t0, int64_t t1, int32_t* cnt) {
  const int lane = threadIdx.x & 15, row = threadIdx.x >> 4;
  float bias[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = 16 * j + lane;
    bias[j] = a.bias && e < a.experts ? a.bias[e] : 0.0f;
  }
  for (int64_t tb = t0; tb < t1; tb += kRouteThreads / 16) {
    const int64_t t = tb + row;
    int id;
    float w;
    route_token<NV, SCORED>(a, t < t1 ? t : t1 - 1, lane, bias, id, w);
    if (lane < a.k && t < t1) {
      a.ids[t * a.k + lane] = id;
      a.weights[t * a.k + lane] = w;
      if (id >= 0) atomicAdd(&cnt[id], 1);
    }
  }
}

// Rows of the workgroup's assignments.  before[e]: assignments of expert e in
// earlier workgroups; total[e]: in all.  The waves take consecutive spans of
// the assignments; a wave counts its span per expert, and after a prefix over
// the waves ranks its assignments 64 at a time (lanes of equal expert by
// ballots over the bits of the expert number).
struct RouteLds {
  int32_t total[kMoeMaxExperts];
  int32_t start[kMoeMaxExperts + 1];                     // padded row offsets
  int32_t run[kRouteWaves][kMoeMaxExperts];              // next row of (wave, expert)
};

__device__ __forceinline__ uint64_t lanes_of_same(int v, bool on) {
  uint64_t m = __ballot(on);
#pragma unroll
  for (int b = 0; b < 9; ++b) {                          // experts <= 512
    const uint64_t s = __ballot((v >> b) & 1);
    m &= ((v >> b) & 1) ? s : ~s;
  }
  return m;
}

// before[e] is in run[0][e] and total[] filled on entry (a barrier has passed).
__device__ __forceinline__ void route_place(const RouteArgs& a, int64_t t0, int64_t t1, RouteLds& s, bool first) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = a.experts;
  // padded offsets: exclusive prefix over the experts by the first wave
  if (wave == 0) {
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      const int n = e < E ? (s.total[e] + a.align - 1) / a.align * a.align : 0;
      int inc = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(inc, d, 64);
        if (lane >= d) inc += up;
      }
      if (e < E) s.start[e] = carry + inc - n;
      carry += __shfl(inc, 63, 64);
    }
    if (lane == 0) s.start[E] = carry;
  }
  __syncthreads();
  const int64_t n0 = t0 * a.k, n1 = t1 * a.k;
  const int64_t span = (((n1 - n0) + kRouteWaves - 1) / kRouteWaves + 63) / 64 * 64;
  const int64_t w0 = n0 + wave * span, w1 = w0 + span < n1 ? w0 + span : n1;
  for (int e = tid; e < E; e += kRouteThreads) s.run[0][e] += s.start[e];
  for (int i = tid; i < (kRouteWaves - 1) * E; i += kRouteThreads) s.run[1 + i / E][i % E] = 0;
  __syncthreads();
  // counts of wave w go to row w + 1 and are summed down the waves
  if (wave + 1 < kRouteWaves)
    for (int64_t i = w0 + lane; i < w1; i += 64) {
      const int id = a.ids[i];
      if (id >= 0) atomicAdd(&s.run[wave + 1][id], 1);
    }
  __syncthreads();
  for (int e = tid; e < E; e += kRouteThreads)
    for (int w = 1; w < kRouteWaves; ++w) s.run[w][e] += s.run[w - 1][e];
  __syncthreads();
  for (int64_t i0 = w0; i0 < w1; i0 += 64) {
    const int64_t i = i0 + lane;
    const int id = i < w1 ? a.ids[i] : -1;
    const uint64_t same = lanes_of_same(id, id >= 0);
    int row = -1;
    if (id >= 0) {
      const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
      row = s.run[wave][id] + rank;
    }
    // the reads above before the writes, the writes before the next reads
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (id >= 0 && (same >> lane) == 1) s.run[wave][id] = row + 1;   // the last lane of the expert
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (i < w1) a.row_of[i] = row;
    if (row >= 0 && row < a.rows) a.src[row] = (int32_t)i;
  }
  if (first)
    for (int e = tid; e <= E; e += kRouteThreads) a.offsets[e] = s.start[e];
}

// Rows of no assignment: the padding of each group and the rows past the last.
__device__ __forceinline__ void route_fill(const RouteArgs& a, const RouteLds& s, int blk, int nblk) {
  for (int e = blk; e < a.experts; e += nblk)
    for (int64_t r = (int64_t)s.start[e] + s.total[e] + threadIdx.x; r < s.start[e + 1]; r += kRouteThreads)
      if (r < a.rows) a.src[r] = -1;
  for (int64_t r = s.start[a.experts] + (int64_t)blk * kRouteThreads + threadIdx.x; r < a.rows;
       r += (int64_t)nblk * kRouteThreads)
    a.src[r] = -1;
}

// Everything in one workgroup (few tokens: launches cost more than the work).
template <int NV, bool SCORED>
__global__ __launch_bounds__(kRouteThreads) void k_moe_route_small(RouteArgs a) {
  __shared__ RouteLds s;
  const int tid = threadIdx.x;
  for (int e = tid; e < a.experts; e += kRouteThreads) s.total[e] = s.run[0][e] = 0;
  __syncthreads();
  route_select<NV, SCORED>(a, 0, a.tokens, s.total);
  __threadfence_block();                                 // ids written above are read below by other waves
  __syncthreads();
  route_place(a, 0, a.tokens, s, true);
  route_fill(a, s, 0, 1);
}

template <int NV, bool SCORED>
__global__ __launch_bounds__(kRouteThreads) void k_moe_select(RouteArgs a) {
  __shared__ int32_t cnt[kMoeMaxExperts];
  const int span = route_span(a.tokens);
  const int64_t t0 = (int64_t)blockIdx.x * span, t1 = t0 + span < a.tokens ? t0 + span : a.tokens;
  for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) cnt[e] = 0;
  __syncthreads();
  route_select<NV, SCORED>(a, t0, t1, cnt);
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) a.hist[(int64_t)blockIdx.x * a.experts + e] = cnt[e];
}

__global__ __launch_bounds__(kRouteThreads) void k_moe_place(RouteArgs a) {
  __shared__ RouteLds s;
  const int tid = threadIdx.x, E = a.experts, nblk = gridDim.x, blk = blockIdx.x;
  const int span = route_span(a.tokens);
  const int64_t t0 = (int64_t)blk * span, t1 = t0 + span < a.tokens ? t0 + span : a.tokens;
  for (int e = tid; e < E; e += kRouteThreads) s.total[e] = s.run[0][e] = 0;
  __syncthreads();
  // counts of all workgroups: slices of them by the threads of each expert
  const int slices = E <= kRouteThreads ? kRouteThreads / E : 1;
  const int e = tid % E, sl = tid / E;
  if (sl < slices) {
    int all = 0, before = 0;
#pragma unroll 16
    for (int b = sl; b < nblk; b += slices) {
      const int v = a.hist[(int64_t)b * E + e];
      all += v;
      before += b < blk ? v : 0;
    }
    atomicAdd(&s.total[e], all);
    atomicAdd(&s.run[0][e], before);
  }
  __syncthreads();
  route_place(a, t0, t1, s, blk == 0);
  route_fill(a, s, blk, nblk);
}

// Gradient of the weights with respect to the logits, one token per 16 lanes.
template <int NV>
__global__ __launch_bounds__(256) void k_moe_route_bwd(const void* logits, bool f32, int64_t tokens, int experts,
                                                       int k, const int32_t* __restrict__ ids,
                                                       const float* __restrict__ d_w, bool sig, bool normalize,
                                                       float scale, void* d_logits) {
  // the slots' gradients are scattered into the token's row here, each 16 lanes
  // (of one wave) their own
  __shared__ float scat[16][NV * 16];
  const int lane = threadIdx.x & 15, row = threadIdx.x >> 4;
  const bool full = !sig && !normalize;
  for (int64_t tb = (int64_t)blockIdx.x * 16; tb < tokens; tb += (int64_t)gridDim.x * 16) {
    const bool live = tb + row < tokens;
    const int64_t t = live ? tb + row : tokens - 1;
    int id = lane < k ? ids[t * k + lane] : -1;
    if ((unsigned)id >= (unsigned)experts) id = -1;
    const bool on = id >= 0;
    const float dp = on ? scale * d_w[t * k + lane] : 0.0f;
    const float sel = on ? logit_at(logits, f32, t * experts + id) : kNegInf;
    float l[NV];
    float ds = 0.0f;                                     // this lane's slot: gradient of its logit
    float mean = 0.0f, m = 0.0f, sum = 1.0f;
    if (full) {
      load_logits<NV>(logits, f32, t, experts, lane, l);
      full_softmax_stats<NV>(l, m, sum);
      const float p = on ? expf(sel - m) / sum : 0.0f;
      mean = row_sum(dp * p);
      ds = dp;                                           // joined with the rest below
    } else if (normalize) {
      const float p = row_softmax(sig && on ? log_sigmoid(sel) : sel, on);
      mean = row_sum(dp * p);
      ds = on ? p * (dp - mean) : 0.0f;
      if (sig && on) ds *= sigmoid(-sel);                // d log(sigmoid) = sigmoid(-l)
    } else if (on) {
      ds = dp * (sigmoid(sel) * sigmoid(-sel));
    }
    const bool any = row_max(on ? 1u : 0u) != 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) scat[row][16 * j + lane] = 0.0f;
    // one wave's LDS operations stay in order; the fences keep the compiler's
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (on) scat[row][id] = ds;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = 16 * j + lane;
      float d = scat[row][e];
      if (full) d = any && l[j] > kNegInf ? (expf(l[j] - m) / sum) * (d - mean) : 0.0f;
      if (live && e < experts) {
        if (f32) static_cast<float*>(d_logits)[t * experts + e] = d;
        else static_cast<uint16_t*>(d_logits)[t * experts + e] = bf16_rne(d);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// ---------------------------------------------------------------- rows to the experts and back

// Rows move in pieces of 8 columns per lane, 512 per wave (AL: 16-byte aligned
// rows; else pieces of any alignment, see load_raw).

// out[p] = x[src[p] / k], zeros where src[p] is no assignment.  A token's rows
// are far apart in expert order, so each XCD takes one of `slabs` column slabs (of
// slab pieces) over all rows, eight slabs at a time: the tokens' part of it, read k
// times, stays in its L2.  LR lanes per row, 64 / LR rows per wave; four pieces in
// flight, of as many rows (AL) or of one.  Bound by HBM writes: 8,192 tokens x 2,
// 4,096 columns into 16,896 rows 38 us, 5.5 TB/s of rows read once per token and
// written once.  Stores past the cache are 3% faster here and send the product
// that reads the rows to HBM, so they are not used.
template <bool AL, int LR>
__global__ __launch_bounds__(256) void k_moe_gather(const uint16_t* __restrict__ x, int64_t tokens, int64_t cols,
                                                    int k, const int32_t* __restrict__ src, int64_t rows,
                                                    uint16_t* __restrict__ out, int slabs, int slab) {
  constexpr int RW = 64 / LR, U = AL ? 4 : 1, V = 4 / U;
  const int lane = threadIdx.x & (LR - 1), n = (int)cols;
  const int across = slabs < 8 ? slabs : 8;
  const unsigned per = gridDim.x / slabs, q = blockIdx.x / across;
  const int c0 = (int)(q / per * across + blockIdx.x % across) * slab * 8, c1 = min(n, c0 + slab * 8);
  const int64_t wave = (int64_t)(q % per) * 4 + (threadIdx.x >> 6), nw = (int64_t)per * 4;
  for (int64_t p0 = wave * (U * RW) + (threadIdx.x & 63) / LR; p0 < rows; p0 += nw * (U * RW)) {
    const uint16_t* xr[U];
    int have[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t p = p0 + i * RW;
      int a = p < rows ? src[p] : -1;
      if (LR == 64) a = __builtin_amdgcn_readfirstlane(a);
      const int64_t t = a >= 0 ? a / k : -1;
      have[i] = t >= 0 && t < tokens ? n : 0;
      xr[i] = x + (have[i] ? t : 0) * cols;
    }
    for (int c = c0 + lane * 8; c < c1; c += V * LR * 8) {
      Raw<uint16_t> v[U][V];
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = load_raw<AL>(xr[i], c + j * LR * 8, have[i]);
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          end_piece<AL>(v[i][j], c + j * LR * 8, have[i]);
          if (p0 + i * RW < rows) store_raw<AL>(out + (p0 + i * RW) * cols, c + j * LR * 8, n, v[i][j]);
        }
    }
  }
}

// out[t] = sum over the slots j, in order, of w[t, j] y[row_of[t, j]] (w null: 1).
// One wave per token and 512 columns, the slots' pieces in flight together; bound
// by HBM.  8,192 tokens x 2, 4,096 columns: 31 us, 6.6 TB/s.
template <bool AL>
__global__ __launch_bounds__(256) void k_moe_combine(const uint16_t* __restrict__ y, int64_t rows, int64_t cols,
                                                     const int32_t* __restrict__ row_of,
                                                     const float* __restrict__ w, int64_t tokens, int k,
                                                     uint16_t* __restrict__ out) {
  const int lane = threadIdx.x & 63, n = (int)cols;
  const int64_t slabs = (cols + 511) / 512, units = tokens * slabs;
  const int64_t nw = (int64_t)gridDim.x * 4;
  for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < units; u += nw) {
    const int64_t t = u / slabs;
    const int c = (int)(u - t * slabs) * 512 + lane * 8;
    float acc[8] = {};
#pragma unroll 4
    for (int j = 0; j < k; ++j) {
      const int p = row_of[t * k + j];
      const bool on = p >= 0 && p < rows;
      const float wj = on ? (w ? w[t * k + j] : 1.0f) : 0.0f;
      Raw<uint16_t> v = load_raw<AL>(y + (on ? (int64_t)p : 0) * cols, c, on ? n : 0);
      if (on) {
        end_piece<AL>(v, c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = __builtin_fmaf(wj, raw_at(v, e), acc[e]);
      }
    }
    store8<AL>(out + t * cols, c, n, acc);
  }
}

// d_y[p] = w d_out[t], d_w[t, j] = <d_out[t], y[p]> for the assignment (t, j) of
// row p; rows of none get zeros, slots of none d_w = 0.  One wave per row: a
// row's gradient and its dot product come from one pass, and no two rows write
// one place: a row writes a slot that names it, and a slot whose row is out of
// range or names another is cleared, so every d_w is written once whatever the
// two arrays hold.  Bound by HBM: 8,192 tokens x 2, 4,096 columns 62 us, 5.5 TB/s.
template <bool AL>
__global__ __launch_bounds__(256) void k_moe_combine_bwd(const uint16_t* __restrict__ d_out,
                                                         const uint16_t* __restrict__ y, int64_t tokens,
                                                         int64_t cols, int k, const int32_t* __restrict__ src,
                                                         const int32_t* __restrict__ row_of,
                                                         const float* __restrict__ w, int64_t rows,
                                                         uint16_t* __restrict__ d_y, float* __restrict__ d_w) {
  const int lane = threadIdx.x & 63, n = (int)cols;
  const int64_t nw = (int64_t)gridDim.x * 4, slots = tokens * k;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < slots; i += nw * 64)
    if (const int r = row_of[i]; r < 0 || r >= rows || src[r] != i) d_w[i] = 0.0f;
  for (int64_t p = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); p < rows; p += nw) {
    const int a = __builtin_amdgcn_readfirstlane(src[p]);
    const bool on = a >= 0 && a < slots;
    const int64_t t = on ? a / k : 0;
    const float wa = on ? w[a] : 0.0f;
    const bool own = on && row_of[a] == p;
    const uint16_t *g = d_out + t * cols, *yr = y + p * cols;
    const int have = on ? n : 0;
    uint16_t* o = d_y + p * cols;
    float dot = 0.0f;
    for (int c = lane * 8; c < n; c += 2 * 512) {
      Raw<uint16_t> gv[2], yv[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        gv[i] = load_raw<AL>(g, c + i * 512, have);
        yv[i] = load_raw<AL>(yr, c + i * 512, have);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        end_piece<AL>(gv[i], c + i * 512, have);
        end_piece<AL>(yv[i], c + i * 512, have);
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = raw_at(gv[i], e);
          dot = __builtin_fmaf(v, raw_at(yv[i], e), dot);
          z[e] = v * wa;
        }
        store8<AL>(o, c + i * 512, n, z);
      }
    }
    dot = wave_sum(dot);
    if (own && lane == 0) d_w[a] = dot;
  }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Workgroups for `waves` waves of work, four per workgroup, at most 64 per
// compute unit (against 8, with whole rows left over for some: combine of 8,192 x
// 2 rows of 4,096 30.4 us against 31.3, its gradient 61.9 against 62.9).
unsigned wave_grid(int64_t waves) {
  const int64_t n = (waves + 3) / 4, cap = (int64_t)(device_cus() > 0 ? device_cus() : 256) * 64;
  return (unsigned)(n < cap ? n : cap);
}

}  // namespace

int64_t moe_route_hist_bytes(int64_t tokens, int experts) {
  const int span = route_span(tokens);
  const int64_t blocks = (tokens + span - 1) / span;
  return blocks > 1 ? blocks * experts * (int64_t)sizeof(int32_t) : 0;
}

namespace {

template <bool SCORED>
hipError_t run_route(const RouteArgs& a, hipStream_t s) {
  const int span = route_span(a.tokens);
  const unsigned blocks = (unsigned)((a.tokens + span - 1) / span);
#define BSQ_ROUTE(NV)                                                                              \
  if (blocks <= 1) {                                                                                \
    hipLaunchKernelGGL((k_moe_route_small<NV, SCORED>), dim3(1), dim3(kRouteThreads), 0, s, a);      \
    return hipGetLastError();                                                                       \
  }                                                                                                 \
  hipLaunchKernelGGL((k_moe_select<NV, SCORED>), dim3(blocks), dim3(kRouteThreads), 0, s, a)
  if (a.experts <= 16) { BSQ_ROUTE(1); }
  else if (a.experts <= 32) { BSQ_ROUTE(2); }
  else if (a.experts <= 64) { BSQ_ROUTE(4); }
  else if (a.experts <= 128) { BSQ_ROUTE(8); }
  else if (a.experts <= 256) { BSQ_ROUTE(16); }
  else { BSQ_ROUTE(32); }
#undef BSQ_ROUTE
  hipLaunchKernelGGL(k_moe_place, dim3(blocks), dim3(kRouteThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t s) {
  return a.scored ? run_route<true>(a, s) : run_route<false>(a, s);
}

hipError_t launch_moe_route_bwd(const void* logits, bool f32, int64_t tokens, int experts, int k,
                                const int32_t* ids, const float* d_w, bool sigmoid, bool normalize,
                                float scale, void* d_logits, hipStream_t s) {
  const dim3 grid(wave_grid((tokens + 3) / 4)), block(256);
#define BSQ_BWD(NV)                                                                                  \
  hipLaunchKernelGGL(k_moe_route_bwd<NV>, grid, block, 0, s, logits, f32, tokens, experts, k, ids, d_w, \
                     sigmoid, normalize, scale, d_logits)
  if (experts <= 16) BSQ_BWD(1);
  else if (experts <= 32) BSQ_BWD(2);
  else if (experts <= 64) BSQ_BWD(4);
  else if (experts <= 128) BSQ_BWD(8);
  else if (experts <= 256) BSQ_BWD(16);
  else BSQ_BWD(32);
#undef BSQ_BWD
  return hipGetLastError();
}

hipError_t launch_moe_gather(const void* x, int64_t tokens, int64_t cols, int k, const int32_t* src,
                             int64_t rows, void* out, hipStream_t s) {
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  uint16_t* op = static_cast<uint16_t*>(out);
  const bool al = cols % 8 == 0 && al16(x) && al16(out);
  // Column slabs where no two share a 128-byte line (4,093 tokens x 4 of 2,048:
  // 16.6 us against 20.8 with whole rows; odd widths lose 3-13%, their lines being
  // written from two XCDs), as narrow as keeps the tokens' part in 3 MiB of an L2
  // (8,192 x 6 of 2,048: 43 us in 16 slabs, 50 in 8), but at least 128 columns
  // (16,384 x 8 of 2,048: 207 us in 32 slabs, 140 in 8) and only while the output
  // fits the 256 MiB behind the L2s, past which short pieces cost more than they
  // save (8,192 x 16 of 2,048, 545 MB: 162 us in 16 slabs, 132 in 8).
  int slabs = 1;
  if (al && cols % 64 == 0 && (reinterpret_cast<uintptr_t>(out) & 127) == 0) {
    slabs = cols >= 1024 ? 8 : cols >= 512 ? 4 : cols >= 256 ? 2 : 1;
    if (slabs == 8 && rows * cols * 2 <= (int64_t)256 << 20) {
      int64_t m = 1;
      const auto fits = [&] { return tokens * cols * 2 <= 8 * m * ((int64_t)3 << 20); };
      while (!fits() && cols / (8 * m) >= 256) m *= 2;
      if (fits()) slabs = (int)(8 * m);
    }
  }
  const int slab = (int)((cols + 64 * (int64_t)slabs - 1) / (64 * (int64_t)slabs)) * 8;
#define BSQ_GATHER(LR)                                                                              \
  {                                                                                                  \
    const dim3 grid(wave_grid((rows + 256 / LR - 1) / (256 / LR)) * slabs), block(256);               \
    if (al)                                                                                          \
      hipLaunchKernelGGL((k_moe_gather<true, LR>), grid, block, 0, s, xp, tokens, cols, k, src, rows, op, slabs, slab);  \
    else                                                                                             \
      hipLaunchKernelGGL((k_moe_gather<false, LR>), grid, block, 0, s, xp, tokens, cols, k, src, rows, op, slabs, slab); \
  }
  if (slab <= 8) BSQ_GATHER(8)
  else if (slab <= 16) BSQ_GATHER(16)
  else if (slab <= 32) BSQ_GATHER(32)
  else BSQ_GATHER(64)
#undef BSQ_GATHER
  return hipGetLastError();
}

hipError_t launch_moe_combine(const void* y, int64_t rows, int64_t cols, const int32_t* row_of,
                              const float* w, int64_t tokens, int k, void* out, hipStream_t s) {
  const uint16_t* yp = static_cast<const uint16_t*>(y);
  uint16_t* op = static_cast<uint16_t*>(out);
  const dim3 grid(wave_grid(tokens * ((cols + 511) / 512))), block(256);
  if (cols % 8 == 0 && al16(y) && al16(out))
    hipLaunchKernelGGL(k_moe_combine<true>, grid, block, 0, s, yp, rows, cols, row_of, w, tokens, k, op);
  else
    hipLaunchKernelGGL(k_moe_combine<false>, grid, block, 0, s, yp, rows, cols, row_of, w, tokens, k, op);
  return hipGetLastError();
}

hipError_t launch_moe_combine_bwd(const void* d_out, const void* y, int64_t tokens, int64_t cols, int k,
                                  const int32_t* src, const int32_t* row_of, const float* w,
                                  int64_t rows, void* d_y, float* d_w, hipStream_t s) {
  const dim3 grid(wave_grid(rows > 0 ? rows : 1)), block(256);
  const uint16_t *gp = static_cast<const uint16_t*>(d_out), *yp = static_cast<const uint16_t*>(y);
  uint16_t* op = static_cast<uint16_t*>(d_y);
  if (cols % 8 == 0 && al16(d_out) && al16(y) && al16(d_y))
    hipLaunchKernelGGL(k_moe_combine_bwd<true>, grid, block, 0, s, gp, yp, tokens, cols, k, src, row_of, w, rows, op, d_w);
  else
    hipLaunchKernelGGL(k_moe_combine_bwd<false>, grid, block, 0, s, gp, yp, tokens, cols, k, src, row_of, w, rows, op, d_w);
  return hipGetLastError();
}

}  // namespace bsq
