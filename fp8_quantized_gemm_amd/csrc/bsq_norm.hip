// Norms around a block with its gate and residual scale, and their gradient:
//   n = o * rstd_o * w_post,  r = alpha * x + g . n,  h = r * rstd_r * w_pre
// with rstd_v = 1 / sqrt(mean(v^2) + eps) over a row.  The contract is in
// include/bsq.h.  Everything is FP32 between the loads and one rounding at each
// store; h is taken from r before its rounding.
//
// Both directions are one pass over the rows (HBM-bound): a group of TPR
// threads holds one row in registers, CH pieces of 8 columns per thread, so x, o
// (forward) and d_r, d_h, r, o (backward) are read once.  Workgroups walk the
// rows, so the weights of a thread's columns stay in registers, and load the next
// row while the current one is reduced.
#include "bsq_internal.hpp"
#include "bsq_wave.hpp"

namespace bsq {

namespace {

// Weights of a piece, `fill` where there are none.
template <bool AL>
__device__ __forceinline__ void load_w(const float* w, int col, int cols, float fill, float (&y)[8]) {
  if (!w) {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = fill;
    return;
  }
  Raw<float> r = load_raw<AL>(w, col, cols);
  end_piece<AL>(r, col, cols);
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = raw_at(r, j);
}

// Sum over the 16 lanes of a DPP row or, with L 32, two of them, in every lane.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  v += u2f(dpp_or0<0xB1, 0xF>(f2u(v)));
  v += u2f(dpp_or0<0x4E, 0xF>(f2u(v)));
  v += u2f(dpp_or0<0x141, 0xF>(f2u(v)));
  v += u2f(dpp_or0<0x140, 0xF>(f2u(v)));
  if constexpr (L == 32) v += __shfl_xor(v, 16, 64);
  return v;
}

// Sums of NV values over the TPR threads of a row group, in every thread of it.
// red: LDS of [NV][waves of the block], a different one for successive calls
// (the caller alternates), so one barrier per call suffices.
template <int TPR, int NV>
__device__ __forceinline__ void group_sum(float (&v)[NV], float* red) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (TPR < 64) v[i] = lanes_sum<TPR>(v[i]);
    else v[i] = wave_sum(v[i]);
  }
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int wave = threadIdx.x >> 6, g0 = wave / W * W;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) red[i * 16 + wave] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += red[i * 16 + g0 + w];
      v[i] = s;
    }
  }
}

// ---------------------------------------------------------------- forward

// At least 256 threads per workgroup: BT / TPR rows at a time, grid-stride.
template <typename T, bool AL, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR, 4) void k_block_norm(NormFwd a) {
  constexpr int BT = TPR < 256 ? 256 : TPR, RPB = BT / TPR;
  __shared__ float red[2][16];
  __shared__ uint32_t mred[16];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int cols = (int)a.cols;
  const float inv = 1.0f / (float)cols;
  const bool has_o = a.o != nullptr, both = a.w_pre && a.w_post;
  const T* x = static_cast<const T*>(a.x);
  const uint16_t* o = static_cast<const uint16_t*>(a.o);
  const uint16_t* gf = a.gate_kind == kGateFull ? static_cast<const uint16_t*>(a.gate) : nullptr;
  const auto col = [&](int c) { return (c * TPR + t) * 8; };
  // the columns' weights: w_post times a channel gate, and w_pre
  float wq[CH][8], wp[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    load_w<AL>(a.w_post, col(c), cols, 1.0f, wq[c]);
    load_w<AL>(a.w_pre, col(c), cols, 0.0f, wp[c]);
    if (a.gate_kind == kGateChannel) {
      float g[8];
      load_w<AL>(static_cast<const float*>(a.gate), col(c), cols, 1.0f, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) wq[c][j] *= g[j];
    }
  }
  Raw<T> xr[CH];
  Raw<uint16_t> orow[CH], gr[CH];
  const auto load = [&](int64_t b) {
    const int64_t row = b * RPB + sub, base = (row < a.rows ? row : a.rows - 1) * a.cols;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      xr[c] = load_raw<AL>(x + base, col(c), cols);
      if (has_o) orow[c] = load_raw<AL>(o + base, col(c), cols);
      if (gf) gr[c] = load_raw<AL>(gf + base, col(c), cols);
    }
  };
  uint32_t hmax = 0;
  const int64_t trips = (a.rows + RPB - 1) / RPB;
  int64_t b = blockIdx.x;
  if (b < trips) load(b);
  while (b < trips) {
    const int64_t row = b * RPB + sub;
    const bool live = row < a.rows;
    const int64_t base = (live ? row : a.rows - 1) * a.cols;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      end_piece<AL>(xr[c], col(c), cols);
      if (has_o) end_piece<AL>(orow[c], col(c), cols);
      if (gf) end_piece<AL>(gr[c], col(c), cols);
    }
    float r[CH][8];
    float rq = 1.0f;
    if (a.w_post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v = raw_at(orow[c], j);
          s[0] = __builtin_fmaf(v, v, s[0]);
        }
#pragma unroll
      for (int c = 0; c < CH; ++c) forget(orow[c]);
      group_sum<TPR, 1>(s, red[0]);
      rq = 1.0f / __builtin_sqrtf(s[0] * inv + a.eps);
      if (live && t == 0 && a.rstd_post) a.rstd_post[row] = rq;
    }
    if (a.gate_kind == kGateRow) rq *= static_cast<const float*>(a.gate)[live ? row : a.rows - 1];
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v = raw_at(xr[c], j);
        if (has_o) {
          float n = raw_at(orow[c], j) * rq * wq[c][j];
          if (gf) n *= raw_at(gr[c], j);
          v = __builtin_fmaf(a.alpha, v, n);
        }
        r[c][j] = v;
        s[0] = __builtin_fmaf(v, v, s[0]);
      }
    const int64_t next = b + gridDim.x;
    if (next < trips) load(next);                     // in flight during the second reduction and the stores
    if (has_o && live) {
#pragma unroll
      for (int c = 0; c < CH; ++c) store8<AL>(static_cast<T*>(a.r) + base, col(c), cols, r[c]);
    }
    if (a.w_pre) {
      group_sum<TPR, 1>(s, red[1]);
      const float rs = 1.0f / __builtin_sqrtf(s[0] * inv + a.eps);
      if (live && t == 0 && a.rstd_pre) a.rstd_pre[row] = rs;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          y[j] = r[c][j] * rs * wp[c][j];
          // amax of the stored values: rounding to BF16 is monotone, so the
          // rounding of the maximum is the maximum of the rounded
          if (live) hmax = max(hmax, f2u(y[j]) & 0x7FFFFFFFu);
        }
        if (live) store8<AL>(static_cast<uint16_t*>(a.h) + base, col(c), cols, y);
      }
    }
    // red[0] and red[1] are each written once per trip, with the other's barrier
    // in between only when both norms run
    if (TPR > 64 && !both) __syncthreads();
    b = next;
  }
  if (a.amax) {
    hmax = wave_max_dpp(hmax);
    if ((threadIdx.x & 63) == 0) mred[threadIdx.x >> 6] = hmax;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < BT / 64; ++i) hmax = max(hmax, mred[i]);
      const float m = u2f((uint32_t)bf16_rne(u2f(hmax)) << 16);
      if (gridDim.x == 1) *a.amax = m;                // no other writer: no clearing launch before
      else atomicMax(reinterpret_cast<unsigned int*>(a.amax), f2u(m));
    }
  }
}

// ---------------------------------------------------------------- backward

// One pass over the rows, each workgroup BT / TPR rows at a time.  With G, rn, on
// as in include/bsq.h, two column sums carry all column gradients:
//   d_w_pre = sum d_h rn;  T = sum G on (times a row or full gate):
//   d_w_post = g T and d_gate = w_post T for a channel gate.
// They stay in registers over all rows of the workgroup and go to the workspace
// once, [workgroup][2][cols]; k_col_sum adds them in workgroup order (no atomics:
// repeated calls give the same bits).
// The two row means need one reduction only: with q = g w_post on,
//   G = d_r + rs (a - rn m1),  m1 = mean(a rn)
//   mean(G q) = mean(d_r q) + rs (mean(a q) - m1 mean(rn q)).
template <typename T, bool AL, int TPR, int CH>
__global__ __launch_bounds__(TPR < 512 ? 512 : TPR, CH > 1 ? 2 : 4) void k_block_norm_bwd(NormBwd a) {
  constexpr int BT = TPR < 512 ? 512 : TPR, RPB = BT / TPR;
  __shared__ float red[2][4 * 16];
  // CH 1: [8][BT], the fold over the row groups.  CH 2: the columns' weights
  // ([2][CH][2][BT] of float4, a thread's own), whose registers would spill.
  extern __shared__ __attribute__((aligned(16))) float fold[];
  float4* held = reinterpret_cast<float4*>(fold);
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int cols = (int)a.cols;
  const float inv = 1.0f / (float)cols;
  const bool has_o = a.o != nullptr, pre = a.w_pre != nullptr, post = a.w_post != nullptr;
  const T *d_r = static_cast<const T*>(a.d_r), *r = static_cast<const T*>(a.r);
  const uint16_t *d_h = static_cast<const uint16_t*>(a.d_h), *o = static_cast<const uint16_t*>(a.o);
  const uint16_t* gf = a.gate_kind == kGateFull ? static_cast<const uint16_t*>(a.gate) : nullptr;
  // two ones: with more than one piece a missing full gate is all ones, because a
  // choice per piece kept all pieces' gates unpacked (91 spilled registers)
  constexpr uint32_t kOnes = 0x3F803F80u;
  const auto col = [&](int c) { return (c * TPR + t) * 8; };
  // the columns' weights: in registers with one piece per thread, in LDS with two
  float wq1[8], wp1[8], sp[CH][8], st[CH][8];
  const auto hold = [&](int k, int c, const float (&v)[8]) {
    held[((k * CH + c) * 2) * BT + threadIdx.x] = make_float4(v[0], v[1], v[2], v[3]);
    held[((k * CH + c) * 2 + 1) * BT + threadIdx.x] = make_float4(v[4], v[5], v[6], v[7]);
  };
  const auto take = [&](int k, int c, float (&v)[8]) {
    const float4 x = held[((k * CH + c) * 2) * BT + threadIdx.x], y = held[((k * CH + c) * 2 + 1) * BT + threadIdx.x];
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
  };
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    load_w<AL>(a.w_post, col(c), cols, 1.0f, wq1);
    load_w<AL>(a.w_pre, col(c), cols, 0.0f, wp1);
    if (a.gate_kind == kGateChannel) {
      float g[8];
      load_w<AL>(static_cast<const float*>(a.gate), col(c), cols, 1.0f, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) wq1[j] *= g[j];
    }
    if constexpr (CH > 1) {
      hold(0, c, wq1);
      hold(1, c, wp1);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sp[c][j] = st[c][j] = 0.0f;
  }
  int par = 0;
  const int64_t trips = (a.rows + RPB - 1) / RPB;
  for (int64_t b = blockIdx.x; b < trips; b += gridDim.x, par ^= 1) {
    const int64_t row = b * RPB + sub;
    const bool live = RPB == 1 || row < a.rows;
    const int64_t rw = live ? row : a.rows - 1;
    const int64_t base = rw * a.cols;
    Raw<T> dr[CH], rr[CH];
    Raw<uint16_t> dh[CH], orow[CH], gr[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (d_r) {
        dr[c] = load_raw<AL>(d_r + base, col(c), cols);
      } else {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) dr[c].v[i] = u32x4{0u, 0u, 0u, 0u};
      }
      if (pre) {
        dh[c] = load_raw<AL>(d_h + base, col(c), cols);
        rr[c] = load_raw<AL>(r + base, col(c), cols);
      } else {
        dh[c].v[0] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) rr[c].v[i] = u32x4{0u, 0u, 0u, 0u};
      }
      if (has_o) orow[c] = load_raw<AL>(o + base, col(c), cols);
      else orow[c].v[0] = u32x4{0u, 0u, 0u, 0u};
      if (gf) gr[c] = load_raw<AL>(gf + base, col(c), cols);
      else if (CH > 1) gr[c].v[0] = u32x4{kOnes, kOnes, kOnes, kOnes};
    }
    const float rs = pre ? a.rstd_pre[rw] : 0.0f;
    const float rp = post ? a.rstd_post[rw] : 1.0f;
    const float grow = a.gate_kind == kGateRow ? static_cast<const float*>(a.gate)[rw] : 1.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (d_r) end_piece<AL>(dr[c], col(c), cols);
      if (pre) end_piece<AL>(dh[c], col(c), cols);
      if (pre) end_piece<AL>(rr[c], col(c), cols);
      if (has_o) end_piece<AL>(orow[c], col(c), cols);
      if (gf) end_piece<AL>(gr[c], col(c), cols);
    }
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if constexpr (CH > 1) {
        asm volatile("" ::: "memory");                   // one piece at a time: fewer registers
        __builtin_amdgcn_sched_barrier(0);
        take(0, c, wq1);
        take(1, c, wp1);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float h = raw_at(dh[c], j), rn = raw_at(rr[c], j) * rs, av = h * wp1[j];
        float q = raw_at(orow[c], j) * rp * wq1[j];
        if (CH > 1 || gf) q *= raw_at(gr[c], j);
        s[0] = __builtin_fmaf(av, rn, s[0]);
        s[1] = __builtin_fmaf(raw_at(dr[c], j), q, s[1]);
        s[2] = __builtin_fmaf(av, q, s[2]);
        s[3] = __builtin_fmaf(rn, q, s[3]);
      }
      // rows past the last add nothing to the column sums (a factor of 0 would
      // turn the last row's infinities into NaN)
      if (live) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sp[c][j] = __builtin_fmaf(raw_at(dh[c], j), raw_at(rr[c], j) * rs, sp[c][j]);
      }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      forget(dr[c]);
      forget(rr[c]);
      forget(dh[c]);
      forget(orow[c]);
      if (CH > 1 || gf) forget(gr[c]);
    }
    group_sum<TPR, 4>(s, red[par]);
    const float m1 = s[0] * inv;
    const float tot = s[1] + rs * (s[2] - m1 * s[3]);   // sum of G q, a row gate left out
    const float m2 = tot * grow * inv;
    if (a.gate_kind == kGateRow && live && t == 0) static_cast<float*>(a.d_gate)[row] = tot;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if constexpr (CH > 1) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        take(0, c, wq1);
        take(1, c, wp1);
      }
      float y[8], z[8], dg[8], Gg[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float av = raw_at(dh[c], j) * wp1[j], rn = raw_at(rr[c], j) * rs;
        const float G = __builtin_fmaf(rs, __builtin_fmaf(-m1, rn, av), raw_at(dr[c], j));
        y[j] = has_o ? a.alpha * G : G;
        const float on = raw_at(orow[c], j) * rp;
        const float g = CH > 1 ? raw_at(gr[c], j) * grow : gf ? raw_at(gr[c], j) : grow;
        Gg[j] = G * g;
        dg[j] = G * wq1[j] * on;                        // full gate
        z[j] = Gg[j] * wq1[j];
        if (post) z[j] = rp * __builtin_fmaf(-m2, on, z[j]);
      }
      if (live) {
#pragma unroll
        for (int j = 0; j < 8; ++j) st[c][j] = __builtin_fmaf(Gg[j], raw_at(orow[c], j) * rp, st[c][j]);
        store8<AL>(static_cast<T*>(a.d_x) + base, col(c), cols, y);
        if (has_o) store8<AL>(static_cast<uint16_t*>(a.d_o) + base, col(c), cols, z);
        if (gf) store8<AL>(static_cast<uint16_t*>(a.d_gate) + base, col(c), cols, dg);
      }
    }
  }
  // fold the row groups of the workgroup in LDS, then one partial row each
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k == 0 ? !pre : !has_o) continue;
      float (&v)[8] = k == 0 ? sp[c] : st[c];
      if constexpr (RPB > 1) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) fold[j * BT + threadIdx.x] = v[j];
        __syncthreads();
        if (sub == 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float f = 0.0f;
            for (int q = 0; q < RPB; ++q) f += fold[j * BT + q * TPR + t];
            v[j] = f;
          }
        }
      }
      if (sub == 0) store8<AL>(a.part + ((int64_t)blockIdx.x * 2 + k) * a.cols, col(c), cols, v);
    }
  }
}

// Sums of the nblk partials in order: 16 slices of them by the 16 waves of a
// workgroup, folded in slice order.  blockIdx.y 0: d_w_pre; 1: T, from which
// d_w_post (times a channel gate) and a channel gate's gradient (times w_post).
__global__ __launch_bounds__(1024) void k_col_sum(const float* __restrict__ part, int nblk, int64_t cols,
                                                  float* d_w_pre, float* d_w_post, float* d_gate,
                                                  const float* w_post, const float* gate) {
  __shared__ float s[16][64];
  if (blockIdx.y == 0 ? !d_w_pre : !d_w_post && !d_gate) return;
  const int lane = threadIdx.x & 63, sl = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  const int per = (nblk + 15) / 16, b0 = sl * per, b1 = min(nblk, b0 + per);
  float v = 0.0f;
  if (c < cols) {
    const float* p = part + (int64_t)blockIdx.y * cols + c;
#pragma unroll 8
    for (int b = b0; b < b1; ++b) v += p[(int64_t)b * 2 * cols];
  }
  s[sl][lane] = v;
  __syncthreads();
  if (sl != 0 || c >= cols) return;
  for (int i = 1; i < 16; ++i) v += s[i][lane];
  if (blockIdx.y == 0) {
    d_w_pre[c] = v;
  } else {
    if (d_w_post) d_w_post[c] = gate ? gate[c] * v : v;
    if (d_gate) d_gate[c] = w_post ? w_post[c] * v : v;
  }
}

// Threads per row and 8-column pieces per thread (the backward turns 1,024 x 2 into
// 512 x 4, whose 256 registers per thread hold the column sums: 4,096 x 16,384,
// BF16, 314 us -> 178 us).
struct NormCfg {
  int tpr, ch;
};
NormCfg norm_cfg(int64_t cols) {
  if (cols <= 128) return {16, 1};
  if (cols <= 256) return {32, 1};
  if (cols <= 512) return {64, 1};
  if (cols <= 1024) return {128, 1};
  if (cols <= 2048) return {256, 1};
  if (cols <= 4096) return {512, 1};
  if (cols <= 8192) return {1024, 1};
  return {1024, 2};
}

template <typename T, bool AL, int TPR, int CH>
hipError_t run_fwd(const NormFwd& a, hipStream_t s) {
  constexpr int BT = TPR < 256 ? 256 : TPR, RPB = BT / TPR;
  const int64_t trips = (a.rows + RPB - 1) / RPB;
  const int64_t cap = (int64_t)device_cus() * (BT < 1024 ? 1536 / BT : 2);
  // an amax of two trips: one workgroup, which needs no clearing launch (2 rows of
  // 4,096: 11.7 against 14.9 us a call, 4.2 against 4.8 us in a graph; 3 rows take
  // longer in a graph, 5.5 against 4.8)
  const unsigned grid = a.amax && trips <= 2 ? 1 : (unsigned)(trips < cap || cap <= 0 ? trips : cap);
  if (a.amax && grid > 1) {
    const hipError_t e = launch_zero_amax(a.amax, nullptr, s);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_block_norm<T, AL, TPR, CH>), dim3(grid), dim3(BT), 0, s, a);
  return hipGetLastError();
}

template <typename T, bool AL>
hipError_t pick_fwd(const NormFwd& a, hipStream_t s) {
  const NormCfg c = norm_cfg(a.cols);
  if (c.tpr == 16) return run_fwd<T, AL, 16, 1>(a, s);
  if (c.tpr == 32) return run_fwd<T, AL, 32, 1>(a, s);
  if (c.tpr == 64) return run_fwd<T, AL, 64, 1>(a, s);
  if (c.tpr == 128) return run_fwd<T, AL, 128, 1>(a, s);
  if (c.tpr == 256) return run_fwd<T, AL, 256, 1>(a, s);
  if (c.tpr == 512) return run_fwd<T, AL, 512, 1>(a, s);
  return c.ch == 1 ? run_fwd<T, AL, 1024, 1>(a, s) : run_fwd<T, AL, 1024, 2>(a, s);
}

template <typename T, bool AL, int TPR, int CH>
hipError_t run_bwd(const NormBwd& a, unsigned grid, hipStream_t s) {
  constexpr int BT = TPR < 512 ? 512 : TPR;
  constexpr int LDS = CH > 1 ? 2 * CH * 8 * BT * 4 : BT > TPR ? BT * 8 * 4 : 0;
  const void* fn = reinterpret_cast<const void*>(&k_block_norm_bwd<T, AL, TPR, CH>);
  if (LDS > 64 * 1024 && set_lds_limit(fn, LDS) != hipSuccess) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_block_norm_bwd<T, AL, TPR, CH>), dim3(grid), dim3(BT), LDS, s, a);
  return hipGetLastError();
}

template <typename T, bool AL>
hipError_t pick_bwd(const NormBwd& a, unsigned grid, hipStream_t s) {
  const NormCfg c = norm_cfg(a.cols);
  if (c.tpr == 16) return run_bwd<T, AL, 16, 1>(a, grid, s);
  if (c.tpr == 32) return run_bwd<T, AL, 32, 1>(a, grid, s);
  if (c.tpr == 64) return run_bwd<T, AL, 64, 1>(a, grid, s);
  if (c.tpr == 128) return run_bwd<T, AL, 128, 1>(a, grid, s);
  if (c.tpr == 256) return run_bwd<T, AL, 256, 1>(a, grid, s);
  if (c.tpr == 512) return run_bwd<T, AL, 512, 1>(a, grid, s);
  return c.ch == 1 ? run_bwd<T, AL, 1024, 1>(a, grid, s) : run_bwd<T, AL, 512, 4>(a, grid, s);
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Workgroups of the backward pass: at most 512 (two per compute unit of the
// 256; one where the weights fill its LDS), so that the partial column sums
// stay small next to the tensors.
unsigned bwd_grid(int64_t rows, int64_t cols) {
  const NormCfg c = norm_cfg(cols);
  const int rpb = (c.tpr < 512 ? 512 : c.tpr) / c.tpr;
  const int64_t trips = (rows + rpb - 1) / rpb, most = c.ch > 1 ? 256 : 512;
  return (unsigned)(trips < most ? trips : most);
}

}  // namespace

hipError_t launch_block_norm(const NormFwd& a, hipStream_t s) {
  const bool vec = a.cols % 8 == 0 && al16(a.x) && al16(a.o) && al16(a.w_post) && al16(a.w_pre) && al16(a.r) &&
                   al16(a.h) && (a.gate_kind == kGateNone || a.gate_kind == kGateRow || al16(a.gate));
  if (a.f32) return vec ? pick_fwd<float, true>(a, s) : pick_fwd<float, false>(a, s);
  return vec ? pick_fwd<uint16_t, true>(a, s) : pick_fwd<uint16_t, false>(a, s);
}

int64_t block_norm_bwd_part_bytes(int64_t rows, int64_t cols) {
  return (int64_t)bwd_grid(rows, cols) * 2 * cols * (int64_t)sizeof(float);
}

hipError_t launch_block_norm_bwd(const NormBwd& a, hipStream_t s) {
  const bool full = a.gate_kind == kGateFull, chan = a.gate_kind == kGateChannel;
  const bool vec = a.cols % 8 == 0 && al16(a.r) && al16(a.o) && al16(a.d_r) && al16(a.d_h) && al16(a.w_post) &&
                   al16(a.w_pre) && al16(a.d_x) && al16(a.d_o) && al16(a.part) &&
                   (!(full || chan) || al16(a.gate)) && (!full || al16(a.d_gate));
  const unsigned grid = bwd_grid(a.rows, a.cols);
  hipError_t e = hipSuccess;
  if (a.rows > 0) {                                 // the column sums of no rows are zero
    if (a.f32) e = vec ? pick_bwd<float, true>(a, grid, s) : pick_bwd<float, false>(a, grid, s);
    else e = vec ? pick_bwd<uint16_t, true>(a, grid, s) : pick_bwd<uint16_t, false>(a, grid, s);
  }
  if (e != hipSuccess) return e;
  float* d_gate = chan ? static_cast<float*>(a.d_gate) : nullptr;
  if (a.d_w_pre || a.d_w_post || d_gate)
    hipLaunchKernelGGL(k_col_sum, dim3((unsigned)((a.cols + 63) / 64), 2), dim3(1024), 0, s, a.part,
                       a.rows > 0 ? (int)grid : 0, a.cols, a.d_w_pre, a.d_w_post, d_gate, a.w_post,
                       chan ? static_cast<const float*>(a.gate) : nullptr);
  return hipGetLastError();
}

}  // namespace bsq
