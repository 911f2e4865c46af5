// Norms around a block with its gate and residual scale, and their gradient:
//   n = o * rstd_o * w_post,  r = alpha * x + g . n,  h = r * rstd_r * w_pre
// with rstd_v = 1 / sqrt(mean(v^2) + eps) over a row.  The contract is in
// include/bsq.h.  Everything is FP32 between the loads and one rounding at each
// store; h is taken from r before its rounding.
//
// Both directions are one pass over the rows (HBM-bound): a group of TPR
// threads holds one row in registers, CH pieces of 8 columns per thread, so x, o
// (forward) and d_r, d_h, r, o (backward) are read once.
#include "bsq_internal.hpp"
#include "bsq_wave.hpp"

namespace bsq {

namespace {

// Column of element j of piece c of thread t: pieces of 8 consecutive columns
// (VEC 8: 16-byte accesses, cols % 8 == 0 and aligned), or single columns
// strided over the group (VEC 1: any cols).
template <int VEC, int TPR>
__device__ __forceinline__ int col_of(int c, int j, int t) {
  return VEC == 8 ? (c * TPR + t) * 8 + j : (c * 8 + j) * TPR + t;
}

template <int VEC, int TPR>
__device__ __forceinline__ void load8(const uint16_t* p, int c, int t, int cols, float* y) {
  if constexpr (VEC == 8) {
    const int col = col_of<8, TPR>(c, 0, t);
    const uint4 v = col < cols ? *reinterpret_cast<const uint4*>(p + col) : make_uint4(0, 0, 0, 0);
    bf16x8_to_f32(v, y);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = col_of<1, TPR>(c, j, t);
      y[j] = col < cols ? u2f((uint32_t)p[col] << 16) : 0.0f;
    }
  }
}
template <int VEC, int TPR>
__device__ __forceinline__ void load8(const float* p, int c, int t, int cols, float* y) {
  if constexpr (VEC == 8) {
    const int col = col_of<8, TPR>(c, 0, t);
    float4 a = make_float4(0, 0, 0, 0), b = a;
    if (col < cols) {
      a = *reinterpret_cast<const float4*>(p + col);
      b = *reinterpret_cast<const float4*>(p + col + 4);
    }
    y[0] = a.x; y[1] = a.y; y[2] = a.z; y[3] = a.w;
    y[4] = b.x; y[5] = b.y; y[6] = b.z; y[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = col_of<1, TPR>(c, j, t);
      y[j] = col < cols ? p[col] : 0.0f;
    }
  }
}
template <int VEC, int TPR>
__device__ __forceinline__ void store8(uint16_t* p, int c, int t, int cols, const float* y) {
  if constexpr (VEC == 8) {
    const int col = col_of<8, TPR>(c, 0, t);
    if (col < cols) *reinterpret_cast<uint4*>(p + col) = f32_to_bf16x8(y);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = col_of<1, TPR>(c, j, t);
      if (col < cols) p[col] = bf16_rne(y[j]);
    }
  }
}
template <int VEC, int TPR>
__device__ __forceinline__ void store8(float* p, int c, int t, int cols, const float* y) {
  if constexpr (VEC == 8) {
    const int col = col_of<8, TPR>(c, 0, t);
    if (col < cols) {
      *reinterpret_cast<float4*>(p + col) = make_float4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<float4*>(p + col + 4) = make_float4(y[4], y[5], y[6], y[7]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = col_of<1, TPR>(c, j, t);
      if (col < cols) p[col] = y[j];
    }
  }
}

// Sums of NV values over the TPR threads of a row group, in every thread of it.
// red: LDS of [NV][waves of the block], a different one for successive calls
// (the caller alternates), so one barrier per call suffices.
template <int TPR, int NV>
__device__ __forceinline__ void group_sum(float (&v)[NV], float* red) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
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

// 256 threads at least per workgroup: BT / TPR rows at a time, grid-stride.
template <typename T, int VEC, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_block_norm(NormFwd a) {
  constexpr int BT = TPR < 256 ? 256 : TPR, RPB = BT / TPR;
  __shared__ float red[2][16];
  __shared__ uint32_t mred[16];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int cols = (int)a.cols;
  const float inv = 1.0f / (float)cols;
  uint32_t hmax = 0;
  const int64_t trips = (a.rows + RPB - 1) / RPB;
  for (int64_t b = blockIdx.x; b < trips; b += gridDim.x) {
    const int64_t row = b * RPB + sub;
    const bool live = row < a.rows;
    const int64_t base = (live ? row : a.rows - 1) * a.cols;
    float r[CH][8];
    const T* x = static_cast<const T*>(a.x) + base;
#pragma unroll
    for (int c = 0; c < CH; ++c) load8<VEC, TPR>(x, c, t, cols, r[c]);
    if (a.o) {
      float o[CH][8];
      const uint16_t* op = static_cast<const uint16_t*>(a.o) + base;
#pragma unroll
      for (int c = 0; c < CH; ++c) load8<VEC, TPR>(op, c, t, cols, o[c]);
      if (a.w_post) {
        float s[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) s[0] += o[c][j] * o[c][j];
        group_sum<TPR, 1>(s, red[0]);
        const float rs = 1.0f / __builtin_sqrtf(s[0] * inv + a.eps);
        if (live && t == 0 && a.rstd_post) a.rstd_post[row] = rs;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          float w[8];
          load8<VEC, TPR>(a.w_post, c, t, cols, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[c][j] = o[c][j] * rs * w[j];
        }
      }
      if (a.gate_kind == kGateRow) {
        const float g = static_cast<const float*>(a.gate)[live ? row : a.rows - 1];
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) o[c][j] *= g;
      } else if (a.gate_kind != kGateNone) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          float g[8];
          if (a.gate_kind == kGateChannel)
            load8<VEC, TPR>(static_cast<const float*>(a.gate), c, t, cols, g);
          else
            load8<VEC, TPR>(static_cast<const uint16_t*>(a.gate) + base, c, t, cols, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[c][j] *= g[j];
        }
      }
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) r[c][j] = a.alpha * r[c][j] + o[c][j];
      if (live) {
        T* rp = static_cast<T*>(a.r) + base;
#pragma unroll
        for (int c = 0; c < CH; ++c) store8<VEC, TPR>(rp, c, t, cols, r[c]);
      }
    }
    if (a.w_pre) {
      float s[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] += r[c][j] * r[c][j];
      group_sum<TPR, 1>(s, red[1]);
      const float rs = 1.0f / __builtin_sqrtf(s[0] * inv + a.eps);
      if (live && t == 0 && a.rstd_pre) a.rstd_pre[row] = rs;
      uint16_t* hp = static_cast<uint16_t*>(a.h) + base;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float w[8];
        load8<VEC, TPR>(a.w_pre, c, t, cols, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = r[c][j] * rs * w[j];
        if (live) {
          store8<VEC, TPR>(hp, c, t, cols, w);
          // amax of the stored values: rounding to BF16 is monotone, so the
          // rounding of the maximum is the maximum of the rounded
#pragma unroll
          for (int j = 0; j < 8; ++j) hmax = max(hmax, f2u(w[j]) & 0x7FFFFFFFu);
        }
      }
    }
    // red[0] and red[1] are each written once per trip, with the other's
    // barrier in between only when both norms run
    if (TPR > 64 && !(a.w_pre && a.o && a.w_post)) __syncthreads();
  }
  if (a.amax) {
    hmax = wave_max_dpp(hmax);
    if ((threadIdx.x & 63) == 0) mred[threadIdx.x >> 6] = hmax;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < BT / 64; ++i) hmax = max(hmax, mred[i]);
      const float m = u2f((uint32_t)bf16_rne(u2f(hmax)) << 16);
      if (gridDim.x == 1) *a.amax = m;             // no other writer: no clearing launch before
      else atomicMax(reinterpret_cast<unsigned int*>(a.amax), f2u(m));
    }
  }
}

// ---------------------------------------------------------------- backward

// One pass over the rows, each workgroup BT / TPR rows at a time; the column
// sums (d_w_pre, d_w_post, a channel gate's) stay in registers over all rows of
// the workgroup and go to the workspace once, [workgroup][3][cols]; k_col_sum
// adds them in workgroup order (no atomics: repeated calls give the same bits).
// The two row means need one reduction only: with q = g w_post on,
//   G = d_r + rs (a - rn m1),  m1 = mean(a rn)
//   mean(G q) = mean(d_r q) + rs (mean(a q) - m1 mean(rn q)).
template <typename T, int VEC, int TPR, int CH>
__global__ __launch_bounds__(TPR < 512 ? 512 : TPR) void k_block_norm_bwd(NormBwd a) {
  constexpr int BT = TPR < 512 ? 512 : TPR, RPB = BT / TPR;
  __shared__ float red[2][4 * 16];
  extern __shared__ float fold[];                   // [BT][8] for the fold over the row groups
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int cols = (int)a.cols;
  const float inv = 1.0f / (float)cols;
  float sp[CH][8], sq[CH][8], sg[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) sp[c][j] = sq[c][j] = sg[c][j] = 0.0f;
  int par = 0;
  const int64_t trips = (a.rows + RPB - 1) / RPB;
  for (int64_t b = blockIdx.x; b < trips; b += gridDim.x, par ^= 1) {
    const int64_t row = b * RPB + sub;
    const bool live = row < a.rows;
    const int64_t rw = live ? row : a.rows - 1;
    const int64_t base = rw * a.cols;
    const float rs = a.w_pre ? a.rstd_pre[rw] : 0.0f;
    const float rp = a.w_post ? a.rstd_post[rw] : 1.0f;
    const float grow = a.gate_kind == kGateRow ? static_cast<const float*>(a.gate)[rw] : 1.0f;
    float G[CH][8], av[CH][8], rn[CH][8], on[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (a.d_r) {
        load8<VEC, TPR>(static_cast<const T*>(a.d_r) + base, c, t, cols, G[c]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) G[c][j] = 0.0f;
      }
      if (a.w_pre) {
        float w[8];
        load8<VEC, TPR>(static_cast<const uint16_t*>(a.d_h) + base, c, t, cols, av[c]);
        load8<VEC, TPR>(static_cast<const T*>(a.r) + base, c, t, cols, rn[c]);
        load8<VEC, TPR>(a.w_pre, c, t, cols, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          rn[c][j] *= rs;
          if (live) sp[c][j] += av[c][j] * rn[c][j];
          av[c][j] *= w[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) av[c][j] = rn[c][j] = 0.0f;
      }
      if (a.o) {
        load8<VEC, TPR>(static_cast<const uint16_t*>(a.o) + base, c, t, cols, on[c]);
#pragma unroll
        for (int j = 0; j < 8; ++j) on[c][j] *= rp;
      }
    }
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float wq[8], g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) wq[j] = 1.0f, g[j] = 1.0f;
      if (a.o) {
        if (a.w_post) load8<VEC, TPR>(a.w_post, c, t, cols, wq);
        if (a.gate_kind == kGateChannel) load8<VEC, TPR>(static_cast<const float*>(a.gate), c, t, cols, g);
        else if (a.gate_kind == kGateFull) load8<VEC, TPR>(static_cast<const uint16_t*>(a.gate) + base, c, t, cols, g);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[0] += av[c][j] * rn[c][j];
        if (a.o) {
          const float q = g[j] * wq[j] * on[c][j];
          s[1] += G[c][j] * q;
          s[2] += av[c][j] * q;
          s[3] += rn[c][j] * q;
        }
      }
    }
    group_sum<TPR, 4>(s, red[par]);
    const float m1 = s[0] * inv;
    const float tot = s[1] + rs * (s[2] - m1 * s[3]);   // sum of G g w_post on (row gate left out)
    const float m2 = tot * grow * inv;
    if (a.gate_kind == kGateRow && live && t == 0) static_cast<float*>(a.d_gate)[row] = tot;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        G[c][j] += rs * (av[c][j] - rn[c][j] * m1);
        y[j] = a.o ? a.alpha * G[c][j] : G[c][j];
      }
      if (live) store8<VEC, TPR>(static_cast<T*>(a.d_x) + base, c, t, cols, y);
      if (a.o) {
        float wq[8], g[8], z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) wq[j] = 1.0f, g[j] = grow;
        if (a.w_post) load8<VEC, TPR>(a.w_post, c, t, cols, wq);
        if (a.gate_kind == kGateChannel) load8<VEC, TPR>(static_cast<const float*>(a.gate), c, t, cols, g);
        else if (a.gate_kind == kGateFull) load8<VEC, TPR>(static_cast<const uint16_t*>(a.gate) + base, c, t, cols, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float Gg = G[c][j] * g[j];
          y[j] = G[c][j] * wq[j] * on[c][j];             // d gate
          if (live) {
            sg[c][j] += y[j];
            sq[c][j] += Gg * on[c][j];
          }
          z[j] = a.w_post ? rp * (Gg * wq[j] - on[c][j] * m2) : Gg;
        }
        if (live) {
          store8<VEC, TPR>(static_cast<uint16_t*>(a.d_o) + base, c, t, cols, z);
          if (a.gate_kind == kGateFull) store8<VEC, TPR>(static_cast<uint16_t*>(a.d_gate) + base, c, t, cols, y);
        }
      }
    }
  }
  // fold the row groups of the workgroup in LDS, then one partial row each
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const bool want = k == 0 ? a.w_pre != nullptr : k == 1 ? a.w_post != nullptr : a.gate_kind == kGateChannel;
      if (!want) continue;
      float* v = k == 0 ? sp[c] : k == 1 ? sq[c] : sg[c];
      if constexpr (RPB > 1) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) fold[j * BT + threadIdx.x] = v[j];
        __syncthreads();
        if (sub == 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float s = 0.0f;
            for (int q = 0; q < RPB; ++q) s += fold[j * BT + q * TPR + t];
            v[j] = s;
          }
        }
      }
      if (sub == 0)
        store8<VEC, TPR>(a.part + ((int64_t)blockIdx.x * 3 + k) * a.cols, c, t, cols, v);
    }
  }
}

// out[k][c] = sum over the nblk partials, in order: 16 slices of the partials by
// 16 row groups of a workgroup, folded in slice order.  blockIdx.y = k.
__global__ __launch_bounds__(1024) void k_col_sum(const float* __restrict__ part, int nblk, int64_t cols,
                                                  float* o0, float* o1, float* o2) {
  __shared__ float s[16][64];
  float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (!out) return;
  const int lane = threadIdx.x & 63, sl = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  const int per = (nblk + 15) / 16, b0 = sl * per, b1 = min(nblk, b0 + per);
  float v = 0.0f;
  if (c < cols) {
    const float* p = part + (int64_t)blockIdx.y * cols + c;
#pragma unroll 8
    for (int b = b0; b < b1; ++b) v += p[(int64_t)b * 3 * cols];
  }
  s[sl][lane] = v;
  __syncthreads();
  if (sl == 0 && c < cols) {
    for (int i = 1; i < 16; ++i) v += s[i][lane];
    out[c] = v;
  }
}

// Threads per row and 8-column pieces per thread.
struct NormCfg {
  int tpr, ch;
};
NormCfg norm_cfg(int64_t cols) {
  if (cols <= 512) return {64, 1};
  if (cols <= 2048) return {256, 1};
  if (cols <= 4096) return {256, 2};
  if (cols <= 8192) return {512, 2};
  return {1024, 2};
}

template <typename T, int VEC, int TPR, int CH>
hipError_t run_fwd(const NormFwd& a, hipStream_t s) {
  constexpr int BT = TPR < 256 ? 256 : TPR, RPB = BT / TPR;
  const int64_t trips = (a.rows + RPB - 1) / RPB;
  const int64_t cap = (int64_t)device_cus() * (2048 / BT);
  const unsigned grid = (unsigned)(trips < cap || cap <= 0 ? trips : cap);
  if (a.amax && grid > 1) {
    const hipError_t e = launch_zero_amax(a.amax, nullptr, s);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_block_norm<T, VEC, TPR, CH>), dim3(grid), dim3(BT), 0, s, a);
  return hipGetLastError();
}

template <typename T, int VEC>
hipError_t pick_fwd(const NormFwd& a, hipStream_t s) {
  const NormCfg c = norm_cfg(a.cols);
  if (c.tpr == 64) return run_fwd<T, VEC, 64, 1>(a, s);
  if (c.tpr == 256) return c.ch == 1 ? run_fwd<T, VEC, 256, 1>(a, s) : run_fwd<T, VEC, 256, 2>(a, s);
  if (c.tpr == 512) return run_fwd<T, VEC, 512, 2>(a, s);
  return run_fwd<T, VEC, 1024, 2>(a, s);
}

template <typename T, int VEC, int TPR, int CH>
hipError_t run_bwd(const NormBwd& a, unsigned grid, hipStream_t s) {
  constexpr int BT = TPR < 512 ? 512 : TPR;
  hipLaunchKernelGGL((k_block_norm_bwd<T, VEC, TPR, CH>), dim3(grid), dim3(BT),
                     BT > TPR ? BT * 8 * sizeof(float) : 0, s, a);
  return hipGetLastError();
}

template <typename T, int VEC>
hipError_t pick_bwd(const NormBwd& a, unsigned grid, hipStream_t s) {
  const NormCfg c = norm_cfg(a.cols);
  if (c.tpr == 64) return run_bwd<T, VEC, 64, 1>(a, grid, s);
  if (c.tpr == 256) return c.ch == 1 ? run_bwd<T, VEC, 256, 1>(a, grid, s) : run_bwd<T, VEC, 256, 2>(a, grid, s);
  if (c.tpr == 512) return run_bwd<T, VEC, 512, 2>(a, grid, s);
  return run_bwd<T, VEC, 1024, 2>(a, grid, s);
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Workgroups of the backward pass: at most 512 (two per compute unit of the
// 256), so that the partial column sums stay small next to the tensors.
unsigned bwd_grid(int64_t rows, int64_t cols) {
  const int tpr = norm_cfg(cols).tpr, rpb = (tpr < 512 ? 512 : tpr) / tpr;
  const int64_t trips = (rows + rpb - 1) / rpb;
  return (unsigned)(trips < 512 ? trips : 512);
}

}  // namespace

hipError_t launch_block_norm(const NormFwd& a, hipStream_t s) {
  const bool vec = a.cols % 8 == 0 && al16(a.x) && al16(a.o) && al16(a.w_post) && al16(a.w_pre) && al16(a.r) &&
                   al16(a.h) && (a.gate_kind == kGateNone || a.gate_kind == kGateRow || al16(a.gate));
  if (a.f32) return vec ? pick_fwd<float, 8>(a, s) : pick_fwd<float, 1>(a, s);
  return vec ? pick_fwd<uint16_t, 8>(a, s) : pick_fwd<uint16_t, 1>(a, s);
}

int64_t block_norm_bwd_part_bytes(int64_t rows, int64_t cols) {
  return (int64_t)bwd_grid(rows, cols) * 3 * cols * (int64_t)sizeof(float);
}

hipError_t launch_block_norm_bwd(const NormBwd& a, hipStream_t s) {
  const bool full = a.gate_kind == kGateFull, chan = a.gate_kind == kGateChannel;
  const bool vec = a.cols % 8 == 0 && al16(a.r) && al16(a.o) && al16(a.d_r) && al16(a.d_h) && al16(a.w_post) &&
                   al16(a.w_pre) && al16(a.d_x) && al16(a.d_o) && al16(a.part) &&
                   (!(full || chan) || al16(a.gate)) && (!full || al16(a.d_gate));
  const unsigned grid = bwd_grid(a.rows, a.cols);
  hipError_t e = hipSuccess;
  if (a.rows > 0) {                                 // the column sums of no rows are zero
    if (a.f32) e = vec ? pick_bwd<float, 8>(a, grid, s) : pick_bwd<float, 1>(a, grid, s);
    else e = vec ? pick_bwd<uint16_t, 8>(a, grid, s) : pick_bwd<uint16_t, 1>(a, grid, s);
  }
  if (e != hipSuccess) return e;
  float* o0 = a.w_pre ? a.d_w_pre : nullptr;
  float* o1 = a.w_post ? a.d_w_post : nullptr;
  float* o2 = chan ? static_cast<float*>(a.d_gate) : nullptr;
  if (o0 || o1 || o2)
    hipLaunchKernelGGL(k_col_sum, dim3((unsigned)((a.cols + 63) / 64), 3), dim3(1024), 0, s, a.part, (int)grid,
                       a.cols, o0, o1, o2);
  return hipGetLastError();
}

}  // namespace bsq
