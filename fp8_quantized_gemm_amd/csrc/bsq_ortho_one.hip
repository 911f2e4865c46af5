// Orthogonalisation of small matrices, all steps in one workgroup, and the weight update
// that takes it, for gfx950 (contract in include/bsq.h; the mathematics and what is held
// in how many bits as in bsq_ortho.hip, X itself in FP32).
//
// What bounds small matrices is the launches: 15 products of 4 to 6 us each (200 x 136: 79
// us; 63 here, an update's 78; 256 of 128 x 128: 150, 41).  Here a workgroup of eight waves
// holds a matrix in its compute unit: X in FP32 in the registers of the waves that compute its
// tiles, and in LDS the symmetric matrix E and X's FP16 form, by rows for the Gram matrix and
// then by columns for the product with the polynomial, as the MFMA takes operands with K
// running along a row.  The products read LDS more than they multiply, so a wave computes 32 x
// 32 entries at a time of the symmetric ones, and 32 columns of X under every row of the
// polynomial.  What bounds it is latency: of 200 x 136 LDS is busy for 41% of the time, the
// VALU 40%, the matrix pipe 18%, and the waves, two a SIMD, wait for half of theirs in phases
// that depend on each other.
#include "bsq_ortho.hpp"
#include "bsq_wave.hpp"

#include <algorithm>

namespace bsq {

namespace {

constexpr int kOneWaves = 8;
constexpr int kOneLds = 160 * 1024;

struct NsOne {
  NsSource src;
  int64_t rows, cols;
  int m, n, steps;                         // m <= n; X is m x n
  float eps;
  float coefs[96];                         // 3 per step
  uint16_t* out;                           // or the update's:
  float* w;
  uint16_t* wb;
  float* amax;
  float keep, step;                        // step of X under kS
};

// LDS, all sizes in whole steps of 32 (what is past the matrix is zero): E [32 mb][lt], its
// diagonal, and X [32 mb][lx] or its transpose [32 nb][lt]; rows 16 bytes apart in the banks.
struct OneLds {
  int mb, nb, lt, lx, d, x, bytes;
};
__host__ __device__ inline OneLds one_lds(int m, int n) {
  OneLds o;
  o.mb = (m + 31) / 32;
  o.nb = (n + 31) / 32;
  o.lt = 32 * o.mb + 8;
  o.lx = 32 * o.nb + 8;
  o.d = 32 * o.mb * o.lt * 2;
  o.x = o.d + 32 * o.mb * 4;
  const int r = 32 * o.mb * o.lx, c = 32 * o.nb * o.lt;
  o.bytes = o.x + (r > c ? r : c) * 2;
  return o;
}

// Four FP16 values of row r16, columns c4 .. c4 + 3, to column-major storage f (the block's
// first element): a lane and its neighbour exchange a pair, so that each stores two rows of
// one column at a time.
__device__ __forceinline__ void one_turn(uint16_t* f, int ld, int r16, int c4, ntu2 v) {
  const bool odd = r16 & 1;
  const uint32_t own = odd ? v[1] : v[0], give = odd ? v[0] : v[1];
  const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)give, 0xB1, 0xF, 0xF, false);   // lane ^ 1
  const uint32_t lo = odd ? got : own, hi = odd ? own : got;
  uint16_t* d = f + (c4 + (odd ? 2 : 0)) * ld + (r16 & ~1);
  *reinterpret_cast<uint32_t*>(d) = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
  *reinterpret_cast<uint32_t*>(d + ld) = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

__device__ __forceinline__ ntu4 one_read(const uint16_t* p) { return *reinterpret_cast<const ntu4*>(p); }

// A lane's four elements of a 16 x 16 tile of a matrix, as FP32: one access at any alignment
// where a whole tile's lie together, else one each, read without branches (a load in a
// branch is waited for there) from the nearest element inside.
struct OneTile {
  bool whole;                              // uniform: inside the matrix, rows of X along its rows
  int64_t first;                           // uniform: the tile's first element
  int off[4], len;                         // the lane's from there, how many are inside
};
__device__ __forceinline__ ntf4 one_wide(const float* p) {
  typedef ntf4 U __attribute__((aligned(4)));
  return *reinterpret_cast<const U*>(p);
}
__device__ __forceinline__ ntf4 one_wide(const uint16_t* p) {
  typedef ntu2 U __attribute__((aligned(2)));
  const ntu2 v = *reinterpret_cast<const U*>(p);
  return ntf4{bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])};
}
__device__ __forceinline__ float one_float(float v) { return v; }
__device__ __forceinline__ float one_float(uint16_t v) { return u2f((uint32_t)v << 16); }
template <typename T>
__device__ __forceinline__ void one_load(float (&u)[4], const T* matrix, const OneTile& t) {
  const T* p = matrix + t.first;
  if (t.whole) {
    const ntf4 v = one_wide(p + t.off[0]);
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = v[k];
  } else {
    T v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = p[t.off[k]];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = k < t.len ? one_float(v[k]) : 0.0f;
  }
}
__device__ __forceinline__ void one_store(float* matrix, const float (&u)[4], const OneTile& t) {
  typedef ntf4 U __attribute__((aligned(4)));
  float* p = matrix + t.first;
  if (t.whole) {
    *reinterpret_cast<U*>(p + t.off[0]) = ntf4{u[0], u[1], u[2], u[3]};
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < t.len) p[t.off[k]] = u[k];
  }
}
__device__ __forceinline__ void one_store(uint16_t* matrix, const float (&u)[4], const OneTile& t) {
  typedef ntu2 U __attribute__((aligned(2)));
  uint16_t* p = matrix + t.first;
  if (t.whole) {
    *reinterpret_cast<U*>(p + t.off[0]) = ntu2{pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3])};
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < t.len) p[t.off[k]] = bf16_rne(u[k]);
  }
}

// MB: m in steps of 32; CB: most steps of 32 columns of a wave (it has every eighth).
template <int IN, int MB, int CB>
__global__ __launch_bounds__(kOneWaves * 64) void k_ns_one(NsOne o) {
  constexpr int LOWER = MB * (MB + 1) / 2, PB = (LOWER + kOneWaves - 1) / kOneWaves;   // blocks of E, most of a wave
  constexpr int LT = 32 * MB + 8;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ double parts[kOneWaves];
  const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), lane = t & 63, r16 = lane & 15, c4 = lane >> 4 << 2;
  const int m = o.m, n = o.n;
  const bool wide = o.rows <= o.cols;
  const OneLds L = one_lds(m, n);
  const int lx = L.lx, nb = L.nb;
  uint16_t* E = reinterpret_cast<uint16_t*>(smem);
  float* D = reinterpret_cast<float*>(smem + L.d);
  uint16_t* X = reinterpret_cast<uint16_t*>(smem + L.x);
  const int64_t base = (int64_t)blockIdx.x * m * n;
  // the tile of X whose first element is (r, c), inside the matrix
  int lr = r16, lc = c4;
  const auto tile = [&](int r, int c) {
    OneTile t;
    t.whole = wide && r + 16 <= m && c + 16 <= n;
    t.first = base + (wide ? r * n + c : c * m + r);
    t.len = r + lr < m ? n - c - lc : 0;
    if (r + 16 <= m && c + 16 <= n) {                      // the same for every such tile
#pragma unroll
      for (int k = 0; k < 4; ++k) t.off[k] = wide ? lr * n + lc + k : (lc + k) * m + lr;
    } else {
      const int i = min(lr, m - 1 - r);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = min(lc + k, n - 1 - c);
        t.off[k] = wide ? i * n + j : j * m + i;
      }
    }
    return t;
  };

  // row 16 i + r16, columns 32 q + 16 h + c4 + k with q = w + 8 j
  float x[CB][2 * MB][2][4];
  double sum = 0.0;
  // f(j, i, h, the tile) for each of this wave's tiles that lie in the matrix
  const auto each = [&](const auto& f) {
#pragma unroll
    for (int j = 0; j < CB; ++j)
#pragma unroll
      for (int i = 0; i < 2 * MB; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * i, c = 32 * (w + kOneWaves * j) + 16 * h;
          if (r < m && c < n) f(j, i, h, tile(r, c));
        }
  };
#pragma unroll
  for (int j = 0; j < CB; ++j)
#pragma unroll
    for (int i = 0; i < 2 * MB; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[j][i][h][k] = 0.0f;
  // (all code here runs once, from a cold instruction cache: all loads before the first store,
  // in two passes over the tiles, are 10 us slower)
  each([&](int j, int i, int h, const OneTile& t) {
    float(&u)[4] = x[j][i][h];
    if constexpr (IN == kNsMoment) {
      float g[4];
      one_load(g, o.src.grad, t);
      one_load(u, (const float*)o.src.momentum, t);
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = o.src.mu * u[k] + g[k];
      one_store(o.src.momentum, u, t);
      if (o.src.nesterov) {
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = g[k] + o.src.mu * u[k];
      }
    } else if constexpr (IN == kNsF32) {
      one_load(u, static_cast<const float*>(o.src.x), t);
    } else {
      one_load(u, static_cast<const uint16_t*>(o.src.x), t);
    }
  });
#pragma unroll
  for (int j = 0; j < CB; ++j)
#pragma unroll
    for (int i = 0; i < 2 * MB; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) sum += (double)x[j][i][h][k] * (double)x[j][i][h][k];
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) sum += __shfl_xor(sum, s);
  if (lane == 0) parts[w] = sum;
  __syncthreads();
  sum = 0.0;
#pragma unroll
  for (int i = 0; i < kOneWaves; ++i) sum += parts[i];
  const NsNorm norm = ns_norm(sum, o.eps);
#pragma unroll
  for (int j = 0; j < CB; ++j)
#pragma unroll
    for (int i = 0; i < 2 * MB; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[j][i][h][k] = ns_scaled(x[j][i][h][k], norm);

  // this wave's blocks on and below the diagonal
  int bi[PB], bj[PB];
#pragma unroll
  for (int p = 0; p < PB; ++p) {
    int k = min(w + kOneWaves * p, LOWER - 1), i = 0;
    while (k > i) k -= ++i;
    bi[p] = i;
    bj[p] = k;
  }
  // rows 32 i .. and 32 j .. of p, one step of K
  typedef ntf4 Block[2][2];
  const auto multiply = [&](Block& acc, const uint16_t* p, int ld, int i, int j, int s) {
    const uint16_t *a = p + (32 * i + r16) * ld + 2 * c4 + 32 * s, *b = p + (32 * j + r16) * ld + 2 * c4 + 32 * s;
    const ntu4 a0 = one_read(a), a1 = one_read(a + 16 * ld), b0 = one_read(b), b1 = one_read(b + 16 * ld);
    acc[0][0] = nt_mfma<kNtF16>(b0, a0, acc[0][0]);
    acc[0][1] = nt_mfma<kNtF16>(b1, a0, acc[0][1]);
    acc[1][0] = nt_mfma<kNtF16>(b0, a1, acc[1][0]);
    acc[1][1] = nt_mfma<kNtF16>(b1, a1, acc[1][1]);
  };
  const auto clear = [](Block& acc) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int v = 0; v < 2; ++v) acc[u][v] = ntf4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  // four entries of row r from column c + c4 on, and their mirror
  const auto put = [&](int r, int c, bool mirror, ntu2 v) {
    *reinterpret_cast<ntu2*>(E + (r + r16) * LT + c + c4) = v;
    if (mirror) one_turn(E + c * LT + r, LT, r16, c4, v);
  };

  for (int s = 0; s < o.steps; ++s) {
    const float a = o.coefs[3 * s], b = o.coefs[3 * s + 1], c = o.coefs[3 * s + 2];
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      const int q = w + kOneWaves * j;
      if (q >= nb) break;
#pragma unroll
      for (int i = 0; i < 2 * MB; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<ntu2*>(X + (16 * i + r16) * lx + 32 * q + 16 * h + c4) =
              ntu2{pack_f16x2(x[j][i][h][0], x[j][i][h][1]), pack_f16x2(x[j][i][h][2], x[j][i][h][3])};
    }
    __syncthreads();
    // A = X X^T
#pragma unroll
    for (int p = 0; p < PB; ++p) {
      if (w + kOneWaves * p >= LOWER) break;
      const int i = bi[p], j = bj[p];
      Block acc;
      clear(acc);
#pragma unroll 2
      for (int k = 0; k < nb; ++k) multiply(acc, X, lx, i, j, k);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          ntf4 y = acc[u][v] * (1.0f / kS);
          const int r = 32 * i + 16 * u, e = 32 * j + 16 * v;
          if (r == e) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (r16 == c4 + k) {
                D[r + r16] = y[k] * (1.0f / kS);
                y[k] = 0.0f;
              }
          }
          put(r, e, i != j, ntu2{pack_f16x2(y[0], y[1]), pack_f16x2(y[2], y[3])});
        }
    }
    __syncthreads();
    // a I + b A + c A^2 in registers, and X by columns
    ntu2 y[PB][2][2];
    float d[PB][2];
#pragma unroll
    for (int p = 0; p < PB; ++p) {
      if (w + kOneWaves * p >= LOWER) break;
      const int i = bi[p], j = bj[p];
      Block acc;
      clear(acc);
#pragma unroll 2
      for (int k = 0; k < MB; ++k) multiply(acc, E, LT, i, j, k);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          ntf4 z = acc[u][v] * (c / kS);
          const int r = 32 * i + 16 * u, f = 32 * j + 16 * v;
          const ntu2 e = *reinterpret_cast<const ntu2*>(E + (r + r16) * LT + f + c4);
          const float di = D[r + r16];
          const ntf4 dj = *reinterpret_cast<const ntf4*>(D + f + c4);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (r == f && r16 == c4 + k) {
              d[p][u] = z[k] * (1.0f / kS) + (a + b * di + c * (di * di));
              z[k] = 0.0f;
            } else {
              z[k] = __builtin_fmaf(k & 1 ? f16_hi(e[k >> 1]) : f16_lo(e[k >> 1]), b + c * (di + dj[k]), z[k]);
            }
          }
          y[p][u][v] = ntu2{pack_f16x2(z[0], z[1]), pack_f16x2(z[2], z[3])};
        }
    }
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      const int q = w + kOneWaves * j;
      if (q >= nb) break;
#pragma unroll
      for (int i = 0; i < 2 * MB; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          one_turn(X + (32 * q + 16 * h) * LT + 16 * i, LT, r16, c4,
                   ntu2{pack_f16x2(x[j][i][h][0], x[j][i][h][1]), pack_f16x2(x[j][i][h][2], x[j][i][h][3])});
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < PB; ++p) {
      if (w + kOneWaves * p >= LOWER) break;
      const int i = bi[p], j = bj[p];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int v = 0; v < 2; ++v) put(32 * i + 16 * u, 32 * j + 16 * v, i != j, y[p][u][v]);
        if (i == j && r16 >= c4 && r16 < c4 + 4) D[32 * i + 16 * u + r16] = d[p][u];
      }
    }
    __syncthreads();
    // X <- P X: this wave's columns, held while P's rows pass
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      const int q = w + kOneWaves * j;
      if (q >= nb) break;
      ntu4 f[2][MB];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < MB; ++k) f[h][k] = one_read(X + (32 * q + 16 * h + r16) * LT + 32 * k + 2 * c4);
      // a row of P is loaded while the one before is multiplied, and no earlier
      ntu4 e[2][MB];
      const auto row = [&](int i) {
#pragma unroll
        for (int k = 0; k < MB; ++k) e[i & 1][k] = one_read(E + (16 * i + r16) * LT + 32 * k + 2 * c4);
      };
      row(0);
#pragma unroll
      for (int i = 0; i < 2 * MB; ++i) {
        if (i + 1 < 2 * MB) row(i + 1);
        __builtin_amdgcn_sched_barrier(0);
        ntf4 acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
        for (int k = 0; k < MB; ++k) {
          acc[0] = nt_mfma<kNtF16>(f[0][k], e[i & 1][k], acc[0]);
          acc[1] = nt_mfma<kNtF16>(f[1][k], e[i & 1][k], acc[1]);
        }
        // P's diagonal times X's FP16 form, and the rest of X's rounding times the leading
        // coefficient, or the diagonal in the last two steps (see bsq_ortho.hip)
        const float di = D[16 * i + r16], rest = s + 2 < o.steps ? a : di;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float y = x[j][i][h][k], half = (float)(_Float16)y;
            x[j][i][h][k] = __builtin_fmaf(acc[h][k], 1.0f / kS, __builtin_fmaf(y - half, rest, di * half));
          }
      }
    }
    __syncthreads();
  }

  // the tiles' offsets are computed again: kept through the steps they would cost registers
  asm volatile("" : "+v"(lr), "+v"(lc));
  uint32_t most = 0;
  each([&](int j, int i, int h, const OneTile& t) {
    float y[4];
    if constexpr (IN == kNsMoment) {
      one_load(y, (const float*)o.w, t);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        y[k] = o.keep * y[k] - o.step * x[j][i][h][k];
        if (k < t.len) most = max(most, ((uint32_t)bf16_rne(y[k]) & 0x7FFFu) << 16);
      }
      one_store(o.w, y, t);
      one_store(o.wb, y, t);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = x[j][i][h][k] * (1.0f / kS);
      one_store(o.out, y, t);
    }
  });
  if constexpr (IN == kNsMoment) {
    if (!o.amax) return;
    uint32_t* all = reinterpret_cast<uint32_t*>(parts);
    most = wave_max_dpp(most);
    __syncthreads();
    if (lane == 0) all[w] = most;
    __syncthreads();
    if (t != 0) return;
#pragma unroll
    for (int i = 0; i < kOneWaves; ++i) most = max(most, all[i]);
    uint32_t* p = reinterpret_cast<uint32_t*>(o.amax);
    if (gridDim.x == 1) *p = most;
    else atomicMax(p, most);
  }
}

template <int IN, int MB, int CB>
hipError_t run_one(const NsOne& a, int64_t batch, hipStream_t s) {
  const int lds = one_lds(a.m, a.n).bytes;
  const void* fn = reinterpret_cast<const void*>(&k_ns_one<IN, MB, CB>);
  constexpr int kStatic = kOneWaves * 8;
  if (lds + kStatic > kOneLds || set_lds_limit(fn, kOneLds - kStatic) != hipSuccess) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_ns_one<IN, MB, CB>), dim3((unsigned)batch), dim3(kOneWaves * 64), lds, s, a);
  return hipGetLastError();
}
template <int IN>
hipError_t run_one_any(const NsOne& a, int64_t batch, hipStream_t s) {
  switch ((a.m + 31) / 32) {
    case 1: return run_one<IN, 1, 4>(a, batch, s);
    case 2: return run_one<IN, 2, 3>(a, batch, s);
    case 3: return run_one<IN, 3, 2>(a, batch, s);
    case 4: return run_one<IN, 4, 1>(a, batch, s);
    case 5: return run_one<IN, 5, 1>(a, batch, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

// What the registers of a wave and the LDS of a compute unit hold: 160 x 256, 96 x 512, 64 x
// 768, 32 x 1,024 and what is smaller.  192 x 192 would fit too, but its registers do not
// (86 us; 77 by the products).
bool ortho_in_one(int64_t rows, int64_t cols) {
  const int64_t m = std::min(rows, cols), n = std::max(rows, cols);
  if (m > 160 || n > (m <= 32 ? 1024 : m <= 64 ? 768 : m <= 96 ? 512 : 256)) return false;
  return one_lds((int)m, (int)n).bytes + kOneWaves * 8 <= kOneLds;
}

hipError_t launch_ortho_one(const OrthoArgs& o, hipStream_t s) {
  NsOne a{};
  a.src = NsSource{o.x, o.momentum, static_cast<const uint16_t*>(o.grad), o.mu, o.nesterov ? 1 : 0};
  a.rows = o.rows, a.cols = o.cols;
  a.m = (int)std::min(o.rows, o.cols), a.n = (int)std::max(o.rows, o.cols);
  a.steps = o.steps;
  a.eps = o.eps;
  if (3 * o.steps > (int)(sizeof(a.coefs) / sizeof(float)) || o.batch > 0x7FFFFFFF) return hipErrorInvalidValue;
  std::copy(o.coefs, o.coefs + 3 * o.steps, a.coefs);
  a.out = static_cast<uint16_t*>(o.out);
  a.w = o.w, a.wb = static_cast<uint16_t*>(o.w_bf16), a.amax = o.amax;
  a.keep = o.keep, a.step = o.step / kS;
  if (!o.w) return o.f32 ? run_one_any<kNsF32>(a, o.batch, s) : run_one_any<kNsBf16>(a, o.batch, s);
  if (o.amax && o.batch > 1) {
    hipLaunchKernelGGL(k_ns_zero, dim3(1), dim3(1), 0, s, o.amax);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  return run_one_any<kNsMoment>(a, o.batch, s);
}

}  // namespace bsq
