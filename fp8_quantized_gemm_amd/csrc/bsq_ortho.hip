// Orthogonalisation of matrices by Newton-Schulz products, and the weight update
// that takes it, for gfx950 (contract in include/bsq.h):
//   X = u / (||u||_F + eps);  per step  A = X X^T,  X <- (a I + b A + c A^2) X
//
// X, A and the polynomials are held in FP16 between products, under powers of two
// that keep every entry of a matrix with singular values up to 8 in range and its
// typical entries normal; sums are FP32 (MFMA).  FP16 rather than BF16: the matrix
// rate is the same and each rounding is eight times finer (2^-11 of an entry); on
// gradients of 512 x 1,792 the result is 1.0e-3 (relative, Frobenius) from the 64-bit
// one, against 1.3e-2 with BF16 between products.
//
// Everything is computed on the smaller side m of the matrix, padded with zeros to
// multiples of 64 in both directions (zero rows and columns stay zero), so that the
// products need no edges.
#include "bsq_nt.hpp"
#include "bsq_wave.hpp"

#include <algorithm>

namespace bsq {

namespace {

// Powers of two of the FP16 forms: X and the Gram matrix (entries at most 1.3
// squared with the usual coefficients, typically 1 / sqrt(m n)) and the polynomials
// (entries up to the product of the leading coefficients).
constexpr float kSX = 1024.0f, kSA = 1024.0f, kSP = 256.0f;
constexpr int kParts = 256;              // most workgroups that sum one matrix's squares

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, halfx2{(_Float16)lo, (_Float16)hi});
}
__device__ __forceinline__ float f16_lo(uint32_t w) { return (float)__builtin_bit_cast(halfx2, w).x; }
__device__ __forceinline__ float f16_hi(uint32_t w) { return (float)__builtin_bit_cast(halfx2, w).y; }

// What is orthogonalised: a tensor (BF16, FP32) or the moment of an update.
enum NsInput { kNsBf16 = 0, kNsF32 = 1, kNsMoment = 2 };
struct NsSource {
  const void* x;
  float* momentum;
  const uint16_t* grad;
  float mu;
  int nesterov;
};

__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return lds[0] + lds[1] + lds[2] + lds[3];
}

// The moment of an update (written in place), and the sum of the squares of what is
// orthogonalised, in 64 bits (the squares of FP32 values leave FP32's range), one
// part per workgroup.  Bound by HBM.
template <int IN>
__global__ __launch_bounds__(256) void k_ns_moment(NsSource src, int64_t n, double* __restrict__ part) {
  __shared__ double lds[4];
  const int64_t base = (int64_t)blockIdx.y * n;
  double sum = 0.0;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 2048) {
    const int len = (int)min((int64_t)8, n - i);
    float u[8];
    if constexpr (IN == kNsMoment) {
      float* m = src.momentum + base + i;
      const uint16_t* g = src.grad + base + i;
      Raw<uint16_t> gr = load_raw<false>(g, 0, len);
      Raw<float> mr = load_raw<false>(m, 0, len);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float gv = raw_at(gr, j), mv = src.mu * raw_at(mr, j) + gv;
        mr.v[j >> 2][j & 3] = f2u(mv);
        u[j] = src.nesterov ? gv + src.mu * mv : mv;
      }
      store_raw<false>(m, 0, len, mr);
    } else if constexpr (IN == kNsF32) {
      const Raw<float> r = load_raw<false>(static_cast<const float*>(src.x) + base + i, 0, len);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = raw_at(r, j);
    } else {
      const Raw<uint16_t> r = load_raw<false>(static_cast<const uint16_t*>(src.x) + base + i, 0, len);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = raw_at(r, j);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < len) sum += (double)u[j] * (double)u[j];
  }
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = sum;
}

// X0 in FP16 in the matrix's own orientation (a [rows64][cols64]) and transposed
// (at), 64 x 64 elements a turn, zeros in the padding.
template <int IN>
__global__ __launch_bounds__(256) void k_ns_scale(NsSource src, int64_t rows, int64_t cols, int parts,
                                                  const double* __restrict__ part, float eps, uint16_t* __restrict__ a,
                                                  uint16_t* __restrict__ at, int64_t rows64, int64_t cols64, int turns) {
  constexpr int LD = 66;
  __shared__ double lds[4];
  __shared__ uint16_t tile[64 * LD];
  const int t = threadIdx.x;
  const double sum = block_sum(t < parts ? part[(int64_t)blockIdx.y * parts + t] : 0.0, lds);
  const float inv = (float)((double)kSX / (sqrt(sum) + (double)eps));
  const int64_t base = (int64_t)blockIdx.y * rows * cols, pad = (int64_t)blockIdx.y * rows64 * cols64;
  const int64_t tiles_c = cols64 / 64, tiles = rows64 / 64 * tiles_c;
  for (int k = 0; k < turns; ++k) {
    const int64_t q = (int64_t)blockIdx.x * turns + k;
    if (q >= tiles) return;
    const int64_t r0 = q / tiles_c * 64, c0 = q % tiles_c * 64;
    const int64_t r = r0 + (t >> 2), c = c0 + (t & 3) * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = (int)c + 8 * h;
      float u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = 0.0f;
      if (r < rows && col < cols) {
        const int64_t row = base + r * cols;
        if constexpr (IN == kNsMoment) {
          Raw<uint16_t> gr = load_raw<false>(src.grad + row, col, (int)cols);
          Raw<float> mr = load_raw<false>((const float*)src.momentum + row, col, (int)cols);
          end_piece<false>(gr, col, (int)cols);
          end_piece<false>(mr, col, (int)cols);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            u[j] = src.nesterov ? raw_at(gr, j) + src.mu * raw_at(mr, j) : raw_at(mr, j);
        } else if constexpr (IN == kNsF32) {
          Raw<float> xr = load_raw<false>(static_cast<const float*>(src.x) + row, col, (int)cols);
          end_piece<false>(xr, col, (int)cols);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] = raw_at(xr, j);
        } else {
          Raw<uint16_t> xr = load_raw<false>(static_cast<const uint16_t*>(src.x) + row, col, (int)cols);
          end_piece<false>(xr, col, (int)cols);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] = raw_at(xr, j);
        }
      }
      ntu4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = pack_f16x2(u[2 * j] * inv, u[2 * j + 1] * inv);
      *reinterpret_cast<ntu4*>(a + pad + r * cols64 + col) = v;
      uint32_t* d = reinterpret_cast<uint32_t*>(tile + (t >> 2) * LD + (t & 3) * 16 + 8 * h);
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = v[j];
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int cc = t >> 2, rr = (t & 3) * 16 + 8 * h;
      ntu4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = (uint32_t)tile[(rr + 2 * j) * LD + cc] | ((uint32_t)tile[(rr + 2 * j + 1) * LD + cc] << 16);
      *reinterpret_cast<ntu4*>(at + pad + (c0 + cc) * rows64 + r0 + rr) = v;
    }
    __syncthreads();
  }
}

__global__ void k_ns_zero(float* p) { *p = 0.0f; }

// ---------------------------------------------------------------- epilogues

// FP16(alpha sum + beta add + gamma I), and its transpose: of a symmetric product the
// tile on the other side of the diagonal, else the matrix in its other orientation.
struct EpiNs {
  static constexpr bool kTrans = true;
  uint16_t* c;
  uint16_t* ct;
  const uint16_t* add;           // null: none
  int64_t ldc, ldt, stride, M, N;
  float alpha, beta, gamma;
  struct Row {};
  struct Col {};
  __device__ __forceinline__ Row row(int, int64_t) const { return Row{}; }
  __device__ __forceinline__ Col col(int, int64_t) const { return Col{}; }
  __device__ __forceinline__ ntu2 pack4(int e, int64_t m, int64_t n, const Row&, const Col&, ntf4 v) const {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = alpha * v[i];
    if (add) {
      const ntu2 w = *reinterpret_cast<const ntu2*>(add + e * stride + min(m, M - 1) * ldc + min(n, N - 4));
      y[0] += beta * f16_lo(w[0]);
      y[1] += beta * f16_hi(w[0]);
      y[2] += beta * f16_lo(w[1]);
      y[3] += beta * f16_hi(w[1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] += m == n + i ? gamma : 0.0f;
    }
    return ntu2{pack_f16x2(y[0], y[1]), pack_f16x2(y[2], y[3])};
  }
  __device__ __forceinline__ void store(int e, int64_t m, int64_t n, const ntu4& v) {
    if (m < M && n < N) *reinterpret_cast<ntu4*>(c + e * stride + m * ldc + n) = v;
  }
  __device__ __forceinline__ void store_t(int e, int64_t n, int64_t m, const ntu4& v) {
    if (m < M && n < N) *reinterpret_cast<ntu4*>(ct + e * stride + n * ldt + m) = v;
  }
  __device__ __forceinline__ void finish(int) {}
};

// BF16(alpha sum) of the matrix without its padding.
struct EpiNsOut {
  static constexpr bool kTrans = false;
  uint16_t* out;
  int64_t rows, cols;
  float alpha;
  struct Row {};
  struct Col {};
  __device__ __forceinline__ Row row(int, int64_t) const { return Row{}; }
  __device__ __forceinline__ Col col(int, int64_t) const { return Col{}; }
  __device__ __forceinline__ ntu2 pack4(int, int64_t, int64_t, const Row&, const Col&, ntf4 v) const {
    return ntu2{pack_bf16x2(alpha * v[0], alpha * v[1]), pack_bf16x2(alpha * v[2], alpha * v[3])};
  }
  __device__ __forceinline__ void store(int e, int64_t m, int64_t n, const ntu4& v) {
    if (m >= rows || n >= cols) return;
    Raw<uint16_t> r;
    r.v[0] = v;
    store_raw<false>(out + (e * rows + m) * cols, (int)n, (int)cols, r);
  }
  __device__ __forceinline__ void store_t(int, int64_t, int64_t, const ntu4&) {}
  __device__ __forceinline__ void finish(int) {}
};

// w <- keep w - step O, its BF16 copy and that copy's largest magnitude.  O passes
// through LDS in FP16, whose rounding is below the products' own error.
struct EpiNsUpdate {
  static constexpr bool kTrans = false;
  float* w;
  uint16_t* wb;
  float* amax;                   // null: none
  int64_t rows, cols;
  float alpha, keep, step;
  uint32_t most;
  struct Row {};
  struct Col {};
  __device__ __forceinline__ Row row(int, int64_t) const { return Row{}; }
  __device__ __forceinline__ Col col(int, int64_t) const { return Col{}; }
  __device__ __forceinline__ ntu2 pack4(int, int64_t, int64_t, const Row&, const Col&, ntf4 v) const {
    return ntu2{pack_f16x2(alpha * v[0], alpha * v[1]), pack_f16x2(alpha * v[2], alpha * v[3])};
  }
  __device__ __forceinline__ void store(int e, int64_t m, int64_t n, const ntu4& v) {
    if (m >= rows || n >= cols) return;
    const int64_t at = (e * rows + m) * cols + n;
    const int len = (int)min((int64_t)8, cols - n);
    Raw<float> r = load_raw<false>(w + at, 0, len);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = keep * raw_at(r, i) - step * (i & 1 ? f16_hi(v[i >> 1]) : f16_lo(v[i >> 1]));
    Raw<uint16_t> b;
#pragma unroll
    for (int i = 0; i < 4; ++i) b.v[0][i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r.v[i >> 2][i & 3] = f2u(y[i]);
      if (i < len) most = max(most, i & 1 ? b.v[0][i >> 1] & 0x7FFF0000u : b.v[0][i >> 1] << 17 >> 1);
    }
    store_raw<false>(w + at, 0, len, r);
    store_raw<false>(wb + at, 0, len, b);
  }
  __device__ __forceinline__ void store_t(int, int64_t, int64_t, const ntu4&) {}
  __device__ __forceinline__ void finish(int) {
    if (!amax) return;
    const uint32_t m = wave_max_dpp(most);
    if ((threadIdx.x & 63) == 0) atomicMax(reinterpret_cast<uint32_t*>(amax), m);
  }
};

template <typename Epi>
hipError_t product(const uint16_t* a, const uint16_t* b, int64_t M, int64_t N, int64_t K, int64_t batch, bool sym,
                   const Epi& epi, hipStream_t s) {
  const NtArgs g{reinterpret_cast<const uint8_t*>(a), reinterpret_cast<const uint8_t*>(b), M, N, (uint32_t)(2 * K),
                 2 * M * K, 2 * N * K, (int)batch, sym};
  return run_nt_direct<kNtF16, 4, 4, 1, 1, 4>(g, epi, s);
}

struct NsSizes {
  int64_t rows64, cols64, m, n;          // padded; m <= n
  int64_t x, sq;                         // elements of one X and of one m x m matrix
  int64_t parts_bytes, bytes;
  int parts;
};
bool ns_sizes(int64_t batch, int64_t rows, int64_t cols, NsSizes* z) {
  z->rows64 = (rows + 63) / 64 * 64;
  z->cols64 = (cols + 63) / 64 * 64;
  z->m = std::min(z->rows64, z->cols64);
  z->n = std::max(z->rows64, z->cols64);
  // 32-bit offsets of a tile's rows and of a tile count
  if (z->n >= ((int64_t)1 << 22) || batch > 65535) return false;
  z->x = z->m * z->n;
  z->sq = z->m * z->m;
  const int64_t n = rows * cols;
  z->parts = (int)std::max<int64_t>(1, std::min<int64_t>(kParts, (n + 16383) / 16384));
  z->parts_bytes = (batch * z->parts * 8 + 255) / 256 * 256;
  z->bytes = z->parts_bytes + batch * 2 * (3 * z->x + 4 * z->sq);
  return true;
}

}  // namespace

int64_t ortho_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
  NsSizes z;
  return ns_sizes(batch, rows, cols, &z) ? z.bytes : -1;
}

hipError_t launch_ortho(const OrthoArgs& o, hipStream_t s) {
  NsSizes z;
  if (!ns_sizes(o.batch, o.rows, o.cols, &z)) return hipErrorInvalidValue;
  double* part = static_cast<double*>(o.workspace);
  uint16_t* p = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(o.workspace) + z.parts_bytes);
  const int64_t B = o.batch, X = B * z.x, S = B * z.sq;
  // x [m][n] and its transposes xt, xn [n][m]; the m x m matrices
  uint16_t *x = p, *xt = p + X, *xn = p + 2 * X, *ga = p + 3 * X, *q = ga + S, *t = q + S, *pp = t + S;
  const bool wide = z.rows64 == z.m;                       // rows <= cols: x has the matrix's own orientation

  const NsSource src{o.x, o.momentum, static_cast<const uint16_t*>(o.grad), o.mu, o.nesterov ? 1 : 0};
  const dim3 gm((unsigned)z.parts, (unsigned)B);
  const int64_t tiles = z.rows64 / 64 * (z.cols64 / 64);
  const int turns = (int)std::min<int64_t>(4, (tiles * B + 2047) / 2048);
  const dim3 gs((unsigned)((tiles + turns - 1) / turns), (unsigned)B);
  uint16_t *own = wide ? x : xt, *other = wide ? xt : x;
#define BSQ_NS_IN(IN)                                                                                              \
  hipLaunchKernelGGL(k_ns_moment<IN>, gm, dim3(256), 0, s, src, o.rows * o.cols, part);                            \
  hipLaunchKernelGGL(k_ns_scale<IN>, gs, dim3(256), 0, s, src, o.rows, o.cols, z.parts, part, o.eps, own, other,   \
                     z.rows64, z.cols64, turns)
  if (o.w) {
    BSQ_NS_IN(kNsMoment);
  } else if (o.f32) {
    BSQ_NS_IN(kNsF32);
  } else {
    BSQ_NS_IN(kNsBf16);
  }
#undef BSQ_NS_IN
  if (o.amax) hipLaunchKernelGGL(k_ns_zero, dim3(1), dim3(1), 0, s, o.amax);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;

  const auto square = [&](const uint16_t* a, const uint16_t* b, uint16_t* c, int64_t K, const uint16_t* add, float alpha,
                          float beta, float gamma) {
    const EpiNs epi{c, c, add, z.m, z.m, z.sq, z.m, z.m, alpha, beta, gamma};
    return product(a, b, z.m, z.m, K, B, true, epi, s);
  };
  for (int i = 0; i < o.steps; ++i) {
    const float* c = o.coefs + 3 * i;
    const bool last = i + 1 == o.steps;
    e = square(x, x, ga, z.n, nullptr, kSA / (kSX * kSX), 0.0f, 0.0f);
    if (e != hipSuccess) return e;
    e = square(ga, ga, q, z.m, ga, c[2] * (kSP / (kSA * kSA)), c[1] * (kSP / kSA), c[0] * kSP);
    if (e != hipSuccess) return e;
    if (!last) {
      const EpiNs epi{xn, x, nullptr, z.m, z.n, z.x, z.n, z.m, 1.0f / kSP, 0.0f, 0.0f};
      e = product(xt, q, z.n, z.m, z.m, B, false, epi, s);
      std::swap(xt, xn);
    } else {
      const uint16_t *l = wide ? q : xt, *r = wide ? xt : q;
      const float alpha = 1.0f / (kSP * kSX);
      if (o.w) {
        const EpiNsUpdate epi{o.w, static_cast<uint16_t*>(o.w_bf16), o.amax, o.rows, o.cols, alpha, o.keep, o.step, 0u};
        e = product(l, r, z.rows64, z.cols64, z.m, B, false, epi, s);
      } else {
        const EpiNsOut epi{static_cast<uint16_t*>(o.out), o.rows, o.cols, alpha};
        e = product(l, r, z.rows64, z.cols64, z.m, B, false, epi, s);
      }
    }
    if (e != hipSuccess) return e;
  }
  (void)t;
  (void)pp;
  return hipSuccess;
}

}  // namespace bsq
