// Orthogonalisation of matrices by Newton-Schulz products, and the weight update
// that takes it, for gfx950 (contract in include/bsq.h):
//   X = u / (||u||_F + eps);  per step  A = X X^T,  X <- (a I + b A + c A^2) X
//
// The products run on the FP16 MFMA (FP32 sums), and what they leave is held so that the
// result stays near the 64-bit one, where small roundings near singular value zero are
// multiplied by a in every step:
//  * X as an FP16 matrix X' and the FP16 rest x of its rounding (22 bits).  With D the diagonal
//    of the polynomial P and O the rest of it, the MFMAs form O X', the epilogue adds D X' and,
//    in place of P x, a multiple of x: a x (a the step's leading coefficient, the product of
//    both of a pair), but D x in the last two phases.
//    What that leaves out is (P - a) x, or (P - D) x.  P is a I where singular values are near
//    zero, which each later step multiplies by its a again (3.4^4 in all, and 3.4^7 of eight
//    steps): there the first form leaves out nothing, the second a - D, which is not small
//    unless the matrix has full rank.  Where they are not, nothing grows, and D is the nearer
//    one.  (D x in every phase: a matrix of rank 1 of 16 x 16 is 2e-2 from the 64-bit result
//    after five steps, 6e-1 after eight; so 1e-3 and 2e-3.  a x in every phase: full rank 1.1e-3
//    for 7e-4.)
//  * the symmetric matrices (A, the polynomials) as their diagonal in FP32 and the rest in
//    FP16, so that the largest entries are not rounded.
// Five steps, relative to the 64-bit result (Frobenius), by these roundings: gradients 3e-4 to
// 1e-3, any rank from 1 to full and singular values over e^5 and e^9 at most 1.5e-3, in pairs of
// steps 3.8e-3 (at rank m / 3), and 5e-3 for fewer than 16 rows; everything in FP16 2e-2, in BF16
// 2e-1 on a matrix of rank 8 over a floor of 1e-2.
//
// Everything is computed on the smaller side m of the matrix, padded with zeros to
// multiples of 64 in both directions (zero rows and columns stay zero), so that the
// products need no edges.
#include "bsq_nt.hpp"
#include "bsq_nt_ring.hpp"
#include "bsq_ortho.hpp"
#include "bsq_wave.hpp"

#include <algorithm>
#include <cmath>

namespace bsq {

__global__ void k_ns_zero(float* p) { *p = 0.0f; }

namespace {

constexpr float kLo = 2048.0f;           // of the rest of X's rounding, at most 2^-11 of X
constexpr int kParts = 256;              // most workgroups that sum one matrix's squares

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

// X0 in FP16 in the matrix's own orientation (a [rows64][cols64]; lo: the rest of its
// rounding) and transposed (at), 64 x 64 elements a turn, zeros in the padding.
template <int IN>
__global__ __launch_bounds__(256) void k_ns_scale(NsSource src, int64_t rows, int64_t cols, int parts,
                                                  const double* __restrict__ part, float eps, uint16_t* __restrict__ a,
                                                  uint16_t* __restrict__ lo, uint16_t* __restrict__ at, int64_t rows64,
                                                  int64_t cols64, int turns) {
  constexpr int LD = 66;
  __shared__ double lds[4];
  __shared__ uint16_t tile[64 * LD];
  const int t = threadIdx.x;
  const double sum = block_sum(t < parts ? part[(int64_t)blockIdx.y * parts + t] : 0.0, lds);
  const NsNorm norm = ns_norm(sum, eps);
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
      ntu4 v, l;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x0 = ns_scaled(u[2 * j], norm), x1 = ns_scaled(u[2 * j + 1], norm);
        v[j] = pack_f16x2_stored(x0, x1);
        l[j] = pack_f16x2((x0 - f16_lo(v[j])) * kLo, (x1 - f16_hi(v[j])) * kLo);
      }
      *reinterpret_cast<ntu4*>(a + pad + r * cols64 + col) = v;
      *reinterpret_cast<ntu4*>(lo + pad + r * cols64 + col) = l;
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

// ---------------------------------------------------------------- epilogues

// A symmetric matrix: the diagonal d [m] in FP32, and e [m][m] in FP16 under kS with zeros
// on the diagonal.
struct NsSquare {
  uint16_t* e;
  float* d;
};

// A wave's part of a padded matrix of rows x cols, both multiples of 16, so that a 16 x 16
// block lies inside or outside as a whole.  Blocks outside are computed on the last one's
// inputs and not stored; a part that lies outside altogether is computed on the first's.
struct NsPart {
  int M, N;                      // rows and columns from the part's first
  bool dead;
  int64_t m0, n0;
  uint32_t lane;                 // the lane's element in a block
  __device__ __forceinline__ void at(int rows, int cols, int64_t m, int64_t n, int r16, int c4) {
    dead = m >= rows || n >= cols;
    m0 = dead ? 0 : m;
    n0 = dead ? 0 : n;
    M = rows - (int)m0;
    N = cols - (int)n0;
    lane = (uint32_t)(r16 * cols + c4);
  }
  // the block's first element, from the part's, in a matrix with rows of cols
  __device__ __forceinline__ int block(int i, int j, int cols) const { return min(16 * i, M - 16) * cols + min(16 * j, N - 16); }
  __device__ __forceinline__ bool inside(int i, int j) const { return !dead && 16 * i < M && 16 * j < N; }
};
// Four 16-bit elements of the lane: a uniform address plus the lane's offset, so that a
// block costs scalar operations only.
__device__ __forceinline__ ntu2 ns_load(const uint16_t* p, int block, uint32_t lane) {
  const uint16_t* q = p + block;
  return *reinterpret_cast<const ntu2*>(reinterpret_cast<const uint8_t*>(q) + 2u * lane);
}

// A symmetric product of two such matrices, the MFMAs having formed the product of their
// FP16 parts: of two different ones (kNsProduct), or a matrix's polynomial (kNsPoly, l is
// r), or of X and its transpose (kNsGram, neither); the tile on the other side of the
// diagonal is stored too.
//   entry (i, j)  alpha sum + r_ij (k0 + k1 dl_i) + l_ij (k0 + k1 dr_j)
//   entry (i, i)  alpha / kS sum + q0 + q1 dl_i + q2 dl_i dr_i, in FP32
enum NsMode { kNsGram = 0, kNsPoly = 1, kNsProduct = 2 };
template <int MODE>
struct EpiNsSquare {
  static constexpr bool kTrans = true;
  static constexpr float kWork = MODE == kNsGram ? 0.0f : MODE == kNsPoly ? 1.0f : 1.4f;
  NsSquare c;
  const uint16_t* l;
  const uint16_t* r;
  const float* dl;
  const float* dr;
  int side;                      // at most 2^22; offsets inside a tile's rows fit 32 bits
  float alpha, k0, k1, q0, q1, q2;
  uint16_t* t;                   // the tile on the other side of the diagonal
  NsPart p;
  int diag, r16, c4;             // block (i, j) holds the diagonal where 16 i + diag is 16 j
  struct Row { float k; };
  struct Col { ntf4 k; };
  struct Add { ntu2 l, r; };
  typedef EpiNothing Fetch;
  __device__ __forceinline__ void at(int e, int64_t m0, int64_t n0, int r16_, int c4_) {
    p.at(side, side, m0, n0, r16_, c4_);
    const int64_t base = (int64_t)e * side, o = (base + p.m0) * side + p.n0;
    t = c.e + (base + p.n0) * side + p.m0;
    c.e += o;
    c.d += base + p.m0;
    if constexpr (MODE != kNsGram) {
      l += o;
      r += o;
      dl += base + p.m0;
      dr += base + p.n0;
    }
    diag = (int)(p.m0 - p.n0);
    r16 = r16_;
    c4 = c4_;
  }
  __device__ __forceinline__ Row row(int i) const {
    if constexpr (MODE == kNsGram) return Row{0.0f};
    else return Row{__builtin_fmaf(k1, dl[min(16 * i, p.M - 16) + r16], k0)};
  }
  __device__ __forceinline__ Col col(int j) const {
    Col k{ntf4{0.0f, 0.0f, 0.0f, 0.0f}};
    if constexpr (MODE != kNsGram) {
      const ntf4 d = *reinterpret_cast<const ntf4*>(dr + min(16 * j, p.N - 16) + c4);
#pragma unroll
      for (int i = 0; i < 4; ++i) k.k[i] = __builtin_fmaf(k1, d[i], k0);
    }
    return k;
  }
  __device__ __forceinline__ void add(Add& x, int i, int j) const {
    if constexpr (MODE != kNsGram) x.r = ns_load(r, p.block(i, j, side), p.lane);
    if constexpr (MODE == kNsProduct) x.l = ns_load(l, p.block(i, j, side), p.lane);
  }
  __device__ __forceinline__ ntu2 pack4(int i, int j, const Row& a, const Col& b, const Add& x, ntf4 v) const {
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      y[k] = alpha * v[k];
      if constexpr (MODE != kNsGram) {
        const float xr = k & 1 ? f16_hi(x.r[k >> 1]) : f16_lo(x.r[k >> 1]);
        if constexpr (MODE == kNsPoly) {
          y[k] = __builtin_fmaf(xr, a.k + b.k[k], y[k]);
        } else {
          const float xl = k & 1 ? f16_hi(x.l[k >> 1]) : f16_lo(x.l[k >> 1]);
          y[k] = __builtin_fmaf(xl, b.k[k], __builtin_fmaf(xr, a.k, y[k]));
        }
      }
    }
    if (16 * i + diag == 16 * j && p.inside(i, j)) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (r16 == c4 + k) {
          float d = alpha * (1.0f / kS) * v[k];
          if constexpr (MODE != kNsGram) {
            const float u = dl[16 * i + r16], w = dr[16 * j + r16];
            d += q0 + q1 * u + q2 * (u * w);
          }
          c.d[16 * i + r16] = d;
          y[k] = 0.0f;
        }
    }
    return ntu2{pack_f16x2(y[0], y[1]), pack_f16x2(y[2], y[3])};
  }
  __device__ __forceinline__ void fetch(Fetch&, int, int) const {}
  __device__ __forceinline__ void store(int m, int n, const ntu4& v, const Fetch&) {
    if (!p.dead && m < p.M && n < p.N) *reinterpret_cast<ntu4*>(c.e + (uint32_t)(m * side + n)) = v;
  }
  __device__ __forceinline__ void store_t(int n, int m, const ntu4& v) {
    if (!p.dead && m < p.M && n < p.N) *reinterpret_cast<ntu4*>(t + (uint32_t)(n * side + m)) = v;
  }
  __device__ __forceinline__ void finish(uint8_t*) {}
};

// What the products P X (X in the matrix's own orientation, rows x cols) add to the MFMAs'
// sum of P's FP16 part and X's: P's diagonal times X's, and its rest times own d + lead, d
// being the diagonal's entry: a number (own 0), or the diagonal itself (own 1, lead 0).  In
// units of X under kS.  WIDE: rows <= cols, the diagonal runs along the rows.
template <bool WIDE>
struct NsApply {
  const uint16_t* hi;
  const uint16_t* lo;
  const float* d;
  int rows, cols;
  float own, lead;               // both over kLo
  NsPart p;
  int r16, c4;
  struct Row { float d, e; };
  struct Col { ntf4 d; };
  struct Add { ntu2 hi, lo; };
  __device__ __forceinline__ int64_t at(int e, int64_t m0, int64_t n0, int r16_, int c4_) {
    p.at(rows, cols, m0, n0, r16_, c4_);
    const int64_t o = ((int64_t)e * rows + p.m0) * cols + p.n0;
    hi += o;
    lo += o;
    d += WIDE ? (int64_t)e * rows + p.m0 : (int64_t)e * cols + p.n0;
    r16 = r16_;
    c4 = c4_;
    return o;
  }
  __device__ __forceinline__ Row row(int i) const {
    if constexpr (!WIDE) return Row{0.0f, 0.0f};
    const float v = d[min(16 * i, p.M - 16) + r16];
    return Row{v, __builtin_fmaf(own, v, lead)};
  }
  __device__ __forceinline__ Col col(int j) const {
    if constexpr (WIDE) return Col{ntf4{0.0f, 0.0f, 0.0f, 0.0f}};
    else return Col{*reinterpret_cast<const ntf4*>(d + min(16 * j, p.N - 16) + c4)};
  }
  __device__ __forceinline__ void add(Add& x, int i, int j) const {
    const int b = p.block(i, j, cols);
    x.hi = ns_load(hi, b, p.lane);
    x.lo = ns_load(lo, b, p.lane);
  }
  __device__ __forceinline__ void sums(const Row& a, const Col& b, const Add& o, ntf4 v, float (&y)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float h = i & 1 ? f16_hi(o.hi[i >> 1]) : f16_lo(o.hi[i >> 1]);
      const float l = i & 1 ? f16_hi(o.lo[i >> 1]) : f16_lo(o.lo[i >> 1]);
      const float x = WIDE ? __builtin_fmaf(l, a.e, a.d * h) : __builtin_fmaf(l, __builtin_fmaf(own, b.d[i], lead), b.d[i] * h);
      y[i] = __builtin_fmaf(v[i], 1.0f / kS, x);
    }
  }
};

// The next X: FP16, the rest of its rounding (in place), and its transpose.
template <bool WIDE>
struct EpiNsNext {
  static constexpr bool kTrans = true;
  static constexpr float kWork = 1.7f;
  NsApply<WIDE> x;
  uint16_t* hi;
  uint16_t* lo;
  uint16_t* t;
  typedef typename NsApply<WIDE>::Row Row;
  typedef typename NsApply<WIDE>::Col Col;
  typedef typename NsApply<WIDE>::Add Add;
  typedef EpiNothing Fetch;
  __device__ __forceinline__ void at(int e, int64_t m0, int64_t n0, int r16, int c4) {
    const int64_t o = x.at(e, m0, n0, r16, c4);
    hi += o;
    lo += o;
    t += ((int64_t)e * x.cols + x.p.n0) * x.rows + x.p.m0;
  }
  __device__ __forceinline__ Row row(int i) const { return x.row(i); }
  __device__ __forceinline__ Col col(int j) const { return x.col(j); }
  __device__ __forceinline__ void add(Add& o, int i, int j) const { x.add(o, i, j); }
  __device__ __forceinline__ ntu2 pack4(int i, int j, const Row& a, const Col& b, const Add& o, ntf4 v) const {
    float y[4];
    x.sums(a, b, o, v, y);
    const ntu2 h = {pack_f16x2_stored(y[0], y[1]), pack_f16x2_stored(y[2], y[3])};
    if (x.p.inside(i, j)) {
      float l[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)                          // (y - h) kLo, exact
        l[k] = __builtin_fmaf(k & 1 ? f16_hi(h[k >> 1]) : f16_lo(h[k >> 1]), -kLo, y[k] * kLo);
      uint16_t* q = lo + x.p.block(i, j, x.cols);
      *reinterpret_cast<ntu2*>(reinterpret_cast<uint8_t*>(q) + 2u * x.p.lane) =
          ntu2{pack_f16x2(l[0], l[1]), pack_f16x2(l[2], l[3])};
    }
    return h;
  }
  __device__ __forceinline__ void fetch(Fetch&, int, int) const {}
  __device__ __forceinline__ void store(int m, int n, const ntu4& v, const Fetch&) {
    if (!x.p.dead && m < x.p.M && n < x.p.N) *reinterpret_cast<ntu4*>(hi + (uint32_t)(m * x.cols + n)) = v;
  }
  __device__ __forceinline__ void store_t(int n, int m, const ntu4& v) {
    if (!x.p.dead && m < x.p.M && n < x.p.N) *reinterpret_cast<ntu4*>(t + (uint32_t)(n * x.rows + m)) = v;
  }
  __device__ __forceinline__ void finish(uint8_t*) {}
};

// BF16(X) of the matrix without its padding.
template <bool WIDE>
struct EpiNsOut {
  static constexpr bool kTrans = false;
  static constexpr float kWork = 0.8f;
  NsApply<WIDE> x;
  uint16_t* out;
  int rows, cols;
  int M, N;
  typedef typename NsApply<WIDE>::Row Row;
  typedef typename NsApply<WIDE>::Col Col;
  typedef typename NsApply<WIDE>::Add Add;
  typedef EpiNothing Fetch;
  __device__ __forceinline__ void at(int e, int64_t m0, int64_t n0, int r16, int c4) {
    x.at(e, m0, n0, r16, c4);
    out += ((int64_t)e * rows + m0) * cols + n0;
    M = rows - (int)m0;
    N = cols - (int)n0;
  }
  __device__ __forceinline__ Row row(int i) const { return x.row(i); }
  __device__ __forceinline__ Col col(int j) const { return x.col(j); }
  __device__ __forceinline__ void add(Add& o, int i, int j) const { x.add(o, i, j); }
  __device__ __forceinline__ ntu2 pack4(int, int, const Row& a, const Col& b, const Add& o, ntf4 v) const {
    float y[4];
    x.sums(a, b, o, v, y);
    constexpr float k = 1.0f / kS;
    return ntu2{pack_bf16x2(k * y[0], k * y[1]), pack_bf16x2(k * y[2], k * y[3])};
  }
  __device__ __forceinline__ void fetch(Fetch&, int, int) const {}
  __device__ __forceinline__ void store(int m, int n, const ntu4& v, const Fetch&) {
    if (m >= M || n >= N) return;
    Raw<uint16_t> r;
    r.v[0] = v;
    store_raw<false>(out + (m * cols + n), 0, N - n, r);
  }
  __device__ __forceinline__ void store_t(int, int, const ntu4&) {}
  __device__ __forceinline__ void finish(uint8_t*) {}
};

// w <- keep w - step X, its BF16 copy and that copy's largest magnitude.  X passes
// through LDS in FP16 (2^-11 of an entry, below the products' own error).
template <bool WIDE>
struct EpiNsUpdate {
  static constexpr bool kTrans = false;
  static constexpr float kWork = 1.2f;
  NsApply<WIDE> x;
  float* w;
  uint16_t* wb;
  float* amax;                   // null: none
  int rows, cols;
  float keep, step;              // step of X under kS
  uint32_t most;
  int M, N;
  typedef typename NsApply<WIDE>::Row Row;
  typedef typename NsApply<WIDE>::Col Col;
  typedef typename NsApply<WIDE>::Add Add;
  typedef Raw<float> Fetch;
  __device__ __forceinline__ void at(int e, int64_t m0, int64_t n0, int r16, int c4) {
    x.at(e, m0, n0, r16, c4);
    const int64_t o = ((int64_t)e * rows + m0) * cols + n0;
    w += o;
    wb += o;
    M = rows - (int)m0;
    N = cols - (int)n0;
  }
  __device__ __forceinline__ Row row(int i) const { return x.row(i); }
  __device__ __forceinline__ Col col(int j) const { return x.col(j); }
  __device__ __forceinline__ void add(Add& o, int i, int j) const { x.add(o, i, j); }
  __device__ __forceinline__ ntu2 pack4(int, int, const Row& a, const Col& b, const Add& o, ntf4 v) const {
    float y[4];
    x.sums(a, b, o, v, y);
    return ntu2{pack_f16x2(y[0], y[1]), pack_f16x2(y[2], y[3])};
  }
  __device__ __forceinline__ void fetch(Fetch& r, int m, int n) const {
    if (m < M && n < N) r = load_raw<false>(w + (m * cols + n), 0, min(8, N - n));
  }
  __device__ __forceinline__ void store(int m, int n, const ntu4& v, Fetch& r) {
    if (m >= M || n >= N) return;
    const int at = m * cols + n, len = min(8, N - n);
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
  __device__ __forceinline__ void store_t(int, int, const ntu4&) {}
  // one atomic a workgroup, and none where the maximum is there already: all go to one
  // address (8 x 520 x 1,000: 4,608 of them took 40 us)
  __device__ __forceinline__ void finish(uint8_t* lds) {
    if (!amax) return;
    uint32_t* all = reinterpret_cast<uint32_t*>(lds);
    const uint32_t m = wave_max_dpp(most);
    __syncthreads();                                       // the tile's pieces are read
    if ((threadIdx.x & 63) == 0) all[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x != 0) return;
    const uint32_t b = max(max(all[0], all[1]), max(all[2], all[3]));
    uint32_t* a = reinterpret_cast<uint32_t*>(amax);
    if (b > __hip_atomic_load(a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicMax(a, b);
  }
};

template <typename Epi>
hipError_t product(const OrthoArgs& o, const uint16_t* a, const uint16_t* b, int64_t M, int64_t N, int64_t K, bool sym,
                   const Epi& epi, hipStream_t s) {
  const NtArgs g{reinterpret_cast<const uint8_t*>(a), reinterpret_cast<const uint8_t*>(b), M, N, (uint32_t)(2 * K),
                 2 * M * K, 2 * N * K, (int)o.batch, sym};
  if (o.kernel == kNtChosen) return run_nt_choice<kNtF16, false>(g, nt_choose(g, false, true, true, Epi::kWork), epi, s);
  const int side = nt_side(o.kernel), half = (int)(nt_tiles(g, side, side) / 2);
  const bool cut = o.rest != kNtChosen && half > 0;
  return run_nt_choice<kNtF16, false>(g, NtChoice{o.kernel, cut ? half : -1, o.rest, side / nt_side(o.rest)}, epi, s);
}

struct NsSizes {
  int64_t rows64, cols64, m, n;          // padded; m <= n
  int64_t x, sq;                         // elements of one X and of one m x m matrix
  int64_t parts_bytes, diag_bytes, bytes;
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
  z->diag_bytes = batch * z->m * 4;                        // a multiple of 256
  z->bytes = z->parts_bytes + 4 * z->diag_bytes + batch * 2 * (4 * z->x + 4 * z->sq);
  return true;
}

// P X in the matrix's own orientation, X being x [m][n] and its transpose xt: the next X
// (x, its transpose xn, the rest lo), or the result.  own, lead: NsApply's, in units of X.
struct NsBuffers {
  uint16_t* x;
  uint16_t* xt;
  uint16_t* xn;
  uint16_t* lo;
  NsSquare p;
};
template <bool WIDE>
hipError_t apply(const OrthoArgs& o, const NsSizes& z, const NsBuffers& b, float own, float lead, bool more, hipStream_t s) {
  const uint16_t *l = WIDE ? b.p.e : b.xt, *r = WIDE ? b.xt : b.p.e;
  const NsApply<WIDE> a{WIDE ? b.x : b.xt, b.lo, b.p.d, (int)z.rows64, (int)z.cols64, own / kLo, lead / kLo};
  const auto run = [&](const auto& epi) { return product(o, l, r, z.rows64, z.cols64, z.m, false, epi, s); };
  if (more) return run(EpiNsNext<WIDE>{a, WIDE ? b.x : b.xn, b.lo, WIDE ? b.xn : b.x});
  if (o.w)
    return run(EpiNsUpdate<WIDE>{a, o.w, static_cast<uint16_t*>(o.w_bf16), o.amax, (int)o.rows, (int)o.cols, o.keep,
                                 o.step / kS, 0u, 0, 0});
  return run(EpiNsOut<WIDE>{a, static_cast<uint16_t*>(o.out), (int)o.rows, (int)o.cols, 0, 0});
}

// Steps from step i on that share one Gram matrix, the phase before having been of
// `before`.  After A = X X^T, the next step's Gram matrix is Q A Q with the polynomial
// Q = a I + b A + c A^2, and the product P of both polynomials is applied to X once: two
// steps take 1.5 m^2 n + 2.5 m^3 multiply-adds (symmetric products counted half), one by
// one 3 m^2 n + m^3.  But Q A Q multiplies A's rounding at singular values near zero by
// a^2 until A is formed afresh, so a pair is followed by a single step, and is taken
// where the matrix is far enough from square to have few singular values near zero and
// the a's are small (at most 12; the usual ones 11.9).  Simulated distance from the 64-bit
// result one by one / in pairs with singles between: gradients of 512 x 1,792 4.2e-4,
// 2.9e-4 (2 and 3 steps at once: 6.4e-4), 600 x 800 5.5e-4, 8.0e-4, 1,024 x 1,024 5.9e-4,
// 1.4e-3 (4.1e-3); singular values spread over e^5 at 600 x 800 6.1e-4, 1.9e-3 (9.7e-3; all five
// at once 2.6e-2); rank 128 at 320 x 512 1e-3, 3.8e-3.  16 x 1,408 x 2,048: 1,981 us one by one, 1,788 in pairs;
// but a pair is 7 launches, two steps 6, which is what a small matrix costs (192 x 256: 79 us
// one by one, 93 in pairs).
int phase_steps(const OrthoArgs& o, const NsSizes& z, int i, int before) {
  return z.m > 256 && 3 * z.n >= 4 * z.m && before != 2 && i + 2 <= o.steps &&
                 std::fabs(o.coefs[3 * i] * o.coefs[3 * i + 3]) <= 12.0f
             ? 2
             : 1;
}

}  // namespace

int64_t ortho_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
  NsSizes z;
  return ns_sizes(batch, rows, cols, &z) ? z.bytes : -1;
}

hipError_t launch_ortho(const OrthoArgs& o, hipStream_t s) {
  if (o.kernel == kNtChosen && ortho_in_one(o.rows, o.cols)) return launch_ortho_one(o, s);
  NsSizes z;
  if (!ns_sizes(o.batch, o.rows, o.cols, &z)) return hipErrorInvalidValue;
  double* part = static_cast<double*>(o.workspace);
  float* diag = reinterpret_cast<float*>(static_cast<uint8_t*>(o.workspace) + z.parts_bytes);
  uint16_t* p = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(diag) + 4 * z.diag_bytes);
  const int64_t B = o.batch, X = B * z.x, S = B * z.sq;
  // x [m][n]; its transpose xt and the next one xn [n][m]; lo in the matrix's own orientation
  uint16_t *x = p, *xt = p + X, *xn = p + 2 * X, *lo = p + 3 * X;
  const auto matrix = [&](int i) { return NsSquare{p + 4 * X + i * S, diag + i * B * z.m}; };
  NsSquare ga = matrix(0), q = matrix(1), t = matrix(2), pp = matrix(3);
  // x has the matrix's own orientation.  By the true sizes: on the larger side, where the
  // padded ones are equal, the Gram matrix has singular values zero, along which roundings
  // grow (7 x 5: 2.6e-3 from the 64-bit result against 8e-4)
  const bool wide = o.rows <= o.cols;

  const NsSource src{o.x, o.momentum, static_cast<const uint16_t*>(o.grad), o.mu, o.nesterov ? 1 : 0};
  const dim3 gm((unsigned)z.parts, (unsigned)B);
  const int64_t tiles = z.rows64 / 64 * (z.cols64 / 64);
  const int turns = (int)std::min<int64_t>(4, (tiles * B + 2047) / 2048);
  const dim3 gs((unsigned)((tiles + turns - 1) / turns), (unsigned)B);
  uint16_t *own = wide ? x : xt, *other = wide ? xt : x;
#define BSQ_NS_IN(IN)                                                                                              \
  hipLaunchKernelGGL(k_ns_moment<IN>, gm, dim3(256), 0, s, src, o.rows * o.cols, part);                            \
  hipLaunchKernelGGL(k_ns_scale<IN>, gs, dim3(256), 0, s, src, o.rows, o.cols, z.parts, part, o.eps, own, lo,      \
                     other, z.rows64, z.cols64, turns)
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

  // c = the product of symmetric matrices l and r, or a I + b l + c l^2
  const auto multiply = [&](const NsSquare& l, const NsSquare& r, const NsSquare& c) {
    EpiNsSquare<kNsProduct> epi{c, l.e, r.e, l.d, r.d, (int)z.m};
    epi.alpha = 1.0f / kS, epi.k1 = 1.0f, epi.q2 = 1.0f;
    return product(o, l.e, r.e, z.m, z.m, z.m, true, epi, s);
  };
  const auto polynomial = [&](const NsSquare& l, const NsSquare& c, const float* k) {
    EpiNsSquare<kNsPoly> epi{c, l.e, l.e, l.d, l.d, (int)z.m};
    epi.alpha = k[2] / kS, epi.k0 = 0.5f * k[1], epi.k1 = k[2], epi.q0 = k[0], epi.q1 = k[1], epi.q2 = k[2];
    return product(o, l.e, l.e, z.m, z.m, z.m, true, epi, s);
  };
  int phases = 0;
  for (int i = 0, r = 0; i < o.steps; i += r, ++phases) r = phase_steps(o, z, i, r);
  for (int i = 0, r = 0; i < o.steps; --phases) {
    r = phase_steps(o, z, i, r);
    const bool last = phases <= 2;                         // of two
    const float own = last ? 1.0f : 0.0f, lead = last ? 0.0f : o.coefs[3 * i] * (r == 2 ? o.coefs[3 * i + 3] : 1.0f);
    EpiNsSquare<kNsGram> gram{ga, nullptr, nullptr, nullptr, nullptr, (int)z.m};
    gram.alpha = 1.0f / kS;
    e = product(o, x, x, z.m, z.m, z.n, true, gram, s);
    if (e == hipSuccess) e = polynomial(ga, pp, o.coefs + 3 * i);
    if (r == 2) {
      if (e == hipSuccess) e = multiply(pp, ga, t);
      if (e == hipSuccess) e = multiply(t, pp, ga);
      if (e == hipSuccess) e = polynomial(ga, q, o.coefs + 3 * i + 3);
      if (e == hipSuccess) e = multiply(q, pp, t);
      std::swap(pp, t);
    }
    i += r;
    const NsBuffers b{x, xt, xn, lo, pp};
    if (e == hipSuccess) e = wide ? apply<true>(o, z, b, own, lead, i < o.steps, s) : apply<false>(o, z, b, own, lead, i < o.steps, s);
    if (e != hipSuccess) return e;
    std::swap(xt, xn);
  }
  return hipSuccess;
}

}  // namespace bsq
