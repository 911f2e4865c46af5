// C-ABI entry points of libbsq: argument validation and kernel dispatch.
// The contract of every function is documented in include/bsq.h.
#include "bsq.h"

#include <hip/hip_runtime.h>

#include <map>
#include <mutex>
#include <utility>

#include "bsq_internal.hpp"

namespace bsq {

hipError_t set_lds_limit(const void* fn, int bytes) {
  static std::mutex mu;
  static std::map<std::pair<int, const void*>, hipError_t> done;   // (device, kernel) -> result
  int dev = 0;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_pair(dev, fn);
  const auto it = done.find(key);
  if (it != done.end()) return it->second;
  const hipError_t r = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  try {
    done.emplace(key, r);
  } catch (...) {   // no host memory to remember it: set again by the next call (nothing is thrown through the C entry)
  }
  return r;
}

int device_cus() {
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static int cus[kMaxDevices] = {};   // device -> compute units (0: not looked up yet)
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (cus[dev] == 0 &&
      hipDeviceGetAttribute(&cus[dev], hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    cus[dev] = 0;
  return cus[dev];
}

}  // namespace bsq

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned16_or_null(const void* p) { return p == nullptr || aligned16(p); }

// Device pointers handed to us must at least be 4-byte aligned for scalars.
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bsq_status hip_status(hipError_t e) { return e == hipSuccess ? BSQ_OK : BSQ_EHIP; }

// a * b would exceed 2^48 (no device holds that many elements; the bound also
// keeps every byte offset the kernels form far inside int64).  a, b >= 0.
bool too_many(int64_t a, int64_t b) { return a > 0 && b > (((int64_t)1 << 48) / a); }

// [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + (uintptr_t)nb && pb < pa + (uintptr_t)na;
}

// Checks and dispatch of bs_gemm (static_scratch false: the NVFP4 split
// workspace from the stream-ordered allocator) and bs_gemm_noalloc (true:
// the library's static per-device workspace, nothing allocated).
bsq_status gemm_common(bsq_format fmt, int64_t M, int64_t N, int64_t K, const uint8_t* a_codes,
                       const uint8_t* a_scales, const float* a_amax, const uint8_t* b_codes,
                       const uint8_t* b_scales, const float* b_amax, void* c, int64_t ldc,
                       void* stream, bool static_scratch) {
  if (fmt != BSQ_NVFP4 && fmt != BSQ_MXFP4 && fmt != BSQ_MXFP8 && fmt != BSQ_FP8) return BSQ_EINVAL;
  const bool per_tensor = fmt == BSQ_NVFP4 || fmt == BSQ_FP8;   // alpha from the two amaxes
  if (M < 0 || N < 0 || K < 0) return BSQ_EINVAL;
  if (K % (fmt == BSQ_NVFP4 ? 16 : 32) != 0) return BSQ_EINVAL;
  if (ldc < N || ldc < 0) return BSQ_EINVAL;
  if (too_many(M, K) || too_many(N, K) || too_many(M, ldc)) return BSQ_EINVAL;
  if (M > (int64_t)256 * 0x7FFFFF || N > (int64_t)256 * 0x7FFFFF) return BSQ_EINVAL;
  if (M == 0 || N == 0) return BSQ_OK;
  if (!c || ((reinterpret_cast<uintptr_t>(c) & 1u) != 0)) return BSQ_EINVAL;
  if (K > 0) {
    if (!a_codes || !b_codes) return BSQ_EINVAL;
    if (fmt != BSQ_FP8 && (!a_scales || !b_scales)) return BSQ_EINVAL;
  }
  if (per_tensor && (!a_amax || !b_amax)) return BSQ_EINVAL;
  const bsq::Fmt f = fmt == BSQ_NVFP4 ? bsq::kNVFP4
                     : fmt == BSQ_MXFP4 ? bsq::kMXFP4
                     : fmt == BSQ_MXFP8 ? bsq::kMXFP8 : bsq::kFP8;
  void* scratch = nullptr;
  size_t scratch_bytes = 0;
  if (static_scratch && fmt == BSQ_NVFP4) {
    if (bsq::gemm_nvfp4_static_scratch(&scratch, &scratch_bytes) != hipSuccess) return BSQ_EHIP;
    if (bsq::gemm_nvfp4_scratch_bytes(M, N, K, a_codes, a_scales, b_codes, b_scales) > scratch_bytes)
      return BSQ_EUNSUPPORTED;
  }
  return hip_status(bsq::launch_gemm(f, M, N, K, a_codes, a_scales, a_amax, b_codes, b_scales,
                                     b_amax, c, ldc, scratch, scratch_bytes,
                                     static_cast<hipStream_t>(stream)));
}

// Shared checks and dispatch of the SwiGLU forward (dh null) and backward.
bsq_status swiglu_common(const void* y, const void* dh, int64_t rows, int64_t f, int rht_col,
                         uint16_t signs, void* out, float* amax_row, float* amax_col, void* stream) {
  if (rows < 0 || f < 0 || rows % 16 != 0 || f % 16 != 0) return BSQ_EINVAL;
  if (too_many(rows, 2 * f)) return BSQ_EINVAL;
  if (!aligned4(amax_row) || !aligned4(amax_col)) return BSQ_EINVAL;
  if (f >= ((int64_t)1 << 25)) return BSQ_EINVAL;    // 16 rows of y per buffer resource
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool amax = amax_row || amax_col;
  if (rows * f == 0) return amax ? hip_status(bsq::launch_zero_amax(amax_row, amax_col, s)) : BSQ_OK;
  const bool bwd = dh != nullptr;
  if (!y || !out || !aligned16(y) || !aligned16(out) || !aligned16_or_null(dh)) return BSQ_EINVAL;
  const int64_t ybytes = rows * f * 4, obytes = rows * f * (bwd ? 4 : 2);
  if (overlap(out, obytes, y, ybytes) || (bwd && overlap(out, obytes, dh, rows * f * 2)))
    return BSQ_EINVAL;
  if (amax) {
    const hipError_t e = bsq::launch_zero_amax(amax_row, amax_col, s);
    if (e != hipSuccess) return BSQ_EHIP;
  }
  return hip_status(bsq::launch_swiglu(y, dh, rows, f, amax ? (rht_col ? 2 : 1) : 0, signs, out,
                                       amax_row, amax_col, s));
}

bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

// Alignment of an element of a BF16 (false) or FP32 (true) array.
bool aligned_elem(const void* p, bool f32) { return f32 ? aligned4(p) : aligned2(p); }

bool valid_dtype(bsq_dtype t) { return t == BSQ_BF16 || t == BSQ_F32; }

// Checks shared by block_norm and its backward; 0 = fine.
bsq_status norm_checks(int64_t rows, int64_t cols, bsq_dtype type, const void* o, const float* w_post,
                       bsq_gate kind, const void* gate, const float* w_pre) {
  if (rows < 0 || cols < 1 || too_many(rows, cols) || !valid_dtype(type)) return BSQ_EINVAL;
  if (kind < BSQ_GATE_NONE || kind > BSQ_GATE_FULL) return BSQ_EINVAL;
  if (cols > 16384) return BSQ_EUNSUPPORTED;
  if (!aligned4(w_post) || !aligned4(w_pre) || !aligned2(o)) return BSQ_EINVAL;
  if (rows == 0) return BSQ_OK;                            // empty tensors have null pointers
  if (!o && (w_post || kind != BSQ_GATE_NONE)) return BSQ_EINVAL;
  if (!o && !w_pre) return BSQ_EINVAL;                     // nothing to compute
  if ((kind != BSQ_GATE_NONE) != (gate != nullptr)) return BSQ_EINVAL;
  if (!aligned_elem(gate, kind != BSQ_GATE_FULL)) return BSQ_EINVAL;
  return BSQ_OK;
}

bsq_status route_checks(int64_t tokens, int experts, int k) {
  if (tokens < 0 || experts < 1 || k < 1 || k > experts) return BSQ_EINVAL;
  if (experts > bsq::kMoeMaxExperts || k > bsq::kMoeMaxK) return BSQ_EUNSUPPORTED;
  if (tokens > 0x7FFFFFFF / k) return BSQ_EINVAL;
  return BSQ_OK;
}

bsq_status moe_rows_of(int64_t tokens, int experts, int k, int align, int64_t* rows) {
  const bsq_status st = route_checks(tokens, experts, k);
  if (st != BSQ_OK) return st;
  if (align < 1 || align > 512) return BSQ_EINVAL;
  const int64_t n = tokens * k;
  int64_t r = n;
  if (align > 1) r = (n + (n < experts ? n : experts) * (int64_t)(align - 1) + 511) / 512 * 512;
  if (r > 0x7FFFFFFF) return BSQ_EINVAL;
  *rows = r;
  return BSQ_OK;
}

// moe_route; scored: moe_route_score_bias.
bsq_status route_common(const void* logits, bsq_dtype type, int64_t tokens, int experts, int k,
                        const float* bias, bool scored, bsq_scoring scoring, int normalize, float scale,
                        int align, int64_t rows, int32_t* experts_out, float* weights, int32_t* offsets,
                        int32_t* row_of, int32_t* src, void* workspace, int64_t workspace_bytes,
                        void* stream) {
  int64_t need = 0;
  const bsq_status st = moe_rows_of(tokens, experts, k, align, &need);
  if (st != BSQ_OK) return st;
  if (!valid_dtype(type) || (scoring != BSQ_SOFTMAX && scoring != BSQ_SIGMOID)) return BSQ_EINVAL;
  if (rows < need || rows > 0x7FFFFFFF) return BSQ_EINVAL;
  if (!offsets || !aligned4(offsets) || (rows > 0 && !src) || !aligned4(src)) return BSQ_EINVAL;
  if (scored && !bias) return BSQ_EINVAL;
  if (tokens > 0 && (!logits || !experts_out || !weights || !row_of)) return BSQ_EINVAL;
  if (!aligned_elem(logits, type == BSQ_F32) || !aligned4(bias) || !aligned4(experts_out) ||
      !aligned4(weights) || !aligned4(row_of) || !aligned4(workspace))
    return BSQ_EINVAL;
  const int64_t hist = bsq::moe_route_hist_bytes(tokens, experts);
  if (hist > 0 && (!workspace || workspace_bytes < hist)) return BSQ_EINVAL;
  const bsq::RouteArgs a{logits, type == BSQ_F32, tokens, experts, k, bias, scored, scoring == BSQ_SIGMOID,
                         normalize != 0, scale, align, rows, experts_out, weights, offsets, row_of,
                         src, static_cast<int32_t*>(workspace)};
  return hip_status(bsq::launch_moe_route(a, static_cast<hipStream_t>(stream)));
}

// Element counts and pointers of the token <-> expert row movers.
bsq_status mover_checks(int64_t tokens, int64_t cols, int k, int64_t rows) {
  if (tokens < 0 || cols < 0 || k < 1 || rows < 0 || rows > 0x7FFFFFFF) return BSQ_EINVAL;
  if (tokens > 0x7FFFFFFF / k || too_many(tokens, cols) || too_many(rows, cols)) return BSQ_EINVAL;
  return cols > (1 << 30) ? BSQ_EUNSUPPORTED : BSQ_OK;  // the kernels' column indexes are 32 bits
}

bsq_status grouped_format(bsq_format fmt, bsq::Fmt* f) {
  if (fmt == BSQ_FP8) return BSQ_EUNSUPPORTED;
  if (fmt != BSQ_NVFP4 && fmt != BSQ_MXFP4 && fmt != BSQ_MXFP8) return BSQ_EINVAL;
  *f = fmt == BSQ_NVFP4 ? bsq::kNVFP4 : fmt == BSQ_MXFP4 ? bsq::kMXFP4 : bsq::kMXFP8;
  return BSQ_OK;
}

}  // namespace

extern "C" {

const char* bsq_status_string(bsq_status status) {
  switch (status) {
    case BSQ_OK: return "BSQ_OK";
    case BSQ_EINVAL: return "BSQ_EINVAL: invalid argument (null pointer, size or alignment)";
    case BSQ_EUNSUPPORTED: return "BSQ_EUNSUPPORTED: combination not defined by the recipe";
    case BSQ_EHIP: return "BSQ_EHIP: HIP launch error";
    default: return "BSQ_UNKNOWN";
  }
}

bsq_status nvfp4_quantize(const void* x, int64_t rows, int64_t cols, int block_rows,
                          bsq_rounding rnd, uint64_t seed, uint32_t offset, int rht,
                          uint16_t rht_signs, const float* amax_in, uint8_t* codes,
                          uint8_t* scales, float* amax_out, void* stream) {
  if (rows < 0 || cols < 0 || cols % 16 != 0 || too_many(rows, cols)) return BSQ_EINVAL;
  if (block_rows != 1 && block_rows != 16) return BSQ_EINVAL;
  if (rnd != BSQ_RNE && rnd != BSQ_SR) return BSQ_EINVAL;
  if (block_rows == 16 && rows % 16 != 0) return BSQ_EINVAL;
  if (amax_in == nullptr && amax_out == nullptr) return BSQ_EINVAL;
  if (!aligned4(amax_in) || !aligned4(amax_out)) return BSQ_EINVAL;
  if (block_rows == 16 && (rnd == BSQ_SR || rht)) return BSQ_EUNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t n = rows * cols;
  if (n == 0) {
    if (amax_out) return hip_status(bsq::launch_zero_amax(amax_out, nullptr, s));
    return BSQ_OK;
  }
  if (!x || !codes || !scales) return BSQ_EINVAL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return BSQ_EINVAL;

  const float* amax = amax_in;
  hipError_t e;
  if (amax_in == nullptr) {
    e = bsq::launch_zero_amax(amax_out, nullptr, s);
    if (e != hipSuccess) return BSQ_EHIP;
    e = bsq::launch_amax_flat(x, n / 8, rht != 0, rht_signs, amax_out, nullptr, s);
    if (e != hipSuccess) return BSQ_EHIP;
    amax = amax_out;
  } else if (amax_out != nullptr && amax_out != amax_in) {
    e = bsq::launch_copy_amax(amax_in, amax_out, s);
    if (e != hipSuccess) return BSQ_EHIP;
  }
  if (block_rows == 1)
    e = bsq::launch_quant_flat(bsq::kNVFP4, rnd == BSQ_SR, rht != 0, x, n / 8, amax, rht_signs,
                               seed, offset, codes, scales, s);
  else
    e = bsq::launch_quant_tile(bsq::kNVFP4, false, false, true, x, rows, cols, true, false, amax,
                               amax, 0, seed, offset, codes, scales, nullptr, nullptr, s);
  return hip_status(e);
}

bsq_status mx_quantize(const void* x, int64_t rows, int64_t cols, bsq_format fmt,
                       bsq_rounding rnd, uint64_t seed, uint32_t offset, uint8_t* codes,
                       uint8_t* scales, void* stream) {
  if (rows < 0 || cols < 0 || cols % 32 != 0 || too_many(rows, cols)) return BSQ_EINVAL;
  if (fmt != BSQ_MXFP4 && fmt != BSQ_MXFP8)
    return fmt == BSQ_NVFP4 || fmt == BSQ_FP8 ? BSQ_EUNSUPPORTED : BSQ_EINVAL;
  if (rnd != BSQ_RNE && rnd != BSQ_SR) return BSQ_EINVAL;
  if (fmt == BSQ_MXFP8 && rnd == BSQ_SR) return BSQ_EUNSUPPORTED;
  const int64_t n = rows * cols;
  if (n == 0) return BSQ_OK;
  if (!x || !codes || !scales) return BSQ_EINVAL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return BSQ_EINVAL;
  return hip_status(bsq::launch_quant_flat(fmt == BSQ_MXFP4 ? bsq::kMXFP4 : bsq::kMXFP8,
                                           rnd == BSQ_SR, false, x, n / 8, nullptr, 0, seed,
                                           offset, codes, scales,
                                           static_cast<hipStream_t>(stream)));
}

bsq_status quantize_transpose(const void* x, int64_t rows, int64_t cols, bsq_format fmt,
                              int block_rows, bsq_rounding rnd, uint64_t seed, uint32_t offset,
                              int rht_col, uint16_t rht_signs, uint8_t* codes_row,
                              uint8_t* scales_row, float* amax_row, uint8_t* codes_col,
                              uint8_t* scales_col, float* amax_col, void* stream) {
  if (fmt == BSQ_FP8) return BSQ_EUNSUPPORTED;      // fp8_quantize_transpose
  if (fmt != BSQ_NVFP4 && fmt != BSQ_MXFP4 && fmt != BSQ_MXFP8) return BSQ_EINVAL;
  const bool nv = fmt == BSQ_NVFP4;
  const int blk = nv ? 16 : 32;
  if (rows < 0 || cols < 0 || rows % blk != 0 || cols % blk != 0) return BSQ_EINVAL;
  if (too_many(rows, cols)) return BSQ_EINVAL;
  if (block_rows != 1 && block_rows != 16) return BSQ_EINVAL;
  if (rnd != BSQ_RNE && rnd != BSQ_SR) return BSQ_EINVAL;
  const bool do_row = codes_row || scales_row || (nv && amax_row);
  const bool do_col = codes_col || scales_col || (nv && amax_col);
  if (!do_row && !do_col && rows * cols != 0) return BSQ_EINVAL;   // empty tensors have null pointers
  if (!nv && (block_rows == 16 || rht_col)) return BSQ_EUNSUPPORTED;
  if (fmt == BSQ_MXFP8 && rnd == BSQ_SR) return BSQ_EUNSUPPORTED;
  if (block_rows == 16 && (rnd == BSQ_SR || rht_col)) return BSQ_EUNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows * cols == 0) {                      // empty tensor: only the amax outputs are defined
    if (nv && (!aligned4(amax_row) || !aligned4(amax_col))) return BSQ_EINVAL;
    if (nv && (amax_row || amax_col)) return hip_status(bsq::launch_zero_amax(amax_row, amax_col, s));
    return BSQ_OK;
  }
  if (do_row && (!codes_row || !scales_row || (nv && !amax_row))) return BSQ_EINVAL;
  if (do_col && (!codes_col || !scales_col || (nv && !amax_col))) return BSQ_EINVAL;
  if (!aligned16_or_null(codes_row) || !aligned16_or_null(scales_row) ||
      !aligned16_or_null(codes_col) || !aligned16_or_null(scales_col))
    return BSQ_EINVAL;
  if (nv && (!aligned4(amax_row) || !aligned4(amax_col))) return BSQ_EINVAL;
  float* ar = do_row ? amax_row : nullptr;
  float* ac = do_col ? amax_col : nullptr;
  if (!x || !aligned16(x)) return BSQ_EINVAL;
  // the column RHT amax pass addresses 16 rows (32 * cols bytes) per buffer resource
  if (nv && rht_col && do_col && cols >= ((int64_t)1 << 26)) return BSQ_EINVAL;

  hipError_t e;
  if (nv) {
    e = bsq::launch_zero_amax(ar, ac, s);
    if (e != hipSuccess) return BSQ_EHIP;
    if (rht_col && do_col)
      e = bsq::launch_amax_tile_rht(x, rows, cols, rht_signs, ar, ac, s);
    else
      e = bsq::launch_amax_flat(x, rows * cols / 8, false, 0, ar ? ar : ac, ar ? ac : nullptr, s);
    if (e != hipSuccess) return BSQ_EHIP;
  }
  const bsq::Fmt f = nv ? bsq::kNVFP4 : (fmt == BSQ_MXFP4 ? bsq::kMXFP4 : bsq::kMXFP8);
  e = bsq::launch_quant_tile(f, rnd == BSQ_SR, rht_col != 0 && do_col, block_rows == 16, x, rows,
                             cols, do_row, do_col, ar, ac, rht_signs, seed, offset, codes_row,
                             scales_row, codes_col, scales_col, s);
  return hip_status(e);
}

bsq_status fp8_quantize_transpose(const void* x, int64_t rows, int64_t cols, uint8_t* codes_row,
                                  uint8_t* codes_col, float* amax, void* stream) {
  if (rows < 0 || cols < 0 || rows % 16 != 0 || cols % 16 != 0) return BSQ_EINVAL;
  if (too_many(rows, cols)) return BSQ_EINVAL;
  if (!amax || !aligned4(amax)) return BSQ_EINVAL;
  if (!codes_row && !codes_col && rows * cols != 0) return BSQ_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows * cols == 0) return hip_status(bsq::launch_zero_amax(amax, nullptr, s));
  if (!x || !aligned16(x) || !aligned16_or_null(codes_row) || !aligned16_or_null(codes_col))
    return BSQ_EINVAL;
  hipError_t e = bsq::launch_zero_amax(amax, nullptr, s);
  if (e != hipSuccess) return BSQ_EHIP;
  e = bsq::launch_amax_flat(x, rows * cols / 8, false, 0, amax, nullptr, s);
  if (e != hipSuccess) return BSQ_EHIP;
  return hip_status(bsq::launch_fp8_qt(x, rows, cols, amax, codes_row, codes_col, s));
}

bsq_status quantize_transpose_amax(const void* x, int64_t rows, int64_t cols, int block_rows,
                                   bsq_rounding rnd, uint64_t seed, uint32_t offset, int rht_col,
                                   uint16_t rht_signs, const float* amax_row, const float* amax_col,
                                   uint8_t* codes_row, uint8_t* scales_row, uint8_t* codes_col,
                                   uint8_t* scales_col, void* stream) {
  if (rows < 0 || cols < 0 || rows % 16 != 0 || cols % 16 != 0) return BSQ_EINVAL;
  if (too_many(rows, cols)) return BSQ_EINVAL;
  if (block_rows != 1 && block_rows != 16) return BSQ_EINVAL;
  if (rnd != BSQ_RNE && rnd != BSQ_SR) return BSQ_EINVAL;
  const bool do_row = codes_row || scales_row;
  const bool do_col = codes_col || scales_col;
  if (!do_row && !do_col && rows * cols != 0) return BSQ_EINVAL;   // empty tensors have null pointers
  if (block_rows == 16 && (rnd == BSQ_SR || rht_col)) return BSQ_EUNSUPPORTED;
  // 16x16 tiles encode both orientations under one amax (the codes of x^T
  // are the codes of x transposed), so the caller must pass that one amax
  // for both sides
  if (block_rows == 16 && do_row && do_col && amax_row != amax_col) return BSQ_EINVAL;
  if (rows * cols == 0) return BSQ_OK;
  if (do_row && (!codes_row || !scales_row || !amax_row)) return BSQ_EINVAL;
  if (do_col && (!codes_col || !scales_col || !amax_col)) return BSQ_EINVAL;
  if (!aligned16_or_null(codes_row) || !aligned16_or_null(scales_row) ||
      !aligned16_or_null(codes_col) || !aligned16_or_null(scales_col))
    return BSQ_EINVAL;
  if (!aligned4(amax_row) || !aligned4(amax_col)) return BSQ_EINVAL;
  if (!x || !aligned16(x)) return BSQ_EINVAL;
  return hip_status(bsq::launch_quant_tile(
      bsq::kNVFP4, rnd == BSQ_SR, rht_col != 0 && do_col, block_rows == 16, x, rows, cols, do_row,
      do_col, do_row ? amax_row : nullptr, do_col ? amax_col : nullptr, rht_signs, seed, offset,
      codes_row, scales_row, codes_col, scales_col, static_cast<hipStream_t>(stream)));
}

bsq_status swiglu_amax(const void* y_gu, int64_t rows, int64_t f, int rht_col, uint16_t rht_signs,
                       void* h, float* amax_row, float* amax_col, void* stream) {
  return swiglu_common(y_gu, nullptr, rows, f, rht_col, rht_signs, h, amax_row, amax_col, stream);
}

bsq_status swiglu_backward_amax(const void* y_gu, const void* d_h, int64_t rows, int64_t f,
                                int rht_col, uint16_t rht_signs, void* d_y_gu, float* amax_row,
                                float* amax_col, void* stream) {
  if (rows * f != 0 && !d_h) return BSQ_EINVAL;
  return swiglu_common(y_gu, d_h, rows, f, rht_col, rht_signs, d_y_gu, amax_row, amax_col, stream);
}

bsq_status master_weight_update(float* w32, const void* grad, int64_t n, float lr, void* w_bf16,
                                float* amax, void* stream) {
  if (n < 0 || n % 8 != 0 || too_many(1, n) || !aligned4(amax)) return BSQ_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (n == 0) return amax ? hip_status(bsq::launch_zero_amax(amax, nullptr, s)) : BSQ_OK;
  if (!w32 || !grad || !w_bf16 || !aligned16(w32) || !aligned16(grad) || !aligned16(w_bf16))
    return BSQ_EINVAL;
  if (overlap(w32, n * 4, grad, n * 2) || overlap(w32, n * 4, w_bf16, n * 2) ||
      overlap(grad, n * 2, w_bf16, n * 2))
    return BSQ_EINVAL;
  if (amax) {
    const hipError_t e = bsq::launch_zero_amax(amax, nullptr, s);
    if (e != hipSuccess) return BSQ_EHIP;
  }
  return hip_status(bsq::launch_master_update(w32, grad, n, lr, w_bf16, amax, s));
}

bsq_status nvfp4_expand(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                        void* out, void* stream) {
  if (rows < 0 || cols < 0 || cols % 16 != 0 || too_many(rows, cols)) return BSQ_EINVAL;
  if (rows * cols == 0) return BSQ_OK;
  if (!codes || !scales || !out || !aligned16(out) || (reinterpret_cast<uintptr_t>(codes) & 7u) != 0)
    return BSQ_EINVAL;
  return hip_status(bsq::launch_nvfp4_expand(codes, scales, rows, cols, out,
                                             static_cast<hipStream_t>(stream)));
}

bsq_status bs_gemm_nvfp4_bx(int64_t M, int64_t N, int64_t K, const uint8_t* a_codes,
                            const uint8_t* a_scales, const float* a_amax, const void* b_x,
                            const float* b_amax, void* c, int64_t ldc, void* stream) {
  if (M < 0 || N < 0 || K < 0 || ldc < N) return BSQ_EINVAL;
  if (too_many(M, K) || too_many(N, K) || too_many(M, ldc)) return BSQ_EINVAL;
  if (M > (int64_t)256 * 0x7FFFFF || N > (int64_t)256 * 0x7FFFFF) return BSQ_EINVAL;
  if (M == 0 || N == 0) return BSQ_OK;
  if (!a_codes || !a_scales || !b_x || !a_amax || !b_amax || !c) return BSQ_EINVAL;
  if ((reinterpret_cast<uintptr_t>(c) & 1u) != 0 || !aligned4(a_amax) || !aligned4(b_amax))
    return BSQ_EINVAL;
  if (K == 0 || K % 128 != 0 || !aligned16(a_codes) || !aligned4(a_scales) || !aligned16(b_x) ||
      M * (K / 2) >= ((int64_t)1 << 32) || N * K * 2 >= ((int64_t)1 << 32))
    return BSQ_EUNSUPPORTED;
  return hip_status(bsq::launch_gemm_nvfp4_bx(M, N, K, a_codes, a_scales, a_amax, b_x, b_amax, c,
                                              ldc, static_cast<hipStream_t>(stream)));
}

bsq_status bs_gemm(bsq_format fmt, int64_t M, int64_t N, int64_t K, const uint8_t* a_codes,
                   const uint8_t* a_scales, const float* a_amax, const uint8_t* b_codes,
                   const uint8_t* b_scales, const float* b_amax, void* c, int64_t ldc,
                   void* stream) {
  return gemm_common(fmt, M, N, K, a_codes, a_scales, a_amax, b_codes, b_scales, b_amax, c, ldc,
                     stream, false);
}

bsq_status bs_gemm_noalloc(bsq_format fmt, int64_t M, int64_t N, int64_t K,
                           const uint8_t* a_codes, const uint8_t* a_scales, const float* a_amax,
                           const uint8_t* b_codes, const uint8_t* b_scales, const float* b_amax,
                           void* c, int64_t ldc, void* stream) {
  return gemm_common(fmt, M, N, K, a_codes, a_scales, a_amax, b_codes, b_scales, b_amax, c, ldc,
                     stream, true);
}

bsq_status block_norm(const void* x, bsq_dtype x_type, const void* o, int64_t rows, int64_t cols,
                      const float* w_post, bsq_gate gate_kind, const void* gate, float alpha,
                      const float* w_pre, float eps, void* r, void* h, float* rstd_post,
                      float* rstd_pre, float* amax, void* stream) {
  const bsq_status st = norm_checks(rows, cols, x_type, o, w_post, gate_kind, gate, w_pre);
  if (st != BSQ_OK) return st;
  const bool f32 = x_type == BSQ_F32;
  if (!(eps > 0.0f)) return BSQ_EINVAL;
  if (rows == 0 && amax)
    return aligned4(amax) ? hip_status(bsq::launch_zero_amax(amax, nullptr, static_cast<hipStream_t>(stream)))
                          : BSQ_EINVAL;
  if (rows == 0) return BSQ_OK;
  if ((o != nullptr) != (r != nullptr) || (w_pre != nullptr) != (h != nullptr)) return BSQ_EINVAL;
  if ((rstd_post && !w_post) || (!w_pre && (rstd_pre || amax))) return BSQ_EINVAL;
  if (!aligned_elem(x, f32) || !aligned_elem(r, f32) || !aligned2(h) || !aligned4(rstd_post) ||
      !aligned4(rstd_pre) || !aligned4(amax))
    return BSQ_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!x) return BSQ_EINVAL;
  const int64_t n = rows * cols, xb = n * (f32 ? 4 : 2), gb = gate_kind == BSQ_GATE_FULL ? n * 2 : 0;
  const void* outs[2] = {r, h};
  const int64_t outb[2] = {r ? xb : 0, h ? n * 2 : 0};
  for (int i = 0; i < 2; ++i) {
    if (!outs[i]) continue;
    if (overlap(outs[i], outb[i], x, xb) || (o && overlap(outs[i], outb[i], o, n * 2)) ||
        (gb && overlap(outs[i], outb[i], gate, gb)))
      return BSQ_EINVAL;
  }
  if (r && h && overlap(r, outb[0], h, outb[1])) return BSQ_EINVAL;
  const bsq::NormFwd a{x,     o,   rows, cols, w_post,    (int)gate_kind, gate, alpha,
                       w_pre, eps, r,    h,    rstd_post, rstd_pre,       amax, f32};
  return hip_status(bsq::launch_block_norm(a, s));
}

bsq_status block_norm_backward_workspace(int64_t rows, int64_t cols, int64_t* bytes) {
  if (rows < 0 || cols < 1 || too_many(rows, cols) || !bytes) return BSQ_EINVAL;
  if (cols > 16384) return BSQ_EUNSUPPORTED;
  *bytes = bsq::block_norm_bwd_part_bytes(rows, cols);
  return BSQ_OK;
}

bsq_status block_norm_backward(const void* r, bsq_dtype r_type, const void* o, const void* d_r,
                               const void* d_h, int64_t rows, int64_t cols, const float* w_post,
                               bsq_gate gate_kind, const void* gate, float alpha, const float* w_pre,
                               const float* rstd_post, const float* rstd_pre, void* d_x, void* d_o,
                               void* d_gate, float* d_w_pre, float* d_w_post, void* workspace,
                               int64_t workspace_bytes, void* stream) {
  const bsq_status st = norm_checks(rows, cols, r_type, o, w_post, gate_kind, gate, w_pre);
  if (st != BSQ_OK) return st;
  const bool f32 = r_type == BSQ_F32;
  if ((w_pre != nullptr) != (d_w_pre != nullptr) || (w_post != nullptr) != (d_w_post != nullptr) ||
      ((rows > 0 || gate_kind == BSQ_GATE_CHANNEL) && (gate != nullptr) != (d_gate != nullptr)))
    return BSQ_EINVAL;
  if (!aligned_elem(r, f32) || !aligned_elem(d_r, f32) || !aligned_elem(d_x, f32) || !aligned2(d_h) ||
      !aligned2(d_o) || !aligned4(rstd_post) || !aligned4(rstd_pre) || !aligned4(d_w_pre) ||
      !aligned4(d_w_post) || !aligned_elem(d_gate, gate_kind != BSQ_GATE_FULL))
    return BSQ_EINVAL;
  if (rows > 0) {
    if (!d_x || (o != nullptr) != (d_o != nullptr)) return BSQ_EINVAL;
    if ((w_pre != nullptr) != (d_h != nullptr) || (w_pre && (!rstd_pre || !r)) || (w_post && !rstd_post))
      return BSQ_EINVAL;
    if (!w_pre && !d_r) return BSQ_EINVAL;                 // no incoming gradient
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < bsq::block_norm_bwd_part_bytes(rows, cols))
      return BSQ_EINVAL;
    const int64_t n = rows * cols, xb = n * (f32 ? 4 : 2);
    const bool full = gate_kind == BSQ_GATE_FULL;
    const void* outs[3] = {d_x, d_o, full ? d_gate : nullptr};
    const int64_t outb[3] = {xb, n * 2, n * 2};
    const void* ins[5] = {r, o, d_r, d_h, full ? gate : nullptr};
    const int64_t inb[5] = {xb, n * 2, xb, n * 2, n * 2};
    for (int i = 0; i < 3; ++i) {
      if (!outs[i]) continue;
      for (int j = 0; j < 5; ++j)
        if (ins[j] && overlap(outs[i], outb[i], ins[j], inb[j])) return BSQ_EINVAL;
      for (int j = 0; j < i; ++j)
        if (outs[j] && overlap(outs[i], outb[i], outs[j], outb[j])) return BSQ_EINVAL;
    }
  }
  const bsq::NormBwd a{r,     o,         d_r,      d_h, rows, cols,   w_post,  (int)gate_kind, gate,
                       alpha, w_pre,     rstd_post, rstd_pre, d_x, d_o, d_gate, d_w_pre, d_w_post,
                       static_cast<float*>(workspace), f32};
  return hip_status(bsq::launch_block_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

bsq_status moe_rows(int64_t tokens, int experts, int k, int align, int64_t* rows) {
  if (!rows) return BSQ_EINVAL;
  return moe_rows_of(tokens, experts, k, align, rows);
}

bsq_status moe_route_workspace(int64_t tokens, int experts, int k, int64_t* bytes) {
  if (!bytes) return BSQ_EINVAL;
  const bsq_status st = route_checks(tokens, experts, k);
  if (st != BSQ_OK) return st;
  *bytes = bsq::moe_route_hist_bytes(tokens, experts);
  return BSQ_OK;
}

bsq_status moe_route(const void* logits, bsq_dtype type, int64_t tokens, int experts, int k,
                     const float* bias, bsq_scoring scoring, int normalize, float scale, int align,
                     int64_t rows, int32_t* experts_out, float* weights, int32_t* offsets,
                     int32_t* row_of, int32_t* src, void* workspace, int64_t workspace_bytes,
                     void* stream) {
  return route_common(logits, type, tokens, experts, k, bias, false, scoring, normalize, scale, align, rows,
                      experts_out, weights, offsets, row_of, src, workspace, workspace_bytes, stream);
}

bsq_status moe_route_score_bias(const void* logits, bsq_dtype type, int64_t tokens, int experts, int k,
                                const float* score_bias, bsq_scoring scoring, int normalize, float scale,
                                int align, int64_t rows, int32_t* experts_out, float* weights,
                                int32_t* offsets, int32_t* row_of, int32_t* src, void* workspace,
                                int64_t workspace_bytes, void* stream) {
  return route_common(logits, type, tokens, experts, k, score_bias, true, scoring, normalize, scale, align, rows,
                      experts_out, weights, offsets, row_of, src, workspace, workspace_bytes, stream);
}

bsq_status moe_route_backward(const void* logits, bsq_dtype type, int64_t tokens, int experts, int k,
                              const int32_t* experts_in, const float* d_weights, bsq_scoring scoring,
                              int normalize, float scale, void* d_logits, void* stream) {
  const bsq_status st = route_checks(tokens, experts, k);
  if (st != BSQ_OK) return st;
  if (!valid_dtype(type) || (scoring != BSQ_SOFTMAX && scoring != BSQ_SIGMOID)) return BSQ_EINVAL;
  if (tokens == 0) return BSQ_OK;
  const bool f32 = type == BSQ_F32;
  if (!logits || !experts_in || !d_weights || !d_logits || !aligned_elem(logits, f32) ||
      !aligned_elem(d_logits, f32) || !aligned4(experts_in) || !aligned4(d_weights))
    return BSQ_EINVAL;
  const int64_t lb = tokens * experts * (f32 ? 4 : 2);
  if (overlap(d_logits, lb, logits, lb)) return BSQ_EINVAL;
  return hip_status(bsq::launch_moe_route_bwd(logits, f32, tokens, experts, k, experts_in, d_weights,
                                              scoring == BSQ_SIGMOID, normalize != 0, scale, d_logits,
                                              static_cast<hipStream_t>(stream)));
}

bsq_status moe_gather(const void* x, int64_t tokens, int64_t cols, int k, const int32_t* src,
                      int64_t rows, void* out, void* stream) {
  const bsq_status st = mover_checks(tokens, cols, k, rows);
  if (st != BSQ_OK) return st;
  if (rows * cols == 0) return BSQ_OK;
  if ((tokens > 0 && !x) || !src || !out || !aligned2(x) || !aligned4(src) || !aligned2(out))
    return BSQ_EINVAL;
  if (overlap(out, rows * cols * 2, x, tokens * cols * 2)) return BSQ_EINVAL;
  return hip_status(bsq::launch_moe_gather(x, tokens, cols, k, src, rows, out, static_cast<hipStream_t>(stream)));
}

bsq_status moe_combine(const void* y, int64_t rows, int64_t cols, const int32_t* row_of,
                       const float* weights, int64_t tokens, int k, void* out, void* stream) {
  const bsq_status st = mover_checks(tokens, cols, k, rows);
  if (st != BSQ_OK) return st;
  if (tokens * cols == 0) return BSQ_OK;
  if ((rows > 0 && !y) || !row_of || !out || !aligned2(y) || !aligned4(row_of) || !aligned4(weights) ||
      !aligned2(out))
    return BSQ_EINVAL;
  if (overlap(out, tokens * cols * 2, y, rows * cols * 2)) return BSQ_EINVAL;
  return hip_status(bsq::launch_moe_combine(y, rows, cols, row_of, weights, tokens, k, out,
                                            static_cast<hipStream_t>(stream)));
}

bsq_status moe_combine_backward(const void* d_out, const void* y, int64_t tokens, int64_t cols, int k,
                                const int32_t* src, const int32_t* row_of, const float* weights,
                                int64_t rows, void* d_y, float* d_weights, void* stream) {
  const bsq_status st = mover_checks(tokens, cols, k, rows);
  if (st != BSQ_OK) return st;
  if (tokens == 0 && rows * cols == 0) return BSQ_OK;
  if (tokens > 0 && (!row_of || !weights || !d_weights)) return BSQ_EINVAL;
  if (tokens * cols > 0 && !d_out) return BSQ_EINVAL;
  if (rows > 0 && !src) return BSQ_EINVAL;
  if (rows * cols > 0 && (!y || !d_y)) return BSQ_EINVAL;
  if (!aligned2(d_out) || !aligned2(y) || !aligned2(d_y) || !aligned4(src) || !aligned4(row_of) ||
      !aligned4(weights) || !aligned4(d_weights))
    return BSQ_EINVAL;
  if (rows * cols > 0 &&
      (overlap(d_y, rows * cols * 2, y, rows * cols * 2) || overlap(d_y, rows * cols * 2, d_out, tokens * cols * 2)))
    return BSQ_EINVAL;
  return hip_status(bsq::launch_moe_combine_bwd(d_out, y, tokens, cols, k, src, row_of, weights, rows, d_y,
                                                d_weights, static_cast<hipStream_t>(stream)));
}

bsq_status bs_gemm_grouped(bsq_format fmt, int experts, const int32_t* offsets, int64_t rows, int64_t N,
                           int64_t K, const uint8_t* a_codes, const uint8_t* a_scales,
                           const float* a_amax, const uint8_t* b_codes, const uint8_t* b_scales,
                           const float* b_amax, int b_amax_n, void* c, int64_t ldc, void* stream) {
  bsq::Fmt f;
  const bsq_status st = grouped_format(fmt, &f);
  if (st != BSQ_OK) return st;
  if (experts < 1 || experts > 4096 || rows < 0 || rows > 0x7FFFFFFF || N < 0 || K < 0) return BSQ_EINVAL;
  if (N > 0x7FFFFFFF) return BSQ_EINVAL;
  if (K % (fmt == BSQ_NVFP4 ? 16 : 32) != 0 || ldc < N) return BSQ_EINVAL;
  if (too_many(rows, K) || too_many(N, K) || too_many(rows, ldc) || too_many(experts, N * K)) return BSQ_EINVAL;
  if (rows == 0 || N == 0) return BSQ_OK;
  if (!offsets || !aligned4(offsets) || !c || !aligned2(c)) return BSQ_EINVAL;
  if (K > 0 && (!a_codes || !a_scales || !b_codes || !b_scales || !aligned16(a_codes) || !aligned16(b_codes)))
    return BSQ_EINVAL;
  if (fmt == BSQ_NVFP4 && (!a_amax || !b_amax || !aligned4(a_amax) || !aligned4(b_amax) ||
                           (b_amax_n != 1 && b_amax_n != experts)))
    return BSQ_EINVAL;
  const bsq::GroupedArgs a{f, experts, offsets, rows, N, K, a_codes, a_scales, a_amax,
                           b_codes, b_scales, b_amax, b_amax_n, c, ldc};
  return hip_status(bsq::launch_gemm_grouped(a, static_cast<hipStream_t>(stream)));
}

bsq_status bs_gemm_grouped_wgrad(bsq_format fmt, int experts, const int32_t* offsets, int64_t M, int64_t N,
                                 int64_t rows, const uint8_t* a_codes, const uint8_t* a_scales,
                                 const float* a_amax, const uint8_t* b_codes, const uint8_t* b_scales,
                                 const float* b_amax, void* c, void* stream) {
  bsq::Fmt f;
  const bsq_status st = grouped_format(fmt, &f);
  if (st != BSQ_OK) return st;
  if (experts < 1 || experts > 4096 || rows < 0 || rows > 0x7FFFFFFF || M < 0 || N < 0) return BSQ_EINVAL;
  if (M > 0x7FFFFFFF || N > 0x7FFFFFFF) return BSQ_EINVAL;
  if (rows % (fmt == BSQ_NVFP4 ? 16 : 32) != 0) return BSQ_EINVAL;
  if (too_many(M, rows) || too_many(N, rows) || too_many(M, N) || too_many(experts, M * N)) return BSQ_EINVAL;
  if (M == 0 || N == 0) return BSQ_OK;
  if (!offsets || !aligned4(offsets) || !c || !aligned2(c)) return BSQ_EINVAL;
  if (rows > 0 && (!a_codes || !a_scales || !b_codes || !b_scales || !aligned16(a_codes) || !aligned16(b_codes)))
    return BSQ_EINVAL;
  if (fmt == BSQ_NVFP4 && (!a_amax || !b_amax || !aligned4(a_amax) || !aligned4(b_amax))) return BSQ_EINVAL;
  const bsq::GroupedArgs a{f, experts, offsets, M, N, rows, a_codes, a_scales, a_amax,
                           b_codes, b_scales, b_amax, 1, c, N};
  return hip_status(bsq::launch_gemm_grouped_wgrad(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
