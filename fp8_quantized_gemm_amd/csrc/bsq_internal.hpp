// Internal launch interface between the C-ABI layer and the HIP kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bsq {

enum Fmt { kNVFP4 = 0, kMXFP4 = 1, kMXFP8 = 2, kFP8 = 3 };   // kFP8: per-tensor E4M3

// One-byte (E4M3) elements: MXFP8 and per-tensor FP8.
constexpr bool fp8_elems(int f) { return f == kMXFP8 || f == kFP8; }

// Raises the dynamic-LDS limit of kernel `fn` to `bytes` on the current
// device, once per (device, kernel): later calls return the first call's
// result.  Thread-safe (several host threads may launch at once).
hipError_t set_lds_limit(const void* fn, int bytes);

// Sets *a = 0 and *b = 0 (either may be null).
hipError_t launch_zero_amax(float* a, float* b, hipStream_t s);
// *dst = *src.
hipError_t launch_copy_amax(const float* src, float* dst, hipStream_t s);

// amax over a contiguous BF16 tensor of nchunk 8-element chunks; with rht the
// amax is over the 16-point RHT of each aligned 16-chunk.  Atomically maxes
// into a0 and (if non-null) a1, which must have been zeroed.
hipError_t launch_amax_flat(const void* x, int64_t nchunk, bool rht, uint32_t signs,
                            float* a0, float* a1, hipStream_t s);

// amax of x (into amax_row, may be null) and of the RHT of x^T along rows
// (into amax_col) for x [R, C].
hipError_t launch_amax_tile_rht(const void* x, int64_t R, int64_t C, uint32_t signs,
                                float* amax_row, float* amax_col, hipStream_t s);

// SwiGLU of Y = [G | U] [R, 2F] (R % 16 == 0, F % 4 == 0): with dh null, the
// forward H = silu(G) * U into out [R, F]; else the backward [dG | dU] of dh
// [R, F] into out [R, 2F].  amax_mode 0: no amax; 1: max |out| into both amax
// outputs (either may be null); 2: max |out| into amax_row and the column RHT
// amax (16-row chunks) into amax_col.  Amax outputs must have been zeroed.
hipError_t launch_swiglu(const void* y, const void* dh, int64_t R, int64_t F, int amax_mode,
                         uint32_t signs, void* out, float* amax_row, float* amax_col, hipStream_t s);

// FP32 master-weight update of n elements (n % 8 == 0): w <- w - lr * g
// (BF16 g), wb = BF16 RNE of the new w, and max |wb| into amax (zeroed
// before; may be null).
hipError_t launch_master_update(float* w, const void* g, int64_t n, float lr, void* wb, float* amax,
                                hipStream_t s);

// Rowwise quantization over a contiguous tensor of nchunk 8-element chunks
// (NVFP4 1x16 or MX 1x32 blocks; rows are implied since cols % block == 0).
hipError_t launch_quant_flat(Fmt fmt, bool sr, bool rht, const void* x, int64_t nchunk,
                             const float* amax, uint32_t signs, uint64_t seed, uint32_t offset,
                             uint8_t* codes, uint8_t* scales, hipStream_t s);

// Row and/or column quantization of x [R, C] from one read.
hipError_t launch_quant_tile(Fmt fmt, bool sr, bool rht_col, bool two_d, const void* x,
                             int64_t R, int64_t C, bool do_row, bool do_col,
                             const float* amax_row, const float* amax_col, uint32_t signs,
                             uint64_t seed, uint32_t offset, uint8_t* codes_row,
                             uint8_t* scales_row, uint8_t* codes_col, uint8_t* scales_col,
                             hipStream_t s);

// Per-tensor FP8 codes of x [R, C] (codes_row [R, C]) and of x^T (codes_col
// [C, R]), either may be null, under the already reduced *amax.
hipError_t launch_fp8_qt(const void* x, int64_t R, int64_t C, const float* amax,
                         uint8_t* codes_row, uint8_t* codes_col, hipStream_t s);

// Number of compute units of the current device (cached per device).
int device_cus();

// NVFP4 GEMM (exact FP16 dequant + FP16 MFMA).  scratch: null = workspace of
// the split last wave (see gemm_nvfp4_rx_split) from the stream-ordered
// allocator; otherwise a device buffer of scratch_bytes used for it
// (hipErrorInvalidValue when too small).
hipError_t launch_gemm_nvfp4(int64_t M, int64_t N, int64_t K, const uint8_t* ac, const uint8_t* as,
                             const float* aa, const uint8_t* bc, const uint8_t* bs,
                             const float* ba, void* c, int64_t ldc, void* scratch,
                             size_t scratch_bytes, hipStream_t s);
// The library's static workspace for the NVFP4 GEMM on the current device
// (address looked up once per device) and its size.
hipError_t gemm_nvfp4_static_scratch(void** ptr, size_t* bytes);
// Workspace bytes the NVFP4 GEMM of these operands needs on the current device.
size_t gemm_nvfp4_scratch_bytes(int64_t M, int64_t N, int64_t K, const uint8_t* ac,
                                const uint8_t* as, const uint8_t* bc, const uint8_t* bs);

// The register-expansion NVFP4 GEMM (four waves, codes expanded in registers):
// whether it takes these operands (K % 256 == 0, codes 16-byte and scales
// 4-byte aligned, each operand below 4 GiB), and its launch.
bool gemm_nvfp4_rx_fits(int64_t M, int64_t N, int64_t K, const uint8_t* ac, const uint8_t* as,
                        const uint8_t* bc, const uint8_t* bs);
// Split last wave: when the tiles fill at least one wave of `cus` workgroups
// and leave a last wave of at most cus / 2 tiles (K % 512 == 0, K >= 4096),
// the number of those tiles; each runs as two workgroups over the two K
// halves, which write FP32 partials (kRxSplitTileBytes per tile) that a
// second kernel adds, scales and rounds.  0 = no split.
int gemm_nvfp4_rx_split(int64_t M, int64_t N, int64_t K, int cus);
constexpr size_t kRxSplitTileBytes = (size_t)2 * 256 * 256 * 4;
// tail: gemm_nvfp4_rx_split's count (or 0); part: tail * kRxSplitTileBytes
// bytes of device memory when tail > 0.
hipError_t launch_gemm_nvfp4_rx(int64_t M, int64_t N, int64_t K, const uint8_t* ac,
                                const uint8_t* as, const float* aa, const uint8_t* bc,
                                const uint8_t* bs, const float* ba, void* c, int64_t ldc,
                                int tail, void* part, hipStream_t s);

// NVFP4 GEMM with B pre-expanded to FP16 (bx [N, K] = v * S * 2^-7, from
// launch_nvfp4_expand).  hipErrorNotSupported unless K % 128 == 0, the
// operands are 16-byte aligned (scales 4) and M * K / 2, N * K * 2 < 2^32.
hipError_t launch_gemm_nvfp4_bx(int64_t M, int64_t N, int64_t K, const uint8_t* ac, const uint8_t* as,
                                const float* aa, const void* bx, const float* ba, void* c,
                                int64_t ldc, hipStream_t s);
// FP16 expansion out [R, K] of NVFP4 codes [R, K/2] and scales [R, K/16].
hipError_t launch_nvfp4_expand(const uint8_t* codes, const uint8_t* scales, int64_t R, int64_t K,
                               void* out, hipStream_t s);

// The four-wave MX / per-tensor FP8 GEMM (FMT kMXFP4, kMXFP8, kFP8): whether it
// takes these operands (K % 512 == 0, codes and scales 16-byte aligned, 32-bit
// offsets suffice), and its launch.
template <int FMT>
bool gemm_mx_rx_fits(int64_t M, int64_t N, int64_t K, const uint8_t* ac, const uint8_t* as,
                     const uint8_t* bc, const uint8_t* bs);
template <int FMT>
hipError_t launch_gemm_mx_rx(int64_t M, int64_t N, int64_t K, const uint8_t* ac, const uint8_t* as,
                             const float* aa, const uint8_t* bc, const uint8_t* bs, const float* ba,
                             void* c, int64_t ldc, hipStream_t s);

// C[M, N] = alpha * A . B^T, block-scaled operands, BF16 out.  scratch as
// for launch_gemm_nvfp4 (only NVFP4 uses it).
hipError_t launch_gemm(Fmt fmt, int64_t M, int64_t N, int64_t K, const uint8_t* a_codes,
                       const uint8_t* a_scales, const float* a_amax, const uint8_t* b_codes,
                       const uint8_t* b_scales, const float* b_amax, void* c, int64_t ldc,
                       void* scratch, size_t scratch_bytes, hipStream_t s);

// ---------------------------------------------------------------- block norms

enum GateKind { kGateNone = 0, kGateChannel = 1, kGateRow = 2, kGateFull = 3 };

// block_norm's arguments (include/bsq.h): x, r FP32 when f32, else BF16.
struct NormFwd {
  const void* x;
  const void* o;                  // null: only h = norm(x)
  int64_t rows, cols;
  const float* w_post;            // null: o is not normalised
  int gate_kind;
  const void* gate;
  float alpha;
  const float* w_pre;             // null: no h
  float eps;
  void* r;
  void* h;
  float* rstd_post;
  float* rstd_pre;
  float* amax;
  bool f32;
};
// 1 <= cols <= 16384, rows > 0; any alignment (16-byte pieces where it allows).
hipError_t launch_block_norm(const NormFwd& a, hipStream_t s);

struct NormBwd {
  const void* r;
  const void* o;
  const void* d_r;                // null: zero
  const void* d_h;
  int64_t rows, cols;
  const float* w_post;
  int gate_kind;
  const void* gate;
  float alpha;
  const float* w_pre;
  const float* rstd_post;
  const float* rstd_pre;
  void* d_x;
  void* d_o;
  void* d_gate;
  float* d_w_pre;
  float* d_w_post;
  float* part;                    // block_norm_bwd_part_bytes of device memory
  bool f32;
};
int64_t block_norm_bwd_part_bytes(int64_t rows, int64_t cols);
hipError_t launch_block_norm_bwd(const NormBwd& a, hipStream_t s);

// ---------------------------------------------------------------- expert routing

constexpr int kMoeMaxExperts = 512, kMoeMaxK = 16;

struct RouteArgs {
  const void* logits;             // [tokens, experts], FP32 when f32, else BF16
  bool f32;
  int64_t tokens;
  int experts, k;
  const float* bias;              // null: none
  bool scored;                    // the bias is added to the score, not to the logit
  bool sigmoid, normalize;
  float scale;
  int align;
  int64_t rows;
  int32_t* ids;
  float* weights;
  int32_t* offsets;
  int32_t* row_of;
  int32_t* src;
  int32_t* hist;                  // moe_route_hist_bytes of device memory
};
int64_t moe_route_hist_bytes(int64_t tokens, int experts);
hipError_t launch_moe_route(const RouteArgs& a, hipStream_t s);
hipError_t launch_moe_route_bwd(const void* logits, bool f32, int64_t tokens, int experts, int k,
                                const int32_t* ids, const float* d_w, bool sigmoid, bool normalize,
                                float scale, void* d_logits, hipStream_t s);
hipError_t launch_moe_gather(const void* x, int64_t tokens, int64_t cols, int k, const int32_t* src,
                             int64_t rows, void* out, hipStream_t s);
hipError_t launch_moe_combine(const void* y, int64_t rows, int64_t cols, const int32_t* row_of,
                              const float* w, int64_t tokens, int k, void* out, hipStream_t s);
hipError_t launch_moe_combine_bwd(const void* d_out, const void* y, int64_t tokens, int64_t cols, int k,
                                  const int32_t* src, const int32_t* row_of, const float* w,
                                  int64_t rows, void* d_y, float* d_w, hipStream_t s);

// ---------------------------------------------------------------- expert-grouped GEMM

struct GroupedArgs {
  Fmt fmt;                        // kNVFP4, kMXFP4 or kMXFP8
  int experts;
  const int32_t* offsets;         // [experts + 1], device
  int64_t M, N, K;                // rows: A [M, K], B [experts][N, K]; wgrad: A [M, K], B [N, K], K = rows
  const uint8_t* ac;
  const uint8_t* as;
  const float* aa;
  const uint8_t* bc;
  const uint8_t* bs;
  const float* ba;
  int ba_n;                       // 1 or experts
  void* c;                        // rows: [M, N]; wgrad: [experts][M, N]
  int64_t ldc;
};
// The kernels of the grouped products, by output tile.
enum GroupedKernel {
  kDirect16x64,            // direct loads, K over four waves: any alignment
  kDirect64x64,
  kDirect16x32,            // direct loads, K over eight waves: few tiles and a long K
  kLds16x128,
  kLds32x128,
  kLds64x64,
  kLds64x128,
  kLds128x128,
  k256x256
};
// The kernel the launches below choose for these sizes and alignments, and a launch
// on a given one (hipErrorInvalidValue where it does not take these operands): for
// the tests and measurements of each kernel.
int grouped_kernel(const GroupedArgs& a, bool wgrad);
hipError_t launch_gemm_grouped_on(const GroupedArgs& a, bool wgrad, int kernel, hipStream_t s);
// C rows of group e = alpha A rows . B_e^T; rows of no group are zeroed.
hipError_t launch_gemm_grouped(const GroupedArgs& a, hipStream_t s);
// C_e = alpha A[:, group e] . B[:, group e]^T.
hipError_t launch_gemm_grouped_wgrad(const GroupedArgs& a, hipStream_t s);
// The same products on the 256 x 256 NVFP4 kernel: whether it takes these
// operands (K resp. rows % 256 == 0, codes and scales 16-byte aligned, 32-bit
// offsets), and its launch.
bool gemm_nvfp4_rx_grouped_fits(const GroupedArgs& a, bool wgrad);
hipError_t launch_gemm_nvfp4_rx_grouped(const GroupedArgs& a, bool wgrad, hipStream_t s);
// ... and on the four-wave MX kernel (K resp. rows % 512 == 0, aligned as above).
bool gemm_mx_rx_grouped_fits(const GroupedArgs& a, bool wgrad);
hipError_t launch_gemm_mx_rx_grouped(const GroupedArgs& a, bool wgrad, hipStream_t s);

// ---------------------------------------------------------------- 8-bit integers

// Codes [rows, cols] and decode scales [rows] of the rows of x (BF16).
hipError_t launch_i8_rows(const void* x, int64_t rows, int64_t cols, uint8_t* codes, float* scales, hipStream_t s);
// Row codes [rows, cols] and column codes [cols, rows] (either pair may be null)
// under maxima formed in amax, rows + cols words of device memory.  x 16-byte aligned.
hipError_t launch_i8_qt(const void* x, int64_t rows, int64_t cols, uint8_t* codes_row, float* scales_row,
                        uint8_t* codes_col, float* scales_col, uint32_t* amax, hipStream_t s);

struct Int8Args {
  int64_t M, N, K;                // 0 <= K < 2^17
  const uint8_t* ac;              // [M, K]
  const float* as;                // [M]
  const uint8_t* bc;              // [N, K]
  const float* bs;                // [N]
  const float* bias;              // [N] or null
  void* c;                        // BF16 [M, N]
  int64_t ldc;
};
// The kernels of the plain products (8-bit integers, and the FP16 products of the
// orthogonalisation), by output tile.
enum NtKernel {
  kNtChosen = -1,
  kNtDirect16x64,          // direct loads, K over four waves: any alignment
  kNtDirect64x64,
  kNtRing128,              // LDS ring: rows of whole 16-byte chunks
  kNtRing192,
  kNtRing256,
  kNtRing128x5,
  kNtRing64,
  kNtRing96
};
// kernel: one of the above (hipErrorInvalidValue where it does not take these
// operands), for the tests and measurements of each, or the one that pays.  rest: the tiles
// from number `count` on (at most all) cut for this smaller ring kernel.
hipError_t launch_i8_gemm(const Int8Args& a, hipStream_t s, int kernel = kNtChosen, int rest = kNtChosen, int count = 0);
int i8_kernel(const Int8Args& a);
// x [M, K] (BF16) quantized by rows times a.bc, in one launch: few rows (a.ac, a.as unused).
bool i8_few_rows(const Int8Args& a);
hipError_t launch_i8_linear_few(const void* x, const Int8Args& a, hipStream_t s);

// ---------------------------------------------------------------- orthogonalisation

struct OrthoArgs {
  int64_t batch, rows, cols;      // a stack of matrices, contiguous
  int steps;
  const float* coefs;             // host: 3 per step
  float eps;
  void* workspace;
  // the matrix to orthogonalise: x (BF16, or FP32 when f32), or the moment of an update
  const void* x;
  bool f32;
  void* out;                      // BF16
  // an update (w not null)
  float* w;
  float* momentum;
  const void* grad;               // BF16
  float mu;
  bool nesterov;
  float keep, step;               // w <- keep w - step O
  void* w_bf16;
  float* amax;                    // or null; cleared here
  int kernel = kNtChosen;         // an NtKernel for every product, or the one that pays
  int rest = kNtChosen;           // the second half of its tiles cut for this smaller one
};
int64_t ortho_workspace_bytes(int64_t batch, int64_t rows, int64_t cols);   // -1: too large
hipError_t launch_ortho(const OrthoArgs& a, hipStream_t s);

}  // namespace bsq
