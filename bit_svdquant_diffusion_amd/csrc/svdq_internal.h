// Internal launch interface between the C-ABI glue and the kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "svdq.h"

namespace svdq {

struct Stage1Args {
  int fmt, M, K, r32;   // K: padded to whole 256-channel steps
  int xk;               // the layer's K: X's row stride, and its channels (the rest read as zero)
  const uint16_t* x;    // bf16 [M][xk]
  const float* mu;      // [K]
  const uint16_t* l1s;  // L1 in stage-1 MFMA order
  // activation codes, scales and Z = X_hat L1 over round32(M) rows: codes
  // and Z in fragment order (the layouts of the weight's qw and l2); scales
  // fp32 [K/64][round16(M)] (INT4) or E8M0 bytes in fragment order (MXFP4)
  uint8_t* qx;
  void* sx;
  uint16_t* z;
  uint32_t* flags;   // INT4 GEMM split ticket counters to clear (nflags of them), or null
  int nflags;
  float* zp;         // partial Z per token group and K piece (see ws_layout)
};
// stage 1; with few token groups its K pieces are dealt over the CUs and a
// second kernel adds the partial Z (num_cus sizes that grid)
hipError_t launch_stage1(const Stage1Args& a, int num_cus, hipStream_t st);
hipError_t prepare_stage1();   // one-time per device: kernels' dynamic LDS attribute

struct GemmArgs {
  int fmt, M, N, K, r32;   // N, K: padded (whole 32-row blocks, whole 256-channel steps)
  int ldy;                 // the layer's N: Y's row stride and width (stores past it are dropped)
  int ldk;                 // the layer's K (the group-sum hook's groups)
  // operands in the layouts of Stage1Args and the packed layer (z and l2t
  // unused when r32 == 0)
  const uint8_t* qx;
  const void* sx;
  const uint16_t* z;
  const uint8_t* qw;
  const void* sw;
  const uint16_t* l2t;
  const uint16_t* bias;  // bf16 [N]
  uint16_t* y;           // bf16 [M][ldy]
  // tiled INT4 GEMM: the workspace areas that receive the FP6 copies of qx
  // and qw (the launch fills them before the GEMM; layout in ws_layout)
  uint8_t* qx6;
  uint8_t* qw6;
  // INT4 split of the last tiles: per-tile ticket counters (cleared by
  // stage 1) and fp32 partial tiles, in the workspace
  uint32_t* flags;
  float* part;
  // group-sum test hook (INT4): window and output [mc][nc][K/64], p ==
  // nullptr for the normal epilogue
  int32_t* p;
  int m0, mc, n0, nc;
  // fused next layer (tiled kernels only; nxt_qx == nullptr otherwise):
  // instead of Y, the epilogue writes the next layer's codes and scales (its
  // format, the same as this layer's) of GELU(bf16(Y)) smoothed by nxt_mu
  // (its stage-1 layout, K = this N) and the fp32 partial X_hat L1 of each
  // tile column (256 channels INT4, 384 MXFP4), [N/tile width][M][nxt_r32]
  uint8_t* nxt_qx;
  void* nxt_sx;
  const float* nxt_mu;
  const uint16_t* nxt_l1s;   // next layer's L1 in its stage-1 layout
  float* nxt_zpart;
  int nxt_r32;
};
hipError_t launch_gemm_int4(const GemmArgs& a, int num_cus, hipStream_t st);
// after a fused MLP-up GEMM: Z of the next layer = bf16 of the tile partials
// added in tile order, in fragment order; also clears that layer's split
// counters (its stage 1 does not run)
hipError_t launch_fused_zsum(const float* zpart, int tiles_n, int M, int r32, uint16_t* z, uint32_t* flags,
                             int nflags, hipStream_t st);
// y = GELU(y) in place over n bf16 values (n % 8 == 0): the activation between
// the MLP layers when they are not fused
hipError_t launch_gelu_bf16(uint16_t* y, size_t n, hipStream_t st);
// few tokens (INT4: at most 256, or 769 to 1024; MXFP4: at most 256; no
// group-sum hook): the weight-streaming kernel of either format
bool gemm_small_fits(const GemmArgs& a, int num_cus);
hipError_t launch_gemm_small(const GemmArgs& a, int num_cus, hipStream_t st);
hipError_t launch_gemm_mxfp4(const GemmArgs& a, int num_cus, hipStream_t st);
// one-time per device: the kernels' dynamic LDS attribute
hipError_t prepare_gemm_int4();
hipError_t prepare_gemm_mxfp4();

// The AWQ-style W4A16 linear (layouts in svdq.h): y [M][N] bf16.
struct AwqArgs {
  int M, K, N;
  const uint16_t* x;       // bf16 [M][K]
  const float* inv_s;      // [K]
  const uint8_t* qw;       // [N/16][K/128][64][16]
  const float* scales;     // [N/16][K/128][16]
  const uint8_t* zeros;    // [N/16][K/128][16]
  const uint16_t* bias;    // bf16 [N]
  uint16_t* y;
};
hipError_t launch_awq(const AwqArgs& a, int num_cus, hipStream_t st);
hipError_t prepare_awq();

// Layer norm and its gradients (svdq_norm.hip); strides in elements
struct NormArgs {
  int dtype, pdtype, one_plus, C, G;
  float eps;
  int64_t M, rpg;
  const void* x;
  int64_t ldx;
  const void* w;   // [G][ldw] or null (gain 1)
  int64_t ldw;
  const void* b;   // [G][ldb] or null (0)
  int64_t ldb;
  void* y;
  int64_t ldy;
  float* mean;     // [M], may be null in the forward
  float* rstd;
  // q != nullptr (bf16 rows): instead of y, its E4M3 codes [M][Kp] and block
  // scales (fp8_scale_index over qs_rows rows)
  uint8_t* q;
  uint8_t* qs;
  int Kp;
  int64_t qs_rows;
  uint32_t* tickets;   // kFp8Tickets words to zero for the product, may be null
};
struct NormGradPlan;
struct NormGradArgs {
  NormArgs f;        // x, weight, mean and rstd
  const void* dy;
  int64_t lddy;
  void* dx;
  int64_t lddx;
  void* dw;          // [G][C] of gdtype, may be null
  void* db;
  int gdtype;
  float* part;       // [G][runs][2][C], null when a group is one run
  int once;          // set by launch_norm_grad: x and dy are read past the caches
};
hipError_t launch_norm(const NormArgs& a, int num_cus, hipStream_t st);
hipError_t prepare_norm();
hipError_t launch_norm_grad(const NormGradArgs& g, const NormGradPlan& p, hipStream_t st);

// E4M3 quantizers (svdq_fp8_quant.hip)
// (plain: the scale bytes as svdq_fp8_quantize documents them, not the product's order)
// `tickets`, where given: kFp8Tickets words that the kernel zeroes for the product behind it
hipError_t launch_fp8_quant_rows(const uint16_t* x, int64_t M, int K, uint8_t* q, uint8_t* s, bool plain, uint32_t* tickets,
                                 hipStream_t st);
// one or two matrices bf16 [M][C] quantized along M (codes [C][round128(M)]);
// the first also along C (row codes) and summed over M where asked
struct Fp8QuantT {
  const uint16_t* x;
  int C;
  uint8_t* qt;       // [C][round128(M)], or null
  uint8_t* st;
  uint8_t* q;        // [M][round128(C)], or null
  uint8_t* s;
  float* sums;       // [round128(M)/128][C], or null
};
hipError_t launch_fp8_quant_t(const Fp8QuantT& a, const Fp8QuantT& b, int64_t M, uint32_t* tickets, hipStream_t st);   // 2 kFp8Tickets
// the bias gradient: the blocks' sums per channel
struct Fp8BiasGrad {
  const float* sums;   // [blocks][N]
  int blocks, N;
  uint16_t* db;
};
hipError_t launch_fp8_bias_grad(const Fp8BiasGrad& a, hipStream_t st);
hipError_t launch_fp8_zero(void* p, size_t bytes, int num_cus, hipStream_t st);   // bytes % 4 == 0
hipError_t launch_fp8_pack(const void* w, int dtype, int K, int N, uint8_t* q, uint8_t* s, uint8_t* qt, uint8_t* st,
                           hipStream_t stream);

// out[a_rows][b_rows] = A B^T (+ bias per column): E4M3 codes with the
// contracted channels contiguous and an E8M0 scale per row and 128 of them
// (A; B as well with b_row_scales), or per 128 x 128 block of B
struct Fp8Gemm {
  const uint8_t* a;
  const uint8_t* as;
  int64_t a_rows, lda;
  const uint8_t* b;
  const uint8_t* bs;
  int b_rows;
  int64_t ldb;
  int b_row_scales;
  int64_t K;           // contracted channels
  const uint16_t* bias;
  uint16_t* out;       // bf16 [a_rows][b_rows]
  float* part;         // where fp8_deep has several runs: their sums, and a zeroed ticket per tile
  uint32_t* tickets;
  const uint16_t* x;   // launch_fp8_gemm_small: A as bf16 rows [a_rows][K], or null
};
// bias: that gradient too, by further workgroups, where fp8_gemm_takes_bias
bool fp8_gemm_takes_bias(const Fp8Gemm& g);
hipError_t launch_fp8_gemm(const Fp8Gemm& g, int num_cus, hipStream_t st, const Fp8BiasGrad* bias = nullptr);
hipError_t launch_fp8_gemm_small(const Fp8Gemm& g, int num_cus, hipStream_t st);
hipError_t prepare_fp8();

// A grid of at least n workgroups: a launch's dimension takes fewer than 2^32
// threads, so from 2^20 workgroups on they lie in rows of so many (the last
// row goes past n).
inline dim3 many_groups(int64_t n) {
  const int64_t row = (int64_t)1 << 20;
  return n <= row ? dim3((unsigned)n) : dim3((unsigned)row, (unsigned)((n + row - 1) / row));
}

// shared by the files with C entry points (svdq_api.hip)
enum KernelSets : unsigned { kKernelsNorm = 1, kKernelsFp8 = 2 };
svdq_status check_device(int* cus = nullptr, void** scratch_ptr = nullptr, unsigned kernels = 0);
svdq_status after_launch(hipError_t e, hipStream_t s);

// measured ceilings of the part (not part of the layer): an MFMA-only loop
// (kind 0 scaled FP4, 1 i8, 2 bf16; *flops = its flop count) and a device copy
hipError_t launch_mfma_peak(int kind, int constant, int iters, int grid, float* sink, hipStream_t st, double* flops);
hipError_t launch_copy(const void* src, void* dst, size_t bytes, int num_cus, hipStream_t st);

inline hipError_t launch_gemm(const GemmArgs& a, int num_cus, hipStream_t st) {
  if (a.M == 0) return hipSuccess;
  if (gemm_small_fits(a, num_cus)) return launch_gemm_small(a, num_cus, st);
  return a.fmt == SVDQ_FMT_MXFP4_G32 ? launch_gemm_mxfp4(a, num_cus, st) : launch_gemm_int4(a, num_cus, st);
}

}  // namespace svdq
