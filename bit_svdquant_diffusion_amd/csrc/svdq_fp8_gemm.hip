// The FP8 product: out[m][n] = sum_k 2^(ea + eb) a[m][k] b[n][k] (+ bias[n]),
// a and b E4M3 codes with the contracted channels contiguous, ea and eb the
// exponents of their blocks of 128 channels, on the block-scaled MFMA
// v_mfma_scale_f32_32x32x64_f8f6f4 (16x16x128 with few tokens), which applies
// the scales itself (its sums: the products of eight consecutive channels are
// aligned to the largest's exponent, what lies below 2^-13 of it is dropped,
// and the rest is added in fp32; over 4096 random products the result is
// 1.4e-5 off, a hundredth of its rounding to bf16). The forward's operands are (X, W), the input gradient's
// (dY, W^T), the weight gradient's (dY^T, X^T).
//
// Both operands are plain row-major bytes in memory. A stage is 128 channels
// of both: `buffer_load_dwordx4 ... lds` transfers of eight rows x 128 bytes,
// whose lanes fetch their 16-byte chunks permuted (chunk c of row r goes to
// place c ^ (r / 2 % 8) of its 128-byte row), so that the fragment reads of
// sixteen consecutive rows at one chunk cover all 64 LDS banks once. The
// weight side is the MFMA's operand A, so a lane's accumulators hold one
// token and runs of four output channels.
#include <algorithm>

#include "svdq_gemm_common.h"
#include "svdq_internal.h"
#include "svdq_layout.h"
#include "svdq_types.h"

namespace svdq {

namespace {

typedef __attribute__((address_space(3))) void lds_void;
__device__ __forceinline__ lds_void* lds_ptr(uint8_t* p) { return (lds_void*)p; }
// 16 bytes per lane from the resource to 1 KiB of LDS (a function of its own:
// the host pass does not take the builtin inside a template)
__device__ __forceinline__ void lds_transfer(__amdgpu_buffer_rsrc_t r, uint8_t* dst, uint32_t voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds_ptr(dst), 16, voff, soff, 0, 0);
}
constexpr int kRsrcWord3 = 0x00020000;   // buffer resources: raw bytes
constexpr uint32_t kOutside = 0x7ffffff0u;   // a lane offset past the end of every resource: loads zero

// Tile of BM tokens x BN channels by WGM x WGN waves of TM x TN blocks of
// 32 x 32.
template <int BM_, int BN_, int WGM_, int WGN_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, NW = WGM * WGN;
  static constexpr int WM = BM / WGM, WN = BN / WGN, TM = WM / 32, TN = WN / 32;
  static constexpr int kSlotA = BM * 128, kSlot = (BM + BN) * 128;
  static constexpr int kOpsA = BM / 8 / NW, kOpsB = BN / 8 / NW;   // transfers per wave and stage
  static_assert(kOpsA % 2 == 0 && kOpsB % 2 == 0 && BM % (8 * NW) == 0 && BN % (8 * NW) == 0,
                "every wave issues whole pairs of transfers of both operands");
};

// BROW: B has a scale per row (else per 128 x 128 block: one word per wave
// and four stages, as a wave's channels lie in one block).
template <int BM, int BN, int WGM, int WGN, bool BROW>
__global__ __launch_bounds__(64 * WGM * WGN) __attribute__((amdgpu_waves_per_eu(1)))
void fp8_gemm_kernel(Fp8Gemm g, int tiles_m, int tiles_n, int group_m) {
  typedef Tile<BM, BN, WGM, WGN> TL;
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int TM = TL::TM, TN = TL::TN, SB = BROW ? TN : 1;
  static_assert(128 % TL::WN == 0, "a wave's channels lie in one block of 128");
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, lr = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / TL::WGN, wn = wave % TL::WGN;
  const TileMap tm = map_tile((int)blockIdx.x, tiles_m, tiles_n, group_m);
  const int Ra = (int)g.a_rows, Rb = g.b_rows, K = (int)g.K, KB = (K + 127) / 128;
  const int m0 = __builtin_amdgcn_readfirstlane(tm.tm) * TL::BM, n0 = __builtin_amdgcn_readfirstlane(tm.tn) * TL::BN;
  const int lda = (int)g.lda, ldb = (int)g.ldb;

  // transfers: the tile's rows of each operand as a buffer resource (rows past
  // it read as zeros), a lane's chunk of the two kinds of row octets
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void*)(g.a + (size_t)m0 * lda), 0, min(TL::BM, Ra - m0) * lda, kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc((void*)(g.b + (size_t)n0 * ldb), 0, min(TL::BN, Rb - n0) * ldb, kRsrcWord3);
  const int ck[2] = {(lane & 7) ^ (lane >> 4), (lane & 7) ^ (4 + (lane >> 4))};   // chunk for even and odd octets
  uint32_t va[2], vb[2];
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    va[o] = (uint32_t)((wave * TL::kOpsA * 8 + (lane >> 3)) * lda + 16 * ck[o]);
    vb[o] = (uint32_t)((wave * TL::kOpsB * 8 + (lane >> 3)) * ldb + 16 * ck[o]);
  }
  // transfer i (of kOps) of stage S into slot S % 2; chunks past the contracted
  // channels (and every chunk of a stage past the last) are zeros
#define SVDQ_ISSUE_BEGIN(S)                                                                                 \
  uint8_t* slot_w = smem + ((S) & 1) * TL::kSlot + wave * TL::kOpsA * 1024;                                 \
  const int k0 = (S) * 128;                                                                                 \
  uint32_t ta[2], tb[2];                                                                                    \
  _Pragma("unroll") for (int o = 0; o < 2; ++o) {                                                           \
    const bool out = 16 * ck[o] >= K - k0;                                                                  \
    ta[o] = out ? kOutside : va[o];                                                                         \
    tb[o] = out ? kOutside : vb[o];                                                                         \
  }
#define SVDQ_ISSUE(i)                                                                                       \
  if ((i) < TL::kOpsA)                                                                                      \
    lds_transfer(ra, slot_w + (i) * 1024, ta[(i) & 1], (i) * 8 * lda + k0);                                 \
  else                                                                                                      \
    lds_transfer(rb, slot_w + TL::kSlotA + (wave * (TL::kOpsB - TL::kOpsA) + (i) - TL::kOpsA) * 1024,       \
                 tb[((i) - TL::kOpsA) & 1], ((i) - TL::kOpsA) * 8 * ldb + k0);
  // scale words (four blocks' bytes) of this wave's rows, read one stage
  // ahead: of A (and of B with a scale per row) the words of a lane's rows in
  // the wave's 32-row blocks stand together
  typedef uint32_t words_a __attribute__((ext_vector_type(TM)));
  typedef uint32_t words_b __attribute__((ext_vector_type(TN)));
  const int wrow = m0 + wm * TL::WM, wcol = n0 + wn * TL::WN;
  const uint32_t* pa = reinterpret_cast<const uint32_t*>(g.as) + wrow / 128 * 128 + lr * 4 + wrow % 128 / 32;
  const uint32_t* pb = reinterpret_cast<const uint32_t*>(g.bs) +
                       (BROW ? wcol / 128 * 128 + lr * 4 + wcol % 128 / 32 : min(wcol, Rb - 1) / 128 * ((KB + 3) / 4));
  const int ga = (Ra + 127) / 128 * 128, gb = BROW ? (Rb + 127) / 128 * 128 : 1;   // words between groups of four blocks
  // (rows past the last 128 of the operand, whose outputs are not stored, read its first words)
  if (wrow >= ga) pa = reinterpret_cast<const uint32_t*>(g.as) + lr * 4;
  if (BROW && wcol >= gb) pb = reinterpret_cast<const uint32_t*>(g.bs) + lr * 4;
  words_a na, ca;
  words_b nb, cb;
#define SVDQ_SCALES(S)                                                                                      \
  {                                                                                                         \
    const int grp = min((S), KB - 1) / 4;                                                                   \
    na = *reinterpret_cast<const words_a*>(pa + (size_t)grp * ga);                                          \
    if constexpr (BROW)                                                                                     \
      nb = *reinterpret_cast<const words_b*>(pb + (size_t)grp * gb);                                        \
    else                                                                                                    \
      nb[0] = pb[grp];                                                                                      \
  }
  // LDS addresses of this lane's fragment chunks: rows wm WM + lr (+ 32 t),
  // chunk 4 step + 2 h + e at place chunk ^ (row / 2 % 8)
  const int sw = (lr >> 1) & 7;
  uint32_t at_a[2][2], at_b[2][2];
#pragma unroll
  for (int st = 0; st < 2; ++st)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t c = (uint32_t)((4 * st + 2 * h + e) ^ sw) * 16;
      at_a[st][e] = (wm * TL::WM + lr) * 128 + c;
      at_b[st][e] = TL::kSlotA + (wn * TL::WN + lr) * 128 + c;
    }
// fragment t of the step (B's TN, then A's TM)
#define SVDQ_READ(S, ST, FA, FB, t)                                                                         \
  {                                                                                                         \
    const uint8_t* slot = smem + ((S) & 1) * TL::kSlot + ((t) < TN ? (t) : (t) - TN) * 4096;                \
    const i32x4 lo = *reinterpret_cast<const i32x4*>(slot + ((t) < TN ? at_b[ST][0] : at_a[ST][0]));        \
    const i32x4 hi = *reinterpret_cast<const i32x4*>(slot + ((t) < TN ? at_b[ST][1] : at_a[ST][1]));        \
    ((t) < TN ? FB[(t) < TN ? (t) : 0] : FA[(t) < TN ? 0 : (t) - TN]) =                                     \
        i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};                                      \
  }
#define SVDQ_MFMA(FA, FB)                                                                                   \
  _Pragma("unroll") for (int i = 0; i < TM; ++i) _Pragma("unroll") for (int j = 0; j < TN; ++j)             \
      acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(FB[j], FA[i], acc[j][i], 0, 0, 0,          \
                                                                  (int)cb[BROW ? j : 0], 0, (int)ca[i]);

  f32x16 acc[TN][TM];
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int i = 0; i < TM; ++i) acc[j][i] = f32x16{};
  // Per stage: the first step's fragments are read while the previous stage's
  // second half multiplies, the second step's while the first half does; the
  // next stage's transfers are issued from the start of the stage on, as they
  // take about half of its time (64 bytes a clock) and then the memory's
  // latency. Reads and transfers stand in this order in the source (the
  // compiler does not move LDS reads over transfers into LDS); the scheduling
  // groups place them between the MFMAs: a fragment and a transfer to an MFMA
  // first, then the other transfers. (Left to itself the compiler reuses the
  // fragments' registers and reads only when the multiplications are through.)
  constexpr int kFrags = TM + TN, kMfma = TM * TN, kOps = TL::kOpsA + TL::kOpsB;
  constexpr int kFirst = kMfma / 2, kPerF = kFrags / kFirst, kPerT = kOps / kMfma;
  static_assert(kFirst * kPerF == kFrags && kMfma * kPerT == kOps, "whole fragments and transfers per MFMA");
#define SVDQ_RING_WAIT                                                                                      \
  __builtin_amdgcn_sched_barrier(0);                                                                        \
  __builtin_amdgcn_s_waitcnt(0x0070); /* vmcnt 0, lgkmcnt 0: this stage's transfers, earlier reads */       \
  __builtin_amdgcn_s_barrier();                                                                             \
  __builtin_amdgcn_sched_barrier(0);
#define SVDQ_FIRST_HALF(S)                                                                                  \
  SVDQ_ISSUE_BEGIN((S) + 1)                                                                                 \
  _Pragma("unroll") for (int q = 0; q < kMfma; ++q) {                                                       \
    if (q < kFirst) {                                                                                       \
      _Pragma("unroll") for (int f = 0; f < kPerF; ++f) SVDQ_READ(S, 0, xa, xb, q * kPerF + f)              \
    }                                                                                                       \
    _Pragma("unroll") for (int f = 0; f < kPerT; ++f) { SVDQ_ISSUE(q * kPerT + f) }                         \
  }
#define SVDQ_SECOND_HALF(S)                                                                                 \
  _Pragma("unroll") for (int t = 0; t < TM; ++t) ca[t] = wa[t] >> (8 * ((S) & 3));                          \
  _Pragma("unroll") for (int t = 0; t < SB; ++t) cb[t] = wb[t] >> (8 * ((S) & 3));                          \
  _Pragma("unroll") for (int f = 0; f < kFrags; ++f) SVDQ_READ(S, 1, ya, yb, f)                             \
  SVDQ_MFMA(xa, xb)                                                                                         \
  _Pragma("unroll") for (int q = 0; q < kMfma; ++q) {                                                       \
    __builtin_amdgcn_sched_group_barrier(0x100, 2 * kFrags / kMfma, 0); /* LDS reads */                     \
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                  /* MFMA */                          \
  }
  i32x8 xa[TM], xb[TN], ya[TM], yb[TN];
  {
    SVDQ_ISSUE_BEGIN(0)
#pragma unroll
    for (int q = 0; q < kOps; ++q) { SVDQ_ISSUE(q) }
  }
  SVDQ_SCALES(0)
  {
    SVDQ_RING_WAIT
    const words_a wa = na;
    const words_b wb = nb;
    SVDQ_SCALES(1)
    SVDQ_FIRST_HALF(0)
    SVDQ_SECOND_HALF(0)
  }
  for (int s = 1; s < KB; ++s) {
    SVDQ_RING_WAIT
    const words_a wa = na;
    const words_b wb = nb;
    SVDQ_SCALES(s + 1)
    __builtin_amdgcn_sched_barrier(0);
    SVDQ_FIRST_HALF(s)
    SVDQ_MFMA(ya, yb)
#pragma unroll
    for (int q = 0; q < kMfma; ++q) {
      if (q < kFirst) __builtin_amdgcn_sched_group_barrier(0x100, 2 * kPerF, 0);
      __builtin_amdgcn_sched_group_barrier(0x020, kPerT, 0);   // transfers
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    SVDQ_SECOND_HALF(s)
  }
  SVDQ_MFMA(ya, yb)
#undef SVDQ_MFMA
#undef SVDQ_READ
#undef SVDQ_SCALES
#undef SVDQ_FIRST_HALF
#undef SVDQ_SECOND_HALF
#undef SVDQ_RING_WAIT
#undef SVDQ_ISSUE
#undef SVDQ_ISSUE_BEGIN
  __builtin_amdgcn_s_waitcnt(0x0070);   // the transfers issued past the end land before the LDS is given up
  // A lane holds token m0 + 32 i + lr and channels 32 j + 8 q + 4 h + (0..3).
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int nb = n0 + wn * TL::WN + 32 * j;
    float bv[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      u32x2 w = u32x2{0, 0};
      if (g.bias && nb + 8 * q + 4 * h < g.b_rows) w = *reinterpret_cast<const u32x2*>(g.bias + nb + 8 * q + 4 * h);
      bv[4 * q] = bf16lo(w.x);
      bv[4 * q + 1] = bf16hi(w.x);
      bv[4 * q + 2] = bf16lo(w.y);
      bv[4 * q + 3] = bf16hi(w.y);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int64_t m = m0 + wm * TL::WM + 32 * i + lr;
        uint32_t o[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) o[p] = cvt_bf16x2(acc[j][i][2 * p] + bv[2 * p], acc[j][i][2 * p + 1] + bv[2 * p + 1]);
        // (o[4p], o[4p+1]) is q = 2p, (o[4p+2], o[4p+3]) is q = 2p + 1: after
        // the swap lane half h holds channels 8 h + (0..7) and 16 + 8 h + (0..7)
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const auto r = __builtin_amdgcn_permlane32_swap(o[4 * p + w], o[4 * p + 2 + w], false, false);
            o[4 * p + w] = r[0];
            o[4 * p + 2 + w] = r[1];
          }
        uint16_t* y = g.out + m * g.b_rows + nb + 8 * h;
        if (m < g.a_rows) {
          if (nb < g.b_rows) *reinterpret_cast<u32x4*>(y) = u32x4{o[0], o[1], o[2], o[3]};
          if (nb + 16 < g.b_rows) *reinterpret_cast<u32x4*>(y + 16) = u32x4{o[4], o[5], o[6], o[7]};
        }
    }
  }
}

// Few tokens: the weight stream. A workgroup of eight waves owns 16 NT output
// channels; the waves split the contracted blocks in eight fixed runs (so a
// token's sum does not depend on the launch) and add their sums in order
// through LDS. Weights go from memory to the MFMA's operand registers
// directly: lane (r, c) of v_mfma_f32_16x16x128 holds row r, channels
// 16 c + (0..15) and 64 + 16 c + (0..15) of the block, so each of its two
// 16-byte loads covers 64 contiguous bytes of a row. (The order of the
// channels within a block is free as both operands share it.) With one token
// tile (TT = 1) and QUANT the wave quantizes its tokens' channels itself in
// that layout: the four lanes of a token hold a block.
constexpr int kSmallWaves = 8;
template <int TT, int NT, bool QUANT>
__global__ __launch_bounds__(64 * kSmallWaves) void fp8_small_kernel(Fp8Gemm g) {
  constexpr int kRing = NT * (QUANT ? 2 : TT) >= 4 ? 2 : 4;   // blocks in flight per wave
  __shared__ float red[kSmallWaves][NT * TT * 4][64];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int KB = (int)((g.K + 127) / 128), b0 = KB * wave / kSmallWaves, b1 = KB * (wave + 1) / kSmallWaves;
  const int n0 = blockIdx.x * 16 * NT;
  const uint8_t* wrow[NT];
  const uint8_t* wsc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int n = min(n0 + 16 * t + r, g.b_rows - 1);
    wrow[t] = g.b + (int64_t)n * g.ldb;
    wsc[t] = g.bs + (int64_t)(min(n0 + 16 * t, g.b_rows - 1) / 128) * ((KB + 3) / 4 * 4);
  }
  const uint8_t* arow[TT];
  const uint8_t* asc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int64_t m = min((int64_t)(16 * t + r), g.a_rows - 1);
    arow[t] = QUANT ? reinterpret_cast<const uint8_t*>(g.x + m * g.K) : g.a + m * g.lda;
    asc[t] = QUANT ? nullptr : g.as + fp8_scale_index(g.a_rows, m, 0);
  }
  i32x4 wq[kRing][NT][2];
  u32x4 xv[kRing][TT][QUANT ? 4 : 2];
  uint32_t ws[kRing][NT], xs[kRing][TT];
  auto load = [&](int u, int kb) {
    kb = min(kb, b1 - 1);   // past the run's end: its last block again, not used
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k = kb * 128 + 64 * e + 16 * c;
      const bool in = k < g.K;
#pragma unroll
      for (int t = 0; t < NT; ++t) wq[u][t][e] = in ? *reinterpret_cast<const i32x4*>(wrow[t] + k) : i32x4{0, 0, 0, 0};
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if constexpr (QUANT) {
          const u32x4* p = reinterpret_cast<const u32x4*>(arow[t] + 2 * k);
          xv[u][t][2 * e] = in ? p[0] : u32x4{0, 0, 0, 0};
          xv[u][t][2 * e + 1] = in ? p[1] : u32x4{0, 0, 0, 0};
        } else {
          xv[u][t][e] = *reinterpret_cast<const u32x4*>(arow[t] + k);   // padded to whole blocks
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) ws[u][t] = wsc[t][kb];
    if constexpr (!QUANT) {
#pragma unroll
      for (int t = 0; t < TT; ++t) xs[u][t] = asc[t][(size_t)(kb / 4) * round128(g.a_rows) * 4 + kb % 4];
    }
  };
  f32x4 acc[NT][TT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[n][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (b0 < b1) {
#pragma unroll
    for (int u = 0; u < kRing; ++u) load(u, b0 + u);
    for (int kb = b0; kb < b1; kb += kRing) {
#pragma unroll
      for (int u = 0; u < kRing; ++u) {
        if (kb + u < b1) {
          i32x8 fx[TT];
          int sx[TT];
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            if constexpr (QUANT) {
              uint32_t amax = 0;
#pragma unroll
              for (int i = 0; i < 16; ++i) amax = amax_bf16x2(amax, xv[u][t][i >> 2][i & 3]);
              // the token's other lanes: c ^ 1 (16 lanes on) and c ^ 2 (32)
              auto s1 = __builtin_amdgcn_permlane16_swap(amax, amax, false, false);
              amax = umax(s1[0], s1[1]);
              auto s2 = __builtin_amdgcn_permlane32_swap(amax, amax, false, false);
              amax = umax(s2[0], s2[1]);
              const int e = e4m3_exponent(amax);
              const float sc = exp2_int(e);
              sx[t] = e + 127;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint32_t w0 = xv[u][t][i >> 1][2 * (i & 1)], w1 = xv[u][t][i >> 1][2 * (i & 1) + 1];
                fx[t][i] = (int)e4m3x4(bf16lo(w0), bf16hi(w0), bf16lo(w1), bf16hi(w1), sc);
              }
            } else {
              const u32x4 x0 = xv[u][t][0], x1 = xv[u][t][1];
              fx[t] = i32x8{(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
              sx[t] = (int)xs[u][t];
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const i32x4 w0 = wq[u][n][0], w1 = wq[u][n][1];
            const i32x8 fw = i32x8{w0[0], w0[1], w0[2], w0[3], w1[0], w1[1], w1[2], w1[3]};
#pragma unroll
            for (int t = 0; t < TT; ++t)
              acc[n][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw, fx[t], acc[n][t], 0, 0, 0, (int)ws[u][n], 0, sx[t]);
          }
          if (kb + u + kRing < b1) load(u, kb + u + kRing);
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][(n * TT + t) * 4 + e][lane] = acc[n][t][e];
  __syncthreads();
  // a thread adds the waves' sums of pairs of consecutive channels: value e of
  // lane (r, c) is token 16 t + r, channel n0 + 16 n + 4 c + e
  for (int i = tid; i < NT * TT * 2 * 64; i += 64 * kSmallWaves) {
    const int l = i & 63, pe = (i >> 6) & 1, nt = i >> 7, n = nt / TT, t = nt % TT;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int w = 0; w < kSmallWaves; ++w) {
      s0 += red[w][nt * 4 + 2 * pe][l];
      s1 += red[w][nt * 4 + 2 * pe + 1][l];
    }
    const int64_t m = 16 * t + (l & 15);
    const int col = n0 + 16 * n + 4 * (l >> 4) + 2 * pe;
    if (m < g.a_rows && col < g.b_rows) {
      const uint32_t b = g.bias ? *reinterpret_cast<const uint32_t*>(g.bias + col) : 0u;
      *reinterpret_cast<uint32_t*>(g.out + m * g.b_rows + col) = cvt_bf16x2(s0 + bf16lo(b), s1 + bf16hi(b));
    }
  }
}

typedef Tile<256, 256, 2, 2> TileL;
typedef Tile<128, 128, 2, 2> TileM;

template <class TL, bool BROW>
hipError_t launch_tile(const Fp8Gemm& g, hipStream_t st) {
  const int tm = (int)((g.a_rows + TL::BM - 1) / TL::BM), tn = (g.b_rows + TL::BN - 1) / TL::BN;
  hipLaunchKernelGGL((fp8_gemm_kernel<TL::BM, TL::BN, TL::WGM, TL::WGN, BROW>), dim3((unsigned)(tm * tn)), dim3(64 * TL::NW), 2 * TL::kSlot, st, g, tm, tn, 8);
  return hipGetLastError();
}
template <class TL, bool BROW>
hipError_t prepare_tile() {
  return hipFuncSetAttribute((const void*)fp8_gemm_kernel<TL::BM, TL::BN, TL::WGM, TL::WGN, BROW>, hipFuncAttributeMaxDynamicSharedMemorySize, 2 * TL::kSlot);
}

}  // namespace

hipError_t prepare_fp8() {
  for (hipError_t e : {prepare_tile<TileL, false>(), prepare_tile<TileL, true>(), prepare_tile<TileM, false>(),
                       prepare_tile<TileM, true>()})
    if (e != hipSuccess) return e;
  return hipSuccess;
}

bool fp8_gemm_small_fits(const Fp8Gemm& g) { return g.a_rows <= 64 && !g.b_row_scales; }

hipError_t launch_fp8_gemm_small(const Fp8Gemm& g, int num_cus, hipStream_t st) {
  (void)num_cus;
  const dim3 b(64 * kSmallWaves);
  if (g.x) {
    hipLaunchKernelGGL((fp8_small_kernel<1, 1, true>), dim3((g.b_rows + 15) / 16), b, 0, st, g);
  } else if (g.a_rows <= 16) {
    hipLaunchKernelGGL((fp8_small_kernel<1, 1, false>), dim3((g.b_rows + 15) / 16), b, 0, st, g);
  } else if (g.a_rows <= 32) {
    hipLaunchKernelGGL((fp8_small_kernel<2, 1, false>), dim3((g.b_rows + 15) / 16), b, 0, st, g);
  } else {
    hipLaunchKernelGGL((fp8_small_kernel<4, 1, false>), dim3((g.b_rows + 15) / 16), b, 0, st, g);
  }
  return hipGetLastError();
}

hipError_t launch_fp8_gemm(const Fp8Gemm& g, int num_cus, hipStream_t st) {
  if (fp8_gemm_small_fits(g)) return launch_fp8_gemm_small(g, num_cus, st);
  const int64_t large = ((g.a_rows + 255) / 256) * ((g.b_rows + 255) / 256);
  if (large >= num_cus)
    return g.b_row_scales ? launch_tile<TileL, true>(g, st) : launch_tile<TileL, false>(g, st);
  return g.b_row_scales ? launch_tile<TileM, true>(g, st) : launch_tile<TileM, false>(g, st);
}

}  // namespace svdq
