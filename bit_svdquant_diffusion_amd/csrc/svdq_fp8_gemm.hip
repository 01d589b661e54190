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
__device__ __forceinline__ void store_16(__amdgpu_buffer_rsrc_t r, u32x4 v, int off) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, 0);
}
__device__ __forceinline__ void store_16_once(__amdgpu_buffer_rsrc_t r, u32x4 v, int off) {   // non-temporal
  __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, 2);
}
constexpr int kRsrcWord3 = 0x00020000;   // buffer resources: raw bytes
constexpr uint32_t kOutside = 0x7ffffff0u;   // a lane offset past the end of every resource: loads zero

// Tile of BM tokens x BN channels by WGM x WGN waves of TM x TN blocks of
// 32 x 32.
template <int BM_, int BN_, int WGM_, int WGN_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, NW = WGM * WGN;
  static constexpr int WM = BM / WGM, WN = BN / WGN, TM = WM / 32, TN = WN / 32;
  // LDS: a ring of five units, a unit one operand's 128 channels of a stage
  static constexpr int kUnit = (BM > BN ? BM : BN) * 128, kUnits = 5, kLds = kUnits * kUnit;
  static constexpr int kOpsA = BM / 8 / NW, kOpsB = BN / 8 / NW, kOps = kOpsA + kOpsB;   // transfers per wave and stage
  static constexpr int kFrags = TM + TN, kMfma = TM * TN;   // fragments and MFMAs per wave and half stage
  static constexpr int kStores = 2 * TM * TN;               // 16-byte stores per wave and tile
  static_assert(kOpsA % 2 == 0 && kOpsB % 2 == 0 && BM % (8 * NW) == 0 && BN % (8 * NW) == 0,
                "every wave issues whole pairs of transfers of both operands");
  static_assert(kOpsA + kStores < 64 && kFrags <= kMfma, "vmcnt range; a fragment or less to an MFMA");
  // transfers issued up to MFMA q of a first half
  static constexpr int ops_until(int q) { return q * kOps / kMfma; }
};

// Scheduling groups of a first half: to MFMA q a fragment's two LDS reads
// while there are any, and the transfers that are due; of a second half: the
// reads spread evenly.
template <class TL, int Q>
__device__ __forceinline__ void spread_first() {
  if constexpr (Q < TL::kFrags) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
  constexpr int kDue = TL::ops_until(Q + 1) - TL::ops_until(Q);
  if constexpr (kDue > 0) __builtin_amdgcn_sched_group_barrier(0x020, kDue, 0);
  __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  if constexpr (Q + 1 < TL::kMfma) spread_first<TL, Q + 1>();
}
template <class TL, int Q>
__device__ __forceinline__ void spread_second() {
  constexpr int kDue = (Q + 1) * 2 * TL::kFrags / TL::kMfma - Q * 2 * TL::kFrags / TL::kMfma;
  if constexpr (kDue > 0) __builtin_amdgcn_sched_group_barrier(0x100, kDue, 0);
  __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  if constexpr (Q + 1 < TL::kMfma) spread_second<TL, Q + 1>();
}

// The bf16 pairs of a lane's 16 channels 8 q + 4 h + (0..3) of row lr of a
// 32 x 32 block, o[2 q], o[2 q + 1], exchanged so that o[0..3] are channels
// 8 h + 16 (lr / 16) + (0..7) of row lr % 16 and o[4..7] of row lr % 16 + 16
__device__ __forceinline__ void spread_rows(uint32_t (&o)[8]) {
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int w = 0; w < 2; ++w) {   // to channels 16 p + 8 h + (0..7) of row lr
      const auto r = __builtin_amdgcn_permlane32_swap(o[4 * p + w], o[4 * p + 2 + w], false, false);
      o[4 * p + w] = r[0];
      o[4 * p + 2 + w] = r[1];
    }
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const auto r = __builtin_amdgcn_permlane16_swap(o[w], o[4 + w], false, false);
    o[w] = r[0];
    o[4 + w] = r[1];
  }
}

// wait until at most N vector-memory operations are outstanding and all LDS
// reads have returned, then the workgroup's barrier; nothing moves across
template <int N>
__device__ __forceinline__ void ring_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

// BROW: B has a scale per row (else per 128 x 128 block).
//
// Persistent workgroups of four waves (one a SIMD, so a wave has 512
// registers: 256 accumulators and two sets of fragments) walk their tiles; the
// stages of all their tiles are one sequence. LDS is a ring of five units
// A0 B0 A1 B1 A2 ...: while stage s is read, B of stage s + 1 and then A of
// stage s + 2 are fetched into the units that stage s - 1 was read from, so A
// has two stages' time to arrive and B, fetched first, one. Near a tile's end
// these are the next tile's, which arrive while the tile is stored.
//
// Per stage: the first step's fragments are read while the previous stage's
// second half multiplies, the second step's while the first half does. Reads
// and transfers stand in their order in the source (the compiler does not
// move LDS reads over transfers into LDS) and the scheduling groups place
// them between the MFMAs. (Left to itself the compiler reuses the fragments'
// registers and reads only when the multiplications are through.)
//
// Measured, with the quantizer's launch: 8192^3 397 us (2.77 PFLOP/s; a
// library's product alone 390 to 425) with inputs that stay in the caches and
// 425 with three sets in turn, 4608 tokens 3072 -> 12288 150 us (2.32) with
// either. The matrix units are busy 52% of that: random codes draw so much power that an
// MFMA loop alone reaches 3.4 to 3.9 of its 5 PFLOP/s, and a stage's 64 KB
// come from L2s that miss for a third of it.
template <int BM, int BN, int WGM, int WGN, bool BROW>
__global__ __launch_bounds__(64 * WGM * WGN) __attribute__((amdgpu_waves_per_eu(1)))
void fp8_gemm_kernel(Fp8Gemm g, int tiles_m, int tiles_n, int group_m) {
  typedef Tile<BM, BN, WGM, WGN> TL;
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int TM = TL::TM, TN = TL::TN;
  constexpr bool kOneBlock = !BROW && 128 % TL::WN == 0;   // a wave's channels lie in one block of 128
  constexpr int SB = kOneBlock ? 1 : TN;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, lr = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WGN, wn = wave % WGN;
  // KR blocks of 128 channels; at least three stages (the rest multiply zeros), so
  // that fetching two stages ahead never passes the next tile
  const int Ra = (int)g.a_rows, Rb = g.b_rows, K = (int)g.K, KR = (K + 127) / 128, KB = max(KR, 3);
  const int lda = (int)g.lda, ldb = (int)g.ldb;
  const int ntiles = tiles_m * tiles_n, grid = (int)gridDim.x;
  // Outputs of more than 64 MB are written past the caches, where they would
  // push out the operands and not stay (4608 x 12288, 113 MB: 150 us against
  // 159, with a GELU that reads them right after 217 either way; 8192 x 8192,
  // 134 MB: 428 against 436; 4608 x 6144, 57 MB: 80.5 against 83.4, so the
  // border could lie lower, were a reader never next).
  const bool once = (int64_t)Ra * Rb > (int64_t)32000000;

  // Transfers: a tile's rows of an operand as a buffer resource (rows past it
  // read as zeros: gfx950 checks the lane's and the scalar offset together
  // against the resource's size); a lane's chunk of the even and the odd row
  // octets.
  const int ck[2] = {(lane & 7) ^ (lane >> 4), (lane & 7) ^ (4 + (lane >> 4))};
  uint32_t va[2], vb[2];
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    va[o] = (uint32_t)((wave * TL::kOpsA * 8 + (lane >> 3)) * lda + 16 * ck[o]);
    vb[o] = (uint32_t)((wave * TL::kOpsB * 8 + (lane >> 3)) * ldb + 16 * ck[o]);
  }
#define SVDQ_RSRC_A(m0) \
  __builtin_amdgcn_make_buffer_rsrc((void*)(g.a + (size_t)(m0) * lda), 0, min(BM, Ra - (m0)) * lda, kRsrcWord3)
#define SVDQ_RSRC_B(n0) \
  __builtin_amdgcn_make_buffer_rsrc((void*)(g.b + (size_t)(n0) * ldb), 0, min(BN, Rb - (n0)) * ldb, kRsrcWord3)
  // the fetched stages: operand, channel offset, LDS unit
  __amdgpu_buffer_rsrc_t fa_res, fb_res;
  int fa_k = 0, fb_k = 0;
  uint32_t fa_unit = 0, fb_unit = TL::kUnit;
  // chunks past the contracted channels are zeros
#define SVDQ_FETCH_BEGIN                                                                                    \
  uint32_t ta[2], tb[2];                                                                                    \
  _Pragma("unroll") for (int o = 0; o < 2; ++o) {                                                           \
    ta[o] = 16 * ck[o] >= K - fa_k ? kOutside : va[o];                                                      \
    tb[o] = 16 * ck[o] >= K - fb_k ? kOutside : vb[o];                                                      \
  }
#define SVDQ_FETCH_A(i) \
  lds_transfer(fa_res, smem + fa_unit + (wave * TL::kOpsA + (i)) * 1024, ta[(i) & 1], (i) * 8 * lda + fa_k);
#define SVDQ_FETCH_B(i) \
  lds_transfer(fb_res, smem + fb_unit + (wave * TL::kOpsB + (i)) * 1024, tb[(i) & 1], (i) * 8 * ldb + fb_k);
  // the next stage of an operand; past the tile's last the next tile's first
#define SVDQ_FETCHED(X, NEXT)                                                                               \
  {                                                                                                         \
    f##X##_unit = f##X##_unit >= 3 * TL::kUnit ? f##X##_unit - 3 * TL::kUnit : f##X##_unit + 2 * TL::kUnit;  \
    f##X##_k += 128;                                                                                        \
    if (f##X##_k >= KB * 128) {                                                                             \
      f##X##_k = 0;                                                                                         \
      f##X##_res = NEXT;                                                                                    \
    }                                                                                                       \
  }
  // LDS offsets in a unit of this lane's fragment chunks: rows wm WM + lr
  // (+ 32 t), chunk 4 step + 2 h + e at place chunk ^ (row / 2 % 8)
  const int sw = (lr >> 1) & 7;
  uint32_t at_a[2][2], at_b[2][2];
#pragma unroll
  for (int st = 0; st < 2; ++st)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t c = (uint32_t)((4 * st + 2 * h + e) ^ sw) * 16;
      at_a[st][e] = (wm * TL::WM + lr) * 128 + c;
      at_b[st][e] = (wn * TL::WN + lr) * 128 + c;
    }
  // fragment t of step ST (B's TN, then A's TM)
#define SVDQ_READ(ST, FA, FB, t)                                                                            \
  {                                                                                                         \
    const uint8_t* unit = smem + ((t) < TN ? rb_unit + (t) * 4096 : ra_unit + ((t) - TN) * 4096);           \
    const i32x4 lo = *reinterpret_cast<const i32x4*>(unit + ((t) < TN ? at_b[ST][0] : at_a[ST][0]));        \
    const i32x4 hi = *reinterpret_cast<const i32x4*>(unit + ((t) < TN ? at_b[ST][1] : at_a[ST][1]));        \
    ((t) < TN ? FB[(t) < TN ? (t) : 0] : FA[(t) < TN ? 0 : (t) - TN]) =                                     \
        i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};                                      \
  }
#define SVDQ_MFMA(FA, FB)                                                                                   \
  _Pragma("unroll") for (int i = 0; i < TM; ++i) _Pragma("unroll") for (int j = 0; j < TN; ++j)             \
      acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(FB[j], FA[i], acc[j][i], 0, 0, 0,          \
                                                                  (int)cb[kOneBlock ? 0 : j], 0, (int)ca[i]);
  // Scale words (four blocks' bytes) of this wave's rows, read a stage ahead.
  // The words of a lane's rows in four 32-row blocks stand together, so a wave
  // whose rows lie in one run of 128 reads them with one load.
  constexpr bool kVecA = 128 % TL::WM == 0, kVecB = BROW && 128 % TL::WN == 0;
  uint32_t na[TM], nb[SB], wa[TM], wb[SB], ca[TM], cb[SB];
  const uint32_t *pa[kVecA ? 1 : TM], *pb[kVecB ? 1 : SB];
  const size_t ga = (size_t)round128(Ra), gb = BROW ? (size_t)round128(Rb) : 1;   // words between groups of four blocks
  // (rows past the operand, whose outputs are not stored, read its first words)
#define SVDQ_SCALE_ROWS(m0, n0)                                                                             \
  _Pragma("unroll") for (int t = 0; t < (kVecA ? 1 : TM); ++t) {                                            \
    const int blk = (m0) + wm * TL::WM + 32 * t;                                                            \
    pa[t] = reinterpret_cast<const uint32_t*>(g.as) + lr * 4 + (blk < Ra ? blk / 128 * 128 + blk % 128 / 32 : 0); \
  }                                                                                                         \
  _Pragma("unroll") for (int t = 0; t < (kVecB ? 1 : SB); ++t) {                                            \
    const int blk = (n0) + wn * TL::WN + 32 * t;                                                            \
    pb[t] = reinterpret_cast<const uint32_t*>(g.bs) +                                                       \
            (BROW ? lr * 4 + (blk < Rb ? blk / 128 * 128 + blk % 128 / 32 : 0) : min(blk, Rb - 1) / 128 * ((KR + 3) / 4)); \
  }
#define SVDQ_SCALES(S)                                                                                      \
  {                                                                                                         \
    const int grp = min((S), KR - 1) / 4;                                                                   \
    if constexpr (kVecA)                                                                                    \
      memcpy(na, __builtin_assume_aligned(pa[0] + grp * ga, TM * 4), sizeof(na));                           \
    else                                                                                                    \
      _Pragma("unroll") for (int t = 0; t < TM; ++t) na[t] = pa[kVecA ? 0 : t][grp * ga];                   \
    if constexpr (kVecB)                                                                                    \
      memcpy(nb, __builtin_assume_aligned(pb[0] + grp * gb, SB * 4), sizeof(nb));                           \
    else                                                                                                    \
      _Pragma("unroll") for (int t = 0; t < SB; ++t) nb[t] = pb[kVecB ? 0 : t][grp * gb];                   \
  }
#define SVDQ_TAKE_SCALES                                                                                    \
  _Pragma("unroll") for (int t = 0; t < TM; ++t) wa[t] = na[t];                                             \
  _Pragma("unroll") for (int t = 0; t < SB; ++t) wb[t] = nb[t];
  // a stage's first half reads its first step and fetches; the multiplication
  // that belongs to it is the previous stage's second half
#define SVDQ_FIRST_HALF                                                                                     \
  {                                                                                                         \
    SVDQ_FETCH_BEGIN                                                                                        \
    _Pragma("unroll") for (int q = 0; q < TL::kMfma; ++q) {                                                 \
      if (q < TL::kFrags) SVDQ_READ(0, xa, xb, q)                                                           \
      _Pragma("unroll") for (int f = TL::ops_until(q); f < TL::ops_until(q + 1); ++f) {                     \
        if (f < TL::kOpsB) {                                                                                \
          SVDQ_FETCH_B(f)                                                                                   \
        } else {                                                                                            \
          SVDQ_FETCH_A(f - TL::kOpsB)                                                                       \
        }                                                                                                   \
      }                                                                                                     \
    }                                                                                                       \
  }
#define SVDQ_SECOND_HALF(S)                                                                                 \
  {                                                                                                         \
    _Pragma("unroll") for (int t = 0; t < TM; ++t) ca[t] = wa[t] >> (8 * (min((S), KR - 1) & 3));            \
    _Pragma("unroll") for (int t = 0; t < SB; ++t) cb[t] = wb[t] >> (8 * (min((S), KR - 1) & 3));            \
    _Pragma("unroll") for (int f = 0; f < TL::kFrags; ++f) SVDQ_READ(1, ya, yb, f)                          \
    SVDQ_MFMA(xa, xb)                                                                                       \
    spread_second<TL, 0>();                                                                                 \
    SVDQ_FETCHED(b, nb_res)                                                                                 \
    SVDQ_FETCHED(a, na_res)                                                                                 \
    ra_unit = ra_unit >= 3 * TL::kUnit ? ra_unit - 3 * TL::kUnit : ra_unit + 2 * TL::kUnit;                 \
    rb_unit = rb_unit >= 3 * TL::kUnit ? rb_unit - 3 * TL::kUnit : rb_unit + 2 * TL::kUnit;                 \
  }

  f32x16 acc[TN][TM];
  i32x8 xa[TM], xb[TN], ya[TM], yb[TN];
  uint32_t ra_unit = 0, rb_unit = TL::kUnit;   // the units of the stage being read
  int t_cur = (int)blockIdx.x;
  // Where some workgroups have one tile fewer they start about a third of a
  // tile later (a stage takes 1.6 us): then not all tiles' outputs go to
  // memory at the same time, whose 33 MB take longer than a stage (3.4 rounds
  // at 4608 x 12288 outputs over 3072 channels, the whole call 149 us against
  // 161; 2.5 rounds at 4608 x 9216 114 against 121).
  if (ntiles > grid && ntiles % grid != 0 && t_cur >= ntiles % grid)
    for (int i = 0; i < KB / 2; ++i) __builtin_amdgcn_s_sleep(32);   // 2048 cycles
  TileMap tm = map_tile(t_cur, tiles_m, tiles_n, group_m);
  int m0 = __builtin_amdgcn_readfirstlane(tm.tm) * BM, n0 = __builtin_amdgcn_readfirstlane(tm.tn) * BN;
  fa_res = SVDQ_RSRC_A(m0);
  fb_res = SVDQ_RSRC_B(n0);
  bool first = true;
  while (true) {
    // the next tile (none: resources of no bytes, whose transfers are zeros)
    const int t_next = t_cur + grid;
    const bool more = t_next < ntiles;
    const TileMap tn = map_tile(more ? t_next : t_cur, tiles_m, tiles_n, group_m);
    const int m_next = __builtin_amdgcn_readfirstlane(tn.tm) * BM, n_next = __builtin_amdgcn_readfirstlane(tn.tn) * BN;
    __amdgpu_buffer_rsrc_t na_res = SVDQ_RSRC_A(m_next), nb_res = SVDQ_RSRC_B(n_next);
    if (!more) na_res = nb_res = __builtin_amdgcn_make_buffer_rsrc(nullptr, 0, 0, kRsrcWord3);
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int i = 0; i < TM; ++i) acc[j][i] = f32x16{};
    if (first) {
      // A0, B0, A1
      SVDQ_SCALE_ROWS(m0, n0)
      SVDQ_SCALES(0)
      __builtin_amdgcn_sched_barrier(0);
      SVDQ_FETCH_BEGIN
#pragma unroll
      for (int i = 0; i < TL::kOpsA; ++i) { SVDQ_FETCH_A(i) }
#pragma unroll
      for (int i = 0; i < TL::kOpsB; ++i) { SVDQ_FETCH_B(i) }
      SVDQ_FETCHED(a, na_res)
      SVDQ_FETCHED(b, nb_res)
#pragma unroll
      for (int o = 0; o < 2; ++o) ta[o] = 16 * ck[o] >= K - fa_k ? kOutside : va[o];
#pragma unroll
      for (int i = 0; i < TL::kOpsA; ++i) { SVDQ_FETCH_A(i) }
      SVDQ_FETCHED(a, na_res)
      first = false;
      ring_barrier<TL::kOpsA>();   // all but A1
    } else {
      ring_barrier<TL::kOpsA + TL::kStores>();   // A1 and the last tile's stores may be outstanding
    }
    SVDQ_TAKE_SCALES
    SVDQ_SCALES(1)
    __builtin_amdgcn_sched_barrier(0);
    SVDQ_FIRST_HALF
    SVDQ_SECOND_HALF(0)
    for (int s = 1; s < KB; ++s) {
      ring_barrier<TL::kOpsA>();   // all but A of the stage after
      SVDQ_TAKE_SCALES
      SVDQ_SCALES(s + 1)
      __builtin_amdgcn_sched_barrier(0);
      SVDQ_FIRST_HALF
      SVDQ_MFMA(ya, yb)
      spread_first<TL, 0>();
      __builtin_amdgcn_sched_barrier(0);
      SVDQ_SECOND_HALF(s)
    }
    __builtin_amdgcn_sched_barrier(0);
    SVDQ_SCALE_ROWS(m_next, n_next)   // (without a next tile this tile's again)
    SVDQ_SCALES(0)
    // All bias words before the first store: vector memory completes in order,
    // so the wait for a later load is a wait for the stores before it (151 us
    // against 149 at 4608 x 12288 outputs over 3072 channels).
    u32x2 bias[TN][4];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        bias[j][q] = u32x2{0, 0};
        if (g.bias) bias[j][q] = *reinterpret_cast<const u32x2*>(g.bias + min(n0 + wn * TL::WN + 32 * j + 8 * q + 4 * h, Rb - 4));
      }
    __builtin_amdgcn_sched_barrier(0);
    SVDQ_MFMA(ya, yb)

    // A lane holds token m0 + 32 i + lr and channels 32 j + 8 q + 4 h + (0..3);
    // spread_rows leaves it channels at_c .. at_c + 7 of tokens lr % 16 and
    // lr % 16 + 16, so that a store fills 64 contiguous bytes of sixteen rows.
    // Every store is issued by every wave, as the ring's waits count them: the
    // resource drops rows past the operand, and channels past it are sent past
    // its end.
    const int at_c = 8 * h + (lr & 16);
    const int nrec = min(BM, Ra - m0) * Rb * 2;
    const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(g.out + (size_t)m0 * Rb, 0, nrec, kRsrcWord3);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int col = n0 + wn * TL::WN + 32 * j;
      float bv[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const u32x2 w = bias[j][q];
        bv[4 * q] = bf16lo(w.x);
        bv[4 * q + 1] = bf16hi(w.x);
        bv[4 * q + 2] = bf16lo(w.y);
        bv[4 * q + 3] = bf16hi(w.y);
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        uint32_t o[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) o[p] = cvt_bf16x2(acc[j][i][2 * p] + bv[2 * p], acc[j][i][2 * p + 1] + bv[2 * p + 1]);
        spread_rows(o);
        const int off = ((wm * TL::WM + 32 * i + (lr & 15)) * Rb + col + at_c) * 2;
        const u32x4 v0 = u32x4{o[0], o[1], o[2], o[3]}, v1 = u32x4{o[4], o[5], o[6], o[7]};
        const int off0 = col + at_c < Rb ? off : nrec, off1 = col + at_c < Rb ? off + 32 * Rb : nrec;
        if (once) {
          store_16_once(out, v0, off0);
          store_16_once(out, v1, off1);
        } else {
          store_16(out, v0, off0);
          store_16(out, v1, off1);
        }
      }
    }
    if (!more) break;
    t_cur = t_next;
    m0 = m_next;
    n0 = n_next;
  }
  __builtin_amdgcn_s_waitcnt(0);   // the transfers past the end land before the LDS is given up
#undef SVDQ_RSRC_A
#undef SVDQ_RSRC_B
#undef SVDQ_FETCH_BEGIN
#undef SVDQ_FETCH_A
#undef SVDQ_FETCH_B
#undef SVDQ_FETCHED
#undef SVDQ_READ
#undef SVDQ_MFMA
#undef SVDQ_SCALE_ROWS
#undef SVDQ_SCALES
#undef SVDQ_TAKE_SCALES
#undef SVDQ_FIRST_HALF
#undef SVDQ_SECOND_HALF
}

// A few tokens: the weight stream, in one launch. A workgroup of W waves owns
// 16 output channels; the waves take the contracted blocks in turn and add
// their sums in order through LDS. Weights go from memory to the
// MFMA's operand registers directly, kRing blocks of a wave in flight:
// lane (r, c) of v_mfma_f32_16x16x128 holds row r, channels 16 c + (0..15) and
// 64 + 16 c + (0..15) of the block, so each of its two 16-byte loads covers 64
// contiguous bytes of a row. (The order of the channels within a block is free
// as both operands share it.) While its first weights arrive the workgroup
// quantizes all the tokens, into LDS: they are few enough, and come from the
// cache. (With every wave quantizing its own runs' channels the codes took
// as many registers as the weights and their exchange stood between the
// loads: 1.7 times as long for one token, 3072 -> 12288, which takes 8.2 us
// now, its weights alone 7.9 at the rate of a copy.)
// CODES: the tokens are codes already (a norm's) and only copied.
constexpr int kSmallPad = 16;   // bytes between rows of codes in LDS
template <int W, int kRing, bool CODES>
__global__ __launch_bounds__(64 * W) void fp8_small_kernel(Fp8Gemm g) {
  extern __shared__ __align__(16) uint8_t smem[];   // codes [a_rows][round128(K) + kSmallPad], scale bytes [a_rows][KB]
  __shared__ float red[W][4][64];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int K = (int)g.K, M = (int)g.a_rows, KB = (K + 127) / 128;
  const int nb = (KB - wave + W - 1) / W;   // this wave's blocks: wave, wave + W, ...
  const int n0 = blockIdx.x * 16;   // b_rows % 16 == 0
  const uint8_t* wrow = g.b + (int64_t)(n0 + r) * g.ldb;
  const uint8_t* wsc = g.bs + (int64_t)(n0 / 128) * ((KB + 3) / 4 * 4);
  const int ldx = KB * 128 + kSmallPad;
  const uint8_t* arow = smem + min(r, M - 1) * ldx;
  uint8_t* scales = smem + M * ldx;
  const uint8_t* asc = scales + min(r, M - 1) * KB;
  i32x4 wq[kRing][2];
  uint32_t ws[kRing];
  auto load = [&](int u, int i) {
    if (i >= nb) return;
    const int kb = wave + W * i;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k = kb * 128 + 64 * e + 16 * c;
      wq[u][e] = k < K ? *reinterpret_cast<const i32x4*>(wrow + k) : i32x4{0, 0, 0, 0};
    }
    ws[u] = wsc[kb];
  };
#pragma unroll
  for (int u = 0; u < kRing; ++u) load(u, u);
  const int n_out = n0 + 4 * c + 2 * (wave & 1);   // the output channels of a thread of the first two waves
  const uint32_t bias = g.bias ? *reinterpret_cast<const uint32_t*>(g.bias + n_out) : 0u;
  // eight lanes a block, 16 channels a lane
  const int per_row = KB * 8, items = M * per_row;
  for (int i = tid; i < items; i += 64 * W) {
    const int m = i / per_row, k = (i - m * per_row) * 16;
    if constexpr (CODES) {
      *reinterpret_cast<u32x4*>(smem + m * ldx + k) = *reinterpret_cast<const u32x4*>(g.a + (size_t)m * g.lda + k);
      if ((tid & 7) == 0) scales[m * KB + k / 128] = g.as[fp8_scale_index(M, m, k / 128)];
      continue;
    }
    u32x4 v0 = u32x4{0, 0, 0, 0}, v1 = v0;
    if (k < K) {
      const u32x4* p = reinterpret_cast<const u32x4*>(g.x + (size_t)m * K + k);
      v0 = p[0];
      v1 = p[1];
    }
    uint32_t amax = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) amax = amax_bf16x2(amax_bf16x2(amax, v0[q]), v1[q]);
    const int e = e4m3_exponent(max_dpp8(amax));
    const float sc = exp2_int(e);
    *reinterpret_cast<u32x4*>(smem + m * ldx + k) =
        u32x4{e4m3x4(bf16lo(v0[0]), bf16hi(v0[0]), bf16lo(v0[1]), bf16hi(v0[1]), sc),
              e4m3x4(bf16lo(v0[2]), bf16hi(v0[2]), bf16lo(v0[3]), bf16hi(v0[3]), sc),
              e4m3x4(bf16lo(v1[0]), bf16hi(v1[0]), bf16lo(v1[1]), bf16hi(v1[1]), sc),
              e4m3x4(bf16lo(v1[2]), bf16hi(v1[2]), bf16lo(v1[3]), bf16hi(v1[3]), sc)};
    if ((tid & 7) == 0) scales[m * KB + k / 128] = (uint8_t)(e + 127);
  }
  __syncthreads();
  f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < nb; i += kRing) {
#pragma unroll
    for (int u = 0; u < kRing; ++u) {
      if (i + u < nb) {
        const int kb = wave + W * (i + u);
        const uint8_t* p = arow + kb * 128 + 16 * c;
        const i32x4 x0 = *reinterpret_cast<const i32x4*>(p), x1 = *reinterpret_cast<const i32x4*>(p + 64);
        const i32x4 w0 = wq[u][0], w1 = wq[u][1];
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            i32x8{w0[0], w0[1], w0[2], w0[3], w1[0], w1[1], w1[2], w1[3]},
            i32x8{x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]}, acc, 0, 0, 0, (int)ws[u], 0, (int)asc[kb]);
        load(u, i + u + kRing);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) red[wave][e][lane] = acc[e];
  __syncthreads();
  // a thread adds the waves' sums of two consecutive channels: value e of
  // lane (r, c) is token r, channel n0 + 4 c + e
  if (tid < 128) {
    const int pe = tid >> 6;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      s0 += red[w][2 * pe][lane];
      s1 += red[w][2 * pe + 1][lane];
    }
    if (r < M)
      *reinterpret_cast<uint32_t*>(g.out + (size_t)r * g.b_rows + n_out) = cvt_bf16x2(s0 + bf16lo(bias), s1 + bf16hi(bias));
  }
}

// Few tiles (fp8_deep): 64 x 64 outputs a workgroup, and where those do not
// fill the CUs a tile's contracted blocks in several runs (`chunk` blocks, a
// multiple of four), whose fp32 sums the workgroup that comes last to the
// tile's ticket adds in order. There is
// little work a CU, so a stage's time is the wait for its transfers: LDS is a
// ring of D whole stages with all but one in flight. Per stage: the wait for
// the next one, the barrier, the transfers into the slot of the stage whose
// fragments have been read, the next stage's fragment reads, and this one's
// multiplications behind them. Four waves hold 32 x 32 each. Scale words (four
// stages' bytes) are read four stages ahead.
//
// With D = 5 the ring is half of a CU's LDS and the ticket's word goes past it,
// so a CU has one workgroup (these launches have no more product tiles than
// CUs; workgroups of the bias gradient behind them wait for a CU that is
// done), with D = 3 three. Measured: a stage takes 0.28 us without its
// transfers (the LDS reads), 0.3 to 0.45 with them (the misses of the L2s).
// Tiles of 64 x 128 and 128 x 128 took as long or longer wherever they are
// fewer than the CUs (12288 channels, 64 tokens, 3072 outputs: 1% and 7%
// longer; 2064, 1003 and 1552: 2% less and 12% longer).
constexpr int kDeepStage = 2 * 64 * 128, kDeepOps = 4;   // bytes of a stage; transfers per wave and stage
template <int D, bool BROW>
__global__ __launch_bounds__(256) void fp8_deep_kernel(Fp8Gemm g, int tiles_m, int tiles_n, int chunk, int runs, Fp8BiasGrad bias) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int all = tiles_m * tiles_n * runs;
  if ((int)blockIdx.x >= all) {
    bias_grad_32<256>(bias.sums, bias.blocks, bias.N, ((int)blockIdx.x - all) * 32, bias.db, reinterpret_cast<float*>(smem));
    return;
  }
  __shared__ int ticket_last;
  static_assert(D - 2 <= 4, "scale words are four stages ahead of their use, the transfers no more");
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, lr = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int Ra = (int)g.a_rows, Rb = g.b_rows, K = (int)g.K, KR = (K + 127) / 128;
  const int lda = (int)g.lda, ldb = (int)g.ldb;
  // an XCD (workgroups 8 apart) takes consecutive tiles of one run of
  // channels, those of the same weights next to each other
  const int xcd = (int)blockIdx.x & 7;
  const int t = xcd * (all >> 3) + min(xcd, all & 7) + ((int)blockIdx.x >> 3);
  const int m0 = t % tiles_m * 64, tn_ = t / tiles_m, n0 = tn_ % tiles_n * 64, run = tn_ / tiles_n;
  const int s0 = run * chunk, s1 = min(KR, s0 + chunk);

  // Transfers: the first two waves' are A's row octets, the others' B's; rows
  // past the operand read as zeros.
  const __amdgpu_buffer_rsrc_t ra =
      __builtin_amdgcn_make_buffer_rsrc((void*)(g.a + (size_t)m0 * lda), 0, min(64, Ra - m0) * lda, kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rb =
      __builtin_amdgcn_make_buffer_rsrc((void*)(g.b + (size_t)n0 * ldb), 0, min(64, Rb - n0) * ldb, kRsrcWord3);
  const int ck0 = (lane & 7) ^ (lane >> 4);   // the lane's chunk of the even octets; of the odd ones ^ 4
  auto fetch = [&](int s, int slot) {
    const int k = s * 128;
    uint8_t* dst = smem + slot * kDeepStage + wave * kDeepOps * 1024;
    const __amdgpu_buffer_rsrc_t res = wave < 2 ? ra : rb;
    const int ld = wave < 2 ? lda : ldb;
#pragma unroll
    for (int i = 0; i < kDeepOps; ++i) {
      const int ck = (i & 1) ? ck0 ^ 4 : ck0;
      lds_transfer(res, dst + i * 1024, s < s1 && 16 * ck < K - k ? (uint32_t)((lane >> 3) * ld + 16 * ck) : kOutside,
                   ((wave & 1) * kDeepOps + i) * 8 * ld + k);
    }
  };
  // LDS offsets in a stage of this lane's fragment chunks: rows (+ 32 t),
  // chunk 4 step + 2 h + e at place chunk ^ (row / 2 % 8)
  const int sw = (lr >> 1) & 7;
  uint32_t at[2][2];
#pragma unroll
  for (int st = 0; st < 2; ++st)
#pragma unroll
    for (int e = 0; e < 2; ++e) at[st][e] = (uint32_t)(lr * 128 + ((4 * st + 2 * h + e) ^ sw) * 16);
  const uint32_t base_a = wm * 4096, base_b = 8192 + wn * 4096;
  // scale words of this lane's rows (rows past the operand read its first words)
  const int row0 = m0 + wm * 32, col0 = n0 + wn * 32;
  const size_t ga = (size_t)round128(Ra), gb = BROW ? (size_t)round128(Rb) : 1;
  const uint32_t* pa = reinterpret_cast<const uint32_t*>(g.as) + lr * 4 + (row0 < Ra ? row0 / 128 * 128 + row0 % 128 / 32 : 0);
  const uint32_t* pb = reinterpret_cast<const uint32_t*>(g.bs) +
                       (BROW ? lr * 4 + (col0 < Rb ? col0 / 128 * 128 + col0 % 128 / 32 : 0) : n0 / 128 * ((KR + 3) / 4));
  uint32_t na, nb;
  auto scales = [&](int grp) {
    grp = min(grp, (KR - 1) / 4);
    na = pa[grp * ga];
    nb = pb[grp * gb];
  };
  f32x16 acc = f32x16{};
  i32x8 fa[2][2], fb[2][2];   // a stage's fragments: set, step
  auto read = [&](int set, int slot) {
    const uint8_t* stage = smem + slot * kDeepStage;
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const i32x4 b0 = *reinterpret_cast<const i32x4*>(stage + base_b + at[st][0]);
      const i32x4 b1 = *reinterpret_cast<const i32x4*>(stage + base_b + at[st][1]);
      const i32x4 a0 = *reinterpret_cast<const i32x4*>(stage + base_a + at[st][0]);
      const i32x4 a1 = *reinterpret_cast<const i32x4*>(stage + base_a + at[st][1]);
      fb[set][st] = i32x8{b0[0], b0[1], b0[2], b0[3], b1[0], b1[1], b1[2], b1[3]};
      fa[set][st] = i32x8{a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
    }
  };
  scales(s0 / 4);
  u32x2 bw[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    bw[q] = u32x2{0, 0};
    if (g.bias) bw[q] = *reinterpret_cast<const u32x2*>(g.bias + min(col0 + 8 * q + 4 * h, Rb - 4));
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int u = 0; u < D - 1; ++u) fetch(s0 + u, u);
  ring_barrier<(D - 2) * kDeepOps>();   // the first stage
  fetch(s0 + D - 1, D - 1);
  __builtin_amdgcn_sched_barrier(0);
  read(0, 0);
  int slot = 0;
  for (int s = s0; s < s1; s += 4) {
    const uint32_t wa = na, wb = nb;
    scales(s / 4 + 1);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (s + u < s1) {
        // the next stage has arrived, and every wave has read this one
        ring_barrier<(D - 2) * kDeepOps>();
        fetch(s + u + D, slot);
        __builtin_amdgcn_sched_barrier(0);
        slot = slot + 1 == D ? 0 : slot + 1;
        read((u + 1) & 1, slot);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int st = 0; st < 2; ++st)
          acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[u & 1][st], fa[u & 1][st], acc, 0, 0, 0,
                                                                (int)(wb >> (8 * u)), 0, (int)(wa >> (8 * u)));
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(0);   // the transfers past the end land before the LDS is given up

  if (runs > 1) {
    // The sums go through the device's coherence point and not the XCD's L2
    // (relaxed atomics of agent scope, of 8 bytes), so that no cache has to be
    // written back or invalidated: with an agent-scope release and acquire the
    // call takes 25.8 us for 64 tokens, 12288 -> 3072, with the acquire alone
    // 20.7, this way 15.7; a second kernel that adds the runs took as long as
    // this and a launch (2.8 us of host time) more. Each store has reached that point before the
    // ticket is taken (the wait), and no XCD can hold an older copy: a kernel
    // starts with nothing of this memory in its caches, a run's sums fill whole
    // lines (the workspace is used from a multiple of 256 bytes on), and only
    // the tile's last workgroup reads them.
    const int tile = t % (tiles_m * tiles_n);
    auto part = [&](int r, int q) {
      return reinterpret_cast<uint64_t*>(g.part) + ((size_t)((tile * runs + r) * 4 + wave) * 8 + q) * 64 + lane;
    };
#pragma unroll
    for (int q = 0; q < 8; ++q)
      __hip_atomic_store(part(run, q), (uint64_t)__float_as_uint(acc[2 * q + 1]) << 32 | __float_as_uint(acc[2 * q]),
                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __builtin_amdgcn_s_waitcnt(0);   // every wave's sums have landed ...
    __syncthreads();                  // ... before the ticket is taken
    if (tid == 0)
      ticket_last = __hip_atomic_fetch_add(g.tickets + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == (uint32_t)runs;
    __syncthreads();
    if (!ticket_last) return;
    acc = f32x16{};
#pragma unroll 4
    for (int r = 0; r < runs; ++r) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint64_t v = __hip_atomic_load(part(r, q), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        acc[2 * q] += __uint_as_float((uint32_t)v);
        acc[2 * q + 1] += __uint_as_float((uint32_t)(v >> 32));
      }
    }
  }
  // a lane holds token row0 + lr and channels col0 + 8 q + 4 h + (0..3)
  uint32_t o[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    o[2 * q] = cvt_bf16x2(acc[4 * q] + bf16lo(bw[q].x), acc[4 * q + 1] + bf16hi(bw[q].x));
    o[2 * q + 1] = cvt_bf16x2(acc[4 * q + 2] + bf16lo(bw[q].y), acc[4 * q + 3] + bf16hi(bw[q].y));
  }
  spread_rows(o);
  const int row = row0 + (lr & 15), c = col0 + 8 * h + (lr & 16);
  if (c >= Rb) return;
  uint16_t* p = g.out + (size_t)row * Rb + c;
  if (row < Ra) *reinterpret_cast<u32x4*>(p) = u32x4{o[0], o[1], o[2], o[3]};
  if (row + 16 < Ra) *reinterpret_cast<u32x4*>(p + (size_t)16 * Rb) = u32x4{o[4], o[5], o[6], o[7]};
}

typedef Tile<256, 256, 2, 2> TileL;
typedef Tile<256, 192, 2, 2> TileW;
typedef Tile<128, 128, 2, 2> TileM;
// The 32 workgroups of an XCD take 4 tile-rows x 8 tile-columns (8 x 4 take
// 4% longer at 8192^3, 16 x 2 8%).
constexpr int kGroupM = 4;

template <class TL, bool BROW>
hipError_t launch_tile(const Fp8Gemm& g, int num_cus, hipStream_t st) {
  const int tm = (int)((g.a_rows + TL::BM - 1) / TL::BM), tn = (g.b_rows + TL::BN - 1) / TL::BN;
  const int resident = num_cus * (int)(160 * 1024 / TL::kLds);   // workgroups that the LDS holds
  hipLaunchKernelGGL((fp8_gemm_kernel<TL::BM, TL::BN, TL::WGM, TL::WGN, BROW>), dim3((unsigned)std::min(tm * tn, resident)),
                     dim3(64 * TL::NW), TL::kLds, st, g, tm, tn, kGroupM);
  return hipGetLastError();
}
template <class TL, bool BROW>
hipError_t prepare_tile() {
  return hipFuncSetAttribute((const void*)fp8_gemm_kernel<TL::BM, TL::BN, TL::WGM, TL::WGN, BROW>,
                             hipFuncAttributeMaxDynamicSharedMemorySize, TL::kLds);
}

}  // namespace

hipError_t prepare_fp8() {
  for (hipError_t e : {prepare_tile<TileW, false>(), prepare_tile<TileW, true>(), prepare_tile<TileL, false>(), prepare_tile<TileL, true>(), prepare_tile<TileM, false>(),
                       prepare_tile<TileM, true>()})
    if (e != hipSuccess) return e;
  for (const void* f : {(const void*)fp8_deep_kernel<5, false>, (const void*)fp8_deep_kernel<5, true>,
                        (const void*)fp8_small_kernel<16, 2, false>, (const void*)fp8_small_kernel<16, 2, true>}) {
    const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, 5 * kDeepStage);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_fp8_gemm_small(const Fp8Gemm& g, int num_cus, hipStream_t st) {
  const int KB = (int)((g.K + 127) / 128), grid = g.b_rows / 16;
  const size_t lds = (size_t)g.a_rows * (KB * 128 + kSmallPad + KB);
  // Where a wave of eight has more than four blocks and no CU has two
  // workgroups, sixteen share them (one token, 12288 -> 3072: 9.4 us against
  // 9.9, 8192 -> 4096 7.8 against 8.8; with 24 blocks, 3072 -> 3072, 4.2 us
  // either way, and with more workgroups, 3072 -> 12288, eight take 7.9 us and
  // sixteen 8.3).
  const dim3 n((unsigned)grid);
  if (grid <= num_cus && KB > 32) {
    if (g.x) hipLaunchKernelGGL((fp8_small_kernel<16, 2, false>), n, dim3(1024), lds, st, g);
    else hipLaunchKernelGGL((fp8_small_kernel<16, 2, true>), n, dim3(1024), lds, st, g);
  } else {
    if (g.x) hipLaunchKernelGGL((fp8_small_kernel<8, 3, false>), n, dim3(512), lds, st, g);
    else hipLaunchKernelGGL((fp8_small_kernel<8, 3, true>), n, dim3(512), lds, st, g);
  }
  return hipGetLastError();
}

namespace {
template <bool BROW>
hipError_t launch_deep(const Fp8Gemm& g, const Fp8Deep& p, const Fp8BiasGrad* bias, hipStream_t st) {
  const int tm = (int)((g.a_rows + 63) / 64), tn = (g.b_rows + 63) / 64, all = tm * tn * p.runs;
  const Fp8BiasGrad b = bias ? *bias : Fp8BiasGrad{nullptr, 0, 0, nullptr};
  const dim3 grid((unsigned)(all + (b.N + 31) / 32));
  if (all <= kFp8Cus)
    hipLaunchKernelGGL((fp8_deep_kernel<5, BROW>), grid, dim3(256), 5 * kDeepStage, st, g, tm, tn, p.chunk, p.runs, b);
  else
    hipLaunchKernelGGL((fp8_deep_kernel<3, BROW>), grid, dim3(256), 3 * kDeepStage, st, g, tm, tn, p.chunk, p.runs, b);
  return hipGetLastError();
}
}  // namespace

// (a launch of its own takes 2 us more: 777 tokens, 1552 -> 2064, 28.1 us
// against 30.1, 64 tokens, 3072 -> 3072, 24.6 against 26.7)
bool fp8_gemm_takes_bias(const Fp8Gemm& g) { return fp8_deep(g.a_rows, g.b_rows, g.K).runs > 0; }

hipError_t launch_fp8_gemm(const Fp8Gemm& g, int num_cus, hipStream_t st, const Fp8BiasGrad* bias) {
  const Fp8Deep p = fp8_deep(g.a_rows, g.b_rows, g.K);
  if (p.runs > 0) return g.b_row_scales ? launch_deep<true>(g, p, bias, st) : launch_deep<false>(g, p, bias, st);
  // The tile of least cost, a cost being the rounds of tiles over the CUs times
  // a round's time relative to TileL's, as measured on the products of K from
  // 2048 to 12288: TileW 0.85 (it fills the CUs where TileL's rounds do not:
  // the weight gradient of 12288 x 3072 over 4608 tokens 175 us, TileL 188,
  // TileM 203), TileM 0.62 with two tiles a CU and 0.5 with one (640 x 3072
  // outputs over 12288 channels 58 us, TileL 110, TileW 97; 4608 x 3072 over
  // 12288 207 us, TileL 165, TileW 243).
  auto tiles = [&](int bm, int bn) { return ((g.a_rows + bm - 1) / bm) * ((g.b_rows + bn - 1) / bn); };
  auto rounds = [&](int64_t n, int64_t at_once) { return (float)((n + at_once - 1) / at_once); };
  const int64_t nm = tiles(TileM::BM, TileM::BN);
  const float cost_l = rounds(tiles(TileL::BM, TileL::BN), num_cus);
  const float cost_w = 0.85f * rounds(tiles(TileW::BM, TileW::BN), num_cus);
  const float cost_m = nm <= num_cus ? 0.5f : 0.62f * rounds(nm, 2 * num_cus);
  if (cost_m <= cost_l && cost_m <= cost_w)
    return g.b_row_scales ? launch_tile<TileM, true>(g, num_cus, st) : launch_tile<TileM, false>(g, num_cus, st);
  if (cost_w < cost_l)
    return g.b_row_scales ? launch_tile<TileW, true>(g, num_cus, st) : launch_tile<TileW, false>(g, num_cus, st);
  return g.b_row_scales ? launch_tile<TileL, true>(g, num_cus, st) : launch_tile<TileL, false>(g, num_cus, st);
}

}  // namespace svdq
