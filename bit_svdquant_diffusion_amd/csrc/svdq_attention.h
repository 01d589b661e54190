// Device-side pieces that the attention kernels share: tiles of 64 rows (keys,
// or queries) of a head in LDS, the fragments read from them, and the products.
//
// A tile's rows are 64 or 128 elements of two bytes, of which the products take
// DP (32, 64, 96 or 128: the head's D and zeros behind it). They come by
// `buffer_load_dwordx4 ... lds` transfers of 1 KiB, whose lanes fetch their
// 16-byte chunks permuted: chunk c of row r lies at place c ^ place(r). Both kinds of fragment then meet every LDS bank
// evenly: 32 rows at one chunk (an operand whose contraction runs along the
// head), and, by the transposing read ds_read_b64_tr_b16, columns of 8 rows at
// four chunks (an operand whose contraction runs along the rows).
//
// MFMA 32x32x16 contracts 16 elements in two halves of the wave, eight a lane.
// The result of a 32 x 32 product has, in lane l, column l % 32 and the rows
// 8 (i / 4) + 4 (l / 32) + i % 4, i = 0..15. Where such a result is the next
// product's operand B, contracted along those rows, its registers 8 t .. 8 t
// + 7 stand for the rows 16 t + 4 h + (0..3) and 16 t + 8 + 4 h + (0..3): they
// are used as they are, and operand A takes its columns in that order, too.
#pragma once
#include "svdq_internal.h"
#include "svdq_types.h"

namespace svdq {

constexpr int kAttnRows = kAttnTile;   // of a tile

struct AttnUnits {};   // in the place of AttnParts where a workgroup has a unit
template <bool PARTS>
struct AttnDealOf {
  typedef AttnUnits type;
};
template <>
struct AttnDealOf<true> {
  typedef AttnParts type;
};
template <bool PARTS>
using AttnDeal = typename AttnDealOf<PARTS>::type;
__device__ __forceinline__ AttnPiece piece_of(const AttnArgs& a, const AttnUnits&, int place) {
  return attn_piece(a.cost, a.plan, place);
}
__device__ __forceinline__ AttnPiece piece_of(const AttnArgs& a, const AttnParts& deal, int place) {
  return attn_piece(a.cost, a.plan, deal.at[place]);
}

// Units are cut into parts where there are fewer than CUs, and then workgroups
// have eight waves.
template <int W, int KW>
constexpr bool kAttnCut = W * KW == 8;
inline hipError_t attn_shared_memory(const void* kernel, int bytes) {
  return hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

template <typename T>
__device__ __forceinline__ f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (__is_same(T, Bf16))
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// two floats rounded to a packed pair
template <typename T>
__device__ __forceinline__ uint32_t cvt_x2(float lo, float hi) {
  if constexpr (__is_same(T, Bf16))
    return cvt_bf16x2(lo, hi);
  else
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, f16x2));
}

// registers 8 t .. 8 t + 7 of a result as an operand B
template <typename T>
__device__ __forceinline__ u32x4 as_operand(const f32x16& v, int t) {
  return u32x4{cvt_x2<T>(v[8 * t], v[8 * t + 1]), cvt_x2<T>(v[8 * t + 2], v[8 * t + 3]), cvt_x2<T>(v[8 * t + 4], v[8 * t + 5]),
               cvt_x2<T>(v[8 * t + 6], v[8 * t + 7])};
}

// what that rounding took off, rounded itself: with both parts a product has
// 2^-17 (bf16) or 2^-22 (fp16) of its operand's rounding left
template <typename T>
__device__ __forceinline__ u32x4 as_operand_rest(const f32x16& v, u32x4 whole, int t) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    if constexpr (__is_same(T, Bf16)) {
      lo = bf16lo(whole[i]);
      hi = bf16hi(whole[i]);
    } else {
      const uint32_t pair = whole[i];   // (a vector's element taken as another type as it stands is its first)
      const f16x2 x = __builtin_bit_cast(f16x2, pair);
      lo = (float)x[0];
      hi = (float)x[1];
    }
    o[i] = cvt_x2<T>(v[8 * t + 2 * i] - lo, v[8 * t + 2 * i + 1] - hi);
  }
  return o;
}
template <typename T, int NP>
__device__ __forceinline__ void as_operands(const f32x16& v, int t, u32x4 (&o)[NP]) {
  o[0] = as_operand<T>(v, t);
  if constexpr (NP == 2) o[1] = as_operand_rest<T>(v, o[0], t);
}

// the other half wave's value of the same column
__device__ __forceinline__ float max_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// 16 (4) bytes a lane from `r` + voff, zeros past r's end, to 1 KiB (256 bytes)
// of LDS. In assembly, because the compiler lets every transposing LDS read
// wait for all transfers that it knows of, those of the next tile among them:
// here tile_barrier alone waits. (No register is written, and the compiler's
// own counted waits only become stricter by what it does not count.)
__device__ __forceinline__ void lds_transfer_16(u32x4 r, const void* dst, uint32_t voff) {
  uint32_t m0;
  asm volatile(
      "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %1, 0 offen lds\n\ts_mov_b32 m0, %0"
      : "=&s"(m0)
      : "s"(r), "v"(voff), "s"((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)dst)
      : "memory");
}
__device__ __forceinline__ void lds_transfer_4(u32x4 r, const void* dst, uint32_t voff) {
  uint32_t m0;
  asm volatile(
      "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dword %2, %1, 0 offen lds\n\ts_mov_b32 m0, %0"
      : "=&s"(m0)
      : "s"(r), "v"(voff), "s"((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)dst)
      : "memory");
}
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 read_tr(const uint8_t* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}
constexpr uint32_t kPastEnd = 0x7ffffff0u;   // a lane offset past the end of every resource: loads zeros
// a buffer resource of raw bytes
__device__ __forceinline__ u32x4 rows_resource(const void* base, int bytes) {
  const uint64_t at = (uint64_t)base;
  return u32x4{(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, (uint32_t)bytes, 0x00020000u};
}

// all transfers have arrived and all LDS reads returned, then the workgroup's
// barrier; nothing moves across
__device__ __forceinline__ void tile_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

// The order of what stands before in its block, for the scheduler: AHEAD LDS
// reads, then the products with STEP further reads after each while there are
// any. (Left to itself the compiler may read a fragment right before its
// product and wait for it: the forward at 4608 tokens 270 us against 244.)
template <int PRODUCTS, int READS, int STEP, int AHEAD, int I = 0>
__device__ __forceinline__ void sched_products() {
  if constexpr (I == 0) __builtin_amdgcn_sched_group_barrier(0x100, AHEAD < READS ? AHEAD : READS, 0);
  if constexpr (I < PRODUCTS) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (AHEAD + (I + 1) * STEP <= READS) __builtin_amdgcn_sched_group_barrier(0x100, STEP, 0);
    sched_products<PRODUCTS, READS, STEP, AHEAD, I + 1>();
  }
}

template <int DP>
struct AttnTile {
  static constexpr int kRow = DP > 64 ? 128 : 64, kRowBytes = kRow * 2, kChunks = kRow / 8, kBytes = kAttnRows * kRowBytes;
  static constexpr int kTransfers = kBytes / 1024, kRowsEach = 64 / kChunks;
  static constexpr int kSteps = DP / 16, kBlocks = DP / 32;

  static __device__ __forceinline__ int place(int row) {
    return kRow == 128 ? ((row & 3) << 2) | ((row >> 2) & 3) : (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
  }
  // transfer j, this lane: its row of the tile and the chunk of the head
  static __device__ __forceinline__ int row_of(int j, int lane) { return j * kRowsEach + lane / kChunks; }
  static __device__ __forceinline__ int chunk_of(int j, int lane) { return (lane % kChunks) ^ place(row_of(j, lane)); }

  // this lane's places in a tile: `straight` for operand A of rows 32 b + l %
  // 32 and head elements 16 step + 8 h + (0..7); `turned[u]` for the head
  // elements 32 blk + l % 32 of rows 16 t + 8 u + 4 h + (0..3)
  struct Lane {
    uint32_t straight, turned[2];
    __device__ __forceinline__ explicit Lane(int lane) {
      const int h = lane >> 5, lr = lane & 31, i = lane & 15;
      straight = lr * kRowBytes + ((h ^ place(lr)) << 4);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = 8 * u + 4 * h + (i >> 2), chunk = 2 * ((lane >> 4) & 1) + ((i >> 1) & 1);
        turned[u] = row * kRowBytes + ((chunk ^ place(row)) << 4) + (i & 1) * 8;
      }
    }
  };
  // operand A from rows 32 b .. of the tile, contracted along the head
  static __device__ __forceinline__ u32x4 straight(const uint8_t* tile, const Lane& at, int b, int step) {
    return *reinterpret_cast<const u32x4*>(tile + (at.straight ^ (uint32_t)(step << 5)) + b * 32 * kRowBytes);
  }
  // operand A of head elements 32 blk .., contracted along rows 16 t .. of the tile
  static __device__ __forceinline__ u32x4 turned(const uint8_t* tile, const Lane& at, int t, int blk) {
    const u32x2 a = read_tr(tile + (at.turned[0] ^ (uint32_t)(blk << 6)) + t * 16 * kRowBytes);
    const u32x2 b = read_tr(tile + (at.turned[1] ^ (uint32_t)(blk << 6)) + t * 16 * kRowBytes);
    return u32x4{a[0], a[1], b[0], b[1]};
  }
};

// A result of head elements (rows) by 32 columns, block blk, as 16-byte chunks
// of the columns' rows in memory: o[p] is chunk 4 blk + 2 p + h of column l % 32
template <typename T>
__device__ __forceinline__ void head_chunks(const f32x16& v, float factor, u32x4 (&o)[2]) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = cvt_x2<T>(v[8 * p + 2 * k] * factor, v[8 * p + 2 * k + 1] * factor);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const auto r = __builtin_amdgcn_permlane32_swap(w[k], w[2 + k], false, false);
      w[k] = r[0];
      w[2 + k] = r[1];
    }
    o[p] = u32x4{w[0], w[1], w[2], w[3]};
  }
}

}  // namespace svdq
