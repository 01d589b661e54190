// Attention, forward: of each query row, over the keys j that it sees,
//
//   s_j = scale q . k_j,  m = max s_j,  o = sum exp(s_j - m) v_j / sum exp(s_j - m),
//   lse = m + log sum exp(s_j - m).
//
// One pass over the keys with the running maximum and sum: a workgroup holds
// 32 NB query rows a wave, K and V pass by in tiles of 64 keys. The product is
// taken as S^T = K Q^T, so that a lane's registers hold one query's scores:
// the maximum and the sum are the lane's own but for one exchange between the
// half waves, and exp(S^T) is in the right registers to be the operand B of
// O^T = V^T P^T. The heads that share a key head are rows of the same tiles
// (row r is query r / G, head r % G), so K and V are read once for them.
#include <algorithm>

#include "svdq_attention.h"
#include "svdq_internal.h"
#include "svdq_layout.h"

namespace svdq {

namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// W waves of NB blocks of 32 query rows; DP the padded head. Two waves a SIMD
// (up to 256 registers), so that one's products run under the other's
// exponentials: 4608 tokens, 24 heads of 128 with a mask 252 us (1.03
// PFLOP/s), with one wave a SIMD 411, with one of two blocks 355, with
// workgroups of four waves instead of eight 270.
template <typename T, int DP, int W, int NB>
__global__ __launch_bounds__(64 * W, 2) void attn_fwd_kernel(AttnArgs a) {
  typedef AttnTile<DP> TL;
  constexpr int NT = TL::kTransfers / W;   // transfers of a wave for one tile
  __shared__ __align__(1024) uint8_t smem[2][2][TL::kBytes];
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, lr = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const AttnPlace at = attn_place(a, blockIdx.x, true);
  const int G = a.G, R = a.Lq * G, D = a.D;
  const int b = at.hb / a.Hk, hk = at.hb % a.Hk;
  const T* qp = static_cast<const T*>(a.q.p) + b * a.q.batch + (int64_t)hk * G * a.q.head;
  const T* kp = static_cast<const T*>(a.k.p) + b * a.k.batch + hk * a.k.head;
  const T* vp = static_cast<const T*>(a.v.p) + b * a.v.batch + hk * a.v.head;
  const uint8_t* mask = a.mask ? a.mask + b * a.mask_batch : nullptr;

  // this lane's rows and the last keys that they see
  const int r0 = at.block * (32 * NB * W) + wave * (32 * NB);
  u32x4 qf[NB][TL::kSteps];
  int last[NB];   // of a row without keys (and past the last row) below 0
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int r = r0 + 32 * n + lr, i = r / G;
    const T* row = qp + (int64_t)i * a.q.token + (int64_t)(r - i * G) * a.q.head;
    last[n] = r >= R ? -1 : a.causal ? min(i + a.Lk - a.Lq, a.Lk - 1) : a.Lk - 1;
#pragma unroll
    for (int s = 0; s < TL::kSteps; ++s) {
      const int d = 16 * s + 8 * h;
      qf[n][s] = r < R && d < D ? *reinterpret_cast<const u32x4*>(row + d) : u32x4{0, 0, 0, 0};
    }
  }
  // the keys of this workgroup: those of its last row, in its part of the split
  const int r_end = min(R, (at.block + 1) * (32 * NB * W));
  int k_end = a.causal ? min(a.Lk, (r_end - 1) / G + a.Lk - a.Lq + 1) : a.Lk;
  k_end = min(k_end, (at.split + 1) * a.split_keys);
  const int k_begin = at.split * a.split_keys;
  const int tiles = k_end > k_begin ? (k_end - k_begin + kAttnRows - 1) / kAttnRows : 0;
  // what every and what any row of this wave sees
  const int w_first = a.causal ? r0 / G + a.Lk - a.Lq : a.Lk - 1;
  const int w_last = r0 >= R ? -1 : a.causal ? (min(r0 + 32 * NB, R) - 1) / G + a.Lk - a.Lq : a.Lk - 1;

  // transfers
  uint32_t vk[NT], vv[NT];
  int row_of[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int j = wave * NT + n, c = TL::chunk_of(j, lane);
    row_of[n] = TL::row_of(j, lane);
    vk[n] = c * 8 < D ? (uint32_t)((row_of[n] * a.k.token + c * 8) * 2) : kPastEnd;
    vv[n] = c * 8 < D ? (uint32_t)((row_of[n] * a.v.token + c * 8) * 2) : kPastEnd;
  }
  auto fetch = [&](int k0, int stage, uint64_t keep) {
    const int rows = min(kAttnRows, a.Lk - k0);
    const auto rk = rows_resource(kp + k0 * a.k.token, (int)((rows - 1) * a.k.token + D) * 2);
    const auto rv = rows_resource(vp + k0 * a.v.token, (int)((rows - 1) * a.v.token + D) * 2);
    uint8_t *tk = smem[stage][0] + wave * NT * 1024, *tv = smem[stage][1] + wave * NT * 1024;
    // (a key that the mask drops is not read: whatever stands there, it is zero)
    if (keep == ~0ull) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        lds_transfer_16(rk, tk + n * 1024, vk[n]);
        lds_transfer_16(rv, tv + n * 1024, vv[n]);
      }
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const bool in = keep >> row_of[n] & 1;
        lds_transfer_16(rk, tk + n * 1024, in ? vk[n] : kPastEnd);
        lds_transfer_16(rv, tv + n * 1024, in ? vv[n] : kPastEnd);
      }
    }
  };
  // the mask's byte of key `lane` of a tile
  auto mask_byte = [&](int k0) -> int {
    const int k = k0 + lane;
    return k < a.Lk ? (mask ? (int)mask[k] : 1) : 0;
  };

  f32x16 o[TL::kBlocks][NB];
  float m[NB], l[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    m[n] = -__builtin_inff();
    l[n] = 0.f;
#pragma unroll
    for (int i = 0; i < TL::kBlocks; ++i) o[i][n] = f32x16{};
  }
  const typename TL::Lane pl(lane);
  uint64_t keep = 0, next_keep = 0;
  int next_byte = 0;
  if (tiles > 0) {
    next_keep = __ballot(mask_byte(k_begin) != 0);
    fetch(k_begin, 0, next_keep);
    next_byte = mask_byte(k_begin + kAttnRows);
  }
  for (int t = 0, k0 = k_begin; t < tiles; ++t, k0 += kAttnRows) {
    keep = next_keep;
    tile_barrier();
    if (t + 1 < tiles) {
      next_keep = __ballot(next_byte != 0);
      fetch(k0 + kAttnRows, (t + 1) & 1, next_keep);
      next_byte = mask_byte(k0 + 2 * kAttnRows);
    }
    if (k0 > w_last || keep == 0) continue;   // nothing that this wave's rows see
    const uint8_t *tk = smem[t & 1][0], *tv = smem[t & 1][1];
    f32x16 s[2][NB];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int n = 0; n < NB; ++n) s[kb][n] = f32x16{};
#pragma unroll
    for (int st = 0; st < TL::kSteps; ++st)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const u32x4 kf = TL::straight(tk, pl, kb, st);
#pragma unroll
        for (int n = 0; n < NB; ++n) s[kb][n] = mma<T>(kf, qf[n][st], s[kb][n]);
      }
    if (keep != ~0ull || k0 + kAttnRows - 1 > w_first) {
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const int lim = last[n] - k0 - 4 * h;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          const uint32_t bits = (uint32_t)(keep >> (32 * kb)) >> (4 * h);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int c = 8 * (i / 4) + i % 4;
            s[kb][n][i] = (bits >> c & 1) && 32 * kb + c <= lim ? s[kb][n][i] : -__builtin_inff();
          }
        }
      }
    }
    u32x4 p[4][NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      float top = s[0][n][0];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, s[kb][n][i]);
      top = max_halves(top) * a.scale_log2;
      // The maximum that is subtracted follows the true one when that is more
      // than 8 (in base 2) above it: up to there the probabilities stay below
      // 2^8, which neither the sums nor either type's rounding minds, and most
      // tiles leave the accumulators as they are.
      if (__any(top > m[n] + 8.f)) {
        const float mn = __builtin_fmaxf(m[n], top);
        const float f = m[n] == mn ? 1.f : __builtin_amdgcn_exp2f(m[n] - mn);
        m[n] = mn;
        l[n] *= f;
#pragma unroll
        for (int i = 0; i < TL::kBlocks; ++i) o[i][n] *= f;
      }
      const float base = m[n] == -__builtin_inff() ? 0.f : m[n];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[kb][n][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][n][i], a.scale_log2, -base));
          l[n] += s[kb][n][i];
        }
        p[2 * kb][n] = as_operand<T>(s[kb][n], 0);
        p[2 * kb + 1][n] = as_operand<T>(s[kb][n], 1);
      }
    }
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
#pragma unroll
      for (int i = 0; i < TL::kBlocks; ++i) {
        const u32x4 vf = TL::turned(tv, pl, kt, i);
#pragma unroll
        for (int n = 0; n < NB; ++n) o[i][n] = mma<T>(vf, p[kt][n], o[i][n]);
      }
  }
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int r = r0 + 32 * n + lr, i = r / G, g = r - i * G;
    const float sum = sum_halves(l[n]);
    const float f = sum == 0.f ? 0.f : 1.f / sum, lse2 = m[n] + __builtin_log2f(sum);   // (no key: -inf)
    if (r >= R) continue;
    if (a.splits > 1) {
      const int64_t row = (at.split * (int64_t)a.B * a.Hk + at.hb) * R + r;
      if (h == 0) a.part_lse[row] = lse2;
#pragma unroll
      for (int blk = 0; blk < TL::kBlocks; ++blk)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int d = 32 * blk + 8 * q + 4 * h;
          if (d < D)
            *reinterpret_cast<f32x4*>(a.part + row * D + d) =
                f32x4{o[blk][n][4 * q], o[blk][n][4 * q + 1], o[blk][n][4 * q + 2], o[blk][n][4 * q + 3]} * f;
        }
      continue;
    }
    const int head = hk * G + g;
    if (h == 0) a.lse[((int64_t)b * a.H + head) * a.Lq + i] = lse2 * kLn2;
    T* row = static_cast<T*>(a.o.p) + b * a.o.batch + i * a.o.token + head * a.o.head;
#pragma unroll
    for (int blk = 0; blk < TL::kBlocks; ++blk) {
      u32x4 c[2];
      head_chunks<T>(o[blk][n], f, c);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int d = 32 * blk + 16 * q + 8 * h;
        if (d < D) *reinterpret_cast<u32x4*>(row + d) = c[q];
      }
    }
  }
}

// The parts of a row's keys joined, a wave half (32 lanes of four elements) a
// row: with the parts' lse, o = sum 2^(lse_s - m) o_s / sum 2^(lse_s - m).
template <typename T>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  const int R = a.Lq * a.G, lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.B * a.Hk * R, row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  float m = -__builtin_inff();
  for (int s = 0; s < a.splits; ++s) m = __builtin_fmaxf(m, a.part_lse[s * rows + row]);
  const float base = m == -__builtin_inff() ? 0.f : m;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
  const int d = lane * 4;
  for (int s = 0; s < a.splits; ++s) {
    const float w = __builtin_amdgcn_exp2f(a.part_lse[s * rows + row] - base);
    sum += w;
    if (d < a.D) o += *reinterpret_cast<const f32x4*>(a.part + (s * rows + row) * a.D + d) * w;
  }
  const int hb = (int)(row / R), r = (int)(row % R), i = r / a.G, head = hb % a.Hk * a.G + r - i * a.G, b = hb / a.Hk;
  o *= sum == 0.f ? 0.f : 1.f / sum;
  if (lane == 0) a.lse[((int64_t)b * a.H + head) * a.Lq + i] = (m + __builtin_log2f(sum)) * kLn2;
  if (d < a.D)
    *reinterpret_cast<u32x2*>(static_cast<T*>(a.o.p) + b * a.o.batch + i * a.o.token + head * a.o.head + d) =
        u32x2{cvt_x2<T>(o[0], o[1]), cvt_x2<T>(o[2], o[3])};
}

template <typename T>
hipError_t launch_fwd(const AttnArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.blocks * a.splits * a.B * a.Hk)), block(512);
  if (a.D <= 64)
    hipLaunchKernelGGL((attn_fwd_kernel<T, 64, 8, 1>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((attn_fwd_kernel<T, 128, 8, 1>), grid, block, 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t rows = (int64_t)a.B * a.H * a.Lq;
  hipLaunchKernelGGL((attn_join_kernel<T>), dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attention(const AttnArgs& a, hipStream_t st) {
  return a.dtype == SVDQ_DT_BF16 ? launch_fwd<Bf16>(a, st) : launch_fwd<Half>(a, st);
}

}  // namespace svdq
