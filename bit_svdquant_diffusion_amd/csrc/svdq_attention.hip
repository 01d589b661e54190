// Attention, forward: of each query row, over the keys j that it sees,
//
//   s_j = scale q . k_j,  m = max s_j,  o = sum exp(s_j - m) v_j / sum exp(s_j - m),
//   lse = m + log sum exp(s_j - m).
//
// One pass over the keys with the running maximum and sum: a workgroup holds
// 32 query rows a wave, K and V pass by in tiles of 64 keys. The product is
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

constexpr float kLn2 = 0.69314718055994530942f;

// Up to here a row's reference (in base 2) is off by half a step of fp32, 2^-5 at
// most, which its largest probability has room for; from 2^30 on it would be off
// by more than fp32's exponents hold.
constexpr float kFarScore = 0x1p20f;
__device__ __forceinline__ float reference(float m, float scale_log2) {
  return m == -__builtin_inff() ? 0.f : m * scale_log2;
}
// what m scale_log2 is above the reference that the sums have
__device__ __forceinline__ float reference_off(float m, float base, float scale_log2) {
  return m == -__builtin_inff() || __builtin_fabsf(base) > kFarScore ? 0.f : __builtin_fmaf(m, scale_log2, -base);
}

// W waves of 32 query rows, KW times (each way takes every KW-th tile); DP the
// padded head; NP operands for probabilities. Two waves a SIMD (up to 256
// registers), so that one's products run under the other's exponentials: 4608
// tokens, 24 heads of 128 with a mask 245 us (1.06 PFLOP/s), with one wave a
// SIMD 411, with one of two blocks 355, with workgroups of four waves instead of
// eight 270. What bounds it: a tile's
// exponentials, maxima, sums and roundings take the vector unit as long as its
// products the matrix unit (40% of the cycles), at a clock that power holds
// near 2 GHz; LDS is busy a fifth of the time. One query over 65536 keys
// streams caches of 268 MB in turn at 4.8 TB/s (56 us; a call with the join 61).
template <typename T, int DP, int W, int KW, int NP, bool PARTS>
__global__ __launch_bounds__(64 * W * KW) __attribute__((amdgpu_waves_per_eu(DP <= 64 ? 4 : 2, DP <= 64 ? 4 : 2))) void attn_fwd_kernel(AttnArgs a, AttnDeal<PARTS> deal) {
  typedef AttnTile<DP> TL;
  constexpr int NT = TL::kTransfers / W;   // transfers of a wave for one tile
  extern __shared__ __align__(1024) uint8_t smem[];   // [KW][2][K, V][kBytes]
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, lr = lane & 31;
  const int w_id = __builtin_amdgcn_readfirstlane(tid >> 6), wave = KW == 1 ? w_id : w_id % W, way = KW == 1 ? 0 : w_id / W;
  const int G = a.G, R = a.Lq * G, D = a.D;
  const typename TL::Lane pl(lane);
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
  const int place = attn_place(a.plan, blockIdx.x);
  const AttnPiece at = piece_of(a, deal, place);
  const int b = at.hb / a.Hk, hk = at.hb % a.Hk;
  const T* qp = static_cast<const T*>(a.q.p) + b * a.q.batch + (int64_t)hk * G * a.q.head;
  const T* kp = static_cast<const T*>(a.k.p) + b * a.k.batch + hk * a.k.head;
  const T* vp = static_cast<const T*>(a.v.p) + b * a.v.batch + hk * a.v.head;
  const uint8_t* mask = a.mask ? a.mask + b * a.mask_batch : nullptr;

  // this lane's rows and the last keys that they see
  const int r0 = at.block * (32 * W) + wave * 32;
  u32x4 qf[TL::kSteps];
  const int r = r0 + lr, query = attn_query(a.group, r), g = r - query * G;
  const T* q_row = qp + (int64_t)query * a.q.token + (int64_t)g * a.q.head;
  const int last = r >= R ? -1 : a.causal ? min(query + a.Lk - a.Lq, a.Lk - 1) : a.Lk - 1;   // of a row without keys below 0
#pragma unroll
  for (int s = 0; s < TL::kSteps; ++s) {
    const int d = 16 * s + 8 * h;
    qf[s] = r < R && d < D ? *reinterpret_cast<const u32x4*>(q_row + d) : u32x4{0, 0, 0, 0};
  }
  const int k_begin = (at.first + way) * kAttnRows, k_end = at.last * kAttnRows, rounds = (at.last - at.first + KW - 1) / KW;
  // what every and what any row of this wave sees
  const int w_first = a.causal ? attn_query(a.group, r0) + a.Lk - a.Lq : a.Lk - 1;
  const int w_last = r0 >= R ? -1 : a.causal ? attn_query(a.group, min(r0 + 32, R) - 1) + a.Lk - a.Lq : a.Lk - 1;

  auto fetch = [&](int k0, int stage, uint64_t keep) {
    const int rows = min(kAttnRows, a.Lk - k0);
    const auto rk = rows_resource(kp + k0 * a.k.token, (int)((rows - 1) * a.k.token + D) * 2);
    const auto rv = rows_resource(vp + k0 * a.v.token, (int)((rows - 1) * a.v.token + D) * 2);
    uint8_t *tk = smem + (way * 2 + stage) * 2 * TL::kBytes + wave * NT * 1024, *tv = tk + TL::kBytes;
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

  // Of a row: m, the score (before the scale) that its maximum is taken at, and
  // the reference of its sums in base 2, base = fp32(m scale_log2), so that a
  // probability is one fused product. Where that is far from zero its rounding
  // is no longer small beside 1: there (far: a row of the wave) the reference
  // is m scale_log2 itself, and m is subtracted before the scale.
  f32x16 o[TL::kBlocks];
  float m = -__builtin_inff(), base = 0.f, l = 0.f;
  bool far = false;
#pragma unroll
  for (int i = 0; i < TL::kBlocks; ++i) o[i] = f32x16{};
  uint64_t now, keep = 0;   // which keys of the tile, and of the next, take part
  int next_byte = 0;
  constexpr int kStep = KW * kAttnRows;
  if (k_begin < k_end) {
    keep = __ballot(mask_byte(k_begin) != 0);
    fetch(k_begin, 0, keep);
    next_byte = mask_byte(k_begin + kStep);
  }
  for (int t = 0, k0 = k_begin; t < rounds; ++t, k0 += kStep) {
    now = keep;
    tile_barrier();
    if (k0 + kStep < k_end) {
      keep = __ballot(next_byte != 0);
      fetch(k0 + kStep, (t + 1) & 1, keep);
      next_byte = mask_byte(k0 + 2 * kStep);
    }
    const uint8_t *tk = smem + (way * 2 + (t & 1)) * 2 * TL::kBytes, *tv = tk + TL::kBytes;
    if (k0 > w_last || now == 0 || (KW > 1 && k0 >= k_end)) continue;   // nothing that this wave's rows see
    f32x16 s[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
      s[kb] = f32x16{};
#pragma unroll
    for (int st = 0; st < TL::kSteps; ++st)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const u32x4 kf = TL::straight(tk, pl, kb, st);
        s[kb] = mma<T>(kf, qf[st], s[kb]);
      }
    sched_products<2 * TL::kSteps, 2 * TL::kSteps, 1, 4>();
    if (now != ~0ull || k0 + kAttnRows - 1 > w_first) {
      const int lim = last - k0 - 4 * h;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const uint32_t bits = (uint32_t)(now >> (32 * kb)) >> (4 * h);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = 8 * (i / 4) + i % 4;
          s[kb][i] = (bits >> c & 1) && 32 * kb + c <= lim ? s[kb][i] : -__builtin_inff();
        }
      }
    }
    u32x4 p[4][NP];
    float top = s[0][0];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, s[kb][i]);
    top = max_halves(top);
    // The maximum that is subtracted follows the true one when that is more
    // than 8 (in base 2) above it: up to there the probabilities stay below
    // 2^8, which neither the sums nor either type's rounding minds, and most
    // tiles leave the accumulators as they are.
    if (__any((top - m) * a.scale_log2 > 8.f)) {
      const float mn = __builtin_fmaxf(m, top), bn = reference(mn, a.scale_log2);
      const float step = (m - mn) * a.scale_log2 + (reference_off(mn, bn, a.scale_log2) - reference_off(m, base, a.scale_log2));
      const float f = m == mn ? 1.f : __builtin_amdgcn_exp2f(step);
      m = mn;
      base = bn;
      far = __any(__builtin_fabsf(bn) > kFarScore);
      l *= f;
#pragma unroll
      for (int i = 0; i < TL::kBlocks; ++i) o[i] *= f;
    }
    float sub = base;
    if (far) {
      const bool before = __builtin_fabsf(sub) > kFarScore;   // (this row's)
      const float off = before ? m : 0.f;
      sub = before ? 0.f : sub;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[kb][i] -= off;
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[kb][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][i], a.scale_log2, -sub));
        l += s[kb][i];
      }
      as_operands<T>(s[kb], 0, p[2 * kb]);
      as_operands<T>(s[kb], 1, p[2 * kb + 1]);
    }
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
#pragma unroll
      for (int i = 0; i < TL::kBlocks; ++i) {
        const u32x4 vf = TL::turned(tv, pl, kt, i);
#pragma unroll
        for (int w = 0; w < NP; ++w) o[i] = mma<T>(vf, p[kt][w], o[i]);
      }
    sched_products<4 * TL::kBlocks * NP, 8 * TL::kBlocks, 2, 8>();
  }
  float lo = reference_off(m, base, a.scale_log2);   // what the reference of the sums is below m scale_log2
  if constexpr (KW > 1) {   // the second way's results join the first's
    f32x4* box = reinterpret_cast<f32x4*>(smem) + wave * (4 * TL::kBlocks * 64) + lane;
    f32x4* stat = reinterpret_cast<f32x4*>(smem + W * TL::kBlocks * 4096) + wave * 64 + lane;
    tile_barrier();
    if (way == 1) {
#pragma unroll
      for (int i = 0; i < TL::kBlocks; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          box[(4 * i + q) * 64] = f32x4{o[i][4 * q], o[i][4 * q + 1], o[i][4 * q + 2], o[i][4 * q + 3]};
      *stat = f32x4{m, l, lo, 0.f};
    }
    tile_barrier();
    if (way == 1) return;
    const f32x4 other = *stat;
    const float top = __builtin_fmaxf(m, other[0]), from = top == -__builtin_inff() ? 0.f : top;
    const float f = __builtin_amdgcn_exp2f((m - from) * a.scale_log2 - lo);
    const float fo = __builtin_amdgcn_exp2f((other[0] - from) * a.scale_log2 - other[2]);
    m = top;
    base = reference(top, a.scale_log2);
    lo = 0.f;
    l = l * f + other[1] * fo;
#pragma unroll
    for (int i = 0; i < TL::kBlocks; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 v = box[(4 * i + q) * 64];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][4 * q + k] = o[i][4 * q + k] * f + v[k] * fo;
      }
  }
  const float sum = sum_halves(l);
  const float f = sum == 0.f ? 0.f : 1.f / sum, lse2 = base + __builtin_log2f(sum);   // (no key: -inf)
  if (r >= R) return;
  if (PARTS && !at.whole) {
    const int64_t row = (int64_t)place * a.part_rows + r - at.block * (32 * W);
    if (h == 0) reinterpret_cast<f32x2*>(a.part_stat)[row] = f32x2{m, sum * __builtin_amdgcn_exp2f(-lo)};
#pragma unroll
    for (int blk = 0; blk < TL::kBlocks; ++blk)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int d = 32 * blk + 8 * q + 4 * h;
        if (d < D)
          *reinterpret_cast<f32x4*>(a.part + row * D + d) =
              f32x4{o[blk][4 * q], o[blk][4 * q + 1], o[blk][4 * q + 2], o[blk][4 * q + 3]} * f;
      }
    return;
  }
  const int head = hk * G + g;
  if (h == 0) a.lse[((int64_t)b * a.H + head) * a.Lq + query] = lse2 * kLn2;
  T* row = static_cast<T*>(a.o.p) + b * a.o.batch + query * a.o.token + head * a.o.head;
#pragma unroll
  for (int blk = 0; blk < TL::kBlocks; ++blk) {
    u32x4 c[2];
    head_chunks<T>(o[blk], f, c);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int d = 32 * blk + 16 * q + 8 * h;
      if (d < D) *reinterpret_cast<u32x4*>(row + d) = c[q];
    }
  }
}

// The parts of units joined: with the parts' maxima (before the scale) and sums,
// w_s = l_s 2^((m_s - m) scale_log2), o = sum w_s o_s / sum w_s. WAYS half waves (32 lanes of four elements) have a row,
// each every WAYS-th part; theirs are then joined in order through LDS.
template <typename T, int WAYS>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, AttnJoins joins) {
  constexpr int ROWS = 8 / WAYS;
  __shared__ float ms[8], sums[8];
  __shared__ f32x4 os[8][32];
  const AttnJoin at = joins.at[blockIdx.x];
  const int hb = at.unit / a.plan.blocks, block = at.unit - hb * a.plan.blocks;
  const int lane = threadIdx.x & 31, half = threadIdx.x >> 5, way = half % WAYS;
  const int in = (int)blockIdx.y * ROWS + half / WAYS, r = block * a.cost.block + in, d = lane * 4;
  const bool live = in < a.part_rows && r < a.Lq * a.G;
  float m = -__builtin_inff(), sum = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  if (live) {
    for (int w = way; w < at.parts; w += WAYS) m = __builtin_fmaxf(m, a.part_stat[((int64_t)(at.first + w) * a.part_rows + in) * 2]);
    const float base = m == -__builtin_inff() ? 0.f : m;
    for (int w = way; w < at.parts; w += WAYS) {
      const int64_t row = (int64_t)(at.first + w) * a.part_rows + in;
      const f32x2 stat = reinterpret_cast<const f32x2*>(a.part_stat)[row];
      const float f = stat[1] * __builtin_amdgcn_exp2f((stat[0] - base) * a.scale_log2);
      sum += f;
      if (d < a.D) o += *reinterpret_cast<const f32x4*>(a.part + row * a.D + d) * f;
    }
  }
  if constexpr (WAYS > 1) {
    if (lane == 0) {
      ms[half] = m;
      sums[half] = sum;
    }
    os[half][lane] = o;
    __syncthreads();
    if (way != 0) return;
    float top = m;
#pragma unroll
    for (int i = 1; i < WAYS; ++i) top = __builtin_fmaxf(top, ms[half + i]);
    const float base = top == -__builtin_inff() ? 0.f : top;
    const float own = __builtin_amdgcn_exp2f((m - base) * a.scale_log2);
    o *= own;
    sum *= own;
#pragma unroll
    for (int i = 1; i < WAYS; ++i) {
      const float f = __builtin_amdgcn_exp2f((ms[half + i] - base) * a.scale_log2);
      sum = __builtin_fmaf(sums[half + i], f, sum);
      o += os[half + i][lane] * f;
    }
    m = top;
  }
  if (!live) return;
  const int i = attn_query(a.group, r), head = hb % a.Hk * a.G + r - i * a.G, b = hb / a.Hk;
  o *= sum == 0.f ? 0.f : 1.f / sum;
  if (lane == 0) a.lse[((int64_t)b * a.H + head) * a.Lq + i] = (reference(m, a.scale_log2) + __builtin_log2f(sum)) * kLn2;
  if (d < a.D)
    *reinterpret_cast<u32x2*>(static_cast<T*>(a.o.p) + b * a.o.batch + i * a.o.token + head * a.o.head + d) =
        u32x2{cvt_x2<T>(o[0], o[1]), cvt_x2<T>(o[2], o[3])};
}

template <int DP, int KW>
constexpr int kFwdLds = 4 * KW * AttnTile<DP>::kBytes;

template <typename T, int DP, int W, int KW, int NP>
hipError_t launch_fwd(const AttnArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.plan.grid), block(64 * W * KW);
  if constexpr (kAttnCut<W, KW>)
    if (a.plan.each) {
      AttnParts deal;
      attn_parts(a.cost, a.plan, &deal);
      hipLaunchKernelGGL((attn_fwd_kernel<T, DP, W, KW, NP, true>), grid, block, (kFwdLds<DP, KW>), st, a, deal);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      AttnJoins joins;
      const int units = attn_joins(a.plan, deal, &joins);
      // with many parts a row, all of a workgroup for one
      const bool deep = a.plan.grid >= 12 * units;
      const dim3 rows((unsigned)units, (unsigned)(deep ? a.part_rows : (a.part_rows + 7) / 8));
      if (deep)
        hipLaunchKernelGGL((attn_join_kernel<T, 8>), rows, dim3(256), 0, st, a, joins);
      else
        hipLaunchKernelGGL((attn_join_kernel<T, 1>), rows, dim3(256), 0, st, a, joins);
      return hipGetLastError();
    }
  hipLaunchKernelGGL((attn_fwd_kernel<T, DP, W, KW, NP, false>), grid, block, (kFwdLds<DP, KW>), st, a, AttnUnits{});
  return hipGetLastError();
}
template <typename T, int DP>
hipError_t launch_fwd(const AttnArgs& a, hipStream_t st) {
  const bool wide = a.cost.block == 8 * kAttnWave;
  if constexpr (DP == 32) {
    if (a.cost.ways == 2) return launch_fwd<T, DP, 4, 2, 2>(a, st);
    return wide ? launch_fwd<T, DP, 8, 1, 2>(a, st) : launch_fwd<T, DP, 4, 1, 2>(a, st);
  } else {
    if (a.cost.fine) return launch_fwd<T, DP, 8, 1, 2>(a, st);
    if (a.cost.ways == 2) return launch_fwd<T, DP, 4, 2, 1>(a, st);
    return wide ? launch_fwd<T, DP, 8, 1, 1>(a, st) : launch_fwd<T, DP, 4, 1, 1>(a, st);
  }
}
template <typename T>
hipError_t launch_fwd(const AttnArgs& a, hipStream_t st) {
  if (a.D <= 32) return launch_fwd<T, 32>(a, st);
  if (a.D <= 64) return launch_fwd<T, 64>(a, st);
  return a.D <= 96 ? launch_fwd<T, 96>(a, st) : launch_fwd<T, 128>(a, st);
}

template <typename T, int DP, int W, int KW, int NP>
hipError_t prepare_fwd() {
  hipError_t e = attn_shared_memory((const void*)attn_fwd_kernel<T, DP, W, KW, NP, false>, kFwdLds<DP, KW>);
  if constexpr (kAttnCut<W, KW>)
    if (e == hipSuccess) e = attn_shared_memory((const void*)attn_fwd_kernel<T, DP, W, KW, NP, true>, kFwdLds<DP, KW>);
  return e;
}
template <typename T, int DP>
hipError_t prepare_fwd_of() {
  for (hipError_t e : {prepare_fwd<T, DP, 4, 1, 1>(), prepare_fwd<T, DP, 4, 2, 1>(), prepare_fwd<T, DP, 8, 1, 1>(),
                       prepare_fwd<T, DP, 8, 1, 2>()})
    if (e != hipSuccess) return e;
  return hipSuccess;
}
template <typename T>
hipError_t prepare_fwd() {
  for (hipError_t e : {prepare_fwd<T, 32, 4, 1, 2>(), prepare_fwd<T, 32, 4, 2, 2>(), prepare_fwd<T, 32, 8, 1, 2>(),
                       prepare_fwd_of<T, 64>(), prepare_fwd_of<T, 96>(), prepare_fwd_of<T, 128>()})
    if (e != hipSuccess) return e;
  return hipSuccess;
}

}  // namespace

hipError_t prepare_attention() {
  const hipError_t e = prepare_fwd<Bf16>();
  return e != hipSuccess ? e : prepare_fwd<Half>();
}

hipError_t launch_attention(const AttnArgs& a, hipStream_t st) {
  return a.dtype == SVDQ_DT_BF16 ? launch_fwd<Bf16>(a, st) : launch_fwd<Half>(a, st);
}

}  // namespace svdq
