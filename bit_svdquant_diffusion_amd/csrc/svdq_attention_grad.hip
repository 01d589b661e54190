// Attention's gradients, the probabilities recomputed from the forward's lse:
//
//   p = exp(scale q k^T - lse),  delta = sum_d do o,  ds = p (do v^T - delta),
//   dv = p^T do,  dk = scale ds^T q,  dq = scale ds k.
//
// Two passes over the scores, each with its results in registers, so that no
// sum is joined by atomics and every order is fixed: one holds 32 keys a
// wave (dk, dv) while the query rows pass by in tiles of 64, one holds 32
// query rows (dq) while the keys do. That is seven products instead of five,
// against a float of traffic per pair of a row and a tile of keys for joining
// dq. As in the forward, the products whose results are the next ones'
// operands are taken so that the held side is the columns, and the heads of a
// key head are rows of the same tiles, which sums a shared head's gradients.
//
// fp16 holds 2^-24 at least. Gradients and probabilities go well below that,
// so p enters its product times 2^10, and ds times the power of two that
// brings the largest value it could have, 2 D max|do| max|v|, to 2^15; both
// are taken out of the sums in fp32. The largest |v| is that of all keys, also
// for one key's ds: delta is do . o, which any key that the row sees may make
// large. bf16 has fp32's exponents and needs none.
#include <algorithm>

#include "svdq_attention.h"
#include "svdq_internal.h"
#include "svdq_layout.h"

namespace svdq {

namespace {

constexpr float kProbScale = 1024.f;   // of fp16 probabilities

template <typename T>
constexpr bool kScaled = !__is_same(T, Bf16);

// the largest magnitude of eight packed fp16 values and m
template <typename T>
__device__ __forceinline__ float amax_x8(float m, u32x4 w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t pair = w[i];   // (a vector's element taken as another type as it stands is its first)
    const f16x2 v = __builtin_bit_cast(f16x2, pair);
    m = __builtin_fmaxf(m, __builtin_fmaxf(__builtin_fabsf((float)v[0]), __builtin_fabsf((float)v[1])));
  }
  return m;
}
template <typename T>
__device__ __forceinline__ float dot_x2(float s, uint32_t a, uint32_t b) {
  if constexpr (__is_same(T, Bf16)) {
    return __builtin_fmaf(bf16hi(a), bf16hi(b), __builtin_fmaf(bf16lo(a), bf16lo(b), s));
  } else {
    const f16x2 x = __builtin_bit_cast(f16x2, a), y = __builtin_bit_cast(f16x2, b);
    return __builtin_fmaf((float)x[1], (float)y[1], __builtin_fmaf((float)x[0], (float)y[0], s));
  }
}

// fp16: the largest |v| of runs of keys (of those that the mask keeps),
// sixteen lanes a key.
template <typename T>
__global__ __launch_bounds__(256) void attn_top_v_kernel(AttnGradArgs g) {
  const AttnArgs& a = g.f;
  __shared__ float red[16];
  const int hb = blockIdx.y, b = hb / a.Hk, hk = hb % a.Hk, lane = threadIdx.x & 15, slot = threadIdx.x >> 4;
  float top = 0.f;
  u32x4 x[kAttnKeyRun / 16];   // (all loads at once)
#pragma unroll
  for (int k = 0; k < kAttnKeyRun / 16; ++k) {
    const int key = blockIdx.x * kAttnKeyRun + k * 16 + slot, at = min(key, a.Lk - 1);
    const bool in = key < a.Lk && lane * 8 < a.D && (!a.mask || a.mask[b * a.mask_batch + at]);
    x[k] = *reinterpret_cast<const u32x4*>(static_cast<const T*>(a.v.p) + b * a.v.batch + at * a.v.token + hk * a.v.head +
                                           (lane * 8 < a.D ? lane * 8 : 0));
    if (!in) x[k] = u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int k = 0; k < kAttnKeyRun / 16; ++k) top = amax_x8<T>(top, x[k]);
  const uint32_t m = max_dpp16(__float_as_uint(top));   // (magnitudes: their bits are in order)
  if (lane == 0) red[slot] = __uint_as_float(m);
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = red[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) v = __builtin_fmaxf(v, red[i]);
    g.top_v[(int64_t)hb * g.key_runs + blockIdx.x] = v;
  }
}

// the largest of n values, the same in every lane
__device__ __forceinline__ float wave_top(const float* p, int n, int lane) {
  float x = 0.f;
  for (int i = lane; i < n; i += 64) x = __builtin_fmaxf(x, p[i]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x = __builtin_fmaxf(x, __shfl_xor(x, d));
  return x;
}
// The power of two of a ds whose do and v are at most x and y: |dp - delta| is
// at most 2 D x y, which it brings below 2^15.
__device__ __forceinline__ float ds_scale(int D, float x, float y) {
  const float top = 2.f * (float)D * x * y;   // (at most 2^8 2^16 2^16)
  if (!(top > 0.f) || !(top < 0x1p100f)) return 1.f;
  const int e = (int)(__float_as_uint(top) >> 23) - 126;   // 2^e > top >= 2^(e - 1)
  return exp2_int(min(15 - e, 100));
}

// The second way's results join the first's through LDS, I-th of a wave's sums.
template <int DP, int W, int I>
__device__ __forceinline__ f32x4* join_place(uint8_t* smem, int wave, int lane) {
  return reinterpret_cast<f32x4*>(smem) + (I * W + wave) * (AttnTile<DP>::kBlocks * 256) + lane;
}
template <int DP, int W, int I>
__device__ __forceinline__ void join_put(uint8_t* smem, int wave, int lane, const f32x16 (&v)[AttnTile<DP>::kBlocks]) {
  f32x4* to = join_place<DP, W, I>(smem, wave, lane);
#pragma unroll
  for (int i = 0; i < AttnTile<DP>::kBlocks; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      to[(4 * i + q) * 64] = f32x4{v[i][4 * q], v[i][4 * q + 1], v[i][4 * q + 2], v[i][4 * q + 3]};
}
template <int DP, int W, int I>
__device__ __forceinline__ void join_add(uint8_t* smem, int wave, int lane, f32x16 (&v)[AttnTile<DP>::kBlocks]) {
  const f32x4* from = join_place<DP, W, I>(smem, wave, lane);
#pragma unroll
  for (int i = 0; i < AttnTile<DP>::kBlocks; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x4 x = from[(4 * i + q) * 64];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i][4 * q + k] += x[k];
    }
}

// dk and dv of 32 keys a wave; the query rows pass by. With heads of 128
// the accumulators and the K fragments take 160 of the 256 registers that two
// waves a SIMD leave, so V's fragments wait in LDS (4608 tokens, 24 heads, of
// the same step: 574 us against 760 with V in registers, of which 53 spill, 768
// with one wave a SIMD and two blocks of keys, 870 with workgroups of four
// waves; now 530, 0.99 PFLOP/s, with the matrix unit busy 45% of the cycles).
template <typename T, int DP, int W, int KW, int NP, bool PARTS>
__global__ __launch_bounds__(64 * W * KW) __attribute__((amdgpu_waves_per_eu(DP == 32 ? 4 : 2, DP == 32 ? 4 : 2))) void attn_dkv_kernel(AttnGradArgs g, AttnDeal<PARTS> deal) {
  typedef AttnTile<DP> TL;
  const AttnArgs& a = g.f;
  constexpr int NT = TL::kTransfers / W;
  static_assert(KW == 1 || DP < 128, "V is held for each way");
  extern __shared__ __align__(1024) uint8_t smem[];   // [KW][2][q, do][kBytes], then V where it is held there
  constexpr bool kHoldV = DP < 128;   // in registers, else in LDS
  uint8_t* held = smem + 4 * TL::kBytes;
  __shared__ __align__(1024) float stats[KW][2][2][kAttnRows];   // -lse / scale and -delta of a tile's rows
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, lr = lane & 31;
  const int w_id = __builtin_amdgcn_readfirstlane(tid >> 6), wave = KW == 1 ? w_id : w_id % W, way = KW == 1 ? 0 : w_id / W;
  const int G = a.G, R = a.Lq * G, D = a.D;
  const typename TL::Lane pl(lane);
  const int place = attn_place(a.plan, blockIdx.x);
  const AttnPiece at = piece_of(a, deal, place);
  const int b = at.hb / a.Hk, hk = at.hb % a.Hk;
  const T* qp = static_cast<const T*>(a.q.p) + b * a.q.batch + (int64_t)hk * G * a.q.head;
  const T* dop = static_cast<const T*>(g.dout.p) + b * g.dout.batch + (int64_t)hk * G * g.dout.head;
  const int64_t Rp = g.rows_padded;
  const float *lse = g.lse + at.hb * Rp, *delta = g.delta + at.hb * Rp;
  const float c = kScaled<T> ? ds_scale(D, wave_top(g.top_do + at.hb * g.row_blocks, g.row_blocks, lane),
                                        wave_top(g.top_v + at.hb * g.key_runs, g.key_runs, lane))
                             : 1.f;
  const float dsc = c / kProbScale, fk = a.scale / c;   // the factor of ds (of fp16 probabilities); of dk

  // this lane's keys, as operand B (of both products that give scores)
  const int key0 = at.block * (32 * W) + wave * 32;
  u32x4 kf[TL::kSteps], vf[TL::kSteps];
  const int key = key0 + lr;
  const bool live = key < a.Lk && (!a.mask || a.mask[b * a.mask_batch + key]);
  const int first = a.causal ? max(key - (a.Lk - a.Lq), 0) * G : 0;   // the first row that sees the key
  const T* kr = static_cast<const T*>(a.k.p) + b * a.k.batch + key * a.k.token + hk * a.k.head;
  const T* vr = static_cast<const T*>(a.v.p) + b * a.v.batch + key * a.v.token + hk * a.v.head;
#pragma unroll
  for (int s = 0; s < TL::kSteps; ++s) {
    const int d = 16 * s + 8 * h;
    const bool in = live && d < D;
    kf[s] = in ? *reinterpret_cast<const u32x4*>(kr + d) : u32x4{0, 0, 0, 0};
    const u32x4 v = in ? *reinterpret_cast<const u32x4*>(vr + d) : u32x4{0, 0, 0, 0};
    if constexpr (kHoldV)
      vf[s] = v;
    else   // (read by this wave alone)
      *reinterpret_cast<u32x4*>(held + wave * 32 * TL::kRowBytes + (pl.straight ^ (s << 5))) = v;
  }
  const uint8_t* my_v = held + (kHoldV ? 0 : wave * 32 * TL::kRowBytes);
  // rows that see no key at all are read as zeros
  int dead = 0;
  if (a.causal) {
    int k = 0;   // the first key that the mask keeps
    if (a.mask) {
      const uint8_t* mask = a.mask + b * a.mask_batch;
      uint64_t some = 0;
      for (; k < a.Lk && some == 0; k += 64) some = __ballot(k + lane < a.Lk && mask[k + lane]);
      k = some ? k - 64 + __builtin_ctzll(some) : a.Lk;
    }
    dead = min(max(k - (a.Lk - a.Lq), 0), a.Lq) * G;
  }
  const int r_begin = (at.first + way) * kAttnRows, r_end = at.last * kAttnRows, rounds = (at.last - at.first + KW - 1) / KW;
  const int w_first = a.causal ? max(key0 - (a.Lk - a.Lq), 0) * G : 0;
  const int w_all = a.causal ? max(key0 + 31 - (a.Lk - a.Lq), 0) * G : 0;   // from here on rows see all of the wave's keys

  auto fetch = [&](int row0, int stage) {
    const int i0 = attn_query(a.group, row0), i1 = attn_query(a.group, min(row0 + kAttnRows, R) - 1);
    // the heads of the queries i0 .. i1
    const auto rq = rows_resource(qp + i0 * a.q.token, (int)((i1 - i0) * a.q.token + (G - 1) * a.q.head + D) * 2);
    const auto rd = rows_resource(dop + i0 * g.dout.token, (int)((i1 - i0) * g.dout.token + (G - 1) * g.dout.head + D) * 2);
    uint8_t *tq = smem + (way * 2 + stage) * 2 * TL::kBytes + wave * NT * 1024, *td = tq + TL::kBytes;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int j = wave * NT + n, ch = TL::chunk_of(j, lane), r = row0 + TL::row_of(j, lane);
      const int i = attn_query(a.group, r), hd = r - i * G;
      const bool in = r < R && r >= dead && ch * 8 < D;
      lds_transfer_16(rq, tq + n * 1024, in ? (uint32_t)(((i - i0) * a.q.token + hd * a.q.head + ch * 8) * 2) : kPastEnd);
      lds_transfer_16(rd, td + n * 1024, in ? (uint32_t)(((i - i0) * g.dout.token + hd * g.dout.head + ch * 8) * 2) : kPastEnd);
    }
    if (wave < 2) {   // (rows up to whole tiles are there)
      const auto rs = rows_resource((wave == 0 ? lse : delta) + row0, kAttnRows * 4);
      lds_transfer_4(rs, reinterpret_cast<uint8_t*>(stats[way][stage][wave]), lane * 4);
    }
  };

  f32x16 dk[TL::kBlocks], dv[TL::kBlocks];
#pragma unroll
  for (int i = 0; i < TL::kBlocks; ++i)
    dk[i] = dv[i] = f32x16{};
  constexpr int kStep = KW * kAttnRows;
  if (r_begin < r_end) fetch(r_begin, 0);
  for (int t = 0, row0 = r_begin; t < rounds; ++t, row0 += kStep) {
    tile_barrier();
    if (row0 + kStep < r_end) fetch(row0 + kStep, (t + 1) & 1);
    if (KW > 1 && row0 >= r_end) continue;
    const uint8_t *tq = smem + (way * 2 + (t & 1)) * 2 * TL::kBytes, *td = tq + TL::kBytes;
    const float *tl = stats[way][t & 1][0], *tD = stats[way][t & 1][1];
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) {
      if (row0 + 32 * rb + 31 < w_first) continue;   // none of these rows sees a key of this wave
      // The scores' accumulators start with -lse / scale, those of do v^T with
      // -delta, each row's in its registers.
      f32x16 s, dp;
      u32x4 p[2][NP];
      auto start = [&](const float* rows, f32x16& to) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(rows + 32 * rb + 8 * q + 4 * h);
#pragma unroll
          for (int i = 0; i < 4; ++i) to[4 * q + i] = v[i];
        }
      };
      const bool part = row0 + 32 * rb < w_all;
      start(tl, s);
#pragma unroll
      for (int st = 0; st < TL::kSteps; ++st) {
        const u32x4 qf = TL::straight(tq, pl, rb, st);
        s = mma<T>(qf, kf[st], s);
      }
      sched_products<TL::kSteps, 4 + TL::kSteps, 1, 8>();
#pragma unroll
      for (int i = 0; i < 16; ++i)
        s[i] = __builtin_amdgcn_exp2f(kScaled<T> ? __builtin_fmaf(s[i], a.scale_log2, 10.f) : s[i] * a.scale_log2);
      if (part) {
        const int lim = first - row0 - 32 * rb - 4 * h;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 8 * (i / 4) + i % 4 >= lim ? s[i] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) as_operands<T>(s, u, p[u]);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < TL::kBlocks; ++i) {
          const u32x4 df = TL::turned(td, pl, 2 * rb + u, i);
#pragma unroll
          for (int w = 0; w < NP; ++w) dv[i] = mma<T>(df, p[u][w], dv[i]);
        }
      start(tD, dp);
#pragma unroll
      for (int st = 0; st < TL::kSteps; ++st) {
        const u32x4 df = TL::straight(td, pl, rb, st);
        if constexpr (kHoldV)
          dp = mma<T>(df, vf[st], dp);
        else
          dp = mma<T>(df, TL::straight(my_v, pl, 0, st), dp);
      }
      sched_products<2 * TL::kBlocks * NP + TL::kSteps, 4 * TL::kBlocks + (kHoldV ? 1 : 2) * TL::kSteps, 2, 4>();
#pragma unroll
      for (int i = 0; i < 16; ++i) dp[i] *= kScaled<T> ? s[i] * dsc : s[i];
      if (part) {   // (do may hold what times 0 is NaN)
        const int lim = first - row0 - 32 * rb - 4 * h;
#pragma unroll
        for (int i = 0; i < 16; ++i) dp[i] = 8 * (i / 4) + i % 4 >= lim ? dp[i] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) as_operands<T>(dp, u, p[u]);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < TL::kBlocks; ++i) {
          const u32x4 qf = TL::turned(tq, pl, 2 * rb + u, i);
#pragma unroll
          for (int w = 0; w < NP; ++w) dk[i] = mma<T>(qf, p[u][w], dk[i]);
        }
      sched_products<2 * TL::kBlocks * NP, 4 * TL::kBlocks, 2, 4>();
    }
  }
  if constexpr (KW > 1) {
    const bool second = way == 1;
    tile_barrier();
    if (second) {
      join_put<DP, W, 0>(smem, wave, lane, dk);
      join_put<DP, W, 1>(smem, wave, lane, dv);
    }
    tile_barrier();
    if (second) return;
    join_add<DP, W, 0>(smem, wave, lane, dk);
    join_add<DP, W, 1>(smem, wave, lane, dv);
  }
  const float fv = kScaled<T> ? 1.f / kProbScale : 1.f;
  if (key >= a.Lk) return;
  if (PARTS && !at.whole) {
    float* row = a.part + ((int64_t)place * a.part_rows + key - at.block * (32 * W)) * 2 * D;
#pragma unroll
    for (int blk = 0; blk < TL::kBlocks; ++blk)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int d = 32 * blk + 8 * q + 4 * h;
        if (d >= D) continue;
        f32x4 x, y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = live ? dk[blk][4 * q + i] * fk : 0.f;
          y[i] = live ? dv[blk][4 * q + i] * fv : 0.f;
        }
        *reinterpret_cast<f32x4*>(row + d) = x;
        *reinterpret_cast<f32x4*>(row + D + d) = y;
      }
    return;
  }
  T* to_dk = static_cast<T*>(g.dk.p) + b * g.dk.batch + key * g.dk.token + hk * g.dk.head;
  T* to_dv = static_cast<T*>(g.dv.p) + b * g.dv.batch + key * g.dv.token + hk * g.dv.head;
#pragma unroll
  for (int blk = 0; blk < TL::kBlocks; ++blk) {
    u32x4 x[2], y[2];
    head_chunks<T>(dk[blk], fk, x);
    head_chunks<T>(dv[blk], fv, y);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int d = 32 * blk + 16 * q + 8 * h;
      if (d >= D) continue;
      *reinterpret_cast<u32x4*>(to_dk + d) = live ? x[q] : u32x4{0, 0, 0, 0};   // (a dropped key has no gradient)
      *reinterpret_cast<u32x4*>(to_dv + d) = live ? y[q] : u32x4{0, 0, 0, 0};
    }
  }
}

// dq of 32 query rows a wave; the keys pass by, as in the forward (4608
// tokens, 24 heads of 128: 350 us, 1.12 PFLOP/s, the matrix unit busy 45% of
// the cycles). It also leaves what the keys' pass starts its sums with.
template <typename T, int DP, int W, int KW, int NP, bool PARTS>
__global__ __launch_bounds__(64 * W * KW) __attribute__((amdgpu_waves_per_eu(DP == 32 ? 4 : 2, DP == 32 ? 4 : 2))) void attn_dq_kernel(AttnGradArgs g, AttnDeal<PARTS> deal) {
  typedef AttnTile<DP> TL;
  const AttnArgs& a = g.f;
  constexpr int NT = TL::kTransfers / W;
  extern __shared__ __align__(1024) uint8_t smem[];   // [KW][2][K, V][kBytes]
  __shared__ float tops[W];
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, lr = lane & 31;
  const int w_id = __builtin_amdgcn_readfirstlane(tid >> 6), wave = KW == 1 ? w_id : w_id % W, way = KW == 1 ? 0 : w_id / W;
  const int G = a.G, R = a.Lq * G, D = a.D;
  const typename TL::Lane pl(lane);
  uint32_t vk[NT], vv[NT];
  int row_of[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int j = wave * NT + n, ch = TL::chunk_of(j, lane);
    row_of[n] = TL::row_of(j, lane);
    vk[n] = ch * 8 < D ? (uint32_t)((row_of[n] * a.k.token + ch * 8) * 2) : kPastEnd;
    vv[n] = ch * 8 < D ? (uint32_t)((row_of[n] * a.v.token + ch * 8) * 2) : kPastEnd;
  }
  const int place = attn_place(a.plan, blockIdx.x);
  const AttnPiece at = piece_of(a, deal, place);
  const int b = at.hb / a.Hk, hk = at.hb % a.Hk;
  const T* qp = static_cast<const T*>(a.q.p) + b * a.q.batch + (int64_t)hk * G * a.q.head;
  const T* dop = static_cast<const T*>(g.dout.p) + b * g.dout.batch + (int64_t)hk * G * g.dout.head;
  const T* kp = static_cast<const T*>(a.k.p) + b * a.k.batch + hk * a.k.head;
  const T* vp = static_cast<const T*>(a.v.p) + b * a.v.batch + hk * a.v.head;
  const uint8_t* mask = a.mask ? a.mask + b * a.mask_batch : nullptr;
  const T* op = static_cast<const T*>(a.o.p) + b * a.o.batch + (int64_t)hk * G * a.o.head;
  const int64_t Rp = g.rows_padded;
  const float top_v = kScaled<T> ? wave_top(g.top_v + at.hb * g.key_runs, g.key_runs, lane) : 0.f;

  const int r0 = at.block * (32 * W) + wave * 32;
  u32x4 qf[TL::kSteps], df[TL::kSteps];
  const int r = r0 + lr, query = attn_query(a.group, r), hd = r - query * G;
  const int last = r >= R ? -1 : a.causal ? min(query + a.Lk - a.Lq, a.Lk - 1) : a.Lk - 1;
  float top_do = 0.f, sum = 0.f;
#pragma unroll
  for (int s = 0; s < TL::kSteps; ++s) {
    const int d = 16 * s + 8 * h;
    const bool in = r < R && d < D;
    qf[s] = in ? *reinterpret_cast<const u32x4*>(qp + query * a.q.token + hd * a.q.head + d) : u32x4{0, 0, 0, 0};
    df[s] = in ? *reinterpret_cast<const u32x4*>(dop + query * g.dout.token + hd * g.dout.head + d) : u32x4{0, 0, 0, 0};
    const u32x4 o = in ? *reinterpret_cast<const u32x4*>(op + query * a.o.token + hd * a.o.head + d) : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w) sum = dot_x2<T>(sum, df[s][w], o[w]);
    if constexpr (kScaled<T>) top_do = amax_x8<T>(top_do, df[s]);
  }
  // -lse / scale and -delta; of a row without keys (and behind the last
  // row) -infinity, which makes its probabilities zero, and 0
  const float l = r < R ? a.lse[((int64_t)b * a.H + hk * G + hd) * a.Lq + query] : -__builtin_inff();
  const bool none = l == -__builtin_inff();
  float lse = none ? l : -l / a.scale;   // (negative, as delta)
  sum = sum_halves(sum);
  const float delta = none ? 0.f : -sum;
  if (at.starts && way == 0) {   // for the keys' gradients, which start with them
    if (h == 0) g.lse[at.hb * Rp + r] = lse;
    if (h == 1) g.delta[at.hb * Rp + r] = delta;
  }
  lse *= a.scale_log2;   // in base 2
  float c = 1.f, wg_top = 0.f;
  if constexpr (kScaled<T>) {
    top_do = none ? 0.f : max_halves(top_do);   // (a row that sees no key may hold anything)
    c = ds_scale(D, top_do, top_v);
    wg_top = top_do;
  }
  if (kScaled<T> && at.starts) {   // (all waves)
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) wg_top = __builtin_fmaxf(wg_top, __shfl_xor(wg_top, d));
    if (lane == 0 && way == 0) tops[wave] = wg_top;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int w = 1; w < W; ++w) wg_top = __builtin_fmaxf(wg_top, tops[w]);
      g.top_do[at.hb * g.row_blocks + at.block] = wg_top;
    }
  }
  const int k_begin = (at.first + way) * kAttnRows, k_end = at.last * kAttnRows, rounds = (at.last - at.first + KW - 1) / KW;
  const int w_first = a.causal ? attn_query(a.group, r0) + a.Lk - a.Lq : a.Lk - 1;
  const int w_last = r0 >= R ? -1 : a.causal ? attn_query(a.group, min(r0 + 32, R) - 1) + a.Lk - a.Lq : a.Lk - 1;

  auto fetch = [&](int k0, int stage, uint64_t keep) {
    const int rows = min(kAttnRows, a.Lk - k0);
    const auto rk = rows_resource(kp + k0 * a.k.token, (int)((rows - 1) * a.k.token + D) * 2);
    const auto rv = rows_resource(vp + k0 * a.v.token, (int)((rows - 1) * a.v.token + D) * 2);
    uint8_t *tk = smem + (way * 2 + stage) * 2 * TL::kBytes + wave * NT * 1024, *tv = tk + TL::kBytes;
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
  auto mask_byte = [&](int k0) -> int {
    const int k = k0 + lane;
    return k < a.Lk ? (mask ? (int)mask[k] : 1) : 0;
  };

  f32x16 dq[TL::kBlocks];
#pragma unroll
  for (int i = 0; i < TL::kBlocks; ++i)
    dq[i] = f32x16{};
  uint64_t keep = 0, next_keep = 0;
  int next_byte = 0;
  constexpr int kStep = KW * kAttnRows;
  if (k_begin < k_end) {
    next_keep = __ballot(mask_byte(k_begin) != 0);
    fetch(k_begin, 0, next_keep);
    next_byte = mask_byte(k_begin + kStep);
  }
  for (int t = 0, k0 = k_begin; t < rounds; ++t, k0 += kStep) {
    keep = next_keep;
    tile_barrier();
    if (k0 + kStep < k_end) {
      next_keep = __ballot(next_byte != 0);
      fetch(k0 + kStep, (t + 1) & 1, next_keep);
      next_byte = mask_byte(k0 + 2 * kStep);
    }
    if (k0 > w_last || keep == 0 || (KW > 1 && k0 >= k_end)) continue;
    const uint8_t *tk = smem + (way * 2 + (t & 1)) * 2 * TL::kBytes, *tv = tk + TL::kBytes;
    const bool part = keep != ~0ull || k0 + kAttnRows - 1 > w_first;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      f32x16 s, dp;
      s = f32x16{};
#pragma unroll
      for (int i = 0; i < 16; ++i) dp[i] = delta;
#pragma unroll
      for (int st = 0; st < TL::kSteps; ++st) {
        const u32x4 f = TL::straight(tk, pl, kb, st);
        s = mma<T>(f, qf[st], s);
      }
#pragma unroll
      for (int st = 0; st < TL::kSteps; ++st) {
        const u32x4 f = TL::straight(tv, pl, kb, st);
        dp = mma<T>(f, df[st], dp);
      }
      sched_products<2 * TL::kSteps, 2 * TL::kSteps, 1, 4>();
      u32x4 ds[2][NP];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], a.scale_log2, lse));
        dp[i] *= kScaled<T> ? p * c : p;
      }
      if (part) {
        const int lim = last - k0 - 32 * kb - 4 * h;
        const uint32_t bits = (uint32_t)(keep >> (32 * kb)) >> (4 * h);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int at_key = 8 * (i / 4) + i % 4;
          dp[i] = (bits >> at_key & 1) && at_key <= lim ? dp[i] : 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) as_operands<T>(dp, u, ds[u]);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < TL::kBlocks; ++i) {
          const u32x4 f = TL::turned(tk, pl, 2 * kb + u, i);
#pragma unroll
          for (int w = 0; w < NP; ++w) dq[i] = mma<T>(f, ds[u][w], dq[i]);
        }
      sched_products<2 * TL::kBlocks * NP, 4 * TL::kBlocks, 2, 8>();
    }
  }
  if constexpr (KW > 1) {
    const bool second = way == 1;
    tile_barrier();
    if (second) join_put<DP, W, 0>(smem, wave, lane, dq);
    tile_barrier();
    if (second) return;
    join_add<DP, W, 0>(smem, wave, lane, dq);
  }
  const float f = a.scale / c;
  if (r >= R) return;
  if (PARTS && !at.whole) {
    float* row = a.part + ((int64_t)place * a.part_rows + r - at.block * (32 * W)) * D;
#pragma unroll
    for (int blk = 0; blk < TL::kBlocks; ++blk)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int d = 32 * blk + 8 * q + 4 * h;
        if (d < D)
          *reinterpret_cast<f32x4*>(row + d) = f32x4{dq[blk][4 * q], dq[blk][4 * q + 1], dq[blk][4 * q + 2],
                                                     dq[blk][4 * q + 3]} * f;
      }
    return;
  }
  T* row = static_cast<T*>(g.dq.p) + b * g.dq.batch + query * g.dq.token + (hk * G + hd) * g.dq.head;
#pragma unroll
  for (int blk = 0; blk < TL::kBlocks; ++blk) {
    u32x4 x[2];
    head_chunks<T>(dq[blk], f, x);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int d = 32 * blk + 16 * q + 8 * h;
      if (d < D) *reinterpret_cast<u32x4*>(row + d) = x[q];
    }
  }
}

// The parts of units added in order, a half wave a row: rows of dq, or
// of dk and dv side by side.
template <typename T, bool KEYS>
__global__ __launch_bounds__(256) void attn_grad_join_kernel(AttnGradArgs g, AttnJoins joins) {
  const AttnArgs& a = g.f;
  const AttnJoin at = joins.at[blockIdx.x];
  const int hb = at.unit / a.plan.blocks, block = at.unit - hb * a.plan.blocks;
  const int lane = threadIdx.x & 31, in = (int)blockIdx.y * 8 + (threadIdx.x >> 5), r = block * a.cost.block + in;
  const int width = KEYS ? 2 * a.D : a.D, b = hb / a.Hk, hk = hb % a.Hk, i = attn_query(a.group, r);
  if (in >= a.part_rows || r >= a.cost.held) return;
  for (int d = lane * 4; d < width; d += 128) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int w = 0; w < at.parts; w += 8) {   // eight loads at a time
      f32x4 u[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        u[k] = w + k < at.parts
                   ? *reinterpret_cast<const f32x4*>(a.part + ((int64_t)(at.first + w + k) * a.part_rows + in) * width + d)
                   : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 8; ++k) v += u[k];
    }
    T* to;
    if (!KEYS)
      to = static_cast<T*>(g.dq.p) + b * g.dq.batch + i * g.dq.token + (hk * a.G + r - i * a.G) * g.dq.head + d;
    else if (d < a.D)
      to = static_cast<T*>(g.dk.p) + b * g.dk.batch + r * g.dk.token + hk * g.dk.head + d;
    else
      to = static_cast<T*>(g.dv.p) + b * g.dv.batch + r * g.dv.token + hk * g.dv.head + d - a.D;
    *reinterpret_cast<u32x2*>(to) = u32x2{cvt_x2<T>(v[0], v[1]), cvt_x2<T>(v[2], v[3])};
  }
}

template <typename T, int DP, int W, int KW, int NP, bool KEYS, bool PARTS>
constexpr auto grad_kernel() {
  if constexpr (KEYS)
    return attn_dkv_kernel<T, DP, W, KW, NP, PARTS>;
  else
    return attn_dq_kernel<T, DP, W, KW, NP, PARTS>;
}
template <int DP, int W, int KW, bool KEYS>
constexpr int kGradLds = 4 * KW * AttnTile<DP>::kBytes + (KEYS && DP == 128 ? W * kAttnWave * AttnTile<DP>::kRowBytes : 0);

template <typename T, int DP, int W, int KW, int NP, bool KEYS>
hipError_t launch_pass(AttnGradArgs g, const AttnCost& cost, const AttnPlan& plan, hipStream_t st) {
  if (plan.grid == 0) return hipSuccess;
  g.f.cost = cost;
  g.f.plan = plan;
  g.f.part_rows = (int)attn_part_rows(cost);
  const dim3 grid((unsigned)plan.grid), block(64 * W * KW);
  if constexpr (kAttnCut<W, KW>)
    if (plan.each) {
      AttnParts deal;
      attn_parts(cost, plan, &deal);
      hipLaunchKernelGGL((grad_kernel<T, DP, W, KW, NP, KEYS, true>()), grid, block, (kGradLds<DP, W, KW, KEYS>), st, g, deal);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      AttnJoins joins;
      const dim3 rows((unsigned)attn_joins(plan, deal, &joins), (unsigned)((g.f.part_rows + 7) / 8));
      hipLaunchKernelGGL((attn_grad_join_kernel<T, KEYS>), rows, dim3(256), 0, st, g, joins);
      return hipGetLastError();
    }
  hipLaunchKernelGGL((grad_kernel<T, DP, W, KW, NP, KEYS, false>()), grid, block, (kGradLds<DP, W, KW, KEYS>), st, g, AttnUnits{});
  return hipGetLastError();
}
// (heads above 96: a workgroup of keys has eight waves, see attn_key_cost)
template <typename T, int DP, bool KEYS>
hipError_t launch_pass(const AttnGradArgs& g, const AttnCost& cost, const AttnPlan& plan, hipStream_t st) {
  constexpr int NP = DP == 32 ? 2 : 1;
  if constexpr (DP > 32)
    if (cost.fine) return launch_pass<T, DP, 8, 1, 2, KEYS>(g, cost, plan, st);
  if constexpr (!KEYS || DP < 128)
    if (cost.ways == 2) return launch_pass<T, DP, 4, 2, NP, KEYS>(g, cost, plan, st);
  if constexpr (!KEYS || DP < 128)
    if (cost.block == 4 * kAttnWave) return launch_pass<T, DP, 4, 1, NP, KEYS>(g, cost, plan, st);
  return launch_pass<T, DP, 8, 1, NP, KEYS>(g, cost, plan, st);
}

template <typename T, int DP>
hipError_t launch_bwd(const AttnGradArgs& g, const AttnGradWs& w, hipStream_t st) {
  const AttnArgs& a = g.f;
  hipError_t e = hipSuccess;
  if constexpr (kScaled<T>) {
    if (g.key_runs > 0 && a.Lq > 0) {
      hipLaunchKernelGGL((attn_top_v_kernel<T>), dim3((unsigned)g.key_runs, (unsigned)(a.B * a.Hk)), dim3(256), 0, st, g);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  // (dq's pass leaves what dk and dv's starts with)
  if ((e = launch_pass<T, DP, false>(g, w.rows, w.dq, st)) != hipSuccess) return e;
  return launch_pass<T, DP, true>(g, w.keys, w.dkv, st);
}

template <typename T>
hipError_t launch_bwd(const AttnGradArgs& g, const AttnGradWs& w, hipStream_t st) {
  if (g.f.D <= 32) return launch_bwd<T, 32>(g, w, st);
  if (g.f.D <= 64) return launch_bwd<T, 64>(g, w, st);
  return g.f.D <= 96 ? launch_bwd<T, 96>(g, w, st) : launch_bwd<T, 128>(g, w, st);
}

template <typename T, int DP, int W, int KW, int NP, bool KEYS>
hipError_t prepare_pass() {
  constexpr int lds = kGradLds<DP, W, KW, KEYS>;
  hipError_t e = attn_shared_memory((const void*)grad_kernel<T, DP, W, KW, NP, KEYS, false>(), lds);
  if constexpr (kAttnCut<W, KW>)
    if (e == hipSuccess) e = attn_shared_memory((const void*)grad_kernel<T, DP, W, KW, NP, KEYS, true>(), lds);
  return e;
}
template <typename T, int DP, bool KEYS>
hipError_t prepare_of() {
  constexpr int NP = DP == 32 ? 2 : 1;
  hipError_t e = prepare_pass<T, DP, 8, 1, NP, KEYS>();
  if constexpr (!KEYS || DP < 128) {
    if (e == hipSuccess) e = prepare_pass<T, DP, 4, 1, NP, KEYS>();
    if (e == hipSuccess) e = prepare_pass<T, DP, 4, 2, NP, KEYS>();
  }
  if constexpr (DP > 32)
    if (e == hipSuccess) e = prepare_pass<T, DP, 8, 1, 2, KEYS>();
  return e;
}
template <typename T>
hipError_t prepare_bwd() {
  for (hipError_t e : {prepare_of<T, 32, false>(), prepare_of<T, 64, false>(), prepare_of<T, 96, false>(), prepare_of<T, 128, false>(),
                       prepare_of<T, 32, true>(), prepare_of<T, 64, true>(), prepare_of<T, 96, true>(), prepare_of<T, 128, true>()})
    if (e != hipSuccess) return e;
  return hipSuccess;
}

}  // namespace

hipError_t prepare_attention_grad() {
  const hipError_t e = prepare_bwd<Bf16>();
  return e != hipSuccess ? e : prepare_bwd<Half>();
}

hipError_t launch_attention_grad(const AttnGradArgs& g, const AttnGradWs& w, hipStream_t st) {
  return g.f.dtype == SVDQ_DT_BF16 ? launch_bwd<Bf16>(g, w, st) : launch_bwd<Half>(g, w, st);
}

}  // namespace svdq
