// Attention's gradients, the probabilities recomputed from the forward's lse:
//
//   p = exp(scale q k^T - lse),  delta = sum_d do o,  ds = p (do v^T - delta),
//   dv = p^T do,  dk = scale ds^T q,  dq = scale ds k.
//
// Two passes over the scores, each with its results in registers, so that no
// sum is joined by atomics and every order is fixed: one holds 32 NB keys a
// wave (dk, dv) while the query rows pass by in tiles of 64, one holds 32 NB
// query rows (dq) while the keys do. That is seven products instead of five,
// against a float of traffic per pair of a row and a tile of keys for joining
// dq. As in the forward, the products whose results are the next ones'
// operands are taken so that the held side is the columns, and the heads of a
// key head are rows of the same tiles, which sums a shared head's gradients.
//
// fp16 holds 2^-24 at least. Gradients and probabilities go well below that,
// so p enters its product times 2^10, and ds times the power of two that
// brings the largest value it could have, 2 D max|do| max|v|, to 2^15; both
// are taken out of the sums in fp32. bf16 has fp32's exponents and needs none.
#include <algorithm>

#include "svdq_attention.h"
#include "svdq_internal.h"
#include "svdq_layout.h"

namespace svdq {

namespace {

constexpr float kProbScale = 1024.f;   // of fp16 probabilities

template <typename T>
constexpr bool kScaled = !__is_same(T, Bf16);

// The largest magnitude of two packed values, as float bits, and m
template <typename T>
__device__ __forceinline__ float amax_x2(float m, uint32_t w) {
  if constexpr (__is_same(T, Bf16)) {
    return __builtin_fmaxf(m, __builtin_fmaxf(__builtin_fabsf(bf16lo(w)), __builtin_fabsf(bf16hi(w))));
  } else {
    const f16x2 v = __builtin_bit_cast(f16x2, w);
    return __builtin_fmaxf(m, __builtin_fmaxf(__builtin_fabsf((float)v[0]), __builtin_fabsf((float)v[1])));
  }
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

// Per query row, in the order of the tiles' rows: -lse / scale (-infinity for
// a row without keys, whose probabilities are then zero) and -delta, which the
// products' accumulators start with; the same up to whole tiles. Sixteen lanes a row. For fp16 also the
// largest |do| of each workgroup's rows and, by further workgroups, the
// largest |v| of runs of keys.
template <typename T>
__global__ __launch_bounds__(256) void attn_rows_kernel(AttnGradArgs g) {
  const AttnArgs& a = g.f;
  __shared__ float red[16];
  const int R = a.Lq * a.G, D = a.D, hb = blockIdx.y, b = hb / a.Hk, hk = hb % a.Hk;
  const int lane = threadIdx.x & 15, slot = threadIdx.x >> 4;
  float top = 0.f;
  if ((int)blockIdx.x < g.row_blocks) {
    const int64_t Rp = (int64_t)g.row_blocks * kAttnPrepRows;
#pragma unroll
    for (int k = 0; k < kAttnPrepRows / 16; ++k) {
      const int r = blockIdx.x * kAttnPrepRows + k * 16 + slot, i = r / a.G, head = hk * a.G + r - i * a.G;
      float s = 0.f;
      if (r < R && lane * 8 < D) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(static_cast<const T*>(g.dout.p) + b * g.dout.batch +
                                                        i * g.dout.token + head * g.dout.head + lane * 8);
        const u32x4 y = *reinterpret_cast<const u32x4*>(static_cast<const T*>(a.o.p) + b * a.o.batch + i * a.o.token +
                                                        head * a.o.head + lane * 8);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          s = dot_x2<T>(s, x[w], y[w]);
          if (kScaled<T>) top = amax_x2<T>(top, x[w]);
        }
      }
      s = add_dpp16(s);
      if (lane == 0) {
        const float lse = r < R ? a.lse[((int64_t)b * a.H + head) * a.Lq + i] : -__builtin_inff();
        const bool none = lse == -__builtin_inff();
        g.lse[hb * Rp + r] = none ? -__builtin_inff() : -lse / a.scale;
        g.delta[hb * Rp + r] = none ? 0.f : -s;
      }
    }
  } else if (kScaled<T>) {
    const int k0 = (blockIdx.x - g.row_blocks) * kAttnPrepRows;
#pragma unroll
    for (int k = 0; k < kAttnPrepRows / 16; ++k) {
      const int key = k0 + k * 16 + slot;
      if (key < a.Lk && lane * 8 < D && (!a.mask || a.mask[b * a.mask_batch + key])) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(static_cast<const T*>(a.v.p) + b * a.v.batch + key * a.v.token +
                                                        hk * a.v.head + lane * 8);
#pragma unroll
        for (int w = 0; w < 4; ++w) top = amax_x2<T>(top, x[w]);
      }
    }
  }
  if (!kScaled<T>) return;
  const uint32_t m = max_dpp16(__float_as_uint(top));   // (magnitudes: their bits are in order)
  if (lane == 0) red[slot] = __uint_as_float(m);
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = red[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) v = __builtin_fmaxf(v, red[i]);
    g.tops[(int64_t)hb * (g.row_blocks + g.key_blocks) + blockIdx.x] = v;
  }
}

// The power of two of a head's ds, from its largest |do| and |v|.
template <typename T>
__device__ __forceinline__ float ds_scale(const AttnGradArgs& g, int hb, int lane) {
  if constexpr (!kScaled<T>) return 1.f;
  if (g.row_blocks == 0) return 1.f;   // (no queries)
  const float* p = g.tops + (int64_t)hb * (g.row_blocks + g.key_blocks);
  float x = 0.f, y = 0.f;
  for (int i = lane; i < g.row_blocks + g.key_blocks; i += 64) {
    if (i < g.row_blocks)
      x = __builtin_fmaxf(x, p[i]);
    else
      y = __builtin_fmaxf(y, p[i]);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    x = __builtin_fmaxf(x, __shfl_xor(x, d));
    y = __builtin_fmaxf(y, __shfl_xor(y, d));
  }
  const float top = 2.f * (float)g.f.D * x * y;   // (at most 2^9 2^16 2^16)
  // 2^e > top >= 2^(e - 1): times 2^(15 - e) it is below 2^15
  if (!(top > 0.f) || !(top < 0x1p100f)) return 1.f;
  const int e = (int)(__float_as_uint(top) >> 23) - 126;
  return exp2_int(min(15 - e, 100));
}

// dk and dv of 32 NB keys a wave; the query rows pass by. With heads of 128
// the accumulators and the K fragments take 160 of the 256 registers that two
// waves a SIMD leave, so V's fragments wait in LDS (4608 tokens, 24 heads: 574
// us against 760 with V in registers, of which 53 spill, 768 with one wave a
// SIMD and two blocks of keys, 870 with workgroups of four waves).
template <typename T, int DP, int W, int NB>
__global__ __launch_bounds__(64 * W, 2) void attn_dkv_kernel(AttnGradArgs g) {
  typedef AttnTile<DP> TL;
  const AttnArgs& a = g.f;
  constexpr int NT = TL::kTransfers / W;
  __shared__ __align__(1024) uint8_t smem[2][2][TL::kBytes];
  constexpr bool kHoldV = DP == 64;   // in registers, else in LDS
  __shared__ __align__(1024) uint8_t held[kHoldV ? 16 : W * NB * 32 * TL::kRowBytes];
  __shared__ __align__(1024) float stats[2][2][kAttnRows];   // -lse / scale and -delta of a tile's rows
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, lr = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const AttnPlace at = attn_place(a, blockIdx.x, false);
  const int G = a.G, R = a.Lq * G, D = a.D;
  const int b = at.hb / a.Hk, hk = at.hb % a.Hk;
  const T* qp = static_cast<const T*>(a.q.p) + b * a.q.batch + (int64_t)hk * G * a.q.head;
  const T* dop = static_cast<const T*>(g.dout.p) + b * g.dout.batch + (int64_t)hk * G * g.dout.head;
  const int64_t Rp = (int64_t)g.row_blocks * kAttnPrepRows;
  const float *lse = g.lse + at.hb * Rp, *delta = g.delta + at.hb * Rp;
  const float c = ds_scale<T>(g, at.hb, lane), dsc = kScaled<T> ? c / kProbScale : 1.f;

  // this lane's keys, as operand B (of both products that give scores)
  const int key0 = at.block * (32 * NB * W) + wave * (32 * NB);
  u32x4 kf[NB][TL::kSteps], vf[kHoldV ? NB : 1][TL::kSteps];
  bool live[NB];
  int first[NB];   // the first row that sees the key
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int key = key0 + 32 * n + lr;
    live[n] = key < a.Lk && (!a.mask || a.mask[b * a.mask_batch + key]);
    first[n] = a.causal ? max(key - (a.Lk - a.Lq), 0) * G : 0;
    const T* kr = static_cast<const T*>(a.k.p) + b * a.k.batch + key * a.k.token + hk * a.k.head;
    const T* vr = static_cast<const T*>(a.v.p) + b * a.v.batch + key * a.v.token + hk * a.v.head;
#pragma unroll
    for (int s = 0; s < TL::kSteps; ++s) {
      const int d = 16 * s + 8 * h;
      const bool in = live[n] && d < D;
      kf[n][s] = in ? *reinterpret_cast<const u32x4*>(kr + d) : u32x4{0, 0, 0, 0};
      const u32x4 v = in ? *reinterpret_cast<const u32x4*>(vr + d) : u32x4{0, 0, 0, 0};
      if constexpr (kHoldV)
        vf[n][s] = v;
      else   // (read by this wave alone)
        *reinterpret_cast<u32x4*>(held + (wave * NB + n) * 32 * TL::kRowBytes + (typename TL::Lane(lane).straight ^ (s << 5))) = v;
    }
  }
  const uint8_t* my_v = held + (kHoldV ? 0 : wave * NB * 32 * TL::kRowBytes);
  // the rows of this workgroup: from its first key's first on, in its part of
  // the split. Rows that see no key at all are read as zeros.
  const int wg_key = at.block * (32 * NB * W);
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
  const int r_first = a.causal ? max(wg_key - (a.Lk - a.Lq), 0) * G : 0;
  const int r_begin = max(r_first / kAttnRows * kAttnRows, at.split * a.split_keys);
  const int r_end = min(R, (at.split + 1) * a.split_keys);
  const int tiles = r_end > r_begin ? (r_end - r_begin + kAttnRows - 1) / kAttnRows : 0;
  const int w_first = a.causal ? max(key0 - (a.Lk - a.Lq), 0) * G : 0;
  const int w_all = a.causal ? max(key0 + 32 * NB - 1 - (a.Lk - a.Lq), 0) * G : 0;   // from here on rows see all of the wave's keys

  auto fetch = [&](int row0, int stage) {
    const int i0 = row0 / G, i1 = min(row0 + kAttnRows - 1, R - 1) / G;
    // the heads of the queries i0 .. i1
    const auto rq = rows_resource(qp + i0 * a.q.token, (int)((i1 - i0) * a.q.token + (G - 1) * a.q.head + D) * 2);
    const auto rd = rows_resource(dop + i0 * g.dout.token, (int)((i1 - i0) * g.dout.token + (G - 1) * g.dout.head + D) * 2);
    uint8_t *tq = smem[stage][0] + wave * NT * 1024, *td = smem[stage][1] + wave * NT * 1024;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int j = wave * NT + n, ch = TL::chunk_of(j, lane), r = row0 + TL::row_of(j, lane);
      const int i = G == 1 ? r : r / G, hd = r - i * G;
      const bool in = r < R && r >= dead && ch * 8 < D;
      lds_transfer_16(rq, tq + n * 1024, in ? (uint32_t)(((i - i0) * a.q.token + hd * a.q.head + ch * 8) * 2) : kPastEnd);
      lds_transfer_16(rd, td + n * 1024, in ? (uint32_t)(((i - i0) * g.dout.token + hd * g.dout.head + ch * 8) * 2) : kPastEnd);
    }
    if (wave < 2) {   // (rows up to whole tiles are there)
      const auto rs = rows_resource((wave == 0 ? lse : delta) + row0, kAttnRows * 4);
      lds_transfer_4(rs, reinterpret_cast<uint8_t*>(stats[stage][wave]), lane * 4);
    }
  };

  f32x16 dk[TL::kBlocks][NB], dv[TL::kBlocks][NB];
#pragma unroll
  for (int i = 0; i < TL::kBlocks; ++i)
#pragma unroll
    for (int n = 0; n < NB; ++n) dk[i][n] = dv[i][n] = f32x16{};
  const typename TL::Lane pl(lane);
  if (tiles > 0) fetch(r_begin, 0);
  for (int t = 0, row0 = r_begin; t < tiles; ++t, row0 += kAttnRows) {
    tile_barrier();
    if (t + 1 < tiles) fetch(row0 + kAttnRows, (t + 1) & 1);
    const uint8_t *tq = smem[t & 1][0], *td = smem[t & 1][1];
    const float *tl = stats[t & 1][0], *tD = stats[t & 1][1];
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) {
      if (row0 + 32 * rb + 31 < w_first) continue;   // none of these rows sees a key of this wave
      // The scores' accumulators start with -lse / scale, those of do v^T with
      // -delta, each row's in its registers.
      f32x16 s[NB], dp[NB];
      u32x4 p[2][NB];
      auto start = [&](const float* rows, f32x16(&to)[NB]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(rows + 32 * rb + 8 * q + 4 * h);
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) to[n][4 * q + i] = v[i];
        }
      };
      const bool part = row0 + 32 * rb < w_all;
      start(tl, s);
#pragma unroll
      for (int st = 0; st < TL::kSteps; ++st) {
        const u32x4 qf = TL::straight(tq, pl, rb, st);
#pragma unroll
        for (int n = 0; n < NB; ++n) s[n] = mma<T>(qf, kf[n][st], s[n]);
      }
#pragma unroll
      for (int n = 0; n < NB; ++n) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[n][i] = __builtin_amdgcn_exp2f(kScaled<T> ? __builtin_fmaf(s[n][i], a.scale_log2, 10.f) : s[n][i] * a.scale_log2);
        if (part) {
          const int lim = first[n] - row0 - 32 * rb - 4 * h;
#pragma unroll
          for (int i = 0; i < 16; ++i) s[n][i] = 8 * (i / 4) + i % 4 >= lim ? s[n][i] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) p[u][n] = as_operand<T>(s[n], u);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < TL::kBlocks; ++i) {
          const u32x4 df = TL::turned(td, pl, 2 * rb + u, i);
#pragma unroll
          for (int n = 0; n < NB; ++n) dv[i][n] = mma<T>(df, p[u][n], dv[i][n]);
        }
      start(tD, dp);
#pragma unroll
      for (int st = 0; st < TL::kSteps; ++st) {
        const u32x4 df = TL::straight(td, pl, rb, st);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          if constexpr (kHoldV)
            dp[n] = mma<T>(df, vf[n][st], dp[n]);
          else
            dp[n] = mma<T>(df, TL::straight(my_v, pl, n, st), dp[n]);
        }
      }
#pragma unroll
      for (int n = 0; n < NB; ++n) {
#pragma unroll
        for (int i = 0; i < 16; ++i) dp[n][i] *= kScaled<T> ? s[n][i] * dsc : s[n][i];
        if (part) {   // (do may hold what times 0 is NaN)
          const int lim = first[n] - row0 - 32 * rb - 4 * h;
#pragma unroll
          for (int i = 0; i < 16; ++i) dp[n][i] = 8 * (i / 4) + i % 4 >= lim ? dp[n][i] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) p[u][n] = as_operand<T>(dp[n], u);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < TL::kBlocks; ++i) {
          const u32x4 qf = TL::turned(tq, pl, 2 * rb + u, i);
#pragma unroll
          for (int n = 0; n < NB; ++n) dk[i][n] = mma<T>(qf, p[u][n], dk[i][n]);
        }
    }
  }
  const float fv = kScaled<T> ? 1.f / kProbScale : 1.f, fk = a.scale / c;
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int key = key0 + 32 * n + lr;
    if (key >= a.Lk) continue;
    if (a.splits > 1) {
      float* row = a.part + (((int64_t)at.split * a.B * a.Hk + at.hb) * a.Lk + key) * 2 * D;
#pragma unroll
      for (int blk = 0; blk < TL::kBlocks; ++blk)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int d = 32 * blk + 8 * q + 4 * h;
          if (d >= D) continue;
          f32x4 x, y;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = live[n] ? dk[blk][n][4 * q + i] * fk : 0.f;
            y[i] = live[n] ? dv[blk][n][4 * q + i] * fv : 0.f;
          }
          *reinterpret_cast<f32x4*>(row + d) = x;
          *reinterpret_cast<f32x4*>(row + D + d) = y;
        }
      continue;
    }
    T* kr = static_cast<T*>(g.dk.p) + b * g.dk.batch + key * g.dk.token + hk * g.dk.head;
    T* vr = static_cast<T*>(g.dv.p) + b * g.dv.batch + key * g.dv.token + hk * g.dv.head;
#pragma unroll
    for (int blk = 0; blk < TL::kBlocks; ++blk) {
      u32x4 x[2], y[2];
      head_chunks<T>(dk[blk][n], fk, x);
      head_chunks<T>(dv[blk][n], fv, y);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int d = 32 * blk + 16 * q + 8 * h;
        if (d >= D) continue;
        *reinterpret_cast<u32x4*>(kr + d) = live[n] ? x[q] : u32x4{0, 0, 0, 0};   // (a dropped key has no gradient)
        *reinterpret_cast<u32x4*>(vr + d) = live[n] ? y[q] : u32x4{0, 0, 0, 0};
      }
    }
  }
}

// dq of 32 NB query rows a wave; the keys pass by, as in the forward (4608
// tokens, 24 heads of 128: 345 us, 1.13 PFLOP/s).
template <typename T, int DP, int W, int NB>
__global__ __launch_bounds__(64 * W, 2) void attn_dq_kernel(AttnGradArgs g) {
  typedef AttnTile<DP> TL;
  const AttnArgs& a = g.f;
  constexpr int NT = TL::kTransfers / W;
  __shared__ __align__(1024) uint8_t smem[2][2][TL::kBytes];
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, lr = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const AttnPlace at = attn_place(a, blockIdx.x, true);
  const int G = a.G, R = a.Lq * G, D = a.D;
  const int b = at.hb / a.Hk, hk = at.hb % a.Hk;
  const T* qp = static_cast<const T*>(a.q.p) + b * a.q.batch + (int64_t)hk * G * a.q.head;
  const T* dop = static_cast<const T*>(g.dout.p) + b * g.dout.batch + (int64_t)hk * G * g.dout.head;
  const T* kp = static_cast<const T*>(a.k.p) + b * a.k.batch + hk * a.k.head;
  const T* vp = static_cast<const T*>(a.v.p) + b * a.v.batch + hk * a.v.head;
  const uint8_t* mask = a.mask ? a.mask + b * a.mask_batch : nullptr;
  const int64_t Rp = (int64_t)g.row_blocks * kAttnPrepRows;
  const float c = ds_scale<T>(g, at.hb, lane);

  const int r0 = at.block * (32 * NB * W) + wave * (32 * NB);
  u32x4 qf[NB][TL::kSteps], df[NB][TL::kSteps];
  int last[NB];
  float lse[NB], delta[NB];   // both negative
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int r = r0 + 32 * n + lr, i = r / G, hd = r - i * G;
    last[n] = r >= R ? -1 : a.causal ? min(i + a.Lk - a.Lq, a.Lk - 1) : a.Lk - 1;
    lse[n] = r < R ? g.lse[at.hb * Rp + r] * a.scale_log2 : -__builtin_inff();   // in base 2
    delta[n] = r < R ? g.delta[at.hb * Rp + r] : 0.f;
#pragma unroll
    for (int s = 0; s < TL::kSteps; ++s) {
      const int d = 16 * s + 8 * h;
      const bool in = r < R && d < D;
      qf[n][s] = in ? *reinterpret_cast<const u32x4*>(qp + i * a.q.token + hd * a.q.head + d) : u32x4{0, 0, 0, 0};
      df[n][s] = in ? *reinterpret_cast<const u32x4*>(dop + i * g.dout.token + hd * g.dout.head + d) : u32x4{0, 0, 0, 0};
    }
  }
  const int r_end = min(R, (at.block + 1) * (32 * NB * W));
  int k_end = a.causal ? min(a.Lk, (r_end - 1) / G + a.Lk - a.Lq + 1) : a.Lk;
  k_end = min(k_end, (at.split + 1) * a.split_keys);
  const int k_begin = at.split * a.split_keys;
  const int tiles = k_end > k_begin ? (k_end - k_begin + kAttnRows - 1) / kAttnRows : 0;
  const int w_first = a.causal ? r0 / G + a.Lk - a.Lq : a.Lk - 1;
  const int w_last = r0 >= R ? -1 : a.causal ? (min(r0 + 32 * NB, R) - 1) / G + a.Lk - a.Lq : a.Lk - 1;

  uint32_t vk[NT], vv[NT];
  int row_of[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int j = wave * NT + n, ch = TL::chunk_of(j, lane);
    row_of[n] = TL::row_of(j, lane);
    vk[n] = ch * 8 < D ? (uint32_t)((row_of[n] * a.k.token + ch * 8) * 2) : kPastEnd;
    vv[n] = ch * 8 < D ? (uint32_t)((row_of[n] * a.v.token + ch * 8) * 2) : kPastEnd;
  }
  auto fetch = [&](int k0, int stage, uint64_t keep) {
    const int rows = min(kAttnRows, a.Lk - k0);
    const auto rk = rows_resource(kp + k0 * a.k.token, (int)((rows - 1) * a.k.token + D) * 2);
    const auto rv = rows_resource(vp + k0 * a.v.token, (int)((rows - 1) * a.v.token + D) * 2);
    uint8_t *tk = smem[stage][0] + wave * NT * 1024, *tv = smem[stage][1] + wave * NT * 1024;
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

  f32x16 dq[TL::kBlocks][NB];
#pragma unroll
  for (int i = 0; i < TL::kBlocks; ++i)
#pragma unroll
    for (int n = 0; n < NB; ++n) dq[i][n] = f32x16{};
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
    if (k0 > w_last || keep == 0) continue;
    const uint8_t *tk = smem[t & 1][0], *tv = smem[t & 1][1];
    const bool part = keep != ~0ull || k0 + kAttnRows - 1 > w_first;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      f32x16 s[NB], dp[NB];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        s[n] = f32x16{};
#pragma unroll
        for (int i = 0; i < 16; ++i) dp[n][i] = delta[n];
      }
#pragma unroll
      for (int st = 0; st < TL::kSteps; ++st) {
        const u32x4 f = TL::straight(tk, pl, kb, st);
#pragma unroll
        for (int n = 0; n < NB; ++n) s[n] = mma<T>(f, qf[n][st], s[n]);
      }
#pragma unroll
      for (int st = 0; st < TL::kSteps; ++st) {
        const u32x4 f = TL::straight(tv, pl, kb, st);
#pragma unroll
        for (int n = 0; n < NB; ++n) dp[n] = mma<T>(f, df[n][st], dp[n]);
      }
      u32x4 ds[2][NB];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][i], a.scale_log2, lse[n]));
          dp[n][i] *= kScaled<T> ? p * c : p;
        }
        if (part) {
          const int lim = last[n] - k0 - 32 * kb - 4 * h;
          const uint32_t bits = (uint32_t)(keep >> (32 * kb)) >> (4 * h);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int at_key = 8 * (i / 4) + i % 4;
            dp[n][i] = (bits >> at_key & 1) && at_key <= lim ? dp[n][i] : 0.f;
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) ds[u][n] = as_operand<T>(dp[n], u);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < TL::kBlocks; ++i) {
          const u32x4 f = TL::turned(tk, pl, 2 * kb + u, i);
#pragma unroll
          for (int n = 0; n < NB; ++n) dq[i][n] = mma<T>(f, ds[u][n], dq[i][n]);
        }
    }
  }
  const float f = a.scale / c;
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int r = r0 + 32 * n + lr, i = r / G, hd = hk * G + r - i * G;
    if (r >= R) continue;
    if (a.splits > 1) {
      float* row = a.part + (((int64_t)at.split * a.B * a.Hk + at.hb) * R + r) * D;
#pragma unroll
      for (int blk = 0; blk < TL::kBlocks; ++blk)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int d = 32 * blk + 8 * q + 4 * h;
          if (d < D)
            *reinterpret_cast<f32x4*>(row + d) = f32x4{dq[blk][n][4 * q], dq[blk][n][4 * q + 1], dq[blk][n][4 * q + 2],
                                                       dq[blk][n][4 * q + 3]} * f;
        }
      continue;
    }
    T* row = static_cast<T*>(g.dq.p) + b * g.dq.batch + i * g.dq.token + hd * g.dq.head;
#pragma unroll
    for (int blk = 0; blk < TL::kBlocks; ++blk) {
      u32x4 x[2];
      head_chunks<T>(dq[blk][n], f, x);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int d = 32 * blk + 16 * q + 8 * h;
        if (d < D) *reinterpret_cast<u32x4*>(row + d) = x[q];
      }
    }
  }
}

// The parts' sums added in order, a wave half a row: rows of dq, or of dk and
// dv side by side.
template <typename T>
__global__ __launch_bounds__(256) void attn_grad_join_kernel(AttnGradArgs g, int keys) {
  const AttnArgs& a = g.f;
  const int n = keys ? a.Lk : a.Lq * a.G, width = keys ? 2 * a.D : a.D, lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.B * a.Hk * n, row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int hb = (int)(row / n), r = (int)(row % n), b = hb / a.Hk, hk = hb % a.Hk, i = r / a.G;
  for (int d = lane * 4; d < width; d += 128) {
    f32x4 v = *reinterpret_cast<const f32x4*>(a.part + row * width + d);
    for (int s = 1; s < a.splits; ++s) v += *reinterpret_cast<const f32x4*>(a.part + (s * rows + row) * width + d);
    T* to;
    if (!keys)
      to = static_cast<T*>(g.dq.p) + b * g.dq.batch + i * g.dq.token + (hk * a.G + r - i * a.G) * g.dq.head + d;
    else if (d < a.D)
      to = static_cast<T*>(g.dk.p) + b * g.dk.batch + r * g.dk.token + hk * g.dk.head + d;
    else
      to = static_cast<T*>(g.dv.p) + b * g.dv.batch + r * g.dv.token + hk * g.dv.head + d - a.D;
    *reinterpret_cast<u32x2*>(to) = u32x2{cvt_x2<T>(v[0], v[1]), cvt_x2<T>(v[2], v[3])};
  }
}

template <typename T>
hipError_t launch_bwd(const AttnGradArgs& args, const AttnGradPlan& plan, hipStream_t st) {
  AttnGradArgs g = args;
  const dim3 block(256);
  const int heads = g.f.B * g.f.Hk;
  hipError_t e;
  if (g.row_blocks > 0) {   // (no queries: dk and dv are zeros)
    hipLaunchKernelGGL((attn_rows_kernel<T>), dim3((unsigned)(g.row_blocks + g.key_blocks), (unsigned)heads), block, 0, st, g);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  for (int keys = 1; keys >= 0; --keys) {
    const AttnSplit& s = keys ? plan.dkv : plan.dq;
    if (s.blocks == 0) continue;
    g.f.blocks = s.blocks;
    g.f.splits = s.splits;
    g.f.split_keys = s.each;
    const dim3 grid((unsigned)(s.blocks * s.splits * heads));
    if (keys && g.f.D <= 64)
      hipLaunchKernelGGL((attn_dkv_kernel<T, 64, 8, 1>), grid, dim3(512), 0, st, g);
    else if (keys)
      hipLaunchKernelGGL((attn_dkv_kernel<T, 128, 8, 1>), grid, dim3(512), 0, st, g);
    else if (g.f.D <= 64)
      hipLaunchKernelGGL((attn_dq_kernel<T, 64, 8, 1>), grid, dim3(512), 0, st, g);
    else
      hipLaunchKernelGGL((attn_dq_kernel<T, 128, 8, 1>), grid, dim3(512), 0, st, g);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (s.splits > 1) {
      const int64_t rows = (int64_t)heads * (keys ? g.f.Lk : g.f.Lq * g.f.G);
      hipLaunchKernelGGL((attn_grad_join_kernel<T>), dim3((unsigned)((rows + 7) / 8)), block, 0, st, g, keys);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_attention_grad(const AttnGradArgs& g, const AttnGradPlan& plan, hipStream_t st) {
  return g.f.dtype == SVDQ_DT_BF16 ? launch_bwd<Bf16>(g, plan, st) : launch_bwd<Half>(g, plan, st);
}

}  // namespace svdq
