// Layer norm of rows, affine or modulated per group of rows, and its
// gradients. With g the row's gain (1, weight or 1 + weight) and b its bias,
//
//   mean = sum_c x / C,  rstd = (sum_c (x - mean)^2 / C + eps)^(-1/2)
//   xhat = (x - mean) rstd,  y = xhat g + b
//   d = dy g,  dx = rstd (d - mean_c(d) - xhat mean_c(d xhat))
//   dweight = sum over the group's rows of dy xhat,  dbias = sum of dy.
//
// Both passes are bound by memory: one read of x (and dy), one write of y
// (dx). A team of lanes holds a row in registers, up to 16 elements a lane, so
// the two-pass variance (which keeps its digits when |mean| is far above the
// deviation) and the backward's two sums cost no second read: a quarter or
// half wave, a wave, or up to sixteen waves, with the next row's loads in
// flight. All sums are in fp32: per lane, then a fixed butterfly over the
// wave, then the waves in order. 9216 x 3072 bf16 takes 23.1 us forward and
// 34.8 backward, 4.9 TB/s both, as a large copy does.
#include <algorithm>

#include "svdq_internal.h"
#include "svdq_layout.h"
#include "svdq_types.h"

namespace svdq {

namespace {

constexpr int kMaxWaves = kNormWaves;

// Sums over a team for n rows at once, the same in each of its lanes: LANES
// of a wave, or W whole waves (first .. first + W - 1 of the workgroup). The
// caller alternates two areas, so one barrier per call is enough.
template <int n, int LANES>
__device__ __forceinline__ void team_sum(float (&v)[n], float (*red)[n], int wave, int first, int W, int lane) {
#pragma unroll
  for (int r = 0; r < n; ++r) v[r] = lanes_sum<LANES>(v[r]);
  if (LANES < 64 || W == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int r = 0; r < n; ++r) red[wave][r] = v[r];
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < n; ++r) {
    float s = red[first][r];
    for (int w = 1; w < W; ++w) s += red[first + w][r];
    v[r] = s;
  }
}

// Where this lane's vectors of a row lie: NV of them, TH vectors apart. Only
// the last can end the row (the launches choose no more vectors than needed).
template <int NV, int VEC>
struct Place {
  Window<VEC> last;
  int first, step;
  bool in_row;   // the last vector holds elements of its own
  __device__ __forceinline__ Place(int tid, int TH, int C)
      : last(window<VEC>((tid + (NV - 1) * TH) * VEC, C)), first(tid * VEC), step(TH * VEC),
        in_row((tid + (NV - 1) * TH) * VEC < C) {}
  __device__ __forceinline__ int at(int j) const { return j == NV - 1 ? last.at : first + j * step; }
  __device__ __forceinline__ int len(int j) const { return j == NV - 1 ? last.len : VEC; }
};

template <int NV, int VEC>
__device__ __forceinline__ void load_gain(const NormArgs& a, int64_t group, const Place<NV, VEC>& pl, float (&gain)[NV][VEC]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (a.w) {
      load_params<VEC>(a.w, a.pdtype, group * a.ldw, pl.at(j), pl.len(j), gain[j]);
      if (a.one_plus) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) gain[j][i] += 1.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) gain[j][i] = 1.f;
    }
  }
}

// Forward. Teams of 64 / SUB lanes, or of W waves (SUB = 1), take consecutive
// rows. QUANT: instead of y, its bf16 values' E4M3 codes and the
// scales of their blocks of 128 (sixteen lanes of a wave hold a block) in the
// layout of the FP8 product's operand.
template <typename T, int NV, int SUB, bool QUANT>
__global__ __launch_bounds__(64 * kMaxWaves) void norm_fwd_kernel(NormArgs a, int W, int per, int extra) {
  constexpr int VEC = kVec<T>, LANES = 64 / SUB;
  __shared__ float red[2][2][kMaxWaves][1];
  const int lane = threadIdx.x & 63, wg_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wg_teams = W == 1 ? (int)(blockDim.x >> 6) * SUB : 1;
  const int local = W > 1 ? 0 : SUB == 1 ? wg_wave : (int)threadIdx.x / LANES;
  const int TH = LANES * W, tid = W > 1 ? (int)threadIdx.x : (int)threadIdx.x % LANES;
  // team t's rows: per or, of the first `extra` teams, per + 1
  const int team = (int)blockIdx.x * wg_teams + local, C = a.C, last_row = (int)a.M - 1;
  const int m_begin = team * per + min(team, extra), m_end = min(m_begin + per + (team < extra ? 1 : 0), last_row + 1);
  const int steps = per + (extra > 0 ? 1 : 0);   // of every team (a barrier is the workgroup's)
  const float fc = (float)C;
  if constexpr (QUANT) {
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i < kFp8Tickets; i += blockDim.x) a.tickets[i] = 0;
  }
  const Place<NV, VEC> pl(tid, TH, C);
  Vec<T> next[NV];
  auto fetch = [&](int m) {
    const T* row = static_cast<const T*>(a.x) + min(m, last_row) * a.ldx;   // (a row past the team's is not used)
#pragma unroll
    for (int j = 0; j < NV; ++j) next[j] = load_vec<T>(row, pl.at(j), pl.len(j));
  };
  fetch(m_begin);
  float gain[NV][VEC], shift[NV][VEC];
  int64_t group_end;   // where the loaded group's rows end
  auto load_group = [&](int m) {
    const int64_t group = (uint32_t)m / (uint32_t)a.rpg;
    group_end = (group + 1) * a.rpg;
    load_gain(a, group, pl, gain);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (a.b) {
        load_params<VEC>(a.b, a.pdtype, group * a.ldb, pl.at(j), pl.len(j), shift[j]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) shift[j][i] = 0.f;
      }
    }
  };
  load_group(min(m_begin, last_row));
  for (int k = 0, m = m_begin; k < steps; ++k, ++m) {
    float v[NV][VEC], mean[1] = {0.f}, rstd[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j][i] = next[j].at(i);
    if (k + 1 < steps) fetch(m + 1);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) mean[0] += j == NV - 1 ? own_or_0(v[j][i], pl.last.own[i]) : v[j][i];
    team_sum<1, LANES>(mean, red[k & 1][0], wg_wave, 0, W, lane);
    mean[0] /= fc;   // (the division, correctly rounded: a constant row has its value as mean)
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[j][i] -= mean[0];
        const float d = j == NV - 1 ? own_or_0(v[j][i], pl.last.own[i]) : v[j][i];
        rstd[0] = __builtin_fmaf(d, d, rstd[0]);
      }
    team_sum<1, LANES>(rstd, red[k & 1][1], wg_wave, 0, W, lane);
    if (m >= m_end) continue;   // (its lanes take part in the next step's sums, if there is one)
    const float rs = 1.0f / __builtin_sqrtf(rstd[0] / fc + a.eps);
    if (m >= group_end) load_group(m);
    if (tid == 0) {
      if (a.mean) a.mean[m] = mean[0];
      if (a.rstd) a.rstd[m] = rs;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = __builtin_fmaf(v[j][i] * rs, gain[j][i], shift[j][i]);
      Vec<T> y;
      y.set(o);
      if constexpr (!QUANT) {
        if (j < NV - 1 || pl.in_row) store_vec<T>(static_cast<T*>(a.y) + m * a.ldy, pl.at(j), pl.len(j), y);
      } else {
        // channels past the row (C is a multiple of 16) are zero codes
        const int c = (tid + j * TH) * VEC;
        u32x4 w = y.w;
        if (c >= C) w = u32x4{0, 0, 0, 0};
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = amax_bf16x2(amax, w[i]);
        const int e = e4m3_exponent(max_dpp16(amax));
        const float sc = exp2_int(e);
        const u32x2 q = u32x2{e4m3x4(bf16lo(w[0]), bf16hi(w[0]), bf16lo(w[1]), bf16hi(w[1]), sc),
                              e4m3x4(bf16lo(w[2]), bf16hi(w[2]), bf16lo(w[3]), bf16hi(w[3]), sc)};
        if (c < a.Kp) {
          *reinterpret_cast<u32x2*>(a.q + (size_t)m * a.Kp + c) = q;
          if ((lane & 15) == 0) a.qs[fp8_scale_index(a.qs_rows, m, c / 128)] = (uint8_t)(e + 127);
        }
      }
    }
  }
}

// Backward: dx of a run of rows of one group, and the run's sums of dy xhat
// and dy per channel. A workgroup is a run's teams, which take its rows in
// turn; a lane keeps its channels' sums over its rows, the teams' are added in
// order through LDS at the end, and written once: to the workspace
// [run][2][C] in fp32, or, where a group is one run, as the gradients.
template <typename T, int NV, int SUB, int MAXW>
__global__ __launch_bounds__(64 * MAXW) void norm_bwd_kernel(NormGradArgs g, int W, int runs) {
  constexpr int VEC = kVec<T>, LANES = 64 / SUB;
  const NormArgs& a = g.f;
  extern __shared__ float sums[];   // [team or wave][2][VEC][NV][TH]
  __shared__ float red[2][MAXW][2];
  const int lane = threadIdx.x & 63, wg_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int TH = LANES * W, teams = (int)blockDim.x / TH;
  const int team = SUB == 1 ? wg_wave / W : (int)threadIdx.x / LANES, tid = (int)threadIdx.x - team * TH;
  const uint32_t block = blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= (uint32_t)a.G * (uint32_t)runs) return;
  const int64_t group = block / (uint32_t)runs;
  const int run = (int)(block % (uint32_t)runs), C = a.C;
  // the group's rows in `runs` parts as even as they can be
  const int64_t g_begin = min(group * a.rpg, a.M), g_rows = min(a.rpg, a.M - g_begin);
  const int per = (int)((uint32_t)g_rows / (uint32_t)runs), extra = (int)((uint32_t)g_rows % (uint32_t)runs);
  const int m_begin = (int)g_begin + run * per + min(run, extra), m_end = m_begin + per + (run < extra ? 1 : 0);
  const float fc = (float)C;
  const Place<NV, VEC> pl(tid, TH, C);
  float gain[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) dw[j][i] = db[j][i] = 0.f;
  Vec<T> nx[NV], ndy[NV];
  float nmean = 0.f, nrstd = 0.f;
  auto fetch = [&](int m) {
    m = min(m, m_end - 1);   // past the end: the last row again, not used
    const T *x = static_cast<const T*>(a.x) + m * a.ldx, *dy = static_cast<const T*>(g.dy) + m * g.lddy;
    if (g.once) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        nx[j] = load_vec<T, true>(x, pl.at(j), pl.len(j));
        ndy[j] = load_vec<T, true>(dy, pl.at(j), pl.len(j));
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        nx[j] = load_vec<T>(x, pl.at(j), pl.len(j));
        ndy[j] = load_vec<T>(dy, pl.at(j), pl.len(j));
      }
    }
    nmean = a.mean[m];
    nrstd = a.rstd[m];
  };
  if (m_begin < m_end) {
    fetch(m_begin + team);
    load_gain(a, group, pl, gain);
  }
  int flip = 0;
  // every team makes the same steps (a barrier is the workgroup's)
  for (int base = m_begin; base < m_end; base += teams, flip ^= 1) {
    const int m = base + team;
    float d[NV][VEC], xhat[NV][VEC], s[2] = {0.f, 0.f};
    const float rstd = nrstd;
    const bool live = m < m_end;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float t = ndy[j].at(i);
        xhat[j][i] = (nx[j].at(i) - nmean) * rstd;
        d[j][i] = t * gain[j][i];
        const float own = j == NV - 1 ? own_or_0(d[j][i], pl.last.own[i]) : d[j][i];
        const float own_x = j == NV - 1 ? own_or_0(xhat[j][i], pl.last.own[i]) : xhat[j][i];
        s[0] += own;
        s[1] = __builtin_fmaf(own, own_x, s[1]);
        if (live) {
          dw[j][i] = __builtin_fmaf(t, xhat[j][i], dw[j][i]);
          db[j][i] += t;
        }
      }
    if (base + teams < m_end) fetch(m + teams);
    team_sum<2, LANES>(s, red[flip], wg_wave, team * W, W, lane);
    if (!live) continue;   // (the last step)
    const float a1 = -(s[0] / fc) * rstd, a2 = -(s[1] / fc) * rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = __builtin_fmaf(d[j][i], rstd, __builtin_fmaf(xhat[j][i], a2, a1));
      Vec<T> o;
      o.set(v);
      if (j < NV - 1 || pl.in_row) store_vec<T>(static_cast<T*>(g.dx) + m * g.lddx, pl.at(j), pl.len(j), o);
    }
  }
  if (!g.dw && !g.db) return;
  // The sums of the teams that share a wave, then the others' through LDS, a
  // plane per team (or wave) and gradient: element i of
  // vector j of lane tid at (i NV + j) TH + tid, so that consecutive lanes
  // write, and read, consecutive words.
  const int plane = VEC * NV * TH;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      dw[j][i] = shares_sum<SUB>(dw[j][i]);
      db[j][i] = shares_sum<SUB>(db[j][i]);
      float* p = sums + (team / SUB) * 2 * plane + (i * NV + j) * TH + tid;
      if (team % SUB == 0) {
        p[0] = dw[j][i];
        p[plane] = db[j][i];
      }
    }
  __syncthreads();
  const int n = (C + VEC - 1) / VEC, len = min(C, VEC);
  for (int e = threadIdx.x; e < 2 * n; e += blockDim.x) {   // vector e of dweight, then of dbias
    const int second = e >= n, vec = e - (second ? n : 0), at = C < VEC ? 0 : min(vec * VEC, C - VEC);
    int j = 0;
#pragma unroll
    for (int k = 1; k < NV; ++k) j += vec >= k * TH;
    const float* p = sums + second * plane + j * TH + (vec - j * TH);
    float v[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = p[i * NV * TH];
    for (int t = 1; t < teams / SUB; ++t) {
      p += 2 * plane;
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] += p[i * NV * TH];
    }
    if (g.part) {
      store_params<VEC>(g.part, SVDQ_DT_F32, ((int64_t)block * 2 + second) * C + at, len, v);
    } else {
      void* o = second ? g.db : g.dw;
      if (o) store_params<VEC>(o, g.gdtype, group * C + at, len, v);
    }
  }
}

// The runs' sums of a group added per channel: 32 threads a channel, each
// every 32nd run in order (all its loads at once: there are few workgroups,
// so this is latency), then the 32 in order.
__global__ __launch_bounds__(1024) void norm_param_grad_kernel(NormGradArgs g, int runs) {
  __shared__ float red[32][33];
  const int C = g.f.C, cl = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cl;   // 0 .. 2 C: dweight's channels, then dbias's
  const int64_t group = blockIdx.y;
  const float* p = g.part + (size_t)group * runs * 2 * C;
  float v[kNormRuns / 32], s = 0.f;
#pragma unroll
  for (int i = 0; i < kNormRuns / 32; ++i) v[i] = c < 2 * C && k + 32 * i < runs ? p[(size_t)(k + 32 * i) * 2 * C + c] : 0.f;
#pragma unroll
  for (int i = 0; i < kNormRuns / 32; ++i) s += v[i];
  red[k][cl] = s;
  __syncthreads();
  if (k == 0 && c < 2 * C) {
    float t = red[0][cl];
#pragma unroll
    for (int i = 1; i < 32; ++i) t += red[i][cl];
    void* o = c < C ? g.dw : g.db;
    if (o) store_param(o, g.gdtype, group * C + (c < C ? c : c - C), t);
  }
}

#define SVDQ_NORM_LAUNCH(KERNEL, ...)                                                 \
  if (t.sub == 4)                                                                     \
    hipLaunchKernelGGL((KERNEL(1, 4)), grid, block, lds, st, __VA_ARGS__);            \
  else if (t.sub == 2)                                                                \
    hipLaunchKernelGGL((KERNEL(1, 2)), grid, block, lds, st, __VA_ARGS__);            \
  else if (t.nv == 1)                                                                 \
    hipLaunchKernelGGL((KERNEL(1, 1)), grid, block, lds, st, __VA_ARGS__);            \
  else if (t.nv == 2)                                                                 \
    hipLaunchKernelGGL((KERNEL(2, 1)), grid, block, lds, st, __VA_ARGS__);            \
  else if constexpr (kVec<T> == 4) {                                                  \
    if (t.nv == 3)                                                                    \
      hipLaunchKernelGGL((KERNEL(3, 1)), grid, block, lds, st, __VA_ARGS__);          \
    else                                                                              \
      hipLaunchKernelGGL((KERNEL(4, 1)), grid, block, lds, st, __VA_ARGS__);          \
  }                                                                                   \
  return hipGetLastError();

// The forward's teams are all resident at once, with as even a share of the
// rows as there can be (9216 x 3072 bf16 into twelve outputs in turn: 27.1 us;
// with up to 32 waves a CU asked for, of which 20 fit, 29.6 us).
template <typename T, bool QUANT>
hipError_t launch_fwd(const NormArgs& a, int num_cus, hipStream_t st) {
  const int span = QUANT ? a.Kp : a.C;
  const NormTeam t = norm_team((span + kVec<T> - 1) / kVec<T>, kVec<T>, !QUANT);
  const int e = t.nv * kVec<T>, fit = e <= 12 ? 24 : kVec<T> == 8 ? 20 : 16;   // waves of a CU that its registers hold
  const int wg_waves = t.waves == 1 ? 4 : t.waves, wg_teams = t.waves == 1 ? 4 * t.sub : 1;
  const int64_t M = a.M, most = (int64_t)num_cus * (fit / wg_waves);
  const int64_t wgs = std::min(most, (M + wg_teams - 1) / wg_teams), all = wgs * wg_teams;
  const dim3 grid((unsigned)wgs), block(64 * wg_waves);
  const int per = (int)(M / all), extra = (int)(M % all);
  const size_t lds = 0;
#define SVDQ_FWD(NV, SUB) norm_fwd_kernel<T, NV, SUB, QUANT>
  SVDQ_NORM_LAUNCH(SVDQ_FWD, a, t.waves, per, extra)
#undef SVDQ_FWD
}

constexpr int kNormLds = kMaxWaves * 64 * 16 * 2 * 4;   // a workgroup's teams' sums at most
template <typename T, int NV>
constexpr int kBwdWaves = norm_grad_waves(NV * kVec<T>);

template <typename T>
hipError_t launch_bwd(const NormGradArgs& g, const NormGradPlan& p, hipStream_t st) {
  constexpr int kWide = 16 / kVec<T>;
  const NormTeam t = norm_team((g.f.C + kVec<T> - 1) / kVec<T>, kVec<T>, true);
  // a workgroup's teams: as many as have rows and fit
  const int64_t useful = (p.rows_per_run + t.sub - 1) / t.sub;
  const int wg_teams = (int)std::min<int64_t>(norm_grad_teams(t, kVec<T>) / t.sub, useful) * t.sub;
  const int th = t.waves * 64 / t.sub;
  const dim3 grid = many_groups((int64_t)g.f.G * p.runs), block(th * wg_teams);
  const size_t lds = g.dw || g.db ? (size_t)wg_teams / t.sub * 2 * kVec<T> * t.nv * th * 4 : 0;
  if (t.waves > norm_grad_waves(t.nv * kVec<T>)) {
    hipLaunchKernelGGL((norm_bwd_kernel<T, kWide, 1, kMaxWaves>), grid, block, lds, st, g, t.waves, p.runs);
    return hipGetLastError();
  }
#define SVDQ_BWD(NV, SUB) norm_bwd_kernel<T, NV, SUB, kBwdWaves<T, NV>>
  SVDQ_NORM_LAUNCH(SVDQ_BWD, g, t.waves, p.runs)
#undef SVDQ_BWD
}

template <typename T>
hipError_t prepare_bwd() {
  constexpr int kWide = 16 / kVec<T>, kMid = kWide - kWide / 4;   // (16-bit types: both 2)
  const void* all[] = {(const void*)norm_bwd_kernel<T, 1, 4, kBwdWaves<T, 1>>, (const void*)norm_bwd_kernel<T, 1, 2, kBwdWaves<T, 1>>,
                       (const void*)norm_bwd_kernel<T, 1, 1, kBwdWaves<T, 1>>, (const void*)norm_bwd_kernel<T, 2, 1, kBwdWaves<T, 2>>,
                       (const void*)norm_bwd_kernel<T, kMid, 1, kBwdWaves<T, kMid>>,
                       (const void*)norm_bwd_kernel<T, kWide, 1, kBwdWaves<T, kWide>>,
                       (const void*)norm_bwd_kernel<T, kWide, 1, kMaxWaves>};
  for (const void* f : all) {
    const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, kNormLds);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t prepare_norm() {
  for (hipError_t e : {prepare_bwd<float>(), prepare_bwd<Bf16>(), prepare_bwd<Half>()})
    if (e != hipSuccess) return e;
  return hipSuccess;
}

hipError_t launch_norm(const NormArgs& a, int num_cus, hipStream_t st) {
  if (a.q) return launch_fwd<Bf16, true>(a, num_cus, st);
  if (a.dtype == SVDQ_DT_F32) return launch_fwd<float, false>(a, num_cus, st);
  if (a.dtype == SVDQ_DT_BF16) return launch_fwd<Bf16, false>(a, num_cus, st);
  return launch_fwd<Half, false>(a, num_cus, st);
}

hipError_t launch_norm_grad(const NormGradArgs& args, const NormGradPlan& p, hipStream_t st) {
  // What the caches (256 MB) cannot keep until it is used again is read past
  // them: from 128 MB of x, dy and dx on (9216 x 3072 bf16, 170 MB: 34.4 us
  // against 38.1, 3000 x 9000 bf16, 162 MB: 41.5 against 43.3; 16387 x 517
  // fp32, 102 MB: 21.6 either way; inputs rotating through three sets).
  NormGradArgs g = args;
  g.once = (double)g.f.M * g.f.C * 3 * (g.f.dtype == SVDQ_DT_F32 ? 4 : 2) > 128e6;
  const hipError_t e = g.f.dtype == SVDQ_DT_F32    ? launch_bwd<float>(g, p, st)
                       : g.f.dtype == SVDQ_DT_BF16 ? launch_bwd<Bf16>(g, p, st)
                                                   : launch_bwd<Half>(g, p, st);
  if (e != hipSuccess || !g.part) return e;
  hipLaunchKernelGGL(norm_param_grad_kernel, dim3((2 * g.f.C + 31) / 32, (unsigned)g.f.G), dim3(1024), 0, st, g, p.runs);
  return hipGetLastError();
}

}  // namespace svdq
