// The gated residual with the norms around it, and its gradients. Of a row's
// stream x and a block's output h, with norm(v) = (v - mean) rstd, or v rstd
// (rms),
//
//   hn = h, or norm(h) gp;  s = alpha x + gate hn, rounded;  y = norm(s) g + b
//
//   t = ds + rstd (d - mean_c(d) - shat mean_c(d shat)),  d = dy g
//   dx = alpha t,  dgate = sum t hn,  dg = sum dy shat,  db = sum dy
//   dh = t gate, or with e = t gate:  dgp = sum e hhat,
//   dh = rstd_h (e gp - mean_c(e gp) - hhat mean_c(e gp hhat))
//
// (rms: without the first mean of each). Bound by memory: the forward reads x
// and h and writes s and y, the backward reads s, h, dy and ds and writes dx
// and dh, each once (8192 x 4096 bf16, calls with three sets of inputs in turn:
// 58.5 us, 4.6 TB/s, and 80, 5.0; fp32 8192 x 2048: 47, 5.8, and 75, 5.4). A team
// of lanes holds a row in registers, so the chained sums (up to four) cost no
// second read; the next row's loads are in flight. All sums are in fp32, in an
// order fixed by the sizes: per lane, a butterfly over the wave, the waves in
// order; the parameters' over a run's rows per lane, then the teams and the
// runs in order.
#include <algorithm>
#include <type_traits>

#include "svdq_internal.h"
#include "svdq_layout.h"
#include "svdq_types.h"

namespace svdq {

namespace {

constexpr int kMaxWaves = 16;

// Sums over a team, the same in each of its lanes. The caller alternates
// areas, so one barrier per call is enough.
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
// the last can end the row.
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
  // the lane's own elements for a sum
  __device__ __forceinline__ float own(int j, int i, float v) const { return j == NV - 1 ? own_or_0(v, last.own[i]) : v; }
};

// a group's parameter, `fill` where there is none, plus `add`
template <int NV, int VEC>
__device__ __forceinline__ void load_param(const void* p, int dtype, int64_t row, const Place<NV, VEC>& pl, float fill, float add,
                                           float (&o)[NV][VEC]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (p) {
      load_params<VEC>(p, dtype, row, pl.at(j), pl.len(j), o[j]);
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[j][i] += add;
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[j][i] = fill;
    }
  }
}

// Forward. Teams of 64 / SUB lanes, or of W waves (SUB = 1), take consecutive
// rows: per or, of the first `extra` teams, per + 1.
template <typename T, int NV, int SUB, bool POST>
__global__ __launch_bounds__(64 * kMaxWaves) void residual_fwd_kernel(ResidualArgs a, int W, int per, int extra) {
  constexpr int VEC = kVec<T>, LANES = 64 / SUB;
  __shared__ float red[2][4][kMaxWaves][1];
  const int lane = threadIdx.x & 63, wg_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wg_teams = W == 1 ? (int)(blockDim.x >> 6) * SUB : 1;
  const int local = W > 1 ? 0 : SUB == 1 ? wg_wave : (int)threadIdx.x / LANES;
  const int TH = LANES * W, tid = W > 1 ? (int)threadIdx.x : (int)threadIdx.x % LANES;
  const int team = (int)blockIdx.x * wg_teams + local, C = a.C, last_row = (int)a.M - 1;
  const int m_begin = team * per + min(team, extra), m_end = min(m_begin + per + (team < extra ? 1 : 0), last_row + 1);
  const int steps = per + (extra > 0 ? 1 : 0);   // of every team (a barrier is the workgroup's)
  const float fc = (float)C;
  const Place<NV, VEC> pl(tid, TH, C);
  Vec<T> nx[NV], nh[NV];
  auto fetch = [&](int m) {
    m = min(m, last_row);   // (a row past the team's is not used)
    const T *x = static_cast<const T*>(a.x) + m * a.ldx, *hrow = static_cast<const T*>(a.h) + m * a.ldh;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      nx[j] = load_vec<T>(x, pl.at(j), pl.len(j));
      nh[j] = load_vec<T>(hrow, pl.at(j), pl.len(j));
    }
  };
  fetch(m_begin);
  float gate[NV][VEC], gain[NV][VEC], shift[NV][VEC], pgain[NV][VEC];
  int64_t group_end;
  const float one = a.one_plus ? 1.f : 0.f;
  auto load_group = [&](int m) {
    const int64_t group = (uint32_t)m / (uint32_t)a.rpg;
    group_end = (group + 1) * a.rpg;
    load_param(a.gate, a.pdtype, group * a.ldgate, pl, 1.f, 0.f, gate);
    load_param(a.w, a.pdtype, group * a.ldw, pl, 1.f, one, gain);
    load_param(a.b, a.pdtype, group * a.ldb, pl, 0.f, 0.f, shift);
    if (POST) load_param(a.pw, a.pdtype, group * a.ldpw, pl, 1.f, one, pgain);
  };
  load_group(min(m_begin, last_row));
  for (int k = 0, m = m_begin; k < steps; ++k, ++m) {
    float v[NV][VEC], h[NV][VEC];
    float (*sums)[kMaxWaves][1] = red[k & 1];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[j][i] = nx[j].at(i);
        h[j][i] = nh[j].at(i);
      }
    if (k + 1 < steps) fetch(m + 1);
    // v's mean and rstd; v becomes its difference from the mean
    auto norm = [&](float (&u)[NV][VEC], float (*r0)[1], float (*r1)[1], float& mean, float& rstd) {
      float s[1] = {0.f};
      mean = 0.f;
      if (a.layer) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) s[0] += pl.own(j, i, u[j][i]);
        team_sum<1, LANES>(s, r0, wg_wave, 0, W, lane);
        mean = s[0] / fc;   // (correctly rounded: a constant row has its value as mean)
        s[0] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          u[j][i] -= mean;
          const float d = pl.own(j, i, u[j][i]);
          s[0] = __builtin_fmaf(d, d, s[0]);
        }
      team_sum<1, LANES>(s, r1, wg_wave, 0, W, lane);
      rstd = 1.0f / __builtin_sqrtf(s[0] / fc + a.eps);
    };
    const bool live = m < m_end;
    if (live && m >= group_end) load_group(m);
    float pmean = 0.f, prstd = 1.f, mean, rstd;
    if (POST) {
      norm(h, sums[0], sums[1], pmean, prstd);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) h[j][i] = h[j][i] * prstd * pgain[j][i];
    }
    Vec<T> out[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[j][i] = __builtin_fmaf(gate[j][i], h[j][i], a.alpha * v[j][i]);
        // (an fp32 sum that is then rounded, for every type: fused into the
        // conversion an fp16 row would round the exact sum)
        if constexpr (__is_same(T, Half)) asm("" : "+v"(v[j][i]));
      }
      out[j].set(v[j]);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j][i] = out[j].at(i);   // the norm is of what was written
    }
    norm(v, sums[2], sums[3], mean, rstd);
    if (!live) continue;   // (its lanes take part in the next step's sums, if there is one)
    if (tid == 0 && a.stats) {
      float* st = a.stats + m;
      if (a.layer) {
        *st = mean;
        st += a.M;
      }
      *st = rstd;
      if (POST) {
        st += a.M;
        if (a.layer) {
          *st = pmean;
          st += a.M;
        }
        *st = prstd;
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = __builtin_fmaf(v[j][i] * rstd, gain[j][i], shift[j][i]);
      Vec<T> y;
      y.set(o);
      // (both stores stand behind a barrier that all lanes of the row reach
      // with its values in registers: the outputs may be the inputs)
      if (j < NV - 1 || pl.in_row) {
        store_vec<T>(static_cast<T*>(a.s) + m * a.lds, pl.at(j), pl.len(j), out[j]);
        store_vec<T>(static_cast<T*>(a.y) + m * a.ldy, pl.at(j), pl.len(j), y);
      }
    }
  }
}

// Backward: a workgroup is a run's teams, which take its rows in turn; a lane
// keeps its channels' sums over its rows. The teams' sums are added in order
// through LDS, one parameter after the other (P = 4 with a norm after the
// block, else 3), and written once: to the workspace [run][4][C] in fp32, or,
// where a group is one run, as the gradients.
template <typename T, int NV, int SUB, bool POST, int MAXW>
__global__ __launch_bounds__(64 * MAXW) void residual_bwd_kernel(ResidualGradArgs g, int W, int runs) {
  constexpr int VEC = kVec<T>, LANES = 64 / SUB, P = POST ? 4 : 3;
  const ResidualArgs& a = g.f;
  __shared__ float red[2][2][kMaxWaves][2];
  __shared__ float plane[kMaxWaves * 64 * 8];   // [team (sharing a wave: one)][VEC][NV][TH]
  const int lane = threadIdx.x & 63, wg_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int TH = LANES * W, teams = (int)blockDim.x / TH;
  const int team = SUB == 1 ? wg_wave / W : (int)threadIdx.x / LANES, tid = (int)threadIdx.x - team * TH;
  const uint32_t block = blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= (uint32_t)a.G * (uint32_t)runs) return;
  const int64_t group = block / (uint32_t)runs;
  const int run = (int)(block % (uint32_t)runs), C = a.C;
  const int64_t g_begin = min(group * a.rpg, a.M), g_rows = min(a.rpg, a.M - g_begin);
  const int per = (int)((uint32_t)g_rows / (uint32_t)runs), extra = (int)((uint32_t)g_rows % (uint32_t)runs);
  const int m_begin = (int)g_begin + run * per + min(run, extra), m_end = m_begin + per + (run < extra ? 1 : 0);
  const float fc = (float)C, one = a.one_plus ? 1.f : 0.f;
  const Place<NV, VEC> pl(tid, TH, C);
  float gate[NV][VEC], gain[NV][VEC], pgain[NV][VEC], acc[P][NV][VEC];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[p][j][i] = 0.f;
  Vec<T> ns[NV], nh[NV], ndy[NV], nds[NV];
  float nst[4] = {0.f, 1.f, 0.f, 1.f};   // mean, rstd, and h's
  auto fetch = [&](int m) {
    m = min(m, m_end - 1);   // past the end: the last row again, not used
    const T *s = static_cast<const T*>(a.x) + m * a.ldx, *h = static_cast<const T*>(a.h) + m * a.ldh;
    const T *dy = static_cast<const T*>(g.dy) + m * g.lddy, *ds = static_cast<const T*>(g.ds) + m * g.ldds;
    auto load = [&](auto once) {
      constexpr bool ONCE = decltype(once)::value;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        ns[j] = load_vec<T, ONCE>(s, pl.at(j), pl.len(j));
        ndy[j] = load_vec<T, ONCE>(dy, pl.at(j), pl.len(j));
        nh[j] = load_vec<T, ONCE>(h, pl.at(j), pl.len(j));
        if (g.ds)
          nds[j] = load_vec<T, ONCE>(ds, pl.at(j), pl.len(j));
        else
          nds[j].w = u32x4{0, 0, 0, 0};
      }
    };
    if (g.once)
      load(std::true_type());
    else
      load(std::false_type());
    const float* st = a.stats + m;
    if (a.layer) {
      nst[0] = *st;
      st += a.M;
    }
    nst[1] = *st;
    if (POST) {
      st += a.M;
      if (a.layer) {
        nst[2] = *st;
        st += a.M;
      }
      nst[3] = *st;
    }
  };
  if (m_begin < m_end) {
    fetch(m_begin + team);
    load_param(a.gate, a.pdtype, group * a.ldgate, pl, 1.f, 0.f, gate);
    load_param(a.w, a.pdtype, group * a.ldw, pl, 1.f, one, gain);
    if (POST) load_param(a.pw, a.pdtype, group * a.ldpw, pl, 1.f, one, pgain);
  }
  int flip = 0;
  // every team makes the same steps (a barrier is the workgroup's)
  for (int base = m_begin; base < m_end; base += teams, flip ^= 1) {
    const int m = base + team;
    const bool live = m < m_end;
    const float mean = nst[0], rstd = nst[1], hmean = nst[2], hrstd = nst[3];
    float d[NV][VEC], shat[NV][VEC], h[NV][VEC], t[NV][VEC], s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float dy = ndy[j].at(i);
        shat[j][i] = (ns[j].at(i) - mean) * rstd;
        h[j][i] = nh[j].at(i);
        t[j][i] = nds[j].at(i);
        d[j][i] = dy * gain[j][i];
        const float own = pl.own(j, i, d[j][i]);
        s[0] += own;
        s[1] = __builtin_fmaf(own, pl.own(j, i, shat[j][i]), s[1]);
        if (live) {
          acc[1][j][i] = __builtin_fmaf(dy, shat[j][i], acc[1][j][i]);
          acc[2][j][i] += dy;
        }
      }
    if (base + teams < m_end) fetch(m + teams);
    // Where dx or dh is an input: the vector that ends a row shares elements
    // with the one before it, maybe another wave's, so all loads of the row
    // have returned before the barrier behind which it is stored. (Always
    // waiting for h and ds here: 5003 x 1283 fp16 with a norm after the block
    // 35.2 us against 33.5.)
    if (g.in_place) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    team_sum<2, LANES>(s, red[flip][0], wg_wave, team * W, W, lane);
    const float a1 = a.layer ? -(s[0] / fc) * rstd : 0.f, a2 = -(s[1] / fc) * rstd;
    s[0] = s[1] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        t[j][i] += __builtin_fmaf(d[j][i], rstd, __builtin_fmaf(shat[j][i], a2, a1));
        o[i] = a.alpha * t[j][i];
        float hn = h[j][i];
        d[j][i] = t[j][i] * gate[j][i];   // of hn
        if (POST) {
          h[j][i] = (h[j][i] - hmean) * hrstd;   // hhat
          hn = h[j][i] * pgain[j][i];
          if (live) acc[P - 1][j][i] = __builtin_fmaf(d[j][i], h[j][i], acc[P - 1][j][i]);
          d[j][i] *= pgain[j][i];
          const float own = pl.own(j, i, d[j][i]);
          s[0] += own;
          s[1] = __builtin_fmaf(own, pl.own(j, i, h[j][i]), s[1]);
        }
        if (live) acc[0][j][i] = __builtin_fmaf(t[j][i], hn, acc[0][j][i]);
      }
      Vec<T> out;
      out.set(o);
      if (live && (j < NV - 1 || pl.in_row)) store_vec<T>(static_cast<T*>(g.dx) + m * g.lddx, pl.at(j), pl.len(j), out);
    }
    float b1 = 0.f, b2 = 0.f;
    if (POST) {
      team_sum<2, LANES>(s, red[flip][1], wg_wave, team * W, W, lane);
      b1 = a.layer ? -(s[0] / fc) * hrstd : 0.f;
      b2 = -(s[1] / fc) * hrstd;
    }
    if (!live) continue;   // (the last step)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        o[i] = POST ? __builtin_fmaf(d[j][i], hrstd, __builtin_fmaf(h[j][i], b2, b1)) : d[j][i];
      Vec<T> out;
      out.set(o);
      if (j < NV - 1 || pl.in_row) store_vec<T>(static_cast<T*>(g.dh) + m * g.lddh, pl.at(j), pl.len(j), out);
    }
  }
  // the teams' sums
  const int n = (C + VEC - 1) / VEC, len = min(C, VEC), size = VEC * NV * TH;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (!g.out[p]) continue;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float v = shares_sum<SUB>(acc[p][j][i]);
        if (team % SUB == 0) plane[team / SUB * size + (i * NV + j) * TH + tid] = v;
      }
    __syncthreads();
    for (int vec = threadIdx.x; vec < n; vec += blockDim.x) {
      const int at = C < VEC ? 0 : min(vec * VEC, C - VEC);
      int j = 0;
#pragma unroll
      for (int k = 1; k < NV; ++k) j += vec >= k * TH;
      const float* q = plane + j * TH + (vec - j * TH);
      float v[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = q[i * NV * TH];
      for (int t = 1; t < teams / SUB; ++t) {
        q += size;
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] += q[i * NV * TH];
      }
      if (g.part)
        store_params<VEC>(g.part, SVDQ_DT_F32, ((int64_t)block * 4 + p) * C + at, len, v);
      else
        store_params<VEC>(g.out[p], g.gdtype, group * C + at, len, v);
    }
  }
}

// The runs' sums of a group added per channel: 32 threads a channel, each
// every 32nd run in order, then the 32 in order.
__global__ __launch_bounds__(1024) void residual_join_kernel(ResidualGradArgs g, int runs) {
  __shared__ float red[32][33];
  const int C = g.f.C, cl = threadIdx.x & 31, k = threadIdx.x >> 5, c = blockIdx.x * 32 + cl;
  const int p = blockIdx.z;
  const int64_t group = blockIdx.y;
  if (!g.out[p]) return;   // (the whole workgroup)
  const float* at = g.part + ((size_t)group * runs * 4 + p) * C;
  float v[kResidualRuns / 32], s = 0.f;
#pragma unroll
  for (int i = 0; i < kResidualRuns / 32; ++i) v[i] = c < C && k + 32 * i < runs ? at[(size_t)(k + 32 * i) * 4 * C + c] : 0.f;
#pragma unroll
  for (int i = 0; i < kResidualRuns / 32; ++i) s += v[i];
  red[k][cl] = s;
  __syncthreads();
  if (k == 0 && c < C) {
    float t = red[0][cl];
#pragma unroll
    for (int i = 1; i < 32; ++i) t += red[i][cl];
    store_param(g.out[p], g.gdtype, group * C + c, t);
  }
}

template <typename T, bool POST>
hipError_t launch_fwd(const ResidualArgs& a, int num_cus, hipStream_t st) {
  const ResidualTeam t = residual_team(a.C, kVec<T>, 2);
  const int fit = 16;   // waves of a CU at once (8: 4608 x 2560 with a norm after the block 30 us against 25, 24: 30)
  const int wg_waves = t.waves == 1 ? 4 : t.waves, wg_teams = t.waves == 1 ? 4 * t.sub : 1;
  const int64_t most = (int64_t)num_cus * std::max(1, fit / wg_waves);
  const int64_t wgs = std::min(most, (a.M + wg_teams - 1) / wg_teams), all = wgs * wg_teams;
  const dim3 grid((unsigned)wgs), block(64 * wg_waves);
  const int per = (int)(a.M / all), extra = (int)(a.M % all);
  if (t.sub == 4)
    hipLaunchKernelGGL((residual_fwd_kernel<T, 1, 4, POST>), grid, block, 0, st, a, t.waves, per, extra);
  else if (t.nv == 1)
    hipLaunchKernelGGL((residual_fwd_kernel<T, 1, 1, POST>), grid, block, 0, st, a, t.waves, per, extra);
  else
    hipLaunchKernelGGL((residual_fwd_kernel<T, 2, 1, POST>), grid, block, 0, st, a, t.waves, per, extra);
  return hipGetLastError();
}

template <typename T, bool POST>
hipError_t launch_bwd(const ResidualGradArgs& g, const ResidualGradPlan& p, hipStream_t st) {
  constexpr int NV = kVec<T> == 4 ? 2 : 1;
  constexpr int WAVES = POST ? 12 : kMaxWaves;   // of workgroups whose lanes hold a vector (residual_grad_waves)
  const ResidualTeam t = residual_team(g.f.C, kVec<T>, NV);
  const dim3 grid = many_groups((int64_t)g.f.G * p.runs), block(t.waves * 64 / t.sub * p.teams);
#define SVDQ_RESIDUAL_BWD(NV, SUB, WAVES) \
  hipLaunchKernelGGL((residual_bwd_kernel<T, NV, SUB, POST, WAVES>), grid, block, 0, st, g, t.waves, p.runs)
  if (t.sub == 4)
    SVDQ_RESIDUAL_BWD(1, 4, WAVES);
  else if (t.nv == 2) {
    if constexpr (NV == 2) {
      if (t.waves <= 12)
        SVDQ_RESIDUAL_BWD(2, 1, 12);
      else
        SVDQ_RESIDUAL_BWD(2, 1, kMaxWaves);
    }
  } else if (t.waves <= WAVES)
    SVDQ_RESIDUAL_BWD(1, 1, WAVES);
  else if constexpr (NV == 1 && POST)
    SVDQ_RESIDUAL_BWD(1, 1, kMaxWaves);
#undef SVDQ_RESIDUAL_BWD
  return hipGetLastError();
}

}  // namespace

hipError_t launch_residual(const ResidualArgs& a, int num_cus, hipStream_t st) {
  if (a.dtype == SVDQ_DT_F32) return a.post ? launch_fwd<float, true>(a, num_cus, st) : launch_fwd<float, false>(a, num_cus, st);
  if (a.dtype == SVDQ_DT_BF16) return a.post ? launch_fwd<Bf16, true>(a, num_cus, st) : launch_fwd<Bf16, false>(a, num_cus, st);
  return a.post ? launch_fwd<Half, true>(a, num_cus, st) : launch_fwd<Half, false>(a, num_cus, st);
}

hipError_t launch_residual_grad(const ResidualGradArgs& args, const ResidualGradPlan& p, hipStream_t st) {
  // What the caches (256 MB) cannot keep until it is used again is read past
  // them (three sets of inputs in turn, 8192 x 4096 bf16, 403 MB: 81 us against
  // 93, 8192 x 2048 fp32, 403 MB: 76 against 89, 4608 x 5120 fp32, 566 MB: 122
  // against 128; one set, 4608 x 2560 bf16, 142 MB: 45.5 against 43.2).
  ResidualGradArgs g = args;
  g.once = (double)g.f.M * g.f.C * (g.ds ? 6 : 5) * (g.f.dtype == SVDQ_DT_F32 ? 4 : 2) > 256e6;
  const bool post = g.f.post;
  const hipError_t e = g.f.dtype == SVDQ_DT_F32    ? (post ? launch_bwd<float, true>(g, p, st) : launch_bwd<float, false>(g, p, st))
                       : g.f.dtype == SVDQ_DT_BF16 ? (post ? launch_bwd<Bf16, true>(g, p, st) : launch_bwd<Bf16, false>(g, p, st))
                                                   : (post ? launch_bwd<Half, true>(g, p, st) : launch_bwd<Half, false>(g, p, st));
  if (e != hipSuccess || !g.part) return e;
  hipLaunchKernelGGL(residual_join_kernel, dim3((g.f.C + 31) / 32, (unsigned)g.f.G, g.f.post ? 4 : 3), dim3(1024), 0, st, g, p.runs);
  return hipGetLastError();
}

}  // namespace svdq
