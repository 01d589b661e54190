// Layer norm of rows, affine or modulated per group of rows, and its
// gradients. With g the row's gain (1, weight or 1 + weight) and b its bias,
//
//   mean = sum_c x / C,  rstd = (sum_c (x - mean)^2 / C + eps)^(-1/2)
//   xhat = (x - mean) rstd,  y = xhat g + b
//   d = dy g,  dx = rstd (d - mean_c(d) - xhat mean_c(d xhat))
//   dweight = sum over the group's rows of dy xhat,  dbias = sum of dy.
//
// Both passes are bound by memory: one read of x (and dy), one write of y
// (dx). A workgroup of W waves holds kRows rows in registers, NV 16-byte
// vectors per lane and row, so the two-pass variance (which keeps its digits
// when |mean| is far above the deviation) and the backward's two sums cost no
// second read. All sums are in fp32: per lane, then a fixed butterfly over
// the wave, then the waves in order.
#include <algorithm>

#include "svdq_internal.h"
#include "svdq_layout.h"
#include "svdq_types.h"

namespace svdq {

namespace {

constexpr int kMaxWaves = 8;

// Sums of W waves' values for n rows at once, the same in every wave. `red`
// holds n * kMaxWaves floats; the caller alternates two areas, so one barrier
// per call is enough.
template <int n>
__device__ __forceinline__ void team_sum(float (&v)[n], float* red, int wave, int W, int lane) {
#pragma unroll
  for (int r = 0; r < n; ++r) v[r] = wave_sum(v[r]);
  if (W == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int r = 0; r < n; ++r) red[r * kMaxWaves + wave] = v[r];
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < n; ++r) {
    float s = red[r * kMaxWaves];
    for (int w = 1; w < W; ++w) s += red[r * kMaxWaves + w];
    v[r] = s;
  }
}

// The gain and the bias of this lane's channels for group g
template <int NV, int VEC>
__device__ __forceinline__ void load_gain(const NormArgs& a, int64_t g, int tid, int T, float (&gain)[NV][VEC]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (tid + j * T) * VEC;
    if (a.w) {
      load_params<VEC>(a.w, a.pdtype, g * a.ldw, c, a.C, gain[j]);
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

// Forward. QUANT: instead of y, its bf16 values' E4M3 codes and the scales of
// their blocks of 128 (sixteen lanes of a wave hold a block) in the layout of
// the FP8 product's operand.
template <typename T, int NV, int R, int MAXW, bool QUANT>
__global__ __launch_bounds__(64 * MAXW) void norm_fwd_kernel(NormArgs a, int64_t rows_per_wg) {
  constexpr int VEC = kVec<T>;
  __shared__ float red[2][2][R * kMaxWaves];
  const int tid = threadIdx.x, lane = tid & 63, TH = blockDim.x, W = TH >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t m_begin = (int64_t)blockIdx.x * rows_per_wg, m_end = min(m_begin + rows_per_wg, a.M);
  const int C = a.C;
  const float fc = (float)C;
  float gain[NV][VEC], shift[NV][VEC];
  int64_t group_end = m_begin;   // where the loaded group's rows end
  int flip = 0;
  for (int64_t m0 = m_begin; m0 < m_end; m0 += R, flip ^= 1) {
    Vec<T> x[R][NV];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const T* row = static_cast<const T*>(a.x) + min(m0 + r, m_end - 1) * a.ldx;   // past the end: the last row again
#pragma unroll
      for (int j = 0; j < NV; ++j) x[r][j] = load_vec<T>(row, (tid + j * TH) * VEC, C);
    }
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) mean[r] += x[r][j].at(i);
    }
    team_sum<R>(mean, red[flip][0], wave, W, lane);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] /= fc;   // (the division, correctly rounded: a constant row has its value as mean)
      rstd[r] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float d = x[r][j].at(i) - mean[r];
          // lanes past the row hold zeros that are no part of it
          if ((tid + j * TH) * VEC + i < C) rstd[r] = __builtin_fmaf(d, d, rstd[r]);
        }
    }
    team_sum<R>(rstd, red[flip][1], wave, W, lane);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rstd[r] = 1.0f / __builtin_sqrtf(rstd[r] / fc + a.eps);
      const int64_t m = m0 + r;
      if (m < m_end) {
        if (m >= group_end) {   // uniform: a new group's gain and bias
          const int64_t group = m / a.rpg;
          group_end = (group + 1) * a.rpg;
          load_gain<NV, VEC>(a, group, tid, TH, gain);
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            if (a.b) {
              load_params<VEC>(a.b, a.pdtype, group * a.ldb, (tid + j * TH) * VEC, C, shift[j]);
            } else {
#pragma unroll
              for (int i = 0; i < VEC; ++i) shift[j][i] = 0.f;
            }
          }
        }
        if (tid == 0) {
          if (a.mean) a.mean[m] = mean[r];
          if (a.rstd) a.rstd[m] = rstd[r];
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = (tid + j * TH) * VEC;
          float o[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            o[i] = __builtin_fmaf((x[r][j].at(i) - mean[r]) * rstd[r], gain[j][i], shift[j][i]);
          Vec<T> y;
          y.set(o);
          if constexpr (!QUANT) {
            if (c < C) store_vec<T>(static_cast<T*>(a.y) + m * a.ldy, c, C, y);
          } else {
            // channels past the row (C is a multiple of 16) are zero codes
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
  }
}

// Backward: dx of a run of rows of one group, and the run's sums of dy xhat
// and dy per channel, kept by each lane for its channels over the run's rows
// (a fixed order) and written once at the run's end: to the workspace
// [run][2][C] in fp32, or, where a group is one run, as the gradients.
template <typename T, int NV, int R, int MAXW>
__global__ __launch_bounds__(64 * MAXW) void norm_bwd_kernel(NormGradArgs g, int64_t rows_per_run, int runs) {
  constexpr int VEC = kVec<T>;
  const NormArgs& a = g.f;
  __shared__ float red[2][2 * R * kMaxWaves];
  const int tid = threadIdx.x, lane = tid & 63, TH = blockDim.x, W = TH >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t group = blockIdx.x / runs, run = blockIdx.x % runs;
  const int64_t g_begin = group * a.rpg, g_end = min(g_begin + a.rpg, a.M);
  const int64_t m_begin = g_begin + run * rows_per_run, m_end = min(m_begin + rows_per_run, g_end);
  const int C = a.C;
  const float fc = (float)C;
  float gain[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) dw[j][i] = db[j][i] = 0.f;
  if (m_begin < m_end) load_gain<NV, VEC>(a, group, tid, TH, gain);
  int flip = 0;
  for (int64_t m0 = m_begin; m0 < m_end; m0 += R, flip ^= 1) {
    Vec<T> x[R][NV], dy[R][NV];
    float mean[R], rstd[R], s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t m = min(m0 + r, m_end - 1);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        x[r][j] = load_vec<T>(static_cast<const T*>(a.x) + m * a.ldx, (tid + j * TH) * VEC, C);
        dy[r][j] = load_vec<T>(static_cast<const T*>(g.dy) + m * g.lddy, (tid + j * TH) * VEC, C);
      }
      mean[r] = a.mean[m];
      rstd[r] = a.rstd[m];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[2 * r] = s[2 * r + 1] = 0.f;
      const bool live = m0 + r < m_end;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          // (lanes past the row hold dy = 0 and gain = 0 or 1: they add nothing)
          const float t = dy[r][j].at(i);
          const float xhat = (x[r][j].at(i) - mean[r]) * rstd[r];
          const float d = t * gain[j][i];
          const bool in = (tid + j * TH) * VEC + i < C;
          s[2 * r] += d;
          s[2 * r + 1] = in ? __builtin_fmaf(d, xhat, s[2 * r + 1]) : s[2 * r + 1];
          if (live) {
            dw[j][i] = __builtin_fmaf(t, xhat, dw[j][i]);
            db[j][i] += t;
          }
        }
    }
    team_sum<2 * R>(s, red[flip], wave, W, lane);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (m0 + r < m_end) {
        const float c1 = s[2 * r] / fc, c2 = s[2 * r + 1] / fc;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = (tid + j * TH) * VEC;
          float v[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float xhat = (x[r][j].at(i) - mean[r]) * rstd[r];
            const float d = dy[r][j].at(i) * gain[j][i];
            v[i] = rstd[r] * (d - c1 - xhat * c2);
          }
          Vec<T> o;
          o.set(v);
          if (c < C) store_vec<T>(static_cast<T*>(g.dx) + (m0 + r) * g.lddx, c, C, o);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = (tid + j * TH) * VEC + i;
      if (c < C) {
        if (g.part) {
          float* p = g.part + (size_t)blockIdx.x * 2 * C;
          p[c] = dw[j][i];
          p[C + c] = db[j][i];
        } else {
          if (g.dw) store_param(g.dw, g.gdtype, group * C + c, dw[j][i]);
          if (g.db) store_param(g.db, g.gdtype, group * C + c, db[j][i]);
        }
      }
    }
}

// The runs' sums of a group added per channel: sixteen threads a channel,
// each every sixteenth run in order, then the sixteen in order.
__global__ __launch_bounds__(256) void norm_param_grad_kernel(NormGradArgs g, int runs) {
  __shared__ float red[16][17];
  const int C = g.f.C, cl = threadIdx.x & 15, k = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + cl;   // 0 .. 2 C: dweight's channels, then dbias's
  const int64_t group = blockIdx.y;
  const float* p = g.part + (size_t)group * runs * 2 * C;
  float s = 0.f;
  if (c < 2 * C)
    for (int i = k; i < runs; i += 16) s += p[(size_t)i * 2 * C + c];
  red[k][cl] = s;
  __syncthreads();
  if (k == 0 && c < 2 * C) {
    float t = red[0][cl];
#pragma unroll
    for (int i = 1; i < 16; ++i) t += red[i][cl];
    void* o = c < C ? g.dw : g.db;
    if (o) store_param(o, g.gdtype, group * C + (c < C ? c : c - C), t);
  }
}

// Waves and vectors per lane for a row of n vectors: up to four waves of up to
// four vectors, the pair that leaves the fewest lanes idle (the fewest waves
// among those); wider rows take eight waves, one row at a time (fp32 rows past
// 8192 channels with eight vectors a lane).
struct Team {
  int nv, waves;
};
Team norm_team(int64_t n) {
  if (n > 64 * 4 * 4) return n > 64 * 4 * kMaxWaves ? Team{8, kMaxWaves} : Team{4, kMaxWaves};
  Team best{4, 4};
  int64_t least = 16;
  for (int w = 4; w >= 1; --w) {
    const int nv = (int)((n + 64 * w - 1) / (64 * w));
    if (nv <= 4 && nv * w <= least) {
      least = nv * w;
      best = Team{nv, w};
    }
  }
  return best;
}

#define SVDQ_NORM_LAUNCH(KERNEL, ...)                                                                \
  if (t.waves == kMaxWaves) {                                                                        \
    if constexpr (sizeof(T) == 4) {                                                                  \
      if (t.nv == 8) {                                                                               \
        hipLaunchKernelGGL((KERNEL(8, 1, kMaxWaves)), dim3(grid), b, 0, st, __VA_ARGS__);            \
        return hipGetLastError();                                                                    \
      }                                                                                              \
    }                                                                                                \
    hipLaunchKernelGGL((KERNEL(4, 1, kMaxWaves)), dim3(grid), b, 0, st, __VA_ARGS__);                \
    return hipGetLastError();                                                                        \
  }                                                                                                  \
  switch (t.nv) {                                                                                    \
    case 1: hipLaunchKernelGGL((KERNEL(1, 2, 4)), dim3(grid), b, 0, st, __VA_ARGS__); break;         \
    case 2: hipLaunchKernelGGL((KERNEL(2, 2, 4)), dim3(grid), b, 0, st, __VA_ARGS__); break;         \
    case 3: hipLaunchKernelGGL((KERNEL(3, 2, 4)), dim3(grid), b, 0, st, __VA_ARGS__); break;         \
    default: hipLaunchKernelGGL((KERNEL(4, 2, 4)), dim3(grid), b, 0, st, __VA_ARGS__); break;        \
  }                                                                                                  \
  return hipGetLastError();

template <typename T, bool QUANT>
hipError_t launch_fwd(const NormArgs& a, int num_cus, hipStream_t st) {
  const int64_t span = QUANT ? a.Kp : a.C;
  const Team t = norm_team((span + kVec<T> - 1) / kVec<T>);
  const int64_t most = (int64_t)num_cus * 32 / t.waves;   // eight waves a SIMD
  const int64_t per = std::max<int64_t>(1, (a.M + most - 1) / most);
  const unsigned grid = (unsigned)((a.M + per - 1) / per);
  const dim3 b(64 * t.waves);
#define SVDQ_FWD(NV, R, MAXW) norm_fwd_kernel<T, NV, R, MAXW, QUANT>
  SVDQ_NORM_LAUNCH(SVDQ_FWD, a, per)
#undef SVDQ_FWD
}

template <typename T>
hipError_t launch_bwd(const NormGradArgs& g, const NormGradPlan& p, hipStream_t st) {
  const Team t = norm_team((g.f.C + kVec<T> - 1) / kVec<T>);
  const unsigned grid = (unsigned)((int64_t)g.f.G * p.runs);
  const dim3 b(64 * t.waves);
#define SVDQ_BWD(NV, R, MAXW) norm_bwd_kernel<T, NV, R, MAXW>
  SVDQ_NORM_LAUNCH(SVDQ_BWD, g, p.rows_per_run, p.runs)
#undef SVDQ_BWD
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, int num_cus, hipStream_t st) {
  if (a.q) return launch_fwd<Bf16, true>(a, num_cus, st);
  if (a.dtype == SVDQ_DT_F32) return launch_fwd<float, false>(a, num_cus, st);
  if (a.dtype == SVDQ_DT_BF16) return launch_fwd<Bf16, false>(a, num_cus, st);
  return launch_fwd<Half, false>(a, num_cus, st);
}

hipError_t launch_norm_grad(const NormGradArgs& g, const NormGradPlan& p, hipStream_t st) {
  const hipError_t e = g.f.dtype == SVDQ_DT_F32    ? launch_bwd<float>(g, p, st)
                       : g.f.dtype == SVDQ_DT_BF16 ? launch_bwd<Bf16>(g, p, st)
                                                   : launch_bwd<Half>(g, p, st);
  if (e != hipSuccess || !g.part) return e;
  hipLaunchKernelGGL(norm_param_grad_kernel, dim3((2 * g.f.C + 15) / 16, (unsigned)g.f.G), dim3(256), 0, st, g, p.runs);
  return hipGetLastError();
}

}  // namespace svdq
