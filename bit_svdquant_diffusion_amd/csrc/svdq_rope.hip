// Rotary positions of several axes (time, height, width, ...). Pair j of a
// head's elements, (2 j, 2 j + 1) or (j, j + pairs), belongs to an axis and
// turns by p = position[axis] freq[j]:
//
//   (u, v) -> (u cos p - v sin p, u sin p + v cos p)
//
// and by -p for the gradient. What lies behind the pairs passes through.
//
// Bound by memory: q and k are read and written once, in one launch (4608
// tokens, 24 + 24 heads of 128, bf16, calls with three sets of inputs in turn:
// 28.9 us, 3.9 TB/s; the kernel alone in a trace 22, 5.1). A workgroup takes a
// few tokens and a share of their heads; it first puts the tokens' cosines and
// sines into LDS. The angle is formed in 64 bits, as turns,
// and only its fraction of a turn is rounded to 32 (at position 10^6 the 32-bit
// product would be 0.06 off).
#include <algorithm>

#include "svdq_internal.h"
#include "svdq_types.h"

namespace svdq {

namespace {

constexpr int kRopeTokens = 4, kRopeMaxDim = 256;

template <typename T, bool HALF>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a, int token_blocks, int heads_each) {
  constexpr int VEC = kVec<T>;
  __shared__ float cs[kRopeTokens][2][kRopeMaxDim / 2];
  const int b = blockIdx.x / token_blocks, l0 = (int)(blockIdx.x % token_blocks) * kRopeTokens;
  const int tokens = min(kRopeTokens, a.L - l0), D = a.D, P = a.pairs;
  for (int e = threadIdx.x; e < tokens * (D / 2); e += 256) {
    const int t = e / (D / 2), j = e - t * (D / 2);
    float c = 1.f, s = 0.f;
    if (j < P) {
      int axis = 0;
#pragma unroll
      for (int i = 1; i < 4; ++i) axis += i < a.axes && j >= a.first[i];
      const int64_t at = b * a.pos_batch + (int64_t)(l0 + t) * a.axes + axis;
      const double p = a.pos_dtype == SVDQ_POS_F32 ? (double)static_cast<const float*>(a.pos)[at]
                                                   : (double)static_cast<const int*>(a.pos)[at];
      double turns = p * a.freqs[j] * 0.15915494309189533577;   // 1 / (2 pi)
      turns -= __builtin_rint(turns);
      sincospif(2.f * (float)(a.inverse ? -turns : turns), &s, &c);
    }
    cs[t][0][j] = c;
    cs[t][1][j] = s;
  }
  __syncthreads();
  // items: a vector (HALF: the two of its pairs) of a head of a token
  const int turned = HALF ? P / VEC : 0, per_row = HALF ? turned + (D - 2 * P) / VEC : D / VEC;
  const int h0 = (int)blockIdx.y * heads_each, h1 = min(h0 + heads_each, a.H[0] + a.H[1]);
  const int items = tokens * (h1 - h0) * per_row;
  for (int e = threadIdx.x; e < items; e += 256) {
    const int row = e / per_row, j = e - row * per_row, t = row / (h1 - h0);
    int head = h0 + row - t * (h1 - h0);
    const int which = head >= a.H[0];
    head -= which ? a.H[0] : 0;
    const Heads &x = a.x[which], &y = a.y[which];
    const T* in = static_cast<const T*>(x.p) + b * x.batch + (l0 + t) * x.token + head * x.head;
    T* out = static_cast<T*>(y.p) + b * y.batch + (l0 + t) * y.token + head * y.head;
    if constexpr (!HALF) {
      Vec<T> v = load_vec<T>(in, j * VEC, VEC);
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        const float c = cs[t][0][j * (VEC / 2) + i], s = cs[t][1][j * (VEC / 2) + i], p = v.at(2 * i), q = v.at(2 * i + 1);
        const bool turns = j * (VEC / 2) + i < P;   // (what lies behind the pairs keeps its bits)
        o[2 * i] = turns ? __builtin_fmaf(p, c, -(q * s)) : p;
        o[2 * i + 1] = turns ? __builtin_fmaf(p, s, q * c) : q;
      }
      v.set(o);
      store_vec<T>(out, j * VEC, VEC, v);
    } else if (j < turned) {
      Vec<T> v = load_vec<T>(in, j * VEC, VEC), w = load_vec<T>(in, P + j * VEC, VEC);
      float o[VEC], q[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float c = cs[t][0][j * VEC + i], s = cs[t][1][j * VEC + i], p = v.at(i), r = w.at(i);
        o[i] = __builtin_fmaf(p, c, -(r * s));
        q[i] = __builtin_fmaf(p, s, r * c);
      }
      v.set(o);
      w.set(q);
      store_vec<T>(out, j * VEC, VEC, v);
      store_vec<T>(out, P + j * VEC, VEC, w);
    } else {
      const int at = 2 * P + (j - turned) * VEC;
      store_vec<T>(out, at, VEC, load_vec<T>(in, at, VEC));
    }
  }
}

template <typename T>
hipError_t launch_rope_as(const RopeArgs& a, hipStream_t st) {
  const int heads = a.H[0] + a.H[1], blocks = (a.L + kRopeTokens - 1) / kRopeTokens;
  // with few tokens the heads are dealt over workgroups, four or more each
  const int64_t all = (int64_t)blocks * a.B;
  const int shares = (int)std::max<int64_t>(1, std::min<int64_t>((heads + 3) / 4, 1024 / all));
  const int each = (heads + shares - 1) / shares;
  const dim3 grid((unsigned)all, (unsigned)((heads + each - 1) / each));
  if (a.half)
    hipLaunchKernelGGL((rope_kernel<T, true>), grid, dim3(256), 0, st, a, blocks, each);
  else
    hipLaunchKernelGGL((rope_kernel<T, false>), grid, dim3(256), 0, st, a, blocks, each);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t st) {
  if (a.dtype == SVDQ_DT_F32) return launch_rope_as<float>(a, st);
  if (a.dtype == SVDQ_DT_BF16) return launch_rope_as<Bf16>(a, st);
  return launch_rope_as<Half>(a, st);
}

}  // namespace svdq
