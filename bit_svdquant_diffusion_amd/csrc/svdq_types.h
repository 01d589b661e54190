// Device-side element types of the layer norm: vectors of 16 bytes of bf16,
// fp16 or fp32 read from and written to addresses aligned to one element
// (gfx950 global loads and stores take any alignment), and wave-wide sums.
#pragma once
#include <string.h>

#include "svdq_device.h"

namespace svdq {

struct Bf16 {
  uint16_t bits;
};
typedef _Float16 Half;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<Half>(Half v) { return (float)v; }
template <>
__device__ __forceinline__ float to_f32<Bf16>(Bf16 v) { return __uint_as_float((uint32_t)v.bits << 16); }

// one rounding, to nearest even (NaN stays NaN)
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ Half from_f32<Half>(float v) { return (Half)v; }
template <>
__device__ __forceinline__ Bf16 from_f32<Bf16>(float v) { return Bf16{__builtin_bit_cast(uint16_t, (__bf16)v)}; }

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);   // elements of a 16-byte vector

// 16 bytes of a row, kept packed in four registers; at(i) unpacks an element
template <typename T>
struct Vec {
  u32x4 w;
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[i]);
    } else if constexpr (__is_same(T, Bf16)) {
      return i & 1 ? bf16hi(w[i >> 1]) : bf16lo(w[i >> 1]);
    } else {
      return (float)__builtin_bit_cast(Half, (uint16_t)(w[i >> 1] >> (16 * (i & 1))));
    }
  }
  // the roundings of v
  __device__ __forceinline__ void set(const float (&v)[kVec<T>]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4)
        w[i] = __float_as_uint(v[i]);
      else if constexpr (__is_same(T, Bf16))
        w[i] = cvt_bf16x2(v[2 * i], v[2 * i + 1]);
      else
        w[i] = (uint32_t)__builtin_bit_cast(uint16_t, (Half)v[2 * i]) |
               ((uint32_t)__builtin_bit_cast(uint16_t, (Half)v[2 * i + 1]) << 16);
    }
  }
};

// The n elements of a row of C that the lane with vector c / n handles. Where
// the row ends inside the vector it is moved back to end with the row, so that
// one wide access serves (its first elements are then another lane's, too:
// `own` is zero for them and all ones for the lane's own, and what both lanes
// write is the same). A row shorter than a vector is taken element by element
// (len < n). A lane past the row reads the row's end and owns nothing.
template <int n>
struct Window {
  int at, len;
  uint32_t own[n];
};
template <int n>
__device__ __forceinline__ Window<n> window(int c, int C) {
  Window<n> w;
  w.at = C < n ? 0 : min(c, C - n);
  w.len = min(C, n);
#pragma unroll
  for (int i = 0; i < n; ++i) w.own[i] = w.at + i >= c && w.at + i < C ? ~0u : 0u;
  return w;
}
__device__ __forceinline__ float own_or_0(float v, uint32_t own) { return __uint_as_float(__float_as_uint(v) & own); }

typedef u32x4 __attribute__((aligned(2))) u32x4_any;   // at any element's address

// ONCE: past the caches (non-temporal)
template <typename T, bool ONCE = false>
__device__ __forceinline__ Vec<T> load_vec(const T* row, int at, int len) {
  Vec<T> o;
  if (len == kVec<T>) {   // uniform
    const u32x4_any* p = reinterpret_cast<const u32x4_any*>(row + at);
    if constexpr (ONCE)
      o.w = __builtin_nontemporal_load(p);
    else
      o.w = *p;
  } else {
    o.w = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i)
      if (i < len) {
        if constexpr (sizeof(T) == 4)
          o.w[i] = __float_as_uint(row[i]);
        else
          o.w[i >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, row[i]) << (16 * (i & 1));
      }
  }
  return o;
}
template <typename T>
__device__ __forceinline__ void store_vec(T* row, int at, int len, const Vec<T>& o) {
  if (len == kVec<T>) {
    memcpy(row + at, &o.w, 16);
  } else {
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i)
      if (i < len) {
        if constexpr (sizeof(T) == 4)
          row[i] = __uint_as_float(o.w[i]);
        else
          row[i] = __builtin_bit_cast(T, (uint16_t)(o.w[i >> 1] >> (16 * (i & 1))));
      }
  }
}

// a window's parameters as floats, in any of the three types (a uniform
// branch); zeros past the row
template <int n, typename P>
__device__ __forceinline__ void load_params_as(const P* p, int at, int len, float* o) {
  if (len == n) {
    P v[n];
    memcpy(v, p + at, sizeof(v));
#pragma unroll
    for (int i = 0; i < n; ++i) o[i] = to_f32<P>(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) o[i] = i < len ? to_f32<P>(p[i]) : 0.f;
  }
}
template <int n>
__device__ __forceinline__ void load_params(const void* p, int dtype, int64_t row, int at, int len, float* o) {
  if (dtype == SVDQ_DT_F32)
    load_params_as<n>(static_cast<const float*>(p) + row, at, len, o);
  else if (dtype == SVDQ_DT_BF16)
    load_params_as<n>(static_cast<const Bf16*>(p) + row, at, len, o);
  else
    load_params_as<n>(static_cast<const Half*>(p) + row, at, len, o);
}
__device__ __forceinline__ void store_param(void* p, int dtype, int64_t at, float v) {
  if (dtype == SVDQ_DT_F32)
    static_cast<float*>(p)[at] = v;
  else if (dtype == SVDQ_DT_BF16)
    static_cast<Bf16*>(p)[at] = from_f32<Bf16>(v);
  else
    static_cast<Half*>(p)[at] = from_f32<Half>(v);
}

template <int n, typename P>
__device__ __forceinline__ void store_params_as(P* p, int len, const float* v) {
  P o[n];
#pragma unroll
  for (int i = 0; i < n; ++i) o[i] = from_f32<P>(v[i]);
  if (len == n) {
    memcpy(p, o, sizeof(o));
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i)
      if (i < len) p[i] = o[i];
  }
}
template <int n>
__device__ __forceinline__ void store_params(void* p, int dtype, int64_t at, int len, const float* v) {
  if (dtype == SVDQ_DT_F32)
    store_params_as<n>(static_cast<float*>(p) + at, len, v);
  else if (dtype == SVDQ_DT_BF16)
    store_params_as<n>(static_cast<Bf16*>(p) + at, len, v);
  else
    store_params_as<n>(static_cast<Half*>(p) + at, len, v);
}

// Butterflies over 16 lanes with DPP moves (quad permutes for distances 1 and
// 2, then the mirrored half row and row, whose lanes hold the other halves'
// sums), then over the rows with the gfx950 lane swaps: every lane ends with
// the result, in one fixed order.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_mov(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;
__device__ __forceinline__ float add_dpp16(float v) {
  v += __uint_as_float(dpp_mov<kDppXor1>(__float_as_uint(v)));
  v += __uint_as_float(dpp_mov<kDppXor2>(__float_as_uint(v)));
  v += __uint_as_float(dpp_mov<kDppHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(dpp_mov<kDppMirror>(__float_as_uint(v)));
  return v;
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
// the largest of 8 lanes' (a half row's) or 16 lanes' (a row's) values
__device__ __forceinline__ uint32_t max_dpp8(uint32_t v) {
  v = umax(v, dpp_mov<kDppXor1>(v));
  v = umax(v, dpp_mov<kDppXor2>(v));
  return umax(v, dpp_mov<kDppHalfMirror>(v));
}
__device__ __forceinline__ uint32_t max_dpp16(uint32_t v) {
  v = max_dpp8(v);
  return umax(v, dpp_mov<kDppMirror>(v));
}
// sums over 16, 32 or 64 lanes
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  v = add_dpp16(v);
  if constexpr (LANES >= 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  if constexpr (LANES == 64) {
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(b[0]) + __uint_as_float(b[1]);
  }
  return v;
}

// sums over the lanes at the same place of a wave's SHARES parts
template <int SHARES>
__device__ __forceinline__ float shares_sum(float v) {
  if constexpr (SHARES == 4) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  if constexpr (SHARES >= 2) {
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(b[0]) + __uint_as_float(b[1]);
  }
  return v;
}

// ---------------------------------------------------------------------------
// E4M3 blocks of 128 with a power-of-two scale
// ---------------------------------------------------------------------------
// The exponent of a block whose largest magnitude has the float bits `amax`
// (sign cleared): the least e >= -126 with amax 2^-e <= 448 = 1.75 2^8. An
// infinity or a NaN (the largest bits of all) gives 120; its element then
// becomes the NaN code, and so do the sums it enters.
__device__ __forceinline__ int e4m3_exponent(uint32_t amax) {
  const int e = (int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : (e > 120 ? 120 : e);
}
// E4M3 codes of four values times 2^-e: v_cvt_scalef32_pk_fp8_f32 divides by
// the (normal) scale exactly and rounds once, to nearest even; |v| 2^-e <= 448
// never overflows; infinities and NaN become the NaN code.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float scale) {
  typedef __attribute__((ext_vector_type(2))) short s16x2;
  s16x2 r = {0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, scale, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, scale, true);
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// the larger magnitude bits of a packed bf16 pair and m (as float bits)
__device__ __forceinline__ uint32_t amax_bf16x2(uint32_t m, uint32_t w) {
  m = umax(m, (w << 16) & 0x7fffffffu);
  return umax(m, w & 0x7fff0000u);
}

// The bias gradient of 32 channels (n0 on) by a workgroup of THREADS: 32 chains
// a channel, each every 32nd block in order with eight loads at a time (there
// are few workgroups, so this is latency), then the 32 in order. `red` holds
// 32 * 33 floats of LDS.
template <int THREADS>
__device__ __forceinline__ void bias_grad_32(const float* sums, int blocks, int N, int n0, uint16_t* db, float* red) {
  const int cl = threadIdx.x & 31, n = n0 + cl;
#pragma unroll
  for (int k = threadIdx.x >> 5; k < 32; k += THREADS / 32) {
    float s = 0.f;
    for (int i = k; i < blocks; i += 8 * 32) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = n < N && i + 32 * u < blocks ? sums[(size_t)(i + 32 * u) * N + n] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
    red[k * 33 + cl] = s;
  }
  __syncthreads();
  if (threadIdx.x < 32 && n < N) {
    float t = red[cl];
#pragma unroll
    for (int i = 1; i < 32; ++i) t += red[i * 33 + cl];
    db[n] = from_f32<Bf16>(t).bits;
  }
}

}  // namespace svdq
