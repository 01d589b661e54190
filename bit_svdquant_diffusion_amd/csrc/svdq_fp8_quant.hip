// E4M3 quantizers of the FP8 linear: for a block of 128 values v,
//
//   e = the least e >= -126 with max|v| 2^-e <= 448,  code = rne_e4m3(v 2^-e),
//
// the scale byte e + 127 (E8M0). A power of two makes the quotient exact, so
// a code is one correct rounding of v / scale, and the block-scaled MFMA
// applies the scale by itself. Memory-bound: bf16 in once, codes out once.
#include <algorithm>

#include "svdq_internal.h"
#include "svdq_layout.h"
#include "svdq_types.h"

namespace svdq {

namespace {

// Blocks along the rows: eight lanes a block, 16 channels (32 bytes) a lane; a
// wave takes 1024 channels of a row (two rows' took 0.5 us longer for 1003
// rows). `plain` scales: [blocks / 4][M][4]. Channels in [K, Kp) get zero
// codes (K % 16 == 0: whole lanes).
__global__ __launch_bounds__(256) void fp8_quant_rows_kernel(const uint16_t* x, uint32_t units, uint32_t chunks, int64_t M, int K,
                                                             int Kp, int plain, uint8_t* q, uint8_t* s, uint32_t* tickets) {
  const uint32_t block = blockIdx.y * gridDim.x + blockIdx.x;
  if (tickets && block == 0 && threadIdx.x < kFp8Tickets) tickets[threadIdx.x] = 0;
  const uint32_t unit = block * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= units) return;
  const uint32_t row = unit / chunks;
  const int lane = threadIdx.x & 63, at = (int)(unit - row * chunks) * 1024 + lane * 16;
  u32x4 v0 = u32x4{0, 0, 0, 0}, v1 = v0;
  if (at < K) {
    const uint16_t* p = x + (size_t)row * K + at;
    v0 = *reinterpret_cast<const u32x4*>(p);
    v1 = *reinterpret_cast<const u32x4*>(p + 8);
  }
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) amax = amax_bf16x2(amax_bf16x2(amax, v0[i]), v1[i]);
  const int e = e4m3_exponent(max_dpp8(amax));
  const float sc = exp2_int(e);
  if (at < Kp) {
    *reinterpret_cast<u32x4*>(q + (size_t)row * Kp + at) =
        u32x4{e4m3x4(bf16lo(v0[0]), bf16hi(v0[0]), bf16lo(v0[1]), bf16hi(v0[1]), sc),
              e4m3x4(bf16lo(v0[2]), bf16hi(v0[2]), bf16lo(v0[3]), bf16hi(v0[3]), sc),
              e4m3x4(bf16lo(v1[0]), bf16hi(v1[0]), bf16lo(v1[1]), bf16hi(v1[1]), sc),
              e4m3x4(bf16lo(v1[2]), bf16hi(v1[2]), bf16lo(v1[3]), bf16hi(v1[3]), sc)};
    const int kb = at / 128;
    if ((lane & 7) == 0) s[plain ? ((size_t)(kb / 4) * M + row) * 4 + kb % 4 : fp8_scale_index(M, row, kb)] = (uint8_t)(e + 127);
  }
}

// A 128 x 128 tile of a bf16 matrix [M][C], read once: codes with blocks
// along the tokens, transposed ([C][Mp]), and where asked codes with blocks
// along the channels and the tile's sums per channel. A thread holds four
// consecutive tokens of 8 channels, so four tokens' codes of a channel are one
// word of the transposed tile, which leaves through LDS in whole 128-byte
// rows. Sums and maxima over the 32 token groups go through LDS in order (rows
// past M are zeros).
//
// Measured, both matrices with row codes and sums: 4608 tokens of 3072 and
// 12288 channels 48 us (268 MB in and out, 5.6 TB/s: the inputs come partly
// from the caches); 777 of 1552 and 2064 10.0 us, of which 4.5 go when the two
// kinds of codes are not stored and 3.2 are the launch and the loads.
constexpr int kTLd = 33;   // words of a transposed row in LDS (32 and one against bank conflicts)
__global__ __launch_bounds__(512) void fp8_quant_t_kernel(Fp8QuantT ma, Fp8QuantT mb, int64_t M, int64_t blocks_a,
                                                          uint32_t* tickets) {
  if (blockIdx.x == 0 && threadIdx.x < 2 * kFp8Tickets) tickets[threadIdx.x] = 0;
  __shared__ uint32_t lds[2 * 32 * 128];   // maxima and sums [32][128] each, then codes [128][kTLd]
  __shared__ uint32_t red[2][4][128];
  __shared__ float col_scale[128];
  const bool second = blockIdx.x >= blocks_a;
  const Fp8QuantT& t = second ? mb : ma;
  const int64_t blk = second ? blockIdx.x - blocks_a : blockIdx.x;
  const int ct = (t.C + 127) / 128;
  const int64_t tm = blk / ct, Mp = round128(M);
  const int c0 = (int)(blk - tm * ct) * 128, tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
  const int64_t m0 = tm * 128 + rg * 4;
  const int c = c0 + cg * 8;
  u32x4 v[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    v[p] = u32x4{0, 0, 0, 0};
    if (m0 + p < M && c < t.C) v[p] = *reinterpret_cast<const u32x4*>(t.x + (m0 + p) * t.C + c);
  }
  // value of token p, channel i of this thread
  auto val = [&](int p, int i) { return (i & 1) ? bf16hi(v[p][i >> 1]) : bf16lo(v[p][i >> 1]); };
  if (t.qt) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int p = 0; p < 4; ++p) m = umax(m, __float_as_uint(val(p, i)) & 0x7fffffffu);
      lds[rg * 128 + cg * 8 + i] = m;
    }
  }
  if (t.sums) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      lds[32 * 128 + rg * 128 + cg * 8 + i] = __float_as_uint((val(0, i) + val(1, i)) + (val(2, i) + val(3, i)));
  }
  if (t.q) {
    const int Cp = (int)round128(t.C);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) amax = amax_bf16x2(amax, v[p][i]);
      const int e = e4m3_exponent(max_dpp16(amax));
      const float sc = exp2_int(e);
      if (m0 + p < M) {
        *reinterpret_cast<u32x2*>(t.q + (size_t)(m0 + p) * Cp + c) =
            u32x2{e4m3x4(val(p, 0), val(p, 1), val(p, 2), val(p, 3), sc), e4m3x4(val(p, 4), val(p, 5), val(p, 6), val(p, 7), sc)};
        if (cg == 0) t.s[fp8_scale_index(M, m0 + p, c0 / 128)] = (uint8_t)(e + 127);
      }
    }
  }
  if (!t.qt && !t.sums) return;
  __syncthreads();
  const int quarter = tid >> 7, rc = tid & 127;   // reductions: channel rc, token groups 8 quarter .. +8
  if (t.qt) {
    uint32_t amax = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) amax = umax(amax, lds[(8 * quarter + k) * 128 + rc]);
    red[0][quarter][rc] = amax;
  }
  if (t.sums) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += __uint_as_float(lds[32 * 128 + (8 * quarter + k) * 128 + rc]);
    red[1][quarter][rc] = __float_as_uint(sum);
  }
  __syncthreads();
  if (quarter == 0 && t.qt) {
    const int e = e4m3_exponent(umax(umax(red[0][0][rc], red[0][1][rc]), umax(red[0][2][rc], red[0][3][rc])));
    col_scale[rc] = exp2_int(e);
    if (c0 + rc < t.C) t.st[fp8_scale_index(t.C, c0 + rc, tm)] = (uint8_t)(e + 127);
  }
  if (quarter == 1 && t.sums && c0 + rc < t.C)
    t.sums[(size_t)tm * t.C + c0 + rc] = (__uint_as_float(red[1][0][rc]) + __uint_as_float(red[1][1][rc])) +
                                         (__uint_as_float(red[1][2][rc]) + __uint_as_float(red[1][3][rc]));
  if (!t.qt) return;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i)
    lds[(cg * 8 + i) * kTLd + rg] = e4m3x4(val(0, i), val(1, i), val(2, i), val(3, i), col_scale[cg * 8 + i]);
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int ch = p * 64 + (tid >> 3), part = tid & 7;   // eight lanes write a channel's 128 codes
    if (c0 + ch < t.C) {
      const uint32_t* w = lds + ch * kTLd + part * 4;
      *reinterpret_cast<u32x4*>(t.qt + (size_t)(c0 + ch) * Mp + tm * 128 + part * 16) = u32x4{w[0], w[1], w[2], w[3]};
    }
  }
}

__global__ __launch_bounds__(1024) void fp8_bias_grad_kernel(Fp8BiasGrad a) {
  __shared__ float red[32 * 33];
  bias_grad_32<1024>(a.sums, a.blocks, a.N, blockIdx.x * 32, a.db, red);
}

__global__ __launch_bounds__(256) void fp8_zero_kernel(uint32_t* p, size_t n) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) p[i] = 0;
}

// A weight matrix [N][K]: one scale per 128 x 128 block, codes [N][K] and,
// for the input's gradient, transposed [K][N] with the scales transposed. One
// workgroup a block; a thread holds four output rows of 16 channels. The
// largest finite value gives the scale: infinities and NaN are the NaN code
// under any, and the block's other channels keep their values. (A token's
// block needs no such care, as all of its row's sums are NaN.)
template <typename T>
__global__ __launch_bounds__(256) void fp8_pack_kernel(const T* w, int K, int N, uint8_t* q, uint8_t* s, uint8_t* qt,
                                                       uint8_t* st) {
  __shared__ uint32_t lds[128 * kTLd];
  __shared__ uint32_t red[4];
  const int k0 = blockIdx.x * 128, n0 = blockIdx.y * 128, tid = threadIdx.x, cg = tid & 7, rg = tid >> 3;
  const int k = k0 + cg * 16;
  float v[4][16];
  uint32_t amax = 0;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int n = n0 + rg * 4 + p;
#pragma unroll
    for (int i = 0; i < 16; i += kVec<T>) {
      Vec<T> in;
      in.w = u32x4{0, 0, 0, 0};
      if (n < N && k < K) in = load_vec<T>(w + (size_t)n * K, k + i, kVec<T>);
#pragma unroll
      for (int t = 0; t < kVec<T>; ++t) {
        v[p][i + t] = in.at(t);
        const uint32_t mag = __float_as_uint(v[p][i + t]) & 0x7fffffffu;
        amax = umax(amax, mag < 0x7f800000u ? mag : 0u);
      }
    }
  }
  amax = max_dpp16(amax);
  amax = umax(amax, (uint32_t)__shfl_xor((int)amax, 16));
  amax = umax(amax, (uint32_t)__shfl_xor((int)amax, 32));
  if ((tid & 63) == 0) red[tid >> 6] = amax;
  __syncthreads();
  const int e = e4m3_exponent(umax(umax(red[0], red[1]), umax(red[2], red[3])));
  const float sc = exp2_int(e);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int n = n0 + rg * 4 + p;
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = e4m3x4(v[p][4 * i], v[p][4 * i + 1], v[p][4 * i + 2], v[p][4 * i + 3], sc);
    if (n < N && k < K) *reinterpret_cast<u32x4*>(q + (size_t)n * K + k) = o;
  }
  if (tid == 0) {
    // a row's last block also writes the row's padding (zeros)
    const int rk = fp8_block_row(K), rn = fp8_block_row(N);
    s[(size_t)blockIdx.y * rk + blockIdx.x] = (uint8_t)(e + 127);
    if (blockIdx.x == gridDim.x - 1)
      for (int i = gridDim.x; i < rk; ++i) s[(size_t)blockIdx.y * rk + i] = 0;
    if (st) {
      st[(size_t)blockIdx.x * rn + blockIdx.y] = (uint8_t)(e + 127);
      if (blockIdx.y == gridDim.y - 1)
        for (int i = gridDim.y; i < rn; ++i) st[(size_t)blockIdx.x * rn + i] = 0;
    }
  }
  if (!qt) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) lds[(cg * 16 + i) * kTLd + rg] = e4m3x4(v[0][i], v[1][i], v[2][i], v[3][i], sc);
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int ch = p * 32 + rg;
    if (k0 + ch < K && n0 + cg * 16 < N) {
      const uint32_t* o = lds + ch * kTLd + cg * 4;
      *reinterpret_cast<u32x4*>(qt + (size_t)(k0 + ch) * N + n0 + cg * 16) = u32x4{o[0], o[1], o[2], o[3]};
    }
  }
}

}  // namespace

hipError_t launch_fp8_quant_rows(const uint16_t* x, int64_t M, int K, uint8_t* q, uint8_t* s, bool plain, uint32_t* tickets,
                                 hipStream_t st) {
  const int Kp = (int)round128(K), chunks = (Kp + 1023) / 1024;
  const int64_t units = M * chunks;
  const dim3 grid = many_groups((units + 3) / 4);   // (at most 2^30 units)
  hipLaunchKernelGGL(fp8_quant_rows_kernel, grid, dim3(256), 0, st, x, (uint32_t)units, (uint32_t)chunks, M, K, Kp, plain ? 1 : 0,
                     q, s, tickets);
  return hipGetLastError();
}

hipError_t launch_fp8_quant_t(const Fp8QuantT& a, const Fp8QuantT& b, int64_t M, uint32_t* tickets, hipStream_t st) {
  const int64_t rows = (M + 127) / 128;
  const int64_t na = a.x ? rows * ((a.C + 127) / 128) : 0, nb = b.x ? rows * ((b.C + 127) / 128) : 0;
  if (na + nb == 0) return hipSuccess;
  hipLaunchKernelGGL(fp8_quant_t_kernel, dim3((unsigned)(na + nb)), dim3(512), 0, st, a, b, M, na, tickets);
  return hipGetLastError();
}

hipError_t launch_fp8_bias_grad(const Fp8BiasGrad& a, hipStream_t st) {
  hipLaunchKernelGGL(fp8_bias_grad_kernel, dim3((a.N + 31) / 32), dim3(1024), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_fp8_zero(void* p, size_t bytes, int num_cus, hipStream_t st) {
  const size_t n = bytes / 4;
  const unsigned grid = (unsigned)std::min<size_t>((n + 255) / 256, (size_t)num_cus * 8);
  hipLaunchKernelGGL(fp8_zero_kernel, dim3(grid), dim3(256), 0, st, (uint32_t*)p, n);
  return hipGetLastError();
}

hipError_t launch_fp8_pack(const void* w, int dtype, int K, int N, uint8_t* q, uint8_t* s, uint8_t* qt, uint8_t* st,
                           hipStream_t stream) {
  const dim3 grid((K + 127) / 128, (N + 127) / 128), b(256);
  if (dtype == SVDQ_DT_F32)
    hipLaunchKernelGGL(fp8_pack_kernel<float>, grid, b, 0, stream, (const float*)w, K, N, q, s, qt, st);
  else if (dtype == SVDQ_DT_BF16)
    hipLaunchKernelGGL(fp8_pack_kernel<Bf16>, grid, b, 0, stream, (const Bf16*)w, K, N, q, s, qt, st);
  else
    hipLaunchKernelGGL(fp8_pack_kernel<Half>, grid, b, 0, stream, (const Half*)w, K, N, q, s, qt, st);
  return hipGetLastError();
}

}  // namespace svdq
