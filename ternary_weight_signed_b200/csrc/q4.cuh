// 4-bit g128 weights (layout in include/ternary_b200.h): pack, unpack, and the
// producer side, which folds the rotation into a dense matrix and rounds every
// 128-group to q in -8..7 with s = fp16(fp32(max|w'| / 7)).
//
// The fold works in fp64 like prepare.cuh's (one warp per row and 1024-block): for
// bf16 and fp16 input its sums are exact, so codes and scales do not depend on
// summation order.  Without a fold the values are fp32 as they come.  17408 x 5120
// bf16 folded: about 390 us, by the latency of its fp64 sums at 16 warps an SM; 1024 x
// 5120 fp32 unfolded: 8 us.
#pragma once
#include "prepare.cuh"
#include "tb_device.cuh"

namespace tb {

constexpr float kQ4MaxScale = 8188.f;  // 8 s stays inside fp16

// One thread per 16 codes -> 8 packed bytes.
__global__ void q4_pack_kernel(const int4* __restrict__ codes, uint2* __restrict__ out, int64_t n,
                               uint32_t* counter) {
  const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  uint32_t bad = 0;
  if (i < n) {
    const int4 v = codes[i];
    const int8_t* c = reinterpret_cast<const int8_t*>(&v);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int q = c[j] < -8 ? -8 : (c[j] > 7 ? 7 : c[j]);
      bad += q != c[j] ? 1u : 0u;
      w[j >> 3] |= static_cast<uint32_t>(q + 8) << (4 * (j & 7));
    }
    out[i] = make_uint2(w[0], w[1]);
  }
  count_invalid(bad, counter);
}

__global__ void q4_unpack_kernel(const uint2* __restrict__ in, int4* __restrict__ codes, int64_t n) {
  const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (i >= n) return;
  const uint2 v = in[i];
  int4 o;
  int8_t* c = reinterpret_cast<int8_t*>(&o);
#pragma unroll
  for (int j = 0; j < 16; ++j)
    c[j] = static_cast<int8_t>(static_cast<int>(((j < 8 ? v.x : v.y) >> (4 * (j & 7))) & 15u) - 8);
  codes[i] = o;
}

// The group scale of a group's largest |w'|, and its reciprocal for q4_code.
__device__ __forceinline__ __half q4_scale(double amax) {
  const float sf = static_cast<float>(__ddiv_rn(amax, 7.0));
  return __float2half_rn(sf < kQ4MaxScale ? sf : kQ4MaxScale);
}

// q + 8 for the value v (exact(): the same in fp64), s > 0 and inv = 1 / s.  The
// fp32 quotient is off by less than 3 2^-24 of it (v's rounding, inv's and the
// product's), under 1.5e-6 as |v / s| < 8; only within 4e-6 of a border between two
// codes does the fp64 quotient decide (32 instructions saved on the others).
template <typename F>
__device__ __forceinline__ uint32_t q4_code(float v, float inv, __half s, F&& exact) {
  const float r = v * inv;
  float q = rintf(r);
  if (fabsf(fabsf(r - q) - 0.5f) < 4e-6f) q = static_cast<float>(rint(__ddiv_rn(exact(), static_cast<double>(__half2float(s)))));
  return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(q, -8.f), 7.f)) + 8);
}

// Folded: grid ceil(K / 1024) * ceil(N / kPwWarps) blocks, one warp per (row, block).
template <typename TIn>
__global__ void __launch_bounds__(32 * kPwWarps)
    q4_fold_kernel(const TIn* __restrict__ w, const int8_t* __restrict__ signs, uint8_t* __restrict__ packed,
                   uint16_t* __restrict__ scales, int64_t N, int K) {
  __shared__ __align__(16) double xbuf[kPwWarps][512];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nblk = K / kHB;
  const int blk = static_cast<int>(blockIdx.x % nblk);
  const int64_t row = static_cast<int64_t>(blockIdx.x / nblk) * kPwWarps + warp;
  if (row >= N) return;  // a whole warp; nothing below synchronises beyond the warp
  const int G = K >> 7;
  const int64_t at = row * K + static_cast<int64_t>(blk) * kHB;
  double v[32];
  pw_load_folded<TIn>(w + at, signs + static_cast<int64_t>(blk) * kHB, xbuf[warp], lane, v);
  double m = 0.0;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = fmax(m, fabs(v[i]));
  m = fmax(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmax(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const __half s = q4_scale(m);
  const float sf = __half2float(s), inv = sf > 0.f ? 1.f / sf : 0.f;
  uint32_t wd[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 32; ++i)
    wd[i >> 3] |= (sf > 0.f ? q4_code(static_cast<float>(v[i]), inv, s, [&] { return v[i]; }) : 8u) << (4 * (i & 7));
  if ((lane & 3) == 0) scales[row * G + blk * 8 + (lane >> 2)] = __half_as_ushort(s);
  *reinterpret_cast<uint4*>(packed + (at >> 1) + 16 * lane) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
}

// Not folded: every value is one of fp32, and a warp takes eight 128-groups of a
// row, four values of each a lane (the same grid).
template <typename TIn>
__global__ void __launch_bounds__(32 * kPwWarps)
    q4_round_kernel(const TIn* __restrict__ w, uint8_t* __restrict__ packed, uint16_t* __restrict__ scales, int64_t N,
                    int K, bool vec) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nblk = (K + kHB - 1) / kHB, G = K >> 7;
  const int g0 = static_cast<int>(blockIdx.x % nblk) * 8, ng = min(8, G - g0);
  const int64_t row = static_cast<int64_t>(blockIdx.x / nblk) * kPwWarps + warp;
  if (row >= N) return;
  const TIn* src = w + row * K + 128 * g0 + 4 * lane;
  float v[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= ng) break;
    const TIn* p = src + 128 * j;
    if (vec) {
      if constexpr (sizeof(TIn) == 4) {
        const float4 f = *reinterpret_cast<const float4*>(p);
        v[j][0] = f.x, v[j][1] = f.y, v[j][2] = f.z, v[j][3] = f.w;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        const TIn* h = reinterpret_cast<const TIn*>(&u);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][e] = to_f32<TIn>(h[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j][e] = to_f32<TIn>(p[e]);
    }
  }
  // lane j takes the scale of group j
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= ng) break;
    const float a = fmaxf(fmaxf(fabsf(v[j][0]), fabsf(v[j][1])), fmaxf(fabsf(v[j][2]), fabsf(v[j][3])));
    const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
    if (lane == j) m = top;
  }
  const __half mine = q4_scale(static_cast<double>(m));
  const float mine_inv = __half2float(mine) > 0.f ? 1.f / __half2float(mine) : 0.f;
  if (lane < ng) scales[row * G + g0 + lane] = __half_as_ushort(mine);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= ng) break;
    const __half s = __ushort_as_half(static_cast<uint16_t>(__shfl_sync(0xffffffffu, static_cast<uint32_t>(__half_as_ushort(mine)), j)));
    const float inv = __shfl_sync(0xffffffffu, mine_inv, j);
    uint32_t c = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c |= (inv > 0.f ? q4_code(v[j][e], inv, s, [&] { return static_cast<double>(v[j][e]); }) : 8u) << (4 * e);
    *reinterpret_cast<uint16_t*>(packed + ((row * K + 128 * (g0 + j)) >> 1) + 2 * lane) = static_cast<uint16_t>(c);
  }
}

}  // namespace tb
