// 4-bit g128 weights (layout in include/ternary_b200.h): pack, unpack, and the
// producer side, which folds the rotation into a dense matrix and rounds every
// 128-group to q in -8..7 with s = fp16(fp32(max|w'| / 7)).
//
// The producer works in fp64 like prepare.cuh (same fold, one warp per row and
// 1024-block): for bf16 and fp16 input the fold's sums are exact, so codes and
// scales do not depend on summation order.
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

// grid: ceil(K / 1024) * ceil(N / kPwWarps) blocks, one warp per (row, block).
template <typename TIn>
__global__ void __launch_bounds__(32 * kPwWarps)
    q4_prepare_kernel(const TIn* __restrict__ w, const int8_t* __restrict__ signs, uint8_t* __restrict__ packed,
                      uint16_t* __restrict__ scales, int64_t N, int K) {
  __shared__ __align__(16) double xbuf[kPwWarps][512];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nblk = (K + kHB - 1) / kHB;
  const int blk = static_cast<int>(blockIdx.x % nblk);
  const int64_t row = static_cast<int64_t>(blockIdx.x / nblk) * kPwWarps + warp;
  if (row >= N) return;  // a whole warp; nothing below synchronises beyond the warp
  const int G = K >> 7;
  const int64_t at = row * K + static_cast<int64_t>(blk) * kHB;
  double v[32];
  if (signs != nullptr) {
    pw_load_folded<TIn>(w + at, signs + static_cast<int64_t>(blk) * kHB, xbuf[warp], lane, v);
  } else {
    const bool in = blk * kHB + 32 * lane < K;  // K % 128 == 0: whole groups of four lanes
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = in ? static_cast<double>(to_f32<TIn>(w[at + 32 * lane + i])) : 0.0;
  }
  double m = 0.0;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = fmax(m, fabs(v[i]));
  m = fmax(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmax(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const float sf = static_cast<float>(__ddiv_rn(m, 7.0));
  const __half s16 = __float2half_rn(sf < kQ4MaxScale ? sf : kQ4MaxScale);
  const double s = static_cast<double>(__half2float(s16));
  uint32_t wd[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const double q = s > 0.0 ? rint(__ddiv_rn(v[i], s)) : 0.0;
    wd[i >> 3] |= static_cast<uint32_t>(static_cast<int>(fmin(fmax(q, -8.0), 7.0)) + 8) << (4 * (i & 7));
  }
  const int g = blk * 8 + (lane >> 2);
  if (g < G) {
    if ((lane & 3) == 0) scales[row * G + g] = __half_as_ushort(s16);
    *reinterpret_cast<uint4*>(packed + (at >> 1) + 16 * lane) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
  }
}

}  // namespace tb
