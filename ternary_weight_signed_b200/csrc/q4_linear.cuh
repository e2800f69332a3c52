// Linear layer with 4-bit g128 weights:
//   y[m, n] = sum_g s[n, g] sum_{k in g} q[n, k] x'[m, k].
//
// x' (scaled, rotated) goes to the workspace as fp32; then one warp per output
// row takes the row's groups, a lane four codes of each.
#pragma once
#include "norm.cuh"
#include "tb_device.cuh"

namespace tb {

constexpr int kQ4Warps = 8;
constexpr int kQ4Tokens = 8;  // tokens per pass over a weight row

__global__ void q4_convert_kernel(const void* __restrict__ x, int xt, const float* __restrict__ x_scales, int group,
                                  float* __restrict__ out, int64_t n, int K) {
  const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (i >= n) return;
  float v;
  if (xt == DT_INT8) {
    v = static_cast<float>(static_cast<const int8_t*>(x)[i]);
  } else if (xt == DT_E4M3) {
    v = __half2float(__nv_cvt_fp8_to_halfraw(static_cast<const __nv_fp8_storage_t*>(x)[i], __NV_E4M3));
  } else {
    v = load_as_f32(x, i, xt);
  }
  if (x_scales != nullptr) v *= x_scales[i / group];
  out[i] = v;
}

__global__ void __launch_bounds__(32 * kQ4Warps)
    q4_linear_kernel(const float* __restrict__ x, const uint8_t* __restrict__ packed,
                     const uint16_t* __restrict__ scales, void* __restrict__ y, int yt, int64_t M, int64_t N, int K) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kQ4Warps + warp;
  if (n >= N) return;
  const int G = K / 128;
  const uint16_t* codes = reinterpret_cast<const uint16_t*>(packed + n * (K / 2));
  for (int64_t m0 = 0; m0 < M; m0 += kQ4Tokens) {
    float acc[kQ4Tokens];
#pragma unroll
    for (int t = 0; t < kQ4Tokens; ++t) acc[t] = 0.f;
    for (int g = 0; g < G; ++g) {
      const uint32_t c = codes[32 * g + lane];
      const float s = __half2float(__ushort_as_half(scales[n * G + g]));
#pragma unroll
      for (int t = 0; t < kQ4Tokens; ++t) {
        if (m0 + t >= M) break;
        const float4 v = *reinterpret_cast<const float4*>(x + (m0 + t) * K + 128 * g + 4 * lane);
        const float d = v.x * (static_cast<int>(c & 15u) - 8) + v.y * (static_cast<int>((c >> 4) & 15u) - 8) +
                        v.z * (static_cast<int>((c >> 8) & 15u) - 8) + v.w * (static_cast<int>(c >> 12) - 8);
        acc[t] += s * d;
      }
    }
#pragma unroll
    for (int t = 0; t < kQ4Tokens; ++t) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
      if (lane == 0 && m0 + t < M) store_from_f32(y, (m0 + t) * N + n, yt, acc[t]);
    }
  }
}

// ---------------------------------------------------------------------------
// Activation prep: x (bf16, fp16, or 8 bits with scales), rotated when signs is
// non-null, as fp16 in the order that a packed word is unpacked in (k = 0, 4, 1,
// 5, 2, 6, 3, 7 inside 8), with one fp32 factor a token.  The factor is the
// power of two that brings the row's largest magnitude under 2^15 (rotated: 2^10,
// a block's sums can grow 32-fold), so that bf16 rows of any size keep their 8
// bits in fp16; an 8-bit row with one scale is exact as it is and its scale is
// the factor.  Values below 2^-29 of the row's largest lose bits.
// One block of 128 threads a row; two passes over it (the second hits L2).
template <typename TIn>
__device__ __forceinline__ void q4_load8(const TIn* p, float v[8]) { load8<TIn>(p, v); }
template <>
__device__ __forceinline__ void q4_load8<int8_t>(const int8_t* p, float v[8]) { load_signs8(p, v); }
template <>
__device__ __forceinline__ void q4_load8<__nv_fp8_e4m3>(const __nv_fp8_e4m3* p, float v[8]) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? u.x : u.y;
    const __half2_raw r =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(r));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

template <typename TIn>
__global__ void __launch_bounds__(kHThreads)
    q4_prep_kernel(const TIn* __restrict__ x, const float* __restrict__ x_scales, int group,
                   const int8_t* __restrict__ signs, __half* __restrict__ out, float* __restrict__ factor, int K) {
  constexpr bool k8 = sizeof(TIn) == 1;
  __shared__ float sm[kHB];
  __shared__ uint32_t red[kHThreads / 32];
  pdl_launch_dependents();
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, G = K / 128;
  const TIn* xr = x + row * K;
  // the largest magnitude of the row as fp32 bits (NaN and infinity above all)
  float f = 1.f;    // x' = x f
  float out_f = 1.f;  // x = x' out_f
  if (!k8 || group == 128) {
    uint32_t mb = 0;
    if constexpr (k8) {
      for (int g = tid; g < G; g += kHThreads) mb = max(mb, abs_bits(x_scales[row * G + g] * 448.f));
    } else {
      for (int k = 8 * tid; k < K; k += 8 * kHThreads) {
        float v[8];
        q4_load8<TIn>(xr + k, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) mb = max(mb, abs_bits(v[i]));
      }
    }
    mb = block_max_bits(mb, red);
    // 2^e <= largest < 2^(e+1); a row that holds a NaN or an infinity stays as it is
    const int top = signs != nullptr ? 9 : 14;
    const int e = mb >= kInfBits ? 0 : max(static_cast<int>(mb >> 23) - 127, -96) - top;
    f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    out_f = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  } else {
    out_f = x_scales[row];
  }
  if (tid == 0) factor[row] = out_f;
  for (int k = 8 * tid; k < K; k += 8 * kHThreads) {
    float v[8];
    q4_load8<TIn>(xr + k, v);
    float c = f;
    if constexpr (k8) {
      if (group == 128) c *= x_scales[row * G + (k >> 7)];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= c;
    if constexpr (!k8) {
      if (signs != nullptr) {
        float d[8];
        load_signs8(signs + k, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= d[i];
        fwht1024(v, sm);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= kHNorm;
      }
    }
    const float o[8] = {v[0], v[4], v[1], v[5], v[2], v[6], v[3], v[7]};
    store8<__half>(out + row * K + k, o);
  }
}

}  // namespace tb
