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

}  // namespace tb
