// RMS norm of activation rows with the residual's addition, the block
// rotation and the rounding to 8 bits in one pass over memory.
//
//   h = round(x + r),  n_k = h_k w_k / sqrt(mean h^2 + eps),
//   n_b <- H (d_b * n_b) / 32 per 1024-block (optional),
//   y = n, or per group scale = max|n| / Q and y = round(n / scale).
//
// One block per row; the row is held in shared memory as fp32.
#pragma once
#include <cuda_fp8.h>

#include "hadamard.cuh"
#include "tb_device.cuh"

namespace tb {

constexpr int kNormThreads = 256;
constexpr int kNormMaxK = 32768;

// dtype codes of the C ABI as the kernels get them
enum : int { DT_BF16 = 0, DT_FP16 = 1, DT_FP32 = 2, DT_INT8 = 3, DT_E4M3 = 5 };

__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, int dt) {
  switch (dt) {
    case DT_BF16: return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    case DT_FP16: return __half2float(static_cast<const __half*>(p)[i]);
    default: return static_cast<const float*>(p)[i];
  }
}

__device__ __forceinline__ void store_from_f32(void* p, int64_t i, int dt, float v) {
  switch (dt) {
    case DT_BF16: static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v); break;
    case DT_FP16: static_cast<__half*>(p)[i] = __float2half_rn(v); break;
    default: static_cast<float*>(p)[i] = v; break;
  }
}

// 8-bit code of v = n / scale
__device__ __forceinline__ uint8_t code8(float v, int dt) {
  if (dt == DT_INT8) {
    const int q = __float2int_rn(v);  // NaN gives 0
    return static_cast<uint8_t>(static_cast<int8_t>(q < -127 ? -127 : (q > 127 ? 127 : q)));
  }
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3));
}

struct NormParams {
  const void* x;
  const void* residual;
  void* residual_out;
  const void* weight;
  const int8_t* signs;
  void* y;
  float* y_scales;
  int64_t K;
  int group;  // 0: floating output
  int xt, rt, wt, yt;
  float eps;
};

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s += red[w];
  __syncthreads();
  return s;
}

// Largest absolute value as its fp32 bits: NaN above infinity above the rest.
__device__ __forceinline__ uint32_t block_max_bits(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t s = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s = max(s, red[w]);
  __syncthreads();
  return s;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

constexpr uint32_t kInfBits = 0x7F800000u;
constexpr uint32_t kTinyBits = (127u - 100u) << 23;  // 2^-100

// Scale of a group with this largest |n| (as bits), and the factor that takes
// n to n / scale.
__device__ __forceinline__ void group_scale(uint32_t amax_bits, float q, float* scale, float* inv) {
  const float amax = __uint_as_float(amax_bits);
  if (amax_bits >= kInfBits) {
    *scale = *inv = __uint_as_float(0x7FC00000u);
  } else if (amax_bits < kTinyBits) {
    *scale = *inv = 0.f;
  } else {
    *scale = amax / q;
    *inv = q / amax;
  }
}

__global__ void __launch_bounds__(kNormThreads) rms_norm_kernel(const NormParams p) {
  extern __shared__ float row[];
  __shared__ float red[kNormThreads / 32];
  const int tid = threadIdx.x, K = static_cast<int>(p.K);
  const int64_t base = static_cast<int64_t>(blockIdx.x) * p.K;
  float ss = 0.f;
  for (int k = tid; k < K; k += kNormThreads) {
    float h = load_as_f32(p.x, base + k, p.xt);
    if (p.residual != nullptr) {
      h += load_as_f32(p.residual, base + k, p.rt);
      store_from_f32(p.residual_out, base + k, p.rt, h);
      h = load_as_f32(p.residual_out, base + k, p.rt);
    }
    row[k] = h;
    ss += h * h;
  }
  ss = block_sum(ss, red);
  float inv;
  if (ss < 1e30f && ss > 1e-20f) {
    inv = 1.f / sqrtf(ss / static_cast<float>(K) + p.eps);
  } else {
    // squares that leave fp32's range: sum them scaled by a power of two
    uint32_t mb = 0;
    for (int k = tid; k < K; k += kNormThreads) mb = max(mb, abs_bits(row[k]));
    mb = block_max_bits(mb, reinterpret_cast<uint32_t*>(red));
    const int e = mb >= kInfBits ? 0 : (mb == 0 ? 0 : ilogbf(__uint_as_float(mb)));
    float s2 = 0.f;
    for (int k = tid; k < K; k += kNormThreads) {
      const float h = ldexpf(row[k], -e);
      s2 += h * h;
    }
    s2 = block_sum(s2, red);
    inv = static_cast<float>(1.0 / sqrt(ldexp(static_cast<double>(s2) / K, 2 * e) + static_cast<double>(p.eps)));
  }
  for (int k = tid; k < K; k += kNormThreads) {
    float n = row[k] * inv;
    if (p.weight != nullptr) n *= load_as_f32(p.weight, k, p.wt);
    if (p.signs != nullptr) n *= static_cast<float>(p.signs[k]);
    row[k] = n;
  }
  __syncthreads();
  if (p.signs != nullptr) {
    for (int h = 1; h < kHB; h <<= 1) {
      for (int i = tid; i < K / 2; i += kNormThreads) {
        const int a = 2 * (i & ~(h - 1)) + (i & (h - 1));
        const float u = row[a], v = row[a + h];
        row[a] = u + v;
        row[a + h] = u - v;
      }
      __syncthreads();
    }
    for (int k = tid; k < K; k += kNormThreads) row[k] *= kHNorm;
    __syncthreads();
  }
  if (p.group == 0) {
    for (int k = tid; k < K; k += kNormThreads) store_from_f32(p.y, base + k, p.yt, row[k]);
    return;
  }
  const float q = p.yt == DT_INT8 ? 127.f : 448.f;
  uint8_t* y = static_cast<uint8_t*>(p.y);
  if (p.group == K) {
    uint32_t mb = 0;
    for (int k = tid; k < K; k += kNormThreads) mb = max(mb, abs_bits(row[k]));
    mb = block_max_bits(mb, reinterpret_cast<uint32_t*>(red));
    float scale, is;
    group_scale(mb, q, &scale, &is);
    if (tid == 0) p.y_scales[blockIdx.x] = scale;
    for (int k = tid; k < K; k += kNormThreads) y[base + k] = code8(row[k] * is, p.yt);
    return;
  }
  // groups of 128: one warp each, in turn
  const int warp = tid >> 5, lane = tid & 31, G = K / 128;
  for (int g = warp; g < G; g += kNormThreads / 32) {
    uint32_t mb = 0;
    for (int j = lane; j < 128; j += 32) mb = max(mb, abs_bits(row[128 * g + j]));
    mb = __reduce_max_sync(0xffffffffu, mb);
    float scale, is;
    group_scale(mb, q, &scale, &is);
    if (lane == 0) p.y_scales[static_cast<int64_t>(blockIdx.x) * G + g] = scale;
    for (int j = lane; j < 128; j += 32) y[base + 128 * g + j] = code8(row[128 * g + j] * is, p.yt);
  }
}

}  // namespace tb
