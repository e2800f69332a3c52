// RMS norm of activation rows with the residual's addition, the block
// rotation and the rounding to 8 bits in one pass over memory.
//
//   h = round(x + r),  n_k = h_k w_k / sqrt(mean h^2 + eps),
//   n_b <- H (d_b * n_b) / 32 per 1024-block (optional),
//   y = n, or per group scale = max|n| / Q and y = round(n / scale).
//
// Bound by HBM past a few hundred rows (16384 x 5120, fp32 residual, e4m3 groups:
// 148 us over one set of buffers, 0.96 of the measured copy rate; 152 to 162 over
// three), rotated by latency (2048 x 5120: 20.4 us; 20 warps an SM issue in half of the
// cycles and wait for their rows' copies and the transposes about equally), by the
// launch and two passes of latency for one row (2.7 us).  Rows over 16384 values go
// without copies and spill (2048 x 17408 127 us, 0.35 of the copy rate; rotated 137).
// A row stays in registers between its one load and its one store: a
// thread holds NV pieces of 8 values (16-byte loads of 16-bit types), a block a
// row, and the blocks walk the rows.  In the rotated kernel a warp holds a whole
// 1024-block, so the transform needs no block-wide barrier: distances 1-4, 256 and
// 512 are in a lane, 8-128 after a transpose through 4 KB of shared memory and back
// (128 wavefronts a block; 160 shuffles would be the other way).
#pragma once
#include <cuda_fp8.h>

#include "hadamard.cuh"
#include "tb_device.cuh"

namespace tb {

constexpr int kNormRotFloats = 4 * 264;  // a warp's transpose buffer: 8 floats of padding every 256

// dtype codes of the C ABI as the kernels get them
enum : int { DT_BF16 = 0, DT_FP16 = 1, DT_FP32 = 2, DT_INT8 = 3, DT_E4M3 = 5 };

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
  int64_t M;
  int K;
  int group;  // 0: floating output
  int xt, rt, wt, yt;
  float eps;
  bool vec;    // every pointer that is read or written in pieces starts on 16 bytes
  bool stall;  // failure-detection test: no copies
};

// Largest absolute value as its fp32 bits: NaN above infinity above the rest.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

constexpr uint32_t kInfBits = 0x7F800000u;
constexpr uint32_t kTinyBits = (127u - 100u) << 23;  // 2^-100

// Block-wide reductions with one barrier each: `red` holds two sets of 32 words
// that consecutive reductions use in turn.
struct BlockReduce {
  uint32_t* red;
  int set;
  __device__ __forceinline__ uint32_t* next() {
    set ^= 32;
    return red + set;
  }
  // kAny: and whether `any` holds for one of the threads, in every thread's `any`.
  template <bool kAny = false>
  __device__ __forceinline__ float sum(float v, bool* any = nullptr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (nw == 1) {
      if constexpr (kAny) *any = __any_sync(0xffffffffu, *any);
      return v;
    }
    uint32_t* r = next();
    if (lane == 0) r[threadIdx.x >> 5] = __float_as_uint(v);
    if constexpr (kAny)
      *any = __syncthreads_or(*any);
    else
      __syncthreads();
    v = lane < nw ? __uint_as_float(r[lane]) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  __device__ __forceinline__ uint32_t max_bits(uint32_t v) {
    v = __reduce_max_sync(0xffffffffu, v);
    const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (nw == 1) return v;
    uint32_t* r = next();
    if (lane == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, lane < nw ? r[lane] : 0u);
  }
};

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

// f(T()) with T the floating type of the code dt: one branch around all of a
// row's pieces instead of one in each.
template <typename F>
__device__ __forceinline__ void with_type(int dt, F&& f) {
  if (dt == DT_BF16)
    f(__nv_bfloat16());
  else if (dt == DT_FP16)
    f(__half());
  else
    f(0.f);
}

// 8 values at element i; vec: by 16-byte accesses.
template <typename T>
__device__ __forceinline__ void norm_load8(const void* p, int64_t i, bool vec, float (&v)[8]) {
  const T* q = static_cast<const T*>(p) + i;
  if (vec) {
    load8<T>(q, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = to_f32<T>(q[e]);
  }
}

template <typename T>
__device__ __forceinline__ void norm_store8(void* p, int64_t i, bool vec, const float (&v)[8]) {
  T* q = static_cast<T*>(p) + i;
  if (vec) {
    store8<T>(q, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = from_f32<T>(v[e]);
  }
}

// The values k0 .. k0 + 7 of a row of K at element base, those outside it zero.
template <typename T>
__device__ __forceinline__ void norm_load_cut(const void* p, int64_t base, int k0, int K, bool vec, float (&v)[8]) {
  if (k0 >= 0 && k0 + 8 <= K) {
    norm_load8<T>(p, base + k0, vec, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = k0 + e >= 0 && k0 + e < K ? to_f32<T>(static_cast<const T*>(p)[base + k0 + e]) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void norm_store_cut(void* p, int64_t base, int k0, int K, bool vec, const float (&v)[8]) {
  if (k0 >= 0 && k0 + 8 <= K) {
    norm_store8<T>(p, base + k0, vec, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k0 + e >= 0 && k0 + e < K) static_cast<T*>(p)[base + k0 + e] = from_f32<T>(v[e]);
  }
}

// Rounds v to T, pairs at a time (the same conversions as store8's).
template <typename T>
__device__ __forceinline__ void norm_round8(float (&v)[8]) {
  if constexpr (!__is_same(T, float)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float2 f;
      if constexpr (__is_same(T, __half))
        f = __half22float2(__floats2half2_rn(v[2 * e], v[2 * e + 1]));
      else
        f = __bfloat1622float2(__floats2bfloat162_rn(v[2 * e], v[2 * e + 1]));
      v[2 * e] = f.x;
      v[2 * e + 1] = f.y;
    }
  }
}

// Codes of 8 values n with n / scale = n inv.
__device__ __forceinline__ void norm_store_codes8(uint8_t* p, int64_t i, int dt, bool vec, const float (&v)[8],
                                                  float inv) {
  uint32_t w[2] = {0u, 0u};
  if (dt == DT_INT8) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e >> 2] |= static_cast<uint32_t>(code8(v[e] * inv, DT_INT8)) << (8 * (e & 3));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(v[2 * e] * inv, v[2 * e + 1] * inv),
                                                                  __NV_SATFINITE, __NV_E4M3))
                   << (16 * (e & 1));
  }
  if (vec) {
    *reinterpret_cast<uint2*>(p + i) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[i + e] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
  }
}

// Two butterflies at once: (a, b) <- (a + b, a - b) on pairs of floats (packed
// fp32 adds; a - b as a + b (-1), the same rounding).
__device__ __forceinline__ void butterfly2(float2& a, float2& b) {
  const unsigned long long minus = 0xBF800000BF800000ull;
  unsigned long long s, d;
  const unsigned long long x = *reinterpret_cast<unsigned long long*>(&a), y = *reinterpret_cast<unsigned long long*>(&b);
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(s) : "l"(x), "l"(y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(y), "l"(minus), "l"(x));
  a = *reinterpret_cast<float2*>(&s);
  b = *reinterpret_cast<float2*>(&d);
}

// Transform of 32 values (16 pairs) over all five index bits.
__device__ __forceinline__ void norm_fwht32(float2 (&u)[16]) {
#pragma unroll
  for (int l = 0; l < 16; ++l) u[l] = make_float2(u[l].x + u[l].y, u[l].x - u[l].y);
#pragma unroll
  for (int h = 1; h < 16; h <<= 1)
#pragma unroll
    for (int l = 0; l < 16; ++l)
      if ((l & h) == 0) butterfly2(u[l], u[l + h]);
}

// Unnormalised transform of the warp's 1024 values: piece j of lane l holds
// 256 j + 8 l .. + 7.  buf: kNormRotFloats floats of the warp's own.
__device__ __forceinline__ void norm_fwht(float (&v)[4][8], float* buf, int lane) {
  float2 u[16];
#pragma unroll
  for (int l = 0; l < 16; ++l) u[l] = make_float2(v[l >> 2][2 * (l & 3)], v[l >> 2][2 * (l & 3) + 1]);
  norm_fwht32(u);  // over e and j
  // transpose: lane 8 j + i takes the values 256 j + 8 l + i over l
#pragma unroll
  for (int l = 0; l < 16; l += 2)
    *reinterpret_cast<float4*>(buf + 264 * (l >> 2) + 8 * lane + 2 * (l & 3)) =
        make_float4(u[l].x, u[l].y, u[l + 1].x, u[l + 1].y);
  __syncwarp();
  float* col = buf + 264 * (lane >> 3) + (lane & 7);
#pragma unroll
  for (int l = 0; l < 16; ++l) u[l] = make_float2(col[16 * l], col[16 * l + 8]);
  norm_fwht32(u);  // over the lane
#pragma unroll
  for (int l = 0; l < 16; ++l) {
    col[16 * l] = u[l].x;
    col[16 * l + 8] = u[l].y;
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) load8<float>(buf + 264 * j + 8 * lane, v[j]);
  __syncwarp();  // buf may be written again
}

// Layouts of a row over the threads: a piece is 8 consecutive values, piece j of
// thread t at 8 (j T + t) (rotated: at 1024 warp + 256 j + 8 lane).  Shifted (K % 8
// != 0): pieces are cut at multiples of 8 of the element's number in the whole
// tensor, so that those inside a row are 16-byte accesses whatever its start, and only
// a row's first and last piece go value by value.
enum : int { NORM_PIECES = 0, NORM_ROTATED = 1, NORM_SHIFTED = 2 };

// The weights from element k on (ones when there are none), in the rotated kernel
// with the signs on them: exact in the weights' own type.
template <typename T, int kMode>
__device__ __forceinline__ void norm_weight8(const NormParams& p, int k, float (&w)[8]) {
  if (p.weight != nullptr) {
    norm_load8<T>(p.weight, k, p.vec, w);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.f;
  }
  if constexpr (kMode == NORM_ROTATED) {
    const uint2 s = *reinterpret_cast<const uint2*>(p.signs + k);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      w[e] = __uint_as_float(__float_as_uint(w[e]) ^ (((e < 4 ? s.x : s.y) << (24 - 8 * (e & 3))) & 0x80000000u));
  }
}

// kBulk: the rows come through shared memory, each by one or two bulk copies
// issued a row ahead (enough beside three to six blocks on an SM; two rows ahead
// leave room for fewer blocks: 170 against 149 us for 16384 x 5120), so that the
// copies of the next row run while a row is reduced, rotated and stored, and the
// weights (with the signs) lie there too; for many rows (16-byte accesses only).
// A block whose wait for a row gives up asks for no further row: after the row's
// barrier all its threads leave, the first once its copy has landed.

template <int NV, int kMode, int kMaxThreads, bool kBulk>
__global__ void __launch_bounds__(kMaxThreads, kMaxThreads <= 320 ? 2 : 1) rms_norm_kernel(const NormParams p) {
  extern __shared__ __align__(16) float norm_smem[];
  __shared__ uint32_t red[64];
  __shared__ uint64_t bar;
  pdl_launch_dependents();
  const int tid = threadIdx.x, T = blockDim.x, warp = tid >> 5, lane = tid & 31, K = p.K;
  BlockReduce reduce{red, 0};
  int cut = 0;  // shifted: values of the row's first piece that belong to the row before
  auto at = [&](int j) {
    return kMode == NORM_ROTATED ? 1024 * warp + 256 * j + 8 * lane : 8 * (j * T + tid) - cut;
  };
  auto in = [&](int j) { return kMode == NORM_ROTATED || at(j) < K; };
  uint8_t* weights = reinterpret_cast<uint8_t*>(norm_smem + (kMode == NORM_ROTATED ? (T >> 5) * kNormRotFloats : 0));
  const int w_size = p.wt == DT_FP32 ? 4 : 2;
  uint8_t* stage = weights + K * w_size;
  const uint32_t x_bytes = static_cast<uint32_t>(K) * (p.xt == DT_FP32 ? 4 : 2);
  const uint32_t r_bytes = p.residual == nullptr ? 0u : static_cast<uint32_t>(K) * (p.rt == DT_FP32 ? 4 : 2);
  auto fetch = [&](int64_t row) {
    if (p.stall || row >= p.M) return;
    mbar_arrive_expect_tx(&bar, x_bytes + r_bytes);
    bulk_load(stage, static_cast<const uint8_t*>(p.x) + row * x_bytes, x_bytes, &bar);
    if (r_bytes != 0) bulk_load(stage + x_bytes, static_cast<const uint8_t*>(p.residual) + row * r_bytes, r_bytes, &bar);
  };
  if constexpr (kBulk) {
    if (tid == 0) {
      mbar_init(&bar, 1);
      fence_mbar_init();
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (in(j)) {
        with_type(p.wt, [&](auto tw) {
          float w[8];
          norm_weight8<decltype(tw), kMode>(p, at(j), w);
          norm_store8<decltype(tw)>(weights, at(j), true, w);
        });
      }
    __syncthreads();
  }
  pdl_wait();
  if constexpr (kBulk) {
    if (tid == 0) fetch(blockIdx.x);
  }
  uint32_t phase = 0;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const int64_t base = row * K;
    float v[NV][8];
    bool gave_up = false;
    if constexpr (kMode == NORM_SHIFTED) {
      cut = p.vec ? static_cast<int>(base & 7) : 0;
      with_type(p.xt, [&](auto tx) {
#pragma unroll
        for (int j = 0; j < NV; ++j) norm_load_cut<decltype(tx)>(p.x, base, at(j), K, p.vec, v[j]);
      });
      if (p.residual != nullptr) {
        with_type(p.rt, [&](auto tr) {
          float r[NV][8];  // all loads before the first store
#pragma unroll
          for (int j = 0; j < NV; ++j) norm_load_cut<decltype(tr)>(p.residual, base, at(j), K, p.vec, r[j]);
#pragma unroll
          for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] += r[j][e];
            norm_round8<decltype(tr)>(v[j]);
            norm_store_cut<decltype(tr)>(p.residual_out, base, at(j), K, p.vec, v[j]);
          }
        });
      }
    } else {
      if constexpr (kBulk) gave_up = !mbar_wait(&bar, phase, FAULT_WAIT_FULL);
      const void* xp = kBulk ? static_cast<const void*>(stage) : p.x;
      const int64_t xbase = kBulk ? 0 : base;
      const bool vec = kBulk || p.vec;
      with_type(p.xt, [&](auto tx) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (in(j)) {
            norm_load8<decltype(tx)>(xp, xbase + at(j), vec, v[j]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = 0.f;
          }
        }
      });
      if (p.residual != nullptr) {
        const void* rp = kBulk ? static_cast<const void*>(stage + x_bytes) : p.residual;
        with_type(p.rt, [&](auto tr) {
          auto add = [&](int j, const float (&r)[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] += r[e];
            norm_round8<decltype(tr)>(v[j]);
            if (!gave_up) norm_store8<decltype(tr)>(p.residual_out, base + at(j), vec, v[j]);
          };
          if constexpr (kBulk) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
              if (in(j)) {
                float r[8];
                norm_load8<decltype(tr)>(rp, at(j), true, r);
                add(j, r);
              }
          } else {
            float r[NV][8];  // all loads before the first store
#pragma unroll
            for (int j = 0; j < NV; ++j)
              if (in(j)) norm_load8<decltype(tr)>(rp, base + at(j), vec, r[j]);
#pragma unroll
            for (int j = 0; j < NV; ++j)
              if (in(j)) add(j, r[j]);
          }
        });
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(v[j][e], v[j][e], ss);
    ss = reduce.sum<kBulk>(ss, &gave_up);
    if constexpr (kBulk) {
      if (gave_up) {
        if (tid == 0 && !p.stall) mbar_wait(&bar, phase, FAULT_WAIT_FULL);
        return;
      }
      // every thread has its values in registers: the stage takes the next row
      if (tid == 0) fetch(row + gridDim.x);
      phase ^= 1u;
    }
    float inv;
    if (ss < 1e30f && ss > 1e-20f) {
      inv = 1.f / sqrtf(ss / static_cast<float>(K) + p.eps);
    } else {
      // squares that leave fp32's range: sum them scaled by a power of two
      uint32_t mb = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) mb = max(mb, abs_bits(v[j][e]));
      mb = reduce.max_bits(mb);
      const int ex = mb >= kInfBits ? 0 : (mb == 0 ? 0 : ilogbf(__uint_as_float(mb)));
      float s2 = 0.f;
      for (int j = 0; j < NV; ++j)
        for (int e = 0; e < 8; ++e) {
          const float h = ldexpf(v[j][e], -ex);
          s2 += h * h;
        }
      s2 = reduce.sum(s2);
      inv = static_cast<float>(1.0 / sqrt(ldexp(static_cast<double>(s2) / K, 2 * ex) + static_cast<double>(p.eps)));
    }
    if constexpr (kMode == NORM_ROTATED) inv *= kHNorm;  // the transform's 1/32
    if constexpr (kMode == NORM_SHIFTED) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] *= inv;
      if (p.weight != nullptr)
        with_type(p.wt, [&](auto tw) {
          const decltype(tw)* src = static_cast<const decltype(tw)*>(p.weight);
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int k = at(j) + e;
              if (k >= 0 && k < K) v[j][e] *= to_f32(src[k]);
            }
        });
    } else {
      with_type(p.wt, [&](auto tw) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (in(j)) {
            float w[8];
            if constexpr (kBulk)
              norm_load8<decltype(tw)>(weights, at(j), true, w);
            else
              norm_weight8<decltype(tw), kMode>(p, at(j), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = v[j][e] * inv * w[e];
          }
      });
    }
    if constexpr (kMode == NORM_ROTATED) norm_fwht(v, norm_smem + warp * kNormRotFloats, lane);
    if (p.group == 0) {
      if constexpr (kMode == NORM_SHIFTED) {
        with_type(p.yt, [&](auto ty) {
#pragma unroll
          for (int j = 0; j < NV; ++j) norm_store_cut<decltype(ty)>(p.y, base, at(j), K, p.vec, v[j]);
        });
      } else {
        with_type(p.yt, [&](auto ty) {
#pragma unroll
          for (int j = 0; j < NV; ++j)
            if (in(j)) norm_store8<decltype(ty)>(p.y, base + at(j), kBulk || p.vec, v[j]);
        });
      }
      continue;
    }
    const float q = p.yt == DT_INT8 ? 127.f : 448.f;
    uint8_t* y = static_cast<uint8_t*>(p.y);
    uint32_t mb[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      mb[j] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) mb[j] = max(mb[j], abs_bits(v[j][e]));
    }
    float scale, is;
    if (p.group == K) {
#pragma unroll
      for (int j = 1; j < NV; ++j) mb[0] = max(mb[0], mb[j]);
      group_scale(reduce.max_bits(mb[0]), q, &scale, &is);
      if (tid == 0) p.y_scales[row] = scale;
      if constexpr (kMode == NORM_SHIFTED) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (at(j) >= 0 && at(j) + 8 <= K) {
            norm_store_codes8(y, base + at(j), p.yt, p.vec, v[j], is);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (at(j) + e >= 0 && at(j) + e < K) y[base + at(j) + e] = code8(v[j][e] * is, p.yt);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (in(j)) norm_store_codes8(y, base + at(j), p.yt, p.vec, v[j], is);
      }
    } else if constexpr (kMode != NORM_SHIFTED) {
      // groups of 128: 16 lanes of a piece
      const int64_t G = K / 128;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) mb[j] = max(mb[j], __shfl_xor_sync(0xffffffffu, mb[j], o));
        group_scale(mb[j], q, &scale, &is);
        if (in(j)) {
          if ((lane & 15) == 0) p.y_scales[row * G + (at(j) >> 7)] = scale;
          norm_store_codes8(y, base + at(j), p.yt, p.vec, v[j], is);
        }
      }
    }
  }
}

}  // namespace tb
