// 4-bit g128 weights (layout in include/ternary_b200.h): pack, unpack, and the
// producer side, which folds the rotation into a dense matrix and rounds every
// 128-group to q in -8..7 with s = fp16(fp32(max|w'| / 7)).
//
// The fold's codes and scales are those of exact sums (fp32 with a bound on its error
// where that decides them, else exact fp32 slices, else fp64), so they do not depend on
// summation order.  Without a fold the values are fp32 as they come.  17408 x 5120 bf16
// folded, with its unpacking: 260 us (412 us with all sums in fp64, 359
// with all in exact slices); 1024 x 5120 fp32 unfolded: 8 us.
#pragma once
#include "norm.cuh"
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

// One (row, 1024-block) folded in fp64: any input.  xb: 512 doubles of the warp's own.
template <typename TIn>
__device__ __noinline__ void q4_fold_block_fp64(const TIn* __restrict__ w, const int8_t* __restrict__ signs,
                                                uint8_t* __restrict__ packed, uint16_t* __restrict__ scales, int lane,
                                                double* xb) {
  double v[32];
  pw_load_folded<TIn>(w, signs, xb, lane, v);
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
  if ((lane & 3) == 0) scales[lane >> 2] = __half_as_ushort(s);
  *reinterpret_cast<uint4*>(packed + 16 * lane) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
}

// One (row, 1024-block) folded exactly.
//
// 16-bit input is folded in fp32.  With the block scaled by a power of two to
// |u| < 2, u = h + l with h a multiple of 2^-12 and l one of 2^-26, |l| <= 2^-13: 1024
// of either add up to less than 2^24 of their units, so every sum of the two
// transforms is exact in fp32, and so is their sum in fp64.  A value that needs more
// than the two slices (a bf16 below 2^-19 of 2, 3 blocks in 1000 of normal weights)
// and fp32 input send the block to the fp64 fold.
template <typename TIn>
__device__ __noinline__ void q4_fold_block(const TIn* __restrict__ src, const int8_t* __restrict__ sg,
                                           uint8_t* __restrict__ dst, uint16_t* __restrict__ sdst, int lane, bool vec,
                                           float* buf) {
  if constexpr (sizeof(TIn) == 2) {
    float h[4][8], l[4][8];
    uint32_t mb = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = 256 * j + 8 * lane;
      norm_load8<TIn>(src, k, vec, h[j]);
      const uint2 s = *reinterpret_cast<const uint2*>(sg + k);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[j][e] = __uint_as_float(__float_as_uint(h[j][e]) ^ (((e < 4 ? s.x : s.y) << (24 - 8 * (e & 3))) & 0x80000000u));
        mb = max(mb, abs_bits(h[j][e]));
      }
    }
    mb = __reduce_max_sync(0xffffffffu, mb);
    const int E = static_cast<int>(mb >> 23) - 127;  // 2^E <= largest < 2^(E+1)
    bool fits = E >= -100 && E <= 100;
    const float scale_in = __uint_as_float(static_cast<uint32_t>(127 - (fits ? E : 0)) << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = h[j][e] * scale_in;
        // adding 1.5 2^11 (2^-3) rounds to a multiple of 2^-12 (2^-26)
        h[j][e] = __fsub_rn(__fadd_rn(u, 0x1.8p11f), 0x1.8p11f);
        const float r = __fsub_rn(u, h[j][e]);
        l[j][e] = __fsub_rn(__fadd_rn(r, 0.1875f), 0.1875f);
        fits = fits && l[j][e] == r;
      }
    if (__all_sync(0xffffffffu, fits)) {
      norm_fwht(h, buf, lane);
      norm_fwht(l, buf, lane);
      const float out = __uint_as_float(static_cast<uint32_t>(127 + E - 5) << 23);  // 2^E / 32
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // the group's largest |w'|, exact: of the values whose fp32 sum is largest
        float f[8], m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[e] = h[j][e] + l[j][e];
          m = fmaxf(m, fabsf(f[e]));
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        double top = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (fabsf(f[e]) == m) top = fmax(top, fabs(static_cast<double>(h[j][e]) + static_cast<double>(l[j][e])));
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
        const __half s = q4_scale(top * static_cast<double>(out));
        const float sf = __half2float(s), inv = sf > 0.f ? 1.f / sf * out : 0.f;
        uint32_t wd = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          wd |= (sf > 0.f ? q4_code(f[e], inv, s,
                                    [&] {
                                      return (static_cast<double>(h[j][e]) + static_cast<double>(l[j][e])) *
                                             static_cast<double>(out);
                                    })
                          : 8u)
                << (4 * e);
        *reinterpret_cast<uint32_t*>(dst + 128 * j + 4 * lane) = wd;
        if ((lane & 15) == 0) sdst[2 * j + (lane >> 4)] = __half_as_ushort(s);
      }
      return;
    }
  }
  q4_fold_block_fp64<TIn>(src, sg, dst, sdst, lane, reinterpret_cast<double*>(buf));
}

// Folded: grid K / 1024 * N blocks of one warp (warps of one block would wait for those
// of them that fold exactly).
//
// First a plain fp32 transform with a bound on its error: ten levels of sums of at
// most U = sum |u| round by less than 10.1 2^-24 U in all.  Where neither a scale nor a
// code can depend on that error (four blocks in five of normal weights), it is done; the
// others are folded exactly.  Either way the bits are those of exact arithmetic.
//
// Bound by instruction fetch (straight-line code, each warp at another place in it) and
// latency, so the most blocks an SM holds: 32 of 64 registers 260 us, 24 of 80 294, 16
// of 128 392; two warps a block 275, four 303, eight 367.
template <typename TIn>
__global__ void __launch_bounds__(32, 32)
    q4_fold_kernel(const TIn* __restrict__ w, const int8_t* __restrict__ signs, uint8_t* __restrict__ packed,
                   uint16_t* __restrict__ scales, int K, bool vec) {
  __shared__ __align__(16) float buf[kNormRotFloats];  // (the fp64 fold takes 1024 of them)
  const int lane = threadIdx.x;
  const int nblk = K / kHB;
  const int blk = static_cast<int>(blockIdx.x % nblk);
  const int64_t row = blockIdx.x / nblk;
  const int64_t at = row * K + static_cast<int64_t>(blk) * kHB;
  const TIn* src = w + at;
  const int8_t* sg = signs + static_cast<int64_t>(blk) * kHB;
  uint8_t* dst = packed + (at >> 1);
  uint16_t* sdst = scales + at / 128;
  float v[4][8], sum = 0.f;
  uint32_t mb = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = 256 * j + 8 * lane;
    norm_load8<TIn>(src, k, vec, v[j]);
    const uint2 s = *reinterpret_cast<const uint2*>(sg + k);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[j][e] = __uint_as_float(__float_as_uint(v[j][e]) ^ (((e < 4 ? s.x : s.y) << (24 - 8 * (e & 3))) & 0x80000000u));
      mb = max(mb, abs_bits(v[j][e]));
      sum += fabsf(v[j][e]);
    }
  }
  mb = __reduce_max_sync(0xffffffffu, mb);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  // |w'| stays far from the ends of fp32 (an empty or a wild block is folded exactly)
  bool sure = mb > (27u << 23) && mb < (227u << 23);
  norm_fwht(v, buf, lane);
  const float err = sum * 6.03e-7f;  // 10.1 2^-24, with room for the rounding of the sum itself
  float m[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m[j] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m[j] = fmaxf(m[j], fabsf(v[j][e]));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], o));
  }
  // lane g < 8 takes the scale of group g (piece g / 2, half g % 2); it is sure where
  // both ends of the interval round to it
  float mine = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float o = __shfl_sync(0xffffffffu, m[j], 16 * (lane & 1));
    if ((lane >> 1) == j) mine = o;
  }
  const double hi = (static_cast<double>(mine) + static_cast<double>(err)) * 0.03125;
  const double lo = (static_cast<double>(mine) - static_cast<double>(err)) * 0.03125;
  const __half s_hi = q4_scale(hi);
  const float sf = __half2float(s_hi);
  if (lane < 8)
    sure = sure && lo > 0.0 && __half_as_ushort(q4_scale(lo)) == __half_as_ushort(s_hi) && sf >= 6.2e-5f && sf < kQ4MaxScale;
  const float inv_mine = 0.03125f / sf;
  uint32_t wd[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float inv = __shfl_sync(0xffffffffu, inv_mine, 2 * j + (lane >> 4));
    // |r| <= 7.01: no code is clipped.  r is off by err inv and three roundings
    const float edge = 0.5f - (err * inv * 1.01f + 2e-6f);
    uint32_t acc = 0x88888888u;
    float worst = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float q = fmaf(v[j][e], inv, 12582912.f);  // the nearest integer in the mantissa
      worst = fmaxf(worst, fabsf(v[j][e] * inv - (q - 12582912.f)));
      acc += (__float_as_uint(q) - 0x4B400000u) << (4 * e);
    }
    wd[j] = acc;
    sure = sure && worst < edge;
  }
  if (!__all_sync(0xffffffffu, sure)) {
    q4_fold_block<TIn>(src, sg, dst, sdst, lane, vec, buf);
    return;
  }
  if (lane < 8) sdst[lane] = __half_as_ushort(s_hi);
#pragma unroll
  for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t*>(dst + 128 * j + 4 * lane) = wd[j];
}

// Not folded: every value is one of fp32, and a warp takes eight 128-groups of a
// row, four values of each a lane (the same grid).
template <typename TIn>
__global__ void __launch_bounds__(32 * kPwWarps)
    q4_round_kernel(const TIn* __restrict__ w, uint8_t* __restrict__ packed, uint16_t* __restrict__ scales, int64_t N,
                    int K, bool vec) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nblk = (K - 1) / kHB + 1, G = K >> 7;  // (K + 1023 may pass 2^31)
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
