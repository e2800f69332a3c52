// Linear layer with 4-bit g128 weights:
//   y[m, n] = sum_g s[n, g] sum_{k in g} q[n, k] x'[m, k].
//
// Here: the activation prep (rotation, fp16 with a factor per token) that the
// pair GEMM and the rotated decode read, and the decode kernel for few tokens.
#pragma once
#include "gemm_pair.cuh"
#include "norm.cuh"
#include "tb_device.cuh"

namespace tb {

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

// ---------------------------------------------------------------------------
// Decode: up to 16 tokens.  The weights are read once and everything else has
// to fit beside that stream, so the kernel is built around it:
//   * a lane reads 16 bytes = 32 codes of a row, four lanes a row's 128-group,
//     straight into registers, one step ahead of the arithmetic; the codes are
//     never staged (nothing else of the CTA reads them);
//   * the products run on mma.sync m16n8k16 with the weights as the 16 rows and
//     the tokens as the 8 columns: q is exact in bf16 and in fp16, the products
//     are exact in fp32 and a group is summed in the fp32 accumulators (8 MMAs),
//     then scaled by s once.  A mask and a shift unpack two codes (k, k + 4) of
//     a packed word at a time, and x' is laid out in shared memory in that order,
//     one 16-byte load a lane for two MMAs.  The tensor pipe is not what binds
//     here; staging the unpacked codes for tcgen05 would move them twice more.
//   * rows are spread over the CTAs, the groups of K over Wk of a CTA's warps
//     (fp32 partial sums joined in shared memory in a fixed order) and, when x'
//     of all tokens does not fit one CTA, over the S CTAs of a cluster, which
//     read each other's partial sums through distributed shared memory.
// No atomics: the bits do not depend on scheduling.
constexpr int kQ4DecMaxThreads = 512;
constexpr int kQ4DecMaxM = 16;

enum : int { Q4X_BF16 = 0, Q4X_FP16 = 1, Q4X_INT8 = 2, Q4X_E4M3 = 3, Q4X_PREP = 4 };

struct Q4DecodeParams {
  const void* x;
  const float* group_scales;  // [M, G] of an 8-bit x, or NULL
  const float* factor;        // [M] or NULL
  const uint8_t* packed;
  const uint16_t* scales;
  void* y;
  int64_t N;
  int M, K, xmode, yt;
  int R, nblocks;  // rows of a block, blocks (a cluster takes every nclusters-th)
  int Wt, Wk;      // row-tile classes x K classes of a CTA's warps
  int S, Gs;       // cluster size, 128-groups of a CTA's K slice
};

__host__ __device__ constexpr int q4_dec_gp(int tpw) { return tpw >= 3 ? 1 : 4 / tpw; }
__host__ __device__ constexpr int64_t q4_dec_x_bytes(int M, int Gs) { return int64_t(256) * M * Gs; }
__host__ __device__ constexpr int64_t q4_dec_xs_bytes(int M, int Gs, bool xg) {
  return xg ? int64_t(4) * 8 * ((M + 7) / 8) * Gs : 0;
}
__host__ __device__ constexpr int64_t q4_dec_part_bytes(int M, int rows, int Wk) { return int64_t(4) * Wk * M * rows; }

template <typename TX>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (__is_same(TX, __half))
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes s and s + 4 of a packed word as the pair (q_s, q_{s+4}): the code set
// into the mantissa of 128 (bf16) or 1024 (fp16), then the bias taken off, both exact.
template <typename TX, int s>
__device__ __forceinline__ uint32_t q4_pair(uint32_t w) {
  if constexpr (__is_same(TX, __half)) {
    const uint32_t v = ((s < 2 ? w : w >> 8) & ((s & 1) ? 0x00F000F0u : 0x000F000Fu)) | 0x64006400u;
    const __half2 h = *reinterpret_cast<const __half2*>(&v);
    const __half2 q = (s & 1) ? __hfma2(h, __float2half2_rn(0.0625f), __float2half2_rn(-72.f))
                              : __hadd2(h, __float2half2_rn(-1032.f));
    return *reinterpret_cast<const uint32_t*>(&q);
  } else {
    const uint32_t v = ((w >> (4 * s)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 q =
        __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&v), __float2bfloat162_rn(-136.f));
    return *reinterpret_cast<const uint32_t*>(&q);
  }
}

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// 8 consecutive values of x in the order (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ uint4 q4_x8(const void* x, int64_t at, int xmode) {
  if (xmode == Q4X_PREP) return __ldcg(reinterpret_cast<const uint4*>(static_cast<const __half*>(x) + at));
  if (xmode <= Q4X_FP16) {
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at));
    return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                      __byte_perm(v.y, v.w, 0x7632));
  }
  const uint2 u = __ldcg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(x) + at));
  uint4 o;
  if (xmode == Q4X_INT8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(static_cast<float>(static_cast<int8_t>(u.x >> (8 * i))),
                                                     static_cast<float>(static_cast<int8_t>(u.y >> (8 * i))));
      (&o.x)[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t pair = __byte_perm(u.x, u.y, 0x0040u + 0x0011u * i);  // bytes i and i + 4
      const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(pair & 0xFFFFu), __NV_E4M3);
      (&o.x)[i] = static_cast<uint32_t>(r.x) | (static_cast<uint32_t>(r.y) << 16);
    }
  }
  return o;
}

// NT: token tiles of 8; TPW: 16-row tiles of a warp; TX: type of the products;
// XG: x has a scale per token and group.
template <int NT, int TPW, typename TX, bool XG>
__global__ void __launch_bounds__(kQ4DecMaxThreads, 1) q4_decode_kernel(const Q4DecodeParams p) {
  constexpr int GP = q4_dec_gp(TPW);  // groups a step: about 8 16-byte loads in flight a lane
  extern __shared__ __align__(16) uint8_t q4_smem[];
  const int M = p.M, T = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;
  const int rank = p.S > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int cluster = static_cast<int>(blockIdx.x) / p.S, nclusters = static_cast<int>(gridDim.x) / p.S;
  const int G = p.K >> 7, G0 = rank * p.Gs, Gn = max(0, min(p.Gs, G - G0));
  const int rows = 16 * TPW * p.Wt;  // of the partial sums' layout
  uint4* xf = reinterpret_cast<uint4*>(q4_smem);
  float* xsg = reinterpret_cast<float*>(q4_smem + q4_dec_x_bytes(M, p.Gs));
  float* part = reinterpret_cast<float*>(q4_smem + q4_dec_x_bytes(M, p.Gs) + q4_dec_xs_bytes(M, p.Gs, XG));

  const int wt = warp % p.Wt, wk = warp / p.Wt;
  const bool active = wk < p.Wk;
  const int nstep = active && Gn > wk * GP ? (Gn - wk * GP + p.Wk * GP - 1) / (p.Wk * GP) : 0;
  const int64_t stride8 = int64_t(4) * p.K;  // bytes of 8 rows

  uint4 w[GP][TPW][2];
  uint16_t sc[GP][TPW][2];
  auto load = [&](int blk, int j) {
    const int64_t row0 = static_cast<int64_t>(blk) * p.R;
    const int lim = static_cast<int>(min(static_cast<int64_t>(p.R), p.N - row0)) - 16 * TPW * wt - r;  // rows from r on
    const int64_t row = row0 + 16 * TPW * wt + r;
    const int g0 = (j * p.Wk + wk) * GP;
    const uint8_t* src = p.packed + row * (p.K >> 1) + static_cast<int64_t>(G0 + g0) * 64 + 16 * c;
    const uint16_t* ssrc = p.scales + row * G + G0 + g0;
#pragma unroll
    for (int gg = 0; gg < GP; ++gg) {
#pragma unroll
      for (int h = 0; h < 2 * TPW; ++h) {
        const bool ok = 8 * h < lim && g0 + gg < Gn;
        w[gg][h >> 1][h & 1] = ok ? ldg_stream(src + h * stride8 + 64 * gg) : make_uint4(0, 0, 0, 0);
        sc[gg][h >> 1][h & 1] = ok ? __ldg(ssrc + static_cast<int64_t>(8 * h) * G + gg) : uint16_t(0);
      }
    }
  };

  pdl_launch_dependents();
  if (nstep > 0) load(cluster, 0);  // weights do not wait for the previous kernel
  pdl_wait();
  for (int m = 0; m < M; ++m) {
    const int64_t base = static_cast<int64_t>(m) * p.K + static_cast<int64_t>(G0) * 128;
    for (int q = tid; q < 16 * Gn; q += T)  // q = 16 g + 4 c + i: codes 32 c + 8 i of group g
      xf[((q >> 4) * 4 + (q & 3)) * 4 * M + 4 * m + ((q >> 2) & 3)] = q4_x8(p.x, base + 8 * q, p.xmode);
  }
  if constexpr (XG) {
    for (int q = tid; q < 8 * NT * Gn; q += T) {
      const int g = q / (8 * NT), m = q - 8 * NT * g;
      xsg[q] = m < M ? __ldcg(p.group_scales + static_cast<int64_t>(m) * G + G0 + g) : 0.f;
    }
  }
  __syncthreads();

  for (int blk = cluster; blk < p.nblocks; blk += nclusters) {
    float acc[TPW][NT][4];
#pragma unroll
    for (int tt = 0; tt < TPW; ++tt)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[tt][t][e] = 0.f;
    for (int j = 0; j < nstep; ++j) {
      uint4 cw[GP][TPW][2];
      float cs[GP][TPW][2];
#pragma unroll
      for (int gg = 0; gg < GP; ++gg)
#pragma unroll
        for (int h = 0; h < 2 * TPW; ++h) {
          cw[gg][h >> 1][h & 1] = w[gg][h >> 1][h & 1];
          cs[gg][h >> 1][h & 1] = __half2float(__ushort_as_half(sc[gg][h >> 1][h & 1]));
        }
      // the next step's loads, over the end of the block
      if (j + 1 < nstep)
        load(blk, j + 1);
      else if (blk + nclusters < p.nblocks)
        load(blk + nclusters, 0);
#pragma unroll
      for (int gg = 0; gg < GP; ++gg) {
        const int g = (j * p.Wk + wk) * GP + gg;
        if (g >= Gn) break;  // the whole warp
        float d[TPW][NT][4];
#pragma unroll
        for (int tt = 0; tt < TPW; ++tt)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[tt][t][e] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 b[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t)
            b[t] = 8 * t + r < M ? xf[(g * 4 + i) * 4 * M + 32 * t + lane] : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int tt = 0; tt < TPW; ++tt) {
            const uint32_t lo = (&cw[gg][tt][0].x)[i], hi = (&cw[gg][tt][1].x)[i];
            uint32_t a0 = q4_pair<TX, 0>(lo), a1 = q4_pair<TX, 0>(hi), a2 = q4_pair<TX, 1>(lo), a3 = q4_pair<TX, 1>(hi);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816<TX>(d[tt][t], a0, a1, a2, a3, b[t].x, b[t].y);
            a0 = q4_pair<TX, 2>(lo), a1 = q4_pair<TX, 2>(hi), a2 = q4_pair<TX, 3>(lo), a3 = q4_pair<TX, 3>(hi);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816<TX>(d[tt][t], a0, a1, a2, a3, b[t].z, b[t].w);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float f0 = 1.f, f1 = 1.f;
          if constexpr (XG) {
            const float2 f = *reinterpret_cast<const float2*>(xsg + g * 8 * NT + 8 * t + 2 * c);
            f0 = f.x;
            f1 = f.y;
          }
#pragma unroll
          for (int tt = 0; tt < TPW; ++tt) {
            const float s0 = cs[gg][tt][0], s1 = cs[gg][tt][1];
            acc[tt][t][0] += (XG ? s0 * f0 : s0) * d[tt][t][0];
            acc[tt][t][1] += (XG ? s0 * f1 : s0) * d[tt][t][1];
            acc[tt][t][2] += (XG ? s1 * f0 : s1) * d[tt][t][2];
            acc[tt][t][3] += (XG ? s1 * f1 : s1) * d[tt][t][3];
          }
        }
      }
    }
    // partial sums [wk][token][row], joined over wk and then over the cluster
    if (active) {
#pragma unroll
      for (int tt = 0; tt < TPW; ++tt)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int m = 8 * t + 2 * c + (e & 1);
            if (m < M) part[(wk * M + m) * rows + 16 * (TPW * wt + tt) + r + 8 * (e >> 1)] = acc[tt][t][e];
          }
    }
    __syncthreads();
    const int64_t row0 = static_cast<int64_t>(blk) * p.R;
    const int nr = static_cast<int>(min(static_cast<int64_t>(p.R), p.N - row0));
    if (p.S > 1) {
      for (int o = tid; o < M * rows; o += T) {
        float v = part[o];
        for (int q = 1; q < p.Wk; ++q) v += part[q * M * rows + o];
        part[o] = v;
      }
      cluster_sync_all();
    }
    const int terms = p.S > 1 ? p.S : p.Wk;
    for (int o = tid * p.S + rank; o < M * nr; o += T * p.S) {
      const int m = o / nr, row = o - m * nr, at = m * rows + row;
      float v;
      if (p.S > 1) {
        v = 0.f;
        for (int q = 0; q < terms; ++q) v += ld_cluster_f32(cluster_map(smem_u32(part + at), q));
      } else {
        v = part[at];
        for (int q = 1; q < terms; ++q) v += part[q * M * rows + at];
      }
      if (p.factor != nullptr) v *= __ldcg(p.factor + m);
      store_from_f32(p.y, m * p.N + row0 + row, p.yt, v);
    }
    if (p.S > 1)
      cluster_sync_all();  // no CTA overwrites (or leaves) what its peers still read
    else
      __syncthreads();
  }
}

}  // namespace tb
