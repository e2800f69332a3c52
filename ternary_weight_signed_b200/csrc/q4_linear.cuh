// Linear layer with 4-bit g128 weights:
//   y[m, n] = sum_g s[n, g] sum_{k in g} q[n, k] x'[m, k].
//
// Here: the activation prep of the tcgen05 kernels (q4_mid.cuh, gemm_pair.cuh) and
// the decode kernel for up to 16 tokens with its own.
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
// One block a row, a thread for 8 values up to 8192 of them; longer rows are read
// twice (the second time from L2).
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
__global__ void __launch_bounds__(1024)
    q4_prep_kernel(const TIn* __restrict__ x, const float* __restrict__ x_scales, int group,
                   const int8_t* __restrict__ signs, __half* __restrict__ out, float* __restrict__ factor, int K) {
  constexpr bool k8 = sizeof(TIn) == 1;
  extern __shared__ __align__(16) float prep_smem[];  // rotated: 1024 floats per 128 threads
  __shared__ uint32_t red[64];
  pdl_launch_dependents();
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, T = blockDim.x, G = K / 128;
  const uint32_t k0 = 8 * tid, width = K, step = 8 * T;  // unsigned: k passes K, which may be next to 2^31
  const TIn* xr = x + row * K;
  float f = 1.f;      // x' = x f
  float out_f = 1.f;  // x = x' out_f
  float v[8];
  pdl_wait();
  if (k0 < width) q4_load8<TIn>(xr + k0, v);
  if (!k8 || group == 128) {
    // the largest magnitude of the row, or the largest scale of its groups (their codes
    // are under 2^9), as fp32 bits (NaN and infinity above all)
    uint32_t mb = 0;
    if constexpr (k8) {
      for (int g = tid; g < G; g += T) mb = max(mb, abs_bits(x_scales[row * G + g]));
    } else {
      for (uint32_t k = k0; k < width; k += step) {
        float u[8];
        if (k == k0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) u[i] = v[i];
        } else {
          q4_load8<TIn>(xr + k, u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) mb = max(mb, abs_bits(u[i]));
      }
    }
    mb = BlockReduce{red, 0}.max_bits(mb);
    // x' = x 2^-e: the largest comes to 2^top and more, under 2^(top + 1), or as near
    // as an fp32 factor takes it; a row that holds a NaN or an infinity stays as it is
    const int top = k8 ? 5 : (signs != nullptr ? 9 : 14);
    const int e = mb >= kInfBits ? 0 : max(static_cast<int>(mb >> 23) - 127 - top, -126);
    f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    out_f = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  } else {
    out_f = x_scales[row];
  }
  if (tid == 0) factor[row] = out_f;
  for (uint32_t k = k0; k < width; k += step) {
    if (k != k0) q4_load8<TIn>(xr + k, v);
    float c = f;
    if constexpr (k8) {
      if (group == 128) c *= x_scales[row * G + (k >> 7)];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= c;
    if constexpr (!k8) {
      if (signs != nullptr) {  // T is a multiple of 128 and K of 1024: whole groups of 128 threads
        float d[8];
        load_signs8(signs + k, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= d[i];
        fwht1024_group(v, prep_smem + 1024 * (tid >> 7), tid & 127, 1 + (tid >> 7));
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
// to fit beside that stream.
//   * The products run on mma.sync m16n8k32 in 8-bit integers, 16 weight rows by 8
//     columns, exact: the codes c = q + 8 as they are (a mask and a shift, 3
//     instructions for 8 codes), x' as 8-bit planes of a fixed-point number, a
//     column per plane and token.  Every group has its own power of two: three
//     planes hold a value to 2^-22 of its group's largest, two to 2^-15, and an int8
//     is one.  The sums of a group start from -8 sum x, which takes the bias off,
//     plus the bits of 1.5 2^23, which makes the integer sum a float's mantissa: one
//     subtraction instead of a conversion.  The groups are added in fp32.
//   * Measured on B200, cycles an MMA on one of the SM's four tensor pipes:
//     m16n8k16 f16 and m16n8k32 s8 8 with constant operands and 15-16 with ones that
//     change, m16n8k32 e4m3 35 (no pipe of its own).  The f16 form unpacks a 16 x 128
//     tile in 88 instructions, this one in 24 (1 x 17408 x 5120: 24.1 against 13.7 us
//     when it replaced it).  tcgen05 wants the codes unpacked to 8 or 16 bits in tensor
//     memory first; past 16 tokens that pays (q4_mid.cuh).
//   * One token, 17408 x 5120: 11.3 to 11.8 us a call (0.60 to 0.63 of the measured HBM
//     rate), of which 5 us stream; 151936 x 5120: 78.9 us (0.79).  bf16 tokens of 17408 x
//     5120 / 5120 x 17408, us: 2 11.8 / 14.6, 4 15.0 / 18.6, 5 17.3 / 19.1, 8 17.1 / 19.8, 16
//     24.1 / (q4_mid.cuh, 26.0).
//   * Each warp streams its own rows: boxes of up to 16 rows x 128 bytes (256
//     codes) by TMA into a ring of its own, refilled by the warp itself, so no warp
//     waits for another inside the loop.  K is spread over Wk of a CTA's warps
//     (fp32 partial sums joined in shared memory in a fixed order) and, when x' does
//     not fit one CTA, over the S CTAs of a cluster, which read each other's partial
//     sums through distributed shared memory.  No atomics: the bits do not depend on
//     scheduling.
constexpr int kQ4DecWarps = 16;      // of a CTA, one CTA an SM
constexpr int kQ4DecMaxM = 16;
constexpr int kQ4DecSlots = 2;       // boxes in flight a warp; 3 and 4 delay the loads of x behind them: 13.0 -> 13.8 us
// Tokens whose planes every CTA makes itself; more, and a rotated x, get them from a
// launch of its own.  In the CTAs / by the launch, us: 1 x 17408 x 5120 11.4 / 13.2, 4 x 15.0 /
// 16.4, 8 x 17.1 / 17.3; 4 x 5120 x 17408 18.7 / 18.8, 5 x 19.3 / 19.1, 8 x 21.7 / 19.8; int8 8 x
// 1024 x 5120 7.5 / 6.7.
constexpr int kQ4DecInCta = 4;

constexpr int kQ4MagicBits = 0x4B400000;   // 1.5 2^23; adding an integer below 2^22 to the bits adds it to the value
constexpr float kQ4Magic = 12582912.f;

enum : int { Q4X_BF16 = 0, Q4X_FP16 = 1, Q4X_INT8 = 2, Q4X_E4M3 = 3, Q4X_IMAGE = 4 };

// Planes of a value: three where they cost no column tile more than two would.
__host__ __device__ constexpr int q4_planes(int xmode, int M) { return xmode == Q4X_INT8 ? 1 : (M <= 5 ? 3 : 2); }

struct Q4DecodeParams {
  const void* x;
  const float* x_scales;  // of an 8-bit x, or of an image: [G][C], then the sums [G][C]
  const uint16_t* scales;
  void* y;
  int64_t N;
  int M, K, xmode, x_group, yt;
  int P, C;         // planes, columns = planes x tokens
  int rw, nblocks;  // rows of a warp's box; row blocks of Wt rw rows (a cluster takes every nclusters-th)
  int Wt, Wk;       // row classes x K classes of a CTA's warps
  int S, Gs;        // cluster size, 128-groups of a CTA's K slice (even)
  int part_at;      // byte offset of the partial sums in shared memory
  bool stall;       // failure-detection test: no copies
};

constexpr int kQ4DecBoxRows = 16;
constexpr int kQ4DecBoxBytes = kQ4DecBoxRows * 128;
// shared memory: rings | barriers | x planes [Gs][2][C][4] x 16 bytes | factors, sums [Gs][8 NT] each | partial sums
// (these over x where a CTA has one row block; rings and barriers are never written over:
// copies may be in flight after a wait that gave up)
// kb boxes (2 kb groups) a slot: two where x' is copied and leaves room, for half the
// waits and scale loads a group (16 x 17408 x 5120 25.2 -> 24.1 us); one where the CTA
// makes the planes itself, whose loads of x two would delay (1 x 6144 x 5120 6.6 -> 7.0)
__host__ __device__ constexpr int q4_dec_ring_bytes(int kb) { return kQ4DecWarps * kQ4DecSlots * kb * kQ4DecBoxBytes; }
constexpr int kQ4DecBarBytes = 8 * kQ4DecWarps * kQ4DecSlots;
__host__ __device__ constexpr int64_t q4_dec_x_bytes(int C, int Gs) { return int64_t(128) * C * Gs; }
__host__ __device__ constexpr int64_t q4_dec_f_bytes(int C, int Gs) { return int64_t(64) * ((C + 7) / 8) * Gs; }
__host__ __device__ constexpr int64_t q4_dec_part_bytes(int C, int rows, int Wk) { return int64_t(4) * Wk * C * rows; }

// Planes, factors and sums of a 128-group of one token, 32 consecutive values v a
// lane: lane c of the four that call this together holds the codes 32 c ..; lanes
// without a group of their own are not live and store nothing.  xs multiplies the
// group's values.  Column n of the group goes to dst[h C 4 + 4 n + c], h the half
// of the lane's codes.
__device__ __forceinline__ void q4_store_planes(const float (&v)[32], bool int8, float xs, int P, int M, int m, int C,
                                                uint4* dst, float* fdst, int* sdst, bool live) {
  const int c = threadIdx.x & 3;
  float f = 1.f, inv = 1.f;
  if (!int8) {
    uint32_t mb = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) mb = max(mb, abs_bits(v[j]));
    mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
    mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
    // the largest under 2^22 (three planes) or 1.9921 2^14 (two: the higher one stays under 128)
    const int top = P == 3 ? 21 : 14;
    // (steps of 2^-126 at least: 1 / step is an fp32 number)
    const int e = min(max(static_cast<int>((mb + (P == 3 ? 0u : 0x10200u)) >> 23) - 127, top - 126), 128);
    f = __uint_as_float(static_cast<uint32_t>(127 + top - e) << 23);
    inv = mb >= kInfBits ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(127 - top + e) << 23);
  }
  inv *= xs;
  int s[3] = {0, 0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[3][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // nearest integers as the mantissas of 1.5 2^23 + v f, then their signed
      // base-256 digits: with 128 added to every digit they are the bytes, and
      // flipping the top bits takes it off again
      uint32_t x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[j] = (__float_as_uint(fmaf(v[16 * h + 8 * i + j], f, kQ4Magic)) +
                (0x00808080u - static_cast<uint32_t>(kQ4MagicBits))) ^ 0x00808080u;
      // byte p of the values (0, 2, 4, 6) and (1, 3, 5, 7): 4 x 4 byte transposes
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const uint32_t lo = __byte_perm(x[o], x[o + 2], 0x5140), hi = __byte_perm(x[o + 4], x[o + 6], 0x5140);
        w[0][2 * i + o] = __byte_perm(lo, hi, 0x5410);
        w[1][2 * i + o] = __byte_perm(lo, hi, 0x7632);
        w[2][2 * i + o] =
            __byte_perm(__byte_perm(x[o], x[o + 2], 0x0062), __byte_perm(x[o + 4], x[o + 6], 0x0062), 0x5410);
      }
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) {  // plane p: digit p, column P - 1 - p of the token
#pragma unroll
      for (int o = 0; o < 4; ++o) s[p] = __dp4a(static_cast<int>(w[p][o]), 0x01010101, s[p]);
      if (p < P && live) dst[h * 4 * C + 4 * ((P - 1 - p) * M + m) + c] = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
    }
  }
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    s[p] += __shfl_xor_sync(0xffffffffu, s[p], 1);
    s[p] += __shfl_xor_sync(0xffffffffu, s[p], 2);
    if (p < P && live && c == 0) {
      const int n = (P - 1 - p) * M + m;
      fdst[n] = inv;
      sdst[n] = kQ4MagicBits - 8 * s[p];
    }
    inv *= 256.f;
  }
}

__device__ __forceinline__ void q4_load8_any(const void* x, int64_t at, int xmode, float v[8]) {
  switch (xmode) {
    case Q4X_BF16: load8<__nv_bfloat16>(static_cast<const __nv_bfloat16*>(x) + at, v); break;
    case Q4X_FP16: load8<__half>(static_cast<const __half*>(x) + at, v); break;
    case Q4X_INT8: q4_load8<int8_t>(static_cast<const int8_t*>(x) + at, v); break;
    default: q4_load8<__nv_fp8_e4m3>(static_cast<const __nv_fp8_e4m3*>(x) + at, v); break;
  }
}

// The planes of all tokens, once for the whole grid of the decode kernel (more
// than kQ4DecInCta tokens, or a rotated x): image [G][2][C][4] x 16 bytes, then
// factors and sums, [G][C] each.  grid (ceil(K / 1024), M), 128 threads: they
// load (and rotate) 8 values each, and the first 32 make the planes of the
// block's eight groups.
__global__ void __launch_bounds__(kHThreads)
    q4_planes_kernel(const void* __restrict__ x, int xmode, const float* __restrict__ x_scales, int group,
                     const int8_t* __restrict__ signs, uint4* __restrict__ image, float* __restrict__ factors, int M,
                     int K, int P, int C) {
  __shared__ __align__(16) float sm[kHB + 8 * 32];  // 32 values and 8 of padding a lane
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, m = blockIdx.y, G = K / 128;
  const int k = blockIdx.x * kHB + 8 * tid;
  float v[8] = {};
  if (k < K) q4_load8_any(x, static_cast<int64_t>(m) * K + k, xmode, v);
  if (signs != nullptr) {
    float d[8];
    load_signs8(signs + k, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= d[i];
    fwht1024(v, sm);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= kHNorm;
  }
  store8<float>(sm + 40 * (tid >> 2) + 8 * (tid & 3), v);
  __syncthreads();
  if (tid >= 32) return;
  float u[32];
#pragma unroll
  for (int j = 0; j < 32; j += 8) load8<float>(sm + 40 * tid + j, u + j);
  const bool live = blockIdx.x * kHB + 32 * tid < K;  // K % 128 == 0: whole groups of four lanes
  const int g = live ? blockIdx.x * 8 + (tid >> 2) : 0;
  const bool x8 = xmode == Q4X_INT8 || xmode == Q4X_E4M3;
  const float xs = x8 ? x_scales[group == 128 ? static_cast<int64_t>(m) * G + g : m] : 1.f;
  q4_store_planes(u, xmode == Q4X_INT8, xs, P, M, m, C, image + static_cast<int64_t>(g) * 8 * C,
                  factors + static_cast<int64_t>(g) * C,
                  reinterpret_cast<int*>(factors + static_cast<int64_t>(G + g) * C), live);
}

// c += a b, a: 16 x 32 unsigned, b: 32 x 8 signed bytes.
__device__ __forceinline__ void mma_u8s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// NT: column tiles of 8; KB: boxes of a slot.
template <int NT, int KB>
__global__ void __launch_bounds__(32 * kQ4DecWarps, 1)
    q4_decode_kernel(const __grid_constant__ CUtensorMap tm_w, const Q4DecodeParams p) {
  constexpr int kSlot = KB * kQ4DecBoxBytes, kSG = 2 * KB;  // bytes and 128-groups of a slot
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int M = p.M, C = p.C, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int T = 32 * kQ4DecWarps;
  const int r = lane >> 2, c = lane & 3;
  const int rho = (r >> 1) + 4 * (r & 1);  // the fragment's row r is row rho of its 8: no bank conflict below
  const int rank = p.S > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int cluster = static_cast<int>(blockIdx.x) / p.S, nclusters = static_cast<int>(gridDim.x) / p.S;
  const int G = p.K >> 7, G0 = rank * p.Gs, Gn = max(0, min(p.Gs, G - G0));
  uint8_t* ring = smem + warp * kQ4DecSlots * kSlot;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + q4_dec_ring_bytes(KB)) + warp * kQ4DecSlots;
  uint4* xf = reinterpret_cast<uint4*>(smem + q4_dec_ring_bytes(KB) + kQ4DecBarBytes);
  float* xsg = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(xf) + q4_dec_x_bytes(C, p.Gs));
  int* xsum = reinterpret_cast<int*>(xsg + p.Gs * 8 * NT);
  float* part = reinterpret_cast<float*>(smem + p.part_at);

  const int wt = warp % p.Wt, wk = warp / p.Wt;
  const int nbox = (Gn + kSG - 1) / kSG;  // slots' worth in the slice
  const int nb = wk < p.Wk && nbox > wk ? (nbox - wk + p.Wk - 1) / p.Wk : 0;  // this warp's, per row block
  const int mine = (p.nblocks - cluster + nclusters - 1) / nclusters;  // row blocks of this cluster
  const int total = mine * nb;
  const int R = p.Wt * p.rw;
  const uint32_t bytes = static_cast<uint32_t>(p.rw) * 128u * KB;

  // the producer's place: block and box index of the next box to fetch
  int fb = 0, fj = 0, fs = 0;
  auto fetch = [&]() {
    if (p.stall) return;
    const int row = (cluster + fb * nclusters) * R + wt * p.rw;
    mbar_arrive_expect_tx(&bars[fs], bytes);
#pragma unroll
    for (int b = 0; b < KB; ++b)
      tma_load_2d(ring + fs * kSlot + b * kQ4DecBoxBytes, &tm_w, (G0 + kSG * (wk + p.Wk * fj) + 2 * b) * 64, row, &bars[fs]);
    if (++fj == nb) {
      fj = 0;
      ++fb;
    }
    if (++fs == kQ4DecSlots) fs = 0;
  };
  if (lane == 0) {
    for (int s = 0; s < kQ4DecSlots; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
    for (int s = 0; s < kQ4DecSlots && s < total; ++s) fetch();  // weights do not wait for the previous kernel
  }
  // scales of this lane's rows (rho, rho + 8), fetched a box ahead
  uint16_t sn[kSG][2];
  auto load_scales = [&](int ib, int j) {
    const int64_t row = static_cast<int64_t>(cluster + ib * nclusters) * R + wt * p.rw + rho;
    const int g = kSG * (wk + p.Wk * j);
    const uint16_t* src = p.scales + row * G + G0 + g;
    const int left = static_cast<int>(min(p.N - row, static_cast<int64_t>(p.rw - rho)));  // rows from rho on
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int gg = 0; gg < kSG; ++gg)
        sn[gg][h] = 8 * h < left && g + gg < Gn ? __ldg(src + 8 * h * G + gg) : uint16_t(0);
  };
  if (nb > 0) load_scales(0, 0);
  pdl_launch_dependents();
  pdl_wait();
  if (p.xmode == Q4X_IMAGE) {
    const uint4* src = static_cast<const uint4*>(p.x) + static_cast<int64_t>(G0) * 8 * C;
    for (int q = tid; q < 8 * C * Gn; q += T) xf[q] = __ldcg(src + q);
    for (int q = tid; q < C * Gn; q += T) {
      const int g = q / C, n = q - g * C;
      xsg[g * 8 * NT + n] = __ldcg(p.x_scales + static_cast<int64_t>(G0) * C + q);
      xsum[g * 8 * NT + n] = __ldcg(reinterpret_cast<const int*>(p.x_scales) + static_cast<int64_t>(G + G0) * C + q);
    }
  } else {
    // four lanes make the planes of one token's group
    const bool x8 = p.xmode == Q4X_INT8 || p.xmode == Q4X_E4M3;
    const int items = M * Gn;
    for (int q0 = 8 * warp; q0 < items; q0 += T / 4) {
      const bool live = q0 + (lane >> 2) < items;
      const int q = live ? q0 + (lane >> 2) : q0;
      const int m = q / Gn, g = q - m * Gn;
      float v[32];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        q4_load8_any(p.x, static_cast<int64_t>(m) * p.K + static_cast<int64_t>(G0 + g) * 128 + 32 * c + 8 * j, p.xmode,
                     v + 8 * j);
      const float xs = x8 ? p.x_scales[p.x_group == 128 ? static_cast<int64_t>(m) * G + G0 + g : m] : 1.f;
      q4_store_planes(v, p.xmode == Q4X_INT8, xs, p.P, M, m, C, xf + g * 8 * C, xsg + g * 8 * NT, xsum + g * 8 * NT,
                      live);
    }
  }
  __syncthreads();

  bool ok = true;
  int slot = 0;
  uint32_t phase = 0;
  int done = 0;
  for (int ib = 0; ib < mine; ++ib) {
    const int64_t row0 = static_cast<int64_t>(cluster + ib * nclusters) * R;
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
    if (nb > 0 && ib > 0) load_scales(ib, 0);
    for (int j = 0; j < nb && ok; ++j) {
      float sc[kSG][2];
#pragma unroll
      for (int h = 0; h < 2 * kSG; ++h) sc[h >> 1][h & 1] = __half2float(__ushort_as_half(sn[h >> 1][h & 1]));
      if (j + 1 < nb) load_scales(ib, j + 1);
      if (!__all_sync(0xffffffffu, mbar_wait(&bars[slot], phase, FAULT_WAIT_FULL))) {
        ok = false;
        break;
      }
      const uint8_t* boxes = ring + slot * kSlot + rho * 128;
      const int g0 = kSG * (wk + p.Wk * j);
#pragma unroll
      for (int gg = 0; gg < kSG; ++gg) {
        const uint8_t* box = boxes + (gg >> 1) * kQ4DecBoxBytes;
        const int g = min(g0 + gg, Gn - 1);  // past an odd end: any x', the scales are zero
        const uint4* xg = xf + g * 8 * C + lane;
        uint4 b[NT][2];
        int2 d0[NT];
        float2 f[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const bool col = 8 * t + r < C;
          b[t][0] = col ? xg[32 * t] : make_uint4(0, 0, 0, 0);
          b[t][1] = col ? xg[4 * C + 32 * t] : make_uint4(0, 0, 0, 0);
          d0[t] = *reinterpret_cast<const int2*>(xsum + g * 8 * NT + 8 * t + 2 * c);
          f[t] = *reinterpret_cast<const float2*>(xsg + g * 8 * NT + 8 * t + 2 * c);
        }
        const int at = 16 * ((4 * (gg & 1) + c) ^ rho);  // the 128-byte swizzle of a box row
        const uint4 lo = *reinterpret_cast<const uint4*>(box + at);
        const uint4 hi = *reinterpret_cast<const uint4*>(box + 1024 + at);
        int d[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          d[t][0] = d[t][2] = d0[t].x;
          d[t][1] = d[t][3] = d0[t].y;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t wl = (&lo.x)[i], wh = (&hi.x)[i];
          const uint32_t a0 = wl & 0x0F0F0F0Fu, a1 = wh & 0x0F0F0F0Fu;
          const uint32_t a2 = (wl >> 4) & 0x0F0F0F0Fu, a3 = (wh >> 4) & 0x0F0F0F0Fu;
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma_u8s8(d[t], a0, a1, a2, a3, (&b[t][i >> 1].x)[2 * (i & 1)], (&b[t][i >> 1].x)[2 * (i & 1) + 1]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float s0 = sc[gg][0], s1 = sc[gg][1];
          acc[t][0] += s0 * f[t].x * (__int_as_float(d[t][0]) - kQ4Magic);
          acc[t][1] += s0 * f[t].y * (__int_as_float(d[t][1]) - kQ4Magic);
          acc[t][2] += s1 * f[t].x * (__int_as_float(d[t][2]) - kQ4Magic);
          acc[t][3] += s1 * f[t].y * (__int_as_float(d[t][3]) - kQ4Magic);
        }
      }
      __syncwarp();  // every lane has read the box
      ++done;
      if (lane == 0 && done + kQ4DecSlots <= total) fetch();
      if (++slot == kQ4DecSlots) {
        slot = 0;
        phase ^= 1u;
      }
    }
    // partial sums [token][row][wk, plane], joined over warps, planes and the cluster
    const int rows = kQ4DecBoxRows * p.Wt, terms = p.Wk * p.P;
    if (mine == 1) __syncthreads();  // they may lie over x'
    if (wk < p.Wk) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int n = 8 * t + 2 * c + e;
          if (n >= C) continue;
          const int pl = (n >= M) + (n >= 2 * M), m = n - pl * M;
          float* dst = part + (m * rows + kQ4DecBoxRows * wt + rho) * terms + wk * p.P + pl;
          dst[0] = acc[t][e];
          dst[8 * terms] = acc[t][e + 2];
        }
    }
    __syncthreads();
    auto joined = [&](int at) {
      const float* s = part + at * terms;
      float v = s[0];
#pragma unroll 4
      for (int q = 1; q < terms; ++q) v += s[q];
      return v;
    };
    if (p.S > 1) {
      // the first term's place takes the CTA's sum (only its own thread reads it before)
      for (int o = tid; o < M * rows; o += T) part[o * terms] = joined(o);
      cluster_sync_all();
    }
    for (int o = tid * p.S + rank; o < M * R; o += T * p.S) {
      const int m = o / R, row = o - m * R;
      const int w = row / p.rw, at = m * rows + kQ4DecBoxRows * w + row - w * p.rw;
      if (row0 + row >= p.N) continue;
      float v;
      if (p.S > 1) {
        v = 0.f;
        for (int q = 0; q < p.S; ++q) v += ld_cluster_f32(cluster_map(smem_u32(part + at * terms), q));
      } else {
        v = joined(at);
      }
      store_from_f32(p.y, m * p.N + row0 + row, p.yt, v);
    }
    if (p.S > 1)
      cluster_sync_all();  // no CTA overwrites (or leaves) what its peers still read
    else
      __syncthreads();
  }
  // after a wait that gave up: the copies still in flight land before the CTA leaves
  if (!ok && lane == 0 && !p.stall) {
    for (int s = 0; s < kQ4DecSlots && s < total - done; ++s) {
      const int at = slot + s;
      mbar_wait(&bars[at % kQ4DecSlots], phase ^ (at >= kQ4DecSlots ? 1u : 0u), FAULT_WAIT_FULL);
    }
  }
}

}  // namespace tb
