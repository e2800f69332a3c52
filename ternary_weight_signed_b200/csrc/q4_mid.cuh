// Linear layer with 4-bit g128 weights for 17 to 128 tokens: tcgen05 on one CTA.
//
// The same mathematics as the pair GEMM (gemm_pair.cuh): the weights are the
// MMA's M side, unpacked to fp16(s q) straight into tensor memory as operand A,
// x' (fp16 with a factor per token) comes by TMA into shared memory as operand B,
// the sums of all of K stay in tensor memory.  What differs is what few tokens
// want:
//   * one-CTA MMAs.  Measured on B200 with A in tensor memory and a commit every 8,
//     cycles per M = 128, K = 16 instruction: 26 at N = 32, 33 at 64, 65 at 128, 128
//     at 256; a CTA pair's M = 256 takes 130 at every N up to 256.  Up to 128 tokens
//     an SM's 128 weight rows so cost half or less on their own.
//   * K split over a cluster of S CTAs when there are fewer 128-row tiles than SMs:
//     each CTA leaves its sums in shared memory as fp32, and after the cluster's
//     barrier each adds its share of the tokens over the S CTAs in rank order
//     (no atomics).
// Bound: the copies of the codes and the L2 reads of x' by every tile (BT * K * 2
// bytes a tile); the MMAs take 5.6 us of 17408 x 5120 at 64 tokens.  Measured with
// the prep: 21.9 us at 32 tokens, 23.3 at 64, 26.2 at 128 (the pair GEMM: 34.7), held by
// the round trip between the unpack warps and the MMAs.
// The codes come in boxes of 128 rows x 128 bytes, two stages at a time: a TMA copy
// of 64-byte rows runs at 2.6 TB/s over the device, one of 128-byte rows at 4 and
// more (measured alone, launches included).
// Warps: 0 copies x', 18 the codes, 1 issues the MMAs (and owns tensor memory),
// 2-17 unpack, four sets of four (set j takes the stages j, j + 4, ..), and read D.
// Hand-offs: wfull / wfree (a box of codes landed / is in the registers of its
// eight warps), full (x' of a stage landed), ready (a stage's A is written), done
// (its MMAs are done: x' and A slot free), accum (D complete).  Every wait is
// bounded; a role that gives up stops waiting and the CTA still leaves in order.
#pragma once
#include "gemm_pair.cuh"
#include "norm.cuh"
#include "q4_linear.cuh"
#include "tb_device.cuh"

namespace tb {

constexpr int kQmThreads = kGpThreads + 32;
constexpr int kQmWBytes = 128 * 128;  // a box of codes: 128 rows x 256 codes
constexpr int kQmWSlots = 4;
constexpr int kQmDCols = 128;         // D columns (tokens) at most; the A ring follows
// x' stages: a multiple of the unpack sets, so that a wait names its phase by parity.
__host__ __device__ constexpr int qm_stages(int bt) { return bt <= 64 ? 8 : 4; }
// Slots of the A ring: where the stages allow, more than the sets, so that a set
// that has written a stage goes on to its next one before its MMAs are done.
__host__ __device__ constexpr int qm_a_slots(int bt) { return bt <= 64 ? 6 : 4; }
__host__ __device__ constexpr int qm_smem_bytes(int bt) {
  return kQmWSlots * kQmWBytes + qm_stages(bt) * bt * 256 + 1024 + 256;
}
static_assert(kQmDCols + 6 * kGpACols <= kGpTmemCols, "TMEM budget");
// kind::f16, D fp32, A and B fp16 K-major, M = 128, N = bt
__host__ __device__ constexpr uint32_t qm_idesc(int bt) {
  return (1u << 4) | (static_cast<uint32_t>(bt >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void umma_ts_f16(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

struct Q4MidParams {
  int M, N, K, S, yt;
  void* y;
  const uint16_t* scales;
  const float* factor;  // of each token
};

// BT: tokens (a multiple of 32).  grid: S * tiles CTAs, the S of a tile one cluster.
template <int BT>
__global__ void __launch_bounds__(kQmThreads, 1)
    q4_mid_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                  const Q4MidParams p) {
  constexpr int kX = BT * 256, kAtom = kX / 2, ST = qm_stages(BT), SA = qm_a_slots(BT);
  constexpr int kCols = BT / kGpSets;
  static_assert(kAtom % 1024 == 0 && ST % kGpSets == 0 && SA <= ST && kQmWSlots % 2 == 0, "rings");
  static_assert(ST * kX + kQmWSlots * kQmWBytes >= BT * 128 * 4, "the sums of a split tile lie over the rings");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* wring = smem + ST * kX;
  uint64_t* full = reinterpret_cast<uint64_t*>(wring + kQmWSlots * kQmWBytes);
  uint64_t* ready = full + ST;
  uint64_t* done = ready + ST;
  uint64_t* wfull = done + ST;
  uint64_t* wfree = wfull + kQmWSlots;
  uint64_t* accum = wfree + kQmWSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accum + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.S > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int n0 = static_cast<int>(blockIdx.x) / p.S * 128;
  // stages in pairs; an odd last 128-group is followed by one past the end (x' and
  // the scales are zero there)
  const int G = p.K >> 7, pairs = (G + 1) >> 1;
  const int p0 = static_cast<int>(static_cast<int64_t>(pairs) * rank / p.S);
  const int np = static_cast<int>(static_cast<int64_t>(pairs) * (rank + 1) / p.S) - p0;  // at least one
  const int kb0 = 2 * p0, nk = 2 * np;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&ready[s], 4);
      mbar_init(&done[s], 1);
    }
    for (int s = 0; s < kQmWSlots; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wfree[s], 2 * 4);
    }
    mbar_init(accum, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kGpTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_d = *tmem_slot;
  const uint32_t tmem_a = tmem_d + kQmDCols;

  if (warp == 18) {
    if (lane == 0 && !test_stall_copies()) {  // (failure-detection test: no copies)
      int j = 0;
      for (; j < np; ++j) {
        const int s = j % kQmWSlots;
        if (j >= kQmWSlots && !mbar_wait(&wfree[s], ((j / kQmWSlots) & 1) ^ 1, FAULT_WAIT_EMPTY)) break;
        mbar_arrive_expect_tx(&wfull[s], kQmWBytes);
        tma_load_2d(wring + s * kQmWBytes, &tm_w, (p0 + j) * 128, n0, &wfull[s]);  // does not wait for the prep kernel
      }
      // the last copies issued land before the CTA may leave
      for (int h = j > kQmWSlots ? j - kQmWSlots : 0; h < j; ++h)
        if (!mbar_wait(&wfull[h % kQmWSlots], (h / kQmWSlots) & 1, FAULT_WAIT_FULL)) break;
    }
  } else if (warp == 0) {
    if (lane == 0) {
      pdl_wait();
      int g = 0;
      for (; g < nk; ++g) {
        const int s = g % ST;
        if (g >= ST && !mbar_wait(&done[s], ((g / ST) & 1) ^ 1, FAULT_WAIT_EMPTY)) break;
        uint8_t* st = smem + s * kX;
        mbar_arrive_expect_tx(&full[s], kX);
        tma_load_2d(st, &tm_x, (kb0 + g) * 128, 0, &full[s]);
        tma_load_2d(st + kAtom, &tm_x, (kb0 + g) * 128 + 64, 0, &full[s]);
      }
      for (int h = g > ST ? g - ST : 0; h < g; ++h)
        if (!mbar_wait(&full[h % ST], (h / ST) & 1, FAULT_WAIT_FULL)) break;
    }
  } else if (warp == 1) {
    // The whole warp walks the stages with uniform operands and one elected lane
    // issues: 26 cycles an MMA at N = 32 and 33 at 64, against 56-69 from a branch on
    // the lane, where every operand is moved to the uniform registers first.
    const uint32_t d = __shfl_sync(0xffffffffu, tmem_d, 0), a0 = d + kQmDCols;
    const uint32_t x0 = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
    for (int g = 0; g < nk; ++g) {
      const int s = g % ST;
      const bool go = mbar_wait(&full[s], (g / ST) & 1, FAULT_WAIT_ACT) && mbar_wait(&ready[s], (g / ST) & 1, FAULT_WAIT_FULL);
      if (!__all_sync(0xffffffffu, go)) break;
      tc_fence_after();
      const uint32_t a = a0 + static_cast<uint32_t>((g % SA) * kGpACols);
      const uint64_t b = umma_desc_sw128(x0 + static_cast<uint32_t>(s * kX));
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // the descriptor's address is in 16-byte units
          umma_ts_f16(d, a + 8 * kk, b + ((kk >> 2) * kAtom + 32 * (kk & 3)) / 16, qm_idesc(BT), (g | kk) != 0 ? 1u : 0u);
        umma_commit(&done[s]);
      }
      __syncwarp();
    }
    if (elect_one()) umma_commit(accum);  // also after a wait that gave up: whoever waits stops waiting
    __syncwarp();
  } else {
    const int q = warp & 3, set = (warp - 2) >> 2, r = 32 * q + lane, n = n0 + r;
    const uint32_t lane_addr = static_cast<uint32_t>(32 * q) << 16;
    const uint16_t* srow = p.scales + static_cast<int64_t>(n) * G + kb0;
    const int ng = min(nk, G - kb0);  // stages with a scale
    uint16_t s_next = n < p.N && set < ng ? srow[set] : uint16_t(0);
    bool ok = true;
    for (int g = set; g < nk; g += kGpSets) {
      const int s = g % ST;
      const __half sc = __ushort_as_half(s_next);
      s_next = n < p.N && g + kGpSets < ng ? srow[g + kGpSets] : uint16_t(0);
      const int j = g >> 1, ws = j % kQmWSlots;
      if (!__all_sync(0xffffffffu, mbar_wait(&wfull[ws], (j / kQmWSlots) & 1, FAULT_WAIT_FULL))) {
        ok = false;
        break;
      }
      // rows of 128 bytes, 128B-swizzled: 16-byte chunk u at u ^ r % 8
      const uint8_t* wrow = wring + ws * kQmWBytes + r * 128;
      uint4 wv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) wv[u] = *reinterpret_cast<const uint4*>(wrow + 16 * ((4 * (g & 1) + u) ^ (r & 7)));
      __syncwarp();
      if (lane == 0) mbar_arrive(&wfree[ws]);  // the codes are in registers
      // The MMAs of stage g - SA are done with this A slot.  Parity names the phase: at
      // its stage g - 4 this warp saw those of g - 4 - SA done, and stage g - SA + ST
      // cannot be done before this warp's stage g.
      if (g >= SA &&
          !__all_sync(0xffffffffu, mbar_wait(&done[(g - SA) % ST], ((g - SA) / ST) & 1, FAULT_WAIT_MMA))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const __half2 s2 = __halves2half2(sc, sc);
      const uint32_t ta = tmem_a + lane_addr + static_cast<uint32_t>((g % SA) * kGpACols);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t o[32];
#pragma unroll
        for (int wd = 0; wd < 8; ++wd) gp_unpack_q4((&wv[0].x)[8 * half + wd], s2, o + 4 * wd);
        tmem_st32(ta + static_cast<uint32_t>(32 * half), o);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ready[s]);
    }
    // D: this warp's 32 rows and kCols of the tokens
    float f[kCols];
    if (p.S == 1) {
      pdl_wait();  // the factors come from the prep kernel; they are padded to 256 tokens
#pragma unroll
      for (int j = 0; j < kCols; j += 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(p.factor + set * kCols + j));
        f[j] = v.x, f[j + 1] = v.y, f[j + 2] = v.z, f[j + 3] = v.w;
      }
    }
    const bool got = __all_sync(0xffffffffu, mbar_wait(accum, 0, FAULT_WAIT_EPILOGUE, 4));
    if (ok && got) {
      tc_fence_after();
      uint32_t v[kCols];
      tmem_ld_cols<kCols>(tmem_d + lane_addr + static_cast<uint32_t>(set * kCols), v);
      tmem_ld_wait();
      tc_fence_before();
      if (p.S > 1) {
        float* sums = reinterpret_cast<float*>(smem) + set * kCols * 128 + r;  // [token][row]
#pragma unroll
        for (int j = 0; j < kCols; ++j) sums[j * 128] = __uint_as_float(v[j]);
      } else if (n < p.N) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          const int m = set * kCols + j;
          if (m < p.M) store_from_f32(p.y, static_cast<int64_t>(m) * p.N + n, p.yt, __uint_as_float(v[j]) * f[j]);
        }
      }
    }
  }
  if (p.S > 1) {
    __syncwarp();
    cluster_sync_all();
    // tokens rank, rank + S, ..; the rows along the threads
    if (warp >= 2 && warp < 18) {
      const int t = threadIdx.x - 64, row = t & 127;
      pdl_wait();
      if (n0 + row < p.N) {
        constexpr int kBatch = 4;  // tokens whose loads are in flight together
        for (int m0 = rank + p.S * (t >> 7); m0 < p.M; m0 += 4 * p.S * kBatch) {
          float v[kBatch] = {}, f[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) f[i] = __ldcg(p.factor + min(m0 + 4 * p.S * i, p.M - 1));
          for (int c = 0; c < p.S; ++c) {
            float u[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
              u[i] = ld_cluster_f32(cluster_map(
                  smem_u32(smem) + static_cast<uint32_t>(min(m0 + 4 * p.S * i, BT - 1) * 128 + row) * 4u, c));
#pragma unroll
            for (int i = 0; i < kBatch; ++i) v[i] += u[i];
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int m = m0 + 4 * p.S * i;
            if (m < p.M) store_from_f32(p.y, static_cast<int64_t>(m) * p.N + n0 + row, p.yt, v[i] * f[i]);
          }
        }
      }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();  // no CTA leaves while its peers read its sums
  } else {
    __syncwarp();
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_d, kGpTmemCols);
  }
}

}  // namespace tb
