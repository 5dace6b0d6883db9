// Linear layer on 8-bit rows: out[m, n] = bf16(sa[m] sw[n] sum_k A[m, k] W[n, k] + b[n]) with A and W
// in e4m3, one fp32 scale per row of each, products accumulated in fp32.
//
// Four kernels:
//   - lin8_rows_kernel for a few rows of A, bound by the weights' bytes (7 x 6144 x 4096: 6.0 us, 4.2 TB/s);
//   - lin8_tile_kernel, 128 x 128 tiles, one CTA per SM;
//   - lin8_split_kernel, 128 x 128 tiles with K split over a cluster, where tiles are few (33 x 4096 x
//     4096: 7.2 us, 12.9 unsplit);
//   - lin8_pair_kernel, 256 x 256 tiles on two SMs (8191 x 4096 x 4096: 95 us, 2.9 PFLOP/s).
// Tile kernel: persistent tcgen05 kind::f8f6f4, one CTA per SM of 10 warps in the roles of the bf16
// GEMM (TMA producer, MMA issuer, 8 epilogue warps; the accumulator double-buffered in TMEM).  A
// stage is 128 bytes deep, which is 128 values of K here (four K = 32 MMAs) where it is 64 in bf16,
// so a byte of shared memory feeds twice the work.  K past its end is zero-filled by the loads,
// rows past M and columns past N are cut by the stores.
#pragma once

#include "cluster.cuh"
#include "op_status.cuh"

namespace vit {

constexpr int LIN8_BM = 128;
constexpr int LIN8_BK = 128;  // bytes of K per stage
constexpr int LIN8_EPI_WARPS = 8;
constexpr int LIN8_THREADS = 64 + 32 * LIN8_EPI_WARPS;
constexpr int DEV_TIMEOUT_LIN8 = 0x300;

struct Lin8Params {
  int M, N, K;
  const float* sa;    // [M]
  const float* sw;    // [N]
  const float* bias;  // [N] or NULL
  unsigned long long wait_ns;
};

struct Lin8Cfg {
  static constexpr int BN = 128;
  static constexpr int STAGES = 6;
  static constexpr int A_BYTES = LIN8_BM * LIN8_BK;
  static constexpr int B_BYTES = BN * LIN8_BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int EPI_WARP_BYTES = 4096;  // 32 rows x 64 bf16 (128-byte rows, 128B swizzle)
  static constexpr int OFF_EPI = STAGES * STAGE_BYTES;
  static constexpr int OFF_BAR = OFF_EPI + LIN8_EPI_WARPS * EPI_WARP_BYTES;
  static constexpr int BAR_BYTES = 256;
  static constexpr int SMEM_BYTES = OFF_BAR + BAR_BYTES + 1024;  // + alignment slack
  static constexpr uint32_t TMEM_COLS = 2 * BN;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(8 * (2 * STAGES + 5) + 8 <= BAR_BYTES, "barrier area");
};

// D[tmem] (+)= A[smem] * B[smem]^T, 8-bit inputs, fp32 accumulator (kind::f8f6f4, K = 32).
__device__ __forceinline__ void tc_mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, "
      "p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::f8f6f4 with e4m3 A and B (format 0), fp32 D, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4)                                 // D format: f32
         | (static_cast<uint32_t>(N >> 3) << 17)   // N / 8
         | (static_cast<uint32_t>(M >> 4) << 24);  // M / 16
}

// One warp's part of a tile (rows row0 .. row0 + 31, columns n0 .. n0 + COLS - 1): scales, bias,
// bf16, 64 columns per TMA store through the warp's staging buffer.  N is a multiple of 8, so
// a group of 8 columns is either inside or outside.
template <int COLS>
__device__ __forceinline__ void lin8_epilogue(const Lin8Params& p, const CUtensorMap* tmO, uint32_t taddr, int row0,
                                              int n0, float sa, uint8_t* obuf) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int g = 0; g < COLS / 64; ++g) {
    if (n0 + g * 64 >= p.N) break;
    if (lane == 0) tma_store_wait_read0();  // the previous store has left the staging buffer
    __syncwarp();
#pragma unroll
    for (int cc = 0; cc < 2; ++cc) {
      float v[32];
      tmem_ld32(taddr + g * 64 + cc * 32, v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int n = n0 + g * 64 + cc * 32 + k * 8;
        float4 s0 = make_float4(0.f, 0.f, 0.f, 0.f), s1 = s0, b0 = s0, b1 = s0;
        if (n < p.N) {
          s0 = __ldg(reinterpret_cast<const float4*>(p.sw + n));
          s1 = __ldg(reinterpret_cast<const float4*>(p.sw + n + 4));
          if (p.bias != nullptr) {
            b0 = __ldg(reinterpret_cast<const float4*>(p.bias + n));
            b1 = __ldg(reinterpret_cast<const float4*>(p.bias + n + 4));
          }
        }
        const float* a = v + 8 * k;
        uint4 w;
        w.x = pack_bf16x2(fmaf(a[0] * sa, s0.x, b0.x), fmaf(a[1] * sa, s0.y, b0.y));
        w.y = pack_bf16x2(fmaf(a[2] * sa, s0.z, b0.z), fmaf(a[3] * sa, s0.w, b0.w));
        w.z = pack_bf16x2(fmaf(a[4] * sa, s1.x, b1.x), fmaf(a[5] * sa, s1.y, b1.y));
        w.w = pack_bf16x2(fmaf(a[6] * sa, s1.z, b1.z), fmaf(a[7] * sa, s1.w, b1.w));
        const int chunk = (cc * 4 + k) ^ (lane & 7);
        *reinterpret_cast<uint4*>(obuf + lane * 128 + chunk * 16) = w;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(tmO, obuf, n0 + g * 64, row0);
      tma_store_commit();
    }
  }
}

__global__ void __launch_bounds__(LIN8_THREADS, 1)
    lin8_tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmO, Lin8Params p, int* status) {
  using Cfg = Lin8Cfg;
  constexpr int BN = Cfg::BN, STAGES = Cfg::STAGES;
  constexpr int COLS = BN / 2;  // columns an epilogue warp takes
  int* gstatus = op_status(status);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * Cfg::A_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 32 * LIN8_EPI_WARPS);
    }
    mbar_init(mma_done, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmO);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, Cfg::TMEM_COLS);
    tmem_relinquish();
  }
  // everything above touches only this CTA's shared and tensor memory; global memory from here on
  pdl_wait();
  if (threadIdx.x == 0) *abort_flag = op_stopped(status) ? 1 : 0;
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const bool skip = *abort_flag != 0;

  const int num_m = (p.M + LIN8_BM - 1) / LIN8_BM;
  const int num_n = (p.N + BN - 1) / BN;
  const int num_tiles = num_m * num_n;
  const int KB = (p.K + LIN8_BK - 1) / LIN8_BK;

  if (!skip && warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- TMA producer
    int stage = 0;
    uint32_t phase = 0;
    int issued_parity[STAGES];
#pragma unroll
    for (int s = 0; s < STAGES; ++s) issued_parity[s] = -1;
    for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x) {
      const int mb = tile / num_n;
      const int nb = tile - mb * num_n;
      bool ok = true;
      for (int kb = 0; kb < KB; ++kb) {
        if (!mbar_wait<32>(&empty[stage], phase ^ 1u, abort_flag, gstatus, DEV_TIMEOUT_LIN8 + 1, p.wait_ns)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[stage], Cfg::STAGE_BYTES);
        tma_load_2d(sA + stage * Cfg::A_BYTES, &tmA, kb * LIN8_BK, mb * LIN8_BM, &full[stage]);
        tma_load_2d(sB + stage * Cfg::B_BYTES, &tmB, kb * LIN8_BK, nb * BN, &full[stage]);
        issued_parity[stage] = static_cast<int>(phase);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
    }
    if (*abort_flag) {
      // let every issued tile land before the CTA can exit and release its shared memory
      for (int s = 0; s < STAGES; ++s)
        if (issued_parity[s] >= 0) mbar_wait_drain(&full[s], static_cast<uint32_t>(issued_parity[s]));
    }
  } else if (!skip && warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3(LIN8_BM, BN);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < num_tiles && ok; tile += gridDim.x) {
        if (!mbar_wait<32>(&tempty[acc], acc_phase ^ 1u, abort_flag, gstatus, DEV_TIMEOUT_LIN8 + 2, p.wait_ns)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait<32>(&full[stage], phase, abort_flag, gstatus, DEV_TIMEOUT_LIN8 + 3, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + stage * Cfg::A_BYTES);
          const uint32_t b0 = smem_u32(sB + stage * Cfg::B_BYTES);
#pragma unroll
          for (int k = 0; k < LIN8_BK / 32; ++k)
            tc_mma_f8_ss(d_tmem, sdesc_sw128(a0 + k * 32, 16, 1024), sdesc_sw128(b0 + k * 32, 16, 1024), idesc,
                         (kb | k) != 0 ? 1u : 0u);
          tc_commit(&empty[stage]);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit(&tfull[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      tc_commit(mma_done);
    }
    __syncwarp();
  } else if (!skip && warp >= 2) {
    // ---------------------------------------------------------------- epilogue
    const int e = warp - 2;
    const int q = warp & 3;
    const int half = e >> 2;
    uint8_t* obuf = smem + Cfg::OFF_EPI + e * Cfg::EPI_WARP_BYTES;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x) {
      const int mb = tile / num_n;
      const int nb = tile - mb * num_n;
      const int row0 = mb * LIN8_BM + q * 32;
      const float sa = row0 + lane < p.M ? __ldg(p.sa + row0 + lane) : 0.f;
      if (!mbar_wait_warp<32>(&tfull[acc], acc_phase, abort_flag, gstatus, DEV_TIMEOUT_LIN8 + 4, p.wait_ns)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>(acc * BN + half * COLS);
      __syncwarp();
      if (row0 < p.M) lin8_epilogue<COLS>(p, &tmO, taddr, row0, nb * BN + half * COLS, sa, obuf);
      tc_fence_before();
      mbar_arrive(&tempty[acc]);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (lane == 0) tma_store_wait0();  // every TMA store of this warp has completed
    __syncwarp();
  }

  // ---------------------------------------------------------------- teardown
  __syncthreads();
  if (warp == 1) {
    if (!skip && lane == 0) mbar_wait_drain(mma_done, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
  }
}

// ------------------------------------------------------------------------------------------------
// Paired variant: a 2-CTA cluster computes a 256 x 256 tile with M = 256 MMAs (cta_group::2), as the
// bf16 GEMM does: each CTA loads its 128 rows of A and its 128 of the 256 rows of W and keeps its 128
// accumulator rows.  Both producers count their bytes on the leader's full barrier; the leader
// issues the MMAs and commits to both CTAs' barriers; epilogue warps release the accumulator on the
// leader's.  No load uses cluster multicast.
struct Lin8PairCfg {
  static constexpr int BN = 256;
  static constexpr int STAGES = 6;
  static constexpr int A_BYTES = LIN8_BM * LIN8_BK;
  static constexpr int B_BYTES = (BN / 2) * LIN8_BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int OFF_EPI = STAGES * STAGE_BYTES;
  static constexpr int OFF_BAR = OFF_EPI + LIN8_EPI_WARPS * 4096;
  static constexpr int BAR_BYTES = 256;
  static constexpr int SMEM_BYTES = OFF_BAR + BAR_BYTES + 1024;
  static constexpr uint32_t TMEM_COLS = 512;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(8 * (2 * STAGES + 5) + 8 <= BAR_BYTES, "barrier area");
};

__device__ __forceinline__ void tc_mma_f8_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                  uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, "
      "p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ int peer_int(const void* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return v;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(LIN8_THREADS, 1)
    lin8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmO, Lin8Params p, int* status) {
  using Cfg = Lin8PairCfg;
  constexpr int BN = Cfg::BN, STAGES = Cfg::STAGES;
  int* gstatus = op_status(status);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * Cfg::A_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * LIN8_EPI_WARPS);  // one arrival per epilogue warp of each CTA
    }
    mbar_init(mma_done, 1);
    fence_mbar_init_cluster();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmO);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, Cfg::TMEM_COLS);
    tmem_relinquish_pair();
  }
  // everything above touches only this cluster's shared and tensor memory; global memory from here on
  pdl_wait();
  if (threadIdx.x == 0) *abort_flag = op_stopped(status) ? 1 : 0;
  pdl_launch_dependents();
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const bool skip = peer_int(const_cast<int*>(abort_flag), 0) != 0;  // the leader decides for both

  const int num_n = (p.N + BN - 1) / BN;
  const int num_tiles = ((p.M + 2 * LIN8_BM - 1) / (2 * LIN8_BM)) * num_n;
  const int KB = (p.K + LIN8_BK - 1) / LIN8_BK;
  const int cid = static_cast<int>(blockIdx.x >> 1);
  const int ncl = static_cast<int>(gridDim.x >> 1);

  if (!skip && warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- TMA producer (both CTAs)
    int stage = 0;
    uint32_t phase = 0;
    int issued_parity[STAGES];
#pragma unroll
    for (int s = 0; s < STAGES; ++s) issued_parity[s] = -1;
    bool ok = true, any = false;
    for (int tile = cid; tile < num_tiles && ok; tile += ncl) {
      const int mb = tile / num_n;
      const int nb = tile - mb * num_n;
      for (int kb = 0; kb < KB; ++kb) {
        if (!mbar_wait<32>(&empty[stage], phase ^ 1u, abort_flag, gstatus, DEV_TIMEOUT_LIN8 + 5, p.wait_ns)) {
          ok = false;
          break;
        }
        if (leader) mbar_arrive_expect_tx(&full[stage], 2 * Cfg::STAGE_BYTES);
        const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
        tma_load_2d_pair(sA + stage * Cfg::A_BYTES, &tmA, kb * LIN8_BK, (mb * 2 + rank) * LIN8_BM, bar);
        tma_load_2d_pair(sB + stage * Cfg::B_BYTES, &tmB, kb * LIN8_BK, nb * BN + rank * (BN / 2), bar);
        issued_parity[stage] = static_cast<int>(phase);
        any = true;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (*abort_flag) {
      // let every issued copy land before the CTA can exit: the leader sees both CTAs' bytes; the other
      // one cannot see its own and pauses instead (200 us)
      if (leader) {
        for (int s = 0; s < STAGES; ++s)
          if (issued_parity[s] >= 0) mbar_wait_drain(&full[s], static_cast<uint32_t>(issued_parity[s]));
      } else if (any) {
        for (const unsigned long long t0 = global_ns(); global_ns() - t0 < 200000ull;) {
        }
      }
    }
  } else if (!skip && warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (leader)
    if (leader && lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3(2 * LIN8_BM, BN);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int tile = cid; tile < num_tiles && ok; tile += ncl) {
        if (!mbar_wait<32>(&tempty[acc], acc_phase ^ 1u, abort_flag, gstatus, DEV_TIMEOUT_LIN8 + 6, p.wait_ns)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait<32>(&full[stage], phase, abort_flag, gstatus, DEV_TIMEOUT_LIN8 + 7, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + stage * Cfg::A_BYTES);
          const uint32_t b0 = smem_u32(sB + stage * Cfg::B_BYTES);
#pragma unroll
          for (int k = 0; k < LIN8_BK / 32; ++k)
            tc_mma_f8_ss_pair(d_tmem, sdesc_sw128(a0 + k * 32, 16, 1024), sdesc_sw128(b0 + k * 32, 16, 1024), idesc,
                              (kb | k) != 0 ? 1u : 0u);
          tc_commit_pair_mc(&empty[stage], 0x3);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit_pair_mc(&tfull[acc], 0x3);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      tc_commit_pair_mc(mma_done, 0x3);
    }
    __syncwarp();
  } else if (!skip && warp >= 2) {
    // ---------------------------------------------------------------- epilogue (both CTAs)
    const int e = warp - 2;
    const int q = warp & 3;
    const int half = e >> 2;
    uint8_t* obuf = smem + Cfg::OFF_EPI + e * 4096;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int tile = cid; tile < num_tiles; tile += ncl) {
      const int mb = tile / num_n;
      const int nb = tile - mb * num_n;
      const int row0 = (mb * 2 + rank) * LIN8_BM + q * 32;
      const float sa = row0 + lane < p.M ? __ldg(p.sa + row0 + lane) : 0.f;
      if (!mbar_wait_warp<32>(&tfull[acc], acc_phase, abort_flag, gstatus, DEV_TIMEOUT_LIN8 + 8, p.wait_ns)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>(acc * BN + half * (BN / 2));
      __syncwarp();
      if (row0 < p.M) lin8_epilogue<BN / 2>(p, &tmO, taddr, row0, nb * BN + half * (BN / 2), sa, obuf);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (lane == 0) tma_store_wait0();
    __syncwarp();
  }

  // ---------------------------------------------------------------- teardown
  __syncthreads();
  if (warp == 1 && !skip && lane == 0) mbar_wait_drain(mma_done, 0);  // the pair's MMAs are done
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();  // no CTA leaves while the other may still signal its barriers or use its memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
  }
}

// ------------------------------------------------------------------------------------------------
// K split over a cluster of SPLITS (2, 4 or 8) CTAs, for work of few tiles: each CTA takes a part of
// the steps of K of one 128 x 128 tile, puts its fp32 accumulator into its shared memory (over the ring,
// which is empty by then), and sums a slice of 128 / SPLITS columns over the cluster in the order
// of the ranks.
struct Lin8SplitCfg {
  static constexpr int STAGES = 6;
  static constexpr int STAGE_BYTES = 2 * LIN8_BM * LIN8_BK;
  static constexpr int OFF_BAR = STAGES * STAGE_BYTES;
  static constexpr int SMEM_BYTES = OFF_BAR + 256 + 1024;
  static_assert(STAGES * STAGE_BYTES >= 128 * 128 * 4, "room for the accumulator");
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

template <int SPLITS>
__global__ void __launch_bounds__(LIN8_THREADS, 1)
    lin8_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, Lin8Params p,
                      __nv_bfloat16* out, int64_t ldo, int* status) {
  using Cfg = Lin8SplitCfg;
  constexpr int STAGES = Cfg::STAGES;
  int* gstatus = op_status(status);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* mma_done = empty + STAGES;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(mma_done, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 128);
    tmem_relinquish();
  }
  pdl_wait();
  if (threadIdx.x == 0) *abort_flag = op_stopped(status) ? 1 : 0;
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const bool skip = *abort_flag != 0;
  const int num_n = (p.N + 127) / 128;
  const int tile = static_cast<int>(blockIdx.x) / SPLITS;
  const int mb = tile / num_n;
  const int nb = tile - mb * num_n;
  const int KB = (p.K + LIN8_BK - 1) / LIN8_BK;
  const int kb0 = static_cast<int>(static_cast<long long>(KB) * rank / SPLITS);
  const int kb1 = static_cast<int>(static_cast<long long>(KB) * (rank + 1) / SPLITS);
  bool ok = !skip;

  if (!skip && warp == 0 && lane == 0) {
    int stage = 0;
    uint32_t phase = 0;
    int issued_parity[STAGES];
#pragma unroll
    for (int s = 0; s < STAGES; ++s) issued_parity[s] = -1;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait<32>(&empty[stage], phase ^ 1u, abort_flag, gstatus, DEV_TIMEOUT_LIN8 + 9, p.wait_ns)) break;
      mbar_arrive_expect_tx(&full[stage], Cfg::STAGE_BYTES);
      uint8_t* st = smem + stage * Cfg::STAGE_BYTES;
      tma_load_2d(st, &tmA, kb * LIN8_BK, mb * LIN8_BM, &full[stage]);
      tma_load_2d(st + LIN8_BM * LIN8_BK, &tmB, kb * LIN8_BK, nb * 128, &full[stage]);
      issued_parity[stage] = static_cast<int>(phase);
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (*abort_flag) {
      for (int s = 0; s < STAGES; ++s)
        if (issued_parity[s] >= 0) mbar_wait_drain(&full[s], static_cast<uint32_t>(issued_parity[s]));
    }
  } else if (!skip && warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3(LIN8_BM, 128);
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait<32>(&full[stage], phase, abort_flag, gstatus, DEV_TIMEOUT_LIN8 + 10, p.wait_ns)) break;
        tc_fence_after();
        const uint32_t a0 = smem_u32(smem + stage * Cfg::STAGE_BYTES), b0 = a0 + LIN8_BM * LIN8_BK;
#pragma unroll
        for (int k = 0; k < LIN8_BK / 32; ++k)
          tc_mma_f8_ss(tmem_base, sdesc_sw128(a0 + k * 32, 16, 1024), sdesc_sw128(b0 + k * 32, 16, 1024), idesc,
                       kb > kb0 || k > 0 ? 1u : 0u);
        tc_commit(&empty[stage]);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      tc_commit(mma_done);
    }
    __syncwarp();
  } else if (!skip && warp >= 2) {
    // the accumulator into shared memory: row r at 512 r, its 16-byte chunk c at place c ^ (r % 32)
    ok = mbar_wait_warp<32>(mma_done, 0, abort_flag, gstatus, DEV_TIMEOUT_LIN8 + 11, p.wait_ns) && *abort_flag == 0;
    ok = __all_sync(0xffffffffu, ok);
    const int q = warp & 3, half = (warp - 2) >> 2;
    if (ok && mb * LIN8_BM + q * 32 < p.M) {
      tc_fence_after();
      float* row = reinterpret_cast<float*>(smem) + (q * 32 + lane) * 128;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v[32];
        __syncwarp();
        tmem_ld32(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + half * 64 + c * 32, v);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          *reinterpret_cast<float4*>(row + (((half * 16 + c * 8 + u) ^ lane) << 2)) =
              make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
      }
    }
  }
  __syncwarp();
  cluster_sync_all();  // every CTA's part is in place
  if (ok && warp >= 2) {
    constexpr int per_row = 16 / SPLITS;  // groups of 8 columns a row of this CTA's slice has
    const uint32_t s0 = smem_u32(smem);
    for (int i = threadIdx.x - 64; i < 128 * per_row; i += 32 * LIN8_EPI_WARPS) {
      const int row = i / per_row, g = rank * per_row + i % per_row;
      const int m = mb * LIN8_BM + row, n = nb * 128 + g * 8;
      if (m >= p.M || n >= p.N) continue;
      const uint32_t at0 = s0 + row * 512 + (((2 * g) ^ (row & 31)) << 4);
      const uint32_t at1 = s0 + row * 512 + (((2 * g + 1) ^ (row & 31)) << 4);
      float4 a[SPLITS], b[SPLITS];  // all on their way before the first is used: a remote load takes about 0.4 us
#pragma unroll
      for (int x = 0; x < SPLITS; ++x) {
        a[x] = ld_cluster_f4(mapa_shared(at0, x));
        b[x] = ld_cluster_f4(mapa_shared(at1, x));
      }
      float v[8] = {a[0].x, a[0].y, a[0].z, a[0].w, b[0].x, b[0].y, b[0].z, b[0].w};
#pragma unroll
      for (int x = 1; x < SPLITS; ++x) {
        v[0] += a[x].x;
        v[1] += a[x].y;
        v[2] += a[x].z;
        v[3] += a[x].w;
        v[4] += b[x].x;
        v[5] += b[x].y;
        v[6] += b[x].z;
        v[7] += b[x].w;
      }
      const float sa = __ldg(p.sa + m);
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e] = fmaf(v[e] * sa, __ldg(p.sw + n + e), p.bias != nullptr ? __ldg(p.bias + n + e) : 0.f);
      *reinterpret_cast<uint4*>(out + m * ldo + n) =
          make_uint4(pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]), pack_bf16x2(w[4], w[5]), pack_bf16x2(w[6], w[7]));
    }
  }
  // ---------------------------------------------------------------- teardown
  if (warp == 1 && !skip && lane == 0) mbar_wait_drain(mma_done, 0);
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();  // no CTA leaves while another may still read its part
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 128);
  }
}

// ------------------------------------------------------------------------------------------------
// Few rows of A (new tokens): the weights' bytes bound it, so they are read once, by all SMs, straight
// from global memory into mma.sync fragments.  A CTA takes 16 rows of W (the M side of m16n8k32) and
// NB groups of 8 rows of A (the N side); its warps split K and are joined through shared memory in a
// fixed order.  The order of K inside a 64-byte chunk is free as long as both sides share it, so a
// lane's 16 bytes of a row (chunk byte 16 t) serve as they are as the fragments of two MMAs.

__device__ __forceinline__ void mma16832_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld_stream(const void* p) {  // read once: no place in L1
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ uint4 ld_keep(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

struct Lin8RowsParams {
  Lin8Params p;
  const uint8_t* A;
  const uint8_t* W;
  __nv_bfloat16* out;
  int64_t lda, ldw, ldo;
};

template <int NB, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 16 / WARPS) lin8_rows_kernel(Lin8RowsParams r, int* status) {
  constexpr int U = NB == 1 ? 8 : (NB == 2 ? 6 : 4);  // chunks in flight
  __shared__ float part[WARPS][16][8 * NB + 1];
  const Lin8Params& p = r.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16;
  // the weights on their way into L2 while the kernel ahead finishes (a prefetch takes no value: whoever writes
  // them is still waited for)
  if (threadIdx.x < 16 && n0 + static_cast<int>(threadIdx.x) < p.N)
    prefetch_l2_bulk(r.W + static_cast<int64_t>(n0 + threadIdx.x) * r.ldw, static_cast<uint32_t>(p.K));
  pdl_wait();
  pdl_launch_dependents();
  if (op_stopped(status)) return;
  const int chunks = (p.K + 63) / 64;
  const int c1 = static_cast<int>(static_cast<long long>(chunks) * (warp + 1) / WARPS);
  float acc[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b][0] = acc[b][1] = acc[b][2] = acc[b][3] = 0.f;
  // rows past the end read the last one instead; their results are not written
  const uint8_t* w0 = r.W + static_cast<int64_t>(min(n0 + g, p.N - 1)) * r.ldw + t * 16;
  const uint8_t* w1 = r.W + static_cast<int64_t>(min(n0 + g + 8, p.N - 1)) * r.ldw + t * 16;
  const uint8_t* x0[NB];
#pragma unroll
  for (int x = 0; x < NB; ++x) x0[x] = r.A + static_cast<int64_t>(min(x * 8 + g, p.M - 1)) * r.lda + t * 16;
  auto products = [&](const uint4& a0, const uint4& a1, const uint4 (&b)[NB]) {
#pragma unroll
    for (int x = 0; x < NB; ++x) {
      mma16832_e4m3(acc[x], a0.x, a1.x, a0.y, a1.y, b[x].x, b[x].y);
      mma16832_e4m3(acc[x], a0.z, a1.z, a0.w, a1.w, b[x].z, b[x].w);
    }
  };
  int c = static_cast<int>(static_cast<long long>(chunks) * warp / WARPS);
  const int whole = min(c1, p.K / 64);  // chunks that K does not cut
  for (; c + U <= whole; c += U) {
    uint4 a0[U], a1[U], b[U][NB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      a0[u] = ld_stream(w0 + static_cast<int64_t>(c + u) * 64);
      a1[u] = ld_stream(w1 + static_cast<int64_t>(c + u) * 64);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int x = 0; x < NB; ++x) b[u][x] = ld_keep(x0[x] + static_cast<int64_t>(c + u) * 64);
#pragma unroll
    for (int u = 0; u < U; ++u) products(a0[u], a1[u], b[u]);
  }
  for (; c < c1; ++c) {
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const int64_t at = static_cast<int64_t>(c) * 64;
    const bool in = c * 64 + t * 16 < p.K;
    const uint4 a0 = in ? ld_stream(w0 + at) : zero, a1 = in ? ld_stream(w1 + at) : zero;
    uint4 b[NB];
#pragma unroll
    for (int x = 0; x < NB; ++x) b[x] = in ? ld_keep(x0[x] + at) : zero;
    products(a0, a1, b);
  }
#pragma unroll
  for (int x = 0; x < NB; ++x) {
    part[warp][g][x * 8 + t * 2] = acc[x][0];
    part[warp][g][x * 8 + t * 2 + 1] = acc[x][1];
    part[warp][g + 8][x * 8 + t * 2] = acc[x][2];
    part[warp][g + 8][x * 8 + t * 2 + 1] = acc[x][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * 8 * NB; i += 32 * WARPS) {
    const int n = i & 15, m = i >> 4;
    if (m >= p.M || n0 + n >= p.N) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v += part[w][n][m];
    const float bias = p.bias != nullptr ? __ldg(p.bias + n0 + n) : 0.f;
    r.out[m * r.ldo + n0 + n] = __float2bfloat16_rn(fmaf(v * __ldg(p.sa + m), __ldg(p.sw + n0 + n), bias));
  }
}

}  // namespace vit
