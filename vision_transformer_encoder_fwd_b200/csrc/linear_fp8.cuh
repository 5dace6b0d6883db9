// Linear layer on 8-bit rows: out[m, n] = bf16(sa[m] sw[n] sum_k A[m, k] W[n, k] + b[n]) with A and W
// in e4m3, one fp32 scale per row of each, products accumulated in fp32.
//
// Tile kernel: persistent tcgen05 kind::f8f6f4, one CTA per SM of 10 warps in the roles of the bf16
// GEMM (TMA producer, MMA issuer, 8 epilogue warps; the accumulator double-buffered in TMEM).  A
// stage is 128 bytes deep, which is 128 values of K here (four K = 32 MMAs) where it is 64 in bf16,
// so a byte of shared memory feeds twice the work.  K past its end is zero-filled by the loads,
// rows past M and columns past N are cut by the stores.
#pragma once

#include "op_status.cuh"

namespace vit {

constexpr int LIN8_BM = 128;
constexpr int LIN8_BK = 128;  // bytes of K per stage
constexpr int LIN8_THREADS = 320;
constexpr int LIN8_EPI_WARPS = 8;
constexpr int DEV_TIMEOUT_LIN8 = 0x300;

struct Lin8Params {
  int M, N, K;
  const float* sa;    // [M]
  const float* sw;    // [N]
  const float* bias;  // [N] or NULL
  unsigned long long wait_ns;
};

template <int BN>
struct Lin8Cfg {
  static constexpr int STAGES = (BN == 256) ? 4 : 6;
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

// One warp's half of a tile (rows row0 .. row0 + 31, columns n0 .. n0 + BN/2 - 1): scales, bias,
// bf16, 64 columns per TMA store through the warp's staging buffer.  N is a multiple of 8, so
// a group of 8 columns is either inside or outside.
template <int BN>
__device__ __forceinline__ void lin8_epilogue(const Lin8Params& p, const CUtensorMap* tmO, uint32_t taddr, int row0,
                                              int n0, float sa, uint8_t* obuf) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int g = 0; g < BN / 128; ++g) {
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

template <int BN>
__global__ void __launch_bounds__(LIN8_THREADS, 1)
    lin8_tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmO, Lin8Params p, int* status) {
  using Cfg = Lin8Cfg<BN>;
  constexpr int STAGES = Cfg::STAGES;
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
  if (threadIdx.x == 0) *abort_flag = (*reinterpret_cast<volatile int*>(gstatus) != 0) ? 1 : 0;
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
                             static_cast<uint32_t>(acc * BN + half * (BN / 2));
      __syncwarp();
      if (row0 < p.M) lin8_epilogue<BN>(p, &tmO, taddr, row0, nb * BN + half * (BN / 2), sa, obuf);
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

}  // namespace vit
