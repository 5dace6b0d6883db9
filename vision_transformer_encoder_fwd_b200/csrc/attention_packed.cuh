// Attention over packed sequences for sm_100a (tcgen05 + TMA): head widths 64 and 128, bf16 or fp16,
// grouped heads, queries and keys of different lengths, causal or full.
//
// Sequence i owns query rows cu_q[i] .. cu_q[i+1] - 1 and key rows cu_k[i] .. cu_k[i+1] - 1, of which
// the first len_k[i] are used.  Query row t (of lq) sees keys 0 .. lk - 1, or with `causal` keys
// 0 .. t + lk - lq (the last query sees the last key):
//   out = sum_j softmax_j(scale q . k_j) v_j,    a row that sees nothing is 0.
//
// One CTA per (tile of 128 rows, group of heads), 6 warps.  A row is one query of one head: the heads
// of a tile share a key head, `pack` of them side by side (row t * pack + g), so that short sequences
// with grouped heads still fill a tile.
//   warp 0      TMA: Q once, then K and V blocks of 64 keys in the order the MMAs use them
//   warp 1      TMEM and the MMAs  S = Q K_n^T (both from shared memory), O += P_n V_n
//   warps 2..5  softmax, one row per thread; P is written over S
// There are two S buffers in tensor memory, so that the S of the next block is there when a softmax ends, and two
// CTAs per SM.  The softmax's exponentials (16 a clock and SM on the special-function unit) bound it at
// width 64, the MMAs with them at width 128; what it costs in practice is the latency of a row's chain: S
// from tensor memory, maximum, exponentials, P back, O and the next S (about 1400 clocks for 64 keys, half
// of it hidden by the other CTA).  The MMAs are issued by a thread chosen by elect.sync, which lets the
// compiler keep descriptors in uniform registers (four MMAs and a commit take 135 clocks; 365 under an
// ordinary predicate), with one commit for S and one for O (the copies' slots are freed by the same
// barriers) and K and V in hand before it waits for P.  The running maximum moves only when it grows by
// more than 2^8.
// Measured: 8 x 4101 tokens, 16 heads of 64, 734 us (751 TFLOP/s); 2 x 8192, 16 heads of 128, 875 us (1257
// TFLOP/s); a causal prompt of 8191, 32 heads on 8 of 128, 536-541 us (1020 TFLOP/s).
// What a tile reads past its sequence's last key belongs to somebody else or to nobody and may be
// NaN: scores there are replaced before use, and V's rows there are overwritten with zeros in
// shared memory, since 0 * NaN would reach every row of O.
// The lengths exist only on the device.  The grid is the most tiles that Tq rows in n sequences
// can need; each CTA finds its sequence from cu_q and returns if there is none.
#pragma once

#include <type_traits>

#include "attention.cuh"
#include "op_status.cuh"
#include "rows.cuh"

namespace vit {

constexpr int DEV_TIMEOUT_ATTP = 0x400;

struct AttnPackedParams {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head, o_tok, o_head;  // strides in elements
  const int* cu_q;
  const int* cu_k;
  const int* len_k;  // or NULL
  int n, Tq, Tk, Hq, Hkv, causal;
  int pack, tokens;  // tile kernel: heads and queries a tile
  float scale_log2;  // scale * log2(e)
  unsigned long long wait_ns;
};

// Where a tile of queries lies: sequence bounds, all clamped to the buffers.
struct SeqTile {
  int q0, lq, k0, lk, tile, seq;
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

__device__ __forceinline__ void seq_bounds(const AttnPackedParams& p, int i, SeqTile& s) {
  s.q0 = clampi(p.cu_q[i], 0, p.Tq);
  s.lq = max(0, clampi(p.cu_q[i + 1], 0, p.Tq) - s.q0);
  s.k0 = clampi(p.cu_k[i], 0, p.Tk);
  s.lk = max(0, clampi(p.cu_k[i + 1], 0, p.Tk) - s.k0);
  if (p.len_k != nullptr) s.lk = clampi(p.len_k[i], 0, s.lk);
}

// Finds tile number `want` in the order of the sequences, ceil(lq * mul / bm) tiles each.  One warp; every
// lane gets the answer.  Each round takes 128 sequences, four per lane, with all their bounds, so that up to
// that many cost one trip to memory.  seq = -1: there is no such tile.
__device__ __forceinline__ SeqTile find_tile(const AttnPackedParams& p, int want, int bm, int mul = 1) {
  const int lane = threadIdx.x & 31;
  SeqTile s{0, 0, 0, 0, 0, -1};
  int before = 0;
  for (int base = 0; base < p.n; base += 128) {
    int c[5], k[5], len[4];
#pragma unroll
    for (int u = 0; u < 5; ++u) {
      const int i = min(base + lane * 4 + u, p.n);
      c[u] = clampi(p.cu_q[i], 0, p.Tq);
      k[u] = clampi(p.cu_k[i], 0, p.Tk);
      if (u < 4) len[u] = p.len_k != nullptr ? p.len_k[min(i, p.n - 1)] : 0x7fffffff;
    }
    int cnt[4], sum = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      cnt[u] = (base + lane * 4 + u < p.n) ? (max(0, c[u + 1] - c[u]) * mul + bm - 1) / bm : 0;
      sum += cnt[u];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    if (want < before + total) {
      int at = before + incl - sum;
      SeqTile f{0, 0, 0, 0, 0, -1};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (want >= at && want < at + cnt[u]) {
          f.seq = base + lane * 4 + u;
          f.tile = want - at;
          f.q0 = c[u];
          f.lq = max(0, c[u + 1] - c[u]);
          f.k0 = k[u];
          f.lk = clampi(len[u], 0, max(0, k[u + 1] - k[u]));
        }
        at += cnt[u];
      }
      const int src = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, f.seq >= 0))) - 1;
      s.q0 = __shfl_sync(0xffffffffu, f.q0, src);
      s.lq = __shfl_sync(0xffffffffu, f.lq, src);
      s.k0 = __shfl_sync(0xffffffffu, f.k0, src);
      s.lk = __shfl_sync(0xffffffffu, f.lk, src);
      s.tile = __shfl_sync(0xffffffffu, f.tile, src);
      s.seq = __shfl_sync(0xffffffffu, f.seq, src);
      return s;
    }
    before += total;
  }
  return s;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) { return pack_bf16x2(lo, hi); }
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// idesc_bf16 with the input format of T (fp16: format 0).
template <typename T>
__host__ __device__ constexpr uint32_t idesc_of(int M, int N, bool b_mn_major) {
  return std::is_same<T, __half>::value ? idesc_bf16(M, N, b_mn_major) & ~((1u << 7) | (1u << 10))
                                        : idesc_bf16(M, N, b_mn_major);
}

// Maximum that keeps a NaN.
__device__ __forceinline__ float maxn(float a, float b) { return max_nan(a, b); }

// m * c as the softmax's exponents subtract it: 0 for a row that has seen no key yet (its P are 0), NaN
// for a maximum of +infinity, whose row has no softmax.
__device__ __forceinline__ float max_offset(float m, float c) { return m == -INFINITY ? 0.f : fmaf(m, c, m - m); }

// Factor that brings sums at maximum m to the common maximum top.
__device__ __forceinline__ float to_max(float m, float top, float c) { return m == top ? 1.f : ex2_approx((m - top) * c); }

// One thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
// Bounded waits, by a whole warp or by one thread, whose slow part stays out of the loops that wait.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* gstatus, int site,
                                       unsigned long long limit) {
  uint64_t* b = static_cast<uint64_t*>(__cvta_shared_to_generic(bar));
  return mbar_wait_warp<32>(b, parity, abort_flag, gstatus, site, limit);
}
__device__ __noinline__ bool wait_one_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* gstatus, int site,
                                           unsigned long long limit) {
  return mbar_wait<32>(static_cast<uint64_t*>(__cvta_shared_to_generic(bar)), parity, abort_flag, gstatus, site, limit);
}
// An arrival without a branch around it.
__device__ __forceinline__ void arrive_if(bool yes, uint32_t bar) {
  asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 st;\n\tsetp.ne.b32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar),
               "r"(yes ? 1 : 0)
               : "memory");
}
__device__ __forceinline__ bool test_bar(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* gstatus, int site,
                                          unsigned long long limit) {
  if (__all_sync(0xffffffffu, test_bar(bar, parity))) return true;
  return wait_slow(bar, parity, abort_flag, gstatus, site, limit);
}
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* gstatus, int site,
                                         unsigned long long limit) {
  return test_bar(bar, parity) || wait_one_slow(bar, parity, abort_flag, gstatus, site, limit);
}

template <int HD>
struct AttnPackedCfg {
  static constexpr int UNIT = 64 * HD * 2;  // a K or V tile of 64 keys, slabs of 64 values
  static constexpr int UNITS = (HD == 64) ? 10 : 5;
  static constexpr int PER_SM = 2;
  static constexpr int Q_BYTES = 128 * HD * 2;
  static constexpr bool ONES = HD == 64;  // row sums by the MMA: a column of ones behind V
  static constexpr int O_COLS = ONES ? 80 : HD;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_RING = OFF_Q + Q_BYTES;
  static constexpr int OFF_ONES = OFF_RING + UNITS * UNIT;
  static constexpr int OFF_BAR = OFF_ONES + (ONES ? 8192 : 0);
  static constexpr int DONE = 8;  // barriers in turn for finished S and for finished O
  static constexpr int SMEM_BYTES = OFF_BAR + 512;
  static constexpr uint32_t TMEM_COLS = 256;
  static constexpr uint32_t TM_S = 0, TM_O = 128;
  static_assert(PER_SM * (SMEM_BYTES + 1024) <= 233472, "CTAs per SM");
  static_assert(DONE > UNITS / 2 + 1, "a slot's barrier is read before it comes round again");
  static_assert(8 * (UNITS + 2 * DONE + 4) + 8 + 8 * 4 <= 512, "barrier area");
};

// 2^x for a pair on the FMA pipe, as exp2_fma2 (off by at most 7.5e-5 of the value, a sixth of what rounding P to
// fp16 may take, less of bf16's), but with a NaN kept and exactly 0 from -126.5 down: the clamp gives j = -127,
// whose power of two has no exponent bits.
__device__ __forceinline__ float2 exp2_fma2_full(float2 x) {
  x.x = max_nan(x.x, -127.0f);
  x.y = max_nan(x.y, -127.0f);
  const float2 t = fadd2(x, make_float2(12582912.0f, 12582912.0f));
  const float2 j = fadd2(t, make_float2(-12582912.0f, -12582912.0f));
  const float2 f = fadd2(x, make_float2(-j.x, -j.y));
  float2 p = ffma2(make_float2(0.0551716685f, 0.0551716685f), f, make_float2(0.242611125f, 0.242611125f));
  p = ffma2(p, f, make_float2(0.693260968f, 0.693260968f));
  p = ffma2(p, f, make_float2(0.999928057f, 0.999928057f));
  const float2 two_j = make_float2(__int_as_float((__float_as_int(t.x) << 23) + 0x3f800000),
                                   __int_as_float((__float_as_int(t.y) << 23) + 0x3f800000));
  return ffma2(p, two_j, make_float2(0.f, 0.f));
}

// P for 64 keys of one row: 2^(s c - mc), rounded, into 32 columns of tensor memory; with SUM returns the
// sum of the unrounded values.  P has V's type because both operands of an MMA have one: half a step of it a
// weight, which is the whole of the difference from 32-bit softmax (error against 64 bits, bf16: 2.3e-3 of the
// result where rounding the result alone gives 1.7e-3).  A remainder as in attn_rows_kernel would double these MMAs.  Masked scores are -infinity.  Every POLY-th pair of exponentials goes to the
// FMA pipe (4th at width 64, 8th at 128: 2nd to 16th were within 5 %, the 2nd slowest).
template <typename T, bool SUM, int POLY>
__device__ __forceinline__ float packed_p64(const float (&s)[64], float c, float mc, uint32_t t_p) {
  const float2 cc = make_float2(c, c);
  const float2 nm = make_float2(-mc, -mc);
  float2 l0 = make_float2(0.f, 0.f), l1 = l0;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    uint32_t pk[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      const int t = b * 32 + u * 2;
      const float2 x = ffma2(make_float2(s[t], s[t + 1]), cc, nm);
      float2 e;
      if ((t >> 1) % POLY == POLY - 1)
        e = exp2_fma2_full(x);
      else
        e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
      if (SUM) {
        if (u & 1)
          l1 = fadd2(l1, e);
        else
          l0 = fadd2(l0, e);
      }
      pk[u] = pack2<T>(e.x, e.y);
    }
    tmem_st16_nowait(t_p + b * 16, pk);
  }
  return (l0.x + l0.y) + (l1.x + l1.y);
}

template <typename T, int HD>
__global__ void __launch_bounds__(ATT_THREADS, AttnPackedCfg<HD>::PER_SM)
    attn_packed_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AttnPackedParams p,
                       int* status) {
  using Cfg = AttnPackedCfg<HD>;
  constexpr int UNITS = Cfg::UNITS, DONE = Cfg::DONE;
  int* gstatus = op_status(status);
  const unsigned long long wlim = p.wait_ns;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled layouts need 1024-byte aligned tiles
    pdl_wait();
    if (threadIdx.x == 0) atomicExch(gstatus, DEV_TIMEOUT_ATTP + 15);
    return;
  }
  uint8_t* ring = smem + Cfg::OFF_RING;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);  // [UNITS]
  uint64_t* s_done = full + UNITS;                                    // [DONE] S of block n
  uint64_t* pv_done = s_done + DONE;                                  // [DONE] O of block n
  uint64_t* p_full = pv_done + DONE;                                  // [2] P in an S buffer
  uint64_t* mma_done = p_full + 2;
  uint64_t* q_full = mma_done + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(q_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  SeqTile* s_tile = reinterpret_cast<SeqTile*>(tmem_holder + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int h0 = blockIdx.y * p.pack;  // first query head
  const int hk = h0 / (p.Hq / p.Hkv);

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < UNITS; ++s) mbar_init(&full[s], 1);
    for (int s = 0; s < DONE; ++s) {
      mbar_init(&s_done[s], 1);
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(&p_full[0], 4);  // a warp's lanes arrive as one
    mbar_init(&p_full[1], 4);
    mbar_init(mma_done, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (Cfg::ONES) {
    // 64 key rows of 128 bytes in the 128-byte-swizzled MN-major layout: 1 at N position 0 of every
    // row (16-byte chunk 0, swizzled to chunk r % 8), 0 elsewhere
    constexpr uint32_t one = std::is_same<T, __half>::value ? 0x3C00u : 0x3F80u;
    uint4* ones = reinterpret_cast<uint4*>(smem + Cfg::OFF_ONES);
    for (int i = threadIdx.x; i < 8192 / 16; i += blockDim.x)
      ones[i] = make_uint4(((i & 7) == ((i >> 3) & 7)) ? one : 0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, Cfg::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();
  if (threadIdx.x == 0) *abort_flag = op_stopped(status) ? 1 : 0;
  if (warp == 2) {
    const SeqTile f = find_tile(p, static_cast<int>(blockIdx.x), p.tokens);
    if (lane == 0) *s_tile = f;
  }
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  SeqTile st = *s_tile;
  const bool skip = *abort_flag != 0 || st.seq < 0;
  // the longest tiles first: with a causal mask the last tile of a sequence sees the most keys
  if (p.causal && !skip) st.tile = (st.lq + p.tokens - 1) / p.tokens - 1 - st.tile;
  const int tok0 = st.tile * p.tokens;
  const int off = st.lk - st.lq;  // causal: query t sees keys 0 .. t + off
  const int kend = p.causal ? clampi(min(tok0 + p.tokens, st.lq) + off, 0, st.lk) : st.lk;
  const int nblk = skip ? 0 : (kend + 63) / 64;
  // place in the ring of the K and V tiles of block n: K0 | K1 V0 | K2 V1 | ... | V(nblk-1)
  auto pos_k = [](int n) { return n == 0 ? 0 : 2 * n - 1; };
  auto pos_v = [nblk](int n) { return n + 1 < nblk ? 2 * n + 2 : 2 * n + 1; };

  if (nblk > 0 && warp == 0 && lane == 0) {
    // ------------------------------------------------------------------ TMA producer
    int issued_parity[UNITS];
#pragma unroll
    for (int s = 0; s < UNITS; ++s) issued_parity[s] = -1;
    const int q_bytes = p.tokens * p.pack * 128;  // of a slab of 64 values
    mbar_arrive_expect_tx(q_full, q_bytes * (HD / 64));
#pragma unroll
    for (int c = 0; c < HD / 64; ++c)
      tma_load_3d(smem + Cfg::OFF_Q + c * 16384, &tmQ, c * 64, h0, st.q0 + tok0, q_full);
    for (int pos = 0; pos < 2 * nblk; ++pos) {
      const int slot = pos % UNITS;
      if (pos >= UNITS) {  // the slot's last tile has been used: K by its S, V by its O
        const int old = pos - UNITS;
        const bool was_k = old == 0 || (old & 1);
        const int b = was_k ? (old + 1) >> 1 : (old >> 1) - 1;
        if (!mbar_wait(&(was_k ? s_done : pv_done)[b % DONE], static_cast<uint32_t>(b / DONE) & 1u, abort_flag, gstatus,
                       DEV_TIMEOUT_ATTP + 1, wlim))
          break;
      }
      const bool is_k = pos == 0 || ((pos & 1) && pos != 2 * nblk - 1);
      const int b = is_k ? (pos + 1) >> 1 : (pos == 2 * nblk - 1 ? nblk - 1 : (pos >> 1) - 1);
      mbar_arrive_expect_tx(&full[slot], Cfg::UNIT);
#pragma unroll
      for (int c = 0; c < HD / 64; ++c)
        tma_load_3d(ring + slot * Cfg::UNIT + c * 8192, is_k ? &tmK : &tmV, c * 64, hk, st.k0 + b * 64, &full[slot]);
      issued_parity[slot] = (pos / UNITS) & 1;
    }
    if (*abort_flag) {
      mbar_wait_drain(q_full, 0);
      for (int s = 0; s < UNITS; ++s)
        if (issued_parity[s] >= 0) mbar_wait_drain(&full[s], static_cast<uint32_t>(issued_parity[s]));
    }
  } else if (nblk > 0 && warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      constexpr uint32_t idesc_s = idesc_of<T>(ATT_BM, 64, false);
      constexpr uint32_t idesc_o = idesc_of<T>(ATT_BM, Cfg::O_COLS, true);
      const uint64_t dq = sdesc_sw128(smem_u32(smem + Cfg::OFF_Q), 16, 1024);
      const uint32_t r0 = smem_u32(ring), ones0 = smem_u32(smem + Cfg::OFF_ONES);
      const uint64_t dk0 = sdesc_sw128(r0, 16, 1024);
      const uint32_t full0 = smem_u32(full), p_full0 = smem_u32(p_full);
      const uint32_t t_s = tmem_base + Cfg::TM_S, t_o = tmem_base + Cfg::TM_O;
      uint32_t kslot = 0, kph = 0;  // of the next K
      auto have_k = [&]() { return wait_one(full0 + kslot * 8, kph, abort_flag, gstatus, DEV_TIMEOUT_ATTP + 3, wlim); };
      auto issue_s = [&](int n) {
        const uint64_t dk = dk0 + kslot * (Cfg::UNIT >> 4);
        const uint32_t d = t_s + 64 * (n & 1);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k)  // 16 values of the width each; 64 a slab
          tc_mma_ss(d, dq + (k >> 2) * (16384 >> 4) + (k & 3) * 2, dk + (k >> 2) * (8192 >> 4) + (k & 3) * 2, idesc_s,
                    k != 0 ? 1u : 0u);
        tc_commit(&s_done[n % DONE]);
        kslot += n == 0 ? 1 : 2;  // K0 | K1 V0 | K2 V1 ...
        if (kslot >= UNITS) {
          kslot -= UNITS;
          kph ^= 1u;
        }
      };
      bool ok = wait_one(smem_u32(q_full), 0, abort_flag, gstatus, DEV_TIMEOUT_ATTP + 2, wlim);
#pragma unroll 1
      for (int n = 0; ok && n < 2 && n < nblk; ++n) {
        ok = have_k();
        tc_fence_after();
        if (ok) issue_s(n);
      }
#pragma unroll 1
      for (int n = 0; ok && n < nblk; ++n) {
        const int pos = pos_v(n);
        const uint32_t slot = static_cast<uint32_t>(pos % UNITS);
        const uint32_t vb = r0 + slot * Cfg::UNIT;
        const uint64_t dv = sdesc_sw128(vb, Cfg::ONES ? ones0 - vb : 8192u, 1024);
        const uint32_t tp = t_s + 64 * (n & 1);
        ok = wait_one(full0 + slot * 8, static_cast<uint32_t>(pos / UNITS) & 1u, abort_flag, gstatus, DEV_TIMEOUT_ATTP + 5,
                      wlim) &&
             (n + 2 >= nblk || have_k()) &&
             wait_one(p_full0 + (n & 1) * 8, static_cast<uint32_t>(n >> 1) & 1u, abort_flag, gstatus, DEV_TIMEOUT_ATTP + 4,
                      wlim);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k) tc_mma_ts(t_o, tp + 8 * k, dv + 128 * k, idesc_o, n > 0 || k > 0 ? 1u : 0u);
        tc_commit(&pv_done[n % DONE]);
        if (n + 2 < nblk) issue_s(n + 2);  // into the buffer that P has just left: MMAs run in order
      }
      tc_commit(mma_done);
    }
    __syncwarp();
  } else if (!skip && warp >= 2) {
    // ------------------------------------------------------------------ softmax
    const int q = warp & 3;
    const int r = q * 32 + lane;
    const int tt = r / p.pack;
    const int tok = tok0 + tt;
    const bool mine = tt < p.tokens && tok < st.lq;
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t t_s = tmem_base + lane_off + Cfg::TM_S;
    const uint32_t t_o = tmem_base + lane_off + Cfg::TM_O;
    // keys this row sees (<= 0: none); rows of nobody go along with the last one
    const int lim = p.causal ? min(st.lk, min(tok, st.lq - 1) + off + 1) : st.lk;
    const uint32_t s_done0 = smem_u32(s_done), p_full0 = smem_u32(p_full);
    const int whole = __reduce_min_sync(0xffffffffu, max(lim, 0)) / 64;  // blocks that every row of the warp sees whole
    const float c = p.scale_log2;
    float m = -INFINITY, mc = 0.f, l = 0.f;  // mc: m c, 0 for a row that has seen no key
    bool ok = true;
    // Two CTAs of an SM that start together stay in step, both at their exponentials and then both not: the one
    // with the upper half of tensor memory begins 0.4 us later (8 x 4101 tokens, 16 heads of 64: 795 -> 749
    // us; 2 x 8192, 16 of 128: 899 -> 874; 0.2 and 0.7 us were within 2 %)
    if (nblk > 4 && (tmem_base & 0xffffu) != 0) __nanosleep(400);
    for (int n = 0; n < nblk; ++n) {
      if (!wait_warp(s_done0 + (n % DONE) * 8, static_cast<uint32_t>(n / DONE) & 1u, abort_flag, gstatus, DEV_TIMEOUT_ATTP + 7,
                     wlim)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t t_b = t_s + 64 * (n & 1);
      float s[64];
      __syncwarp();
      tmem_ld64(t_b, s);
      if (__builtin_expect(n >= whole, 0)) {
        const int valid = lim - n * 64;
#pragma unroll
        for (int t = 0; t < 64; ++t) s[t] = (t < valid) ? s[t] : -INFINITY;
      }
      const float m_new = fmaxf(m, row_max64(s));
      const bool resc = !((m_new - m) * c <= kRescaleLog2) && m_new != -INFINITY;
      if (__builtin_expect(__any_sync(0xffffffffu, resc), 0)) {
        const float alpha = resc ? to_max(m, m_new, c) : 1.f;
        if (resc) {
          m = m_new;
          mc = max_offset(m, c);
        }
        l *= alpha;
        if (n > 0) {
          if (!wait_warp(smem_u32(pv_done) + ((n - 1) % DONE) * 8, static_cast<uint32_t>((n - 1) / DONE) & 1u, abort_flag,
                         gstatus, DEV_TIMEOUT_ATTP + 8, wlim)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int u = 0; u < Cfg::O_COLS; u += 16) {
            float o[16];
            tmem_ld16(t_o + u, o);
            uint32_t ob[16];
#pragma unroll
            for (int t = 0; t < 16; ++t) ob[t] = __float_as_uint(o[t] * alpha);
            tmem_st16(t_o + u, ob);
          }
        }
      }
      if (__builtin_expect(n == nblk - 1 && st.lk < nblk * 64, 0)) {
        // V rows past the sequence's keys: zeros
        const int pos = pos_v(n);
        if (!wait_warp(smem_u32(&full[pos % UNITS]), static_cast<uint32_t>(pos / UNITS) & 1u, abort_flag, gstatus,
                       DEV_TIMEOUT_ATTP + 9, wlim)) {
          ok = false;
          break;
        }
        uint4* vt = reinterpret_cast<uint4*>(ring + (pos % UNITS) * Cfg::UNIT);
        for (int i = (st.lk - n * 64) * 8 + r; i < 512; i += 128) {
#pragma unroll
          for (int a = 0; a < HD / 64; ++a) vt[a * 512 + i] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      l += packed_p64<T, !Cfg::ONES, HD == 64 ? 4 : 8>(s, c, mc, t_b);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      arrive_if(lane == 0, p_full0 + (n & 1) * 8);
    }
    if (ok && nblk > 0) ok = wait_warp(smem_u32(mma_done), 0, abort_flag, gstatus, DEV_TIMEOUT_ATTP + 10, wlim);
    if (ok) {
      tc_fence_after();
      const bool sees = lim > 0 && nblk > 0;
      if (Cfg::ONES && nblk > 0) {
        float ls[16];
        __syncwarp();
        tmem_ld16(t_o + 64, ls);
        l = ls[0];
      }
      const float inv = sees ? 1.0f / l : 0.f;
      T* dst = static_cast<T*>(p.out) + static_cast<int64_t>(st.q0 + tok) * p.o_tok +
               static_cast<int64_t>(h0 + r - tt * p.pack) * p.o_head;
#pragma unroll 1
      for (int u = 0; u < HD; u += 64) {
        float o[64];
        __syncwarp();
        if (nblk > 0) tmem_ld64(t_o + u, o);
        if (mine) {
          uint4* d4 = reinterpret_cast<uint4*>(dst + u);
#pragma unroll
          for (int t = 0; t < 8; ++t)
            d4[t] = sees ? make_uint4(pack2<T>(o[8 * t + 0] * inv, o[8 * t + 1] * inv),
                                      pack2<T>(o[8 * t + 2] * inv, o[8 * t + 3] * inv),
                                      pack2<T>(o[8 * t + 4] * inv, o[8 * t + 5] * inv),
                                      pack2<T>(o[8 * t + 6] * inv, o[8 * t + 7] * inv))
                         : make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
  }

  // ------------------------------------------------------------------ teardown
  __syncthreads();
  if (warp == 1) {
    if (nblk > 0 && lane == 0) mbar_wait_drain(mma_done, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
  }
}

}  // namespace vit
