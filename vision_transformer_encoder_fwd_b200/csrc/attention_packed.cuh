// Attention over packed sequences for sm_100a (tcgen05 + TMA): head widths 64 and 128, bf16 or fp16,
// grouped heads, queries and keys of different lengths, causal or full.
//
// Sequence i owns query rows cu_q[i] .. cu_q[i+1] - 1 and key rows cu_k[i] .. cu_k[i+1] - 1, of which
// the first len_k[i] are used.  Query row t (of lq) sees keys 0 .. lk - 1, or with `causal` keys
// 0 .. t + lk - lq (the last query sees the last key):
//   out = sum_j softmax_j(scale q . k_j) v_j,    a row that sees nothing is 0.
//
// One CTA per (128-query tile, head), 6 warps, two CTAs per SM, in the design of the fixed-length
// kernel (64-key sub-blocks, two S buffers in TMEM that they alternate between, P written over S,
// the running maximum moved only when it grows by more than 2^8):
//   warp 0      TMA: Q once, then K and V tiles of 64 keys in the order the MMAs use them
//   warp 1      TMEM and the MMAs  S_b = Q K_n^T (both from shared memory), O += P_n V_n
//   warps 2..5  softmax, one query row per thread
// How it differs: Q stays in shared memory (at width 128 there is no TMEM left for it: two S buffers
// and O fill the CTA's 256 columns), the row sums are kept in registers at width 128 and by
// the MMA (a column of ones behind V) at width 64.
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
  float scale_log2;  // scale * log2(e)
  unsigned long long wait_ns;
};

// Where a tile of `bm` query rows lies: sequence bounds, all clamped to the buffers.
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

// Finds tile number `want` in the order of the sequences, ceil(lq * mul / bm) tiles each (mul:
// rows per query).  One warp; every lane gets the answer.  Each round takes 128 sequences, four
// per lane, so that up to that many cost one trip to memory.  seq = -1: there is no such tile.
__device__ __forceinline__ SeqTile find_tile(const AttnPackedParams& p, int want, int bm, int mul) {
  const int lane = threadIdx.x & 31;
  SeqTile s;
  s.seq = -1;
  int before = 0;
  for (int base = 0; base < p.n; base += 128) {
    int c[5];
#pragma unroll
    for (int u = 0; u < 5; ++u) c[u] = clampi(p.cu_q[min(base + lane * 4 + u, p.n)], 0, p.Tq);
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
      int at = before + incl - sum, seq = -1, tile = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (want >= at && want < at + cnt[u]) {
          seq = base + lane * 4 + u;
          tile = want - at;
        }
        at += cnt[u];
      }
      const unsigned who = __ballot_sync(0xffffffffu, seq >= 0);
      const int src = __ffs(static_cast<int>(who)) - 1;
      s.seq = __shfl_sync(0xffffffffu, seq, src);
      s.tile = __shfl_sync(0xffffffffu, tile, src);
      seq_bounds(p, s.seq, s);
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

template <int HD>
struct AttnPackedCfg {
  static constexpr int UNIT = 64 * HD * 2;        // one K or V tile
  static constexpr int UNITS = (HD == 64) ? 10 : 5;
  static constexpr int Q_BYTES = 128 * HD * 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_RING = OFF_Q + Q_BYTES;
  static constexpr int OFF_ONES = OFF_RING + UNITS * UNIT;  // width 64: the atom of ones behind V
  static constexpr int OFF_BAR = OFF_ONES + (HD == 64 ? 8192 : 0);
  static constexpr int SMEM_BYTES = OFF_BAR + 256;
  static constexpr bool ONES = HD == 64;
  static constexpr uint32_t TMEM_COLS = 256;
  static constexpr int O_COLS = ONES ? 80 : HD;
  static constexpr uint32_t TM_S = 0, TM_O = 128;
  static_assert(SMEM_BYTES <= 115712, "two CTAs per SM");
  static_assert(8 * (2 * UNITS + 7) + 8 + 4 * 8 <= 256, "barrier area");
};

// Maxima that keep a NaN: a score that is one has to reach its row's output, and the row maximum is
// the way there (the FMA-pipe exponential would lose it).
__device__ __forceinline__ float maxn(float a, float b) { return max_nan(a, b); }
__device__ __forceinline__ float maxn(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float row_maxn64(const float (&s)[64]) {
  float m0 = maxn(s[0], s[1]), m1 = maxn(s[2], s[3]), m2 = maxn(s[4], s[5]), m3 = maxn(s[6], s[7]);
#pragma unroll
  for (int t = 8; t < 64; t += 8) {
    m0 = maxn(m0, s[t], s[t + 1]);
    m1 = maxn(m1, s[t + 2], s[t + 3]);
    m2 = maxn(m2, s[t + 4], s[t + 5]);
    m3 = maxn(m3, s[t + 6], s[t + 7]);
  }
  return maxn(m0, m1, maxn(m2, m3));
}

// m * c as the softmax's exponents subtract it: 0 for a row that has seen no key yet (its P are 0), NaN
// for a maximum of +infinity, whose row has no softmax.
__device__ __forceinline__ float max_offset(float m, float c) { return m == -INFINITY ? 0.f : fmaf(m, c, m - m); }

// P for one row of a 64-key sub-block, as softmax_sub_p with a scale known at launch; returns the
// sum of the unrounded values (used at width 128).
template <typename T, bool MASK, bool SUM>
__device__ __forceinline__ float packed_sub_p(const float (&s)[64], float c, float mc, int valid, uint32_t t_p,
                                              uint64_t* full) {
  const float2 cc = make_float2(c, c);
  const float2 nm = make_float2(-mc, -mc);
  float2 l0 = make_float2(0.f, 0.f), l1 = l0;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    uint32_t pk[16];
#pragma unroll
    for (int u = 0; u < 32; u += 2) {
      const int t = b * 32 + u;
      const float2 x = ffma2(make_float2(s[t], s[t + 1]), cc, nm);
      float2 e;
      if ((t & (kPolyEvery - 1)) == kPolyEvery - 2) {
        e = exp2_fma2(x);
        if (MASK) {
          e.x = (t < valid) ? e.x : 0.f;
          e.y = (t + 1 < valid) ? e.y : 0.f;
        }
      } else {
        e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
      }
      if (SUM) {
        if (u & 2)
          l1 = fadd2(l1, e);
        else
          l0 = fadd2(l0, e);
      }
      pk[u >> 1] = pack2<T>(e.x, e.y);
    }
    tmem_st16_nowait(t_p + b * 16, pk);
  }
  tmem_st_wait();
  tc_fence_before();
  mbar_arrive(full);
  return (l0.x + l0.y) + (l1.x + l1.y);
}

template <typename T, int HD>
__global__ void __launch_bounds__(ATT_THREADS, 2)
    attn_packed_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AttnPackedParams p,
                       int* status) {
  using Cfg = AttnPackedCfg<HD>;
  constexpr int UNITS = Cfg::UNITS;
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
  uint64_t* empty = full + UNITS;                                     // [UNITS]
  uint64_t* s_full = empty + UNITS;                                   // [2]
  uint64_t* p_full = s_full + 2;                                      // [2]
  uint64_t* pv_done = p_full + 2;
  uint64_t* mma_done = pv_done + 1;
  uint64_t* q_full = mma_done + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(q_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  SeqTile* s_tile = reinterpret_cast<SeqTile*>(tmem_holder + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y;
  const int hk = h / (p.Hq / p.Hkv);

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < UNITS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
    }
    mbar_init(pv_done, 1);
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
  if (threadIdx.x == 0) *abort_flag = (*reinterpret_cast<volatile int*>(gstatus) != 0) ? 1 : 0;
  if (warp == 2) {
    const SeqTile f = find_tile(p, static_cast<int>(blockIdx.x), ATT_BM, 1);
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
  if (p.causal && !skip) st.tile = (st.lq + ATT_BM - 1) / ATT_BM - 1 - st.tile;
  const int row0 = st.tile * ATT_BM;
  const int off = st.lk - st.lq;  // causal: row t sees keys 0 .. t + off
  const int kend = p.causal ? clampi(min(row0 + ATT_BM, st.lq) + off, 0, st.lk) : st.lk;
  const int nsub = skip ? 0 : (kend + 63) / 64;
  // ring position of the K and V tiles of sub-block n: K0 | K1 V0 | K2 V1 | ... | V(nsub-1)
  auto pos_k = [](int n) { return n == 0 ? 0 : 2 * n - 1; };
  auto pos_v = [nsub](int n) { return n + 1 < nsub ? 2 * n + 2 : 2 * n + 1; };

  if (nsub > 0 && warp == 0 && lane == 0) {
    // ------------------------------------------------------------------ TMA producer
    int issued_parity[UNITS];
#pragma unroll
    for (int s = 0; s < UNITS; ++s) issued_parity[s] = -1;
    mbar_arrive_expect_tx(q_full, Cfg::Q_BYTES);
#pragma unroll
    for (int c = 0; c < HD / 64; ++c)
      tma_load_3d(smem + Cfg::OFF_Q + c * 16384, &tmQ, c * 64, h, st.q0 + row0, q_full);
    int slot = 0;
    uint32_t ph = 0;
    auto load = [&](const CUtensorMap* tm, int key) {
      if (!mbar_wait(&empty[slot], ph ^ 1u, abort_flag, gstatus, DEV_TIMEOUT_ATTP + 1, wlim)) return false;
      mbar_arrive_expect_tx(&full[slot], Cfg::UNIT);
#pragma unroll
      for (int c = 0; c < HD / 64; ++c) tma_load_3d(ring + slot * Cfg::UNIT + c * 8192, tm, c * 64, hk, key, &full[slot]);
      issued_parity[slot] = static_cast<int>(ph);
      if (++slot == UNITS) {
        slot = 0;
        ph ^= 1u;
      }
      return true;
    };
    bool ok = true;
    for (int n = 0; ok && n <= nsub; ++n) {
      if (n < nsub) ok = load(&tmK, st.k0 + n * 64);
      if (ok && n > 0) ok = load(&tmV, st.k0 + (n - 1) * 64);
    }
    if (*abort_flag) {
      mbar_wait_drain(q_full, 0);
      for (int s = 0; s < UNITS; ++s)
        if (issued_parity[s] >= 0) mbar_wait_drain(&full[s], static_cast<uint32_t>(issued_parity[s]));
    }
  } else if (nsub > 0 && warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_of<T>(ATT_BM, 64, false);
      constexpr uint32_t idesc_o = idesc_of<T>(ATT_BM, Cfg::O_COLS, true);
      const uint32_t q0 = smem_u32(smem + Cfg::OFF_Q);
      const uint32_t r0 = smem_u32(ring);
      const uint32_t ones0 = smem_u32(smem + Cfg::OFF_ONES);
      const uint32_t t_s0 = tmem_base + Cfg::TM_S, t_o0 = tmem_base + Cfg::TM_O;
      auto issue_s = [&](int n) {
        const uint32_t kb = r0 + (pos_k(n) % UNITS) * Cfg::UNIT;
        const uint64_t dq = sdesc_sw128(q0, 16, 1024), dk = sdesc_sw128(kb, 16, 1024);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k)  // 16 values of the width each; 64 per 128-byte atom
          tc_mma_ss(t_s0 + 64 * (n & 1), dq + (k >> 2) * (16384 >> 4) + (k & 3) * 2,
                    dk + (k >> 2) * (8192 >> 4) + (k & 3) * 2, idesc_s, k != 0 ? 1u : 0u);
        tc_commit(&s_full[n & 1]);
        tc_commit(&empty[pos_k(n) % UNITS]);
      };
      auto wait_unit = [&](int pos, int site) {
        const bool got = mbar_wait<32>(&full[pos % UNITS], static_cast<uint32_t>(pos / UNITS) & 1u, abort_flag, gstatus,
                                       DEV_TIMEOUT_ATTP + site, wlim);
        tc_fence_after();
        return got;
      };
      bool ok = mbar_wait<32>(q_full, 0, abort_flag, gstatus, DEV_TIMEOUT_ATTP + 2, wlim) && wait_unit(pos_k(0), 3);
      if (ok) issue_s(0);
      if (ok && nsub > 1) {
        ok = wait_unit(pos_k(1), 3);
        if (ok) issue_s(1);
      }
      for (int n = 0; ok && n < nsub; ++n) {
        ok = mbar_wait<32>(&p_full[n & 1], static_cast<uint32_t>(n >> 1) & 1u, abort_flag, gstatus,
                           DEV_TIMEOUT_ATTP + 4, wlim) &&
             wait_unit(pos_v(n), 5);
        if (!ok) break;
        const uint32_t vb = r0 + (pos_v(n) % UNITS) * Cfg::UNIT;
        const uint64_t dv = sdesc_sw128(vb, Cfg::ONES ? ones0 - vb : 8192u, 1024);
        const uint32_t tp = t_s0 + 64 * (n & 1);
        const uint32_t a_p[4] = {tp, tp + 8, tp + 16, tp + 24};
        const uint64_t b_v[4] = {dv, dv + 128, dv + 256, dv + 384};
        tc_mma_ts_chain4(t_o0, a_p, b_v, idesc_o, n > 0 ? 1u : 0u);
        tc_commit(pv_done);
        tc_commit(&empty[pos_v(n) % UNITS]);
        if (n + 2 < nsub) {
          ok = wait_unit(pos_k(n + 2), 6);
          if (ok) issue_s(n + 2);
        }
      }
      tc_commit(mma_done);
    }
    __syncwarp();
  } else if (!skip && warp >= 2) {
    // ------------------------------------------------------------------ softmax
    const int q = warp & 3;
    const int r = q * 32 + lane;
    const int row = row0 + r;
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t t_s = tmem_base + lane_off + Cfg::TM_S;
    const uint32_t t_o = tmem_base + lane_off + Cfg::TM_O;
    const int lim = p.causal ? min(st.lk, row + off + 1) : st.lk;  // keys this row sees (<= 0: none)
    const float c = p.scale_log2;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int n = 0; n < nsub; ++n) {
      const int buf = n & 1;
      if (!mbar_wait_warp(&s_full[buf], static_cast<uint32_t>(n >> 1) & 1u, abort_flag, gstatus, DEV_TIMEOUT_ATTP + 7,
                          wlim)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float s[64];
      __syncwarp();
      tmem_ld64(t_s + 64 * buf, s);
      const int valid = lim - n * 64;
      const bool part = __any_sync(0xffffffffu, valid < 64);
      if (part) {
#pragma unroll
        for (int t = 0; t < 64; ++t) s[t] = (t < valid) ? s[t] : -INFINITY;
      }
      const float m_new = maxn(m, row_maxn64(s));
      const bool resc = !((m_new - m) * c <= kRescaleLog2) && m_new != -INFINITY;  // a NaN moves it too
      float alpha = 1.f;
      if (resc) {
        alpha = ex2_approx((m - m_new) * c);
        m = m_new;
      }
      if (n > 0 && __any_sync(0xffffffffu, resc)) {
        if (!mbar_wait_warp(pv_done, static_cast<uint32_t>(n - 1) & 1u, abort_flag, gstatus, DEV_TIMEOUT_ATTP + 8,
                            wlim)) {
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
      if (n == nsub - 1 && st.lk < nsub * 64) {
        // V rows past the sequence's keys: zeros
        const int pos = pos_v(n);
        if (!mbar_wait_warp(&full[pos % UNITS], static_cast<uint32_t>(pos / UNITS) & 1u, abort_flag, gstatus,
                            DEV_TIMEOUT_ATTP + 9, wlim)) {
          ok = false;
          break;
        }
        const int from = st.lk - n * 64;
        uint4* vt = reinterpret_cast<uint4*>(ring + (pos % UNITS) * Cfg::UNIT);
        for (int i = from * 8 + r; i < 512; i += 128) {
#pragma unroll
          for (int a = 0; a < HD / 64; ++a) vt[a * 512 + i] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      const float mc = max_offset(m, c);
      __syncwarp();
      l = l * alpha + (part ? packed_sub_p<T, true, !Cfg::ONES>(s, c, mc, valid, t_s + 64 * buf, &p_full[buf])
                            : packed_sub_p<T, false, !Cfg::ONES>(s, c, mc, valid, t_s + 64 * buf, &p_full[buf]));
    }
    if (ok && nsub > 0) ok = mbar_wait_warp(mma_done, 0, abort_flag, gstatus, DEV_TIMEOUT_ATTP + 10, wlim);
    if (ok) {
      tc_fence_after();
      if (Cfg::ONES && nsub > 0) {
        float ls[16];
        __syncwarp();
        tmem_ld16(t_o + 64, ls);
        l = ls[0];
      }
      const float inv = (lim > 0 && nsub > 0) ? 1.0f / l : 0.f;
      T* dst = static_cast<T*>(p.out) + static_cast<int64_t>(st.q0 + row) * p.o_tok + h * p.o_head;
#pragma unroll 1
      for (int u = 0; u < HD; u += 64) {
        float o[64];
        __syncwarp();
        if (nsub > 0) tmem_ld64(t_o + u, o);
        if (row < st.lq) {
          uint4* d4 = reinterpret_cast<uint4*>(dst + u);
#pragma unroll
          for (int t = 0; t < 8; ++t)
            d4[t] = lim > 0 && nsub > 0
                        ? make_uint4(pack2<T>(o[8 * t + 0] * inv, o[8 * t + 1] * inv),
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
    if (nsub > 0 && lane == 0) mbar_wait_drain(mma_done, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
  }
}

}  // namespace vit
