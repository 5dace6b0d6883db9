// Attention over packed sequences for few query rows per sequence (single tokens over a cache, short
// prompts): the same mathematics and arguments as attn_packed_kernel, in 16-row tiles on mma.sync.
//
// With r rows reading a sequence's keys the work is 4 r flops a value of K and V, so below about 64 rows
// the bytes bound it and a 128-row tensor-memory tile is mostly padding.  Here the rows of all query
// heads of one key head (query t, head g of the group: row t * group + g) form 16-row tiles, and
// the keys are the long axis:
//   - The work is a line of units, one per (sequence, key head, row tile, 64-key block) in that
//     order.  Each CTA takes an equal piece of it, wherever sequences begin and end, so that long
//     and short ones balance; lengths are only known on the device, and every CTA adds them up
//     itself.  An item (tile) that a piece boundary cuts leaves partial results (maximum, sum,
//     unnormalised output, fp32) in the workspace, two slots a CTA, and attn_join_kernel joins them in
//     the order of the pieces, so that results do not depend on the order of execution.
//   - Warp 4 feeds a ring of stages: K and V blocks by TMA, and at an item's first block its Q rows
//     by cp.async.  It runs ahead over item boundaries.  Warps 0..3 take 16 keys of each block
//     each, with a running maximum, sum and output of their own, and meet only at the end of an
//     item, through the shared memory of its last stage.
//   - P is kept as a pair of 16-bit numbers (value and remainder, two products with V): the matrix
//     pipe has room to spare, and single tokens keep nearly fp32 accuracy.
// Measured: 64 tokens over caches of 33 to 4096 keys, 32 heads on 8 of 128, 98-101 us (5.1-5.2 TB/s); one token over
// 100003 keys 75 us (5.4 TB/s), over 400003 256 us (6.4 TB/s).
// Scores past a row's last key are replaced before use; V's rows past the sequence's last key are
// overwritten with zeros in shared memory (0 * NaN).
#pragma once

#include "attention_packed.cuh"

namespace vit {

constexpr int DEV_TIMEOUT_ATTR = 0x500;
constexpr int ATTR_THREADS = 160;
constexpr int ATTR_MIN_UNITS = 2;  // least 64-key blocks a CTA takes

template <int HD>
struct AttnRowsCfg {
  static constexpr int K_BYTES = 64 * HD * 2;
  static constexpr int Q_BYTES = 16 * HD * 2;
  static constexpr int STAGE = 2 * K_BYTES + Q_BYTES;  // K | V | Q
  static constexpr int STAGES = HD == 64 ? 4 : 3;
  static constexpr int OFF_BAR = STAGES * STAGE;
  static constexpr int SMEM_BYTES = OFF_BAR + 1536;
  static constexpr int PER_SM = HD == 64 ? 3 : 2;
  static_assert(PER_SM * (SMEM_BYTES + 1024) <= 233472, "CTAs per SM");
};

// Division by a number known at launch (Granlund and Montgomery): n / d for 0 <= n < 2^31, by a multiplier of 33
// bits, ceil(2^(32+l) / d) with l = ceil(log2 d), whose top bit is the n that is added.
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  return {d, static_cast<uint32_t>(((1ull << 32) * ((1ull << l) - d)) / d + 1), l};
}
__device__ __forceinline__ int div_by(int n, const FastDiv& f) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(n), f.mul) + static_cast<uint32_t>(n)) >> f.shift);
}

// Workspace: outputs [2 * CTAs][16][HD], then (maximum, sum) [2 * CTAs][16].
struct AttnRowsParams {
  AttnPackedParams a;
  FastDiv group;  // query heads a key head
  float* part_o;
  float2* part_ml;
};

struct AttnRowsStage {  // what a stage holds
  int q0, rows, row0, off, lk, key0, hk, flags;
};
constexpr int ATTR_FIRST = 1, ATTR_LAST = 2, ATTR_PART = 4, ATTR_ODD = 8;

// Units of a sequence and key head: row tiles and 64-key blocks (one at least, so that rows without
// keys are written too).
__device__ __forceinline__ void rows_shape(const SeqTile& s, int group, long long& nt, int& nb) {
  nt = (static_cast<long long>(s.lq) * group + 15) / 16;
  nb = max(1, (s.lk + 63) / 64);
}

// One warp adds up the units of all sequences, 128 a round (four a lane).  pick(total) names the unit that
// is looked for (< 0 or >= total: none); seq, base: the sequence that holds it (p.n: none) and that one's
// first unit.  Up to 128 sequences are read once, more of them twice.
template <typename F>
__device__ __forceinline__ void rows_scan(const AttnPackedParams& p, int group, F pick, int& seq, long long& base) {
  const int lane = threadIdx.x & 31;
  long long cost[4], sum = 0, incl = 0, total = 0, before = 0;
  auto round = [&](int at) {
    sum = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      cost[u] = 0;
      if (at + lane * 4 + u < p.n) {
        SeqTile s;
        seq_bounds(p, at + lane * 4 + u, s);
        long long nt;
        int nb;
        rows_shape(s, group, nt, nb);
        cost[u] = nt * nb * p.Hkv;
      }
      sum += cost[u];
    }
    incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    return __shfl_sync(0xffffffffu, incl, 31);
  };
  for (int at = 0; at < p.n; at += 128) total += round(at);
  const long long want = pick(total);
  seq = p.n;
  base = 0;
  if (want < 0 || want >= total) return;
  for (int at = 0; at < p.n; at += 128) {
    const long long here = p.n <= 128 ? total : round(at);
    if (want < before + here) {
      const int src = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, want < before + incl))) - 1;
      base = before + __shfl_sync(0xffffffffu, incl - sum, src);
      seq = at + src * 4;
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        const long long c = __shfl_sync(0xffffffffu, cost[u], src);
        if (seq == at + src * 4 + u && want >= base + c) {
          base += c;
          ++seq;
        }
      }
      return;
    }
    before += here;
  }
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Byte offset of 16-byte chunk c (8 values) of row r in a tile of 128-byte rows, `rows` rows a 64-value slab.
__device__ __forceinline__ uint32_t swz(int r, int c, int rows) {
  return static_cast<uint32_t>((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// Two values as a 16-bit pair and the pair of their remainders.
template <typename T>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack2<T>(x, y);
  const T* h = reinterpret_cast<const T*>(&hi);
  lo = pack2<T>(x - to_f32<T>(h[0]), y - to_f32<T>(h[1]));
}
template <typename T, int HD>
__global__ void __launch_bounds__(ATTR_THREADS, AttnRowsCfg<HD>::PER_SM)
    attn_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ AttnRowsParams pr, int* status) {
  using Cfg = AttnRowsCfg<HD>;
  constexpr int STAGES = Cfg::STAGES;
  constexpr int KS = HD / 16;
  const AttnPackedParams& p = pr.a;
  int* gstatus = op_status(status);
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {
    pdl_wait();
    if (threadIdx.x == 0) atomicExch(gstatus, DEV_TIMEOUT_ATTR + 15);
    return;
  }
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);  // [STAGES]
  uint64_t* empty = full + STAGES;
  uint64_t* join = empty + STAGES;  // the consumer warps' meeting point (bounded, unlike a barrier instruction)
  AttnRowsStage* desc = reinterpret_cast<AttnRowsStage*>(smem + Cfg::OFF_BAR + 128);  // [STAGES]
  float2* s_ml0 = reinterpret_cast<float2*>(smem + Cfg::OFF_BAR + 384);               // [2][4][16]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_BAR + 112);
  int* s_count = reinterpret_cast<int*>(smem + Cfg::OFF_BAR + 116);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int group = static_cast<int>(pr.group.d);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 33);
      mbar_init(&empty[s], 4);
    }
    mbar_init(join, 4);
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  pdl_wait();
  if (threadIdx.x == 0) *abort_flag = op_stopped(status) ? 1 : 0;
  long long u = 0, u_end = 0, base = 0, per = 0;
  int seq = 0;
  if (warp == 4) {
    rows_scan(p, group, [&](long long total) {
      per = max(static_cast<long long>(ATTR_MIN_UNITS), (total + gridDim.x - 1) / gridDim.x);
      u = min(total, per * blockIdx.x);
      u_end = min(total, u + per);
      return u;
    }, seq, base);
    if (lane == 0) *s_count = static_cast<int>(min(u_end - u, 0x7fffffffLL));
  }
  pdl_launch_dependents();
  __syncthreads();
  const int count = *abort_flag != 0 ? 0 : *s_count;

  if (warp == 4) {
    // ------------------------------------------------------------------ producer
    if (count > 0) {
      const long long start = u;
      int slot = 0;
      uint32_t ph = 0;
      int issued_parity[STAGES];
#pragma unroll
      for (int s = 0; s < STAGES; ++s) issued_parity[s] = -1;
      bool ok = true;
      SeqTile s;
      long long nt = 0;
      int nb = 1;
      seq_bounds(p, seq, s);
      rows_shape(s, group, nt, nb);
      // the first item of the piece; from there on they are counted up
      const long long item = (u - base) / nb;
      int blk = static_cast<int>(u - base - item * nb);
      int hk = static_cast<int>(item / nt);
      int tile = static_cast<int>(item - hk * nt);
      while (ok && u < u_end) {
        if (hk == p.Hkv) {  // the next sequence that has rows
          hk = 0;
          do seq_bounds(p, ++seq, s);
          while (s.lq == 0 && seq + 1 < p.n);
          rows_shape(s, group, nt, nb);
        }
        const int row0 = tile * 16;
        const int take = static_cast<int>(min(static_cast<long long>(nb - blk), u_end - u));
        const int rows = s.lq * group;
        const int off = s.lk - s.lq;
        const int kend = p.causal ? clampi(div_by(min(row0 + 15, rows - 1), pr.group) + off + 1, 0, s.lk) : s.lk;
        const int part = (blk > 0 || take < nb) ? (ATTR_PART | (u == start ? 0 : ATTR_ODD)) : 0;
        for (int b = 0; b < take; ++b) {
          if (!mbar_wait_warp(&empty[slot], ph ^ 1u, abort_flag, gstatus, DEV_TIMEOUT_ATTR + 1, p.wait_ns)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + slot * Cfg::STAGE;
          if (b == 0) {
            // 16 rows of Q; past the last row the last one again (never written out)
            for (int i = lane; i < 16 * (HD / 8); i += 32) {
              const int r = i / (HD / 8), c = i % (HD / 8);
              const int row = min(row0 + r, rows - 1);
              const int t = div_by(row, pr.group);
              const void* src = static_cast<const T*>(p.q) + static_cast<int64_t>(s.q0 + t) * p.q_tok +
                                static_cast<int64_t>(hk * group + row - t * group) * p.q_head + c * 8;
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(st + 2 * Cfg::K_BYTES) + swz(r, c, 16)),
                           "l"(src)
                           : "memory");
            }
          }
          const int key0 = (blk + b) * 64;
          const bool some = key0 < kend;
          if (lane == 0) {
            AttnRowsStage d;
            d.q0 = s.q0;
            d.rows = rows;
            d.row0 = row0;
            d.off = off;
            d.lk = s.lk;
            d.key0 = key0;
            d.hk = hk;
            d.flags = (b == 0 ? ATTR_FIRST : 0) | (b == take - 1 ? ATTR_LAST : 0) | part;
            desc[slot] = d;
            if (some) {
              mbar_arrive_expect_tx(&full[slot], 2 * Cfg::K_BYTES);
#pragma unroll
              for (int c = 0; c < HD / 64; ++c) tma_load_3d(st + c * 8192, &tmK, c * 64, hk, s.k0 + key0, &full[slot]);
#pragma unroll
              for (int c = 0; c < HD / 64; ++c)
                tma_load_3d(st + Cfg::K_BYTES + c * 8192, &tmV, c * 64, hk, s.k0 + key0, &full[slot]);
            } else {
              mbar_arrive(&full[slot]);
            }
          }
          // each lane's arrival comes once its copies have landed
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&full[slot])) : "memory");
          issued_parity[slot] = static_cast<int>(ph);
          if (++slot == STAGES) {
            slot = 0;
            ph ^= 1u;
          }
        }
        u += take;
        blk = 0;
        if (++tile == nt) {
          tile = 0;
          ++hk;
        }
      }
      if (*abort_flag) {
        for (int i = 0; i < STAGES; ++i)
          if (issued_parity[i] >= 0) mbar_wait_drain(&full[i], static_cast<uint32_t>(issued_parity[i]));
      }
    }
  } else {
    // ------------------------------------------------------------------ consumers: 16 keys of a block each
    const float c = p.scale_log2;
    const int mi = lane >> 3, g = lane >> 2, t4 = lane & 3;
    uint32_t qf[KS][4];
    float o[HD / 8][4];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int slot = 0;
    uint32_t ph = 0, jp = 0;
    int s_flip = 0;  // two sets of s_ml: a warp that is done may begin the next item's
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(join);
      const bool met = mbar_wait_warp(join, jp, abort_flag, gstatus, DEV_TIMEOUT_ATTR + 3, p.wait_ns);
      jp ^= 1u;
      return met;
    };
    for (int i = 0; i < count; ++i) {
      if (!mbar_wait_warp(&full[slot], ph, abort_flag, gstatus, DEV_TIMEOUT_ATTR + 2, p.wait_ns)) break;
      const AttnRowsStage d = desc[slot];
      uint8_t* st = smem + slot * Cfg::STAGE;
      const uint32_t sk = smem_u32(st), sv = sk + Cfg::K_BYTES, sq = sv + Cfg::K_BYTES;
      if (d.flags & ATTR_FIRST) {
#pragma unroll
        for (int k = 0; k < KS; ++k) ldsm4(qf[k], sq + swz((mi & 1) * 8 + (lane & 7), k * 2 + (mi >> 1), 16));
#pragma unroll
        for (int n = 0; n < HD / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
      }
      // keys each of this thread's two rows sees, counted from this warp's first key
      const int key = d.key0 + warp * 16;
      int lim[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = min(d.row0 + g + 8 * r, d.rows - 1);
        lim[r] = (p.causal ? min(d.lk, div_by(row, pr.group) + d.off + 1) : d.lk) - key;
      }
      if (__any_sync(0xffffffffu, lim[1] > 0 || lim[0] > 0)) {
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t b[4];
          ldsm4(b, sk + swz(warp * 16 + (mi >> 1) * 8 + (lane & 7), k * 2 + (mi & 1), 64));
          mma16816<T>(s[0], qf[k], b[0], b[1]);
          mma16816<T>(s[1], qf[k], b[2], b[3]);
        }
        if (d.lk - key < 16) {  // V's rows past the last key
          for (int x = lane; x < (16 - (d.lk - key)) * (HD / 8); x += 32) {
            const int r = warp * 16 + (d.lk - key) + x / (HD / 8);
            *reinterpret_cast<uint4*>(st + Cfg::K_BYTES + swz(r, x % (HD / 8), 64)) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        float alpha[2], mc[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (n * 8 + t4 * 2 + e >= lim[r]) s[n][2 * r + e] = -INFINITY;
          float top = maxn(maxn(s[0][2 * r], s[0][2 * r + 1]), maxn(s[1][2 * r], s[1][2 * r + 1]));
          top = maxn(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = maxn(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const float m_new = maxn(m[r], top);
          alpha[r] = to_max(m[r], m_new, c);
          m[r] = m_new;
          mc[r] = max_offset(m_new, c);
        }
        float pv[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) pv[n][e] = ex2_approx(fmaf(s[n][e], c, -mc[e >> 1]));
#pragma unroll
        for (int r = 0; r < 2; ++r)
          l[r] = l[r] * alpha[r] + ((pv[0][2 * r] + pv[0][2 * r + 1]) + (pv[1][2 * r] + pv[1][2 * r + 1]));
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int n = 0; n < HD / 8; ++n) {
            o[n][0] *= alpha[0];
            o[n][1] *= alpha[0];
            o[n][2] *= alpha[1];
            o[n][3] *= alpha[1];
          }
        }
        uint32_t hi[4], lo[4];
        split2<T>(pv[0][0], pv[0][1], hi[0], lo[0]);
        split2<T>(pv[0][2], pv[0][3], hi[1], lo[1]);
        split2<T>(pv[1][0], pv[1][1], hi[2], lo[2]);
        split2<T>(pv[1][2], pv[1][3], hi[3], lo[3]);
#pragma unroll
        for (int n = 0; n < HD / 16; ++n) {
          uint32_t b[4];
          ldsm4t(b, sv + swz(warp * 16 + (mi & 1) * 8 + (lane & 7), n * 2 + (mi >> 1), 64));
          mma16816<T>(o[2 * n], hi, b[0], b[1]);
          mma16816<T>(o[2 * n + 1], hi, b[2], b[3]);
          mma16816<T>(o[2 * n], lo, b[0], b[1]);
          mma16816<T>(o[2 * n + 1], lo, b[2], b[3]);
        }
      }
      if (d.flags & ATTR_LAST) {
        // join the four warps through the stage's K and V, which all have read by then
        float2* s_ml = s_ml0 + s_flip * 64;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
          l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
          if (t4 == 0) s_ml[warp * 16 + g + 8 * r] = make_float2(m[r], l[r]);
        }
        if (!meet()) break;
        float* so = reinterpret_cast<float*>(st) + warp * 16 * HD;
        float w[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = g + 8 * r;
          const float top = maxn(maxn(s_ml[row].x, s_ml[16 + row].x), maxn(s_ml[32 + row].x, s_ml[48 + row].x));
          w[r] = to_max(m[r], top, c);
        }
#pragma unroll
        for (int n = 0; n < HD / 8; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r)  // chunks of 8 values, permuted by row against bank conflicts
            *reinterpret_cast<float2*>(so + (g + 8 * r) * HD + ((n ^ g) << 3) + t4 * 2) =
                make_float2(o[n][2 * r] * w[r], o[n][2 * r + 1] * w[r]);
        if (!meet()) break;
        const int row = threadIdx.x >> 3;
        const int arow = d.row0 + row;
        if (arow < d.rows) {
          float top = s_ml[row].x, sum = 0.f;
#pragma unroll
          for (int x = 1; x < 4; ++x) top = maxn(top, s_ml[x * 16 + row].x);
#pragma unroll
          for (int x = 0; x < 4; ++x) sum += s_ml[x * 16 + row].y * to_max(s_ml[x * 16 + row].x, top, c);
          const int t = div_by(arow, pr.group);
          const bool sees = (p.causal ? min(d.lk, t + d.off + 1) : d.lk) > 0;
          const float inv = sees ? 1.0f / sum : 0.f;
          T* dst = static_cast<T*>(p.out) + static_cast<int64_t>(d.q0 + t) * p.o_tok +
                   static_cast<int64_t>(d.hk * group + arow - t * group) * p.o_head;
          const int cta_slot = 2 * blockIdx.x + ((d.flags & ATTR_ODD) ? 1 : 0);
          float* po = pr.part_o + (static_cast<int64_t>(cta_slot) * 16 + row) * HD;
#pragma unroll
          for (int ch = threadIdx.x & 7; ch < HD / 8; ch += 8) {
            float v[8];
            const float* src = reinterpret_cast<const float*>(st) + row * HD + ((ch ^ (row & 7)) << 3);
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
              float4 a = *reinterpret_cast<const float4*>(src + e);
#pragma unroll
              for (int x = 1; x < 4; ++x) {
                const float4 b = *reinterpret_cast<const float4*>(src + x * 16 * HD + e);
                a.x += b.x;
                a.y += b.y;
                a.z += b.z;
                a.w += b.w;
              }
              v[e] = a.x;
              v[e + 1] = a.y;
              v[e + 2] = a.z;
              v[e + 3] = a.w;
            }
            if (d.flags & ATTR_PART) {
              *reinterpret_cast<float4*>(po + ch * 8) = make_float4(v[0], v[1], v[2], v[3]);
              *reinterpret_cast<float4*>(po + ch * 8 + 4) = make_float4(v[4], v[5], v[6], v[7]);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = sees ? v[e] * inv : 0.f;
              *reinterpret_cast<uint4*>(dst + ch * 8) =
                  make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
            }
          }
          if ((d.flags & ATTR_PART) && (threadIdx.x & 7) == 0)
            pr.part_ml[static_cast<int64_t>(cta_slot) * 16 + row] = make_float2(top, sum);
        }
        fence_proxy_async_smem();  // the stage was written here; the next write is a copy's
        s_flip ^= 1;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
      if (++slot == STAGES) {
        slot = 0;
        ph ^= 1u;
      }
    }
  }
}

// Joins the partial results of the items that piece boundaries cut.  CTA b looks at the boundary
// between pieces b and b + 1 and takes the item there, if that is the first boundary in it.  Its 16
// warps share the item's rows, and several of them a row's parts: one long sequence leaves few items of
// very many parts (8 items of 37 parts took 20 us with a thread's loop over all parts).
constexpr int ATTJ_WARPS = 16;

template <typename T, int HD>
__global__ void __launch_bounds__(32 * ATTJ_WARPS) attn_join_kernel(const __grid_constant__ AttnRowsParams pr, int pieces,
                                                                    int* status) {
  constexpr int V = HD / 32;  // values a lane
  const AttnPackedParams& p = pr.a;
  __shared__ long long s_at[3];
  __shared__ int s_seq;
  // half of the warps' sums: with no more than this the CTA fits beside two of the kernel ahead
  __shared__ float s_o[ATTJ_WARPS / 2][HD];
  __shared__ float s_l[ATTJ_WARPS / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = static_cast<int>(pr.group.d);
  // the lengths were there before the kernel ahead began: only its results have to be waited for
  if (warp == 0) {
    int seq;
    long long base, per = 0, at = 0;
    rows_scan(p, group, [&](long long total) {
      per = max(static_cast<long long>(ATTR_MIN_UNITS), (total + pieces - 1) / pieces);
      return at = per * (blockIdx.x + 1);
    }, seq, base);
    if (lane == 0) {
      s_seq = seq;
      s_at[0] = at;
      s_at[1] = base;
      s_at[2] = per;
    }
  }
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  if (s_seq >= p.n || op_stopped(status)) return;
  const long long at = s_at[0], base = s_at[1], per = s_at[2];
  SeqTile s;
  long long nt;
  int nb;
  seq_bounds(p, s_seq, s);
  rows_shape(s, group, nt, nb);
  const long long item = (at - base) / nb;
  const long long u0 = base + item * nb;
  if (u0 == at || u0 < at - per) return;  // begins here, or taken at an earlier boundary
  const int c0 = static_cast<int>(u0 / per), c1 = static_cast<int>((u0 + nb - 1) / per);
  const int odd = u0 > c0 * per ? 1 : 0;
  const int hk = static_cast<int>(item / nt);
  const int row0 = static_cast<int>(item - hk * nt) * 16;
  const int nrows = min(16, s.lq * group - row0);
  int share = 1;  // warps a row
  while (share * 2 * nrows <= ATTJ_WARPS) share *= 2;
  const int row = warp / share, part = warp % share;
  const float c = p.scale_log2;
  const bool work = row < nrows;
  auto slot = [&](int x) { return (2 * x + (x == c0 ? odd : 0)) * 16 + row; };
  float v[V], sum = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = 0.f;
  if (work) {
    float top = -INFINITY;
    for (int x = c0 + lane; x <= c1; x += 32) top = maxn(top, pr.part_ml[slot(x)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = maxn(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll 4
    for (int x = c0 + part; x <= c1; x += share) {
      const float2 ml = pr.part_ml[slot(x)];
      const float* src = pr.part_o + static_cast<int64_t>(slot(x)) * HD + lane * V;
      const float w = to_max(ml.x, top, c);
      sum = fmaf(ml.y, w, sum);
      float a[V];
      if constexpr (V == 4) {
        const float4 q = *reinterpret_cast<const float4*>(src);
        a[0] = q.x, a[1] = q.y, a[2] = q.z, a[3] = q.w;
      } else {
        const float2 q = *reinterpret_cast<const float2*>(src);
        a[0] = q.x, a[1] = q.y;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = fmaf(a[e], w, v[e]);
    }
  }
  for (int h = share / 2; h > 0; h /= 2) {  // the upper half of a row's warps hands its sums to the lower
    const int at_s = row * h + (part & (h - 1));
    if (work && part >= h && part < 2 * h) {
#pragma unroll
      for (int e = 0; e < V; ++e) s_o[at_s][lane * V + e] = v[e];
      if (lane == 0) s_l[at_s] = sum;
    }
    __syncthreads();
    if (work && part < h) {
      sum += s_l[at_s];
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] += s_o[at_s][lane * V + e];
    }
    __syncthreads();
  }
  if (!work || part != 0) return;
  const int arow = row0 + row;
  const int t = div_by(arow, pr.group);
  const bool sees = (p.causal ? min(s.lk, t + s.lk - s.lq + 1) : s.lk) > 0;
  const float inv = sees ? 1.0f / sum : 0.f;
  T* dst = static_cast<T*>(p.out) + static_cast<int64_t>(s.q0 + t) * p.o_tok +
           static_cast<int64_t>(hk * group + arow - t * group) * p.o_head + lane * V;
#pragma unroll
  for (int e = 0; e < V; e += 2)
    reinterpret_cast<uint32_t*>(dst)[e / 2] = sees ? pack2<T>(v[e] * inv, v[e + 1] * inv) : 0u;
}

}  // namespace vit
