// Attention over packed sequences for few query rows and few keys per sequence (short prompts, the first new
// tokens): the same mathematics and arguments as attn_packed_kernel, one warp per tile of 16 rows and
// key head (rows: query t, head g of the group, row t * group + g), no shared memory at all.
//
// Such work is bound by latency: a warp's keys are few, so that rings, barriers and joins cost more than the
// loads.  A warp reads K and V from global memory straight into mma.sync fragments, 16 bytes a lane:
//   - in S = Q K^T the order of the width's values is free as long as both sides share it, so the 16 bytes of
//     chunk t of a key's 64 values serve as they are as the fragments of two MMAs;
//   - in O = P V the order of the output's columns is free: lane (g, t) reads 8 values from 8 g on of keys 2 t
//     and 2 t + 1, and column g of the j-th 8-column product is value 8 g + j, which leaves each lane
//     with 16 neighbouring values of the result.
// Keys past the last one are read as the last one and masked, so nothing outside a sequence is touched.
// P is kept as a pair of 16-bit numbers, as in attn_rows_kernel.
// Measured: 150 causal prompts of 5 to 24 tokens, 16 heads of 64, 9 us; 64 tokens over 32 keys, 32 heads on 8
// of 128, 5.3 us.
#pragma once

#include "attention_rows.cuh"

namespace vit {

constexpr int ATTS_WARPS = 4;

struct AttnShortParams {
  AttnPackedParams a;
  FastDiv group;
};

__device__ __forceinline__ uint4 ld_g16(const void* p) { return *reinterpret_cast<const uint4*>(p); }

template <typename T, int HD>
__global__ void __launch_bounds__(32 * ATTS_WARPS, HD == 64 ? 4 : 2)
    attn_short_kernel(const __grid_constant__ AttnShortParams pr, int* status) {
  constexpr int NC = HD / 64;  // 64-value slabs of the width
  const AttnPackedParams& p = pr.a;
  const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int hk = blockIdx.y;
  const int group = static_cast<int>(pr.group.d);
  pdl_wait();
  pdl_launch_dependents();
  if (op_stopped(status)) return;
  const SeqTile st = find_tile(p, static_cast<int>(blockIdx.x) * ATTS_WARPS + static_cast<int>(threadIdx.x >> 5), 16, group);
  if (st.seq < 0) return;
  const int rows = st.lq * group;
  const int row0 = st.tile * 16;
  const int off = st.lk - st.lq;
  const float c = p.scale_log2;

  // this lane's two rows; past the last one the last one again (never written out)
  int tq[2], hq[2], lim[2];
  uint4 q[2][2 * NC];  // chunks t and t + 4 of each slab
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = min(row0 + g + 8 * r, rows - 1);
    tq[r] = div_by(row, pr.group);
    hq[r] = hk * group + row - tq[r] * group;
    lim[r] = p.causal ? min(st.lk, tq[r] + off + 1) : st.lk;
    const T* src = static_cast<const T*>(p.q) + static_cast<int64_t>(st.q0 + tq[r]) * p.q_tok + hq[r] * p.q_head;
#pragma unroll
    for (int x = 0; x < 2 * NC; ++x) q[r][x] = ld_g16(src + (x * 4 + t4) * 8);
  }
  const int last = min(row0 + 15, rows - 1);
  const int kend = p.causal ? clampi(div_by(last, pr.group) + off + 1, 0, st.lk) : st.lk;
  const T* kb = static_cast<const T*>(p.k) + static_cast<int64_t>(st.k0) * p.k_tok + hk * p.k_head + t4 * 8;
  const T* vb = static_cast<const T*>(p.v) + static_cast<int64_t>(st.k0) * p.v_tok + hk * p.v_head + g * 8;

  float o[HD / 8][4];
#pragma unroll
  for (int n = 0; n < HD / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  uint4 kf[2][2 * NC], vf[4][NC];
  auto load_k = [&](int key0) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const T* src = kb + static_cast<int64_t>(min(key0 + n * 8 + g, st.lk - 1)) * p.k_tok;
#pragma unroll
      for (int x = 0; x < 2 * NC; ++x) kf[n][x] = ld_g16(src + x * 32);
    }
  };
  auto load_v = [&](int key0) {
#pragma unroll
    for (int y = 0; y < 4; ++y) {  // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
      const T* src = vb + static_cast<int64_t>(min(key0 + t4 * 2 + (y & 1) + (y >> 1) * 8, st.lk - 1)) * p.v_tok;
#pragma unroll
      for (int x = 0; x < NC; ++x) vf[y][x] = ld_g16(src + x * 64);
    }
  };
  if (kend > 0) {
    load_k(0);
    load_v(0);
  }
  for (int key0 = 0; key0 < kend; key0 += 16) {
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int x = 0; x < 2 * NC; ++x) {
        const uint32_t a0[4] = {q[0][x].x, q[1][x].x, q[0][x].y, q[1][x].y};
        const uint32_t a1[4] = {q[0][x].z, q[1][x].z, q[0][x].w, q[1][x].w};
        mma16816<T>(s[n], a0, kf[n][x].x, kf[n][x].y);
        mma16816<T>(s[n], a1, kf[n][x].z, kf[n][x].w);
      }
    if (key0 + 16 < kend) load_k(key0 + 16);
    float alpha[2], mc[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (key0 + n * 8 + t4 * 2 + e >= lim[r]) s[n][2 * r + e] = -INFINITY;
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
#pragma unroll
    for (int n = 0; n < HD / 8; ++n) {
      o[n][0] *= alpha[0];
      o[n][1] *= alpha[0];
      o[n][2] *= alpha[1];
      o[n][3] *= alpha[1];
    }
    uint32_t hi[4], lo[4];
    split2<T>(pv[0][0], pv[0][1], hi[0], lo[0]);
    split2<T>(pv[0][2], pv[0][3], hi[1], lo[1]);
    split2<T>(pv[1][0], pv[1][1], hi[2], lo[2]);
    split2<T>(pv[1][2], pv[1][3], hi[3], lo[3]);
#pragma unroll
    for (int x = 0; x < NC; ++x) {
      const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&vf[0][x]);
      const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&vf[1][x]);
      const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&vf[2][x]);
      const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&vf[3][x]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;  // the j-th 16-bit value of two rows side by side
        const uint32_t b0 = __byte_perm(v0[j >> 1], v1[j >> 1], sel), b1 = __byte_perm(v2[j >> 1], v3[j >> 1], sel);
        mma16816<T>(o[x * 8 + j], hi, b0, b1);
        mma16816<T>(o[x * 8 + j], lo, b0, b1);
      }
    }
    if (key0 + 16 < kend) load_v(key0 + 16);
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    if (row0 + g + 8 * r >= rows) continue;
    const bool sees = lim[r] > 0;
    const float inv = sees ? 1.0f / l[r] : 0.f;
    T* dst = static_cast<T*>(p.out) + static_cast<int64_t>(st.q0 + tq[r]) * p.o_tok + hq[r] * p.o_head;
    // columns 2 t and 2 t + 1 of product j: values 16 t + j and 16 t + 8 + j of the slab
#pragma unroll
    for (int x = 0; x < NC; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 8; j += 2)
          w[j >> 1] = sees ? pack2<T>(o[x * 8 + j][2 * r + e] * inv, o[x * 8 + j + 1][2 * r + e] * inv) : 0u;
        *reinterpret_cast<uint4*>(dst + x * 64 + t4 * 16 + e * 8) = make_uint4(w[0], w[1], w[2], w[3]);
      }
  }
}

}  // namespace vit
