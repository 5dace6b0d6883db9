// Rotary positions: each pair (a, b) of a head's first `rd` values is turned by the angle
// t = position * frequency, (a cos t - b sin t, a sin t + b cos t); the rest of the head is copied.
//
// The angle never exists as a floating number.  The host turns a frequency f (radians per position)
// into the 64-bit fixed-point fraction of a turn F = round(2^64 frac(f / 2 pi)); position * F
// modulo 2^64 is then the exact fraction of a turn at any 64-bit position, with whole turns gone
// by the wrap of unsigned multiplication, and only its top 32 bits go to sincospif (off by at most
// 2^-33 turn, plus 2^-25 of the result by the conversion to fp32).
//
// Bound: bytes (q and k in and out).  A block takes a few tokens; its threads first compute the
// tokens' cosines and sines once into shared memory, then each thread keeps those of its pairs
// in registers and walks the heads with 16-byte loads and stores.
#pragma once

#include "rows.cuh"

namespace vit {

constexpr int ROPE_MAX_PAIRS = 128;  // rd <= 256
constexpr int ROPE_THREADS = 256;

struct RopeParams {
  const void* in[2];   // q, k
  void* out[2];
  int64_t in_tok[2], in_head[2], out_tok[2], out_head[2];  // strides in elements
  int heads[2];
  const void* pos;     // [axes, T]
  int64_t T;
  int d, rd, axes;
  int pos64;           // positions are int64, else int32
  int tokens;          // tokens per block
  float sign;          // -1: the inverse rotation
  float gain;          // factor on cosine and sine
  unsigned long long turn[ROPE_MAX_PAIRS];
};

// HALF: pair i is (i, i + rd/2), else (2 i, 2 i + 1).  E values per access (1: any alignment).
template <typename T, bool HALF, int E>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ float2 cs[];  // [tokens][n]
  constexpr bool VEC = E > 1;
  const int n = p.rd >> 1;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int ntok = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.T - tok0));
  pdl_wait();
  pdl_launch_dependents();
  const int per_axis = n / p.axes;
  for (int i = threadIdx.x; i < ntok * n; i += ROPE_THREADS) {
    const int tk = i / n;
    const int j = i - tk * n;
    const int64_t at = static_cast<int64_t>(j / per_axis) * p.T + tok0 + tk;
    const long long pos = p.pos64 ? static_cast<const long long*>(p.pos)[at] : static_cast<const int*>(p.pos)[at];
    const unsigned long long ph = static_cast<unsigned long long>(pos) * p.turn[j];
    // the top 32 bits as a signed fraction of a turn in [-1/2, 1/2), times 2 (sincospi's half turns)
    const float half_turns = static_cast<float>(static_cast<int>(ph >> 32)) * 4.656612873077393e-10f;
    float s, c;
    sincospif(half_turns, &s, &c);
    cs[i] = make_float2(c * p.gain, s * p.gain * p.sign);
  }
  __syncthreads();
  // a chunk is one thread's share of a head: E pairs (HALF), or E values (E = 1: one pair), or E
  // values behind the rotated part
  constexpr int PAIRS = HALF ? E : (VEC ? E / 2 : 1);
  const int rot = n / PAIRS;
  const int tail = (p.d - p.rd) / E;
  const int chunks = rot + tail;
  const int lanes = max(1, min(p.heads[0] + p.heads[1], ROPE_THREADS / max(1, chunks * ntok)));
  const int total = ntok * lanes * chunks;
  for (int i = threadIdx.x; i < total; i += ROPE_THREADS) {
    const int ch = i % chunks;
    const int hl = (i / chunks) % lanes;
    const int tk = i / (chunks * lanes);
    const int64_t tok = tok0 + tk;
    float2 w[PAIRS];
    if (ch < rot) {
#pragma unroll
      for (int u = 0; u < PAIRS; ++u) w[u] = cs[tk * n + ch * PAIRS + u];
    }
    for (int h = hl; h < p.heads[0] + p.heads[1]; h += lanes) {
      const int x = h < p.heads[0] ? 0 : 1;
      const int hh = h - (x ? p.heads[0] : 0);
      const T* src = static_cast<const T*>(p.in[x]) + tok * p.in_tok[x] + hh * p.in_head[x];
      T* dst = static_cast<T*>(p.out[x]) + tok * p.out_tok[x] + hh * p.out_head[x];
      if (ch >= rot) {
        const int c = p.rd + (ch - rot) * E;
        float v[E];
        load_f32<T, E, VEC>(src + c, v);
        store_f32<T, E, VEC>(dst + c, v);
      } else if (HALF) {
        float a[PAIRS], b[PAIRS], ra[PAIRS], rb[PAIRS];
        load_f32<T, PAIRS, VEC>(src + ch * PAIRS, a);
        load_f32<T, PAIRS, VEC>(src + n + ch * PAIRS, b);
#pragma unroll
        for (int u = 0; u < PAIRS; ++u) {
          ra[u] = a[u] * w[u].x - b[u] * w[u].y;
          rb[u] = a[u] * w[u].y + b[u] * w[u].x;
        }
        store_f32<T, PAIRS, VEC>(dst + ch * PAIRS, ra);
        store_f32<T, PAIRS, VEC>(dst + n + ch * PAIRS, rb);
      } else {
        float a[2 * PAIRS], r[2 * PAIRS];
        load_f32<T, 2 * PAIRS, VEC>(src + ch * 2 * PAIRS, a);
#pragma unroll
        for (int u = 0; u < PAIRS; ++u) {
          r[2 * u] = a[2 * u] * w[u].x - a[2 * u + 1] * w[u].y;
          r[2 * u + 1] = a[2 * u] * w[u].y + a[2 * u + 1] * w[u].x;
        }
        store_f32<T, 2 * PAIRS, VEC>(dst + ch * 2 * PAIRS, r);
      }
    }
  }
}

}  // namespace vit
