// Rotary positions: each pair (a, b) of a head's first `rd` values is turned by the angle
// t = position * frequency, (a cos t - b sin t, a sin t + b cos t); the rest of the head is copied.
//
// The angle never exists as a floating number.  The host turns a frequency f (radians per position)
// into the 64-bit fixed-point fraction of a turn F = 2^64 frac(f / 2 pi), off by at most 1 unit for frequencies up
// to 1 and 3 up to 2 pi (f / 2 pi in the 64 bits of long double, then rounded).  position * F modulo 2^64 is the
// fraction of a turn: whole turns are gone by the wrap of unsigned multiplication, and F's error counts
// position times (|position| 2^-64 turns: 2^-33 at 2^31, 2^-24 at 2^40).  Rounded to 32 bits, off by at most
// 2^-33 turn more, it goes to sincospif (by the conversion to fp32 2^-25 of it).
//
// Bound: bytes (q and k in and out).  A block takes a few tokens; its threads first compute the
// tokens' cosines and sines once into shared memory, then each thread keeps those of its pairs
// in registers and walks the heads with 16-byte accesses (8-byte ones or single values where
// the layout asks for them), several heads' loads ahead of their use and the first of them ahead of the
// sines.  16383 tokens of 40 heads of 128 in 16 bits, half of each head turned in interleaved pairs: 57 us
// call by call (5.8 TB/s), 55 replayed from a graph, all of it in halves 56; with one access in flight 86 and 96 us.
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

template <int BYTES>
struct RawOf;
template <>
struct RawOf<16> {
  using type = uint4;
};
template <>
struct RawOf<8> {
  using type = uint2;
};
template <>
struct RawOf<4> {
  using type = uint32_t;
};
template <>
struct RawOf<2> {
  using type = uint16_t;
};

// HALF: pair i is (i, i + rd/2), else (2 i, 2 i + 1).  E: values an access.  A chunk is one thread's share
// of a head: two accesses E pairs apart by rd/2 (HALF), one of E values (E / 2 pairs), or one of E values
// behind the turned part.  Interleaved single values (E = 1) take a pair as two accesses side by side.
template <typename T, bool HALF, int E>
__global__ void __launch_bounds__(ROPE_THREADS, (HALF || E == 1) ? 4 : 5) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ float2 cs[];  // [tokens][n]
  using Raw = typename RawOf<E * sizeof(T)>::type;
  constexpr bool TWO = HALF || E == 1;            // a chunk has two accesses
  constexpr int PAIRS = TWO ? E : E / 2;          // pairs a chunk
  constexpr int U = TWO ? 3 : 5;                  // heads in flight a thread
  const int n = p.rd >> 1;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int ntok = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.T - tok0));
  pdl_wait();
  pdl_launch_dependents();
  const int rot = n / PAIRS;
  const int chunks = rot + (p.d - p.rd) / E;
  const int heads = p.heads[0] + p.heads[1];
  const int lanes = max(1, min(heads, ROPE_THREADS / max(1, chunks * ntok)));
  const int total = ntok * lanes * chunks;
  const int second = HALF ? n : 1;  // from a chunk's first access to its second
  // the chunk a thread works on: place, token, first head
  int ch, tk, hl;
  bool turn;
  int64_t tok, at;
  auto take = [&](int i) {
    ch = i % chunks;
    hl = (i / chunks) % lanes;
    tk = i / (chunks * lanes);
    turn = ch < rot;
    tok = tok0 + tk;
    at = turn ? (HALF ? ch * E : ch * 2 * PAIRS) : p.rd + (ch - rot) * E;
  };
  Raw a[U], b[U];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int hu = h + u * lanes;
      if (hu < heads) {
        const int x = hu < p.heads[0] ? 0 : 1;
        const T* s = static_cast<const T*>(p.in[x]) + tok * p.in_tok[x] + at +
                     static_cast<int64_t>(hu - (x ? p.heads[0] : 0)) * p.in_head[x];
        a[u] = *reinterpret_cast<const Raw*>(s);
        if (TWO && turn) b[u] = *reinterpret_cast<const Raw*>(s + second);
      }
    }
  };
  // the first values are on their way while the sines are computed
  bool ahead = static_cast<int>(threadIdx.x) < total;
  if (ahead) {
    take(threadIdx.x);
    load(hl);
  }
  const int per_axis = n / p.axes;
  for (int i = threadIdx.x; i < ntok * n; i += ROPE_THREADS) {
    const int t = i / n;
    const int j = i - t * n;
    const int64_t from = static_cast<int64_t>(j / per_axis) * p.T + tok0 + t;
    const long long pos = p.pos64 ? static_cast<const long long*>(p.pos)[from] : static_cast<const int*>(p.pos)[from];
    const unsigned long long ph = static_cast<unsigned long long>(pos) * p.turn[j];
    // rounded to 32 bits, as a signed fraction of a turn in [-1/2, 1/2), times 2 (sincospi's half turns)
    const float half_turns = static_cast<float>(static_cast<int>((ph + 0x80000000ull) >> 32)) * 4.656612873077393e-10f;
    float s, c;
    sincospif(half_turns, &s, &c);
    cs[i] = make_float2(c * p.gain, s * p.gain * p.sign);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += ROPE_THREADS) {
    if (!ahead) take(i);
    float2 w[PAIRS];
#pragma unroll
    for (int u = 0; u < PAIRS; ++u) w[u] = turn ? cs[tk * n + ch * PAIRS + u] : make_float2(1.f, 0.f);
    for (int h = hl; h < heads; h += lanes * U) {
      if (!ahead) load(h);
      ahead = false;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int hu = h + u * lanes;
        if (hu < heads) {
          const int x = hu < p.heads[0] ? 0 : 1;
          T* o = static_cast<T*>(p.out[x]) + tok * p.out_tok[x] + at +
                 static_cast<int64_t>(hu - (x ? p.heads[0] : 0)) * p.out_head[x];
          if (turn) {
            T* va = reinterpret_cast<T*>(&a[u]);
            T* vb = reinterpret_cast<T*>(&b[u]);
#pragma unroll
            for (int v = 0; v < PAIRS; ++v) {
              T& e0 = TWO ? va[v] : va[2 * v];
              T& e1 = TWO ? vb[v] : va[2 * v + 1];
              const float f0 = to_f32<T>(e0), f1 = to_f32<T>(e1);
              e0 = from_f32<T>(f0 * w[v].x - f1 * w[v].y);
              e1 = from_f32<T>(f0 * w[v].y + f1 * w[v].x);
            }
            if (TWO) *reinterpret_cast<Raw*>(o + second) = b[u];
          }
          *reinterpret_cast<Raw*>(o) = a[u];
        }
      }
    }
  }
}

}  // namespace vit
