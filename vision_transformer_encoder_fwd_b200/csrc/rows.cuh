// Root-mean-square norm of rows with the residual's addition, and rows quantised to 8 bits.
//
//   h = x + r                        (r optional; h is stored back in r's type)
//   y = h * w / sqrt(mean(h^2) + eps)
//   out = y                          (rounded to x's type), or
//   s = max(max_j |y_j|, 2^-100) / 448,  out_j = e4m3(y_j / s)   (448: the largest e4m3 value)
// and the same without the norm (y = x) for quantising weights and activations.
//
// The sum of squares, the norm and the largest magnitude are taken from h in fp32, before its
// rounding.  Both reductions run in one exchange: the common factor 1/sqrt(...) is positive, so
// max |y| = max |h w| / sqrt(...).  An 8-bit value comes from four roundings in fp32 (h, h w, 448 / max, their
// product), which put it on the other side of a step less often than the formula taken step by step in fp32
// (8191 rows of 4096, 12 inputs: 18 values a call not those of 64 bits, 28 step by step).
//
// Bound: bytes (x, r in; h, out written), so each row is read once into registers (8 values per
// 16-byte load of a 16-bit type) and stays there.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"

namespace vit {

constexpr float kE4m3Max = 448.0f;
constexpr float kRowAmaxMin = 7.888609052210118e-31f;  // 2^-100: keeps 448 / amax finite

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// N consecutive values as fp32; VEC: 16-byte aligned, N * sizeof(T) a multiple of 16.
template <typename T, int N, bool VEC>
__device__ __forceinline__ void load_f32(const T* p, float (&v)[N]) {
  if constexpr (VEC) {
    constexpr int PER = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < N / PER; ++i) {
      const uint4 w = reinterpret_cast<const uint4*>(p)[i];
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int j = 0; j < PER; ++j) v[i * PER + j] = to_f32<T>(e[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_f32<T>(p[i]);
  }
}

template <typename T, int N, bool VEC>
__device__ __forceinline__ void store_f32(T* p, const float (&v)[N]) {
  if constexpr (VEC) {
    constexpr int PER = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < N / PER; ++i) {
      uint4 w;
      T* e = reinterpret_cast<T*>(&w);
#pragma unroll
      for (int j = 0; j < PER; ++j) e[j] = from_f32<T>(v[i * PER + j]);
      reinterpret_cast<uint4*>(p)[i] = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = from_f32<T>(v[i]);
  }
}

// Two values to e4m3 (nearest even, saturating; NaN stays NaN), the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// The larger of two values, or NaN if one is: a row's largest magnitude keeps a NaN, as its scale does.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// What the values v = h w of a row are multiplied by on their way to 8 bits: rstd / s with s = top rstd / 448, so
// that rstd drops out and only the quotient is rounded.  `amax` is top rstd; below the smallest one the
// scale is that one's.  There, and where 448 / top is past fp32's range, the factor itself need not have a
// number in fp32 (rstd * 448 / 2^-100 from rstd = 6e5 on, which a row of zeros has for eps = 1e-12): v is brought
// to y = v rstd first (`first`, 1 elsewhere), whose factor 448 / amax is at most 448 * 2^100.  rows_kernel
// multiplies by both everywhere (1 % of its time; a loop of its own for such rows spilled registers: 8191 rows of 4096,
// bf16 residual, 53 us against 48), the ring kernel, which its instructions bound, only where it has to.  A NaN
// as amax, which is the scale's, is every value's.
__device__ __forceinline__ float row_factor(float top, float rstd, float amax, float& first) {
  float f = kE4m3Max / top;
  first = 1.0f;
  if (amax <= kRowAmaxMin || f == INFINITY) {
    first = rstd;
    f = kE4m3Max / max_nan(amax, kRowAmaxMin);
  }
  return amax == amax ? f : amax;
}

struct RowsParams {
  const void* x;
  const void* r;   // residual in, or NULL
  void* h;         // residual out (may be r)
  const void* w;   // weight, or NULL: no norm
  void* out;
  float* scales;   // NULL: out has x's type
  int64_t x_ld, r_ld, h_ld, out_ld;
  int64_t rows;
  int D;
  float eps;
  int w_f32;       // weight type: fp32, else x's type
};

// One row per group of `tpr` threads (a power of two, or the whole block); NV vectors of E values
// per thread, vector v of thread t at element (v * tpr + t) * E.
// RMODE: 0 no residual, 1 residual of x's type, 2 fp32 residual.
// SHIFT: rows that begin anywhere, all operands' at the same place modulo 8 elements (rows of odd width behind one
// another): the vectors are those that lie whole in the row, the up to 7 values before them and after them go to
// one thread each.  The weights, which begin elsewhere, come from the L1 cache one by one, and bound it with their
// instructions (us here and by single values: 8191 rows of 4095 with an fp32 residual to 8 bits 70 and 140, of 4097
// with a bf16 one 59 and 152, of 4093 without 46 and 77; 4000 of 12285 with a bf16 one 116 and 407).
// Bounds that leave enough rows on an SM: 8191 rows of 4096, us with 2 / 3 / 4 blocks of 512: residual of x's type 49 /
// 47 / 68, fp32 60 / 65 / 92; rows of 5701 in single values 72 with one block of 1024, 54 with two.
constexpr int rows_threads(int e, int nv, int rmode, bool shift) { return e == 8 && nv < 4 && rmode == 1 && !shift ? 512 : 1024; }
constexpr int rows_blocks(int e, int nv, int rmode, bool shift) {
  return rows_threads(e, nv, rmode, shift) == 512 ? 3 : nv == 8 ? 2 : 1;
}

template <typename TX, int RMODE, bool OUT8, int E, int NV, bool SHIFT = false>
__global__ void __launch_bounds__(rows_threads(E, NV, RMODE, SHIFT), rows_blocks(E, NV, RMODE, SHIFT))
    rows_kernel(RowsParams p, int tpr) {
  using TR = typename std::conditional<RMODE == 2, float, TX>::type;
  constexpr bool VEC = E > 1;
  static_assert(!SHIFT || E == 8, "vectors of 8 values");
  __shared__ float2 part[32];
  const int grp = threadIdx.x / tpr;
  const int t = threadIdx.x - grp * tpr;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + grp;
  pdl_wait();
  pdl_launch_dependents();
  const bool live = row < p.rows;
  const bool norm = p.w != nullptr;
  // the vectors' part of the row, and the value beside it that is this thread's (-1: none)
  const int begin = SHIFT ? min(static_cast<int>(-(row * p.x_ld) & 7), p.D) : 0;
  const int end = SHIFT ? begin + ((p.D - begin) & ~7) : p.D;
  int extra = -1;
  if (SHIFT && live) {
    if (t < begin) extra = t;
    if (t >= 8 && end + t - 8 < p.D) extra = end + t - 8;
  }
  float h[NV][E], g[NV][E];
  float ss = 0.f, top = 0.f, he = 0.f, ge = 0.f;
  if (SHIFT && extra >= 0) {
    he = to_f32<TX>(static_cast<const TX*>(p.x)[row * p.x_ld + extra]);
    if (RMODE != 0) he += to_f32<TR>(static_cast<const TR*>(p.r)[row * p.r_ld + extra]);
    if (norm) ge = p.w_f32 ? static_cast<const float*>(p.w)[extra] : to_f32<TX>(static_cast<const TX*>(p.w)[extra]);
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = begin + (v * tpr + t) * E;
    if (live && c < end) {
      load_f32<TX, E, VEC>(static_cast<const TX*>(p.x) + row * p.x_ld + c, h[v]);
      if (RMODE != 0) {
        float r[E];
        load_f32<TR, E, VEC>(static_cast<const TR*>(p.r) + row * p.r_ld + c, r);
#pragma unroll
        for (int i = 0; i < E; ++i) h[v][i] += r[i];
      }
      if (norm) {
        if (p.w_f32)
          load_f32<float, E, VEC && !SHIFT>(static_cast<const float*>(p.w) + c, g[v]);
        else
          load_f32<TX, E, VEC && !SHIFT>(static_cast<const TX*>(p.w) + c, g[v]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) h[v][i] = g[v][i] = 0.f;
    }
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = begin + (v * tpr + t) * E;
    if (RMODE != 0 && live && c < end)
      store_f32<TR, E, VEC>(static_cast<TR*>(p.h) + row * p.h_ld + c, h[v]);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      ss = fmaf(h[v][i], h[v][i], ss);
      if (norm) h[v][i] *= g[v][i];
      if (OUT8) top = max_nan(top, fabsf(h[v][i]));
    }
  }
  if (SHIFT) {
    if (RMODE != 0 && extra >= 0) static_cast<TR*>(p.h)[row * p.h_ld + extra] = from_f32<TR>(he);
    ss = fmaf(he, he, ss);
    if (norm) he *= ge;
    if (OUT8) top = max_nan(top, fabsf(he));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o < tpr) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (OUT8) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
  }
  if (tpr > 32) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) part[warp] = make_float2(ss, top);
    __syncthreads();
    const int w0 = grp * (tpr >> 5);
    ss = 0.f;
    top = 0.f;
    for (int i = 0; i < (tpr >> 5); ++i) {
      const float2 q = part[w0 + i];
      ss += q.x;
      top = max_nan(top, q.y);
    }
  }
  if (!live) return;
  const float rstd = norm ? rsqrtf(ss / static_cast<float>(p.D) + p.eps) : 1.0f;
  float mul = rstd, first = 1.0f;
  if (OUT8) {
    const float amax = top * rstd;
    mul = row_factor(top, rstd, amax, first);
    if (t == 0) p.scales[row] = max_nan(amax, kRowAmaxMin) / kE4m3Max;
  }
  if (SHIFT && extra >= 0) {
    if (OUT8)
      static_cast<uint8_t*>(p.out)[row * p.out_ld + extra] = static_cast<uint8_t>(e4m3x2(he * first * mul, 0.f));
    else
      static_cast<TX*>(p.out)[row * p.out_ld + extra] = from_f32<TX>(he * mul);
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = begin + (v * tpr + t) * E;
    if (c >= end) continue;
#pragma unroll
    for (int i = 0; i < E; ++i) h[v][i] = OUT8 ? h[v][i] * first * mul : h[v][i] * mul;
    if (OUT8) {
      uint8_t* o = static_cast<uint8_t*>(p.out) + row * p.out_ld + c;
      if constexpr (E == 8) {
        *reinterpret_cast<uint2*>(o) = make_uint2(e4m3x2(h[v][0], h[v][1]) | e4m3x2(h[v][2], h[v][3]) << 16,
                                                  e4m3x2(h[v][4], h[v][5]) | e4m3x2(h[v][6], h[v][7]) << 16);
      } else {
        for (int i = 0; i < E; ++i) o[i] = static_cast<uint8_t>(e4m3x2(h[v][i], 0.f));
      }
    } else {
      store_f32<TX, E, VEC>(static_cast<TX*>(p.out) + row * p.out_ld + c, h[v]);
    }
  }
}

// The same without a residual for many rows of a 16-bit type: a block (a warp, where a row fits one) takes rows
// r, r + stride, ... and copies STAGES - 1 rows ahead of the one it works on into shared memory, each
// thread the pieces that it will read itself, so that no barrier stands between a copy and its use.
// The register kernel has nothing in flight while a row is summed up and written.  8191 rows of 4096 from
// bf16 to 8 bits: 23 us against 36 (4.4 TB/s); with a residual the ring's shared memory leaves too few
// warps on an SM, and it was slower (fp32 residual 88 us against 60).
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
template <typename TX, bool OUT8, int NV, int STAGES>
__global__ void __launch_bounds__(512) rows_stream_kernel(RowsParams p, int tpr) {
  extern __shared__ uint4 ring[];  // [STAGES][NV][threads], 8 values each
  __shared__ float2 part[2][32];
  const int threads = blockDim.x;
  const int grp = threadIdx.x / tpr;
  const int t = threadIdx.x - grp * tpr;
  const int groups = threads / tpr;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * groups;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + grp;
  const bool norm = p.w != nullptr;
  pdl_wait();
  pdl_launch_dependents();
  auto slot = [&](int stage, int v) { return ring + (stage * NV + v) * threads + threadIdx.x; };
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.rows) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * tpr + t) * 8;
        if (c < p.D) cp_async16(slot(stage, v), static_cast<const TX*>(p.x) + row * p.x_ld + c);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(first + s * stride, s);
  int stage = 0, flip = 0;
  for (int64_t row = first; row < p.rows; row += stride) {
    int ahead = stage + STAGES - 1;
    if (ahead >= STAGES) ahead -= STAGES;
    fetch(row + (STAGES - 1) * stride, ahead);
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
    float h[NV][8];
    float ss = 0.f, top = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * tpr + t) * 8;
      if (c < p.D) {
        const uint4 w8 = *slot(stage, v);
        const TX* e8 = reinterpret_cast<const TX*>(&w8);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] = to_f32<TX>(e8[i]);
        if (norm) {
          float g[8];
          if (p.w_f32)
            load_f32<float, 8, true>(static_cast<const float*>(p.w) + c, g);
          else
            load_f32<TX, 8, true>(static_cast<const TX*>(p.w) + c, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = fmaf(h[v][i], h[v][i], ss);
            h[v][i] *= g[i];
          }
        }
        if (OUT8) {
#pragma unroll
          for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(h[v][i]));
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (OUT8) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (tpr > 32) {  // one barrier a row: the two sets of parts take turns
      if ((threadIdx.x & 31) == 0) part[flip][threadIdx.x >> 5] = make_float2(ss, top);
      __syncthreads();
      ss = 0.f;
      top = 0.f;
      for (int i = 0; i < (tpr >> 5); ++i) {
        const float2 q = part[flip][i];
        ss += q.x;
        top = max_nan(top, q.y);
      }
      flip ^= 1;
    }
    const float rstd = norm ? rsqrtf(ss / static_cast<float>(p.D) + p.eps) : 1.0f;
    float mul = rstd;
    if (OUT8) {
      const float amax = top * rstd;
      float first;
      mul = row_factor(top, rstd, amax, first);
      if (first != 1.0f) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int i = 0; i < 8; ++i) h[v][i] *= first;
      }
      if (t == 0) p.scales[row] = max_nan(amax, kRowAmaxMin) / kE4m3Max;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * tpr + t) * 8;
      if (c >= p.D) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] *= mul;
      if (OUT8)
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + row * p.out_ld + c) =
            make_uint2(e4m3x2(h[v][0], h[v][1]) | e4m3x2(h[v][2], h[v][3]) << 16,
                       e4m3x2(h[v][4], h[v][5]) | e4m3x2(h[v][6], h[v][7]) << 16);
      else
        store_f32<TX, 8, true>(static_cast<TX*>(p.out) + row * p.out_ld + c, h[v]);
    }
    if (++stage == STAGES) stage = 0;
  }
}

}  // namespace vit
