// Host side of the operator entry points in include/vit_ops.h: checks, tensor maps, launches.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/vit_ops.h"
#include "attention_packed.cuh"
#include "attention_rows.cuh"
#include "attention_short.cuh"
#include "host_common.cuh"
#include "linear_fp8.cuh"
#include "rope.cuh"
#include "rows.cuh"

using namespace vit;

namespace {

vit_status fail(vit_status st, const char* msg) {
  set_err("%s", msg);
  return st;
}

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

size_t type_size(int t) { return t == VIT_DT_F32 ? 4 : (t == VIT_DT_E4M3 ? 1 : 2); }

bool real_type(int t) { return t == VIT_DT_BF16 || t == VIT_DT_F16 || t == VIT_DT_F32; }

// Whether vectors of `width` values at i * si + j * sj, 0 <= i < ni, 0 <= j < nj, share a value.
bool overlap_itself(int64_t ni, int64_t si, int64_t nj, int64_t sj, int64_t width) {
  si = std::abs(si);
  sj = std::abs(sj);
  if ((ni > 1 && si < width) || (nj > 1 && sj < width)) return true;
  if (ni <= 1 || nj <= 1) return false;
  const __int128 wi = si, wj = sj;
  if (wi >= (nj - 1) * wj + width || wj >= (ni - 1) * wi + width) return false;  // one inside the other
  // interleaved: for each distance along the shorter axis the nearest ones along the other
  if (ni > nj) {
    std::swap(ni, nj);
    std::swap(si, sj);
  }
  for (int64_t i = 1; i < ni; ++i) {
    const int64_t j = i * si / sj;
    if ((j < nj && i * si - j * sj < width) || (j + 1 < nj && (j + 1) * sj - i * si < width)) return true;
  }
  return false;
}

int current_sms() {
  int dev = 0;
  cudaGetDevice(&dev);
  return device_sms(dev);
}

// ------------------------------------------------------------------ rows
// How rows may be accessed: by vectors from their first value on, by vectors of the buffers that begin at the same
// place in each, or by single values.
enum RowAccess { ROWS_SINGLE, ROWS_SHIFT, ROWS_VEC };
// Layout of a row over threads: E values per access, NV accesses per thread, tpr threads a row.
template <typename TX, int RMODE, bool OUT8>
cudaError_t launch_rows(const RowsParams& p, RowAccess access, cudaStream_t s) {
  const bool vec = access == ROWS_VEC;
  auto go = [&](auto kernel, int tpr) {
    const int block = tpr >= 128 ? tpr : 128;
    const int64_t per = block / tpr;
    return launch_pdl(kernel, dim3(static_cast<unsigned>((p.rows + per - 1) / per)), dim3(block), 0, s, p, tpr);
  };
  auto whole_warps = [](int threads) { return std::min(1024, std::max(32, (threads + 31) / 32 * 32)); };
  // several rows share a block only at 32 threads a row; the vectors of rows that begin anywhere are D / 8 at most
  const int width = access == ROWS_SHIFT ? p.D & ~7 : p.D;
  auto tpr_of = [&](int per_thread) {
    const int t = whole_warps((width + per_thread - 1) / per_thread);
    return t > 32 && t < 128 ? 128 : t;
  };
  // Many rows without a residual go through the ring kernel: from one row a block on it has nothing to gain.  A
  // thread takes 32 values where there are as many, since a row costs it about 100 instructions whatever
  // its share (16 values: 25 us where 32 take 23).
  if constexpr (RMODE == 0 && sizeof(TX) == 2) {
    auto ring = [&](auto nv, int tpr, bool& taken) {
      constexpr int NV = decltype(nv)::value, STAGES = 4;
      const int block = tpr == 32 ? 128 : tpr;  // several rows share a block only where a warp has one
      const int block_rows = block / tpr;
      const int smem = STAGES * NV * block * 16;
      const int64_t at_once = static_cast<int64_t>(std::min(768 / block, 226 * 1024 / (smem + 2048))) * current_sms();
      taken = (p.rows + block_rows - 1) / block_rows > at_once;
      if (!taken) return cudaSuccess;
      static std::atomic<uint64_t> done{0};
      auto kernel = rows_stream_kernel<TX, OUT8, NV, STAGES>;
      cudaError_t e = set_smem_attr_once(kernel, 128 * 1024, done);
      if (e != cudaSuccess) return e;
      return launch_pdl(kernel, dim3(static_cast<unsigned>(at_once)), dim3(block), smem, s, p, tpr);
    };
    if (vec && p.D <= 16384) {
      bool taken = false;
      cudaError_t e;
      if (p.D <= 256)
        e = ring(std::integral_constant<int, 1>{}, 32, taken);
      else if (p.D <= 512)
        e = ring(std::integral_constant<int, 2>{}, 32, taken);
      else
        e = ring(std::integral_constant<int, 4>{},
                 p.D <= 1024 ? 32 : p.D <= 2048 ? 64 : std::max(128, whole_warps((p.D + 31) / 32)), taken);
      if (taken) return e;
    }
  }
  if (vec) {
    // 8 values a thread where that fills 128 threads (16384 rows of 1024: 24-26 us, 28-29 with 16)
    if (p.D <= 256) return go(rows_kernel<TX, RMODE, OUT8, 8, 1>, 32);
    if (p.D <= 512) return go(rows_kernel<TX, RMODE, OUT8, 8, 2>, 32);
    if (p.D <= 2048) return go(rows_kernel<TX, RMODE, OUT8, 8, 1>, tpr_of(8));
    if (p.D <= 8192) return go(rows_kernel<TX, RMODE, OUT8, 8, 2>, tpr_of(16));
    return go(rows_kernel<TX, RMODE, OUT8, 8, 4>, tpr_of(32));
  }
  if (access == ROWS_SHIFT) {
    if (width <= 256) return go(rows_kernel<TX, RMODE, OUT8, 8, 1, true>, 32);
    if (width <= 512) return go(rows_kernel<TX, RMODE, OUT8, 8, 2, true>, 32);
    if (width <= 2048) return go(rows_kernel<TX, RMODE, OUT8, 8, 1, true>, tpr_of(8));
    // 32 values a thread spill (4000 rows of 12285, fp32 residual: 147 us, 129 with 16)
    if (width <= 16384) return go(rows_kernel<TX, RMODE, OUT8, 8, 2, true>, tpr_of(16));
    return go(rows_kernel<TX, RMODE, OUT8, 8, 4, true>, tpr_of(32));
  }
  if (p.D <= 8192) return go(rows_kernel<TX, RMODE, OUT8, 1, 8>, tpr_of(8));
  return go(rows_kernel<TX, RMODE, OUT8, 1, 32>, tpr_of(32));
}

template <typename TX>
cudaError_t launch_rows_t(const RowsParams& p, int rmode, RowAccess access, cudaStream_t s) {
  const bool out8 = p.scales != nullptr;
  if (rmode == 0) return out8 ? launch_rows<TX, 0, true>(p, access, s) : launch_rows<TX, 0, false>(p, access, s);
  if (rmode == 1) return out8 ? launch_rows<TX, 1, true>(p, access, s) : launch_rows<TX, 1, false>(p, access, s);
  return out8 ? launch_rows<TX, 2, true>(p, access, s) : launch_rows<TX, 2, false>(p, access, s);
}

vit_status run_rows(const RowsParams& p, int x_type, int r_type, int w_type, cudaStream_t s) {
  const size_t xs = type_size(x_type);
  const size_t os = p.scales != nullptr ? 1 : xs;
  if (p.D < 1 || p.D > 32768 || p.rows < 0) return fail(VIT_E_SHAPE, "need 1 <= D <= 32768 and rows >= 0");
  if (p.rows == 0) return VIT_OK;
  if (p.rows > 0x7fffffffLL) return fail(VIT_E_SHAPE, "more than 2^31 - 1 rows");
  if (!p.x || !p.out) return fail(VIT_E_INVALID_ARG, "x or out is NULL");
  if (!aligned_to(p.x, xs) || !aligned_to(p.out, os) || !aligned_to(p.scales, 4))
    return fail(VIT_E_INVALID_ARG, "a pointer is not aligned to its element type");
  if (p.x_ld < 0 || (p.rows > 1 && p.out_ld < p.D)) return fail(VIT_E_SHAPE, "leading dimension too small");
  bool vec = p.D % 8 == 0 && aligned16(p.x) && p.x_ld % 8 == 0 && aligned_to(p.out, os == 1 ? 8 : 16) && p.out_ld % 8 == 0;
  bool shift = aligned16(p.x) && aligned_to(p.out, os == 1 ? 8 : 16) && (p.rows == 1 || p.x_ld % 8 == p.out_ld % 8);
  if (p.w != nullptr) {
    if (!aligned_to(p.w, type_size(w_type))) return fail(VIT_E_INVALID_ARG, "weight is not aligned to its type");
    vec = vec && aligned16(p.w);
  }
  if (p.r != nullptr) {
    if (!p.h) return fail(VIT_E_INVALID_ARG, "residual without residual_out");
    if (!aligned_to(p.r, type_size(r_type)) || !aligned_to(p.h, type_size(r_type)))
      return fail(VIT_E_INVALID_ARG, "the residual is not aligned to its type");
    if (p.r_ld < 0 || (p.rows > 1 && p.h_ld < p.D)) return fail(VIT_E_SHAPE, "residual's leading dimension too small");
    vec = vec && aligned16(p.r) && aligned16(p.h) && p.r_ld % 8 == 0 && p.h_ld % 8 == 0;
    shift = shift && aligned16(p.r) && aligned16(p.h) && (p.rows == 1 || (p.r_ld % 8 == p.x_ld % 8 && p.h_ld % 8 == p.x_ld % 8));
  } else if (p.h != nullptr) {
    return fail(VIT_E_INVALID_ARG, "residual_out without residual");
  }
  // An output on an input: row i on row i, which one block reads before it writes, or rows of other blocks would
  // be overwritten before these have read them
  auto other_rows = [&](const void* o, int64_t o_bytes, const void* in, int64_t in_bytes) {
    return o == in && p.rows > 1 && o_bytes != in_bytes;
  };
  const int64_t out_bytes = p.out_ld * static_cast<int64_t>(os), x_bytes = p.x_ld * static_cast<int64_t>(xs);
  if (other_rows(p.out, out_bytes, p.x, x_bytes) || (p.r != nullptr && other_rows(p.h, p.h_ld, p.r, p.r_ld)))
    return fail(VIT_E_SHAPE, "an output on its input has to have the input's rows (the same bytes from row to row)");
  const int rmode = p.r == nullptr ? 0 : (r_type == x_type ? 1 : 2);
  const RowAccess access = vec ? ROWS_VEC : shift ? ROWS_SHIFT : ROWS_SINGLE;
  cudaError_t e;
  if (x_type == VIT_DT_BF16)
    e = launch_rows_t<__nv_bfloat16>(p, rmode, access, s);
  else if (x_type == VIT_DT_F16)
    e = launch_rows_t<__half>(p, rmode, access, s);
  else
    e = p.scales ? (rmode ? launch_rows<float, 1, true>(p, access, s) : launch_rows<float, 0, true>(p, access, s))
                 : (rmode ? launch_rows<float, 1, false>(p, access, s) : launch_rows<float, 0, false>(p, access, s));
  CK(e);
  return VIT_OK;
}

// ------------------------------------------------------------------ tensor maps
// 2-D map of 8-bit rows [rows, K]: box 128 bytes x box_rows, 128-byte swizzle; past the end: zeros.
bool tmap_rows8(CUtensorMap* tm, const void* base, int64_t K, int64_t rows, int64_t ld, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(LIN8_BK), box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D map of a bf16 output [rows, cols]: boxes of 64 columns x 32 rows.
bool tmap_out16(CUtensorMap* tm, void* base, int64_t cols, int64_t rows, int64_t ld) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  cuuint32_t box[2] = {64, 32};
  cuuint32_t estr[2] = {1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D map of heads [tokens, heads, d] of a 16-bit type: box 64 values x box_heads x box_tokens.  The
// values only move, so the type of the map does not matter.
bool tmap_heads(CUtensorMap* tm, const void* base, int d, int heads, int64_t tokens, int64_t head_ld, int64_t tok_ld,
                uint32_t box_tokens, uint32_t box_heads = 1) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  // a head of 64 is 128 bytes: the next 128 are another head's, for another CTA at another time (8 caches of
  // 100003 keys, 8 heads of 64: 308 us; 375 with 256-byte promotion)
  const CUtensorMapL2promotion promotion = d == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  // the stride of a dimension of one is never used, but has to be a valid one
  if (heads == 1) head_ld = d;
  if (tokens == 1) tok_ld = d;
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_ld) * 2, static_cast<cuuint64_t>(tok_ld) * 2};
  cuuint32_t box[3] = {64, box_heads, box_tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promotion,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

vit_status no_map() { return fail(VIT_E_CUDA, "cuTensorMapEncodeTiled refused a tensor map"); }

// ------------------------------------------------------------------ linear
cudaError_t launch_lin8_tile(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o, const Lin8Params& p, int* st,
                             cudaStream_t s, int nsm) {
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = set_smem_attr_once(lin8_tile_kernel, Lin8Cfg::SMEM_BYTES, attr_done);
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>((p.M + 127) / 128) * ((p.N + 127) / 128);
  return launch_pdl(lin8_tile_kernel, dim3(static_cast<unsigned>(std::min<long long>(tiles, nsm))), dim3(LIN8_THREADS),
                    Lin8Cfg::SMEM_BYTES, s, a, b, o, p, st);
}

cudaError_t launch_lin8_pair(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o, const Lin8Params& p, int* st,
                             cudaStream_t s, int nsm) {
  static std::atomic<uint64_t> attr_done{0};
  static std::atomic<int> max_clusters[64];  // by device
  constexpr int smem = Lin8PairCfg::SMEM_BYTES;
  cudaError_t e = set_smem_attr_once(lin8_pair_kernel, smem, attr_done);
  if (e != cudaSuccess) return e;
  int dev = 0;
  cudaGetDevice(&dev);
  int mc = max_clusters[dev & 63].load();
  if (mc == 0) {
    // how many 2-CTA clusters fit on the device at once (an SM can be left without a partner)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (nsm / 2));
    cfg.blockDim = dim3(LIN8_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, lin8_pair_kernel, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = nsm / 2;
    }
    mc = std::max(1, std::min(n, nsm / 2));
    max_clusters[dev & 63].store(mc);
  }
  const long long tiles = static_cast<long long>((p.M + 255) / 256) * ((p.N + 255) / 256);
  return launch_pdl(lin8_pair_kernel, dim3(static_cast<unsigned>(2 * std::min<long long>(tiles, mc))), dim3(LIN8_THREADS), smem,
                    s, a, b, o, p, st);
}

template <int SPLITS>
cudaError_t launch_lin8_split(const CUtensorMap& a, const CUtensorMap& b, const Lin8Params& p, __nv_bfloat16* out,
                              int64_t ldo, int* st, cudaStream_t s) {
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = set_smem_attr_once(lin8_split_kernel<SPLITS>, Lin8SplitCfg::SMEM_BYTES, attr_done);
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>((p.M + 127) / 128) * ((p.N + 127) / 128);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * SPLITS));
  cfg.blockDim = dim3(LIN8_THREADS);
  cfg.dynamicSmemBytes = Lin8SplitCfg::SMEM_BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = SPLITS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, lin8_split_kernel<SPLITS>, a, b, p, out, ldo, st);
}

template <int NB>
cudaError_t launch_lin8_rows(const Lin8RowsParams& r, int* st, cudaStream_t s, int nsm) {
  // All CTAs at once: two of 8 warps on an SM or four of 4 (1 x 8192 x 8192: 14.8 us with 8 warps, in two waves)
  const int ctas = (r.p.N + 15) / 16;
  if (ctas <= 2 * nsm) return launch_pdl(lin8_rows_kernel<NB, 8>, dim3(ctas), dim3(256), 0, s, r, st);
  return launch_pdl(lin8_rows_kernel<NB, 4>, dim3(ctas), dim3(128), 0, s, r, st);
}

// ------------------------------------------------------------------ attention
template <typename T, int HD>
cudaError_t launch_attn_packed(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                               const AttnPackedParams& p, int* st, cudaStream_t s) {
  static std::atomic<uint64_t> attr_done{0};
  constexpr int smem = AttnPackedCfg<HD>::SMEM_BYTES;
  cudaError_t e = set_smem_attr_once(attn_packed_kernel<T, HD>, smem, attr_done);
  if (e != cudaSuccess) return e;
  // n sequences of Tq rows in all need at most this many tiles
  const long long tiles = static_cast<long long>(p.Tq) / p.tokens + p.n;
  return launch_pdl(attn_packed_kernel<T, HD>, dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(p.Hq / p.pack)),
                    dim3(ATT_THREADS), smem, s, q, k, v, p, st);
}

// Which kernel a call takes.  Lengths are on the device: the rule goes by max_q and the key rows there are
// for a sequence on average (a cache's room).  Measured on a B200, us: short / split / tile kernel, for
// sequences x queries x keys, heads on key heads x width:
//   150 x 24 x 24, 16 on 16 x 64     11 / 29 / 52      74 x 24 x 24, 32 on 8 x 128    15 / 41 / 19
//   100 x 96 x 96, 16 on 16 x 64     40 / 64 / 50      74 x 48 x 48, 32 on 8 x 128    40 / 75 / 35
//   40 x 128 x 128, 16 on 16 x 64    25 / 39 / 24      57 x 48 x 48, 16 on 4 x 64      9 / 30 / 12
//   64 x 1 x 64, 32 on 8 x 128      7.3 / 11 / 12      8 x 1 x 128, 32 on 8 x 128    9.0 / 8.3 / 6.4
//   64 x 1 x 128                     13 / 13 / 14      8 x 1 x 512                    28 / 12 / 10
//   64 x 1 x 512                     46 / 33 / 31      8 x 1 x 2048                  153 / 22 / 28
//   300 x 1 x 100, 8 on 1 x 64      7.8 / 11 / 13      96 x 1 x 512, 16 on 16 x 64    52 / 51 / 64
enum AttnKernel { ATTN_TILE, ATTN_SPLIT, ATTN_SHORT };
AttnKernel attention_kernel(const vit_attn_packed* a) {
  const int64_t group = a->heads_q / a->heads_k;
  const int64_t rows = a->max_q * group;
  if (a->max_q <= 0 || a->n == 0 || a->Tq * group > 0x7fffff00LL) return ATTN_TILE;  // rows are counted in 32 bits
  const int64_t keys = a->Tk / a->n;
  const int64_t work = static_cast<int64_t>(a->n) * a->heads_k;  // sequences and key heads
  const bool many = work > 2 * current_sms();
  // the short kernel: 16 x 16 blocks of one warp
  const int64_t blocks = (rows + 15) / 16 * ((keys + 15) / 16);
  if (blocks <= (a->head_dim == 64 ? 36 : 24) && (keys <= 64 || (keys <= 128 && many)) && a->heads_k <= 65535)
    return ATTN_SHORT;
  if (rows > 64 || (keys <= 512 && work <= 4 * current_sms())) return ATTN_TILE;
  return ATTN_SPLIT;
}

template <int HD>
int rows_pieces() { return AttnRowsCfg<HD>::PER_SM * current_sms(); }

size_t rows_workspace(int head_dim) {
  const size_t rows = 16 * 2 * static_cast<size_t>(head_dim == 64 ? rows_pieces<64>() : rows_pieces<128>());
  return rows * head_dim * sizeof(float) + rows * sizeof(float2);
}

template <typename T, int HD>
cudaError_t launch_attn_rows(const CUtensorMap& k, const CUtensorMap& v, const AttnPackedParams& a, int max_q, void* ws,
                             int* st, cudaStream_t s) {
  static std::atomic<uint64_t> attr_done{0};
  constexpr int smem = AttnRowsCfg<HD>::SMEM_BYTES;
  cudaError_t e = set_smem_attr_once(attn_rows_kernel<T, HD>, smem, attr_done);
  if (e != cudaSuccess) return e;
  AttnRowsParams p{a, fast_div(static_cast<uint32_t>(a.Hq / a.Hkv)), static_cast<float*>(ws), nullptr};
  // no more pieces than there can be work for, by the row tiles that max_q promises (any number is right)
  const int64_t tiles = (static_cast<int64_t>(max_q) * p.group.d + 15) / 16;
  const int64_t units = a.Hkv * tiles * (a.Tk / 64 + a.n);
  const int pieces = static_cast<int>(std::min<int64_t>(rows_pieces<HD>(), (units + ATTR_MIN_UNITS - 1) / ATTR_MIN_UNITS));
  p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<size_t>(pieces) * 2 * 16 * HD);
  e = launch_pdl(attn_rows_kernel<T, HD>, dim3(pieces), dim3(ATTR_THREADS), smem, s, k, v, p, st);
  if (e != cudaSuccess || pieces == 1) return e;
  return launch_pdl(attn_join_kernel<T, HD>, dim3(pieces - 1), dim3(32 * ATTJ_WARPS), 0, s, p, pieces, st);
}

template <typename T, int HD>
cudaError_t launch_attn_short(const AttnPackedParams& a, int* st, cudaStream_t s) {
  const AttnShortParams p{a, fast_div(static_cast<uint32_t>(a.Hq / a.Hkv))};
  const int64_t tiles = static_cast<int64_t>(a.Tq) * p.group.d / 16 + a.n;  // at most as many
  return launch_pdl(attn_short_kernel<T, HD>,
                    dim3(static_cast<unsigned>((tiles + ATTS_WARPS - 1) / ATTS_WARPS), static_cast<unsigned>(a.Hkv)),
                    dim3(32 * ATTS_WARPS), 0, s, p, st);
}

vit_status check_attention(const vit_attn_packed* a) {
  if (!a) return fail(VIT_E_INVALID_ARG, "arguments are NULL");
  if (a->type != VIT_DT_BF16 && a->type != VIT_DT_F16) return fail(VIT_E_UNSUPPORTED, "heads must be bf16 or fp16");
  if (a->head_dim != 64 && a->head_dim != 128) return fail(VIT_E_UNSUPPORTED, "head_dim must be 64 or 128");
  if (a->n < 0 || a->Tq < 0 || a->Tk < 0 || a->Tq > 0x3fffffffLL || a->Tk > 0x3fffffffLL || a->heads_q < 1 ||
      a->heads_k < 1 || a->heads_q % a->heads_k || a->heads_q > 65535)
    return fail(VIT_E_SHAPE, "need n >= 0, 0 <= Tq, Tk < 2^30, heads_q (at most 65535) a multiple of heads_k >= 1");
  return VIT_OK;
}

}  // namespace

extern "C" {

vit_status vit_op_rms_norm(const void* x, vit_dtype x_type, int64_t x_ld, const void* residual, int64_t residual_ld,
                           void* residual_out, int64_t residual_out_ld, vit_dtype residual_type, const void* weight,
                           vit_dtype weight_type, float eps, int64_t rows, int32_t D, void* out, vit_dtype out_type,
                           int64_t out_ld, float* scales, vit_stream_t stream) {
  if (!real_type(x_type)) return fail(VIT_E_UNSUPPORTED, "x must be bf16, fp16 or fp32");
  if (out_type != x_type && out_type != VIT_DT_E4M3) return fail(VIT_E_UNSUPPORTED, "out must have x's type or e4m3");
  if ((out_type == VIT_DT_E4M3) != (scales != nullptr) && rows != 0)
    return fail(VIT_E_INVALID_ARG, "scales go with e4m3 rows, and only with them");
  if (weight_type != x_type && weight_type != VIT_DT_F32)
    return fail(VIT_E_UNSUPPORTED, "weight must have x's type or fp32");
  if (residual != nullptr && residual_type != x_type && residual_type != VIT_DT_F32)
    return fail(VIT_E_UNSUPPORTED, "the residual must have x's type or fp32");
  if (!weight) return fail(VIT_E_INVALID_ARG, "weight is NULL");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(VIT_E_INVALID_ARG, "eps must be finite and >= 0");
  RowsParams p{x, residual, residual_out, weight, out, scales, x_ld, residual_ld, residual_out_ld, out_ld, rows, D, eps,
               weight_type == VIT_DT_F32 ? 1 : 0};
  return run_rows(p, x_type, residual_type, weight_type, reinterpret_cast<cudaStream_t>(stream));
}

vit_status vit_op_quant_rows(const void* x, vit_dtype x_type, int64_t x_ld, int64_t rows, int32_t D, void* out,
                             int64_t out_ld, float* scales, vit_stream_t stream) {
  if (!real_type(x_type)) return fail(VIT_E_UNSUPPORTED, "x must be bf16, fp16 or fp32");
  if (!scales && rows != 0) return fail(VIT_E_INVALID_ARG, "scales is NULL");
  RowsParams p{x, nullptr, nullptr, nullptr, out, scales, x_ld, 0, 0, out_ld, rows, D, 0.f, 0};
  return run_rows(p, x_type, x_type, x_type, reinterpret_cast<cudaStream_t>(stream));
}

vit_status vit_op_linear_fp8(const void* A, int64_t lda, const float* a_scales, const void* W, int64_t ldw,
                             const float* w_scales, const float* bias, int32_t M, int32_t N, int32_t K, void* out,
                             int64_t ldo, int32_t* status, uint64_t wait_ns, vit_stream_t stream) {
  if (M < 0 || N < 0 || K < 16 || K % 16 || N % 8)
    return fail(VIT_E_SHAPE, "need M, N >= 0, N a multiple of 8, K >= 16 and a multiple of 16");
  if (M == 0 || N == 0) return VIT_OK;
  if (!A || !a_scales || !W || !w_scales || !out) return fail(VIT_E_INVALID_ARG, "NULL pointer");
  if (!aligned16(A) || !aligned16(W) || !aligned16(out) || !aligned16(w_scales) || !aligned16(bias) ||
      !aligned_to(a_scales, 4) || !aligned_to(status, 4))
    return fail(VIT_E_INVALID_ARG, "A, W, out, w_scales and bias must be 16-byte aligned");
  if ((M > 1 && lda < K) || (N > 1 && ldw < K) || (M > 1 && ldo < N) || lda % 16 || ldw % 16 || ldo % 8)
    return fail(VIT_E_SHAPE, "leading dimensions: at least a row, lda and ldw multiples of 16, ldo of 8");
  const int nsm = current_sms();
  Lin8Params p{M, N, K, a_scales, w_scales, bias, wait_ns};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // Measured on a B200 (148 SMs), us with the weights in L2, row kernel against K split over clusters:
  // M = 16, N = 6144, K = 4096: 7.9 / 12.3; M = 32: 512 x 1024 3.1 / 4.9, 1024 x 4096 5.2 / 6.4, 4096 x 4096
  // 12.7 / 7.2 (every CTA of the row kernel reads all of A, which past 16 rows is most of its bytes).
  if (M <= 16 || (M <= 32 && static_cast<long long>(N) * K <= 1 << 22)) {
    const Lin8RowsParams r{p, static_cast<const uint8_t*>(A), static_cast<const uint8_t*>(W), static_cast<__nv_bfloat16*>(out),
                           M > 1 ? lda : 0, N > 1 ? ldw : 0, M > 1 ? ldo : 0};
    CK(M <= 8 ? launch_lin8_rows<1>(r, status, s, nsm) : M <= 16 ? launch_lin8_rows<2>(r, status, s, nsm)
                                                            : launch_lin8_rows<4>(r, status, s, nsm));
    return VIT_OK;
  }
  CUtensorMap ta, tb, to;
  if (!tmap_rows8(&ta, A, K, M, std::max<int64_t>(lda, K), LIN8_BM) ||
      !tmap_rows8(&tb, W, K, N, std::max<int64_t>(ldw, K), 128) || !tmap_out16(&to, out, N, M, std::max<int64_t>(ldo, N)))
    return no_map();
  const long long steps = (K + LIN8_BK - 1) / LIN8_BK;
  const long long tiles = static_cast<long long>((M + 127) / 128) * ((N + 127) / 128);
  // Few tiles: K over clusters, as long as a CTA keeps four steps.  Against one CTA a tile: 33 x 4096 x
  // 4096 7.2 / 12.9 us, 100 x 1024 x 4096 9.2 / 12.9, 512 x 1024 x 4096 10.0 / 13.3; with two steps a CTA
  // (256 x 1024 x 1024) 7.6 / 7.2.
  int splits = tiles <= nsm / 10 ? 8 : tiles <= nsm / 4 ? 4 : tiles <= nsm / 2 ? 2 : 1;
  while (splits > 1 && steps < 4 * splits) splits /= 2;
  if (splits > 1) {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
    const int64_t ld = M > 1 ? ldo : 0;
    CK(splits == 8 ? launch_lin8_split<8>(ta, tb, p, o, ld, status, s)
                   : splits == 4 ? launch_lin8_split<4>(ta, tb, p, o, ld, status, s)
                                 : launch_lin8_split<2>(ta, tb, p, o, ld, status, s));
    return VIT_OK;
  }
  // A step of K takes 0.28 us of a 128 x 128 tile, 0.40 us of a 256 x 256 tile on two SMs, and the paired
  // kernel 3 us more to start: 1024 x 4096 x 4096 24 us in small tiles, 20.6 paired; 4096^3 71 / 55; 2048 x
  // 1024 x 4096 14.4 / 18.7.
  auto waves = [](long long t, int at_once) { return (t + at_once - 1) / at_once; };
  const long long pair_ns = 400 * steps * waves(static_cast<long long>((M + 255) / 256) * ((N + 255) / 256), nsm / 2) + 3000;
  const long long tile_ns = 280 * steps * waves(tiles, nsm);
  CK(pair_ns < tile_ns ? launch_lin8_pair(ta, tb, to, p, status, s, nsm) : launch_lin8_tile(ta, tb, to, p, status, s, nsm));
  return VIT_OK;
}

vit_status vit_op_rope_freqs(double base, int32_t pairs, int32_t axes, int32_t scaling, double factor,
                             double original_len, double beta_fast, double beta_slow, double* freqs) {
  if (!freqs || !(base > 0.0) || !std::isfinite(base)) return fail(VIT_E_INVALID_ARG, "need base > 0 and room for freqs");
  if (pairs < 1 || axes < 1 || axes > 4 || pairs % axes || pairs > ROPE_MAX_PAIRS)
    return fail(VIT_E_SHAPE, "need 1..128 pairs, a multiple of 1..4 axes");
  if (scaling < VIT_ROPE_PLAIN || scaling > VIT_ROPE_PARTS) return fail(VIT_E_UNSUPPORTED, "unknown scaling");
  if (scaling != VIT_ROPE_PLAIN && !(factor > 0.0 && std::isfinite(factor)))
    return fail(VIT_E_INVALID_ARG, "factor must be positive");
  if (scaling == VIT_ROPE_PARTS && !(original_len > 0.0 && beta_fast > beta_slow))
    return fail(VIT_E_INVALID_ARG, "need original_len > 0 and beta_fast > beta_slow");
  const int p = pairs / axes;
  if (scaling == VIT_ROPE_BASE) {
    if (p < 2) return fail(VIT_E_SHAPE, "a larger base needs two pairs an axis");
    base *= std::pow(factor, static_cast<double>(p) / (p - 1));
  }
  for (int i = 0; i < p; ++i) {
    double f = std::pow(base, -static_cast<double>(i) / p);
    if (scaling == VIT_ROPE_LINEAR) f /= factor;
    if (scaling == VIT_ROPE_PARTS) {
      const double turns = f * original_len / 6.283185307179586476925;
      const double keep = std::min(1.0, std::max(0.0, (turns - beta_slow) / (beta_fast - beta_slow)));
      f = f / factor * (1.0 - keep) + f * keep;
    }
    for (int a = 0; a < axes; ++a) freqs[a * p + i] = f;
  }
  return VIT_OK;
}

vit_status vit_op_rope(const vit_rope_tensor* q, const vit_rope_tensor* k, vit_dtype type, int64_t T, int32_t head_dim,
                       int32_t rotary_dim, const void* positions, int32_t pos64, int32_t axes, const double* freqs,
                       int32_t layout, float gain, int32_t inverse, vit_stream_t stream) {
  if (!real_type(type)) return fail(VIT_E_UNSUPPORTED, "heads must be bf16, fp16 or fp32");
  if (layout != VIT_ROPE_HALF && layout != VIT_ROPE_INTERLEAVED) return fail(VIT_E_UNSUPPORTED, "unknown layout");
  if (T < 0 || axes < 1 || axes > 4 || rotary_dim < 2 || rotary_dim % 2 || rotary_dim > 2 * ROPE_MAX_PAIRS ||
      head_dim < rotary_dim || head_dim > 4096 || (rotary_dim / 2) % axes)
    return fail(VIT_E_SHAPE, "rotary_dim: even, 2..256, at most head_dim (at most 4096), pairs a multiple of 1..4 axes");
  if (!freqs) return fail(VIT_E_INVALID_ARG, "freqs is NULL");
  if (!std::isfinite(gain)) return fail(VIT_E_INVALID_ARG, "gain must be finite");
  const vit_rope_tensor* tq[2] = {q, k};
  const int n = rotary_dim / 2;
  const int size = static_cast<int>(type_size(type));
  // bytes an access: what every chunk's place and every row's stride is a multiple of
  int64_t even = 16 / size;
  auto share = [&even](int64_t v) {
    while (v % even) even /= 2;
  };
  share(layout == VIT_ROPE_HALF ? n : rotary_dim);
  share(head_dim - rotary_dim);
  RopeParams p{};
  for (int i = 0; i < 2; ++i) {
    if (!tq[i] || !tq[i]->in || tq[i]->heads == 0) continue;
    const vit_rope_tensor& t = *tq[i];
    if (t.heads < 0) return fail(VIT_E_SHAPE, "negative number of heads");
    if (!t.out || !aligned_to(t.in, type_size(type)) || !aligned_to(t.out, type_size(type)))
      return fail(VIT_E_INVALID_ARG, "output NULL, or a pointer not aligned to its type");
    if (T > 0 && overlap_itself(T, t.out_token, t.heads, t.out_head, head_dim)) return fail(VIT_E_SHAPE, "heads of an output overlap");
    if (t.in == t.out && ((T > 1 && t.in_token != t.out_token) || (t.heads > 1 && t.in_head != t.out_head)))
      return fail(VIT_E_SHAPE, "an output on its input has to have the input's strides");
    p.in[i] = t.in;
    p.out[i] = t.out;
    p.in_tok[i] = t.in_token;
    p.in_head[i] = t.in_head;
    p.out_tok[i] = t.out_token;
    p.out_head[i] = t.out_head;
    p.heads[i] = t.heads;
    for (int64_t v : {t.in_token, t.in_head, t.out_token, t.out_head}) share(v);
    for (const void* v : {t.in, static_cast<const void*>(t.out)}) share(static_cast<int64_t>(reinterpret_cast<uintptr_t>(v) / size));
  }
  if (T == 0 || p.heads[0] + p.heads[1] == 0) return VIT_OK;
  if (!positions || !aligned_to(positions, pos64 ? 8 : 4)) return fail(VIT_E_INVALID_ARG, "positions NULL or misaligned");
  for (int i = 0; i < n; ++i) {
    if (!std::isfinite(freqs[i])) return fail(VIT_E_INVALID_ARG, "a frequency is not finite");
    // 2^64 times the fraction of a turn, in the 64-bit mantissa of long double
    long double t = static_cast<long double>(freqs[i]) * 0.15915494309189533576888376337251436L;
    if (!(t >= 0.0L && t < 1.0L)) t -= floorl(t);
    t = t * 18446744073709551616.0L + 0.5L;
    p.turn[i] = t >= 18446744073709551616.0L ? 0ull : static_cast<unsigned long long>(t);
  }
  p.pos = positions;
  p.T = T;
  p.d = head_dim;
  p.rd = rotary_dim;
  p.axes = axes;
  p.pos64 = pos64 != 0;
  p.sign = inverse ? -1.f : 1.f;
  p.gain = gain;
  // tokens a block: enough pairs for one sine and cosine per thread, but at least four blocks an SM
  // while the tokens last
  const int64_t spread = std::max<int64_t>(1, T / (4 * current_sms()));
  p.tokens = static_cast<int>(std::min<int64_t>(spread, std::max(1, ROPE_THREADS / n)));
  const int64_t blocks = (T + p.tokens - 1) / p.tokens;
  if (blocks > 0x7fffffffLL) return fail(VIT_E_SHAPE, "too many tokens");
  const size_t smem = static_cast<size_t>(p.tokens) * n * sizeof(float2);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(ROPE_THREADS), smem,
                      reinterpret_cast<cudaStream_t>(stream), p);
  };
  cudaError_t err;
  auto by_layout = [&](auto half_kernel, auto pair_kernel) { return layout == VIT_ROPE_HALF ? go(half_kernel) : go(pair_kernel); };
  auto by_access = [&](auto t) {
    using T = decltype(t);
    constexpr int E = 16 / sizeof(T);
    if (even >= E) return by_layout(rope_kernel<T, true, E>, rope_kernel<T, false, E>);
    if (even >= E / 2) return by_layout(rope_kernel<T, true, E / 2>, rope_kernel<T, false, E / 2>);
    return by_layout(rope_kernel<T, true, 1>, rope_kernel<T, false, 1>);
  };
  if (type == VIT_DT_BF16)
    err = by_access(__nv_bfloat16{});
  else if (type == VIT_DT_F16)
    err = by_access(__half{});
  else
    err = by_access(float{});
  CK(err);
  return VIT_OK;
}

vit_status vit_op_attention_packed_workspace(const vit_attn_packed* a, size_t* bytes) {
  const vit_status st = check_attention(a);
  if (st != VIT_OK) return st;
  if (!bytes) return fail(VIT_E_INVALID_ARG, "bytes is NULL");
  *bytes = attention_kernel(a) == ATTN_SPLIT ? rows_workspace(a->head_dim) : 0;
  return VIT_OK;
}

vit_status vit_op_attention_packed(const vit_attn_packed* a, vit_stream_t stream) {
  const vit_status st = check_attention(a);
  if (st != VIT_OK) return st;
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return fail(VIT_E_INVALID_ARG, "scale must be positive and finite");
  if (a->n == 0 || a->Tq == 0) return VIT_OK;
  if (!a->q || !a->out || !a->cu_q || !a->cu_k || (a->Tk > 0 && (!a->k || !a->v)))
    return fail(VIT_E_INVALID_ARG, "NULL pointer");
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->out) || !aligned_to(a->cu_q, 4) ||
      !aligned_to(a->cu_k, 4) || !aligned_to(a->len_k, 4) || !aligned_to(a->status, 4))
    return fail(VIT_E_INVALID_ARG, "q, k, v and out must be 16-byte aligned");
  const int64_t strides[8] = {a->q_token, a->q_head, a->k_token, a->k_head, a->v_token, a->v_head, a->out_token, a->out_head};
  for (int64_t s : strides)
    if (s % 8 || s < 0 || s >= (1LL << 38)) return fail(VIT_E_SHAPE, "strides must be multiples of 8, not negative");
  if (overlap_itself(a->Tq, a->out_token, a->heads_q, a->out_head, a->head_dim))
    return fail(VIT_E_SHAPE, "heads of out overlap");
  if (static_cast<int64_t>(a->n) + a->Tq > 0x7fffffffLL) return fail(VIT_E_SHAPE, "too many sequences");
  const AttnKernel which = attention_kernel(a);
  const bool rows = which == ATTN_SPLIT;
  if (rows && (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < rows_workspace(a->head_dim)))
    return fail(VIT_E_WORKSPACE, "workspace missing, not 16-byte aligned or too small");
  AttnPackedParams p{};
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.out = a->out;
  p.q_tok = a->q_token;
  p.q_head = a->q_head;
  p.k_tok = a->k_token;
  p.k_head = a->k_head;
  p.v_tok = a->v_token;
  p.v_head = a->v_head;
  p.o_tok = a->out_token;
  p.o_head = a->out_head;
  p.cu_q = a->cu_q;
  p.cu_k = a->cu_k;
  p.len_k = a->len_k;
  p.n = a->n;
  p.Tq = static_cast<int>(a->Tq);
  p.Tk = static_cast<int>(a->Tk);
  p.Hq = a->heads_q;
  p.Hkv = a->heads_k;
  p.causal = a->causal != 0;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.wait_ns = a->wait_ns;
  // As many of the heads that share a key head in a tile as divide their number and fill 120 of 128 rows
  const int group = a->heads_q / a->heads_k;
  p.pack = 1;
  for (int x = 2; x <= std::min(group, 128); ++x)
    if (group % x == 0 && 128 / x * x >= 120) p.pack = x;
  p.tokens = 128 / p.pack;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (which == ATTN_SHORT) {
    if (a->type == VIT_DT_BF16)
      e = a->head_dim == 64 ? launch_attn_short<__nv_bfloat16, 64>(p, a->status, s)
                            : launch_attn_short<__nv_bfloat16, 128>(p, a->status, s);
    else
      e = a->head_dim == 64 ? launch_attn_short<__half, 64>(p, a->status, s)
                            : launch_attn_short<__half, 128>(p, a->status, s);
    CK(e);
    return VIT_OK;
  }
  CUtensorMap tq, tk, tv;
  // without keys nothing is loaded: any valid map will do
  const void* kb = a->Tk > 0 ? a->k : a->q;
  const void* vb = a->Tk > 0 ? a->v : a->q;
  const int64_t tkeys = std::max<int64_t>(1, a->Tk);
  if ((!rows && !tmap_heads(&tq, a->q, a->head_dim, a->heads_q, a->Tq, a->q_head, a->q_token, p.tokens, p.pack)) ||
      !tmap_heads(&tk, kb, a->head_dim, a->heads_k, tkeys, a->k_head, a->k_token, 64) ||
      !tmap_heads(&tv, vb, a->head_dim, a->heads_k, tkeys, a->v_head, a->v_token, 64))
    return no_map();
  if (rows) {
    if (a->type == VIT_DT_BF16)
      e = a->head_dim == 64 ? launch_attn_rows<__nv_bfloat16, 64>(tk, tv, p, a->max_q, a->workspace, a->status, s)
                            : launch_attn_rows<__nv_bfloat16, 128>(tk, tv, p, a->max_q, a->workspace, a->status, s);
    else
      e = a->head_dim == 64 ? launch_attn_rows<__half, 64>(tk, tv, p, a->max_q, a->workspace, a->status, s)
                            : launch_attn_rows<__half, 128>(tk, tv, p, a->max_q, a->workspace, a->status, s);
    CK(e);
    return VIT_OK;
  }
  if (a->type == VIT_DT_BF16)
    e = a->head_dim == 64 ? launch_attn_packed<__nv_bfloat16, 64>(tq, tk, tv, p, a->status, s)
                          : launch_attn_packed<__nv_bfloat16, 128>(tq, tk, tv, p, a->status, s);
  else
    e = a->head_dim == 64 ? launch_attn_packed<__half, 64>(tq, tk, tv, p, a->status, s)
                          : launch_attn_packed<__half, 128>(tq, tk, tv, p, a->status, s);
  CK(e);
  return VIT_OK;
}

vit_status vit_op_poll(vit_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int v = 0;
  const int zero = 0;
  CK(cudaMemcpyFromSymbolAsync(&v, g_op_status, sizeof(v), 0, cudaMemcpyDeviceToHost, s));
  CK(cudaStreamSynchronize(s));
  if (v == 0) return VIT_OK;
  CK(cudaMemcpyToSymbolAsync(g_op_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s));
  CK(cudaStreamSynchronize(s));
  set_err("a kernel gave up on a pipeline wait (site 0x%x)", v);
  return VIT_E_DEVICE_TIMEOUT;
}

}  // extern "C"
