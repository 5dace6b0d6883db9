// Device status of the operator entry points: a caller's word, or, where none is given, one word per
// device in the library that vit_op_poll reads and clears.  A caller's word also stops later kernels on it;
// the library's does not, since calls of others share it.
#pragma once

#include "common.cuh"

namespace vit {

static __device__ int g_op_status;

__device__ __forceinline__ int* op_status(int* given) { return given != nullptr ? given : &g_op_status; }

// Whether an earlier kernel on the caller's word gave up.
__device__ __forceinline__ bool op_stopped(const int* given) {
  return given != nullptr && *reinterpret_cast<const volatile int*>(given) != 0;
}

// mbar_wait by a whole warp with one answer for all lanes: a lane that gives up takes the others
// with it, so that no lane is left behind at a warp-wide instruction.
template <int kPoll = kPollDefault>
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* gstatus,
                                               int site, unsigned long long limit) {
  return __all_sync(0xffffffffu, mbar_wait<kPoll>(bar, parity, abort_flag, gstatus, site, limit));
}

}  // namespace vit
