// ops_common.cuh -- what the serving operators beside the decode step share:
// host-side argument checks and the current-device guard, the 16-bit storage
// types, and the device status word.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mk.h"

namespace mk {
namespace ops {

constexpr int kPageTokens = 64;   // tokens per KV page, as in the decode step

inline mk_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return MK_OK;
  (void)cudaGetLastError();
  if (e == cudaErrorMemoryAllocation) return MK_ERR_OOM;
  return e == cudaErrorInvalidDevice ? MK_ERR_INVALID : MK_ERR_CUDA;
}

// Makes `device` current for one call and puts the caller's device back.
class DeviceGuard {
 public:
  explicit DeviceGuard(int device) {
    err_ = cudaGetDevice(&prev_);
    if (err_ == cudaSuccess && prev_ != device) {
      err_ = cudaSetDevice(device);
      moved_ = err_ == cudaSuccess;
    }
  }
  ~DeviceGuard() {
    if (moved_) (void)cudaSetDevice(prev_);
  }
  DeviceGuard(const DeviceGuard&) = delete;
  DeviceGuard& operator=(const DeviceGuard&) = delete;
  mk_status status() const { return from_cuda(err_); }

 private:
  int prev_ = 0;
  bool moved_ = false;
  cudaError_t err_;
};

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// ------------------------------------------------------------ device side --

// Latches {code, operator, entry, value, limit} in the caller's status word
// (may be null): the first report stays until the caller clears the word.
__device__ inline void report(int32_t* status, int code, int op, int entry, int value, int limit) {
  if (status == nullptr || atomicCAS(status, 0, code) != 0) return;
  status[1] = op;
  status[2] = entry;
  status[3] = value;
  status[4] = limit;
}

template <typename T>
struct Vec8 {   // 8 elements of a 16-bit type as one 16-byte word
  static __device__ __forceinline__ void unpack(uint4 w, float* f);
  static __device__ __forceinline__ uint4 pack(const float* f);
};

template <>
struct Vec8<__nv_bfloat16> {
  static __device__ __forceinline__ void unpack(uint4 w, float* f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

template <>
struct Vec8<__half> {
  static __device__ __forceinline__ void unpack(uint4 w, float* f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

}  // namespace ops
}  // namespace mk
