// ops_step.cu -- what the decode step's form with shared prefixes needs on the
// device besides the serving operators.
#include "ops_common.cuh"
#include "ops_step.h"

namespace mk {
namespace ops {
namespace {

__global__ void add_kernel(uint32_t* counters, const int32_t* pairs, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) counters[pairs[2 * i]] += (uint32_t)pairs[2 * i + 1];
}

__global__ void check_equal_kernel(const int32_t* position, const int32_t* seq_len, int n, int32_t* status) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < n && position[b] != seq_len[b])
    report(status, MK_ERR_DEVICE, MK_OP_SAMPLE, b, position[b], seq_len[b]);
}

}  // namespace

cudaError_t check_equal(const int32_t* position, const int32_t* seq_len, int n, int32_t* status,
                        cudaStream_t stream) {
  check_equal_kernel<<<(n + 31) / 32, 32, 0, stream>>>(position, seq_len, n, status);
  return cudaGetLastError();
}

cudaError_t add_to_counters(uint32_t* counters, const int32_t* pairs, int n, cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  add_kernel<<<(n + 255) / 256, 256, 0, stream>>>(counters, pairs, n);
  return cudaGetLastError();
}

}  // namespace ops
}  // namespace mk
