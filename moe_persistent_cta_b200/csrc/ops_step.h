// ops_step.h -- the serving operators as the decode step calls them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mk.h"

namespace mk {
namespace ops {

// Where the attention of a decode step goes instead of `out`: 32-bit rows
// [batch][query heads][head size] and, for the output projection, per KV head a
// block of frag_bytes with rows of frag_stride floats per entry.
struct StepSink {
  float* out = nullptr;
  uint8_t* frag = nullptr;
  int frag_bytes = 0, frag_stride = 0;
};
mk_status prefix_attention(const mk_prefix_attention_args* args, const StepSink& sink, cudaStream_t stream);

// mk_sample, then the decode loop's state moved on: the drawn token (0 where
// there is none) into next_token, position and seq_len (once if they are one
// buffer) up by one.
mk_status sample(const mk_sample_args* args, int32_t* next_token, int32_t* position, int32_t* seq_len,
                 cudaStream_t stream);

// Reports (MK_ERR_DEVICE, MK_OP_SAMPLE) an entry whose position is not its
// sequence's length: sampled steps advance every entry alone.  Ahead of them, since
// the same test in the sampling kernel cost every call of it 1 %.
cudaError_t check_equal(const int32_t* position, const int32_t* seq_len, int n, int32_t* status,
                        cudaStream_t stream);

// counters[pairs[2 i]] += pairs[2 i + 1] for i < n.
cudaError_t add_to_counters(uint32_t* counters, const int32_t* pairs, int n, cudaStream_t stream);

}  // namespace ops
}  // namespace mk
