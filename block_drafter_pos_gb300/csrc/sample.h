// Truncated sampling: the kernel's arguments and launch.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace df2 {

// Largest vocabulary: sums of 2^19 weights of at most 2^44 stay below 2^64.
constexpr int kSampleMaxVocab = 1 << 19;

struct SampleArgs {
  const void* logits;
  long long row_stride;
  int n_rows, vocab, type;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* uniform;
  int32_t* token;
  float* prob;
  float* kept;
  long long kept_stride;
  int32_t* status;
  int kept_in_place;  // kept overlaps the logits
  int num_sms;
};
cudaError_t launch_sample(const SampleArgs& a, cudaStream_t st);

}  // namespace df2
