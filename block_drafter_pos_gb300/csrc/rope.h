// Rotary positions: argument blocks and launch interfaces.
#pragma once

#include "paged.h"

namespace df2 {

constexpr int kRopeMaxPairs = 128;
constexpr int kRopeMaxDim = 1024, kRopeMaxHeads = 1024;  // of a row, and of a token in all: at most 2^16 items of 16 channels
constexpr int kRopeMaxTokens = 0x7FFFFFF0;                // (a CTA's last token is numbered in 32 bits)

struct RopePlan {
  int rot;              // channels that are turned
  int interleaved;
  float amplitude, sign;  // sign -1: the opposite angle
  unsigned long long turns[kRopeMaxPairs];
};

struct RopeArgs {
  PagedRows x, y, k, ky;  // heads of x to y, of k to ky
  int n_tokens, dim, x_heads, k_heads;
  int x_copy, k_copy;     // whether the channels behind the turned ones are copied (not where a row is turned in place)
  const int32_t* positions;
  RopePlan plan;
};
cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t st);

struct RopeWriteArgs {
  PagedMoveArgs move;     // the keys and values
  PagedRows q, y;         // q.p null: none
  int q_heads, q_copy;
  const int32_t* positions;  // null: the tokens' positions in the cache
  RopePlan plan;
};
cudaError_t launch_rope_write(const RopeWriteArgs& a, int head_dim, int fmt, int num_sms, cudaStream_t st);

}  // namespace df2
