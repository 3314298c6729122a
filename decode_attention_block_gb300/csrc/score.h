// score.h -- workspace and split of spark_token_logprobs (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spark_score.h"

namespace spark {
namespace score {

constexpr int kMaxParts = 64;       // parts a row is split into at most
constexpr int kMaxSplit = 2048;     // (row, part) pairs of a split call at most
constexpr int kPartElems = 4096;    // elements of a part at least: one tile

// what one part of a row leaves for the join
struct alignas(16) Part {
  float m, z, u;
  int bad;
  unsigned long long key[SPARK_MAX_TOP];
};

constexpr size_t kTickets = 256;    // uint32 [kMaxSplit], zero between launches; the error word sits at 0
constexpr size_t kParts = kTickets + 4 * kMaxSplit;
constexpr size_t kTotal = kParts + sizeof(Part) * kMaxSplit;

// Parts per row: enough CTAs for the GPU (about two an SM) where the rows
// alone are too few.
inline int parts_for(int n_rows, int vocab, int sms) {
  int64_t c = (2 * (int64_t)sms + n_rows - 1) / n_rows;
  const int64_t most = vocab / kPartElems;
  if (c > most) c = most;
  if (c > kMaxParts) c = kMaxParts;
  if (c * n_rows > kMaxSplit) c = kMaxSplit / n_rows;
  return c < 1 ? 1 : (int)c;
}

}  // namespace score

cudaError_t launch_score(const void* logits, int64_t ld, int dtype, int n_rows, int vocab, const int32_t* targets, int k,
                         float* logprob, float* entropy, int32_t* top_ids, float* top_logprobs, void* workspace,
                         cudaStream_t st);

}  // namespace spark
