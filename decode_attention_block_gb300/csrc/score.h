// score.h -- workspace and split of spark_token_logprobs (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spark_score.h"

namespace spark {
namespace score {

constexpr int kMaxParts = 64;       // parts a row is split into at most
constexpr int kMaxSplit = 256;      // (row, part) pairs of a split call at most
constexpr int kPartElems = 4096;    // elements of a part at least: one tile
constexpr int kSplitElems = 65536;  // of a row that is split

// what one part of a row leaves for the join
struct alignas(16) Part {
  float m, z, u;
  int bad;
  unsigned long long key[SPARK_MAX_TOP];
};

constexpr size_t kTickets = 256;    // uint32 [kMaxSplit], zero between launches; the error word sits at 0
constexpr size_t kParts = kTickets + 4 * kMaxSplit;
constexpr size_t kTotal = kParts + sizeof(Part) * kMaxSplit;

// Parts per row.  A part's list of alternatives and the join cost more than the
// CTAs gain where there are many: one row of 131072 with 20 alternatives takes
// 22 us whole, 14 in 8 parts and 10.8 in 32; 32 rows 25, 18 and 22; 100 rows 26
// whole and 28 in two; 511 rows 57 and 72.  Rows of 32001 take 12 us whole and
// 10.4 in 8 parts at best, and longer as soon as there are 48 of them.
inline int parts_for(int n_rows, int vocab) {
  if (vocab < kSplitElems) return 1;
  int c = kMaxSplit / n_rows;
  if (c > vocab / kPartElems) c = vocab / kPartElems;
  if (c > kMaxParts) c = kMaxParts;
  return c < 1 ? 1 : c;
}

}  // namespace score

cudaError_t launch_score(const void* logits, int64_t ld, int dtype, int n_rows, int vocab, const int32_t* targets, int k,
                         float* logprob, float* entropy, int32_t* top_ids, float* top_logprobs, void* workspace,
                         cudaStream_t st);

}  // namespace spark
