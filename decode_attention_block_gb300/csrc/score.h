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

// Parts per row: more CTAs for few rows, against a list of alternatives for each
// part and the join.  fp32 rows of 131072, us on the GPU whole and in the parts
// the rule takes, without alternatives, with 20 and with 32:
//     32 rows, 8 parts   22.7 and  8.3   28.5 and 16.8   30.0 and 17.9
//     64 rows, 4 parts   23.2 and 11.4   29.0 and 21.9   30.3 and 24.6
//    100 rows, 2 parts   23.9 and 16.6   29.3 and 28.1   30.8 and 30.6
//    128 rows, 2 parts   24.4 and 17.5   29.8 and 28.8   30.9 and 31.0
// so kMaxSplit ends where a split stops paying (511 rows in two parts: 72
// against 57).  At 65536 two parts of 86 to 128 rows win without alternatives
// (13.3 and 10.9) and lose with them (18.8 and 21.3 with 20 for 100 rows), up to
// 64 rows parts win or lose less than 1 us; rows of 262144 gain throughout (50.3 and 40.0).  Rows of
// 32001 take 12 us whole and 10.4 in 8 parts at best, and longer as soon as
// there are 48 of them: below kSplitElems a row stays whole.
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
