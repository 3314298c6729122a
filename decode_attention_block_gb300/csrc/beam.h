// beam.h -- calls of the beam search kernels and their workspace (internal to
// the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spark_beam.h"

namespace spark {
namespace beam {

constexpr int kMaxParts = 64;      // parts a row is split into at most
constexpr int kMaxPairs = 1024;    // (row, part) pairs of a call at most
constexpr int kPartElems = 8192;   // elements of a part at least: two tiles
// Parts for CTAs as far as they run at once (four an SM).  us on the GPU, fp32 rows
// of 131072, parts of 4096 elements at least and of 8192: one group of 4 beams 13.9
// and 12.7, four 15.8 and 13.7; up to 512 CTAs and up to 300: 16 groups of 4 beams
// 19.1 and 17.5, 32 of 8 35 and 36.5, 8 of 32 (whole rows then, long lists) 51 and 99.
constexpr int kWantedCtas = 512;

// what one part of a row leaves for the join of its group
struct alignas(16) Part {
  float m;
  int bad;   // a NaN or +inf among its logits
  float z, z_rest;  // sum of e^(x - m), as a number and what it leaves
  unsigned long long key[SPARK_MAX_BEAMS];
};

constexpr size_t kTickets = 256;  // uint32 [SPARK_MAX_BATCH], zero between launches; the error word sits at 0
constexpr size_t kParts = kTickets + 4 * SPARK_MAX_BATCH;
constexpr size_t kTotal = kParts + sizeof(Part) * kMaxPairs;

inline int parts_for(int n_rows, int vocab) {
  int c = kWantedCtas / n_rows;
  if (c > vocab / kPartElems) c = vocab / kPartElems;
  if (c > kMaxParts) c = kMaxParts;
  return c < 1 ? 1 : c;
}

struct Select {
  const void* logits;
  int64_t ld;
  int n_groups, n_beams, vocab;
  const float* score;
  const int32_t *done, *length;
  int eos;
  float* new_score;
  int32_t *token, *parent, *new_done, *keep_len, *new_len;
  uint32_t* tickets;
  Part* part;
};

struct States {
  spark_beam_state s[SPARK_MAX_BEAM_STATES];
};

}  // namespace beam

cudaError_t launch_beam_select(const beam::Select& a, int dtype, cudaStream_t st);
cudaError_t launch_beam_reorder(const int32_t* parent, const int32_t* keep, const int32_t* grow, int n_slots,
                                const beam::States& states, int n_states, uint32_t* err, cudaStream_t st);

}  // namespace spark
