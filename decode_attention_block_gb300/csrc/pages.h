// pages.h -- a spark_pages_* call as its launcher takes it, and the layout of
// its workspace (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spark_paged.h"

namespace spark {

// error word bit: the pool has too few free pages
constexpr uint32_t kErrPages = 4u;

namespace pages {

struct Head {
  int32_t bad;       // an argument on the device is out of range
  int32_t n_moves;   // moves the copy kernel carries out
  int32_t below;     // compact: used pages before page n_live
  int32_t totals[8];  // pages counted by each CTA of the plan
};

// rows 0 .. rows - 1 of page src to page dst
struct Move {
  int32_t src, dst, rows, unused;
};

struct Pools {
  void* p[2 * SPARK_MAX_PAGE_POOLS];  // K, V of each layer
};

struct Call {
  Pools pools;
  int32_t n_pools;
  int64_t n_pages;
  int32_t page_size;
  int64_t row_bytes;
  int32_t row_step;  // rows that lie together: a page's first rows are copied in multiples of it
  const int32_t* table;
  int32_t* new_table;
  int32_t n_slots, max_pages;
  const int32_t *parent, *keep, *grow;  // remap; null: compact
  int32_t* n_live;                      // compact
  void* workspace;
};

struct WsLayout {
  size_t head, moves, state, list, total;
};

inline WsLayout ws_layout(int64_t n_pages, int32_t n_slots) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t moves = (size_t)(n_pages > n_slots ? n_pages : n_slots);
  WsLayout L;
  L.head = 256;  // the error word sits at 0
  L.moves = 512;
  L.state = up(L.moves + sizeof(Move) * moves);
  L.list = up(L.state + sizeof(int32_t) * (size_t)n_pages);
  L.total = up(L.list + sizeof(int32_t) * (size_t)n_pages);
  return L;
}

}  // namespace pages

cudaError_t launch_pages(const pages::Call& c, cudaStream_t st);

}  // namespace spark
