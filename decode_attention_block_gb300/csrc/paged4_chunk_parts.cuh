// paged4_chunk_parts.cuh -- what the chunk attention kernels over 4-bit pages
// share (paged4_chunk.cu: one CTA and 32 tokens a group; paged4_pair.cu: two
// CTAs and 64): blocks of pages into fp16 operands in shared memory.
//
// A warp takes a block or half of its rows or dims: plain loads of codes and scales
// into registers, a tile ahead of their use (a block's parts are contiguous, so
// nothing is gained by a copy engine, and no shared memory is spent on bytes that
// are read once), then conversion and 16-byte stores in the layout of
// paged_chunk_parts.cuh.
#pragma once

#include "paged_chunk_parts.cuh"

namespace spark {
namespace chunk4 {

using namespace chunk;

constexpr int kDequant = 8;          // warps
constexpr int kThreads4 = 128 * 2 + 32 * kDequant;
constexpr int kFirstSoft = 4, kFirstDequant = 8;  // warps, in warpgroups: 0 and 1 load queries and issue MMAs
// Registers a thread, by warpgroup (setmaxnreg): each group gives up or takes of
// the launch's 4 x 128 (a dec to more than a thread has is an illegal instruction).
constexpr int kRegsLaunch = 128;  // of 65536 for 512 threads
template <int ISSUE, int SOFT, int DEQUANT>
struct Regs {
  static constexpr int kIssue = ISSUE, kSoft = SOFT, kDequant = DEQUANT;
  static_assert(ISSUE < kRegsLaunch && SOFT > kRegsLaunch && DEQUANT < kRegsLaunch && ISSUE + SOFT + 2 * DEQUANT <= 4 * kRegsLaunch &&
                    ISSUE % 8 + SOFT % 8 + DEQUANT % 8 == 0,
                "registers of the launch");
};

template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// A lane's part of a block: chunk 4 h + lane / 8 of rows lane % 8 and lane % 8 +
// 8, their codes and the two scales of each.  (Eight lanes with rows of their own
// store 16 bytes of each in different banks.)
struct Part {
  uint4 code[2];
  uint32_t scale[2];
};

// Where they lie in a pool: with X the first row's chunk of h = 0, that of h = 1
// is X ^ 64 bytes, and 8 rows further the two have changed places (fp4::turn).
struct Lanes {
  const unsigned char *x0, *x1, *y;
  __device__ __forceinline__ Lanes(const unsigned char* pool, int lane) {
    const int row = lane & 7, c = lane >> 3;
    const uint32_t x = (uint32_t)(row * fp4::kCodes + ((c ^ fp4::turn(row)) << 4));
    x0 = pool + x;
    x1 = pool + (x ^ 64u);
    y = pool + fp4::kScalesAt + row * fp4::kScales + 2 * c;
  }
  static constexpr uint32_t kNone = 0xFFFFFFFFu;
  // half h's part of a block (kNone: zeros)
  __device__ __forceinline__ void load(Part& x, uint32_t block, int h) const {
    if (block == kNone) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x.code[i] = make_uint4(0u, 0u, 0u, 0u);
        x.scale[i] = 0u;
      }
      return;
    }
    const uint64_t at = (uint64_t)block * (uint64_t)fp4::kBlock;
    x.code[0] = __ldcg(reinterpret_cast<const uint4*>((h ? x1 : x0) + at));
    x.code[1] = __ldcg(reinterpret_cast<const uint4*>((h ? x0 : x1) + at + 8 * fp4::kCodes));
#pragma unroll
    for (int i = 0; i < 2; ++i)
      x.scale[i] = __ldcg(reinterpret_cast<const unsigned short*>(y + at + 8 * h + 8 * i * fp4::kScales));
  }
};

// The block of a warp's positions in each of a group's tiles, found for 32 tiles at
// a time, one per lane.
struct Blocks {
  static constexpr int kTiles = 32;
  uint32_t mine;
  // those at x and at the 31 places kPos apart behind it, before `end`
  __device__ __forceinline__ void find(const Args& p, const Cursor& cur, int x, int end, int lane) {
    x += lane * kPos;
    mine = Lanes::kNone;
    if (x < end && x <= cur.g.hi && x + fp4::kRows > cur.g.lo) {
      const int col = paged::page_col(p, x), in_page = (x - col * p.page_size) / fp4::kRows;
      const int page = paged::page_of(p, paged::page_entry(p, cur.s, col));
      // (pages * page_size < 2^31: the blocks of all heads are below 2^30)
      mine = ((uint32_t)page * (uint32_t)(p.page_size / fp4::kRows) + (uint32_t)in_page) * (uint32_t)p.n_kv + (uint32_t)cur.j;
    }
  }
  __device__ __forceinline__ uint32_t of(int tile) const { return __shfl_sync(0xffffffffu, mine, tile % kTiles); }
};

// The part's 32 dims of each row as fp16: with c = lane / 8, line c / 2 of 64
// dims, four 16-byte chunks of a row of 128 bytes, chunk 4 (c % 2) + e of row r at
// (4 (c % 2) + e) ^ (r % 8): the lane's places are at[e] in the line; the second
// row lies `group` bytes behind.
__device__ __forceinline__ void store_part(uint32_t line, const uint32_t (&at)[4], uint32_t group, const Part& x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {x.code[i].x, x.code[i].y, x.code[i].z, x.code[i].w};
    const uint32_t f[2] = {__byte_perm(x.scale[i], 0u, 0x4040u) << 7, __byte_perm(x.scale[i], 0u, 0x4141u) << 7};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t h[4];
      fp4::halves8(w[k], h);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = fp4::mul2(h[j], f[k >> 1]);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(line + at[k] + i * group), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                   : "memory");
    }
  }
}
// Whole rows of a block by a warp: chunk c = lane / 8 ^ 5 (lane / 4 % 2) of four
// rows of each of the block's row groups u < 4, rows 0 1 6 7, 2 3 4 5, then 8
// further.  A group's codes are four lines of 128 bytes, read whole (half lines of
// eight rows cost a load twice the passes of the memory pipe, which these kernels
// are bound by), and eight lanes store 16 bytes each in different banks: their four
// rows and two chunks of either parity differ in (4 (c % 2)) ^ (r % 8).
struct RowLanes {
  const unsigned char *x0, *x1, *y0, *y1;  // codes and scales of groups 0 and 1
  int d0, d1;         // codes from group 0 to 2, from 1 to 3
  uint32_t at0, at1;  // places in the line, of rows of groups 0 and 1, of the chunk's first 16 bytes (the k-th: ^ 16 k)
  int h, line;        // half of the dims, line of it
  __device__ __forceinline__ RowLanes(const unsigned char* pool, int lane) {
    const int s = lane & 3, c = (lane >> 3) ^ ((lane & 4) ? 5 : 0), r0 = s < 2 ? s : s + 4, r1 = s + 2;
    const uint32_t a0 = (uint32_t)(r0 * fp4::kCodes + ((c ^ fp4::turn(r0)) << 4)), a1 = (uint32_t)(r1 * fp4::kCodes + ((c ^ fp4::turn(r1)) << 4));
    x0 = pool + a0;
    x1 = pool + a1;
    y0 = pool + fp4::scale_at(r0, 32 * c);
    y1 = pool + fp4::scale_at(r1, 32 * c);
    d0 = (int)((a0 ^ 64u) - a0) + 8 * fp4::kCodes;
    d1 = (int)((a1 ^ 64u) - a1) + 8 * fp4::kCodes;
    at0 = (uint32_t)(r0 * 128 + (((c & 1) * 4 ^ r0) << 4));
    at1 = (uint32_t)(r1 * 128 + (((c & 1) * 4 ^ r1) << 4));
    h = c >> 2;
    line = (c >> 1) & 1;
  }
};
struct RowPart {
  uint4 code;
  uint32_t scale;
};
template <int U>
__device__ __forceinline__ void load_rows(RowPart& x, const RowLanes& l, uint32_t block) {
  if (block == Lanes::kNone) {
    x.code = make_uint4(0u, 0u, 0u, 0u);
    x.scale = 0u;
    return;
  }
  const uint64_t at = (uint64_t)block * (uint64_t)fp4::kBlock;
  x.code = __ldcg(reinterpret_cast<const uint4*>(((U & 1) ? l.x1 : l.x0) + at + (U < 2 ? 0 : (U & 1) ? l.d1 : l.d0)));
  x.scale = __ldcg(reinterpret_cast<const unsigned short*>(((U & 1) ? l.y1 : l.y0) + at + (U < 2 ? 0 : 8 * fp4::kScales)));
}
// to: the lane's place of the row's first 16 bytes
__device__ __forceinline__ void store_rows(uint32_t to, const RowPart& x) {
  const uint32_t w[4] = {x.code.x, x.code.y, x.code.z, x.code.w};
  const uint32_t f[2] = {__byte_perm(x.scale, 0u, 0x4040u) << 7, __byte_perm(x.scale, 0u, 0x4141u) << 7};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t h[4];
    fp4::halves8(w[k], h);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = fp4::mul2(h[j], f[k >> 1]);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to ^ (uint32_t)(16 * k)), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                 : "memory");
  }
}

// the lane's places
__device__ __forceinline__ void part_places(uint32_t (&at)[4], int lane) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    at[k] = (uint32_t)((lane & 7) * 128 + ((((lane >> 3 & 1) << 2 | k) ^ (lane & 7)) << 4));
}

}  // namespace chunk4
}  // namespace spark
