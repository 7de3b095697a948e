// Where the tiles of the experts' products lie: rows of the groups, blocks of
// rows on a line, and the rows and columns of a place on it. Arithmetic alone,
// for the kernels and for the host, where tests/native/tile_line_check.cpp
// runs it on plans of any content.
//
// Offsets come from a plan's workspace and are taken as they are found: each
// group is cut to its rank's rows, and numbers of row blocks add up to no more
// than the groups of a whole plan can have (`room`), which is also what grids
// are made for. With a whole plan neither changes anything; with any other
// every tile is inside the buffers and their number is bounded.
#pragma once

#include "ep_kernels.hpp"

namespace ep {

// Rows [first, first + rows) of the grouped buffers.
struct Group {
  int first, rows;
};

__host__ __device__ inline Group group_of(const Groups& g, int e) {
  if (!g.off) return Group{(int)(e * g.cap), (int)g.cap};
  const int d = e / g.L, j = e - d * g.L;
  const int32_t* off = g.off + (size_t)d * (g.L + 1) + j;
  const int64_t lo = off[0] < 0 ? 0 : off[0] < g.cap ? off[0] : g.cap;
  const int64_t hi = off[1] < lo ? lo : off[1] < g.cap ? off[1] : g.cap;
  return Group{(int)(d * g.cap + lo), (int)(hi - lo)};
}

// Blocks of br rows in `rows` (fewer than 2^31) rows.
__host__ __device__ inline int blocks_in(int rows, int br) {
  return (int)(((uint32_t)rows + (uint32_t)br - 1) / (uint32_t)br);
}

// Blocks of br rows that the groups of a whole plan have at most, all together.
__host__ __device__ inline int room_of(const Groups& g, int br) {
  if (!g.off) return (int)(g.N * ((g.cap + br - 1) / br));
  const int64_t experts = (int64_t)g.N * g.L;
  return (int)(g.most / br + (experts < g.most ? experts : g.most));
}

// Blocks of an expert, and sums of blocks, within the room: in any order of
// adding a sum is the smaller of the true one and the room.
__host__ __device__ inline int blocks_of(const Groups& g, int e, int br, int room) {
  const int n = blocks_in(group_of(g, e).rows, br);
  return n < room ? n : room;
}
__host__ __device__ inline int add_blocks(int a, int b, int room) {
  return a + b < room ? a + b : room;  // room < 2^28
}

// A tile of a group's rows: `rows` of them from the group's `at`-th on, and
// the tile's column block.
struct Where {
  int expert, first, rows, at, col;
};

__host__ __device__ inline Where where_of(const Group& gr, int e, int br, int rb, int col) {
  const int at = rb * br;
  return Where{e, gr.first + at, gr.rows - at < br ? gr.rows - at : br, at, col};
}

// A workgroup's i-th tile on a line of `all`, or -1, for `grid` workgroups (a
// multiple of 8; workgroup b runs on XCD b % 8): the XCDs take turns with as
// many neighbouring tiles as they have workgroups, so that what several of
// them read is still in the memory-side cache, and share what is left at the
// end evenly.
__host__ __device__ inline int64_t tile_of(int i, int64_t all, int grid, int block) {
  const int slots = grid / 8, xcd = block % 8, slot = block / 8;
  const int64_t before = (int64_t)i * 8 * slots, left = all - before;
  if (left >= 8 * slots) return before + xcd * slots + slot;
  const int each = (int)((left + 7) / 8);
  return left > 0 && slot < each && xcd * each + slot < left ? before + xcd * each + slot : -1;
}

// Row block and column block of the at-th tile of blocks x cols: the tiles go by
// stripes of 16 columns, in those by four rows, in those by 8 columns, so that
// 32 neighbours, an XCD's at one time, are 4 x 8 and need 12 blocks of operands.
struct RowCol {
  int row, col;
};
__host__ __device__ inline RowCol place_of(int at, int blocks, int cols) {
  const int stripe = at / (blocks * 16), in = at - stripe * blocks * 16;
  const int wide = cols - stripe * 16 < 16 ? cols - stripe * 16 : 16;
  const int four = in / (4 * wide), rows = blocks - 4 * four < 4 ? blocks - 4 * four : 4;
  const int left = wide < 8 ? wide : 8, i = in - four * 4 * wide, j = i - rows * left;
  return j < 0 ? RowCol{4 * four + i / left, stripe * 16 + i % left}
               : RowCol{4 * four + j / (wide - left), stripe * 16 + left + j % (wide - left)};
}

// Tile `want` of a line of blocks x cols tiles per expert, `before` row blocks
// of which lie before expert e's. No rows where e has no such tile: only when
// the offsets change while the kernel runs.
__host__ __device__ inline Where tile_at(const Groups& g, int br, int e, int before, int64_t want,
                                         int cols) {
  const Group gr = group_of(g, e);
  const int blocks = blocks_in(gr.rows, br);
  const int64_t at = want - (int64_t)before * cols;
  if (at < 0 || at >= (int64_t)blocks * cols) return Where{e, gr.first, 0, 0, 0};
  const RowCol rc = place_of((int)at, blocks, cols);
  return where_of(gr, e, br, rc.row, rc.col);
}

// The elementwise part's order of the same tiles (see find_tile): the at-th of
// an expert's blocks x cols, by stripes of eight column blocks, row blocks
// inside.
__host__ __device__ inline RowCol stripe_of(int at, int blocks, int cols) {
  const int stripe = at / (blocks * 8);
  const int wide = cols - stripe * 8 < 8 ? cols - stripe * 8 : 8;
  const int in = at - stripe * blocks * 8;
  return RowCol{in / wide, stripe * 8 + in % wide};
}

}  // namespace ep
