// The products' tiles, on the host: the kernels' own arithmetic (ep_tiles.hpp)
// on whole plans and on offsets of any value.
//
// Whole plans: every tile of every group has one workgroup, and one place.
// Any offsets: a bounded number of tiles, each inside its rank's rows and the
// matrix's columns; sums of blocks do not depend on the order of adding. (The
// parts of the backward pass hold as many row blocks as a plan has room for,
// so numbers of blocks inside the room are inside the parts.)
#include <algorithm>
#include <climits>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "ep_tiles.hpp"

using namespace ep;

static std::mt19937_64 rng(7);
static int64_t pick(int64_t lo, int64_t hi) { return std::uniform_int_distribution<int64_t>(lo, hi)(rng); }
// By magnitude, so that small and large numbers are equally likely.
static int64_t spread(int64_t lo, int64_t hi) {
  const int64_t top = std::min(hi, lo + ((int64_t)1 << pick(0, 62 - __builtin_clzll(hi - lo + 2))));
  return pick(lo, std::max(lo, top));
}

#define CHECK(x)                                                              \
  do {                                                                        \
    if (!(x)) {                                                               \
      std::printf("line %d: %s\n", __LINE__, #x);                             \
      std::exit(1);                                                           \
    }                                                                         \
  } while (0)

struct Plan {
  std::vector<int32_t> off;
  Groups g;
  bool whole;
};

static Plan make_plan(int kind) {
  Plan p;
  const int N = (int)pick(1, 8), L = (int)spread(1, 256);
  const int64_t cap = spread(1, (((int64_t)1 << 31) - 1) / N);
  p.off.resize((size_t)N * (L + 1));
  p.whole = kind == 0;
  int64_t rows = 0;
  for (int d = 0; d < N; ++d) {
    int32_t* o = &p.off[(size_t)d * (L + 1)];
    const int64_t top = std::min<int64_t>(cap, spread(1, 40000));
    for (int j = 0; j <= L; ++j) {
      switch (kind) {
        case 0: o[j] = (int32_t)pick(0, top); break;                                  // sorted below
        case 1: o[j] = (int32_t)(j % 2 ? cap : 0); break;                             // every other group is all rows
        case 2: o[j] = (int32_t)(cap - cap * j / L); break;                           // descending
        case 3: o[j] = j % 2 ? INT_MAX : (int32_t)pick(INT_MIN, 0); break;
        case 4: o[j] = (int32_t)pick(INT_MIN, INT_MAX); break;
        default: o[j] = (int32_t)pick(0, cap); break;
      }
    }
    if (kind == 0) {
      std::sort(o, o + L + 1);
      if (pick(0, 1)) std::fill(o, o + (L + 1) / 2, o[0]);                            // empty groups
      o[0] = 0;
      rows += o[L];
    }
  }
  // No more rows than the slots of the call, or than there is room for.
  const int64_t slots = kind == 0 ? rows + pick(0, 50) : spread(1, (int64_t)1 << 26);
  p.g = Groups{p.off.data(), N, L, cap, std::min(slots, N * cap)};
  if (kind == 6) {
    p.g = Groups{nullptr, N, 1, std::min<int64_t>(cap, 30000), 0};
    p.g.most = p.g.N * p.g.cap;
    p.whole = true;
  }
  return p;
}

static void check_where(const Plan& p, const Where& t, int br, int cols) {
  const Groups& g = p.g;
  CHECK(t.expert >= 0 && t.expert < g.N * g.L);
  const int64_t lo = t.expert / g.L * g.cap;
  CHECK(t.rows >= (p.whole ? 1 : 0) && t.rows <= br && t.at >= 0);
  CHECK(t.first >= lo && t.first + (int64_t)t.rows <= lo + g.cap);
  CHECK(t.col >= 0 && t.col < cols);
}

int main() {
  int64_t seen = 0;
  for (int trial = 0; trial < 3000; ++trial) {
    const Plan p = make_plan(trial % 7);
    const Groups& g = p.g;
    const int br = 32 << pick(0, 3), cols = (int)spread(1, 200), experts = g.N * g.L;
    const int room = room_of(g, br);
    CHECK(room >= 0 && room < 1 << 28);
    std::vector<int> ends(experts);
    int64_t true_sum = 0;
    int sum = 0;
    for (int e = 0; e < experts; ++e) {
      const Group gr = group_of(g, e);
      const int64_t lo = e / g.L * g.cap;
      CHECK(gr.rows >= 0 && gr.first >= lo && gr.first + (int64_t)gr.rows <= lo + g.cap);
      CHECK(blocks_in(gr.rows, br) == ((int64_t)gr.rows + br - 1) / br);
      true_sum += blocks_in(gr.rows, br);
      ends[e] = sum = add_blocks(sum, blocks_of(g, e, br, room), room);
      CHECK(sum == std::min<int64_t>(true_sum, room));
    }
    if (p.whole) CHECK(true_sum <= room);
    // The same from the back, and by halves.
    int back = 0, half[2] = {0, 0};
    for (int e = experts - 1; e >= 0; --e) back = add_blocks(back, blocks_of(g, e, br, room), room);
    for (int e = 0; e < experts; ++e)
      half[e % 2] = add_blocks(half[e % 2], blocks_of(g, e, br, room), room);
    CHECK(back == sum && add_blocks(half[0], half[1], room) == sum);

    // The line: all its tiles if there are few, else some.
    const int64_t tiles = (int64_t)sum * cols;
    const int grid = (int)std::min<int64_t>(256, (room * (int64_t)cols + 7) / 8 * 8);
    const bool all = tiles <= 60000;
    std::vector<std::vector<char>> had(all && p.whole ? experts : 0);
    for (size_t e = 0; e < had.size(); ++e)
      had[e].assign((size_t)blocks_in(group_of(g, (int)e).rows, br) * cols, 0);
    int64_t given = 0;
    std::vector<char> turn(all ? tiles : 0, 0);
    for (int b = 0; b < grid; ++b)
      for (int i = 0;; ++i) {
        int64_t want;
        if (all) {
          want = tile_of(i, tiles, grid, b);
          if (want < 0) break;
          CHECK(want < tiles && !turn[want]);
          turn[want] = 1;
        } else {
          if (i == 2) break;
          want = pick(0, tiles - 1);
        }
        ++given;
        const int block = (int)(want / cols);
        const int e = (int)(std::upper_bound(ends.begin(), ends.end(), block) - ends.begin());
        CHECK(e < experts);
        const Where t = tile_at(g, br, e, e > 0 ? ends[e - 1] : 0, want, cols);
        check_where(p, t, br, cols);
        CHECK(t.rows > 0 && t.expert == e);
        if (!had.empty()) {
          char& h = had[e][(size_t)(t.at / br) * cols + t.col];
          CHECK(!h);
          h = 1;
        }
        // The elementwise part's order.
        const Group gr = group_of(g, e);
        const int64_t left = want - (int64_t)(e > 0 ? ends[e - 1] : 0) * cols;
        if (left < INT_MAX / 8) {
          const RowCol rc = stripe_of((int)left, blocks_in(gr.rows, br), cols);
          check_where(p, where_of(gr, e, br, rc.row, rc.col), br, cols);
        }
      }
    if (all) CHECK(given == tiles);
    for (const auto& h : had) CHECK(std::count(h.begin(), h.end(), 1) == (int64_t)h.size());
    // A place that an expert does not have: offsets that changed under way.
    const int e = (int)pick(0, experts - 1);
    const int64_t far = pick(-((int64_t)1 << 40), (int64_t)1 << 40);
    const Where t = tile_at(g, br, e, (int)pick(0, room), far, cols);
    CHECK(t.rows >= 0 && t.rows <= br && t.col >= 0 && t.col < cols);
    seen += given;
  }
  std::printf("tiles %lld\n", (long long)seen);
  return 0;
}
