// Backward pass of the grouped product: dz = dout act'(pre), dx = dz w,
// dw = dz^T x, dbias = column sums of dz.
#include "ep_product_device.hpp"

namespace ep {
namespace {

// --- dz and dbias -----------------------------------------------------------

constexpr int kChunkRows = 32;     // rows of one group per workgroup
constexpr int kActThreads = 256;   // four rows at a time, 64 lanes of 4 columns
constexpr int kActCols = kWave * 4;

struct ActArgs {
  const uint16_t *dout, *pre;
  uint16_t* dz;   // or null
  float* parts;   // [most][W], or null
  int64_t most;   // row blocks that parts has room for: all those of a whole plan
  Groups g;
  int n;          // columns of dout
  int cols;
};

__device__ __forceinline__ void unpack4(const uint2& u, float (&v)[4]) {
  v[0] = bf16_lo(u.x);
  v[1] = bf16_hi(u.x);
  v[2] = bf16_lo(u.y);
  v[3] = bf16_hi(u.y);
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&v)[4]) {
  *(uint2*)p = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// dz of a block of rows and columns, and the columns' sums over the rows: wave
// w takes rows w, w + 4, ... HBM bounds it: 65,536 rows of 2048 + 4096 values to
// 4096 in 262 us, 5.1 TB/s. A small layer (333 tokens of 6 experts, 264 columns)
// takes 11 us, a chain: the offsets, their sum, two batches of loads, the offsets
// again for the parts' place.
template <int ACT>
__global__ __launch_bounds__(kActThreads) void act_grad_kernel(ActArgs a) {
  constexpr bool glu = ACT == EP_ACT_SWIGLU;
  constexpr int waves = kActThreads / kWave, steps = kChunkRows / waves;
  __shared__ int before[waves];
  __shared__ float room[waves][glu ? 2 : 1][kActCols];
  Where t;
  if (!find_tile<kChunkRows, kActThreads>(a.g, a.cols, &t)) return;
  const int wave = threadIdx.x / kWave, lane = lane_id();
  const int c = t.col * kActCols + lane * 4, W = glu ? 2 * a.n : a.n;
  float s[glu ? 2 : 1][4] = {};
  if (c < a.n) {
    // Rows of a wave on their way at once: a sum alone (no activation) reads 65,536
    // rows of 2048 in 54 us with all eight and 55 with four; where dz is written,
    // four take 5 to 9 % less (GELU 173 against 190 us, SwiGLU 249 against 261).
    constexpr int some = ACT == EP_ACT_NONE ? steps : 4;
#pragma unroll 1
    for (int i0 = 0; i0 < steps; i0 += some) {
      uint2 d2[some], z2[some], u2[some];
#pragma unroll
      for (int i = 0; i < some; ++i) {
        const int r = wave + (i0 + i) * waves;
        const int64_t row = t.first + r;
        d2[i] = z2[i] = u2[i] = uint2{0, 0};
        if (r >= t.rows) continue;
        d2[i] = *(const uint2*)(a.dout + row * a.n + c);
        if constexpr (ACT != EP_ACT_NONE) z2[i] = *(const uint2*)(a.pre + row * W + c);
        if constexpr (glu) u2[i] = *(const uint2*)(a.pre + row * W + a.n + c);
      }
#pragma unroll
      for (int i = 0; i < some; ++i) {
        const int r = wave + (i0 + i) * waves;
        if (r >= t.rows) continue;
        const int64_t row = t.first + r;
        float d[4], z[4], u[4], o[4];
        unpack4(d2[i], d);
        unpack4(z2[i], z);
        unpack4(u2[i], u);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if constexpr (ACT == EP_ACT_NONE) {
            o[v] = d[v];
          } else if constexpr (ACT == EP_ACT_GELU) {
            const Normal n = normal_at(z[v]);
            o[v] = d[v] * (n.below + z[v] * n.density);
          } else {
            const float sg = sigmoid(z[v]);
            const float slope = sg * (1.0f + z[v] * (1.0f - sg));
            if constexpr (glu) {
              o[v] = d[v] * u[v] * slope;
              u[v] = d[v] * z[v] * sg;
              s[1][v] += u[v];
            } else {
              o[v] = d[v] * slope;
            }
          }
          s[0][v] += o[v];
        }
        if (ACT != EP_ACT_NONE && a.dz) {
          store4(a.dz + row * W + c, o);
          if constexpr (glu) store4(a.dz + row * W + a.n + c, u);
        }
      }
    }
  }
  if (!a.parts) return;
  // The row block's number among all groups' row blocks: those of the experts
  // before, then those of its own.
  const int limit = room_of(a.g, kChunkRows);
  int mine = 0;
  for (int e = threadIdx.x; e < t.expert; e += kActThreads)
    mine = add_blocks(mine, blocks_of(a.g, e, kChunkRows, limit), limit);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) mine = add_blocks(mine, __shfl_xor(mine, off), limit);
  if (lane == 0) before[wave] = mine;
#pragma unroll
  for (int h = 0; h < (glu ? 2 : 1); ++h)
    *(float4*)&room[wave][h][lane * 4] = float4{s[h][0], s[h][1], s[h][2], s[h][3]};
  __syncthreads();
  const int64_t block = (int64_t)t.at / kChunkRows + before[0] + before[1] + before[2] + before[3];
  const int col = t.col * kActCols + threadIdx.x;
  if (col >= a.n || block >= a.most) return;  // the latter with a broken plan only
#pragma unroll
  for (int h = 0; h < (glu ? 2 : 1); ++h)
    a.parts[block * W + h * a.n + col] =
        room[0][h][threadIdx.x] + room[1][h][threadIdx.x] + room[2][h][threadIdx.x] +
        room[3][h][threadIdx.x];
}

// dbias[e][c]: the parts of e's row blocks. COLS columns per workgroup, and
// groups of COLS lanes that each take every GROUPS-th part, eight of them on
// their way at once.
template <int COLS, int GROUPS>
__global__ __launch_bounds__(COLS * GROUPS) void bias_kernel(const float* parts, int64_t most,
                                                             Groups g, float* dbias, int W) {
  constexpr int threads = COLS * GROUPS;
  __shared__ int before[threads / kWave];
  __shared__ float room[GROUPS][COLS];
  const int e = blockIdx.y, lane = threadIdx.x % COLS, group = threadIdx.x / COLS;
  const int c = blockIdx.x * COLS + lane;
  const int limit = room_of(g, kChunkRows);
  int mine = 0;
  for (int i = threadIdx.x; i < e; i += threads)
    mine = add_blocks(mine, blocks_of(g, i, kChunkRows, limit), limit);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) mine = add_blocks(mine, __shfl_xor(mine, off), limit);
  if (lane_id() == 0) before[threadIdx.x / kWave] = mine;
  __syncthreads();
  int64_t first = 0;
  for (int w = 0; w < threads / kWave; ++w) first += before[w];
  int64_t n = blocks_in(group_of(g, e).rows, kChunkRows);
  if (first + n > most) n = 0;  // of a broken plan
  float s = 0.0f;
  for (int64_t p0 = group; p0 < n; p0 += 8 * GROUPS) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t p = p0 + i * GROUPS;
      v[i] = p < n && c < W ? parts[(first + p) * W + c] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
  }
  room[group][lane] = s;
  __syncthreads();
  if (group != 0 || c >= W) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < GROUPS; ++i) s += room[i][lane];
  dbias[(int64_t)e * W + c] = s;
}

// Many parts per expert (65,536 rows of one: 2048, of 4096 columns) need many
// lanes a column, 11 against 43 us; few (64 experts of 1024 rows: 32) are one
// batch of loads for four lanes, 11 us against 74.
hipError_t run_bias(const float* parts, int64_t most, const Groups& g, float* dbias, int W,
                    hipStream_t stream) {
  const int experts = g.N * g.L;
  if (g.most / experts > 64 * kChunkRows)
    hipLaunchKernelGGL((bias_kernel<32, 32>), dim3((W + 31) / 32, experts), dim3(1024), 0, stream,
                       parts, most, g, dbias, W);
  else
    hipLaunchKernelGGL((bias_kernel<64, 4>), dim3((W + 63) / 64, experts), dim3(256), 0, stream,
                       parts, most, g, dbias, W);
  return hipGetLastError();
}

// --- products ---------------------------------------------------------------

struct GradArgs {
  const uint16_t *dz, *x, *w;
  uint16_t *dx, *dw;
  Groups g;
  int in, W;   // columns of x, of dz
  int rows, cols;
};

struct NoScale {
  __device__ __forceinline__ uint32_t operator()(int, int = 0) const { return kNowhere; }
};

// A tile's output: rows [0, rows) of `out`, columns [c0, cols) of a line of them.
template <typename S>
__device__ __forceinline__ void write_tile(const Tile<S>& tile, uint16_t* out, int rows, int c0,
                                           int cols) {
  const int lane = lane_id();
#pragma unroll
  for (int i = 0; i < S::FR; ++i) {
    const int r = (tile.wr * S::FR + i) * kFrag + lane % 16;
    uint16_t* o = out + (int64_t)r * cols;
#pragma unroll
    for (int j = 0; j < S::FC; j += 2) {
      const int c = c0 + (tile.wc * S::FC + j) * kFrag + column_of_lane();
      float v[8];
      eight_columns(tile.acc[i][j], tile.acc[i][j + 1], v);
      if (r < rows && c < cols) store8(o + c, v);
    }
  }
}

template <int FR, bool ONCE>
using RowsShape = Shape<2, FR, 4, 4, false, true, false, 2, ONCE>;
using RowsSmall = Shape<2, 4, 2, 4, false, true, false, 4>;       // 128 x 128
using RowsFlat = Shape<1, 2, 2, 4, false, true, false, 4, true>;  // 32 x 128

// 64 experts of about 1024 rows, W 4096, in 7168: dx 3.42 ms, dw 3.58 ms, 1.12
// and 1.07 PFLOP/s; the matrix units are busy 60 and 56 % of the time. As in the
// forward pass a CU's intake of operands is what the steps wait for, and groups of
// exactly 1024 rows (dx 3.17 against 3.54 ms) read 9 GB where random sizes read
// 18. The 256-row kernel spills 13 registers, outside its steps.
//
// dx[r][c] = sum over n of dz[r][n] w[n][c], for tiles of more than MIN and at
// most S::BR rows, from t on, while the line has such ones. Returns whether t is
// then a tile of another height.
template <typename S, int MIN, typename L>
__device__ __forceinline__ bool rows_tiles(const GradArgs& a, L& line_, Where& t, uint32_t lds) {
  const int line = a.W * 2, w_line = a.in * 2;
  const auto feed_of = [&](const Where& w) {
    Feed p;
    p.r = (const uint8_t*)a.dz + (int64_t)w.first * line;
    p.r_size = w.rows * line;
    p.r_off = 0;
    p.c_off = w.col * S::BC * 2;
    p.c = (const uint8_t*)a.w + (int64_t)w.expert * a.W * w_line + p.c_off;
    p.c_size = 0;
    p.left = line;
    p.rs = p.cs = nullptr;
    p.rs_size = p.cs_size = 0;
    return p;
  };
  Tile<S> tile(
      lds, line, w_line, [&](int r) { return (uint32_t)(r * line); },
      [&](int r) { return (uint32_t)(r * w_line); }, NoScale{}, NoScale{});
  Feed p = feed_of(t);
  const bool long_enough = p.steps() >= S::stages;
  for (bool primed = false;;) {
    Where n = t;
    const bool more = line_.next(&n);
    const bool same = more && n.rows > MIN && n.rows <= S::BR, chained = same && long_enough;
    const Feed after = feed_of(n);
    tile.run(p, primed, after, chained);
    write_tile(tile, a.dx + (int64_t)t.first * a.in, t.rows, t.col * S::BC, a.in);
    t = n;
    if (!same) return more;
    p = after;
    primed = chained;
  }
}

template <typename S>
__global__ __launch_bounds__(S::threads) void rows_grad_kernel(GradArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::lds_bytes];
  extern __shared__ int ends[];
  Line<S::BR, S::threads> line(a.g, a.cols, ends);
  Where t;
  bool more = line.next(&t);
  while (more) {
    if constexpr (S::BR == 256) {  // in tiles of 64, 128 and 192 rows where they hold the rows
      if (t.rows <= 64) more = rows_tiles<RowsShape<2, true>, 0>(a, line, t, lds_base(lds));
      else if (t.rows <= 128) more = rows_tiles<RowsShape<4, true>, 64>(a, line, t, lds_base(lds));
      else if (t.rows <= 192) more = rows_tiles<RowsShape<6, true>, 128>(a, line, t, lds_base(lds));
      else more = rows_tiles<S, 192>(a, line, t, lds_base(lds));
    } else {
      more = rows_tiles<S, 0>(a, line, t, lds_base(lds));
    }
  }
}

template <typename S>
hipError_t run_rows(GradArgs a, hipStream_t stream) {
  a.cols = (a.in + S::BC - 1) / S::BC;
  hipLaunchKernelGGL(rows_grad_kernel<S>, dim3(line_grid(tile_grid(a.g, S::BR, a.cols))),
                     dim3(S::threads), (size_t)a.g.N * a.g.L * 4, stream, a);
  return hipGetLastError();
}

// The tiles that cost least, of equals the smallest, as in the forward pass.
hipError_t rows_by_cost(const GradArgs& a, hipStream_t stream) {
  const int64_t large = cost_of(a.g, 256, 64, 256, a.in), small = cost_of(a.g, 128, 128, 128, a.in),
                flat = cost_of(a.g, 32, 32, 128, a.in);
  if (flat <= small && flat <= large) return run_rows<RowsFlat>(a, stream);
  if (small <= large) return run_rows<RowsSmall>(a, stream);
  return run_rows<RowsShape<8, false>>(a, stream);
}

// dw[n][c] = sum over the expert's rows r of dz[r][n] x[r][c]. The experts'
// tiles lie on a line, as those of the rows do.
template <typename S>
__global__ __launch_bounds__(S::threads) void weights_grad_kernel(GradArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::lds_bytes];
  const int tiles = a.rows * a.cols, all = tiles * a.g.N * a.g.L;
  const int line = a.W * 2, x_line = a.in * 2;
  struct At {
    int e, r0, c0;
  };
  const auto at_of = [&](int want) {
    const int e = want / tiles;
    const RowCol rc = place_of(want - e * tiles, a.rows, a.cols);
    return At{e, rc.row * S::BR, rc.col * S::BC};
  };
  const auto feed_of = [&](const At& w) {
    const Group g = group_of(a.g, w.e);
    const int first = wave_uniform(g.first), rows = wave_uniform(g.rows);
    Feed p;
    p.r_off = w.r0 * 2;
    p.c_off = w.c0 * 2;
    p.r = (const uint8_t*)a.dz + (int64_t)first * line + p.r_off;
    p.c = (const uint8_t*)a.x + (int64_t)first * x_line + p.c_off;
    p.r_size = p.c_size = 0;
    p.left = rows * 2;
    p.rs = p.cs = nullptr;
    p.rs_size = p.cs_size = 0;
    return p;
  };
  int64_t want = tile_of(0, all, gridDim.x, blockIdx.x);
  if (want < 0) return;
  Tile<S> tile(
      lds_base(lds), line, x_line,
      [&](int r) { return (uint32_t)(r * line); }, [&](int r) { return (uint32_t)(r * x_line); },
      NoScale{}, NoScale{});
  At t = at_of((int)want);
  Feed p = feed_of(t);
  int taken = 1;
  for (bool primed = false;; ++taken) {
    want = tile_of(taken, all, gridDim.x, blockIdx.x);
    const bool more = want >= 0;
    const At n = more ? at_of((int)want) : t;
    const Feed after = feed_of(n);
    const bool chained = more && after.steps() >= S::stages;
    tile.run(p, primed, after, chained);
    write_tile(tile, a.dw + ((int64_t)t.e * a.W + t.r0) * a.in, a.W - t.r0, t.c0, a.in);
    if (!more) return;
    t = n;
    p = after;
    primed = chained;
  }
}

template <typename S>
hipError_t run_weights(GradArgs a, hipStream_t stream) {
  a.rows = (a.W + S::BR - 1) / S::BR;
  a.cols = (a.in + S::BC - 1) / S::BC;
  hipLaunchKernelGGL(weights_grad_kernel<S>,
                     dim3(line_grid(((int64_t)a.g.N * a.g.L * a.rows * a.cols + 7) / 8 * 8)),
                     dim3(S::threads), 0, stream, a);
  return hipGetLastError();
}

// By the same cost; the tiles are of the matrices, E times W x in.
hipError_t weights_by_cost(const GradArgs& a, hipStream_t stream) {
  const int64_t experts = (int64_t)a.g.N * a.g.L;
  const auto cost = [&](int b) {
    return (experts * ((a.W + b - 1) / b) * ((a.in + b - 1) / b) + 255) / 256 * 2 * b;
  };
  if (cost(128) <= cost(256)) return run_weights<Shape<2, 4, 2, 4, true, true, false, 4>>(a, stream);
  return run_weights<Shape<2, 8, 4, 4, true, true, false, 2>>(a, stream);
}

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

Groups groups_of(const Dims& d) {
  const int64_t rows = (int64_t)d.N * d.cap;
  // Without the plan's offsets: as many row blocks as either form has.
  return Groups{nullptr, d.N, d.L, d.cap, rows};
}

// Row blocks, at most: dense groups or the plan's.
int64_t most_blocks(const Dims& d) {
  const Groups g = groups_of(d);
  const int64_t dense = room_of(g, kChunkRows), routed = d.NTR / kChunkRows + d.E + 8;
  return d.E == d.N && dense > routed ? dense : routed;
}

}  // namespace

// A line's tiles are given to as many workgroups as there are; their numbers,
// of 32 x 32 tiles at least, are 32-bit ones. 2^26 blocks of 32 x 64 are outputs
// of 275 GB.
bool line_fits(const Groups& g, int64_t cols) {
  return room_of(g, 32) * ((cols + 63) / 64) < (int64_t)1 << 26;
}

// One workgroup per 32 rows by 256 columns, in a grid of fewer than 2^32 threads.
bool act_grad_fits(const Groups& g, int64_t cols) {
  return tile_grid(g, kChunkRows, (cols + kActCols - 1) / kActCols) * kActThreads <
         (int64_t)1 << 32;
}

int64_t product_grad_bytes(const ep_product& p, const Dims& d) {
  const int64_t W = weight_rows(p);
  const int64_t dz = p.act == EP_ACT_NONE ? 0 : align256((int64_t)d.N * d.cap * W * 2);
  return dz + most_blocks(d) * W * 4;
}

hipError_t launch_product_grad(const ep_product& p, const Dims& d, const Groups& g,
                               const uint16_t* dout, const uint16_t* x, const uint16_t* pre,
                               void* ws, uint16_t* dx, uint16_t* dw, float* dbias,
                               hipStream_t stream) {
  const int W = (int)weight_rows(p);
  const bool none = p.act == EP_ACT_NONE;
  ActArgs act;
  act.dout = dout;
  act.pre = pre;
  act.dz = none || (!dx && !dw) ? nullptr : (uint16_t*)ws;
  act.parts =
      dbias ? (float*)((char*)ws + (none ? 0 : align256((int64_t)d.N * d.cap * W * 2))) : nullptr;
  act.most = most_blocks(d);
  act.g = g;
  act.n = p.out;
  act.cols = (p.out + kActCols - 1) / kActCols;
  hipError_t e = hipSuccess;
  if (g.most > 0 && (act.dz || act.parts)) {
    const auto kernel = p.act == EP_ACT_SWIGLU ? act_grad_kernel<EP_ACT_SWIGLU>
                        : p.act == EP_ACT_SILU ? act_grad_kernel<EP_ACT_SILU>
                        : p.act == EP_ACT_GELU ? act_grad_kernel<EP_ACT_GELU>
                                               : act_grad_kernel<EP_ACT_NONE>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)tile_grid(g, kChunkRows, act.cols)),
                       dim3(kActThreads), 0, stream, act);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dbias) {
    e = run_bias(act.parts, act.most, g, dbias, W, stream);
    if (e != hipSuccess) return e;
  }
  GradArgs a;
  a.dz = none ? dout : (const uint16_t*)ws;
  a.x = x;
  a.w = (const uint16_t*)p.w;
  a.dx = dx;
  a.dw = dw;
  a.g = g;
  a.in = p.in;
  a.W = W;
  a.rows = a.cols = 0;
  if (dx && g.most > 0) {
    e = rows_by_cost(a, stream);
    if (e != hipSuccess) return e;
  }
  if (dw) e = weights_by_cost(a, stream);
  return e;
}

}  // namespace ep
