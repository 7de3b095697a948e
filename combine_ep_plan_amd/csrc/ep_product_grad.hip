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
  float* parts;   // [row blocks][W], or null
  Groups g;
  int n;          // columns of dout
  int cols;
};

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + __expf(-z)); }

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
// w takes rows w, w + 4, ..., all of them on their way at once.
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
    uint2 d2[steps], z2[steps], u2[steps];
#pragma unroll
    for (int i = 0; i < steps; ++i) {
      const int r = wave + i * waves;
      const int64_t row = t.first + r;
      d2[i] = z2[i] = u2[i] = uint2{0, 0};
      if (r >= t.rows) continue;
      d2[i] = *(const uint2*)(a.dout + row * a.n + c);
      if constexpr (ACT != EP_ACT_NONE) z2[i] = *(const uint2*)(a.pre + row * W + c);
      if constexpr (glu) u2[i] = *(const uint2*)(a.pre + row * W + a.n + c);
    }
#pragma unroll
    for (int i = 0; i < steps; ++i) {
      const int r = wave + i * waves;
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
          const float cdf = 0.5f * erfcf(z[v] * -0.70710678118654752f);
          o[v] = d[v] * (cdf + z[v] * 0.39894228040143268f * __expf(-0.5f * z[v] * z[v]));
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
  if (!a.parts) return;
  // The row block's number among all groups' row blocks: those of the experts
  // before, then those of its own.
  int mine = 0;
  for (int e = threadIdx.x; e < t.expert; e += kActThreads)
    mine += (group_of(a.g, e).rows + kChunkRows - 1) / kChunkRows;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) mine += __shfl_xor(mine, off);
  if (lane == 0) before[wave] = mine;
#pragma unroll
  for (int h = 0; h < (glu ? 2 : 1); ++h)
    *(float4*)&room[wave][h][lane * 4] = float4{s[h][0], s[h][1], s[h][2], s[h][3]};
  __syncthreads();
  const int block = t.at / kChunkRows + before[0] + before[1] + before[2] + before[3];
  const int col = t.col * kActCols + threadIdx.x;
  if (col >= a.n) return;
#pragma unroll
  for (int h = 0; h < (glu ? 2 : 1); ++h)
    a.parts[(int64_t)block * W + h * a.n + col] =
        room[0][h][threadIdx.x] + room[1][h][threadIdx.x] + room[2][h][threadIdx.x] +
        room[3][h][threadIdx.x];
}

// dbias[e][c]: the parts of e's row blocks, in order.
__global__ __launch_bounds__(256) void bias_kernel(const float* parts, Groups g, float* dbias,
                                                   int W) {
  __shared__ int sums[256 / kWave];
  const int e = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
  int before = 0;
  for (int i = threadIdx.x; i < e; i += 256)
    before += (group_of(g, i).rows + kChunkRows - 1) / kChunkRows;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) before += __shfl_xor(before, off);
  if (lane_id() == 0) sums[threadIdx.x / kWave] = before;
  __syncthreads();
  const int first = sums[0] + sums[1] + sums[2] + sums[3];
  const int n = (group_of(g, e).rows + kChunkRows - 1) / kChunkRows;
  if (c >= W) return;
  float s = 0.0f;
  for (int i = 0; i < n; ++i) s += parts[(int64_t)(first + i) * W + c];
  dbias[(int64_t)e * W + c] = s;
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

// dx[r][c] = sum over n of dz[r][n] w[n][c].
template <typename S>
__device__ __forceinline__ void rows_tile(const GradArgs& a, const Where& t, uint32_t lds) {
  const int c0 = t.col * S::BC;
  const int64_t line = (int64_t)a.W * 2, w_line = (int64_t)a.in * 2;
  Pair p;
  p.r = (const uint8_t*)a.dz + t.first * line;
  p.r_size = t.rows * line;
  p.r_step = kStep;
  p.c = (const uint8_t*)a.w + (int64_t)t.expert * a.W * w_line + c0 * 2;
  p.c_size = a.W * w_line - c0 * 2;
  p.c_step = kStep / 2 * w_line;
  p.r_line = (uint32_t)line;
  p.c_line = (uint32_t)w_line;
  p.turn = t.col % 8;
  p.k_bytes = line;
  p.rs = p.cs = nullptr;
  p.rs_size = p.cs_size = 0;
  Tile<S> tile;
  tile.run(p, lds, [&](int r) { return (uint32_t)(r * line); },
           [&](int r) { return (uint32_t)(r * w_line); }, NoScale{}, NoScale{});
  const int lane = lane_id();
#pragma unroll
  for (int i = 0; i < S::FR; ++i) {
    const int r = (tile.wr * S::FR + i) * kFrag + lane % 16;
    if (r >= t.rows) continue;
    uint16_t* o = a.dx + (int64_t)(t.first + r) * a.in;
#pragma unroll
    for (int j = 0; j < S::FC; ++j) {
      const int c = c0 + (tile.wc * S::FC + j) * kFrag + lane / 16 * 4;
      const float v[4] = {tile.acc[i][j][0], tile.acc[i][j][1], tile.acc[i][j][2],
                          tile.acc[i][j][3]};
      if (c < a.in) store4(o + c, v);
    }
  }
}

template <int FR, bool ONCE>
using RowsShape = Shape<2, FR, 4, 4, false, true, false, 2, ONCE>;

__global__ __launch_bounds__(512) void rows_grad_kernel(GradArgs a) {
  using S = RowsShape<8, false>;
  static_assert(S::threads == 512, "");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::lds_bytes];
  Where t;
  if (!find_tile<S::BR, S::threads>(a.g, a.cols, &t)) return;
  if (t.rows <= 64) rows_tile<RowsShape<2, true>>(a, t, lds_base(lds));
  else if (t.rows <= 128) rows_tile<RowsShape<4, true>>(a, t, lds_base(lds));
  else if (t.rows <= 192) rows_tile<RowsShape<6, true>>(a, t, lds_base(lds));
  else rows_tile<S>(a, t, lds_base(lds));
}

// dw[n][c] = sum over the expert's rows r of dz[r][n] x[r][c].
template <typename S>
__global__ __launch_bounds__(S::threads) void weights_grad_kernel(GradArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::lds_bytes];
  // The experts' tiles lie on a line that the XCDs share, as in find_tile.
  const int tiles = a.rows * a.cols, all = tiles * a.g.N * a.g.L, stretch = (all + 7) / 8;
  const int slot = blockIdx.x / 8, want = blockIdx.x % 8 * stretch + slot;
  if (slot >= stretch || want >= all) return;
  const int e = want / tiles, at = want - e * tiles, stripe = at / (a.rows * 8);
  const int wide = a.cols - stripe * 8 < 8 ? a.cols - stripe * 8 : 8;
  const int in = at - stripe * a.rows * 8;
  const int r0 = in / wide * S::BR, c0 = (stripe * 8 + in % wide) * S::BC;
  const Group g = group_of(a.g, e);
  const int first = wave_uniform(g.first), rows = wave_uniform(g.rows);
  const int64_t line = (int64_t)a.W * 2, x_line = (int64_t)a.in * 2;
  Pair p;
  p.r = (const uint8_t*)a.dz + first * line + r0 * 2;
  p.r_size = rows * line - r0 * 2;
  p.r_step = kStep / 2 * line;
  p.c = (const uint8_t*)a.x + first * x_line + c0 * 2;
  p.c_size = rows * x_line - c0 * 2;
  p.c_step = kStep / 2 * x_line;
  p.r_line = (uint32_t)line;
  p.c_line = (uint32_t)x_line;
  p.turn = 0;
  p.k_bytes = (int64_t)rows * 2;
  p.rs = p.cs = nullptr;
  p.rs_size = p.cs_size = 0;
  Tile<S> tile;
  tile.run(p, lds_base(lds), [&](int r) { return (uint32_t)(r * line); },
           [&](int r) { return (uint32_t)(r * x_line); }, NoScale{}, NoScale{});
  const int lane = lane_id();
#pragma unroll
  for (int i = 0; i < S::FR; ++i) {
    const int r = r0 + (tile.wr * S::FR + i) * kFrag + lane % 16;
    if (r >= a.W) continue;
    uint16_t* o = a.dw + ((int64_t)e * a.W + r) * a.in;
#pragma unroll
    for (int j = 0; j < S::FC; ++j) {
      const int c = c0 + (tile.wc * S::FC + j) * kFrag + lane / 16 * 4;
      const float v[4] = {tile.acc[i][j][0], tile.acc[i][j][1], tile.acc[i][j][2],
                          tile.acc[i][j][3]};
      if (c < a.in) store4(o + c, v);
    }
  }
}

using WeightsShape = Shape<2, 8, 4, 4, true, true, false, 2>;

int64_t blocks_of(const Groups& g) { return tile_grid(g, kChunkRows, 1); }

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

Groups groups_of(const Dims& d) {
  const int64_t rows = (int64_t)d.N * d.cap;
  // Without the plan's offsets: as many row blocks as either form has.
  return Groups{nullptr, d.N, d.L, d.cap, rows};
}

// Row blocks, at most: dense groups or the plan's.
int64_t most_blocks(const Dims& d) {
  const Groups g = groups_of(d);
  const int64_t dense = blocks_of(g), routed = d.NTR / kChunkRows + d.E + 8;
  return d.E == d.N && dense > routed ? dense : routed;
}

}  // namespace

bool product_fits(const ep_product& p, const Dims& d) {
  // The smallest tiles are 32 x 64 (columns of a SwiGLU tile), 32 x 256 in the
  // elementwise part; no workgroup has more than 512 threads.
  const int64_t rows = d.NTR > d.N * d.cap ? d.NTR : d.N * d.cap;
  const int64_t most = (int64_t)1 << 23, W = weight_rows(p);
  const int64_t tiles = (rows / 32 + d.E + 8) * ((p.out + 63) / 64);
  const int64_t back = (rows / 256 + d.E + 8) * ((p.in + 255) / 256);
  const int64_t weights = d.E * ((W + 255) / 256) * ((p.in + 255) / 256);
  return tiles < most && back < most && weights < most;
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
  const int W = (int)weight_rows(p), experts = d.E;
  const bool none = p.act == EP_ACT_NONE;
  ActArgs act;
  act.dout = dout;
  act.pre = pre;
  act.dz = none || (!dx && !dw) ? nullptr : (uint16_t*)ws;
  act.parts =
      dbias ? (float*)((char*)ws + (none ? 0 : align256((int64_t)d.N * d.cap * W * 2))) : nullptr;
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
    hipLaunchKernelGGL(bias_kernel, dim3((W + 255) / 256, experts), dim3(256), 0, stream,
                       act.parts, g, dbias, W);
    e = hipGetLastError();
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
  a.rows = (W + WeightsShape::BR - 1) / WeightsShape::BR;
  if (dx && g.most > 0) {
    using S = RowsShape<8, false>;
    a.cols = (p.in + S::BC - 1) / S::BC;
    hipLaunchKernelGGL(rows_grad_kernel, dim3((unsigned)tile_grid(g, S::BR, a.cols)),
                       dim3(S::threads), 0, stream, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dw) {
    a.cols = (p.in + WeightsShape::BC - 1) / WeightsShape::BC;
    hipLaunchKernelGGL(weights_grad_kernel<WeightsShape>,
                       dim3((unsigned)((experts * a.rows * a.cols + 7) / 8 * 8)),
                       dim3(WeightsShape::threads), 0,
                       stream, a);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace ep
