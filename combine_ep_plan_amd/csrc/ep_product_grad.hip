// Backward pass of the grouped product: dz = dout act'(pre), dx = dz w,
// dw = dz^T x, dbias = column sums of dz.
#include "ep_product_device.hpp"

namespace ep {
namespace {

// --- dz and dbias -----------------------------------------------------------

constexpr int kChunkRows = 64;   // rows of one group per workgroup
constexpr int kActThreads = 128; // columns / 4

struct ActArgs {
  const uint16_t *dout, *pre;
  uint16_t* dz;   // or null
  float* parts;   // [row blocks][W], or null
  Groups g;
  int n;          // columns of dout
  int cols;
};

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + __expf(-z)); }

__device__ __forceinline__ void load4(const uint16_t* p, float (&v)[4]) {
  const uint2 u = *(const uint2*)p;
  v[0] = bf16_lo(u.x);
  v[1] = bf16_hi(u.x);
  v[2] = bf16_lo(u.y);
  v[3] = bf16_hi(u.y);
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&v)[4]) {
  *(uint2*)p = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// Row blocks before expert e's, for blocks of BR rows: the place of its parts.
template <int ACT>
__global__ __launch_bounds__(kActThreads) void act_grad_kernel(ActArgs a) {
  constexpr bool glu = ACT == EP_ACT_SWIGLU;
  __shared__ int block_at;
  Where t;
  if (!find_tile<kChunkRows, kActThreads>(a.g, a.cols, &t)) return;
  // The row block's number on the line of all groups' row blocks.
  if (a.parts) {
    __shared__ int sums[kActThreads / kWave];
    int before = 0;
    for (int e = threadIdx.x; e < t.expert; e += kActThreads)
      before += (group_of(a.g, e).rows + kChunkRows - 1) / kChunkRows;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) before += __shfl_xor(before, off);
    if (lane_id() == 0) sums[threadIdx.x / kWave] = before;
    __syncthreads();
    if (threadIdx.x == 0) {
      int s = t.at / kChunkRows;
      for (int w = 0; w < kActThreads / kWave; ++w) s += sums[w];
      block_at = s;
    }
    __syncthreads();
  }
  const int c = (t.col * kActThreads + threadIdx.x) * 4;
  if (c >= a.n) return;
  const int W = glu ? 2 * a.n : a.n;
  float s0[4] = {0, 0, 0, 0}, s1[4] = {0, 0, 0, 0};
  for (int r = 0; r < t.rows; ++r) {
    const int64_t row = t.first + r;
    float d[4], z[4], u[4], o[4];
    load4(a.dout + row * a.n + c, d);
    if constexpr (ACT == EP_ACT_NONE) {
#pragma unroll
      for (int v = 0; v < 4; ++v) s0[v] += d[v];
      continue;
    }
    load4(a.pre + row * W + c, z);
    if constexpr (glu) load4(a.pre + row * W + a.n + c, u);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if constexpr (ACT == EP_ACT_GELU) {
        const float cdf = 0.5f * erfcf(z[v] * -0.70710678118654752f);
        o[v] = d[v] * (cdf + z[v] * 0.39894228040143268f * __expf(-0.5f * z[v] * z[v]));
      } else {
        const float s = sigmoid(z[v]);
        const float slope = s * (1.0f + z[v] * (1.0f - s));
        if constexpr (glu) {
          o[v] = d[v] * u[v] * slope;
          u[v] = d[v] * z[v] * s;
          s1[v] += u[v];
        } else {
          o[v] = d[v] * slope;
        }
      }
      s0[v] += o[v];
    }
    if (a.dz) {
      store4(a.dz + row * W + c, o);
      if constexpr (glu) store4(a.dz + row * W + a.n + c, u);
    }
  }
  if (!a.parts) return;
  float* p = a.parts + (int64_t)block_at * W + c;
  *(float4*)p = float4{s0[0], s0[1], s0[2], s0[3]};
  if constexpr (glu) *(float4*)(p + a.n) = float4{s1[0], s1[1], s1[2], s1[3]};
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
__global__ __launch_bounds__(S::threads) void rows_grad_kernel(GradArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::lds_bytes];
  Where t;
  if (!find_tile<S::BR, S::threads>(a.g, a.cols, &t)) return;
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
  tile.run(p, lds_base(lds), [&](int r) { return (uint32_t)(r * line); },
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

// dw[n][c] = sum over the expert's rows r of dz[r][n] x[r][c].
template <typename S>
__global__ __launch_bounds__(S::threads) void weights_grad_kernel(GradArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::lds_bytes];
  const int tiles = a.rows * a.cols, e = blockIdx.x / tiles, at = blockIdx.x - e * tiles;
  const int r0 = at / a.cols * S::BR, c0 = at % a.cols * S::BC;
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

using RowsShape = Shape<2, 8, 4, 4, false, true, false, 2>;
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
  // The smallest tiles are 32 x 64 (columns of a SwiGLU tile), 64 x 512 in the
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
  act.cols = (p.out / 4 + kActThreads - 1) / kActThreads;
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
    a.cols = (p.in + RowsShape::BC - 1) / RowsShape::BC;
    hipLaunchKernelGGL(rows_grad_kernel<RowsShape>,
                       dim3((unsigned)tile_grid(g, RowsShape::BR, a.cols)),
                       dim3(RowsShape::threads), 0, stream, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dw) {
    a.cols = (p.in + WeightsShape::BC - 1) / WeightsShape::BC;
    hipLaunchKernelGGL(weights_grad_kernel<WeightsShape>,
                       dim3((unsigned)(experts * a.rows * a.cols)), dim3(WeightsShape::threads), 0,
                       stream, a);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace ep
