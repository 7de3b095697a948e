// Grouped product of the experts: out = act(x w^T + bias) + residual.
#include "ep_product_device.hpp"

namespace ep {
namespace {

struct FwdArgs {
  const uint8_t *x, *w;
  const float *xs, *ws;
  const uint16_t *bias, *residual;
  uint16_t *pre, *out;
  Groups g;
  int in, n, cols;  // cols: column blocks
};

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == EP_ACT_SILU) return z * sigmoid(z);
  if constexpr (ACT == EP_ACT_GELU) return 0.5f * z * erfcf(z * -0.70710678118654752f);
  return z;
}

__device__ __forceinline__ void add4(float (&v)[4], const uint16_t* p) {
  const uint2 u = *(const uint2*)p;
  v[0] += bf16_lo(u.x);
  v[1] += bf16_hi(u.x);
  v[2] += bf16_lo(u.y);
  v[3] += bf16_hi(u.y);
}

__device__ __forceinline__ void store4(uint16_t* p, const float (&v)[4]) {
  *(uint2*)p = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// One tile. Fragments of a SwiGLU tile alternate: 16 gate rows of w, the 16 up
// rows of the same columns; a lane then holds both of a column.
template <typename S, int ACT>
__device__ __forceinline__ void product_tile(const FwdArgs& a, const Where& t, uint32_t lds) {
  constexpr bool glu = ACT == EP_ACT_SWIGLU;
  constexpr int es = S::FP8 ? 1 : 2, per_tile = glu ? S::BC / 2 : S::BC;
  const int c0 = t.col * per_tile, wrows = glu ? 2 * a.n : a.n;
  const int64_t line = (int64_t)a.in * es;
  const uint8_t* w = a.w + (int64_t)t.expert * wrows * line;
  // Weight row of row r of the tile, beside the tile's first.
  const auto w_row = [&](int r) { return glu ? r / 32 * 16 + r % 16 + (r & 16 ? a.n : 0) : r; };
  Pair p;
  p.r = a.x + (int64_t)t.first * line;
  p.c = w + c0 * line;
  p.r_size = t.rows * line;
  p.c_size = (int64_t)(wrows - c0) * line;
  p.r_step = p.c_step = kStep;
  p.r_line = p.c_line = (uint32_t)line;
  p.turn = t.col % 8;
  p.k_bytes = line;
  p.rs = p.cs = nullptr;
  p.rs_size = p.cs_size = 0;
  const int kb = a.in / 128;
  if constexpr (S::FP8) {
    p.rs = a.xs + (int64_t)t.first * kb;
    p.rs_size = (int64_t)t.rows * kb * 4;
    p.cs = a.ws + (int64_t)t.expert * (wrows / 128) * kb;
    p.cs_size = (int64_t)(wrows / 128) * kb * 4;
  }
  Tile<S> tile;
  tile.run(
      p, lds, [&](int r) { return (uint32_t)(r * line); },
      [&](int r) { return (uint32_t)(w_row(r) * line); },
      [&](int r) { return (uint32_t)(r * kb * 4); },
      [&](int wc, int f) {
        return (uint32_t)((c0 + w_row((wc * S::FC + f) * kFrag)) / 128 * kb * 4);
      });
  const int lane = lane_id();
  const uint16_t* bias = a.bias ? a.bias + (int64_t)t.expert * wrows : nullptr;
#pragma unroll
  for (int i = 0; i < S::FR; ++i) {
    const int r = (tile.wr * S::FR + i) * kFrag + lane % 16;
    if (r >= t.rows) continue;
    const int64_t row = t.first + r;
#pragma unroll
    for (int j = 0; j < S::FC; j += glu ? 2 : 1) {
      const int f = tile.wc * S::FC + j, c = c0 + (glu ? f / 2 : f) * kFrag + lane / 16 * 4;
      if (c >= a.n) continue;
      float z[4], y[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) z[v] = tile.acc[i][j][v];
      if (bias) add4(z, bias + c);
      if (a.pre) store4(a.pre + row * wrows + c, z);
      if constexpr (glu) {
        float up[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) up[v] = tile.acc[i][j + 1][v];
        if (bias) add4(up, bias + a.n + c);
        if (a.pre) store4(a.pre + row * wrows + a.n + c, up);
#pragma unroll
        for (int v = 0; v < 4; ++v) y[v] = activate<EP_ACT_SILU>(z[v]) * up[v];
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) y[v] = activate<ACT>(z[v]);
      }
      if (a.residual) add4(y, a.residual + row * a.n + c);
      store4(a.out + row * a.n + c, y);
    }
  }
}

// S: the kernel's largest tile; T...: smaller ones, in ascending order, of
// which the first that holds the rows is taken.
template <int ACT, typename S>
__device__ __forceinline__ void pick_tile(const FwdArgs& a, const Where& t, uint32_t lds) {
  product_tile<S, ACT>(a, t, lds);
}
template <int ACT, typename S, typename T, typename... U>
__device__ __forceinline__ void pick_tile(const FwdArgs& a, const Where& t, uint32_t lds) {
  if (t.rows <= T::BR) product_tile<T, ACT>(a, t, lds);
  else pick_tile<ACT, S, U...>(a, t, lds);
}

template <typename... S>
constexpr int most_lds() {
  int most = 0;
  ((most = S::lds_bytes > most ? S::lds_bytes : most), ...);
  return most;
}

template <int ACT, typename S, typename... T>
__global__ __launch_bounds__(S::threads) void product_kernel(FwdArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[most_lds<S, T...>()];
  static_assert(((T::threads == S::threads && T::BC == S::BC) && ...),
                "the smaller tiles are the largest one's with fewer rows");
  Where t;
  if (!find_tile<S::BR, S::threads>(a.g, a.cols, &t)) return;
  pick_tile<ACT, S, T...>(a, t, lds_base(lds));
}

template <typename S, typename... T>
hipError_t run(FwdArgs a, int act, hipStream_t stream) {
  const int per_tile = act == EP_ACT_SWIGLU ? S::BC / 2 : S::BC;
  a.cols = (a.n + per_tile - 1) / per_tile;
  const auto kernel = act == EP_ACT_SWIGLU ? product_kernel<EP_ACT_SWIGLU, S, T...>
                      : act == EP_ACT_SILU ? product_kernel<EP_ACT_SILU, S, T...>
                      : act == EP_ACT_GELU ? product_kernel<EP_ACT_GELU, S, T...>
                                           : product_kernel<EP_ACT_NONE, S, T...>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)tile_grid(a.g, S::BR, a.cols)), dim3(S::threads), 0,
                     stream, a);
  return hipGetLastError();
}

template <int FR, bool FP8, int STAGES, bool ONCE = true>
using Rows = Shape<2, FR, 4, 4, false, false, FP8, STAGES, ONCE>;

template <bool FP8>
hipError_t by_rows(const FwdArgs& a, int act, hipStream_t stream) {
  const int64_t mean = a.g.most / (a.g.N * a.g.L);
  if (mean <= 24) return run<Shape<1, 2, 2, 4, false, false, FP8, 4, true>>(a, act, stream);
  return run<Rows<8, FP8, 2, false>, Rows<2, FP8, 3>, Rows<4, FP8, 3>, Rows<6, FP8, 2>>(a, act, stream);
}

}  // namespace

hipError_t launch_product(const ep_product& p, const Groups& g, const void* const x[2],
                          const void* residual, void* pre, void* out, hipStream_t stream) {
  FwdArgs a;
  a.x = (const uint8_t*)x[0];
  a.xs = (const float*)x[1];
  a.w = (const uint8_t*)p.w;
  a.ws = p.w_scale;
  a.bias = (const uint16_t*)p.bias;
  a.residual = (const uint16_t*)residual;
  a.pre = (uint16_t*)pre;
  a.out = (uint16_t*)out;
  a.g = g;
  a.in = p.in;
  a.n = p.out;
  a.cols = 0;
  return p.dtype == EP_DTYPE_E4M3 ? by_rows<true>(a, p.act, stream)
                                  : by_rows<false>(a, p.act, stream);
}

}  // namespace ep
