// Grouped product of the experts: out = act(x w^T + bias) + residual, the
// epilogue applied to the 32-bit sums in registers.
//
// Few rows an expert: the weights' way from HBM bounds it. 256 experts of 128
// rows (7168 values to 2048 by SwiGLU): 3.1 ms, 15.6 GB at 5.0 TB/s; e4m3 1.7 ms.
// Many rows: the matrix units are busy 62 % (e4m3 50 %) of the time, and wait for
// operands from L2 and behind it in the rest. 256 experts of about 1024 rows take 13.6
// ms in bf16 (1.13 PFLOP/s) and 8.1 to 8.4 in e4m3 (1.8 to 1.9); of exactly 1024
// each 11.9 (1.29) and 7.3 (2.1), and read 23 and 11 GB where random sizes read
// 43 and 29: likely neighbouring tiles of different heights leave step over 56 or
// 112 steps of k and no longer find each other's operands in L2. e4m3's scaling, 128
// FMAs beside 32 matrix instructions a step, is about half the matrix work. One
// dense product of 16,384 rows of 7168 to 8192: 1.41 to 1.50 ms, 1.28 to 1.37
// PFLOP/s.
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

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == EP_ACT_SILU) return z * sigmoid(z);
  if constexpr (ACT == EP_ACT_GELU) return z * normal_at(z).below;
  return z;
}

// A tile's output. Fragments of a SwiGLU tile alternate: 16 gate rows of w, the
// 16 up rows of the same columns; a lane then holds both of a column.
template <typename S, int ACT>
__device__ __forceinline__ void write_tile(const FwdArgs& a, const Tile<S>& tile, const Where& t) {
  constexpr bool glu = ACT == EP_ACT_SWIGLU;
  const int lane = lane_id(), c0 = t.col * (glu ? S::BC / 2 : S::BC);
  const int wrows = glu ? 2 * a.n : a.n;
  const uint16_t* bias = a.bias ? a.bias + (int64_t)t.expert * wrows : nullptr;
#pragma unroll
  for (int i = 0; i < S::FR; ++i) {
    const int r = (tile.wr * S::FR + i) * kFrag + lane % 16;
    const bool there = r < t.rows;
    const int64_t row = t.first + r;
#pragma unroll
    for (int j = 0; j < S::FC; j += glu ? 4 : 2) {
      const int f = tile.wc * S::FC + j, c = c0 + (glu ? f / 2 : f) * kFrag + column_of_lane();
      float y[8];
      eight_columns(tile.acc[i][j], tile.acc[i][j + (glu ? 2 : 1)], y);
      float up[8];
      if constexpr (glu) eight_columns(tile.acc[i][j + 1], tile.acc[i][j + 3], up);
      if (!there || c >= a.n) continue;
      if (bias) add8(y, bias + c);
      if (a.pre) store8(a.pre + row * wrows + c, y);
      if constexpr (glu) {
        if (bias) add8(up, bias + a.n + c);
        if (a.pre) store8(a.pre + row * wrows + a.n + c, up);
#pragma unroll
        for (int v = 0; v < 8; ++v) y[v] = activate<EP_ACT_SILU>(y[v]) * up[v];
      } else {
#pragma unroll
        for (int v = 0; v < 8; ++v) y[v] = activate<ACT>(y[v]);
      }
      if (a.residual) add8(y, a.residual + row * a.n + c);
      store8(a.out + row * a.n + c, y);
    }
  }
}

// Tiles of more than MIN and at most S::BR rows, from t on, while the line has
// such ones. Returns whether t is then a tile of another height.
template <typename S, int ACT, int MIN, typename L>
__device__ __forceinline__ bool run_tiles(const FwdArgs& a, L& line_, Where& t, uint32_t lds) {
  constexpr bool glu = ACT == EP_ACT_SWIGLU;
  constexpr int es = S::FP8 ? 1 : 2, per_tile = glu ? S::BC / 2 : S::BC;
  const int wrows = glu ? 2 * a.n : a.n, kb = a.in / 128;
  const int line = a.in * es;
  // Weight row of row r of the tile, beside the tile's first.
  const auto w_row = [&](int r) { return glu ? r / 32 * 16 + r % 16 + (r & 16 ? a.n : 0) : r; };
  const auto feed_of = [&](const Where& w) {
    const int c0 = w.col * per_tile;
    Feed p;
    p.r = a.x + (int64_t)w.first * line;
    p.c = a.w + ((int64_t)w.expert * wrows + c0) * line;
    p.r_size = w.rows * line;
    p.c_size = (wrows - c0) * line;
    p.r_off = p.c_off = 0;
    p.left = line;
    p.rs = p.cs = nullptr;
    p.rs_size = p.cs_size = 0;
    if constexpr (S::FP8) {
      const int64_t block = (int64_t)w.expert * (wrows / 128) + c0 / 128;
      p.rs = a.xs + (int64_t)w.first * kb;
      p.rs_size = w.rows * kb * 4;
      p.cs = a.ws + block * kb;
      p.cs_size = (wrows / 128 - c0 / 128) * kb * 4;
    }
    return p;
  };
  Tile<S> tile(
      lds, line, line, [&](int r) { return (uint32_t)(r * line); },
      [&](int r) { return (uint32_t)(w_row(r) * line); },
      [&](int r) { return (uint32_t)(r * kb * 4); },
      [&](int wc, int f) { return (uint32_t)(w_row((wc * S::FC + f) * kFrag) / 128 * kb * 4); });
  Feed p = feed_of(t);
  const bool long_enough = p.steps() >= S::stages;
  for (bool primed = false;;) {
    Where n = t;
    const bool more = line_.next(&n);
    const bool same = more && n.rows > MIN && n.rows <= S::BR, chained = same && long_enough;
    const Feed after = feed_of(n);
    tile.run(p, primed, after, chained);
    write_tile<S, ACT>(a, tile, t);
    t = n;
    if (!same) return more;
    p = after;
    primed = chained;
  }
}

// S: the kernel's largest tile; T...: smaller ones, in ascending order.
template <int ACT, int MIN, typename S, typename L>
__device__ __forceinline__ bool pick_tiles(const FwdArgs& a, L& line, Where& t, uint32_t lds) {
  return run_tiles<S, ACT, MIN>(a, line, t, lds);
}
template <int ACT, int MIN, typename S, typename T, typename... U, typename L>
__device__ __forceinline__ bool pick_tiles(const FwdArgs& a, L& line, Where& t, uint32_t lds) {
  if (t.rows <= T::BR) return run_tiles<T, ACT, MIN>(a, line, t, lds);
  return pick_tiles<ACT, T::BR, S, U...>(a, line, t, lds);
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
  extern __shared__ int ends[];
  static_assert(((T::threads == S::threads && T::BC == S::BC) && ...),
                "the smaller tiles are the largest one's with fewer rows");
  Line<S::BR, S::threads> line(a.g, a.cols, ends);
  Where t;
  bool more = line.next(&t);
  while (more) more = pick_tiles<ACT, 0, S, T...>(a, line, t, lds_base(lds));
}

template <typename S, typename... T>
hipError_t run(FwdArgs a, int act, hipStream_t stream) {
  const int per_tile = act == EP_ACT_SWIGLU ? S::BC / 2 : S::BC;
  a.cols = (a.n + per_tile - 1) / per_tile;
  const auto kernel = act == EP_ACT_SWIGLU ? product_kernel<EP_ACT_SWIGLU, S, T...>
                      : act == EP_ACT_SILU ? product_kernel<EP_ACT_SILU, S, T...>
                      : act == EP_ACT_GELU ? product_kernel<EP_ACT_GELU, S, T...>
                                           : product_kernel<EP_ACT_NONE, S, T...>;
  hipLaunchKernelGGL(kernel, dim3(line_grid(tile_grid(a.g, S::BR, a.cols))), dim3(S::threads),
                     (size_t)a.g.N * a.g.L * 4, stream, a);
  return hipGetLastError();
}

template <int FR, bool FP8, int STAGES, bool ONCE = true>
using Rows = Shape<2, FR, 4, 4, false, false, FP8, STAGES, ONCE>;

// Tiles of fewer rows and columns, with more steps on their way. In e4m3 the
// compiler has the matrix instruction write accumulator registers here (one
// wave a SIMD leaves it those), and every sum is moved out for its scaling: 64
// moves beside 64 FMAs in a step of 128 x 128, 32 beside 32 in the others. 1 to
// 128 rows of 7168 values by 4096 columns: 32 us, bf16 38 to 40.
template <bool FP8>
using Small = Shape<2, 4, 2, 4, false, false, FP8, 4>;        // 128 x 128
template <bool FP8>
using Flat = Shape<1, 2, 2, 4, false, false, FP8, 4, true>;   // 32 x 128
template <bool FP8>
using Thin = Shape<1, 2, 1, 4, false, false, FP8, 5, true>;   // 32 x 64

// The tiles that cost least, of equals the smallest. Rows of 7168 values by
// 4096 columns: 2048 rows take 150 us in the large ones and 125 in 128 x 128; 256
// rows 126, 53, 50 and 74 in the four; 64 rows 89, 46, 49 and 38. 2048 rows of
// 2048 values by 7168 columns: 54, 69, 189 and 315.
template <bool FP8>
hipError_t by_cost(const FwdArgs& a, int act, hipStream_t stream) {
  using Large = Rows<8, FP8, 2, false>;
  const int64_t cols = act == EP_ACT_SWIGLU ? 2 * a.n : a.n;
  const int64_t large = cost_of(a.g, 256, 64, 256, cols), small = cost_of(a.g, 128, 128, 128, cols),
                flat = cost_of(a.g, 32, 32, 128, cols), thin = cost_of(a.g, 32, 32, 64, cols);
  if (thin <= flat && thin <= small && thin <= large) return run<Thin<FP8>>(a, act, stream);
  if (flat <= small && flat <= large) return run<Flat<FP8>>(a, act, stream);
  if (small <= large) return run<Small<FP8>>(a, act, stream);
  return run<Large, Rows<2, FP8, 3>, Rows<4, FP8, 3>, Rows<6, FP8, 2>>(a, act, stream);
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
  return p.dtype == EP_DTYPE_E4M3 ? by_cost<true>(a, p.act, stream)
                                  : by_cost<false>(a, p.act, stream);
}

}  // namespace ep
