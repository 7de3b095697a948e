// RMS norm with the residual's addition, its output as rows and as the planes
// of a block-fp8 dispatch, and its backward pass.
//
// Forward: h = x + residual rounded to the rows' type, y = h w r with
// r = 1 / sqrt(mean(h^2) + eps). Backward, with g = dy w:
// dx = dsum + r (g - h r^2 mean(g h)), dw = sum over rows of dy h r.
// HBM bounds both: every value is read once and written once, so a row stays
// in registers between its statistics and its output, and the backward pass
// forms r anew from the row it holds anyway instead of reading it.
//
// One workgroup per row, 8 values (16 bytes) per lane and chunk, V chunks per
// thread; the 16 lanes of a DPP row hold one 128-value block of the codes.
//
// 32768 rows of 7168 bf16 values: forward with residual and codes 365 us (2.12
// GB, 5.8 TB/s), backward 311 to 318 + 5 us (1.88 GB, 5.9 to 6.0 TB/s); a copy
// of 4 GiB runs at 4.5 to 4.9 TB/s. One row: 3.5 us, a launch. 4096 rows of 16384
// and of 32768 values: forward 100 and 218 us (6.0 and 5.5 TB/s), backward 100
// and 258 us (5.4 and 4.2: see the four chunks of the backward pass).
#include "ep_device.hpp"
#include "ep_kernels.hpp"
#include "ep_quant_device.hpp"

namespace ep {
namespace {

constexpr int kMaxWaves = 16;  // of a workgroup

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <int DT>
__device__ __forceinline__ void unpack(const u32x4& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == EP_DTYPE_BF16) {
      v[2 * i] = bf16_lo(r[i]);
      v[2 * i + 1] = bf16_hi(r[i]);
    } else {
      const f16x2 h = __builtin_bit_cast(f16x2, (uint32_t)r[i]);
      v[2 * i] = (float)h[0];
      v[2 * i + 1] = (float)h[1];
    }
  }
}

// Rounded to nearest even, both types.
template <int DT>
__device__ __forceinline__ u32x4 pack(const float (&v)[8]) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 f = {v[2 * i], v[2 * i + 1]};
    if constexpr (DT == EP_DTYPE_BF16)
      r[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
    else
      r[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
  }
  return r;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// Sums of N values over the workgroup, in the same order in every run. `room`
// is free again once every thread has passed the next barrier.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*room)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  const int waves = blockDim.x / kWave;
  if (waves == 1) return;
  if (lane_id() == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) room[threadIdx.x / kWave][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
  for (int w = 0; w < waves; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += room[w][i];
}

template <int DT, int V, bool QUANT>
__global__ __launch_bounds__(1024) void norm_kernel(const u32x4* x, const u32x4* residual,
                                                    const u32x4* weight, u32x4* sum, u32x4* y,
                                                    uint2* codes, float* scales, int64_t rows,
                                                    int n16, float per, float eps) {
  __shared__ float room[kMaxWaves][1];
  const int64_t number = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (number >= rows) return;  // whole waves: with blockDim.y > 1 a row is one wave's
  const size_t row = (size_t)number * n16;
  u32x4 raw[V], res[V], wt[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    raw[i] = res[i] = wt[i] = u32x4{0, 0, 0, 0};
    if (c < n16) {
      raw[i] = load_stream(&x[row + c]);
      if (residual) res[i] = load_stream(&residual[row + c]);
      wt[i] = weight[c];
    }
  }
  float h[V][8], ss[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    unpack<DT>(raw[i], h[i]);
    if (residual) {
      float b[8];
      unpack<DT>(res[i], b);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] += b[j];
      // The stream keeps the rounded sum, and its norm is what the next layers
      // and the backward pass see.
      const u32x4 s = pack<DT>(h[i]);
      if (c < n16) store_stream(&sum[row + c], s);
      unpack<DT>(s, h[i]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss[0] = __builtin_fmaf(h[i][j], h[i][j], ss[0]);
  }
  block_sum(ss, room);
  const float r = rsqrtf(ss[0] * per + eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    float w[8];
    unpack<DT>(wt[i], w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= h[i][j] * r;
    if (y && c < n16) store_stream(&y[row + c], pack<DT>(w));
    if constexpr (QUANT) {  // every lane takes part: a block's lanes are all in the row or none
      uint32_t packed[2];
      float scale;
      quantise_values(w, packed, scale);
      if (c < n16) {
        codes[row + c] = uint2{packed[0], packed[1]};
        if (threadIdx.x % 16 == 0) scales[(row + c) / 16] = scale;
      }
    }
  }
}

// Rows number, number + step, ... of a workgroup, or with SIDE of each of its
// waves; with AHEAD the next row's values are on their way while one is worked
// on (registers for it are there up to 512 threads). Each workgroup keeps its
// part of dweight in registers and writes it once: sums in a fixed order,
// without atomics.
template <int DT, int V, int THREADS, bool AHEAD, bool SIDE>
__global__ __launch_bounds__(THREADS) void norm_grad_kernel(const u32x4* dy, const u32x4* h,
                                                         const u32x4* weight, const u32x4* dsum,
                                                         u32x4* dx, float* parts, int64_t rows,
                                                         int n16, float per, float eps) {
  const int64_t number = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  __shared__ float room[2][kMaxWaves][2];
  u32x4 hn[V], dn[V], sn[V], wt[V];  // packed: a row's unpacked values fill the registers
  float dw[V][8];
  const auto load = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      hn[i] = dn[i] = sn[i] = u32x4{0, 0, 0, 0};
      if (c < n16 && r < rows) {
        const size_t at = (size_t)r * n16 + c;
        hn[i] = load_stream(&h[at]);
        dn[i] = load_stream(&dy[at]);
        if (dsum) sn[i] = load_stream(&dsum[at]);
      }
    }
  };
  if (AHEAD) load(number);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    wt[i] = c < n16 ? weight[c] : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  int turn = 0;
  for (int64_t r = number; r < rows; r += step, turn ^= 1) {
    float s[2] = {0.0f, 0.0f};
    u32x4 h0[V], d0[V], add[V];
    if (!AHEAD) load(r);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      h0[i] = hn[i];
      d0[i] = dn[i];
      add[i] = sn[i];
    }
    if (AHEAD) load(r + step);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float hv[8], dv[8], wv[8];
      unpack<DT>(h0[i], hv);
      unpack<DT>(d0[i], dv);
      unpack<DT>(wt[i], wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[0] = __builtin_fmaf(hv[j], hv[j], s[0]);
        s[1] = __builtin_fmaf(dv[j] * wv[j], hv[j], s[1]);
      }
    }
    block_sum(s, room[turn]);  // two rooms in turn: one barrier per row is enough
    const float rs = rsqrtf(s[0] * per + eps);
    const float k = rs * rs * s[1] * per;
    // Unpacked anew, not kept: of 1024 threads each has 128 registers, and 107 more
    // do not fit. The packed row and dweight of four chunks pass them all the same:
    // 31 to 33 registers, 80 bytes a lane, are spilled.
    if constexpr (V > 2) {
#pragma unroll
      for (int i = 0; i < V; ++i) asm volatile("" : "+v"(h0[i]), "+v"(d0[i]), "+v"(wt[i]));
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      float o[8], hv[8], dv[8], wv[8];
      unpack<DT>(add[i], o);
      unpack<DT>(h0[i], hv);
      unpack<DT>(d0[i], dv);
      unpack<DT>(wt[i], wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j] += rs * __builtin_fmaf(-hv[j], k, dv[j] * wv[j]);
        dw[i][j] = __builtin_fmaf(dv[j], hv[j] * rs, dw[i][j]);
      }
      if (c < n16) store_stream(&dx[(size_t)r * n16 + c], pack<DT>(o));
    }
  }
  if (!parts) return;
  if constexpr (SIDE) {  // the waves' sums, in order
    constexpr int waves = THREADS / kWave;
    __shared__ float sums[waves - 1][V * 8][kWave];
    if (threadIdx.y > 0)
#pragma unroll
      for (int j = 0; j < V * 8; ++j) sums[threadIdx.y - 1][j][threadIdx.x] = dw[j / 8][j % 8];
    __syncthreads();
    if (threadIdx.y > 0) return;
    for (int w = 0; w < waves - 1; ++w)
#pragma unroll
      for (int j = 0; j < V * 8; ++j) dw[j / 8][j % 8] += sums[w][j][threadIdx.x];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c >= n16) continue;
    float4* p = (float4*)(parts + ((size_t)blockIdx.x * n16 + c) * 8);
    p[0] = float4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
    p[1] = float4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
  }
}

// Column sums of the parts: 32 columns per workgroup, 32 groups of lanes that
// each take every 32nd part, eight of them on their way at once.
__global__ __launch_bounds__(1024) void norm_weight_kernel(const float* parts, float* dweight,
                                                           int n, int hidden) {
  __shared__ float room[32][33];
  const int lane = threadIdx.x % 32, group = threadIdx.x / 32, col = blockIdx.x * 32 + lane;
  float s = 0.0f;
  for (int p0 = group; p0 < n; p0 += 8 * 32) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int p = p0 + i * 32;
      v[i] = p < n && col < hidden ? parts[(size_t)p * hidden + col] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
  }
  room[group][lane] = s;
  __syncthreads();
  if (group != 0 || col >= hidden) return;
  s = 0.0f;
#pragma unroll
  for (int g = 0; g < 32; ++g) s += room[g][lane];
  dweight[col] = s;
}

// Chunks per thread: two while 1024 threads hold the row, else four. Two make
// the 896 chunks of 7168 values fill seven waves.
int chunks_per_thread(int hidden) { return hidden / 8 <= 2048 ? 2 : 4; }

// Threads of the workgroup that holds a row.
int norm_threads(int hidden) {
  const int per_wave = kWave * chunks_per_thread(hidden);
  return kWave * ((hidden / 8 + per_wave - 1) / per_wave);
}

// Rows of one wave each that share a workgroup: 35,000 rows of 16 values are
// otherwise as many workgroups.
int rows_at_once(int hidden) { return norm_threads(hidden) == kWave ? 8 : 1; }

// A launch holds fewer than 2^32 threads, of at most 1024 per row; more rows
// go in several launches.
constexpr int64_t kRowsPerLaunch = (int64_t)1 << 21;

template <int DT, int V>
hipError_t run_norm(const ep_norm& n, const void* x, const void* residual, void* sum, void* y,
                    uint8_t* codes, float* scales, hipStream_t stream) {
  const dim3 block(norm_threads(n.hidden), rows_at_once(n.hidden));
  const int n16 = n.hidden / 8;
  const auto kernel = codes ? norm_kernel<DT, V, true> : norm_kernel<DT, V, false>;
  const auto from = [&](const void* p, int64_t row) {
    return p ? (u32x4*)const_cast<void*>(p) + row * n16 : nullptr;
  };
  for (int64_t row = 0; row < n.rows; row += kRowsPerLaunch) {
    const int64_t rows = n.rows - row < kRowsPerLaunch ? n.rows - row : kRowsPerLaunch;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((rows + block.y - 1) / block.y)), block, 0, stream, from(x, row),
                       from(residual, row), (const u32x4*)n.weight, from(sum, row), from(y, row),
                       codes ? (uint2*)codes + row * n16 : nullptr,
                       scales ? scales + row * (n16 / 16) : nullptr, rows, n16,
                       1.0f / (float)n.hidden, n.eps);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
auto grad_kernel(int hidden) {
  if (rows_at_once(hidden) > 1) return norm_grad_kernel<DT, 2, 512, true, true>;
  if (chunks_per_thread(hidden) == 4) return norm_grad_kernel<DT, 4, 1024, false, false>;
  return norm_threads(hidden) > 512 ? norm_grad_kernel<DT, 2, 1024, false, false>
                                    : norm_grad_kernel<DT, 2, 512, true, false>;
}

}  // namespace

// Workgroups that together give each of the chip's 256 CUs 1024 threads, but
// at most two: every one of them costs a row of parts. No more than rows need.
int norm_grad_parts(const ep_norm& n) {
  const int threads = norm_threads(n.hidden), side = rows_at_once(n.hidden);
  const int64_t most = threads * side > 512 ? 256 : 512, need = (n.rows + side - 1) / side;
  return (int)(need < most ? need : most);
}

hipError_t launch_rms_norm(const ep_norm& n, const void* x, const void* residual, void* sum,
                           void* y, uint8_t* codes, float* scales, hipStream_t stream) {
  const auto run = n.dtype == EP_DTYPE_BF16
                       ? (chunks_per_thread(n.hidden) == 2 ? run_norm<EP_DTYPE_BF16, 2>
                                                           : run_norm<EP_DTYPE_BF16, 4>)
                       : (chunks_per_thread(n.hidden) == 2 ? run_norm<EP_DTYPE_F16, 2>
                                                           : run_norm<EP_DTYPE_F16, 4>);
  return run(n, x, residual, sum, y, codes, scales, stream);
}

hipError_t launch_rms_norm_grad(const ep_norm& n, const void* dy, const void* h, const void* dsum,
                                void* dx, float* dweight, float* parts, hipStream_t stream) {
  const int blocks = norm_grad_parts(n);
  if (blocks > 0) {
    const auto kernel =
        n.dtype == EP_DTYPE_BF16 ? grad_kernel<EP_DTYPE_BF16>(n.hidden) : grad_kernel<EP_DTYPE_F16>(n.hidden);
    hipLaunchKernelGGL(kernel, dim3(blocks),
                       dim3(norm_threads(n.hidden), rows_at_once(n.hidden)), 0, stream,
                       (const u32x4*)dy, (const u32x4*)h, (const u32x4*)n.weight,
                       (const u32x4*)dsum, (u32x4*)dx, dweight ? parts : nullptr, n.rows,
                       n.hidden / 8, 1.0f / (float)n.hidden, n.eps);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !dweight) return e;
  }
  if (dweight)
    hipLaunchKernelGGL(norm_weight_kernel, dim3((n.hidden + 31) / 32), dim3(1024), 0,
                       stream, parts, dweight, blocks, n.hidden);
  return hipGetLastError();
}

}  // namespace ep
