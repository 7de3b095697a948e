// Backward passes of combine and dispatch.
//
// With out = sum_k w_k y_k over a token's slots k, the gradients are
// dy_k = w_k dout and dw_k = dout . y_k. With grouped row = x of its token,
// dx = sum_k dgrouped_k. HBM bounds both: each expert row is read once, in whole
// rows wherever the plan put them, and a token's dout comes from HBM once (the
// combine kernel reads it anew for every four slots, then from the caches).
//
// One workgroup per token, V chunks of 8 values (16 bytes) per thread.
//
// 8 x 4096 tokens of 7168 values, top-8: 1582 us for combine (7.99 GB, 5.05
// TB/s), 799 us for dispatch (4.70 GB, 5.9 TB/s). 32 x 128 tokens: 195 and 91 us.
#include "ep_device.hpp"
#include "ep_kernels.hpp"

namespace ep {
namespace {

constexpr int kV = 2;        // 16-byte chunks per thread
// Expert rows in flight. Of 1, 2, 4 and 8: combine takes 1591, 1581, 1585 and
// 1589 us, dispatch 823, 835, 839 and 799 (8 x 4096 tokens).
constexpr int kRows = 4, kSumRows = 8;
constexpr int kMaxWaves = 16;

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack2(float a, float b) {  // nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// Row of slot k of the token, or -1 (dropped).
__device__ __forceinline__ int row_of(const int32_t* rows, int k, int R, int64_t rows_in) {
  const int r = k < R ? rows[k] : -1;
  return r >= 0 && r < rows_in ? wave_uniform(r) : -1;
}

template <bool DY, bool DW>
__global__ __launch_bounds__(1024) void combine_grad_kernel(const u32x4* dout, const u32x4* y,
                                                            const float* w, const int32_t* comb_row,
                                                            u32x4* dy, float* dweights, int R,
                                                            int n16, int64_t rows_in) {
  __shared__ float part[kMaxWaves][EP_MAX_TOPK];
  const size_t tok = blockIdx.x;
  const int32_t* rows = comb_row + tok * R;
  const float* wt = w + tok * R;
  const u32x4* src = dout + tok * n16;
  const int wave = threadIdx.x / kWave, span = blockDim.x * kV;
  for (int k0 = 0; k0 < R; k0 += kRows) {
    int row[kRows];
    float dot[kRows];
#pragma unroll
    for (int b = 0; b < kRows; ++b) {
      row[b] = row_of(rows, k0 + b, R, rows_in);
      dot[b] = 0.0f;
    }
    for (int base = 0; base < n16; base += span) {
      u32x4 d[kV], v[kRows][kV];
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int c = base + threadIdx.x + i * blockDim.x;
        d[i] = c < n16 ? src[c] : u32x4{0, 0, 0, 0};
        if constexpr (DW) {
#pragma unroll
          for (int b = 0; b < kRows; ++b)
            v[b][i] = row[b] >= 0 && c < n16 ? load_stream(&y[(size_t)row[b] * n16 + c])
                                             : u32x4{0, 0, 0, 0};
        }
      }
#pragma unroll
      for (int b = 0; b < kRows; ++b) {
        if (row[b] < 0) continue;
        const float wk = DY ? wt[k0 + b] : 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const int c = base + threadIdx.x + i * blockDim.x;
          u32x4 o;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float lo = bf16_lo(d[i][j]), hi = bf16_hi(d[i][j]);
            if constexpr (DW) {
              dot[b] = __builtin_fmaf(lo, bf16_lo(v[b][i][j]), dot[b]);
              dot[b] = __builtin_fmaf(hi, bf16_hi(v[b][i][j]), dot[b]);
            }
            if constexpr (DY) o[j] = pack2(wk * lo, wk * hi);
          }
          if constexpr (DY)
            if (c < n16) store_stream(&dy[(size_t)row[b] * n16 + c], o);
        }
      }
    }
    if constexpr (DW) {
#pragma unroll
      for (int b = 0; b < kRows; ++b) {
        const float s = wave_sum(dot[b]);
        if (lane_id() == 0 && k0 + b < R) part[wave][k0 + b] = s;
      }
    }
  }
  if constexpr (DW) {
    __syncthreads();
    for (int k = threadIdx.x; k < R; k += blockDim.x) {
      float s = 0.0f;
      for (int v = 0; v < (int)blockDim.x / kWave; ++v) s += part[v][k];
      dweights[tok * R + k] = s;
    }
  }
}

__global__ __launch_bounds__(1024) void dispatch_grad_kernel(const u32x4* g, const u32x4* add,
                                                             const int32_t* comb_row, u32x4* dx,
                                                             int R, int n16, int64_t rows_in) {
  const size_t tok = blockIdx.x;
  const int32_t* rows = comb_row + tok * R;
  for (int base = 0; base < n16; base += blockDim.x * kV) {
    float acc[kV][8];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int c = base + threadIdx.x + i * blockDim.x;
      const u32x4 a = add && c < n16 ? load_stream(&add[tok * n16 + c]) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][2 * j] = bf16_lo(a[j]);
        acc[i][2 * j + 1] = bf16_hi(a[j]);
      }
    }
    for (int k0 = 0; k0 < R; k0 += kSumRows) {
      int row[kSumRows];
      u32x4 v[kSumRows][kV];
#pragma unroll
      for (int b = 0; b < kSumRows; ++b) row[b] = row_of(rows, k0 + b, R, rows_in);
#pragma unroll
      for (int b = 0; b < kSumRows; ++b)
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const int c = base + threadIdx.x + i * blockDim.x;
          if (row[b] >= 0)
            v[b][i] = load_stream(&g[(size_t)row[b] * n16 + (c < n16 ? c : n16 - 1)]);
        }
#pragma unroll
      for (int b = 0; b < kSumRows; ++b) {
        if (row[b] < 0) continue;
#pragma unroll
        for (int i = 0; i < kV; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[i][2 * j] += bf16_lo(v[b][i][j]);
            acc[i][2 * j + 1] += bf16_hi(v[b][i][j]);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int c = base + threadIdx.x + i * blockDim.x;
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = pack2(acc[i][2 * j], acc[i][2 * j + 1]);
      if (c < n16) store_stream(&dx[tok * n16 + c], o);
    }
  }
}

// Threads that hold a row at kV chunks each, up to a workgroup's limit; longer
// rows are walked.
int threads_for(int n16) {
  const int waves = (n16 + kWave * kV - 1) / (kWave * kV);
  return kWave * (waves < kMaxWaves ? waves : kMaxWaves);
}

}  // namespace

// NT < 2^26 tokens of at most 1024 threads: the grid holds up to 2^22 whole
// workgroups of that size, so longer batches go in several launches.
constexpr int64_t kTokensPerLaunch = (int64_t)1 << 21;

hipError_t launch_combine_grad(const Dims& d, const uint16_t* dout, const uint16_t* y,
                               const float* w, const PlanPtrs& p, uint16_t* dy, float* dweights,
                               hipStream_t stream) {
  const auto kernel = !dy ? combine_grad_kernel<false, true>
                          : dweights ? combine_grad_kernel<true, true>
                                     : combine_grad_kernel<true, false>;
  const int n16 = d.H / 8;
  for (int64_t at = 0; at < d.NT; at += kTokensPerLaunch) {
    const int64_t n = d.NT - at < kTokensPerLaunch ? d.NT - at : kTokensPerLaunch;
    hipLaunchKernelGGL(kernel, dim3((unsigned)n), dim3(threads_for(n16)), 0, stream,
                       (const u32x4*)dout + at * n16, (const u32x4*)y, w ? w + at * d.R : nullptr,
                       p.comb_row + at * d.R, (u32x4*)dy, dweights ? dweights + at * d.R : nullptr,
                       d.R, n16, (int64_t)d.N * d.cap);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_dispatch_grad(const Dims& d, const uint16_t* dgrouped, const uint16_t* add,
                                const PlanPtrs& p, uint16_t* dx, hipStream_t stream) {
  const int n16 = d.H / 8;
  for (int64_t at = 0; at < d.NT; at += kTokensPerLaunch) {
    const int64_t n = d.NT - at < kTokensPerLaunch ? d.NT - at : kTokensPerLaunch;
    hipLaunchKernelGGL(dispatch_grad_kernel, dim3((unsigned)n), dim3(threads_for(n16)), 0, stream,
                       (const u32x4*)dgrouped, add ? (const u32x4*)add + at * n16 : nullptr,
                       p.comb_row + at * d.R, (u32x4*)dx + at * n16, d.R, n16,
                       (int64_t)d.N * d.cap);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace ep
