// Attention of new tokens over the pages of a cache.
//
// With s_i = scale q.k_i over the keys a row sees, m = max s_i and
// l = sum exp(s_i - m): out = sum exp(s_i - m) v_i / l, lse = m + log l. One
// pass over the keys keeps m, l and the sum, and scales them by
// exp(m_old - m_new) when the maximum grows.
//
// One wave takes one row and head: a lane scores one key of 64, then owns
// every 64th element of the output.
#include "ep_kernels.hpp"
#include "ep_kv_device.hpp"

namespace ep {
namespace {

constexpr int kBlock = 256;
constexpr int kMaxDim = 256;

struct Attend {
  ep_kv_cache c;
  ep_kv_batch b;
  ep_kv_groups g;
  ep_rows q, out;
  float* lse;
  float scale;
  int heads, max_new;
  int32_t* status;
};

template <int QT, int CT>
__global__ __launch_bounds__(kBlock) void attend_kernel(Attend a) {
  __shared__ float q[kBlock / kWave][kMaxDim];
  __shared__ float prob[kBlock / kWave][kWave];
  __shared__ int64_t slot[kBlock / kWave][kWave];
  const int wave = wave_uniform(threadIdx.x / kWave), lane = lane_id();
  const int64_t unit = (int64_t)blockIdx.x * (kBlock / kWave) + wave;
  const int row = wave_uniform((int)(unit / a.heads)), head = wave_uniform((int)(unit % a.heads));
  const int s = row < a.b.n_tokens ? seq_of_row(a.b, row) : -1;
  int64_t n = 0;
  bool skip = s < 0;
  bool bad = false;
  const int dim = a.c.head_dim, bt = a.c.page_tokens;
  if (s >= 0) {
    const int first = first_row(a.b, s), end = a.b.q_off ? a.b.q_off[s + 1] : s + 1;
    n = (int64_t)a.b.lens[s] - (end - first) + (row - first) + 1;
    if (row - first >= a.max_new) skip = bad = true;
    const int64_t cap = (int64_t)a.b.max_pages * bt;
    if (n > cap) {
      n = cap;
      bad = true;
    }
    const uint8_t* p = (const uint8_t*)a.q.p + row * a.q.token_stride + head * a.q.head_stride;
    for (int d = lane; d < dim; d += kWave) q[wave][d] = load1<QT>(p + 2 * d) * a.scale;
  }
  const int kvh = head / (a.heads / a.c.n_heads);
  const uint8_t* kb = (const uint8_t*)a.c.k + kvh * a.c.head_stride;
  const uint8_t* vb = (const uint8_t*)a.c.v + kvh * a.c.head_stride;
  const float ks = CT == EP_DTYPE_E4M3 ? a.c.k_scale[kvh] : 1.0f;
  const float vs = CT == EP_DTYPE_E4M3 ? a.c.v_scale[kvh] : 1.0f;
  float m = -__builtin_inff(), l = 0.0f, o[kMaxDim / kWave] = {};
  for (int64_t t0 = 0; !skip && t0 < n; t0 += kWave) {
    const int64_t t = t0 + lane;
    int64_t at = -1;
    if (t < n) {
      const int32_t p = a.b.tables[(int64_t)s * a.b.max_pages + t / bt];
      if (p >= 0 && p < a.c.n_pages)
        at = p * a.c.page_stride + (t % bt) * a.c.token_stride;
      else
        bad = true;
    }
    float x = -__builtin_inff();
    if (at >= 0) {
      x = 0.0f;
      for (int d = 0; d < dim; d += 8) {
        float f[8];
        load8<CT>(kb + at + d * Fmt<CT>::bytes, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) x += f[i] * q[wave][d + i];
      }
      x *= ks;
    }
    float top = x;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    top = fmaxf(top, m);
    if (top == -__builtin_inff()) continue;
    const float w = __expf(m - top), e = at >= 0 ? __expf(x - top) : 0.0f;
    float sum = e;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) sum += __shfl_xor(sum, d);
    m = top;
    l = l * w + sum;
    prob[wave][lane] = e;
    slot[wave][lane] = at;
#pragma unroll
    for (int i = 0; i < kMaxDim / kWave; ++i) o[i] *= w;
    for (int j = 0; j < kWave; ++j) {
      const int64_t sj = slot[wave][j];
      if (sj < 0) continue;
      const float pj = prob[wave][j];
#pragma unroll
      for (int i = 0; i < kMaxDim / kWave; ++i) {
        const int d = lane + i * kWave;
        if (d < dim) o[i] += pj * load1<CT>(vb + sj + d * Fmt<CT>::bytes);
      }
    }
  }
  if (bad) atomicOr(a.status, EP_STATUS_BAD_PAGE);
  if (skip) return;
  uint8_t* to = (uint8_t*)a.out.p + row * a.out.token_stride + head * a.out.head_stride;
  const float inv = l > 0.0f ? vs / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
  for (int i = 0; i < kMaxDim / kWave; ++i) {
    const int d = lane + i * kWave;
    if (d < dim) store1<QT>(to + 2 * d, o[i] * inv);
  }
  if (a.lse && lane == 0)
    a.lse[(int64_t)row * a.heads + head] = l == 0.0f ? -__builtin_inff() : m + __logf(l);
}

}  // namespace

size_t kv_attend_bytes(const ep_kv_cache&, int, int, int, int, int) { return 256; }

hipError_t launch_kv_attend(const ep_kv_cache& c, const ep_kv_batch& b, const ep_kv_groups& g,
                            int max_new, const ep_rows& q, int n_heads, const ep_rows& out,
                            float* lse, float sm_scale, void*, int32_t* status,
                            hipStream_t stream) {
  const Attend a{c, b, g, q, out, lse, sm_scale, n_heads, max_new, status};
  const unsigned grid = (unsigned)(((int64_t)b.n_tokens * n_heads + 3) / 4);
  const bool e4m3 = c.dtype == EP_DTYPE_E4M3;
  if (b.dtype == EP_DTYPE_BF16) {
    if (e4m3)
      hipLaunchKernelGGL((attend_kernel<EP_DTYPE_BF16, EP_DTYPE_E4M3>), dim3(grid), dim3(kBlock), 0, stream, a);
    else
      hipLaunchKernelGGL((attend_kernel<EP_DTYPE_BF16, EP_DTYPE_BF16>), dim3(grid), dim3(kBlock), 0, stream, a);
  } else if (e4m3) {
    hipLaunchKernelGGL((attend_kernel<EP_DTYPE_F16, EP_DTYPE_E4M3>), dim3(grid), dim3(kBlock), 0, stream, a);
  } else {
    hipLaunchKernelGGL((attend_kernel<EP_DTYPE_F16, EP_DTYPE_F16>), dim3(grid), dim3(kBlock), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace ep
