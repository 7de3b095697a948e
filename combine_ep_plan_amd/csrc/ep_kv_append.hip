// Rotary positions and the write of new K and V into the pages of a cache.
//
// A pair (x, y) at position t turns by a = t * inv_freq: (x cos a - y sin a,
// x sin a + y cos a). The angle is formed and reduced in 64 bits: at a
// position of 10^5 a 32-bit product is off by up to 2^-8 radians.
//
// Bytes bound it: q is read and written once, k and v are read once and
// written once. A block takes a few tokens and forms their sines and cosines
// once, in LDS, for all heads; a work item is a pair of 16-byte chunks (or
// one chunk, where its pairs lie within), so that q can be rotated in place.
#include "ep_kernels.hpp"
#include "ep_kv_device.hpp"

namespace ep {
namespace {

constexpr int kBlock = 256;
constexpr int kMaxTokens = 4;  // tokens of a block
constexpr int kMaxPairs = 128;

struct Append {
  ep_kv_cache c;
  ep_kv_batch b;
  ep_rows q, k, v, q_out;
  ep_rope rope;
  int heads, tokens;  // query heads; tokens per block
  // Items of a row of q or k, and of v, and the powers of two they are laid
  // out by: a thread finds its row and item by a shift.
  int turned, turned_log, plain, plain_log;
  int32_t* status;
};

// Where one token's K and V go: byte offset of its slot, or -1.
struct Token {
  int64_t slot;
  int row;  // -1: no sequence has it
};

__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float a = x * c - y * s, b = x * s + y * c;
  x = a;
  y = b;
}

// x / scale, rounded once. With y = 1 / scale rounded once, q = x y and the
// remainder r = x - scale q (exact), q + r y rounds correctly (Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990); an
// infinite or NaN q stays. Scales whose reciprocals or remainders leave the
// normal range are divided by.
struct Divisor {
  float scale, inv;
  bool plain;

  __device__ __forceinline__ explicit Divisor(float s) : scale(s), inv(1.0f / s) {
    plain = !(fabsf(s) > 0x1p-60f && fabsf(s) < 0x1p60f);
  }
  __device__ __forceinline__ float operator()(float x) const {
    const float q = x * inv;
    const float c = __builtin_fmaf(__builtin_fmaf(-scale, q, x), inv, q);
    return fabsf(q) < __builtin_inff() ? c : q;
  }
};

// One row of a head: reads `from`, writes `to` (as type OUT, divided by
// the scale for an e4m3 cache). Item j of row_items().
template <int IN, int OUT>
__device__ __forceinline__ void row_item(const uint8_t* from, uint8_t* to, int j, int head_dim,
                                         const ep_rope& rope, const float2* cs, float scale) {
  constexpr int ib = Fmt<IN>::bytes, ob = Fmt<OUT>::bytes;
  const Divisor by(scale);
  auto put8 = [&](int d, float* f) {
    if constexpr (OUT == EP_DTYPE_E4M3) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = by.plain ? f[i] / scale : by(f[i]);
    }
    store8<OUT>(to + (int64_t)d * ob, f);
  };
  auto put1 = [&](int d, float f) {
    if constexpr (OUT == EP_DTYPE_E4M3) f = f / scale;
    store1<OUT>(to + (int64_t)d * ob, f);
  };
  const int rot = rope.rot_dim, half = rot / 2;
  const bool split = rope.layout == EP_ROPE_HALF;
  if (rot % (split ? 16 : 8) == 0) {
    const int turned = split ? rot / 16 : rot / 8;
    float f[8];
    if (j >= turned) {
      const int d = rot + 8 * (j - turned);
      load8<IN>(from + (int64_t)d * ib, f);
      put8(d, f);
    } else if (split) {
      float g[8];
      load8<IN>(from + (int64_t)8 * j * ib, f);
      load8<IN>(from + (int64_t)(8 * j + half) * ib, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) turn(f[i], g[i], cs[8 * j + i].x, cs[8 * j + i].y);
      put8(8 * j, f);
      put8(8 * j + half, g);
    } else {
      load8<IN>(from + (int64_t)8 * j * ib, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) turn(f[2 * i], f[2 * i + 1], cs[4 * j + i].x, cs[4 * j + i].y);
      put8(8 * j, f);
    }
  } else if (j < half) {
    const int d = split ? j : 2 * j, e = split ? j + half : 2 * j + 1;
    float x = load1<IN>(from + (int64_t)d * ib), y = load1<IN>(from + (int64_t)e * ib);
    turn(x, y, cs[j].x, cs[j].y);
    put1(d, x);
    put1(e, y);
  } else {
    const int d = rot + j - half;
    put1(d, load1<IN>(from + (int64_t)d * ib));
  }
}

// Items of a rotated row: chunks where the rotated part is whole chunks,
// else pairs and single elements.
int row_items(const ep_rope& rope, int head_dim) {
  const bool split = rope.layout == EP_ROPE_HALF;
  const int rot = rope.rot_dim;
  if (rot % (split ? 16 : 8) == 0) return (split ? rot / 16 : rot / 8) + (head_dim - rot) / 8;
  return rot / 2 + head_dim - rot;
}

template <int IN, int OUT>
__global__ __launch_bounds__(kBlock) void append_kernel(Append a) {
  __shared__ float2 cs[kMaxTokens * kMaxPairs];
  __shared__ Token tok[kMaxTokens];
  __shared__ int64_t at[kMaxTokens];
  const int wave = wave_uniform(threadIdx.x / kWave);
  const int half = a.rope.rot_dim / 2, bt = a.c.page_tokens;
  for (int t = wave; t < a.tokens; t += kBlock / kWave) {
    const int64_t row = (int64_t)blockIdx.x * a.tokens + t;
    Token k{-1, -1};
    int64_t pos = 0;
    bool bad = false;
    const int s = row < a.b.n_tokens ? seq_of_row(a.b, (int)row) : -1;
    if (s >= 0) {
      const int first = first_row(a.b, s), end = a.b.q_off ? a.b.q_off[s + 1] : s + 1;
      pos = (int64_t)a.b.lens[s] - (end - first) + (row - first);
      k.row = (int)row;
      bad = true;
      if (pos >= 0 && pos / bt < a.b.max_pages) {
        const int32_t p = a.b.tables[(int64_t)s * a.b.max_pages + pos / bt];
        if (p >= 0 && p < a.c.n_pages) {
          k.slot = p * a.c.page_stride + (pos % bt) * a.c.token_stride;
          bad = false;
        }
      }
    }
    if (lane_id() == 0) {
      tok[t] = k;
      at[t] = pos;
      if (bad) atomicOr(a.status, EP_STATUS_BAD_PAGE);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.tokens * half; i += kBlock) {
    const int t = i / half, pair = i - t * half;
    const double turns = (double)at[t] * (double)a.rope.inv_freq[pair] * 0.15915494309189533577;
    const float f = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.0f * f, &s, &c);
    cs[t * kMaxPairs + pair] = make_float2(c * a.rope.mscale, s * a.rope.mscale);
  }
  __syncthreads();
  const int heads = a.q.p ? a.heads : 0, kv = a.c.n_heads;
  const int qk = (heads + kv) << a.turned_log, per = qk + (kv << a.plain_log);
  for (int t = 0; t < a.tokens; ++t) {
    const Token k = tok[t];
    if (k.row < 0) continue;
    const float2* sc = cs + t * kMaxPairs;
    for (int i = threadIdx.x; i < per; i += kBlock) {
      if (i < qk) {
        const int h = i >> a.turned_log, j = i & ((1 << a.turned_log) - 1);
        if (j >= a.turned) continue;
        if (h < heads) {
          row_item<IN, IN>((const uint8_t*)a.q.p + k.row * a.q.token_stride + h * a.q.head_stride,
                           (uint8_t*)a.q_out.p + k.row * a.q_out.token_stride +
                               h * a.q_out.head_stride,
                           j, a.c.head_dim, a.rope, sc, 1.0f);
        } else if (k.slot >= 0) {
          const int g = h - heads;
          row_item<IN, OUT>((const uint8_t*)a.k.p + k.row * a.k.token_stride + g * a.k.head_stride,
                            (uint8_t*)a.c.k + k.slot + g * a.c.head_stride, j, a.c.head_dim,
                            a.rope, sc, a.c.k_scale ? a.c.k_scale[g] : 1.0f);
        }
      } else if (k.slot >= 0) {
        const int g = (i - qk) >> a.plain_log, j = (i - qk) & ((1 << a.plain_log) - 1);
        if (j >= a.plain) continue;
        ep_rope none = a.rope;
        none.rot_dim = 0;
        row_item<IN, OUT>((const uint8_t*)a.v.p + k.row * a.v.token_stride + g * a.v.head_stride,
                          (uint8_t*)a.c.v + k.slot + g * a.c.head_stride, j, a.c.head_dim, none, sc,
                          a.c.v_scale ? a.c.v_scale[g] : 1.0f);
      }
    }
  }
}

int log2_up(int n) {
  int l = 0;
  while (1 << l < n) ++l;
  return l;
}

template <int IN, int OUT>
hipError_t launch(const Append& a, hipStream_t stream) {
  const unsigned grid = (unsigned)(((int64_t)a.b.n_tokens + a.tokens - 1) / a.tokens);
  hipLaunchKernelGGL((append_kernel<IN, OUT>), dim3(grid), dim3(kBlock), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const ep_kv_cache& c, const ep_kv_batch& b, const ep_rows& q,
                            int n_heads, const ep_rows& k, const ep_rows& v, const ep_rows& q_out,
                            const ep_rope& rope, int32_t* status, hipStream_t stream) {
  const int turned = row_items(rope, c.head_dim), plain = c.head_dim / 8;
  const Append a{c,      b,     q, k, v, q_out, rope, n_heads, b.n_tokens >= 2048 ? kMaxTokens : 1,
                 turned, log2_up(turned), plain, log2_up(plain), status};
  if (b.dtype == EP_DTYPE_BF16)
    return c.dtype == EP_DTYPE_E4M3 ? launch<EP_DTYPE_BF16, EP_DTYPE_E4M3>(a, stream)
                                    : launch<EP_DTYPE_BF16, EP_DTYPE_BF16>(a, stream);
  return c.dtype == EP_DTYPE_E4M3 ? launch<EP_DTYPE_F16, EP_DTYPE_E4M3>(a, stream)
                                  : launch<EP_DTYPE_F16, EP_DTYPE_F16>(a, stream);
}

}  // namespace ep
