// Rotary positions and the write of new K and V into the pages of a cache.
//
// A pair (x, y) at position t turns by a = t * inv_freq: (x cos a - y sin a,
// x sin a + y cos a). The angle is formed and reduced in 64 bits: at a
// position of 10^5 a 32-bit product is off by up to 2^-8 radians.
//
// Bytes bound it: q is read and written once, k and v are read once and
// written once. 14,900 tokens of 32 + 8 + 8 heads of 128, bf16 to e4m3 (335
// MB), take 67 us: 5.0 TB/s, against 5.7 that a large copy reaches; 10,000 to a
// bf16 cache take 43 us, 5.7 TB/s. With the 5 + 1 + 1 heads of one rank a token
// has items for one wave of a block's four, and 14,900 tokens (53 MB) take 21
// us, 2.6 TB/s. A step of 128 tokens takes 5.5 us, most of it the chain from
// the offsets over the table to the slot, and the launch.
//
// A block takes one token or a few and forms their sines and cosines once, in
// LDS, for all heads; a work item is a pair of 16-byte chunks (or one chunk,
// where its pairs lie within), so that q can be rotated in place. A thread
// keeps its item and goes through the block's tokens, so that rows and scales
// are found once.
#include "ep_kernels.hpp"
#include "ep_kv_device.hpp"

namespace ep {
namespace {

constexpr int kBlock = 256;
constexpr int kAhead = 4;  // tokens whose loads are on their way together
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

// Where one token's rows are, in bytes.
struct Token {
  int64_t slot;     // of the cache; -1: none
  int64_t from[3];  // q, k, v
  int64_t to;       // q_out; -1: no sequence has the token
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

// Items of a row of chunks: 16 bytes of it, or the two halves' 16 bytes that
// turn together.
struct Chunk {
  u32x4 x, y;
};

__device__ __forceinline__ bool by_chunks(const ep_rope& rope) {
  return rope.rot_dim % (rope.layout == EP_ROPE_HALF ? 16 : 8) == 0;
}

// Whether item j of a row turns, and where it starts.
struct Place {
  int d;
  bool turns;
};
__device__ __forceinline__ Place place_of(const ep_rope& rope, int j) {
  const int turned = rope.layout == EP_ROPE_HALF ? rope.rot_dim / 16 : rope.rot_dim / 8;
  return j < turned ? Place{8 * j, true} : Place{rope.rot_dim + 8 * (j - turned), false};
}

template <int IN>
__device__ __forceinline__ void load_chunk(Chunk& c, const uint8_t* from, int j,
                                           const ep_rope& rope) {
  const Place p = place_of(rope, j);
  c.x = load_stream((const u32x4*)(from + p.d * Fmt<IN>::bytes));
  if (p.turns && rope.layout == EP_ROPE_HALF)
    c.y = load_stream((const u32x4*)(from + (p.d + rope.rot_dim / 2) * Fmt<IN>::bytes));
}

template <int IN>
__device__ __forceinline__ void widen8(const u32x4& w, float* f) {
  const auto v = as<typename Fmt<IN>::vec8>(w);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = (float)v[i];
}

template <int OUT>
__device__ __forceinline__ void divide8(const Divisor& by, float* f) {
  if constexpr (OUT == EP_DTYPE_E4M3) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = by.plain ? f[i] / by.scale : by(f[i]);
  }
}

template <int IN, int OUT>
__device__ __forceinline__ void put_chunk(const Chunk& c, uint8_t* to, int j, const ep_rope& rope,
                                          const float2* cs, const Divisor& by) {
  const Place p = place_of(rope, j);
  if (IN == OUT && !p.turns) {
    *(u32x4*)(to + p.d * Fmt<OUT>::bytes) = c.x;
    return;
  }
  float f[8], g[8];
  widen8<IN>(c.x, f);
  if (p.turns && rope.layout == EP_ROPE_HALF) {
    widen8<IN>(c.y, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(f[i], g[i], cs[8 * j + i].x, cs[8 * j + i].y);
    divide8<OUT>(by, g);
    store8<OUT>(to + (p.d + rope.rot_dim / 2) * Fmt<OUT>::bytes, g);
  } else if (p.turns) {
#pragma unroll
    for (int i = 0; i < 4; ++i) turn(f[2 * i], f[2 * i + 1], cs[4 * j + i].x, cs[4 * j + i].y);
  }
  divide8<OUT>(by, f);
  store8<OUT>(to + p.d * Fmt<OUT>::bytes, f);
}

// Item j of a row whose rotated part is no whole chunks: a pair, or a single
// element.
template <int IN, int OUT>
__device__ __forceinline__ void small_item(const uint8_t* from, uint8_t* to, int j,
                                           const ep_rope& rope, const float2* cs, float scale) {
  constexpr int ib = Fmt<IN>::bytes, ob = Fmt<OUT>::bytes;
  auto put1 = [&](int d, float f) {
    if constexpr (OUT == EP_DTYPE_E4M3) f = f / scale;
    store1<OUT>(to + (int64_t)d * ob, f);
  };
  const int rot = rope.rot_dim, half = rot / 2;
  if (j < half) {
    const bool split = rope.layout == EP_ROPE_HALF;
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

template <int IN, int OUT, int TOKENS>
__global__ __launch_bounds__(kBlock) void append_kernel(Append a) {
  __shared__ float2 cs[TOKENS * kMaxPairs];
  __shared__ Token tok[TOKENS];
  __shared__ int64_t at[TOKENS];
  const int half = a.rope.rot_dim / 2, bt = a.c.page_tokens;
  // Token t of the block by lane t of the first wave: the first one's
  // sequence is searched for, the others' lie among the next 64 offsets.
  if (threadIdx.x < kWave) {
    const int lane = threadIdx.x, row0 = wave_uniform(blockIdx.x) * TOKENS, row = row0 + lane;
    const bool have = lane < TOKENS && row < a.b.n_tokens;
    int s = have && row < a.b.n_seqs ? row : -1, first = row, end = row + 1;
    if (a.b.q_off) {
      const int s0 = seq_of_row(a.b, row0);
      s = -1;
      if (s0 >= 0) {
        const int last = a.b.n_seqs - s0;  // offsets s0 .. s0 + last
        const int next = a.b.q_off[s0 + (lane + 1 < last ? lane + 1 : last)];
        int skip = 0;
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) {
          const uint64_t mask = ballot(next <= row0 + t);
          if (lane == t) skip = mask + 1 == 0 ? kWave : __builtin_ctzll(~mask);
        }
        int lo = s0 + skip;
        if (have && skip == kWave)  // more empty sequences than lanes: walk on
          while (lo < a.b.n_seqs && a.b.q_off[lo + 1] <= row) ++lo;
        if (have && lo < a.b.n_seqs) {
          first = a.b.q_off[lo];
          end = a.b.q_off[lo + 1];
          if (first <= row && row < end) s = lo;
        }
      }
    }
    Token k{-1, {0, 0, 0}, -1};
    int64_t pos = 0;
    bool bad = false;
    if (s >= 0) {
      pos = (int64_t)a.b.lens[s] - (end - first) + (row - first);
      k.from[0] = row * a.q.token_stride;
      k.from[1] = row * a.k.token_stride;
      k.from[2] = row * a.v.token_stride;
      k.to = row * a.q_out.token_stride;
      bad = true;
      if (pos >= 0 && pos / bt < a.b.max_pages) {
        const int32_t p = a.b.tables[(int64_t)s * a.b.max_pages + pos / bt];
        if (p >= 0 && p < a.c.n_pages) {
          k.slot = p * a.c.page_stride + (pos % bt) * a.c.token_stride;
          bad = false;
        }
      }
    }
    if (lane < TOKENS) {
      tok[lane] = k;
      at[lane] = pos;
    }
    if (bad) atomicOr(a.status, EP_STATUS_BAD_PAGE);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < TOKENS * half; i += kBlock) {
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
  for (int i = threadIdx.x; i < per; i += kBlock) {
    // The item: of head h of q, k or v; the same one of every token.
    const bool is_v = i >= qk;
    const int log = is_v ? a.plain_log : a.turned_log, at_row = is_v ? i - qk : i;
    const int h = at_row >> log, j = at_row & ((1 << log) - 1);
    if (j >= (is_v ? a.plain : a.turned)) continue;
    const bool is_q = !is_v && h < heads;
    const int g = is_v || is_q ? h : h - heads;
    const int side = is_v ? 2 : is_q ? 0 : 1;
    const uint8_t* from = is_v   ? (const uint8_t*)a.v.p + g * a.v.head_stride
                          : is_q ? (const uint8_t*)a.q.p + g * a.q.head_stride
                                 : (const uint8_t*)a.k.p + g * a.k.head_stride;
    uint8_t* to = is_q ? (uint8_t*)a.q_out.p + g * a.q_out.head_stride
                       : (uint8_t*)(is_v ? a.c.v : a.c.k) + g * a.c.head_stride;
    const float* scales = is_v ? a.c.v_scale : a.c.k_scale;
    const float scale = OUT == EP_DTYPE_E4M3 && !is_q ? scales[g] : 1.0f;
    ep_rope rope = a.rope;
    if (is_v) rope.rot_dim = 0;
    const Divisor by(scale);
    if (by_chunks(rope)) {
      constexpr int n = TOKENS < kAhead ? TOKENS : kAhead;
#pragma unroll 1
      for (int t0 = 0; t0 < TOKENS; t0 += n) {
        Chunk c[n];
#pragma unroll
        for (int t = 0; t < n; ++t)  // a token that no sequence has reads row 0
          load_chunk<IN>(c[t], from + tok[t0 + t].from[side], j, rope);
#pragma unroll
        for (int t = 0; t < n; ++t) {
          const int64_t at_to = is_q ? tok[t0 + t].to : tok[t0 + t].slot;
          if (at_to < 0) continue;
          const float2* sc = cs + (t0 + t) * kMaxPairs;
          if (is_q) put_chunk<IN, IN>(c[t], to + at_to, j, rope, sc, by);
          else put_chunk<IN, OUT>(c[t], to + at_to, j, rope, sc, by);
        }
      }
    } else {
      for (int t = 0; t < TOKENS; ++t) {
        const int64_t at_to = is_q ? tok[t].to : tok[t].slot;
        if (at_to < 0) continue;
        const float2* sc = cs + t * kMaxPairs;
        const uint8_t* x = from + tok[t].from[side];
        if (is_q) small_item<IN, IN>(x, to + at_to, j, rope, sc, 1.0f);
        else small_item<IN, OUT>(x, to + at_to, j, rope, sc, scale);
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
  const dim3 grid((unsigned)(((int64_t)a.b.n_tokens + a.tokens - 1) / a.tokens));
  if (a.tokens == 1)
    hipLaunchKernelGGL((append_kernel<IN, OUT, 1>), grid, dim3(kBlock), 0, stream, a);
  else
    hipLaunchKernelGGL((append_kernel<IN, OUT, kAhead>), grid, dim3(kBlock), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const ep_kv_cache& c, const ep_kv_batch& b, const ep_rows& q,
                            int n_heads, const ep_rows& k, const ep_rows& v, const ep_rows& q_out,
                            const ep_rope& rope, int32_t* status, hipStream_t stream) {
  const int turned = row_items(rope, c.head_dim), plain = c.head_dim / 8;
  // Four tokens of a block have their loads on the way together and share the
  // block's start, which pays once every CU has blocks enough; few tokens
  // finish sooner in blocks of their own. One and four tokens, us, with 32 + 8
  // heads of 128 in bf16: 13.1 and 14.2 at 2,000 tokens, 16.5 and 16.1 at
  // 2,400, 48.0 and 43.4 at 10,000 (an e4m3 cache: 75.4 and 67.7 at 14,900).
  // With 5 + 1 heads: 5.1 and 6.6 at 2,000, 6.7 and 6.9 at 2,400, 8.8 and 7.6 at
  // 4,000, 30.2 and 20.8 at 14,900.
  const int tokens = b.n_tokens >= 2048 ? kAhead : 1;
  const Append a{c,      b,     q, k, v, q_out, rope, n_heads, tokens,
                 turned, log2_up(turned), plain, log2_up(plain), status};
  if (b.dtype == EP_DTYPE_BF16)
    return c.dtype == EP_DTYPE_E4M3 ? launch<EP_DTYPE_BF16, EP_DTYPE_E4M3>(a, stream)
                                    : launch<EP_DTYPE_BF16, EP_DTYPE_BF16>(a, stream);
  return c.dtype == EP_DTYPE_E4M3 ? launch<EP_DTYPE_F16, EP_DTYPE_E4M3>(a, stream)
                                  : launch<EP_DTYPE_F16, EP_DTYPE_F16>(a, stream);
}

}  // namespace ep
