// C ABI of the operators on a paged KV cache: argument checks, workspace
// layout and launches. What depends on device data (page ids, lengths,
// offsets) is checked by the kernels.
#include "ep.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "ep_checks.hpp"
#include "ep_kernels.hpp"

namespace {

using ep::check_aligned16;
using ep::check_ptr;
using ep::DeviceScope;
using ep::fail;
using ep::fail_hip;

constexpr int64_t kMaxBytes = (int64_t)1 << 46;  // of any one buffer or stride

// a * b, or -1 when either is negative or the product passes kMaxBytes.
int64_t mul(int64_t a, int64_t b) {
  int64_t r = 0;
  if (a < 0 || b < 0 || __builtin_mul_overflow(a, b, &r) || r > kMaxBytes) return -1;
  return r;
}

int check_pages(const ep_kv_pages* g, int64_t m) {
  if (!g) return fail(EP_ERR_INVALID_ARG, "null page state");
  if (g->n_seqs < 1 || g->max_pages < 1 || g->n_pages < 1 || g->page_tokens < 1 || g->ranks < 1)
    return fail(EP_ERR_INVALID_ARG, "page state: sizes must be positive");
  if (g->reserved != 0) return fail(EP_ERR_INVALID_ARG, "page state: reserved must be 0");
  if (g->page_bytes < 16 || g->page_bytes % 16 != 0 || g->rank_bytes % 16 != 0)
    return fail(EP_ERR_INVALID_ARG, "page state: page and rank bytes must be multiples of 16");
  const int64_t span = mul(g->n_pages, g->page_bytes);
  if (span < 0 || g->rank_bytes < 0 || g->rank_bytes > kMaxBytes ||
      mul(g->ranks, g->rank_bytes) < 0)
    return fail(EP_ERR_UNSUPPORTED, "page state: pool too large");
  if (g->rank_bytes < span)
    return fail(EP_ERR_INVALID_ARG, "page state: rank_bytes is less than n_pages * page_bytes");
  if (mul(mul(g->n_seqs, g->max_pages), 4) < 0 || mul(g->max_pages, g->page_tokens) < 0)
    return fail(EP_ERR_UNSUPPORTED, "page state: tables too large");
  // One grid row per rank and piece of a page.
  if (g->ranks > 65534 / ep::kv_page_pieces(g->page_bytes))
    return fail(EP_ERR_UNSUPPORTED, "page state: ranks * (8 KB pieces per page) must be < 65535");
  if (m < 0) return fail(EP_ERR_INVALID_ARG, "number of requests must not be negative");
  if (m > EP_KV_MAX_REQUESTS)
    return fail(EP_ERR_UNSUPPORTED, "more than EP_KV_MAX_REQUESTS requests");
  return EP_OK;
}

size_t pages_layout(const ep_kv_pages& g, int64_t m, void* ws, ep::PagesWs* w) {
  const int64_t chunks = ((int64_t)g.n_pages + ep::kKvCompactChunk - 1) / ep::kKvCompactChunk;
  const int64_t n[8] = {g.n_pages, g.n_pages, g.n_pages / 2 + 1, g.n_pages / 2 + 1, g.n_seqs, m, m,
                        chunks + 1};
  int32_t* p[8];
  size_t at = 0;
  for (int i = 0; i < 8; ++i) {
    p[i] = ws ? (int32_t*)((char*)ws + at) : nullptr;
    at += ((size_t)n[i] * 4 + 255) & ~(size_t)255;
  }
  if (w) *w = ep::PagesWs{p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7]};
  return at;
}

// The state's buffers. `tables`: also tables and lengths are used; `pool`:
// also the pool.
int check_state(const ep_kv_pages& g, int64_t m, void* ws, int32_t* status, bool tables,
                bool pool, int dev) {
  if (tables) {
    EP_CHECK(check_ptr(g.tables, dev, "tables", (int64_t)g.n_seqs * g.max_pages * 4));
    EP_CHECK(check_ptr(g.lens, dev, "lens", (int64_t)g.n_seqs * 4));
    EP_CHECK(check_ptr(g.refs, dev, "refs", (int64_t)g.n_pages * 4));
  }
  if (pool) {
    EP_CHECK(check_ptr(g.pool, dev, "pool",
                       (g.ranks - 1) * g.rank_bytes + g.n_pages * g.page_bytes));
    EP_CHECK(check_aligned16(g.pool, "pool"));
  }
  EP_CHECK(check_ptr(ws, dev, "ws", (int64_t)pages_layout(g, m, nullptr, nullptr)));
  EP_CHECK(check_aligned16(ws, "ws"));
  return check_ptr(status, dev, "status", 4);
}

bool known_dtype(int32_t t, bool cache) {
  return t == EP_DTYPE_BF16 || t == EP_DTYPE_F16 || (cache && t == EP_DTYPE_E4M3);
}

int elem_bytes(int32_t t) { return t == EP_DTYPE_E4M3 ? 1 : 2; }

int check_cache(const ep_kv_cache* c) {
  if (!c) return fail(EP_ERR_INVALID_ARG, "null cache");
  if (!known_dtype(c->dtype, true)) return fail(EP_ERR_INVALID_ARG, "cache: unknown dtype");
  if (c->reserved != 0) return fail(EP_ERR_INVALID_ARG, "cache: reserved must be 0");
  if (c->n_pages < 1 || c->page_tokens < 1 || c->n_heads < 1 || c->head_dim < 1)
    return fail(EP_ERR_INVALID_ARG, "cache: sizes must be positive");
  if (c->head_dim % (16 / elem_bytes(c->dtype)) != 0)
    return fail(EP_ERR_INVALID_ARG, "cache: head_dim must be a multiple of 8 (16 for e4m3)");
  if (c->head_dim > 256) return fail(EP_ERR_UNSUPPORTED, "cache: head_dim must be at most 256");
  if (c->n_heads > 65535) return fail(EP_ERR_UNSUPPORTED, "cache: too many heads");
  const int64_t row = (int64_t)c->head_dim * elem_bytes(c->dtype);
  const int64_t st[3] = {c->page_stride, c->token_stride, c->head_stride};
  for (int64_t s : st) {
    if (s < 0 || s % 16 != 0)
      return fail(EP_ERR_INVALID_ARG, "cache: strides must be multiples of 16 and not negative");
    if (s > kMaxBytes) return fail(EP_ERR_UNSUPPORTED, "cache: stride too large");
  }
  if ((c->n_heads > 1 && c->head_stride < row) || (c->page_tokens > 1 && c->token_stride < row) ||
      (c->n_pages > 1 && c->page_stride < row))
    return fail(EP_ERR_INVALID_ARG, "cache: a stride is smaller than a row");
  if (mul(c->n_pages, c->page_stride) < 0 || mul(c->page_tokens, c->token_stride) < 0)
    return fail(EP_ERR_UNSUPPORTED, "cache: too large");
  return EP_OK;
}

int check_cache_ptrs(const ep_kv_cache& c, int dev) {
  const int64_t span = (int64_t)(c.n_pages - 1) * c.page_stride +
                       (int64_t)(c.page_tokens - 1) * c.token_stride +
                       (int64_t)(c.n_heads - 1) * c.head_stride +
                       (int64_t)c.head_dim * elem_bytes(c.dtype);
  EP_CHECK(check_ptr(c.k, dev, "cache.k", span));
  EP_CHECK(check_ptr(c.v, dev, "cache.v", span));
  EP_CHECK(check_aligned16(c.k, "cache.k"));
  EP_CHECK(check_aligned16(c.v, "cache.v"));
  if (c.dtype == EP_DTYPE_E4M3) {
    EP_CHECK(check_ptr(c.k_scale, dev, "cache.k_scale", (int64_t)c.n_heads * 4));
    EP_CHECK(check_ptr(c.v_scale, dev, "cache.v_scale", (int64_t)c.n_heads * 4));
  } else if (c.k_scale || c.v_scale) {
    return fail(EP_ERR_INVALID_ARG, "cache: scales belong to an e4m3 cache only");
  }
  return EP_OK;
}

int check_batch(const ep_kv_batch* b, const ep_kv_cache& c) {
  if (!b) return fail(EP_ERR_INVALID_ARG, "null batch");
  if (!known_dtype(b->dtype, false)) return fail(EP_ERR_INVALID_ARG, "batch: unknown dtype");
  if (c.dtype != EP_DTYPE_E4M3 && c.dtype != b->dtype)
    return fail(EP_ERR_UNSUPPORTED, "the cache's dtype must be the rows' or e4m3");
  if (b->n_seqs < 0 || b->max_pages < 0 || b->n_tokens < 0)
    return fail(EP_ERR_INVALID_ARG, "batch: sizes must not be negative");
  if (b->n_tokens > 0 && b->n_seqs > 0 && b->max_pages < 1)
    return fail(EP_ERR_INVALID_ARG, "batch: max_pages must be positive");
  if (mul(mul(b->n_seqs, b->max_pages), 4) < 0 || mul(b->max_pages, c.page_tokens) < 0)
    return fail(EP_ERR_UNSUPPORTED, "batch: tables too large");
  if (b->n_tokens > (1 << 24)) return fail(EP_ERR_UNSUPPORTED, "batch: n_tokens must be <= 2^24");
  return EP_OK;
}

int check_batch_ptrs(const ep_kv_batch& b, int dev) {
  EP_CHECK(check_ptr(b.tables, dev, "tables", (int64_t)b.n_seqs * b.max_pages * 4));
  EP_CHECK(check_ptr(b.lens, dev, "lens", (int64_t)b.n_seqs * 4));
  if (b.q_off) EP_CHECK(check_ptr(b.q_off, dev, "q_off", ((int64_t)b.n_seqs + 1) * 4));
  return EP_OK;
}

int check_rows(const ep_rows* r, int64_t heads, const ep_kv_batch& b, int head_dim,
               const char* name, int dev) {
  if (!r) return fail(EP_ERR_INVALID_ARG, (std::string("null rows: ") + name).c_str());
  const int64_t row = (int64_t)head_dim * 2;
  if (r->token_stride < 0 || r->head_stride < 0 || (r->token_stride | r->head_stride) & 15)
    return fail(EP_ERR_INVALID_ARG,
                (std::string("strides must be multiples of 16 and not negative: ") + name).c_str());
  if (mul(b.n_tokens, r->token_stride) < 0 || mul(heads, r->head_stride) < 0)
    return fail(EP_ERR_UNSUPPORTED, (std::string("rows too large: ") + name).c_str());
  EP_CHECK(check_ptr(r->p, dev, name,
                     (b.n_tokens - 1) * r->token_stride + (heads - 1) * r->head_stride + row));
  return check_aligned16(r->p, name);
}

// Output rows must not share bytes.
int check_apart(const ep_rows& r, int64_t heads, const ep_kv_batch& b, int head_dim,
                const char* name) {
  const int64_t row = (int64_t)head_dim * 2;
  const bool heads_in = (b.n_tokens == 1 || r.token_stride >= (heads - 1) * r.head_stride + row) &&
                        (heads == 1 || r.head_stride >= row);
  const bool tokens_in = (heads == 1 || r.head_stride >= (b.n_tokens - 1) * r.token_stride + row) &&
                         (b.n_tokens == 1 || r.token_stride >= row);
  if (heads_in || tokens_in) return EP_OK;
  return fail(EP_ERR_INVALID_ARG, (std::string("rows overlap: ") + name).c_str());
}

int check_heads(const ep_kv_cache& c, int32_t n_heads) {
  if (n_heads < 1 || n_heads % c.n_heads != 0)
    return fail(EP_ERR_INVALID_ARG, "n_heads must be a positive multiple of the cache's heads");
  if (n_heads > 65535) return fail(EP_ERR_UNSUPPORTED, "too many heads");
  return EP_OK;
}

}  // namespace

extern "C" {

size_t ep_kv_pages_bytes(const ep_kv_pages* g, int64_t m) {
  if (check_pages(g, m) != EP_OK) return 0;
  return pages_layout(*g, m, nullptr, nullptr);
}

int ep_kv_extend(const ep_kv_pages* g, const int32_t* seqs, const int32_t* add, int64_t m,
                 void* ws, int32_t* status, hipStream_t stream) {
  EP_CHECK(check_pages(g, m));
  DeviceScope scope(stream);
  if (scope.error() != hipSuccess) return fail_hip(scope.error(), "device");
  EP_CHECK(check_state(*g, m, ws, status, true, false, scope.device()));
  EP_CHECK(check_ptr(seqs, scope.device(), "seqs", m * 4));
  EP_CHECK(check_ptr(add, scope.device(), "add", m * 4));
  if (m == 0) return EP_OK;
  ep::PagesWs w;
  pages_layout(*g, m, ws, &w);
  const hipError_t e = ep::launch_kv_extend(*g, seqs, add, (int)m, w, status, stream);
  if (e != hipSuccess) return fail_hip(e, "ep_kv_extend");
  return EP_OK;
}

int ep_kv_fork(const ep_kv_pages* g, const int32_t* parents, const int32_t* children, int64_t m,
               void* ws, int32_t* status, hipStream_t stream) {
  EP_CHECK(check_pages(g, m));
  DeviceScope scope(stream);
  if (scope.error() != hipSuccess) return fail_hip(scope.error(), "device");
  EP_CHECK(check_state(*g, m, ws, status, true, true, scope.device()));
  EP_CHECK(check_ptr(parents, scope.device(), "parents", m * 4));
  EP_CHECK(check_ptr(children, scope.device(), "children", m * 4));
  if (m == 0) return EP_OK;
  ep::PagesWs w;
  pages_layout(*g, m, ws, &w);
  const hipError_t e = ep::launch_kv_fork(*g, parents, children, (int)m, w, status, stream);
  if (e != hipSuccess) return fail_hip(e, "ep_kv_fork");
  return EP_OK;
}

int ep_kv_free(const ep_kv_pages* g, const int32_t* seqs, int64_t m, void* ws, int32_t* status,
               hipStream_t stream) {
  EP_CHECK(check_pages(g, m));
  DeviceScope scope(stream);
  if (scope.error() != hipSuccess) return fail_hip(scope.error(), "device");
  EP_CHECK(check_state(*g, m, ws, status, true, false, scope.device()));
  EP_CHECK(check_ptr(seqs, scope.device(), "seqs", m * 4));
  if (m == 0) return EP_OK;
  const hipError_t e = ep::launch_kv_free(*g, seqs, (int)m, status, stream);
  if (e != hipSuccess) return fail_hip(e, "ep_kv_free");
  return EP_OK;
}

int ep_kv_compact(const ep_kv_pages* g, int32_t* n_live, void* ws, int32_t* status,
                  hipStream_t stream) {
  EP_CHECK(check_pages(g, 0));
  DeviceScope scope(stream);
  if (scope.error() != hipSuccess) return fail_hip(scope.error(), "device");
  EP_CHECK(check_state(*g, 0, ws, status, true, true, scope.device()));
  if (n_live) EP_CHECK(check_ptr(n_live, scope.device(), "n_live", 4));
  ep::PagesWs w;
  pages_layout(*g, 0, ws, &w);
  const hipError_t e = ep::launch_kv_compact(*g, n_live, w, status, stream);
  if (e != hipSuccess) return fail_hip(e, "ep_kv_compact");
  return EP_OK;
}

int ep_kv_copy_pages(const ep_kv_pages* g, const int32_t* src, const int32_t* dst, int64_t m,
                     void* ws, int32_t* status, hipStream_t stream) {
  EP_CHECK(check_pages(g, m));
  DeviceScope scope(stream);
  if (scope.error() != hipSuccess) return fail_hip(scope.error(), "device");
  EP_CHECK(check_state(*g, m, ws, status, false, true, scope.device()));
  EP_CHECK(check_ptr(src, scope.device(), "src", m * 4));
  EP_CHECK(check_ptr(dst, scope.device(), "dst", m * 4));
  if (m == 0) return EP_OK;
  ep::PagesWs w;
  pages_layout(*g, m, ws, &w);
  const hipError_t e = ep::launch_kv_copy_pages(*g, src, dst, (int)m, w, status, stream);
  if (e != hipSuccess) return fail_hip(e, "ep_kv_copy_pages");
  return EP_OK;
}

int ep_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor, double orig_tokens,
                  double beta_fast, double beta_slow, float* inv_freq, float* mscale) {
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 256)
    return fail(EP_ERR_INVALID_ARG, "ep_rope_freqs: rot_dim must be even, from 2 to 256");
  if (!inv_freq || !mscale) return fail(EP_ERR_INVALID_ARG, "ep_rope_freqs: null output");
  if (!(base > 1.0) || !std::isfinite(base))
    return fail(EP_ERR_INVALID_ARG, "ep_rope_freqs: base must be over 1");
  if (scaling < EP_ROPE_NONE || scaling > EP_ROPE_YARN)
    return fail(EP_ERR_INVALID_ARG, "ep_rope_freqs: unknown scaling");
  if (scaling != EP_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(EP_ERR_INVALID_ARG, "ep_rope_freqs: factor must be at least 1");
  double lo = 0.0, hi = 0.0;
  *mscale = 1.0f;
  if (scaling == EP_ROPE_YARN) {
    if (!(orig_tokens > 0.0) || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) ||
        !std::isfinite(orig_tokens) || !std::isfinite(beta_fast))
      return fail(EP_ERR_INVALID_ARG,
                  "ep_rope_freqs: YaRN needs orig_tokens > 0 and beta_fast >= beta_slow > 0");
    // Pair i turns orig / (2 pi base^(2 i / rot)) times; solved for i.
    const auto pair_of = [&](double turns) {
      return rot_dim * std::log(orig_tokens / (turns * 2.0 * M_PI)) / (2.0 * std::log(base));
    };
    lo = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
    hi = std::fmin(std::ceil(pair_of(beta_slow)), rot_dim - 1.0);
    *mscale = (float)(0.1 * std::log(factor) + 1.0);
  }
  if (scaling == EP_ROPE_NTK && rot_dim > 2) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == EP_ROPE_LINEAR) f /= factor;
    if (scaling == EP_ROPE_YARN) {
      const double r = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
      f = f / factor * r + f * (1.0 - r);
    }
    inv_freq[i] = (float)f;
  }
  return EP_OK;
}

int ep_kv_append(const ep_kv_cache* c, const ep_kv_batch* b, const ep_rows* q, int32_t n_heads,
                 const ep_rows* k, const ep_rows* v, const ep_rows* q_out, const ep_rope* rope,
                 int32_t* status, hipStream_t stream) {
  EP_CHECK(check_cache(c));
  EP_CHECK(check_batch(b, *c));
  const bool queries = q && q->p;
  if (queries != (q_out && q_out->p))
    return fail(EP_ERR_INVALID_ARG, "q and q_out must be given together");
  if (queries) EP_CHECK(check_heads(*c, n_heads));
  ep_rope r{nullptr, 0, EP_ROPE_HALF, 1.0f, 0};
  if (rope) {
    r = *rope;
    if (r.rot_dim < 0 || r.rot_dim % 2 != 0 || r.rot_dim > c->head_dim)
      return fail(EP_ERR_INVALID_ARG, "rope: rot_dim must be even and at most head_dim");
    if (r.layout != EP_ROPE_HALF && r.layout != EP_ROPE_INTERLEAVED)
      return fail(EP_ERR_INVALID_ARG, "rope: unknown layout");
    if (r.reserved != 0) return fail(EP_ERR_INVALID_ARG, "rope: reserved must be 0");
  }
  DeviceScope scope(stream);
  if (scope.error() != hipSuccess) return fail_hip(scope.error(), "device");
  const int dev = scope.device();
  EP_CHECK(check_ptr(status, dev, "status", 4));
  if (b->n_tokens == 0 || b->n_seqs == 0) return EP_OK;
  EP_CHECK(check_cache_ptrs(*c, dev));
  EP_CHECK(check_batch_ptrs(*b, dev));
  EP_CHECK(check_ptr(r.inv_freq, dev, "rope.inv_freq", (int64_t)r.rot_dim * 2));
  EP_CHECK(check_rows(k, c->n_heads, *b, c->head_dim, "k", dev));
  EP_CHECK(check_rows(v, c->n_heads, *b, c->head_dim, "v", dev));
  if (queries) {
    EP_CHECK(check_rows(q, n_heads, *b, c->head_dim, "q", dev));
    EP_CHECK(check_rows(q_out, n_heads, *b, c->head_dim, "q_out", dev));
    EP_CHECK(check_apart(*q_out, n_heads, *b, c->head_dim, "q_out"));
    if (q->p == q_out->p &&
        (q->token_stride != q_out->token_stride || q->head_stride != q_out->head_stride))
      return fail(EP_ERR_INVALID_ARG, "q in place needs q_out with the same strides");
  }
  const ep_rows none{nullptr, 0, 0};
  const hipError_t e = ep::launch_kv_append(*c, *b, queries ? *q : none, queries ? n_heads : 0, *k,
                                            *v, queries ? *q_out : none, r, status, stream);
  if (e != hipSuccess) return fail_hip(e, "ep_kv_append");
  return EP_OK;
}

size_t ep_kv_attend_bytes(const ep_kv_cache* c, int32_t n_seqs, int32_t n_groups, int32_t n_tokens,
                          int32_t n_heads, int32_t max_new) {
  if (check_cache(c) != EP_OK || check_heads(*c, n_heads) != EP_OK) return 0;
  if (n_seqs < 0 || n_groups < 0 || n_tokens < 0 || n_tokens > (1 << 24) || max_new < 1) {
    fail(EP_ERR_INVALID_ARG, "ep_kv_attend_bytes: bad sizes");
    return 0;
  }
  if ((int64_t)n_tokens * n_heads >= (int64_t)1 << 31) {
    fail(EP_ERR_UNSUPPORTED, "n_tokens * n_heads must be < 2^31");
    return 0;
  }
  return ep::kv_attend_bytes(*c, n_seqs, n_groups, n_tokens, n_heads, max_new);
}

int ep_kv_attend(const ep_kv_cache* c, const ep_kv_batch* b, const ep_kv_groups* groups,
                 int32_t max_new, const ep_rows* q, int32_t n_heads, const ep_rows* out,
                 float* lse, float sm_scale, void* ws, int32_t* status, hipStream_t stream) {
  EP_CHECK(check_cache(c));
  EP_CHECK(check_batch(b, *c));
  EP_CHECK(check_heads(*c, n_heads));
  if (max_new < 1) return fail(EP_ERR_INVALID_ARG, "max_new must be positive");
  if (!std::isfinite(sm_scale)) return fail(EP_ERR_INVALID_ARG, "sm_scale must be finite");
  ep_kv_groups g{nullptr, nullptr, 0, 0};
  if (groups) g = *groups;
  if (g.n_groups < 0 || g.reserved != 0)
    return fail(EP_ERR_INVALID_ARG, "groups: bad sizes, or reserved not 0");
  if ((int64_t)b->n_tokens * n_heads >= (int64_t)1 << 31)
    return fail(EP_ERR_UNSUPPORTED, "n_tokens * n_heads must be < 2^31");
  DeviceScope scope(stream);
  if (scope.error() != hipSuccess) return fail_hip(scope.error(), "device");
  const int dev = scope.device();
  EP_CHECK(check_ptr(status, dev, "status", 4));
  if (b->n_tokens == 0 || b->n_seqs == 0) return EP_OK;
  EP_CHECK(check_cache_ptrs(*c, dev));
  EP_CHECK(check_batch_ptrs(*b, dev));
  if (g.n_groups > 0) {
    EP_CHECK(check_ptr(g.group_off, dev, "group_off", ((int64_t)g.n_groups + 1) * 4));
    EP_CHECK(check_ptr(g.shared, dev, "shared", (int64_t)g.n_groups * 4));
  }
  EP_CHECK(check_rows(q, n_heads, *b, c->head_dim, "q", dev));
  EP_CHECK(check_rows(out, n_heads, *b, c->head_dim, "out", dev));
  EP_CHECK(check_apart(*out, n_heads, *b, c->head_dim, "out"));
  // Rows of q are read again after others were written.
  if (out->p == q->p) return fail(EP_ERR_INVALID_ARG, "out may not be q");
  if (lse) EP_CHECK(check_ptr(lse, dev, "lse", (int64_t)b->n_tokens * n_heads * 4));
  EP_CHECK(check_ptr(ws, dev, "ws",
                     (int64_t)ep::kv_attend_bytes(*c, b->n_seqs, g.n_groups, b->n_tokens, n_heads,
                                                  max_new)));
  EP_CHECK(check_aligned16(ws, "ws"));
  const hipError_t e = ep::launch_kv_attend(*c, *b, g, max_new, *q, n_heads, *out, lse, sm_scale,
                                            ws, status, stream);
  if (e != hipSuccess) return fail_hip(e, "ep_kv_attend");
  return EP_OK;
}

}  // extern "C"
