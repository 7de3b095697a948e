// A descriptor's checks, the plan workspace's layout and the common prologue
// of the calls that take both, shared by the C ABI's translation units.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "ep.h"
#include "ep_checks.hpp"
#include "ep_kernels.hpp"

namespace ep {

constexpr int64_t kMaxWaves = (int64_t)1 << 26;  // grid.x * 64 threads < 2^32

inline int64_t bound_of(const ep_desc* d) {
  const int64_t L = d->n_experts / d->n_ranks;
  const int64_t m = d->topk > L ? d->topk : L;
  return (int64_t)d->n_ranks * d->tokens * m;
}

// Validate a descriptor and derive sizes. Returns EP_OK or a negative code.
inline int derive(const ep_desc* d, Dims* o) {
  if (!d) return fail(EP_ERR_INVALID_ARG, "null descriptor");
  if (d->n_ranks <= 0 || d->tokens < 0 || d->hidden <= 0 || d->n_experts <= 0 || d->topk <= 0)
    return fail(EP_ERR_INVALID_ARG, "sizes must be positive (tokens may be 0)");
  if (d->n_experts % d->n_ranks != 0)
    return fail(EP_ERR_INVALID_ARG, "n_experts must be a multiple of n_ranks");
  if (d->payload != EP_PAYLOAD_BF16 && d->payload != EP_PAYLOAD_FP8_B128)
    return fail(EP_ERR_INVALID_ARG, "unknown payload");
  if (d->payload == EP_PAYLOAD_BF16 && d->hidden % 8 != 0)
    return fail(EP_ERR_INVALID_ARG, "bf16 payload needs hidden % 8 == 0");
  if (d->payload == EP_PAYLOAD_FP8_B128 && d->hidden % 128 != 0)
    return fail(EP_ERR_INVALID_ARG, "fp8 payload needs hidden % 128 == 0");
  if (d->cap_rows < 0) return fail(EP_ERR_INVALID_ARG, "cap_rows must be >= 0");
  if (d->n_experts > EP_MAX_EXPERTS) return fail(EP_ERR_UNSUPPORTED, "too many experts");
  if (d->topk > EP_MAX_TOPK) return fail(EP_ERR_UNSUPPORTED, "topk too large");
  const int64_t cap = d->cap_rows > 0 ? d->cap_rows : bound_of(d);
  const int64_t NTR = (int64_t)d->n_ranks * d->tokens * d->topk;
  // A zero capacity only arises from the bound with no tokens at all.
  if ((int64_t)d->n_ranks * cap >= ((int64_t)1 << 31))
    return fail(EP_ERR_UNSUPPORTED, "n_ranks * cap_rows must be < 2^31");
  if (NTR >= kMaxWaves) return fail(EP_ERR_UNSUPPORTED, "n_ranks * tokens * topk must be < 2^26");
  o->N = d->n_ranks;
  o->T = d->tokens;
  o->H = d->hidden;
  o->E = d->n_experts;
  o->R = d->topk;
  o->L = d->n_experts / d->n_ranks;
  o->payload = d->payload;
  o->planes = d->payload == EP_PAYLOAD_BF16 ? 1 : 2;
  o->cap = cap;
  o->TR = (int64_t)d->tokens * d->topk;
  o->NT = (int64_t)d->n_ranks * d->tokens;
  o->NTR = NTR;
  if (d->payload == EP_PAYLOAD_BF16) {
    o->row[0] = 2 * (int64_t)d->hidden;
    o->row[1] = 0;
  } else {
    o->row[0] = d->hidden;
    o->row[1] = 4 * (int64_t)(d->hidden / 128);
  }
  const int64_t nch = (o->TR + kPlanChunk - 1) / kPlanChunk;
  o->nchunks = (int)(nch > 0 ? nch : 1);
  // Windowed sender: windows of the largest power-of-two token count whose
  // rows fit kGatherSourceBytes.
  const int64_t tok_bytes = o->row[0] + o->row[1];
  const int64_t src_bytes = (int64_t)d->tokens * tok_bytes;
  o->win = 0;
  o->nwin = 0;
  if (src_bytes > kGatherSourceBytes && src_bytes <= kWindowSourceBytes &&
      NTR * tok_bytes <= kWindowSendBytes) {
    int64_t w = 1;
    while (2 * w * tok_bytes <= kGatherSourceBytes) w *= 2;
    o->win = (int)w;
    o->nwin = (int)((d->tokens + w - 1) / w);
  }
  // Bound on the copy grids: the row copies launch one wave per 1 KB piece
  // of a row (a plane under 1 KB counts as one piece), so one launch stays
  // under 2^26 waves: 2^32 work-items of 64 lanes, the most one dispatch
  // can hold.
  int64_t pieces = 0;
  for (int q = 0; q < o->planes; ++q) pieces += (o->row[q] + 1023) / 1024;
  if (NTR * pieces >= kMaxWaves)
    return fail(EP_ERR_UNSUPPORTED,
                "n_ranks * tokens * topk * (1 KB pieces per row) must be < 2^26");
  return EP_OK;
}

// Plan workspace: int32 arrays, each starting on a 256-byte boundary.
struct Layout {
  size_t off[14];
  size_t bytes;
};

inline Layout layout_of(const Dims& d) {
  const size_t n[14] = {
      (size_t)d.N * d.E,                       // cnt
      (size_t)d.N * (d.E + 1),                 // send_off
      (size_t)d.NTR,                           // send_pos
      (size_t)d.N * (d.N + 1),                 // recv_off
      (size_t)d.N * (d.L + 1),                 // grp_off
      (size_t)d.NTR,                           // grp_pos
      (size_t)d.N * d.E,                       // src_off
      (size_t)d.NTR,                           // comb_row
      (size_t)d.NTR,                           // grp_slot
      (size_t)d.N * d.nchunks * d.E,           // chunk_cnt
      (size_t)d.NTR,                           // send_slot
      (size_t)2 * d.NTR,                       // recv_rows
      (size_t)d.NTR,                           // send_seg
      (size_t)2 * d.N * d.nwin * d.win * d.R,  // win_list (windowed sender only)
  };
  Layout l{};
  size_t at = 0;
  for (int i = 0; i < 14; ++i) {
    l.off[i] = at;
    at += (n[i] * sizeof(int32_t) + 255) & ~(size_t)255;
  }
  l.bytes = at > 0 ? at : 256;
  return l;
}

inline PlanPtrs plan_ptrs(const Dims& d, const void* ws) {
  const Layout l = layout_of(d);
  char* b = (char*)ws;
  PlanPtrs p;
  p.cnt = (int32_t*)(b + l.off[0]);
  p.send_off = (int32_t*)(b + l.off[1]);
  p.send_pos = (int32_t*)(b + l.off[2]);
  p.recv_off = (int32_t*)(b + l.off[3]);
  p.grp_off = (int32_t*)(b + l.off[4]);
  p.grp_pos = (int32_t*)(b + l.off[5]);
  p.src_off = (int32_t*)(b + l.off[6]);
  p.comb_row = (int32_t*)(b + l.off[7]);
  p.grp_slot = (int32_t*)(b + l.off[8]);
  p.chunk_cnt = (int32_t*)(b + l.off[9]);
  p.send_slot = (int32_t*)(b + l.off[10]);
  p.recv_rows = (int32_t*)(b + l.off[11]);
  p.send_seg = (int32_t*)(b + l.off[12]);
  p.win_list = d.win > 0 ? (int32_t*)(b + l.off[13]) : nullptr;
  return p;
}

// rows: rows of every plane buffer (its bytes are rows * row bytes).
inline int check_planes(const Dims& d, const void* const* pl, int dev, const char* name,
                 int64_t rows) {
  if (!pl) return fail(EP_ERR_INVALID_ARG, (std::string("null plane array: ") + name).c_str());
  for (int q = 0; q < d.planes; ++q) {
    int rc = check_ptr(pl[q], dev, name, rows * d.row[q]);
    if (rc != EP_OK) return rc;
    rc = check_aligned16(pl[q], name);
    if (rc != EP_OK) return rc;
  }
  if (d.planes == 1 && pl[1] != nullptr)
    return fail(EP_ERR_INVALID_ARG, (std::string("plane 1 must be NULL for bf16: ") + name).c_str());
  return EP_OK;
}

// Common prologue: descriptor, device scope, workspace pointer.
#define EP_PROLOGUE(desc, stream, ws)                                            \
  ep::Dims dims;                                                                 \
  {                                                                              \
    const int rc_ = ep::derive(desc, &dims);                                     \
    if (rc_ != EP_OK) return rc_;                                                \
  }                                                                              \
  ep::DeviceScope scope(stream);                                                 \
  if (scope.error() != hipSuccess) return ep::fail_hip(scope.error(), "device"); \
  {                                                                              \
    int rc_ = ep::check_ptr(ws, scope.device(), "plan_ws",                       \
                            (int64_t)ep::layout_of(dims).bytes);                 \
    if (rc_ == EP_OK) rc_ = ep::check_aligned16(ws, "plan_ws");                  \
    if (rc_ != EP_OK) return rc_;                                                \
  }                                                                              \
  const ep::PlanPtrs pp = ep::plan_ptrs(dims, ws);

}  // namespace ep
