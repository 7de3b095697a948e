// Pages of a KV cache: extend, fork, free, compact and copy, on the tables,
// lengths, reference counts and pool that the KV push fills.
//
// All of it is integer bookkeeping and page copies, so the bounds are the
// latency of a few dependent launches and, where pages move, the copy rate
// of HBM (2 bytes of traffic per byte moved). Two choices follow:
//   - No free list: a page is free when its count is not positive, and the
//     k-th page handed out is the k-th free one. The list would have to be
//     kept in order under concurrent pushes and pops; finding free pages is
//     one pass over 4 bytes per page (8192 pages: one load per thread and
//     eighth of the pass), by one workgroup that stops as soon as it has
//     enough.
//   - The bookkeeping of the requests runs in one workgroup per call (the
//     prefix sums over requests and the allocation are sequential in
//     nature); page copies and table rows run in a second launch over the
//     whole chip.
#include "ep_device.hpp"
#include "ep_kernels.hpp"

namespace ep {
namespace {

constexpr int kPlan = 1024;               // threads of the planning workgroup
constexpr int kPlanWaves = kPlan / kWave;
constexpr int kScan = 8;                  // refs per thread and pass
constexpr int kBlock = 256;
// A copy's workgroup is one wave that has 8 KB on its way, page sizes being
// mostly powers of two: 268 MB in 32 KB pages take 54 us, 5.0 TB/s, as with
// pieces of 16 KB by four waves.
constexpr int kChunks = 8;                // 16-byte chunks per lane
constexpr int64_t kPieceBytes = (int64_t)kWave * kChunks * 16;
constexpr int32_t kNone = 0x7fffffff;

__device__ __forceinline__ void flag(int32_t* status, int32_t bits) {
  if (bits) atomicOr(status, bits);
}

// Values that other threads of the launch change with atomics are read past
// the vector cache.
__device__ __forceinline__ int32_t load_fresh(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_fresh(int32_t* p, int32_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Barrier after which every thread of the workgroup sees what the others
// stored or changed with atomics: their accesses have reached the L2.
__device__ __forceinline__ void settle() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

// Inclusive sum over the planning workgroup; every thread calls it. `total`
// gets the sum over all threads. `part` holds one value per wave.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part, int64_t* total) {
  const int lane = lane_id(), wave = threadIdx.x / kWave;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int64_t u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  if (lane == kWave - 1) part[wave] = v;
  __syncthreads();
  int64_t before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    const int64_t p = part[w];
    if (w < wave) before += p;
    sum += p;
  }
  *total = sum;
  __syncthreads();
  return v + before;
}

__device__ __forceinline__ void load_refs(const int32_t* refs, int n_pages, int64_t base,
                                          int32_t r[kScan]) {
#pragma unroll
  for (int j = 0; j < kScan; ++j) {
    const int64_t p = base + j * kPlan + threadIdx.x;
    r[j] = refs[p < n_pages ? p : n_pages - 1];
  }
}

// The lowest free pages in ascending order into list[0, min(want, free));
// returns how many were found. Whole workgroup. r: the counts of the first
// pass, loaded ahead.
__device__ __forceinline__ int64_t find_free(const int32_t* refs, int n_pages, int64_t want,
                                             int32_t r[kScan], int32_t* list, int32_t* counts) {
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  int64_t found = 0;
  for (int64_t base = 0; base < n_pages && found < want; base += (int64_t)kPlan * kScan) {
    uint64_t mask[kScan];
    if (base > 0) load_refs(refs, n_pages, base, r);
#pragma unroll
    for (int j = 0; j < kScan; ++j) {
      const int64_t p = base + j * kPlan + threadIdx.x;
      mask[j] = ballot(p < n_pages && r[j] <= 0);
      if (lane == 0) counts[j * kPlanWaves + wave] = __popcll(mask[j]);
    }
    __syncthreads();
    // Sums before (j, wave) over the kScan * kPlanWaves counts, by one wave.
    if (wave == 0) {
      constexpr int kPer = kScan * kPlanWaves / kWave;
      int32_t c[kPer], sum = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        c[k] = counts[lane * kPer + k];
        sum += c[k];
      }
      int32_t incl = sum;
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) {
        const int32_t u = __shfl_up(incl, d);
        if (lane >= d) incl += u;
      }
      int32_t at = incl - sum;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        counts[lane * kPer + k] = at;
        at += c[k];
      }
      if (lane == kWave - 1) counts[kScan * kPlanWaves] = at;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kScan; ++j) {
      const int64_t at = found + counts[j * kPlanWaves + wave] + __popcll(mask[j] & lanes_below());
      if (((mask[j] >> lane) & 1) && at < want)
        list[at] = (int32_t)(base + j * kPlan + threadIdx.x);
    }
    found += counts[kScan * kPlanWaves];
    __syncthreads();
  }
  return found < want ? found : want;
}

// What a call of few requests needs stays in LDS: the marks of up to kMarks
// sequences, the starts of up to kPlan requests and kList pages. A trip
// through memory and back is most of a microsecond, and the planning would
// take four of them.
constexpr int kMarks = 8192, kList = 4096;

struct PagesShared {
  int64_t part[kPlanWaves];
  int32_t counts[kScan * kPlanWaves + 1];
  int32_t first[kMarks], start[kPlan], list[kList];
};

// Pages that hold `n` tokens.
__device__ __forceinline__ int64_t pages_of(int64_t n, int page_tokens) {
  return (n + page_tokens - 1) / page_tokens;
}

__device__ __forceinline__ int64_t used_pages(int32_t len, const ep_kv_pages& g) {
  const int64_t n = pages_of(len > 0 ? len : 0, g.page_tokens);
  return n < g.max_pages ? n : g.max_pages;
}

// What a request needs: -1 when it is out of range, else its pages.
// ADD: a sequence `seq` grows by arg tokens; otherwise child `seq` copies
// parent arg.
template <bool ADD>
__device__ __forceinline__ int64_t need_of(const ep_kv_pages& g, int32_t seq, int32_t arg) {
  if (seq < 0 || seq >= g.n_seqs) return -1;
  const int64_t cap = (int64_t)g.max_pages * g.page_tokens;
  if (ADD) {
    const int64_t len = g.lens[seq];
    if (arg < 0 || len < 0 || len > cap || len + arg > cap || len + arg > 0x7fffffff) return -1;
    return pages_of(len + arg, g.page_tokens) - pages_of(len, g.page_tokens);
  }
  if (arg < 0 || arg >= g.n_seqs || g.lens[seq] != 0) return -1;
  const int64_t len = g.lens[arg];
  if (len < 0 || len > cap) return -1;
  return len % g.page_tokens != 0;
}

// Marks the first request of every sequence, and lays out the needs: start[i]
// = pages needed by the valid requests before i, or -1 for a skipped one.
// Returns the total need. Whole workgroup.
template <bool ADD>
__device__ __forceinline__ int64_t lay_out(const ep_kv_pages& g, const int32_t* seqs,
                                           const int32_t* args, int m, const PagesWs& ws,
                                           PagesShared& sh, int32_t* start_of,
                                           int32_t* status) {
  const bool small = g.n_seqs <= kMarks;
  for (int i = threadIdx.x; i < m; i += kPlan) {
    const int32_t s = seqs[i];
    if (s < 0 || s >= g.n_seqs) continue;
    if (small) sh.first[s] = kNone;
    else store_fresh(&ws.first[s], kNone);
  }
  settle();
  for (int i = threadIdx.x; i < m; i += kPlan) {
    const int32_t s = seqs[i];
    if (s < 0 || s >= g.n_seqs) continue;
    if (small) atomicMin(&sh.first[s], i);
    else atomicMin(&ws.first[s], i);
  }
  settle();
  int64_t base = 0;
  bool bad = false;
  for (int i0 = 0; i0 < m; i0 += kPlan) {
    const int i = i0 + threadIdx.x;
    int64_t need = -1;
    if (i < m) {
      need = need_of<ADD>(g, seqs[i], args[i]);
      if (need >= 0 && (small ? sh.first[seqs[i]] : load_fresh(&ws.first[seqs[i]])) != i)
        need = -1;
      bad |= need < 0;
    }
    const int64_t n = need > 0 ? need : 0;
    int64_t sum;
    const int64_t incl = base + block_scan(n, sh.part, &sum);
    // Starts past the pool's size are never granted: they saturate.
    const int64_t start = incl - n;
    if (i < m) start_of[i] = need < 0 ? -1 : (int32_t)(start < kNone ? start : kNone);
    base += sum;
  }
  if (bad) flag(status, EP_STATUS_BAD_PAGE);
  return base;
}

__global__ __launch_bounds__(kPlan) void extend_kernel(ep_kv_pages g, const int32_t* seqs,
                                                       const int32_t* add, int m, PagesWs ws,
                                                       int32_t* status) {
  __shared__ PagesShared sh;
  int32_t r[kScan];
  load_refs(g.refs, g.n_pages, 0, r);
  int32_t* start_of = m <= kPlan ? sh.start : ws.start;
  const int64_t total = lay_out<true>(g, seqs, add, m, ws, sh, start_of, status);
  int32_t* list = total <= kList ? sh.list : ws.pages;
  const int64_t found = find_free(g.refs, g.n_pages, total, r, list, sh.counts);
  settle();
  for (int i = threadIdx.x / kWave; i < m; i += kPlanWaves) {
    const int64_t start = start_of[i];
    if (start < 0) continue;
    const int32_t s = seqs[i], len = g.lens[s], n = add[i];
    const int64_t have = pages_of(len, g.page_tokens);
    const int64_t need = pages_of((int64_t)len + n, g.page_tokens) - have;
    if (need > 0 && start + need > found) {
      if (lane_id() == 0) flag(status, EP_STATUS_CAPACITY);
      continue;
    }
    int32_t* row = g.tables + (int64_t)s * g.max_pages + have;
    for (int64_t k = lane_id(); k < need; k += kWave) {
      const int32_t p = list[start + k];
      row[k] = p;
      g.refs[p] = 1;
    }
    if (lane_id() == 0) g.lens[s] = len + n;
  }
}

// The plan of a fork: start[i] becomes the new page of request i, -1 where
// it is skipped or refused, -2 where it needs none; len[i] the parent's
// length as it was.
__global__ __launch_bounds__(kPlan) void fork_plan_kernel(ep_kv_pages g, const int32_t* parents,
                                                          const int32_t* children, int m,
                                                          PagesWs ws, int32_t* status) {
  __shared__ PagesShared sh;
  int32_t r[kScan];
  load_refs(g.refs, g.n_pages, 0, r);
  const int64_t total = lay_out<false>(g, children, parents, m, ws, sh, ws.start, status);
  int32_t* list = total <= kList ? sh.list : ws.pages;
  const int64_t found = find_free(g.refs, g.n_pages, total, r, list, sh.counts);
  settle();
  for (int i = threadIdx.x; i < m; i += kPlan) {
    const int64_t start = ws.start[i];
    if (start < 0) continue;
    const int32_t len = g.lens[parents[i]];
    ws.len[i] = len;
    int32_t page = -2;
    if (len % g.page_tokens != 0) {
      page = start < found ? list[start] : -1;
      if (page < 0) flag(status, EP_STATUS_CAPACITY);
    }
    ws.start[i] = page;
  }
}

// Piece q of a page, by one wave.
__device__ __forceinline__ void copy_piece(const uint8_t* src, uint8_t* dst, int q, int64_t n16) {
  RowRegs<kChunks> r;
  const int64_t c0 = (int64_t)q * kWave * kChunks;
  const int n = (int)(n16 - c0 < kWave * kChunks ? n16 - c0 : kWave * kChunks);
  load_row16(r, (const u32x4*)src + c0, 0, n);
  store_row16(r, (u32x4*)dst + c0, 0, n);
}

// Block (i, 0): the child's row, counts and length. Block (i, 1 + r * pieces
// + q): piece q of the partly filled page, in rank r.
__global__ __launch_bounds__(kWave) void fork_apply_kernel(ep_kv_pages g, const int32_t* parents,
                                                            const int32_t* children, PagesWs ws,
                                                            int pieces, int32_t* status) {
  const int i = blockIdx.x;
  const int32_t page = ws.start[i];
  if (page == -1) return;
  const int32_t len = ws.len[i], full = len / g.page_tokens;
  const int32_t* from = g.tables + (int64_t)parents[i] * g.max_pages;
  if (blockIdx.y == 0) {
    int32_t* to = g.tables + (int64_t)children[i] * g.max_pages;
    bool bad = false;
    for (int k = threadIdx.x; k < g.max_pages; k += kWave) {
      int32_t p = -1;
      if (k < full) {
        p = from[k];
        if (p >= 0 && p < g.n_pages) atomicAdd(&g.refs[p], 1);
        else bad = true;
      } else if (k == full && page >= 0) {
        p = page;
        g.refs[p] = 1;
      }
      to[k] = p;
    }
    if (threadIdx.x == 0) g.lens[children[i]] = len;
    if (bad) flag(status, EP_STATUS_BAD_PAGE);
    return;
  }
  if (page < 0) return;
  const int32_t src = from[full];
  if (src < 0 || src >= g.n_pages) {
    if (threadIdx.x == 0) flag(status, EP_STATUS_BAD_PAGE);
    return;
  }
  const int r = (blockIdx.y - 1) / pieces, q = (blockIdx.y - 1) % pieces;
  uint8_t* base = (uint8_t*)g.pool + r * g.rank_bytes;
  copy_piece(base + src * g.page_bytes, base + page * g.page_bytes, q, g.page_bytes / 16);
}

// One block per request. The first request of a sequence is the one that no
// earlier request equals: each block compares its own with those before it
// rather than wait for a launch that marks them. That is quadratic in m, at
// most 16384: 3.1 us for 128 requests, 4.0 for 1024, 8.7 for 4096, 48.8 for
// 16384.
__global__ __launch_bounds__(kBlock) void free_kernel(ep_kv_pages g, const int32_t* seqs,
                                                      int32_t* status) {
  const int i = blockIdx.x;
  const int32_t s = seqs[i];
  bool skip = s < 0 || s >= g.n_seqs;
  for (int j = threadIdx.x; j < i; j += kBlock) skip |= seqs[j] == s;
  if (__syncthreads_or(skip)) {
    if (threadIdx.x == 0) flag(status, EP_STATUS_BAD_PAGE);
    return;
  }
  const int32_t len = g.lens[s];
  const int64_t n = used_pages(len, g);
  bool bad = len < 0 || len > (int64_t)g.max_pages * g.page_tokens;
  int32_t* row = g.tables + (int64_t)s * g.max_pages;
  for (int64_t k = threadIdx.x; k < g.max_pages; k += kBlock) {
    if (k < n) {
      const int32_t p = row[k];
      if (p < 0 || p >= g.n_pages) {
        bad = true;
      } else if (atomicSub(&g.refs[p], 1) <= 0) {
        atomicAdd(&g.refs[p], 1);
        bad = true;
      }
    }
    row[k] = -1;
  }
  __syncthreads();  // every thread has read lens[s]
  if (threadIdx.x == 0) g.lens[s] = 0;
  if (bad) flag(status, EP_STATUS_BAD_PAGE);
}

// ---------------------------------------------------------------------------
// Compaction. counts[c]: used pages of chunk c (kCompact pages each).
// ---------------------------------------------------------------------------
constexpr int kCompact = kKvCompactChunk;
constexpr int kPer = kCompact / kBlock;
// Up to so many chunks every block counts all pages itself, which spares a
// launch (4.5 us for 2048 pages).
constexpr int kCompactAlone = 4;

__device__ __forceinline__ int block_sum(int v, int* part) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
  if (lane_id() == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kBlock / kWave; ++w) s += part[w];
  __syncthreads();
  return s;
}

__global__ __launch_bounds__(kBlock) void compact_count_kernel(ep_kv_pages g, PagesWs ws) {
  __shared__ int part[kBlock / kWave];
  const int64_t base = (int64_t)blockIdx.x * kCompact;
  int n = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int64_t p = base + j * kBlock + threadIdx.x;
    n += p < g.n_pages && g.refs[p] > 0;
  }
  n = block_sum(n, part);
  if (threadIdx.x == 0) ws.counts[blockIdx.x] = n;
}

// Block c ranks the pages of chunk c: with L used pages in all, a used page
// p >= L is mover number used(p) - used(L), a free page p < L is hole number
// p - used(p), where used(x) counts the used pages below x.
__global__ __launch_bounds__(kBlock) void compact_rank_kernel(ep_kv_pages g, PagesWs ws,
                                                              int chunks, int32_t* n_live) {
  __shared__ int part[kBlock / kWave];
  const int c = blockIdx.x;
  int before = 0, all = 0;
  if (chunks <= kCompactAlone) {
    for (int64_t p = threadIdx.x; p < g.n_pages; p += kBlock) {
      const int used = g.refs[p] > 0;
      all += used;
      if (p < (int64_t)c * kCompact) before += used;
    }
  } else {
    for (int j = threadIdx.x; j < chunks; j += kBlock) {
      const int n = ws.counts[j];
      all += n;
      if (j < c) before += n;
    }
  }
  before = block_sum(before, part);
  const int live = block_sum(all, part);
  // used(L): the chunks before L's, and the part of its own chunk.
  const int lc = chunks <= kCompactAlone ? 0 : live / kCompact;
  int below = 0;
  for (int j = threadIdx.x; j < lc; j += kBlock) below += ws.counts[j];
  for (int64_t p = (int64_t)lc * kCompact + threadIdx.x; p < live; p += kBlock)
    below += g.refs[p] > 0;
  below = block_sum(below, part);
  if (c == 0 && threadIdx.x == 0) {
    ws.counts[chunks] = live - below;  // moves
    if (n_live) *n_live = live;
  }
  const int wave = threadIdx.x / kWave;
  int at = before;  // used pages below the block's current row of kBlock pages
  for (int j = 0; j < kPer; ++j) {
    const int64_t p = (int64_t)c * kCompact + j * kBlock + threadIdx.x;
    const bool used = p < g.n_pages && g.refs[p] > 0;
    const uint64_t mask = ballot(used);
    if (lane_id() == 0) part[wave] = __popcll(mask);
    __syncthreads();
    int mine = at + __popcll(mask & lanes_below()), sum = 0;
#pragma unroll
    for (int w = 0; w < kBlock / kWave; ++w) {
      if (w < wave) mine += part[w];
      sum += part[w];
    }
    __syncthreads();
    at += sum;
    if (p >= g.n_pages) continue;
    int32_t rank = -1;
    if (used && p >= live) {
      rank = mine - below;
      ws.src[rank] = (int32_t)p;
    } else if (!used && p < live) {
      ws.dst[p - mine] = (int32_t)p;
    }
    ws.rank[p] = rank;
    ws.pages[p] = -1;  // a mover's new page follows with its copy
  }
}

// Tables (by the first row_blocks waves), pages and counts.
__global__ __launch_bounds__(kWave) void compact_apply_kernel(ep_kv_pages g, PagesWs ws,
                                                              int chunks, int row_blocks,
                                                              int pieces, int32_t* status) {
  const int moves = ws.counts[chunks];
  if ((int)blockIdx.x < row_blocks) {
    bool bad = false;
    for (int s = blockIdx.x; s < g.n_seqs; s += row_blocks) {
      const int64_t n = used_pages(g.lens[s], g);
      int32_t* row = g.tables + (int64_t)s * g.max_pages;
      for (int64_t k = threadIdx.x; k < n; k += kWave) {
        const int32_t p = row[k];
        if (p < 0 || p >= g.n_pages) {
          bad = true;
          continue;
        }
        const int32_t rank = ws.rank[p];
        if (rank >= 0) row[k] = ws.dst[rank];
      }
    }
    if (bad) flag(status, EP_STATUS_BAD_PAGE);
    return;
  }
  const int64_t units = (int64_t)moves * g.ranks * pieces;
  for (int64_t u = blockIdx.x - row_blocks; u < units; u += gridDim.x - row_blocks) {
    const int64_t j = u / ((int64_t)g.ranks * pieces);
    const int rest = (int)(u - j * g.ranks * pieces), r = rest / pieces, q = rest % pieces;
    const int32_t src = ws.src[j], dst = ws.dst[j];
    uint8_t* base = (uint8_t*)g.pool + r * g.rank_bytes;
    copy_piece(base + src * g.page_bytes, base + dst * g.page_bytes, q, g.page_bytes / 16);
    if (rest == 0 && threadIdx.x == 0) {
      g.refs[dst] = g.refs[src];
      g.refs[src] = 0;
      ws.pages[src] = dst;
    }
  }
}

// ---------------------------------------------------------------------------
// Copies by list. owner[p]: the first pair that writes page p.
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool pair_in_range(const ep_kv_pages& g, int32_t s, int32_t d) {
  return s >= 0 && s < g.n_pages && d >= 0 && d < g.n_pages;
}

__global__ __launch_bounds__(kBlock) void copy_clear_kernel(ep_kv_pages g, const int32_t* src,
                                                            const int32_t* dst, int m,
                                                            PagesWs ws) {
  const int i = blockIdx.x * kBlock + threadIdx.x;
  if (i >= m || !pair_in_range(g, src[i], dst[i])) return;
  ws.pages[src[i]] = kNone;
  ws.pages[dst[i]] = kNone;
}

__global__ __launch_bounds__(kBlock) void copy_own_kernel(ep_kv_pages g, const int32_t* src,
                                                          const int32_t* dst, int m, PagesWs ws) {
  const int i = blockIdx.x * kBlock + threadIdx.x;
  if (i >= m || !pair_in_range(g, src[i], dst[i]) || src[i] == dst[i]) return;
  atomicMin(&ws.pages[dst[i]], i);
}

__global__ __launch_bounds__(kWave) void copy_pages_kernel(ep_kv_pages g, const int32_t* src,
                                                            const int32_t* dst, PagesWs ws,
                                                            int pieces, int32_t* status) {
  const int i = blockIdx.x;
  const int32_t s = src[i], d = dst[i];
  const bool ok = pair_in_range(g, s, d);
  if (ok && s == d) return;
  if (!ok || ws.pages[d] != i || ws.pages[s] != kNone) {
    if (threadIdx.x == 0 && blockIdx.y == 0) flag(status, EP_STATUS_BAD_PAGE);
    return;
  }
  const int r = blockIdx.y / pieces, q = blockIdx.y % pieces;
  uint8_t* base = (uint8_t*)g.pool + r * g.rank_bytes;
  copy_piece(base + s * g.page_bytes, base + d * g.page_bytes, q, g.page_bytes / 16);
}

}  // namespace

int64_t kv_page_pieces(int64_t page_bytes) { return (page_bytes + kPieceBytes - 1) / kPieceBytes; }

hipError_t launch_kv_extend(const ep_kv_pages& g, const int32_t* seqs, const int32_t* add, int m,
                            const PagesWs& ws, int32_t* status, hipStream_t stream) {
  hipLaunchKernelGGL(extend_kernel, dim3(1), dim3(kPlan), 0, stream, g, seqs, add, m, ws, status);
  return hipGetLastError();
}

hipError_t launch_kv_fork(const ep_kv_pages& g, const int32_t* parents, const int32_t* children,
                          int m, const PagesWs& ws, int32_t* status, hipStream_t stream) {
  const int pieces = (int)kv_page_pieces(g.page_bytes);
  hipLaunchKernelGGL(fork_plan_kernel, dim3(1), dim3(kPlan), 0, stream, g, parents, children, m,
                     ws, status);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fork_apply_kernel, dim3(m, 1 + g.ranks * pieces), dim3(kWave), 0, stream, g,
                     parents, children, ws, pieces, status);
  return hipGetLastError();
}

hipError_t launch_kv_free(const ep_kv_pages& g, const int32_t* seqs, int m, int32_t* status,
                          hipStream_t stream) {
  hipLaunchKernelGGL(free_kernel, dim3(m), dim3(kBlock), 0, stream, g, seqs, status);
  return hipGetLastError();
}

hipError_t launch_kv_compact(const ep_kv_pages& g, int32_t* n_live, const PagesWs& ws,
                             int32_t* status, hipStream_t stream) {
  const int chunks = (g.n_pages + kCompact - 1) / kCompact;
  const int pieces = (int)kv_page_pieces(g.page_bytes);
  hipError_t e = hipSuccess;
  if (chunks > kCompactAlone) {
    hipLaunchKernelGGL(compact_count_kernel, dim3(chunks), dim3(kBlock), 0, stream, g, ws);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(compact_rank_kernel, dim3(chunks), dim3(kBlock), 0, stream, g, ws, chunks,
                     n_live);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int row_blocks = g.n_seqs < 256 ? g.n_seqs : 256;
  // How many pages move is known on the device only: enough waves to fill the
  // chip several times over, and no more than the moves there can be.
  const int64_t most = ((int64_t)g.n_pages + 1) / 2 * g.ranks * pieces;
  const int waves = (int)(most < 16384 ? most : 16384);
  hipLaunchKernelGGL(compact_apply_kernel, dim3(row_blocks + (waves > 0 ? waves : 1)), dim3(kWave),
                     0, stream, g, ws, chunks, row_blocks, pieces, status);
  return hipGetLastError();
}

hipError_t launch_kv_copy_pages(const ep_kv_pages& g, const int32_t* src, const int32_t* dst,
                                int m, const PagesWs& ws, int32_t* status, hipStream_t stream) {
  const int pieces = (int)kv_page_pieces(g.page_bytes);
  const dim3 flat((m + kBlock - 1) / kBlock);
  hipLaunchKernelGGL(copy_clear_kernel, flat, dim3(kBlock), 0, stream, g, src, dst, m, ws);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(copy_own_kernel, flat, dim3(kBlock), 0, stream, g, src, dst, m, ws);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(copy_pages_kernel, dim3(m, g.ranks * pieces), dim3(kWave), 0, stream, g, src,
                     dst, ws, pieces, status);
  return hipGetLastError();
}

}  // namespace ep
