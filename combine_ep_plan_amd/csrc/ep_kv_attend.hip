// Attention of new tokens over the pages of a cache, leading pages that
// sequences share being read once for all of them.
//
// With s_i = scale q.k_i over the keys a row sees, m = max s_i and
// l = sum exp(s_i - m): out = sum exp(s_i - m) v_i / l, lse = m + log l.
// Both sums are associative once rescaled to a common m, so the keys of a
// row may be cut anywhere: pieces keep (m, l, sum) in 32 bits and a second
// launch joins them.
//
// Units. A prefix unit is a group: all its rows (new tokens x the query heads
// of one KV head) over the shared keys. A suffix unit is a sequence: its rows
// over the keys behind them. Units are cut into items of at most kRows rows
// and one KV head, items into tiles of kTile keys.
//
// Work. The tiles of all items stand in two lines, prefix and suffix items,
// weighted by what they cost. Each of the 8 XCDs takes an equal length of
// both, so that row tiles that read the same keys meet in one L2 and every XCD
// has as much arithmetic (prefix) as reading (suffix) to do; its workgroups
// take equal lengths of what it has, whatever the lengths of the sequences. No
// list of work is kept: every workgroup sums the units itself. A workgroup's
// part of an item is a piece; workgroup w's piece of item i has number w + i,
// which no other piece of the line has, since both only grow along it.
//
// Matrix products. Scores are formed transposed, S^T = K Q^T, with 32x32x16
// products: a lane then holds 16 keys of one row, so that maximum, sum and
// rescale need no more than one exchange between lanes l and l + 32, and the
// probabilities are already laid out as the second operand of
// O^T += V^T P^T. The k order of that product is a free choice as long as
// both sides take it: slot (half h, j) of its step s is key 16 s + 8 (j / 4)
// + 4 h + j % 4, the order the scores come out in. V is read from LDS through
// the transposing read, four keys of one column per lane.
//
// What bounds it (bf16, heads of 128):
// - Many rows over shared pages (12 sequences of up to 256 new tokens, 40
//   heads over 8, 8192 shared keys; 232 GFLOP): 323 us with the join, 0.72
//   PFLOP/s, where a large matrix product reaches 1.35 to 1.6. The matrix
//   units are busy 36 % of the time and the other vector arithmetic 46 %: two
//   waves on a SIMD cover each other only in part. The exponentials, the reads
//   of LDS and the copies to it each account for 5, 5 and 15 % when left out.
// - Many rows over their own keys: a row tile takes all keys of its sequence,
//   those that are hidden from all its rows as well, which is twice the needed
//   operations for a prompt with nothing before it (4096 tokens, 172 GFLOP
//   visible: 474 us).
// - Few rows over a prefix (128 samples of a prompt of 16,384 tokens, 512 keys
//   of their own on average; 339 MB): 124 us with the join, 2.7 TB/s of the 5.7
//   that a copy reaches, the prefix's arithmetic and the waits of short
//   sequences beside each other.
// - Few rows over their own keys (32 to 128 sequences, 4096 to 32,768 keys, 40
//   heads over 8): 4.4 to 5.4 TB/s, 3.4 to 4.7 over one-byte caches.
// - One token over 300 keys: 18.6 us, two launches and some ten dependent
//   loads.
#include <type_traits>

#include "ep_kernels.hpp"
#include "ep_kv_device.hpp"

namespace ep {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint8_t __attribute__((address_space(3))) lds_u8;

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / kWave;
constexpr int kTile = 128;       // keys of a tile
constexpr int kNone = 0x7fffffff;
constexpr int kMostKeys = 0x7fffffff - 1024;
// Rows of an item whose keys the waves share out. With few rows that ends an
// item sooner (4 rows of 64 over one-byte keys in pages of one token: 40 us, 52
// with the rows shared out and three waves idle; 4 rows of 128 over one-byte
// keys: 73 and 81; 5 rows over 16 bits: 113 both). Items of 32 rows would read
// the keys of 33 to 96 rows two or three times: 214 against 120 us for 48 rows,
// 322 against 128 for 96.
constexpr int kRowsSplit = 32;
constexpr int kRowsBlock = 128;  // rows of an item whose rows the waves share out
constexpr int kGroupTable = 64;  // groups whose ranges are kept in LDS
// Costs in the line: of a tile of either kind, and of starting on an item. A
// split tile at half of a block's tile costs short batches 5 to 11 % (25.4
// against 22.9 us for one rank's decode, 34.6 and 31.7 for drafts) and others
// nothing; at one and a half times it drafts 11 %, others 2 to 5 %. An item's
// start at half a tile leaves prompts uneven (500 and 361 us), at four tiles it
// costs 128 samples 5 % (143 and 135).
constexpr int kCostSplit = 4;
constexpr int kCostBlock = 4;
constexpr int kCostItem = 8;

// A unit as the line of work has it.
struct Unit {
  int64_t start;  // in the lines, the suffix line behind the prefix line
  int item;       // first item, among those of its kind
  int row0, rows; // first new token, rows per KV head
  int lo, hi;     // keys
  int seq;        // whose row of the table holds the keys
  int group;      // of a sequence; -1: none
  int len, fresh; // of a sequence: tokens, new ones among them

  __device__ __forceinline__ bool split() const { return rows <= kRowsSplit; }
  __device__ __forceinline__ int tile_rows() const { return split() ? kRowsSplit : kRowsBlock; }
  __device__ __forceinline__ int items() const { return (rows + tile_rows() - 1) / tile_rows(); }
  __device__ __forceinline__ int tiles() const {  // of an item
    return rows > 0 ? (int)(((int64_t)hi - lo + kTile - 1) / kTile) : 0;
  }
  __device__ __forceinline__ int cost() const { return split() ? kCostSplit : kCostBlock; }
  __device__ __forceinline__ int64_t item_length() const {
    const int64_t n = tiles();
    return n > 0 ? kCostItem + n * cost() : 0;
  }
};

struct Attend {
  ep_kv_cache c;
  ep_kv_batch b;
  ep_kv_groups g;
  ep_rows q, out;
  float* lse;
  float scale;
  int heads, share, max_new;  // share: query heads per KV head
  int workers;
  uint32_t page_magic, page_shift;  // t / page_tokens = mulhi(t, magic) >> shift
  // Workspace: the units, with the lengths of the lines behind the last as the
  // starts of two more; per item the workgroups that hold its first and last
  // tile (the last as its complement where the item was written whole); and
  // the pieces' sums and (m, l) by number and row.
  Unit* units;
  int2* span[2];
  float* sum[2];      // [0]: prefix pieces, [1]: suffix pieces
  float2* stat[2];
  int pieces[2], rows[2];  // pieces that fit, rows of each
  int32_t* status;
};

constexpr int kXcds = 8;

// The arguments in the kernel's argument segment: read where they are used.
// As values they would all be loaded at the start and spilled.
typedef const Attend __attribute__((address_space(4))) Args;

__device__ __forceinline__ Args& fresh(Args& a) {
  Args* p = &a;
  asm volatile("" : "+s"(p));
  return *p;
}

struct Shared {
  Unit unit[kBlock];         // of a round
  int64_t part[kWaves];
  int32_t ipart[kWaves], spart[kWaves];
  int32_t group_off[kGroupTable + 1], shared[kGroupTable];
  uint64_t refused;          // bit j: of the first kGroupTable groups
  int32_t any_short, special, first;
  int64_t prefix;  // length of the prefix line
  float stat[2][kWaves][32];
};

// ---------------------------------------------------------------------------
// Units
// ---------------------------------------------------------------------------
__device__ __forceinline__ int clamp_int(int64_t v, int64_t lo, int64_t hi) {
  return (int)(v < lo ? lo : v > hi ? hi : v);
}

// Keys that a row of the table holds; positions stay under 2^31 with room for
// two steps.
template <typename A>
__device__ __forceinline__ int key_cap(const A& a) {
  const int64_t cap = (int64_t)a.b.max_pages * a.c.page_tokens;
  return cap < kMostKeys ? (int)cap : kMostKeys;
}

// Whether number n has a place among `places`. Offsets that contradict each
// other name more items than a batch can have, and may wrap their numbers.
__device__ __forceinline__ bool fits(int64_t n, int places) { return n >= 0 && n < places; }

// A 64-bit value that is equal on all lanes, in scalar registers.
__device__ __forceinline__ int64_t wave_uniform64(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)wave_uniform((int)(uint32_t)v) |
                   (uint64_t)(uint32_t)wave_uniform((int)(v >> 32)) << 32);
}

__device__ __forceinline__ Unit uniform_unit(const Unit& u) {
  Unit t;
  t.start = wave_uniform64(u.start);
  t.item = wave_uniform(u.item);
  t.row0 = wave_uniform(u.row0);
  t.rows = wave_uniform(u.rows);
  t.lo = wave_uniform(u.lo);
  t.hi = wave_uniform(u.hi);
  t.seq = wave_uniform(u.seq);
  t.group = wave_uniform(u.group);
  t.len = wave_uniform(u.len);
  t.fresh = wave_uniform(u.fresh);
  return t;
}

// New tokens between two offsets; 0 where the offsets are not those of a
// batch.
__device__ __forceinline__ int fresh_of(Args& a, int lo, int hi) {
  return lo >= 0 && hi > lo && hi <= a.b.n_tokens ? hi - lo : 0;
}

// Reads the groups' ranges into LDS where they fit; a barrier must follow.
__device__ __forceinline__ void load_groups(Args& a, Shared& sh) {
  const int j = threadIdx.x;
  if (a.g.n_groups > kGroupTable || j > a.g.n_groups || a.g.n_groups == 0) return;
  sh.group_off[j] = a.g.group_off[j];
  if (j < a.g.n_groups) sh.shared[j] = a.g.shared[j];
}

// The group of sequence s, or -1: the last one that starts at or before it.
__device__ __forceinline__ int group_of(Args& a, const int32_t* off, int s) {
  int lo = 0, hi = a.g.n_groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (off[mid] <= s) lo = mid;
    else hi = mid;
  }
  return lo < a.g.n_groups && off[lo] <= s && s < off[lo + 1] ? lo : -1;
}

// The new tokens of sequences s0 .. s1 - 1: the first, and behind the last.
// Offsets out of range are not followed.
struct Span {
  int lo, hi;
  bool in;

  __device__ __forceinline__ Span(Args& a, int s0, int s1)
      : in(s0 >= 0 && s0 <= s1 && s1 <= a.b.n_seqs) {
    lo = in ? s0 : 0;
    hi = in ? s1 : 0;
    if (a.b.q_off) {
      lo = a.b.q_off[lo];
      hi = a.b.q_off[hi];
    } else if (hi > a.b.n_tokens) {
      hi = a.b.n_tokens;
    }
  }
  // Whether the offsets name no such sequences or rows.
  __device__ __forceinline__ bool bad(Args& a) const {
    return !in || (a.b.q_off && (lo < 0 || hi < lo || hi > a.b.n_tokens));
  }
};

// Unit u but for its place; *late: the shared keys reach past the first new
// token, so that rows of the group see different ones of them; *bad: its
// offsets are not those of a batch. Such a unit has no rows. A group that has
// none for that reason shares nothing: its sequences read all their keys
// through their own rows of the table (place_units() sees to that where the
// groups are in LDS).
__device__ __forceinline__ Unit unit_of(Args& a, const Shared& sh, int u, bool* late, bool* bad) {
  const int s = u - a.g.n_groups;
  const bool kept = a.g.n_groups <= kGroupTable;
  int s0 = s, s1 = s + 1;
  if (s < 0) {
    s0 = kept ? sh.group_off[u] : a.g.group_off[u];
    s1 = kept ? sh.group_off[u + 1] : a.g.group_off[u + 1];
  }
  // On their way for both kinds of unit while the group is searched for.
  const int len = a.b.lens[s < 0 ? 0 : s];
  const Span rows(a, s0, s1);
  Unit t;
  t.start = t.item = 0;
  t.seq = s0;
  t.group = u;
  if (s >= 0) {
    t.group = kept ? group_of(a, sh.group_off, s) : group_of(a, a.g.group_off, s);
    if (!kept && t.group >= 0 &&
        Span(a, a.g.group_off[t.group], a.g.group_off[t.group + 1]).bad(a))
      t.group = -1;
  }
  const int shared = t.group < 0 ? 0 : kept ? sh.shared[t.group] : a.g.shared[t.group];
  // An empty group has nobody to share with, wherever it lies.
  *bad = s0 != s1 && rows.bad(a);
  t.row0 = rows.lo;
  const int fresh = *bad ? 0 : fresh_of(a, rows.lo, rows.hi);
  if (s < 0) {
    t.rows = fresh * a.share;
    t.lo = t.len = t.fresh = 0;
    t.hi = t.rows > 0 ? clamp_int(shared, 0, key_cap(a)) : 0;
    *late = false;
  } else {
    t.len = len;
    t.fresh = fresh;
    t.rows = (fresh < a.max_new ? fresh : a.max_new) * a.share;
    t.lo = clamp_int(shared, 0, key_cap(a));
    t.hi = clamp_int(len, t.lo, key_cap(a));
    *late = (int64_t)len - fresh + 1 < shared;
  }
  return t;
}

// Workgroup w of `workers` (a power of two) is number w % per of XCD w / per.
// An XCD's lengths of the two lines of p and s stand one behind the other and
// are cut evenly; [begin, end) is w's part of the line of that kind.
struct Range {
  int64_t begin, end;
};

template <typename A>
__device__ __forceinline__ Range range_of(const A& a, int kind, int w, int64_t p, int64_t s) {
  const int per = a.workers / kXcds, x = w / per, i = w % per;
  const int64_t p0 = p * x / kXcds, p1 = p * (x + 1) / kXcds;
  const int64_t s0 = s * x / kXcds, s1 = s * (x + 1) / kXcds;
  const int64_t np = p1 - p0, n = np + s1 - s0;
  const int64_t lo = (int64_t)((uint64_t)(n * i) / (unsigned)per);
  const int64_t hi = (int64_t)((uint64_t)(n * (i + 1)) / (unsigned)per);
  if (kind == 0) return Range{p0 + (lo < np ? lo : np), p0 + (hi < np ? hi : np)};
  return Range{p + s0 + (lo > np ? lo - np : 0), p + s0 + (hi > np ? hi - np : 0)};
}

// Tiles of an item at `at` whose points lie before x.
__device__ __forceinline__ int tiles_before(const Unit& u, int64_t at, int64_t x) {
  return clamp_int((x - at - kCostItem + u.cost() - 1) / u.cost(), 0, u.tiles());
}

// ---------------------------------------------------------------------------
// Tiles in LDS. Rows of DP elements of 16 bits in chunks of 16 bytes; chunk c
// of key t lies at chunk place_k(t, c) or place_v(t, c) of its row, so that
// the reads below spread over the banks.
// ---------------------------------------------------------------------------
// K is read by 32 lanes that hold 32 keys, chunk 2 step + half of each.
template <int DP>
__device__ __forceinline__ int place_k(int t, int c) {
  return DP == 64 ? c ^ ((t >> 1) & 7) : c ^ (t & 15);
}
// V is read as 64 bytes (4 chunks) of 4 consecutive keys per half wave.
template <int DP>
__device__ __forceinline__ int place_v(int t, int c) {
  return DP == 64 ? c ^ ((((t >> 1) & 1) << 2) | ((t >> 2) & 3))
                  : c ^ (((t & 3) << 2) | ((t >> 2) & 3));
}

// Sixteen e4m3 values as 16-bit ones (exact).
template <int QT>
__device__ __forceinline__ void widen(const u32x4& in, u32x4 out[2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(in[i], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(in[i], true);
    uint32_t w0, w1;
    if constexpr (QT == EP_DTYPE_BF16) {
      w0 = __builtin_amdgcn_perm(__float_as_uint(lo[1]), __float_as_uint(lo[0]), 0x07060302u);
      w1 = __builtin_amdgcn_perm(__float_as_uint(hi[1]), __float_as_uint(hi[0]), 0x07060302u);
    } else {
      w0 = as<uint32_t>(__builtin_amdgcn_cvt_pkrtz(lo[0], lo[1]));
      w1 = as<uint32_t>(__builtin_amdgcn_cvt_pkrtz(hi[0], hi[1]));
    }
    out[i / 2][2 * (i % 2)] = w0;
    out[i / 2][2 * (i % 2) + 1] = w1;
  }
}

// Zeroes the infinities and NaN of a chunk; returns whether there were any.
template <int QT>
__device__ __forceinline__ bool drop_special(u32x4& v) {
  constexpr uint32_t ex = QT == EP_DTYPE_BF16 ? 0x7f80u : 0x7c00u;
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w = v[i];
    if ((w & ex) == ex) {
      w &= 0xffff0000u;
      any = true;
    }
    if ((w & (ex << 16)) == ex << 16) {
      w &= 0xffffu;
      any = true;
    }
    v[i] = w;
  }
  return any;
}

// Which thread this is, opaque to the compiler at every call: what follows
// from it is formed where it is used and not kept in registers across the
// loops over items and tiles, which leave none to spare.
struct Who {
  int tid, lane, half, wave;  // half: of the wave; wave: scalar
};

__device__ __forceinline__ Who who() {
  uint32_t t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return Who{(int)t, (int)(t % kWave), (int)(t % kWave / 32), wave_uniform((int)(t / kWave))};
}

__device__ __forceinline__ int64_t from_lane(int64_t v, int lane) {
  const int at = lane * 4;
  const int lo = __builtin_amdgcn_ds_bpermute(at, (int)(uint32_t)v);
  const int hi = __builtin_amdgcn_ds_bpermute(at, (int)(v >> 32));
  return (int64_t)((uint64_t)(uint32_t)lo | (uint64_t)(uint32_t)hi << 32);
}

// Source of the chunks that hold nothing: the part of a padded row behind the
// head.
__device__ const u32x4 kZeros = {0, 0, 0, 0};

// Starts the copy of 16 bytes per lane to LDS, lane l's to `to` + 16 l. It
// counts as a vector load; nothing waits for it but settle_copies().
__device__ __forceinline__ void copy_to_lds(const uint8_t* from, const lds_u8* to) {
  const int at = wave_uniform((int)(uint32_t)(uintptr_t)to);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(at), "v"(from)
               : "memory", "m0");
}
__device__ __forceinline__ void settle_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// KEYS rows of K and V on their way from the pages to LDS, by THREADS threads
// (whole waves). 16-bit rows of up to 128 elements are copied to LDS without
// passing through registers: a copy fills 1024 bytes of LDS in order, so the
// order of the chunks is made by what each lane reads. Others go through
// registers: e4m3 rows are widened on the way. FULL: the head fills its place.
template <int DP, int QT, int CT, bool FULL, int KEYS, int THREADS>
struct Stage {
  static constexpr int cb = Fmt<CT>::bytes;
  static constexpr bool direct = cb == 2 && DP <= 128;
  static constexpr int chunks = DP * cb / 16;  // 16-byte chunks of a row in the cache
  static constexpr int step = THREADS / chunks;
  static constexpr int n = KEYS / step;
  static_assert(THREADS % chunks == 0 && KEYS % step == 0, "a pass takes whole rows");
  u32x4 k[direct ? 1 : n], v[direct ? 1 : n];
  int64_t at[n];

  // slot: this lane's key's byte offset, lane i holding key i (mod KEYS);
  // -1: none, for which the cache's first row is read. Where each row of this
  // thread's starts.
  __device__ __forceinline__ void find(int64_t slot, int tid) {
    const int64_t from = slot >= 0 ? slot : 0;
#pragma unroll
    for (int j = 0; j < n; ++j) at[j] = from_lane(from, tid / chunks % kWave + j * step);
  }

  // Row j: to LDS at lk and lv where the tiles will be, or to registers.
  __device__ __forceinline__ void copy(int j, const uint8_t* kb, const uint8_t* vb, int tid,
                                       int head_bytes, uint8_t* lk, uint8_t* lv) {
    const int c = tid % chunks;
    if constexpr (direct) {
      const int t = tid / chunks + j * step;
      const int ck = place_k<DP>(t, c) * 16, cv = place_v<DP>(t, c) * 16;
      const int base = wave_uniform(tid / kWave) * (kWave / chunks) + j * step;  // wave's first row
      const uint8_t *pk = kb + ck + at[j], *pv = vb + cv + at[j];
      if constexpr (!FULL) {  // nothing is read past a row
        if (ck >= head_bytes) pk = (const uint8_t*)&kZeros;
        if (cv >= head_bytes) pv = (const uint8_t*)&kZeros;
      }
      copy_to_lds(pk, (const lds_u8*)lk + base * DP * 2);
      copy_to_lds(pv, (const lds_u8*)lv + base * DP * 2);
    } else {
      const int64_t off = at[j] + (c * 16 < head_bytes ? c * 16 : 0);
      k[j] = *(const u32x4*)(kb + off);
      v[j] = *(const u32x4*)(vb + off);
    }
  }

  __device__ __forceinline__ void load(const uint8_t* kb, const uint8_t* vb, int64_t slot, int tid,
                                       int head_bytes, uint8_t* lk, uint8_t* lv) {
    find(slot, tid);
#pragma unroll
    for (int j = 0; j < n; ++j) copy(j, kb, vb, tid, head_bytes, lk, lv);
  }

  // Finishes the tiles. CHECK: rows of V without a slot are zeroed in LDS, and
  // infinities and NaN of the others; returns the lowest key (of this
  // thread's) that holds one, else kNone. What K holds in rows without a slot
  // does not matter: the scores are replaced.
  template <bool CHECK>
  __device__ __forceinline__ int store(uint8_t* lk, uint8_t* lv, uint64_t valid, int tid,
                                       int head_bytes) const {
    const int c = tid % chunks;
    int special = kNone;
    if constexpr (direct) {
      if constexpr (CHECK) {
#pragma unroll
        for (int j = 0; j < n; ++j) {
          const int t = tid / chunks + j * step;
          u32x4* at = (u32x4*)(lv + t * DP * 2 + c * 16);
          u32x4 x = *at;
          if (!((valid >> t) & 1)) {
            *at = u32x4{0, 0, 0, 0};
          } else if (drop_special<QT>(x)) {
            *at = x;
            if (t < special) special = t;
          }
        }
      }
      return special;
    }
    const int whole = c * 16 < head_bytes ? -1 : 0;
#pragma unroll
    for (int j = 0; j < (direct ? 0 : n); ++j) {
      const int t = tid / chunks + j * step;
      const uint32_t keep = (uint32_t)(whole & -(int)((valid >> t) & 1));
      const u32x4 x = k[j] & keep, y = v[j] & keep;
      if constexpr (CT == EP_DTYPE_E4M3) {
        u32x4 wx[2], wy[2];
        widen<QT>(x, wx);
        widen<QT>(y, wy);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (CHECK && drop_special<QT>(wy[i]) && t < special) special = t;
          *(u32x4*)(lk + t * DP * 2 + place_k<DP>(t, 2 * c + i) * 16) = wx[i];
          *(u32x4*)(lv + t * DP * 2 + place_v<DP>(t, 2 * c + i) * 16) = wy[i];
        }
      } else {
        u32x4 z = y;
        if (CHECK && drop_special<QT>(z) && t < special) special = t;
        *(u32x4*)(lk + t * DP * 2 + place_k<DP>(t, c) * 16) = x;
        *(u32x4*)(lv + t * DP * 2 + place_v<DP>(t, c) * 16) = z;
      }
    }
    return special;
  }
};

template <int QT>
__device__ __forceinline__ f32x16 product(const s16x8& x, const s16x8& y, const f32x16& z) {
  if constexpr (QT == EP_DTYPE_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(as<bf16x8>(x), as<bf16x8>(y), z, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(as<f16x8>(x), as<f16x8>(y), z, 0, 0, 0);
}

// What a wave keeps of 32 rows: lane l holds row l % 32; register r of block
// dt of `o` is element 32 dt + 8 (r / 4) + 4 (l / 32) + r % 4 of it.
template <int DP>
struct Rows32 {
  s16x8 q[DP / 16];
  f32x16 o[DP / 32];
  float m, l;      // of scores as the product gives them; l of this lane's keys
  int limit;       // keys below it are seen
  int row;         // in the unit; -1: none

  __device__ __forceinline__ void clear() {
    m = -__builtin_inff();
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < DP / 32; ++i) o[i] = f32x16{};
  }
};

// Lanes l and l + 32 both get a function of their two values.
__device__ __forceinline__ float max_halves(float v) {
  const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
}
__device__ __forceinline__ float add_halves(float v) {
  const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(x[0]) + __uint_as_float(x[1]);
}

// Key of register i, among 32.
__device__ __forceinline__ int key_of(int i, int half) { return 8 * (i / 4) + 4 * half + i % 4; }

// Where a lane reads the tiles: the first chunk of its row of K, and its part
// of the first four keys of V. The chunks of the other steps are an exclusive
// or away, since place_k and place_v are one of the chunk's number.
template <int DP>
struct Reads {
  uint32_t k, v;

  __device__ __forceinline__ Reads(const uint8_t* lk, const uint8_t* lv) {
    const Who me = who();
    const int lane = me.lane, half = me.half, col = lane % 32, i16 = lane % 16;
    const int t = 4 * half + i16 / 4, chunk = lane / 16 % 2 * 2 + i16 % 4 / 2;
    k = (uint32_t)(uintptr_t)(const lds_u8*)lk + col * DP * 2 + place_k<DP>(col, half) * 16;
    v = (uint32_t)(uintptr_t)(const lds_u8*)lv + t * DP * 2 + place_v<DP>(t, chunk) * 16 +
        i16 % 2 * 8;
  }
};

template <typename V>
__device__ __forceinline__ V read_lds(uint32_t at) {
  typedef V __attribute__((address_space(3))) lds_v;
  return *(lds_v*)at;
}

// m need not be the maximum of a row's scores, only near it: it follows when
// they pass it by 2^kSlack, which keeps every weight under 2^kSlack and spares
// the rescale of the sums most of the time (with the maximum itself, some row
// of 32 has a new one in almost every step).
constexpr float kSlack = 8.0f;
// Weights and sums are 2^kRaise times what m alone would make them. In fp16 a
// weight under 2^-14 loses bits and one under 2^-25 is lost, and a thousand
// such keys beside one of large weight and small V are the row's output. The
// type holds 2^15, so 7 powers of two are free above those of the slack.
template <int QT>
constexpr float kRaise = QT == EP_DTYPE_F16 ? 7.0f : 0.0f;

// What the exponents of a row's weights are taken off; nothing seen yet: any
// finite value.
template <int QT>
__device__ __forceinline__ float base_of(float m, float c) {
  return m == -__builtin_inff() ? 0.0f : m * c - kRaise<QT>;
}

// NS * 32 keys in LDS, `at` bytes behind the tiles of `rd`. c > 0: the factor
// of the scores in powers of two. masked: some row does not see some of the
// keys; bit t of `see` says whether this lane's row sees key t.
// between(m) stands behind product m of the scores, m < kScoreProducts.
template <int DP, int NS>
constexpr int kScoreProducts = NS * DP / 16;

template <int DP, int QT, int NS, typename F>
__device__ __forceinline__ void step(Rows32<DP>& r, Reads<DP> rd, int at, float c, bool masked,
                                     uint64_t see, F&& between) {
  rd.k += at;
  rd.v += at;
  // Opaque, so that the few addresses are formed here and not kept.
  asm volatile("" : "+v"(rd.k), "+v"(rd.v));
  f32x16 s[NS];
#pragma unroll
  for (int n = 0; n < NS; ++n) s[n] = f32x16{};
  // kAhead chunks stay on their way from LDS: read one at a time, each
  // product would wait for its own.
  constexpr int kReads = kScoreProducts<DP, NS>, kAhead = 4;
  const auto k_at = [&](int m) {
    return read_lds<s16x8>((rd.k ^ (m / NS << 5)) + 32 * (m % NS) * DP * 2);
  };
  s16x8 kf[kAhead];
#pragma unroll
  for (int m = 0; m < kAhead; ++m) kf[m] = k_at(m);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int m = 0; m < kReads; ++m) {
    s[m % NS] = product<QT>(kf[m % kAhead], r.q[m / NS], s[m % NS]);
    if (m + kAhead < kReads) kf[m % kAhead] = k_at(m + kAhead);
    between(m);
    __builtin_amdgcn_sched_barrier(0);
  }
  // Product m is of 16 keys (m / (DP / 32)) and 32 elements (m % (DP / 32));
  // V for the next ones is on its way, and between the products of one 16
  // keys stands the arithmetic of the next's weights.
  constexpr int kCols = DP / 32, kProducts = NS * 2 * kCols;
  const auto v_at = [&](int m) {
    typedef s16x4 __attribute__((address_space(3))) lds_s16x4;
    const int d = m % kCols, key = m / kCols * 16 * DP * 2;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s16x4*)((rd.v ^ (d << 6)) + key));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s16x4*)((rd.v ^ (d << 6) ^ 32) + key + 8 * DP * 2));
    s16x8 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = lo[j];
      v[4 + j] = hi[j];
    }
    return v;
  };
  s16x8 vf[kAhead];
#pragma unroll
  for (int m = 0; m < kAhead; ++m) vf[m] = v_at(m);
  __builtin_amdgcn_sched_barrier(0);
  if (masked) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      const int bits = (int)(uint32_t)(see >> (32 * n + 4 * who().half));
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t keep = (uint32_t)(bits << (31 - (8 * (i / 4) + i % 4)) >> 31);
        s[n][i] = __uint_as_float((__float_as_uint(s[n][i]) & keep) | (~keep & 0xff800000u));
      }
    }
  }
  float top = s[0][0];
#pragma unroll
  for (int n = 0; n < NS; ++n)
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, s[n][i]);
  top = max_halves(top);
  if (ballot((top - r.m) * c > kSlack)) {
    const float m = fmaxf(r.m, top);
    // exp2(-inf) = 0 where nothing was seen before; rows that still see
    // nothing keep their zeros.
    const float w = m == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f((r.m - m) * c);
    r.l *= w;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) r.o[d][i] *= w;
    r.m = m;
  }
  const float base = base_of<QT>(r.m, c);
  float sum = 0.0f;
  // The weights meet V in the rows' 16-bit type: half a step of it, relative,
  // per weight; the sum of weights is taken before. kRaise keeps small fp16
  // weights from it for longer.
  typename Fmt<QT>::vec8 w[2];
  const auto weights = [&](int g, int j0, int j1) {
#pragma unroll
    for (int j = j0; j < j1; ++j) {
      const float e =
          __builtin_amdgcn_exp2f(__builtin_fmaf(s[g / 2][8 * (g % 2) + j], c, -base));
      sum += e;
      w[g % 2][j] = (typename Fmt<QT>::elem)e;
    }
  };
  weights(0, 0, 8);
#pragma unroll
  for (int m = 0; m < kProducts; ++m) {
    const int g = m / kCols, d = m % kCols;
    r.o[d] = product<QT>(vf[m % kAhead], as<s16x8>(w[g % 2]), r.o[d]);
    if (m + kAhead < kProducts) vf[m % kAhead] = v_at(m + kAhead);
    if (g + 1 < 2 * NS) weights(g + 1, d * 8 / kCols, (d + 1) * 8 / kCols);
    __builtin_amdgcn_sched_barrier(0);
  }
  r.l += sum;
}

// Bits of the keys t0 .. t0 + 63 below `limit`.
__device__ __forceinline__ uint64_t below(int limit, int t0) {
  const int n = limit - t0;
  return n >= 64 ? ~0ull : n <= 0 ? 0 : (1ull << n) - 1;
}

// Bytes of LDS that the tiles take: a workgroup's two halves, or the waves'
// own tiles.
template <int DP>
struct Lds {
  static constexpr int keys = DP <= 128 ? 64 : 32;     // keys of a block step
  static constexpr int half = keys * DP * 2;           // K or V of one
  static constexpr int block = 2 * half * 2;           // two steps
  static constexpr int wave = 2 * 32 * DP * 2;         // K and V of 32 keys
  static constexpr int box = 32 * DP * 4;              // rows on their way out, of a wave
  static constexpr int most = block > kWaves * wave ? block : kWaves * wave;
  static constexpr int bytes = most > kWaves * box ? most : kWaves * box;
};

template <int DP, int QT, int CT, bool FULL>
struct Body {
  Args& a;
  Shared& sh;
  uint8_t* lds;
  Unit u;
  bool prefix;
  int kvh, index, lo_tile, hi_tile;  // index: of the item in its KV head
  const uint8_t *kb, *vb;
  float c;  // factor of the scores, in powers of two; positive
  bool negate;
  int head_bytes;

  // A key's slot is found in two halves, so that the table's entry is on its
  // way while other work is done.
  struct Lookup {
    int32_t page;
    uint32_t in;  // slot within the page; kNone: no key
  };

  __device__ __forceinline__ Lookup look_up(int t) const {
    // Keys past the end read the last one's entry: no branch around the load.
    const int last = t < u.hi ? t : u.hi - 1;
    const uint32_t page = a.page_magic ? __umulhi((uint32_t)last, a.page_magic) >> a.page_shift
                                       : (uint32_t)last;
    const uint32_t in = (uint32_t)last - page * (uint32_t)a.c.page_tokens;
    return Lookup{(a.b.tables + (int64_t)u.seq * a.b.max_pages)[page],
                  t < u.hi ? in : (uint32_t)kNone};
  }

  // Byte offset of the slot, or -1.
  __device__ __forceinline__ int64_t slot_of(const Lookup& l, bool* bad) const {
    const bool in = (uint32_t)l.page < (uint32_t)a.c.n_pages;
    *bad |= !in && l.in != (uint32_t)kNone;
    return in && l.in != (uint32_t)kNone
               ? l.page * a.c.page_stride + (int64_t)l.in * a.c.token_stride : -1;
  }

  __device__ __forceinline__ int token_of(int row) const { return u.row0 + row / a.share; }
  __device__ __forceinline__ int head_of(int row) const {
    return kvh * a.share + row % a.share;
  }

  // The head size, opaque to the compiler: comparisons with it are not worth
  // keeping in registers across the tiles.
  __device__ __forceinline__ int dim() const {
    int d = a.c.head_dim;
    asm volatile("" : "+s"(d));
    return d;
  }

  // Keys below it are seen by a row of the unit.
  __device__ __forceinline__ int limit_of(int row) const {
    const int token = token_of(row);
    if (!prefix) return clamp_int((int64_t)u.len - u.fresh + (token - u.row0) + 1, 0, u.hi);
    if (!sh.any_short) return u.hi;
    int lo = u.seq, hi = a.g.group_off[u.group + 1];
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if ((a.b.q_off ? a.b.q_off[mid] : mid) <= token) lo = mid;
      else hi = mid;
    }
    const int last = a.b.q_off ? a.b.q_off[lo + 1] : lo + 1;
    return clamp_int((int64_t)a.b.lens[lo] - (last - token) + 1, 0, u.hi);
  }

  __device__ __forceinline__ void load_rows(Rows32<DP>& r, int row0) const {
    Args& a = fresh(this->a);
    const Who me = who();
    const int half = me.half, row = row0 + me.lane % 32;
    r.clear();
    r.row = row < u.rows ? row : -1;
    const int have = row < u.rows ? row : u.rows - 1;
    const int token = token_of(have);
    // Rows past the unit's end see what the unit holds, so that they ask
    // for no masking.
    r.limit = row < u.rows ? limit_of(row) : u.hi;
    const uint8_t* p = (const uint8_t*)a.q.p + (int64_t)token * a.q.token_stride +
                       (int64_t)head_of(have) * a.q.head_stride;
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      const int d = 16 * i + 8 * half;
      u32x4 w = {0, 0, 0, 0};
      if (d < dim()) w = *(const u32x4*)(p + 2 * d);
      if (negate) w ^= u32x4{0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u};
      r.q[i] = as<s16x8>(w);
    }
  }

  // The fewest keys that a row of the wave sees.
  __device__ __forceinline__ int least_limit(const Rows32<DP>& r) const {
    int v = r.limit;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_xor(v, d);
      v = o < v ? o : v;
    }
    return wave_uniform(v);
  }

  // Infinities and NaN of V at keys that some rows may not see went to LDS as
  // zeros, since 0 * inf would reach those rows. Here the rows of the piece
  // that see such a key get them, after put() by the whole workgroup: a
  // positive weight changes neither. Keys [t0, end).
  __device__ __forceinline__ void add_special(int64_t number, bool whole, int t0, int end) const {
    Args& a = fresh(this->a);
    __syncthreads();
    const int kind = prefix ? 0 : 1, rows = u.tile_rows();
    if (!whole && !fits(number, a.pieces[kind])) return;
    for (int t = t0; t < end; ++t) {
      bool bad = false;
      const int64_t at = slot_of(look_up(t), &bad);
      if (at < 0) continue;
#pragma unroll 1
      for (int i = threadIdx.x; i < rows * DP; i += kBlock) {
        const int in = i / DP, e = i % DP, row = index * rows + in;
        if (e >= a.c.head_dim || row >= u.rows || t >= limit_of(row)) continue;
        const float x = load1<CT>(vb + at + e * Fmt<CT>::bytes);
        if (fabsf(x) < __builtin_inff()) continue;
        if (whole) {
          uint8_t* to = (uint8_t*)a.out.p + (int64_t)token_of(row) * a.out.token_stride +
                        (int64_t)head_of(row) * a.out.head_stride + 2 * e;
          store1<QT>(to, load1<QT>(to) + x);
        } else {
          float* to = a.sum[kind] + (number * a.rows[kind] + in) * DP + e;
          *to += x;
        }
      }
    }
  }

  // Chunk q (of four floats) of row i of 32 in LDS: moved so that lanes that
  // hold 32 rows and lanes that read whole ones both spread over the banks.
  static constexpr int kChunks = DP / 4;
  __device__ __forceinline__ static int chunk_at(int i, int q) {
    return i * kChunks + (q ^ (i % kChunks));
  }

  // The wave's rows, times f, to LDS.
  __device__ __forceinline__ static void lay_out(const Rows32<DP>& r, f32x4* to, float f) {
    const Who me = who();
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        to[chunk_at(me.lane % 32, 8 * d + 2 * i + me.half)] =
            f32x4{r.o[d][4 * i], r.o[d][4 * i + 1], r.o[d][4 * i + 2], r.o[d][4 * i + 3]} * f;
  }

  // Four elements from e of a row of the unit, to the output or the piece.
  __device__ __forceinline__ void put4(Args& a, int64_t number, bool whole, int row, int e,
                                       const f32x4& x) const {
    const int kind = prefix ? 0 : 1;
    if (!whole) {
      *(f32x4*)(a.sum[kind] + (number * a.rows[kind] + row % u.tile_rows()) * DP + e) = x;
    } else if (e < a.c.head_dim) {
      uint8_t* to = (uint8_t*)a.out.p + (int64_t)token_of(row) * a.out.token_stride +
                    (int64_t)head_of(row) * a.out.head_stride + 2 * e;
      typename Fmt<QT>::elem w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = (typename Fmt<QT>::elem)x[j];
      *(u32x2*)to = u32x2{as<uint16_t>(w[0]) | (uint32_t)as<uint16_t>(w[1]) << 16,
                          as<uint16_t>(w[2]) | (uint32_t)as<uint16_t>(w[3]) << 16};
    }
  }

  // The statistics of a row; m of scores as the product gives them.
  __device__ __forceinline__ void put_stat(Args& a, int64_t number, bool whole, int row, float m,
                                           float l) const {
    const int kind = prefix ? 0 : 1;
    // Scores that are all NaN leave no maximum but a sum: the join has to
    // see it.
    const float n = m == -__builtin_inff() && l == 0.0f ? m : base_of<QT>(m, c);
    if (!whole)
      a.stat[kind][number * a.rows[kind] + row % u.tile_rows()] = make_float2(n, l);
    else if (a.lse)
      a.lse[(int64_t)token_of(row) * a.heads + head_of(row)] =
          l == 0.0f ? -__builtin_inff() : (n + log2f(l)) * 0.69314718055994531f;
  }

  // What the sums of a row are multiplied by where they are the output.
  __device__ __forceinline__ float final_factor(Args& a, float l) const {
    return l == 0.0f ? 0.0f : (CT == EP_DTYPE_E4M3 ? a.c.v_scale[kvh] : 1.0f) / l;
  }

  // Whether a piece of this number has a place (it has, but where the
  // batch's offsets contradict each other).
  __device__ __forceinline__ bool has_place(Args& a, int64_t number, bool whole) const {
    if (whole || fits(number, a.pieces[prefix ? 0 : 1])) return true;
    if (threadIdx.x % kWave == 0) atomicOr(a.status, EP_STATUS_BAD_PAGE);
    return false;
  }

  // A wave's rows to their place: the output where this piece is all there is,
  // else the piece's sums. A lane holds parts of one row; they pass through
  // `box` in LDS, so that whole rows are written at a time.
  __device__ __forceinline__ void put(Rows32<DP>& r, int64_t number, bool whole,
                                      uint8_t* box) const {
    Args& a = fresh(this->a);
    if (!has_place(a, number, whole)) return;
    const Who me = who();
    const int lane = me.lane;
    lay_out(r, (f32x4*)box, whole ? final_factor(a, r.l) : 1.0f);
    const int first = wave_uniform(r.row);  // row of lane 0: always there
    if (r.row >= 0 && me.half == 0) put_stat(a, number, whole, r.row, r.m, r.l);
#pragma unroll 4
    for (int k = 0; k < 32 * kChunks / kWave; ++k) {
      const int i = k * (kWave / kChunks) + lane / kChunks, q = lane % kChunks, row = first + i;
      const f32x4 x = ((const f32x4*)box)[chunk_at(i, q)];
      if (row < u.rows) put4(a, number, whole, row, 4 * q, x);
    }
  }

  // The rows whose keys the waves shared out, from what each left in LDS: the
  // common maximum, then the sums weighted to it.
  __device__ __forceinline__ void put_split(int64_t number, bool whole) const {
    Args& a = fresh(this->a);
    if (!has_place(a, number, whole)) return;
    const Who me = who();
    const int row0 = index * kRowsSplit;
    const int n = u.rows - row0 < kRowsSplit ? u.rows - row0 : kRowsSplit;
    for (int j = me.tid; j < n * kChunks; j += kBlock) {
      const int i = j / kChunks, q = j % kChunks;
      float m[kWaves], top = -__builtin_inff(), l = 0.0f;
      f32x4 x[kWaves], sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        m[w] = sh.stat[0][w][i];
        x[w] = ((const f32x4*)(lds + w * Lds<DP>::box))[chunk_at(i, q)];
        top = fmaxf(top, m[w]);
      }
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = m[w] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f((m[w] - top) * c);
        l += sh.stat[1][w][i] * f;
        sum += x[w] * f;
      }
      put4(a, number, whole, row0 + i, 4 * q, whole ? sum * final_factor(a, l) : sum);
      if (q == 0) put_stat(a, number, whole, row0 + i, top, l);
    }
  }

  // Waves share out the rows: 32 each, all keys.
  __device__ __forceinline__ void block_rows(int64_t number, bool whole) {
    const Who me = who();
    const int tid = me.tid, wave = me.wave, lane = me.lane;
    constexpr int keys = Lds<DP>::keys;
    constexpr uint64_t all = keys == 64 ? ~0ull : (1ull << keys) - 1;
    Stage<DP, QT, CT, FULL, keys, kBlock> st;
    Rows32<DP> r;
    bool bad = false;
    int t0 = u.lo + lo_tile * kTile;
    const int end = hi_tile < u.tiles() ? u.lo + hi_tile * kTile : u.hi;
    int64_t slot = slot_of(look_up(t0 + lane % keys), &bad);
    Lookup next = look_up(t0 + keys + lane % keys);
    st.load(kb, vb, slot, tid, head_bytes, lds, lds + Lds<DP>::half);
    load_rows(r, index * kRowsBlock + wave * 32);
    const int least = least_limit(r);
    // The block's least: keys from there on may be hidden from some row.
    if (lane == 0) sh.ipart[wave] = least;
    __syncthreads();
    int fewest = sh.ipart[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) fewest = sh.ipart[w] < fewest ? sh.ipart[w] : fewest;
    fewest = wave_uniform(fewest);
    const Reads<DP> rd(lds, lds + Lds<DP>::half);
    const bool busy = index * kRowsBlock + wave * 32 < u.rows;
    // A step's tiles are complete once every wave has seen its own copies
    // land and met the others; they may be overwritten when all have met
    // again, in the next step.
    constexpr int kStep = 2 * Lds<DP>::half;
    for (int buf = 0; t0 < end; t0 += keys, buf ^= kStep) {
      uint8_t* lk = lds + buf;
      uint8_t* lv = lk + Lds<DP>::half;
      const uint64_t valid = ballot(slot >= 0) & all;
      const bool edge = t0 + keys > fewest || valid != all;
      if constexpr (decltype(st)::direct) settle_copies();
      int special = kNone;
      if (edge) special = st.template store<true>(lk, lv, valid, tid, head_bytes);
      else st.template store<false>(lk, lv, valid, tid, head_bytes);
      if (special != kNone) atomicMin(&sh.special, t0 + special);
      __syncthreads();
      // The next step's copies are started one by one between the products
      // of the scores: all at once they would hold the wave up, as the
      // vector memory unit takes 64 bytes of a copy per cycle and CU.
      const bool more = t0 + keys < end;
      const bool masked = t0 + keys > least || valid != all;
      const uint64_t see = valid & below(r.limit, t0);
      uint8_t* to = lds + (buf ^ kStep);
      const auto fetch = [&](int m, int of) {
        if (!more) return;
        if (m == 0) {
          slot = slot_of(next, &bad);
          st.find(slot, tid);
        }
        constexpr int n = decltype(st)::n;
        // Copies spread over the products behind the first few.
        const int from = of > n + 3 ? 3 : 0, gap = (of - from) / n > 0 ? (of - from) / n : 1;
#pragma unroll
        for (int j = 0; j < n; ++j)
          if (m == (from + j * gap < of ? from + j * gap : of - 1))
            st.copy(j, kb, vb, tid, head_bytes, to, to + Lds<DP>::half);
        if (m == of - 1) next = look_up(t0 + 2 * keys + lane % keys);
      };
      if (busy) {
        step<DP, QT, keys / 32>(r, rd, buf, c, masked, see, [&](int m) {
          fetch(m, kScoreProducts<DP, keys / 32>);
        });
      } else {
        fetch(0, 1);
      }
    }
    if (bad) atomicOr(a.status, EP_STATUS_BAD_PAGE);
    r.l = add_halves(r.l);
    __syncthreads();  // no wave reads tiles any more
    if (busy) put(r, number, whole, lds + wave * 32 * DP * 4);
    const int special = wave_uniform(sh.special);
    if (special < end) add_special(number, whole, special, end);
    __syncthreads();  // LDS is free for the next item
    if (special != kNone) {
      if (tid == 0) sh.special = kNone;
      __syncthreads();
    }
  }

  // Waves share out the keys: 32 of every 128 each, the same rows; their
  // sums are joined at the end.
  __device__ __forceinline__ void split_keys(int64_t number, bool whole) {
    const Who me = who();
    const int tid = me.tid, wave = me.wave, lane = me.lane;
    Stage<DP, QT, CT, FULL, 32, kWave> st;
    Rows32<DP> r;
    bool bad = false;
    int t0 = u.lo + lo_tile * kTile + wave * 32;
    const int end = hi_tile < u.tiles() ? u.lo + hi_tile * kTile : u.hi;
    uint8_t* lk = lds + wave * Lds<DP>::wave;
    uint8_t* lv = lk + Lds<DP>::wave / 2;
    int64_t slot = -1;
    Lookup next{0, (uint32_t)kNone};
    if (t0 < end) {
      slot = slot_of(look_up(t0 + lane % 32), &bad);
      next = look_up(t0 + kTile + lane % 32);
      st.load(kb, vb, slot, lane, head_bytes, lk, lv);
    }
    load_rows(r, index * kRowsSplit);
    const Reads<DP> rd(lk, lv);
    const int least = least_limit(r);
    for (; t0 < end; t0 += kTile) {
      const uint64_t valid = ballot(slot >= 0) & 0xffffffffull;
      const bool edge = t0 + 32 > least || valid != 0xffffffffull;
      if constexpr (decltype(st)::direct) settle_copies();
      int special = kNone;
      if (edge) special = st.template store<true>(lk, lv, valid, lane, head_bytes);
      else st.template store<false>(lk, lv, valid, lane, head_bytes);
      if (special != kNone) atomicMin(&sh.special, t0 + special);
      if constexpr (!decltype(st)::direct) {
        if (t0 + kTile < end) {
          slot = slot_of(next, &bad);
          st.load(kb, vb, slot, lane, head_bytes, lk, lv);
          next = look_up(t0 + 2 * kTile + lane % 32);
        }
      }
      step<DP, QT, 1>(r, rd, 0, c, edge, valid & below(r.limit, t0), [](int) {});
      if constexpr (decltype(st)::direct) {
        if (t0 + kTile < end) {
          slot = slot_of(next, &bad);
          // The step's reads of the tiles are done: the products took them.
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          st.load(kb, vb, slot, lane, head_bytes, lk, lv);
          next = look_up(t0 + 2 * kTile + lane % 32);
        }
      }
    }
    if (bad) atomicOr(a.status, EP_STATUS_BAD_PAGE);
    r.l = add_halves(r.l);
    // Every wave leaves its sums where its tiles were, as put() does; then all
    // threads join them, 16 bytes at a time.
    f32x4* mine = (f32x4*)(lds + wave * Lds<DP>::box);
    static_assert(Lds<DP>::box == Lds<DP>::wave, "a wave's sums take the place of its tiles");
    lay_out(r, mine, 1.0f);
    if (me.half == 0) {
      sh.stat[0][wave][lane % 32] = r.m;
      sh.stat[1][wave][lane % 32] = r.l;
    }
    __syncthreads();
    put_split(number, whole);
    const int special = wave_uniform(sh.special);
    if (special < end) add_special(number, whole, special, end);
    __syncthreads();  // LDS is free for the next item
    if (special != kNone) {
      if (tid == 0) sh.special = kNone;
      __syncthreads();
    }
  }

  // Tiles [lo_tile, hi_tile) of an item.
  __device__ __forceinline__ void run(int64_t number, bool whole) {
    Args& a = fresh(this->a);
    kb = (const uint8_t*)a.c.k + kvh * a.c.head_stride;
    vb = (const uint8_t*)a.c.v + kvh * a.c.head_stride;
    float f = a.scale * 1.44269504088896341f;
    if (CT == EP_DTYPE_E4M3) f *= a.c.k_scale[kvh];
    negate = f < 0.0f;
    // Equal scores all the same, and no 0 * inf where a key is hidden.
    c = f == 0.0f ? 1e-30f : fabsf(f);
    head_bytes = a.c.head_dim * Fmt<CT>::bytes;
    if (u.split()) split_keys(number, whole);
    else block_rows(number, whole);
  }
};

// Units base .. base + kBlock - 1 into sh.unit, placed behind `at` in the
// line and item[kind] of either kind, all of which move on by theirs.
__device__ __forceinline__ void place_units(Args& a, Shared& sh, int base, int64_t& at,
                                            int32_t item[2]) {
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave, u = base + tid;
  const int count = a.g.n_groups + a.b.n_seqs;
  const bool suffix = u >= a.g.n_groups;
  Unit t;
  int64_t x = 0;
  int32_t y[2] = {0, 0};
  bool late = false, bad = false;
  if (u < count) t = unit_of(a, sh, u, &late, &bad);
  if (blockIdx.x == 0 && bad) atomicOr(a.status, EP_STATUS_BAD_PAGE);
  // Groups in LDS are the first wave's in the first round; where it has the
  // sequences too, nobody waits for it.
  if (a.g.n_groups > 0 && a.g.n_groups <= kGroupTable) {
    uint64_t refused = ballot(!suffix && bad);
    if (count > kWave) {
      if (base == 0 && tid == 0) sh.refused = refused;
      __syncthreads();
      refused = sh.refused;
    }
    if (u < count && suffix && t.group >= 0 && ((refused >> t.group) & 1)) {
      t.group = -1;
      t.lo = 0;
      t.hi = clamp_int(t.len, 0, key_cap(a));
      late = false;
    }
  }
  if (u < count) {
    if (late) sh.any_short = 1;
    if (t.tiles() > 0) {
      y[suffix] = t.items() * a.c.n_heads;
      x = y[suffix] * t.item_length();
    }
  }
  const int64_t x0 = x;
  const int32_t y0 = y[0], y1 = y[1];
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int64_t xo = __shfl_up(x, d);
    const int32_t yo = __shfl_up(y[0], d), zo = __shfl_up(y[1], d);
    if (lane >= d) {
      x += xo;
      y[0] += yo;
      y[1] += zo;
    }
  }
  if (lane == kWave - 1) {
    sh.part[wave] = x;
    sh.ipart[wave] = y[0];
    sh.spart[wave] = y[1];
  }
  __syncthreads();
  int64_t all = 0;
  int32_t all0 = 0, all1 = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) {
      x += sh.part[w];
      y[0] += sh.ipart[w];
      y[1] += sh.spart[w];
    }
    all += sh.part[w];
    all0 += sh.ipart[w];
    all1 += sh.spart[w];
  }
  if (u == a.g.n_groups) sh.prefix = at + x - x0;
  if (u < count) {
    t.start = at + x - x0;
    t.item = suffix ? item[1] + y[1] - y1 : item[0] + y[0] - y0;
    sh.unit[tid] = t;
  }
  at += all;
  item[0] += all0;
  item[1] += all1;
  __syncthreads();
}

template <int DP, int QT, int CT, bool FULL>
__global__ __launch_bounds__(kBlock, DP <= 128 ? 2 : 1) void attend_kernel(Attend) {
  Args& a = *(Args*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Lds<DP>::bytes];
  __shared__ Shared sh;
  const int tid = threadIdx.x;
  const int units = a.g.n_groups + a.b.n_seqs;
  if (tid == 0) {
    sh.any_short = 0;
    sh.special = kNone;  // between items
  }
  load_groups(a, sh);
  __syncthreads();
  // The line's length; a batch of up to kBlock units stays in LDS.
  int64_t total = 0;
  int32_t item[2] = {0, 0};
  for (int base = 0; base < units; base += kBlock) place_units(a, sh, base, total, item);
  total = wave_uniform64(total);
  const int64_t prefix = wave_uniform64(sh.prefix);
  const bool scribe = blockIdx.x == 0;
  const int per_xcd = a.workers / kXcds;
  const int w = blockIdx.x % kXcds * per_xcd + blockIdx.x / kXcds;
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    const Range part = range_of(a, kind, w, prefix, total - prefix);
    const int64_t begin = part.begin, end = part.end;
    const bool write = scribe && kind == 0;
    if (begin == end && !write) continue;
    int64_t at = 0;
    item[0] = item[1] = 0;
    for (int base = 0; base < units && (write || at < end); base += kBlock) {
      const int64_t from = at;
      if (units > kBlock) {
        place_units(a, sh, base, at, item);
        at = wave_uniform64(at);
      } else {
        at = total;
      }
      const int count = units - base < kBlock ? units - base : kBlock;
      if (write && tid < count) a.units[base + tid] = sh.unit[tid];
      if (begin >= at || end <= from || begin == end) continue;
      // From the last item backwards: workgroups that take the same keys for
      // different rows then begin at the keys' start together, and stay in
      // step for as long as they read the same item, so that each tile comes
      // from memory to an XCD about once. The unit that holds the last point,
      // or this round's last one.
      const int64_t stop = tid + 1 < count ? sh.unit[tid + 1].start : at;
      __syncthreads();  // the other line's reads of it
      if (tid == 0) sh.first = count - 1;
      __syncthreads();
      if (tid < count && sh.unit[tid].start < end && end <= stop) sh.first = tid;
      __syncthreads();
      for (int k = wave_uniform(sh.first); k >= 0; --k) {
        const Unit v = uniform_unit(sh.unit[k]);
        const int64_t len = v.item_length();
        if (len == 0) continue;
        const int per = v.items(), n = per * a.c.n_heads, tiles = v.tiles();
        if (v.start + n * len <= begin) break;
        // The last item that starts before `end`.
        const int64_t room = end - v.start < n * len ? end - v.start - 1 : n * len - 1;
        int i = ((room | len) >> 32) == 0 ? (int)((uint32_t)room / (uint32_t)len)
                                          : (int)(room / len);
        for (; i >= 0 && v.start + (i + 1) * len > begin; --i) {
          Body<DP, QT, CT, FULL> b{a, sh, lds};
          b.u = v;
          b.prefix = kind == 0;
          b.kvh = i / per;
          b.index = i % per;
          const int64_t start = v.start + i * len;
          b.lo_tile = tiles_before(v, start, begin);
          b.hi_tile = tiles_before(v, start, end);
          if (b.lo_tile >= b.hi_tile) continue;
          const bool whole = kind == 1 && v.lo == 0 && b.lo_tile == 0 && b.hi_tile == tiles;
          if (tid == 0 && fits(v.item + i, a.pieces[kind] - a.workers)) {
            if (b.lo_tile == 0) a.span[kind][v.item + i].x = w;
            if (b.hi_tile == tiles) a.span[kind][v.item + i].y = whole ? ~w : w;
          }
          b.run((int64_t)v.item + i + w, whole);
        }
      }
    }
  }
  if (scribe && tid == 0) {
    a.units[units].start = prefix;
    a.units[units + 1].start = total;
  }
}

// ---------------------------------------------------------------------------
// Joining the pieces. 16 lanes take a row and head (the chain of loads from
// the row to its pieces is most of the time, and a wave then has four on the
// way), or SHARE times 16 lanes where there are few rows, with the pieces dealt
// out among them.
// ---------------------------------------------------------------------------
constexpr int kJoin = 16;  // lanes

struct Part {
  int64_t start;  // of the row's item, in the lines
  int item, row;  // number of the item, row of the piece
  int w0, n;      // workgroups that may hold pieces of it: w0 .. w0 + n - 1
  bool whole;     // written by the first launch
};

__device__ __forceinline__ Part part_of(const Attend& a, const Unit& u, int kind, int token,
                                        int share_row, int kvh) {
  Part p;
  p.n = 0;
  p.whole = false;
  const int row = (token - u.row0) * a.share + share_row;
  if (u.tiles() == 0 || row < 0 || row >= u.rows) return p;
  const int i = kvh * u.items() + row / u.tile_rows();
  p.start = u.start + i * u.item_length();
  p.item = u.item + i;
  p.row = row % u.tile_rows();
  if (!fits(p.item, a.pieces[kind] - a.workers)) return p;
  const int2 span = a.span[kind][p.item];
  p.w0 = span.x;
  p.whole = span.y < 0;
  p.n = (p.whole ? ~span.y : span.y) - span.x + 1;
  return p;
}

// seq_of_row() by the kJoin lanes that have the same i.
__device__ __forceinline__ int seq_of_row16(const ep_kv_batch& b, int i) {
  if (!b.q_off) return i < b.n_seqs ? i : -1;
  const int lane = lane_id(), at = lane % kJoin;
  int lo = 0, hi = b.n_seqs;  // the answer lies in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + kJoin - 1) / kJoin;
    const int j = lo + at * step;
    const uint64_t mask = ballot(j < hi && b.q_off[j < hi ? j : lo] <= i);
    const uint32_t mine = (uint32_t)(mask >> (lane - at)) & ((1u << kJoin) - 1);
    if (mine == 0) return -1;
    lo += (31 - __builtin_clz(mine)) * step;
    hi = hi < lo + step ? hi : lo + step;
  }
  return lo < b.n_seqs && b.q_off[lo] <= i && i < b.q_off[lo + 1] ? lo : -1;
}

template <int DP, int QT, int SHARE>
__global__ __launch_bounds__(kBlock) void join_kernel(Attend a, int64_t rows) {
  constexpr int kGroups = kBlock / kJoin;   // of a workgroup
  constexpr int kQuads = DP / (4 * kJoin);  // elements 4 * (lane + kJoin q) .. + 3 of a lane
  constexpr int kAhead = 4;                 // pieces read at a time
  __shared__ float box[SHARE > 4 ? kWaves : 1][DP + 2];
  const int at = threadIdx.x % kJoin, group = threadIdx.x / kJoin, part_no = group % SHARE;
  const int count = a.g.n_groups + a.b.n_seqs;
  const int64_t prefix = a.units[count].start, suffix = a.units[count + 1].start - prefix;
  const int64_t stride = (int64_t)gridDim.x * (kGroups / SHARE);
  for (int64_t i = (int64_t)blockIdx.x * (kGroups / SHARE) + group / SHARE; i < rows;
       i += stride) {
    const int token = (int)((uint32_t)i / (uint32_t)a.heads);  // rows < 2^31
    const int head = (int)i - token * a.heads, kvh = head / a.share;
    const int s = seq_of_row16(a.b, token);
    bool done = s < 0;
    Unit su;
    Part part[2];
    part[0].n = part[1].n = 0;
    part[0].whole = part[1].whole = false;
    Unit pu;
    if (!done) {
      su = a.units[a.g.n_groups + s];
      pu = su;
      const int64_t last = (int64_t)su.len - su.fresh + (token - su.row0);
      const bool skip = token - su.row0 >= a.max_new || su.fresh == 0;
      // Skipped rows, and positions behind the table's end.
      if ((skip || last >= key_cap(a)) && at == 0 && part_no == 0)
        atomicOr(a.status, EP_STATUS_BAD_PAGE);
      done = skip;
    }
    if (!done) {
      if (su.group >= 0) {
        pu = a.units[su.group];
        part[0] = part_of(a, pu, 0, token, head % a.share, kvh);
      }
      part[1] = part_of(a, su, 1, token, head % a.share, kvh);
      done = part[1].whole;
    }
    if (SHARE == 1 && done) continue;
    if (SHARE > 1 && __all(done)) continue;  // all groups of a row agree
    const int most = part[0].n + part[1].n;
    float m = -__builtin_inff(), l = 0.0f;
    f32x4 o[kQuads] = {};
    for (int k0 = 0; k0 < most; k0 += kJoin * SHARE) {
      const int k = k0 + at * SHARE + part_no;
      const bool pre = k < part[0].n;
      const Part& p = pre ? part[0] : part[1];
      const Unit& u = pre ? pu : su;
      const int w = p.w0 + (pre ? k : k - part[0].n), kind = pre ? 0 : 1;
      const float* x = nullptr;
      float2 st = make_float2(-__builtin_inff(), 0.0f);
      if (k < most) {
        const Range r = range_of(a, kind, w, prefix, suffix);
        const int64_t number = (int64_t)w + p.item;
        if (tiles_before(u, p.start, r.begin) < tiles_before(u, p.start, r.end) &&
            fits(number, a.pieces[kind])) {
          const int64_t row = number * a.rows[kind] + p.row;
          st = a.stat[kind][row];
          if (st.x != -__builtin_inff()) x = a.sum[kind] + row * DP;
        }
      }
      float top = st.x;
#pragma unroll
      for (int d = 1; d < kJoin; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
      top = fmaxf(top, m);
      if (top == -__builtin_inff()) continue;
      const float scale = __builtin_amdgcn_exp2f(m - top);
      const float wgt = x ? __builtin_amdgcn_exp2f(st.x - top) : 0.0f;
      float sum = wgt * st.y;
#pragma unroll
      for (int d = 1; d < kJoin; d <<= 1) sum += __shfl_xor(sum, d);
      l = l * scale + sum;
      m = top;
#pragma unroll
      for (int q = 0; q < kQuads; ++q) o[q] *= scale;
      const int lane0 = lane_id() - at;
      uint32_t mask = (uint32_t)(ballot(x != nullptr) >> lane0) & ((1u << kJoin) - 1);
      while (mask) {
        f32x4 v[kAhead][kQuads];
        float f[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          // Behind the last piece: the last one again, with no weight.
          const int src = mask ? __builtin_ctz(mask) : -1;
          mask &= mask - 1;
          f[j] = src >= 0 ? __shfl(wgt, lane0 + (src >= 0 ? src : 0)) : 0.0f;
          const float* y = (const float*)__shfl((uint64_t)x, lane0 + (src >= 0 ? src : 0));
#pragma unroll
          for (int q = 0; q < kQuads; ++q)
            v[j][q] = src >= 0 ? *(const f32x4*)(y + 4 * (at + kJoin * q)) : f32x4{};
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
          for (int q = 0; q < kQuads; ++q) o[q] += v[j][q] * f[j];
      }
    }
    if constexpr (SHARE > 1) {
      // The groups of a wave, then the waves.
      float top = m;
#pragma unroll
      for (int d = kJoin; d < kWave; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
      const float f = m == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m - top);
      m = top;
      l *= f;
#pragma unroll
      for (int d = kJoin; d < kWave; d <<= 1) l += __shfl_xor(l, d);
#pragma unroll
      for (int q = 0; q < kQuads; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y = o[q][e] * f;
#pragma unroll
          for (int d = kJoin; d < kWave; d <<= 1) y += __shfl_xor(y, d);
          o[q][e] = y;
        }
    }
    if constexpr (SHARE > 4) {
      const int wave = threadIdx.x / kWave;
      __syncthreads();  // the last row's reads
      if (lane_id() < kJoin) {
#pragma unroll
        for (int q = 0; q < kQuads; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) box[wave][4 * (at + kJoin * q) + e] = o[q][e];
        if (at == 0) {
          box[wave][DP] = m;
          box[wave][DP + 1] = l;
        }
      }
      __syncthreads();
      float top = box[0][DP];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) top = fmaxf(top, box[w][DP]);
      l = 0.0f;
#pragma unroll
      for (int q = 0; q < kQuads; ++q) o[q] = f32x4{};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float mw = box[w][DP];
        const float f = mw == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(mw - top);
        l += box[w][DP + 1] * f;
#pragma unroll
        for (int q = 0; q < kQuads; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[q][e] += box[w][4 * (at + kJoin * q) + e] * f;
      }
      m = top;
    }
    if (part_no != 0 || done) continue;
    uint8_t* to = (uint8_t*)a.out.p + (int64_t)token * a.out.token_stride +
                  (int64_t)head * a.out.head_stride;
    const float vs = a.c.dtype == EP_DTYPE_E4M3 ? a.c.v_scale[kvh] : 1.0f;
    const float inv = l == 0.0f ? 0.0f : vs / l;
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
      const int d = 4 * (at + kJoin * q);
      if (d >= a.c.head_dim) continue;
      typename Fmt<QT>::elem w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = (typename Fmt<QT>::elem)(o[q][e] * inv);
      *(u32x2*)(to + 2 * d) = u32x2{as<uint16_t>(w[0]) | (uint32_t)as<uint16_t>(w[1]) << 16,
                                    as<uint16_t>(w[2]) | (uint32_t)as<uint16_t>(w[3]) << 16};
    }
    if (a.lse && at == 0)
      a.lse[i] = l == 0.0f ? -__builtin_inff() : (m + log2f(l)) * 0.69314718055994531f;
  }
}

struct Layout {
  int dim;  // padded head size
  int workers;
  uint32_t page_magic, page_shift;  // t / page_tokens = mulhi(t, magic) >> shift
  int pieces[2], rows[2];
  size_t units, span[2], stat[2], sum[2], bytes;
};

size_t up(size_t n) { return (n + 255) & ~(size_t)255; }

Layout layout(const ep_kv_cache& c, int n_seqs, int n_groups, int n_tokens, int n_heads,
              int max_new) {
  Layout l{};
  l.dim = c.head_dim <= 64 ? 64 : c.head_dim <= 128 ? 128 : 256;
  l.workers = l.dim <= 128 ? 512 : 256;
  const int64_t rows = (int64_t)n_tokens * (n_heads / c.n_heads);  // per KV head
  const int64_t most = (int64_t)max_new * (n_heads / c.n_heads);
  l.rows[0] = n_groups > 0 ? kRowsBlock : 0;
  l.rows[1] = most <= kRowsSplit ? kRowsSplit : kRowsBlock;
  // Items: one per unit and full tile_rows more; units of few rows take one.
  const int64_t items0 = n_groups > 0 ? (rows / kRowsBlock + n_groups) * c.n_heads : 0;
  const int64_t full = most <= kRowsSplit ? 0 : rows / kRowsBlock;
  const int64_t items1 = (full + (n_seqs < n_tokens ? n_seqs : n_tokens)) * c.n_heads;
  const int64_t p0 = items0 > 0 ? items0 + l.workers : 0, p1 = items1 + l.workers;
  l.pieces[0] = (int)(p0 < 0x7fffffff ? p0 : 0x7fffffff);
  l.pieces[1] = (int)(p1 < 0x7fffffff ? p1 : 0x7fffffff);
  size_t at = 0;
  const int64_t units = (int64_t)n_seqs + n_groups;
  l.units = at;
  at += up((size_t)(units + 2) * sizeof(Unit));
  for (int k = 0; k < 2; ++k) {
    l.span[k] = at;
    at += up((size_t)l.pieces[k] * sizeof(int2));
    l.stat[k] = at;
    at += up((size_t)l.pieces[k] * l.rows[k] * 8);
    l.sum[k] = at;
    at += up((size_t)l.pieces[k] * l.rows[k] * l.dim * 4);
  }
  l.bytes = at;
  return l;
}

template <int DP, int QT, int CT>
hipError_t launch(const Attend& a, hipStream_t stream) {
  // FULL spares the copies of 16-bit rows a comparison per chunk.
  constexpr bool direct = CT != EP_DTYPE_E4M3 && DP <= 128;
  if (direct && a.c.head_dim == DP)
    hipLaunchKernelGGL((attend_kernel<DP, QT, CT, direct>), dim3(a.workers), dim3(kBlock), 0,
                       stream, a);
  else
    hipLaunchKernelGGL((attend_kernel<DP, QT, CT, false>), dim3(a.workers), dim3(kBlock), 0,
                       stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // More lanes to a row where it has many pieces: where items are few, and
  // each is cut for many workgroups (16 pieces per row, 160 rows: 40.6 us with
  // 16 groups, 42.3 with one; 3 pieces, 1200 rows: 110.2 with one, 113.8 with
  // 16; one piece, 5120 rows: 397 and 407).
  const int64_t rows = (int64_t)a.b.n_tokens * a.heads;
  const int64_t items = (int64_t)a.pieces[0] + a.pieces[1] - (a.pieces[0] > 0 ? 2 : 1) * a.workers;
  const int share = a.workers >= 8 * items ? 16 : a.workers >= 3 * items ? 4 : 1;
  const int per = kBlock / kJoin / share;
  const int64_t blocks = (rows + per - 1) / per;
  const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20));
  if (share == 1)
    hipLaunchKernelGGL((join_kernel<DP, QT, 1>), grid, dim3(kBlock), 0, stream, a, rows);
  else if (share == 4)
    hipLaunchKernelGGL((join_kernel<DP, QT, 4>), grid, dim3(kBlock), 0, stream, a, rows);
  else
    hipLaunchKernelGGL((join_kernel<DP, QT, 16>), grid, dim3(kBlock), 0, stream, a, rows);
  return hipGetLastError();
}

template <int DP>
hipError_t launch_dim(const Attend& a, hipStream_t stream) {
  const bool e4m3 = a.c.dtype == EP_DTYPE_E4M3;
  if (a.b.dtype == EP_DTYPE_BF16)
    return e4m3 ? launch<DP, EP_DTYPE_BF16, EP_DTYPE_E4M3>(a, stream)
                : launch<DP, EP_DTYPE_BF16, EP_DTYPE_BF16>(a, stream);
  return e4m3 ? launch<DP, EP_DTYPE_F16, EP_DTYPE_E4M3>(a, stream)
              : launch<DP, EP_DTYPE_F16, EP_DTYPE_F16>(a, stream);
}

}  // namespace

size_t kv_attend_bytes(const ep_kv_cache& c, int n_seqs, int n_groups, int n_tokens, int n_heads,
                       int max_new) {
  return layout(c, n_seqs, n_groups, n_tokens, n_heads, max_new).bytes;
}

hipError_t launch_kv_attend(const ep_kv_cache& c, const ep_kv_batch& b, const ep_kv_groups& g,
                            int max_new, const ep_rows& q, int n_heads, const ep_rows& out,
                            float* lse, float sm_scale, void* ws, int32_t* status,
                            hipStream_t stream) {
  const Layout l = layout(c, b.n_seqs, g.n_groups, b.n_tokens, n_heads, max_new);
  char* p = (char*)ws;
  // For d > 1 with 2^(l - 1) < d <= 2^l: magic = floor(2^(31 + l) / d) + 1 fits
  // 32 bits, and mulhi(t, magic) >> (l - 1) = t / d for t < 2^31, since magic d
  // is past 2^(31 + l) by at most d <= 2^l.
  uint32_t magic = 0, shift = 0;
  if (c.page_tokens > 1) {
    while ((int64_t)1 << (shift + 1) < c.page_tokens) ++shift;
    magic = (uint32_t)(((uint64_t)1 << (32 + shift)) / (uint64_t)c.page_tokens) + 1;
  }
  const Attend a{c,
                 b,
                 g,
                 q,
                 out,
                 lse,
                 sm_scale,
                 n_heads,
                 n_heads / c.n_heads,
                 max_new,
                 l.workers,
                 magic,
                 shift,
                 (Unit*)(p + l.units),
                 {(int2*)(p + l.span[0]), (int2*)(p + l.span[1])},
                 {(float*)(p + l.sum[0]), (float*)(p + l.sum[1])},
                 {(float2*)(p + l.stat[0]), (float2*)(p + l.stat[1])},
                 {l.pieces[0], l.pieces[1]},
                 {l.rows[0], l.rows[1]},
                 status};
  if (l.dim == 64) return launch_dim<64>(a, stream);
  if (l.dim == 128) return launch_dim<128>(a, stream);
  return launch_dim<256>(a, stream);
}

}  // namespace ep
