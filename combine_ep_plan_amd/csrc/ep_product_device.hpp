// Tiles of matrix products over the experts' groups of rows, shared by the
// grouped product and its backward pass.
//
// A workgroup computes C[r][c] = sum_k R[r][k] Cc[c][k] for BR rows (r) and BC
// columns (c). Both operands go to LDS with copies that pass through no
// registers, 128 bytes of k a step, `stages` steps on their way. An operand
// lies in memory either with k dense (rows of 128 bytes in LDS) or with k as
// its slow axis (64 rows of B values in LDS, read with the transposing LDS
// reads). The 16x16 matrix products are laid out so that a lane holds one row
// r (lane % 16) and four neighbouring columns c: register i of a fragment is
// column 4 (lane / 16) + i of its 16.
//
// Reads past an operand's end give zeros (the buffer's bounds), so k may end
// inside a step. Rows and columns past the end of the tile's group or matrix
// compute what nothing stores.
#pragma once

#include <cmath>
#include <utility>

#include "ep_device.hpp"
#include "ep_kernels.hpp"
#include "ep_tiles.hpp"

namespace ep {

typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kStep = 128;     // bytes of k in a step
constexpr int kFrag = 16;      // rows or columns of a fragment
constexpr uint32_t kNowhere = 0x80000000u;  // an offset past every buffer's end

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// Where exp(-z) passes the floats' range (z < -88.7) this is 0; the true value
// times z is under 2^-120 there.
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + __expf(-z)); }

// Density and distribution function of the standard normal distribution at z.
// The tail beyond |z| is the density times Mills' ratio, which is smooth: a
// polynomial in u = 1 / (1 + 0.3 |z|) fitted to it (least squares in the
// relative error, reweighted towards its maximum) is within 2^-20 of the ratio
// for all z. The exponent a = z^2 / 2 adds its roundings, 2.3 a 2^-24 relative
// in density and tail: of all bf16 z, GELU's slope is within 2^-20 of its terms
// up to |z| = 5 and within 2^-18 up to 13, behind which the density is below
// 2^-120. erfcf() takes 140 instructions and made the 32 values of a thread 9
// us of a small backward pass; this takes 20.
struct Normal {
  float density, below;
};
__device__ __forceinline__ Normal normal_at(float z) {
  const float u = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, fabsf(z), 1.0f));
  float m = 4.652415588e-02f;
  m = __builtin_fmaf(m, u, -1.212453768e-01f);
  m = __builtin_fmaf(m, u, 7.356668357e-03f);
  m = __builtin_fmaf(m, u, 9.863400459e-02f);
  m = __builtin_fmaf(m, u, 1.256773323e-01f);
  m = __builtin_fmaf(m, u, 2.238885313e-01f);
  m = __builtin_fmaf(m, u, 2.724575102e-01f);
  m = __builtin_fmaf(m, u, 3.000220060e-01f);
  m = __builtin_fmaf(m, u, 2.999998331e-01f);
  const float density = 0.39894228040143268f * __expf(-0.5f * z * z);
  const float tail = m * u * density;
  return Normal{density, z < 0.0f ? tail : 1.0f - tail};
}

// Bytes [base, base + size) as the buffer instructions take them (raw: 32-bit
// offsets, reads past the end give zeros; no bytes when size is negative).
__device__ __forceinline__ u32x4 buffer_of(const uint8_t* base, int size) {
  const uint64_t p = (uint64_t)(uintptr_t)base;
  return u32x4{(uint32_t)wave_uniform((int)(uint32_t)p),
               (uint32_t)wave_uniform((int)(uint32_t)(p >> 32)),
               (uint32_t)wave_uniform(size > 0 ? size : 0), 0x00020000u};
}

// Starts the copy of 16 (or 4) bytes per lane from offset `at` of the buffer
// to LDS, lane l's to `to` + 16 l (4 l). Nothing waits for it but settle().
// ONCE: nothing else reads the bytes soon (they do not stay in the caches).
template <bool ONCE>
__device__ __forceinline__ void copy16(const u32x4& from, uint32_t at, uint32_t to) {
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
                 :
                 : "s"(to), "v"(at), "s"(from)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(to), "v"(at), "s"(from)
                 : "memory", "m0");
}
__device__ __forceinline__ void copy4(const u32x4& from, uint32_t at, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(to), "v"(at), "s"(from)
               : "memory", "m0");
}

// All but the wave's last N copies have arrived and its reads of LDS are done;
// then all waves' (barrier).
template <int N>
__device__ __forceinline__ void settle() {
  static_assert(N <= 63, "the wait counts to 63");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// f(0), ..., f(N - 1) with compile-time numbers: loops of several hundred
// products and reads whose registers must have fixed names.
template <int... I, typename F>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
  each_of(std::make_integer_sequence<int, N>{}, f);
}

// f(q) for those of n things that stand at slot m when they are spread over
// `slots` slots: q slots / n rounded down is m.
template <int N, int SLOTS, int M, typename F>
__device__ __forceinline__ void spread(F&& f) {
  constexpr int from = (M * N + SLOTS - 1) / SLOTS, to = ((M + 1) * N + SLOTS - 1) / SLOTS;
  each<to - from>([&](auto i) { f(std::integral_constant<int, from + decltype(i)::value>{}); });
}

template <typename V>
__device__ __forceinline__ V read_lds(uint32_t at) {
  typedef V __attribute__((address_space(3))) lds_v;
  return *(lds_v*)(uintptr_t)at;
}

// One operand: B rows (or columns) of the product, T: k is the slow axis.
template <int B, bool T, int WAVES>
struct Operand {
  static constexpr int copies = B * kStep / 1024 / WAVES;  // per wave and step
  static_assert(copies * WAVES * 1024 == B * kStep, "whole copies");
  static constexpr int row = T ? B * 2 : kStep;            // bytes in LDS
  static constexpr int rows = 1024 / row;                  // of a copy
  static_assert(!T || (B % 128 == 0 && rows >= 1 && (copies & (copies - 1)) == 0),
                "the places of a slow-k tile's chunks are by bits of the row");

  // 16-byte chunks of row r are stored at their number ^ turn(r): places that
  // make the reads of a wave meet all banks (they take eight rows of a dense-k
  // tile at a time, rows 0-3 and 8-11 of 16 of a slow-k one).
  static __device__ __forceinline__ constexpr int turn(int r) {
    return T ? ((r & 3) | (r >> 1 & 4)) << 1 : r & 7;
  }

  uint32_t lane_row, lane_chunk;  // of the lane's chunk in a copy, in bytes
  uint32_t copy_at[copies];       // of the copies' first rows, the same for all lanes

  // row_at(r): byte offset of row r of the tile (dense k) or of row r of k
  // (slow k); `line`: from one row to the next inside a copy.
  template <typename F>
  __device__ __forceinline__ void init(F&& row_at, uint32_t line) {
    const int first = wave_uniform(threadIdx.x / kWave) * copies * rows;
    const int lane = lane_id(), r = lane * 16 / row, chunk = lane * 16 % row / 16;
    lane_row = r * line;
    lane_chunk = (chunk ^ turn(first + r)) * 16;
#pragma unroll
    for (int i = 0; i < copies; ++i) copy_at[i] = wave_uniform(row_at(first + i * rows));
  }

  // Whether the lane's chunk lies before the end of k, `left` bytes from the
  // step's start (always, for a slow-k tile: rows behind k are behind the
  // buffer).
  __device__ __forceinline__ bool before(int left) const { return T || (int)lane_chunk < left; }

  // Bytes that a step may read, given those from its first row on (dense k) or
  // the bytes of k that are left and of the first row before the tile (slow k).
  static __device__ __forceinline__ int bytes(int size, int left, int line, int off) {
    if constexpr (!T) return size;
    else return (left < kStep ? left : kStep) / 2 * line - off;
  }

  // Copy i of the wave's.
  template <bool ONCE>
  __device__ __forceinline__ void load(int i, const u32x4& from, uint32_t to, bool there) const {
    const int wave = wave_uniform(threadIdx.x / kWave);
    const uint32_t at = lane_row + (lane_chunk ^ (turn(i * rows) * 16)) + copy_at[i];
    copy16<ONCE>(from, there ? at : kNowhere, to + (wave * copies + i) * 1024);
  }
};

// Where a lane reads fragments of 16 rows: `first` is the wave's first row.
template <int B, bool T, int F>
struct Reads {
  static_assert(!T || (F & (F - 1)) == 0, "a slow-k tile's fragments are by bits");
  uint32_t at;

  __device__ __forceinline__ Reads(int first) {
    const int lane = lane_id(), group = lane / 16, i16 = lane % 16;
    using Op = Operand<B, T, 1>;
    if constexpr (!T) {
      at = (first + i16) * kStep + (group ^ Op::turn(i16)) * 16;
    } else {
      // A group of 16 lanes reads 4 rows of k by 16 columns; lane i gets
      // column i of them.
      const int r = 8 * group + i16 / 4;
      at = r * Op::row + ((first / 16 * 2 + i16 % 4 / 2) ^ Op::turn(r)) * 16 + i16 % 2 * 8;
    }
  }

  // Fragment f of 32 values of k (the kk-th of a step): k = 8 group + j. The
  // places of other chunks are an exclusive or away from the first one's.
  __device__ __forceinline__ s16x8 get(uint32_t base, int f, int kk) const {
    if constexpr (!T) {
      return read_lds<s16x8>(((base + at) ^ (kk * 64)) + f * kFrag * kStep);
    } else {
      typedef s16x4 __attribute__((address_space(3))) lds_s16x4;
      constexpr int row = Operand<B, T, 1>::row;
      const uint32_t a = ((base + at) ^ (f * 32)) + kk * 32 * row;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)a);
      const s16x4 hi =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(a + 4 * row));
      return s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
  }

  // Fragment f of a step's 128 e4m3 values of k: chunks `group` and 4 + group,
  // which meet all banks as above. What counts is that both operands take the
  // same values of k.
  __device__ __forceinline__ i32x8 get8(uint32_t base, int f) const {
    static_assert(!T, "e4m3 operands have k dense");
    const uint32_t a = base + at;
    const u32x4 x = read_lds<u32x4>(a + f * kFrag * kStep);
    const u32x4 y = read_lds<u32x4>((a ^ 64) + f * kFrag * kStep);
    return i32x8{(int)x[0], (int)x[1], (int)x[2], (int)x[3],
                 (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
  }
};

// WR x WC waves of FR x FC fragments of 16 x 16. ONCE: no other workgroup reads
// the columns' operand.
template <int WR_, int FR_, int WC_, int FC_, bool RT_, bool CT_, bool FP8_, int STAGES_,
          bool ONCE_ = false>
struct Shape {
  static constexpr int WR = WR_, FR = FR_, WC = WC_, FC = FC_, stages = STAGES_;
  static constexpr bool RT = RT_, CT = CT_, FP8 = FP8_, ONCE = ONCE_;
  static constexpr int BR = WR * FR * kFrag, BC = WC * FC * kFrag, waves = WR * WC;
  static constexpr int threads = waves * kWave;
  // A stage: the two tiles; for e4m3 the scales of BR rows and of the waves'
  // two blocks of columns, and a place for what the waves without scales copy.
  static constexpr int scales_at = (BR + BC) * kStep;
  static constexpr int scale_slots = BR / kWave + (BR % kWave != 0);
  static constexpr int stage_bytes = scales_at + (FP8 ? (scale_slots + 2) * 256 : 0);
  static constexpr int lds_bytes = stage_bytes * stages;
  // A wave's copies in a step, those of scales with them.
  static constexpr int r_copies = Operand<BR, RT, waves>::copies + (FP8 ? 1 : 0);
  static constexpr int c_copies = Operand<BC, CT, waves>::copies + (FP8 ? 1 : 0);
  static constexpr int copies = r_copies + c_copies;
  static_assert(!FP8 || waves >= scale_slots, "a wave copies the scales of 64 rows");
  static_assert(!FP8 || FC * kFrag <= 128, "a wave's columns lie in one or two blocks of scales");
};

// What a tile multiplies, from some step of k on: the next copies' sources.
struct Feed {
  const uint8_t *r, *c;
  int r_size, c_size;      // dense k: bytes from there to the operand's end
  int r_off, c_off;        // slow k: bytes of a row before the tile
  int left;                // bytes of k, as a dense-k operand counts them (2 per value when bf16)
  const float *rs, *cs;    // e4m3: scales of the rows, [row][k / 128], and of the columns' blocks
  int rs_size, cs_size;

  __device__ __forceinline__ int steps() const { return (left + kStep - 1) / kStep; }
};

// A workgroup's tiles, one after the other. The copies of the next tile's
// first steps start during the last ones of a tile, so that neither the way
// from memory nor the tile's output leaves the matrix units without work for
// long: apart, a tile of 16 steps took 38 us of which 25 were its steps.
template <typename S>
struct Tile {
  f32x4 acc[S::FR][S::FC];
  int wr, wc;  // the wave's place

  using ROperand = Operand<S::BR, S::RT, S::waves>;
  using COperand = Operand<S::BC, S::CT, S::waves>;
  using RReads = Reads<S::BR, S::RT, S::FR>;
  using CReads = Reads<S::BC, S::CT, S::FC>;

  ROperand ro;
  COperand co;
  RReads rr;
  CReads cr;
  int r_line, c_line;           // bytes from one row (of k, where it is slow) to the next
  uint32_t lds, here, last;     // the ring of steps; the places of this one and the one before
  uint32_t rs_lane, cs_lane;    // of the lane's scales
  Feed feed;                    // of the copies that start next
  // Where the copies of a step come from.
  struct {
    u32x4 r, c, rs, cs;
    bool r_there, c_there;
  } from;

  // r_at, c_at: byte offsets of rows (see Operand); rs_at(row), cs_at(wave column, parity of the fragment): byte
  // offsets of scales. The same for all of the workgroup's tiles.
  template <typename FR_AT, typename FC_AT, typename RS_AT, typename CS_AT>
  __device__ __forceinline__ Tile(uint32_t lds, int r_line, int c_line, FR_AT&& r_at,
                                  FC_AT&& c_at, RS_AT&& rs_at, CS_AT&& cs_at)
      : wr(wave_uniform(threadIdx.x / kWave) / S::WC),
        wc(wave_uniform(threadIdx.x / kWave) % S::WC),
        rr(wr * S::FR * kFrag),
        cr(wc * S::FC * kFrag),
        r_line(r_line),
        c_line(c_line),
        lds(lds) {
    ro.init(r_at, (uint32_t)r_line);
    co.init(c_at, (uint32_t)c_line);
    if constexpr (S::FP8) {
      // Waves copy the scales of 64 rows each, the first also those of the
      // columns; the others fill a place that nothing reads.
      const int wave = wave_uniform(threadIdx.x / kWave), lane = lane_id();
      rs_lane = wave * kWave + lane < S::BR ? rs_at(wave * kWave + lane) : kNowhere;
      cs_lane = wave == 0 && lane < 2 * S::WC ? cs_at(lane / 2, lane % 2) : kNowhere;
    }
  }

  // Sets the sources of one step's copies. Behind a tile's last step come those
  // of the tile after it, if there is one (once), else zeros from an empty
  // buffer, so that every stage counts the same number of copies.
  __device__ __forceinline__ void aim(const Feed& after, bool& chained) {
    if (feed.left <= 0) {
      if (chained) feed = after;
      else feed.r_size = feed.c_size = feed.rs_size = feed.cs_size = 0;
      chained = false;
    }
    from.r = buffer_of(feed.r, ROperand::bytes(feed.r_size, feed.left, r_line, feed.r_off));
    from.c = buffer_of(feed.c, COperand::bytes(feed.c_size, feed.left, c_line, feed.c_off));
    from.r_there = ro.before(feed.left);
    from.c_there = co.before(feed.left);
    feed.r += S::RT ? kStep / 2 * (int64_t)r_line : kStep;
    feed.c += S::CT ? kStep / 2 * (int64_t)c_line : kStep;
    feed.r_size -= kStep;
    feed.c_size -= kStep;
    feed.left -= kStep;
    if constexpr (S::FP8) {
      from.rs = buffer_of((const uint8_t*)feed.rs, feed.rs_size);
      from.cs = buffer_of((const uint8_t*)feed.cs, feed.cs_size);
      ++feed.rs;
      ++feed.cs;
      feed.rs_size -= 4;
      feed.cs_size -= 4;
    }
  }
  __device__ __forceinline__ void copy_r(int i, uint32_t to) {
    const int wave = wave_uniform(threadIdx.x / kWave);
    if (i < ROperand::copies)
      ro.template load<false>(i, from.r, to, from.r_there);
    else
      copy4(from.rs, rs_lane,
            to + S::scales_at + (wave < S::scale_slots ? wave : S::scale_slots + 1) * 256);
  }
  __device__ __forceinline__ void copy_c(int i, uint32_t to) {
    const int wave = wave_uniform(threadIdx.x / kWave);
    if (i < COperand::copies)
      co.template load<S::ONCE>(i, from.c, to + S::BR * kStep, from.c_there);
    else
      copy4(from.cs, cs_lane, to + S::scales_at + (S::scale_slots + (wave == 0 ? 0 : 1)) * 256);
  }

  // The products of tile p into acc. primed: its first copies have been started
  // by the run before it. chained: `after` is the tile of the next run, which
  // has at least as many steps as there are stages.
  __device__ __forceinline__ void run(const Feed& p, bool primed, const Feed& after, bool chained) {
    bool to_come = chained;
#pragma unroll
    for (int i = 0; i < S::FR; ++i)
#pragma unroll
      for (int j = 0; j < S::FC; ++j) acc[i][j] = f32x4{};
    if (!primed) {
      // As many copies as there are when a first step begins.
      feed = p;
#pragma unroll
      for (int s = 0; s < S::stages; ++s) {
        aim(after, to_come);
#pragma unroll
        for (int i = 0; i < S::c_copies; ++i) copy_c(i, lds + s * S::stage_bytes);
#pragma unroll
        for (int i = 0; i < S::r_copies; ++i)
          if (s < S::stages - 1 || i < early) copy_r(i, lds + s * S::stage_bytes);
      }
      here = lds;
      last = lds + (S::stages - 1) * S::stage_bytes;
      settle<(S::stages - 2) * S::copies + S::c_copies + early>();
      fetch_first(here);
    }
    const int steps = p.steps();
    for (int s = 0; s < steps; ++s) {
      const uint32_t next =
          here == lds + (S::stages - 1) * S::stage_bytes ? lds : here + S::stage_bytes;
      step(next, [&] { aim(after, to_come); });
      last = here;
      here = next;
    }
    if (!chained) settle<0>();
  }

  // Fragments on their way from LDS while the products before them run: in
  // turn two sets of 32 values of k; for e4m3 a step's fragments of columns and
  // in turn two of rows, with their scales.
  struct {
    s16x8 a[2][S::FP8 ? 1 : S::FC], b[2][S::FP8 ? 1 : S::FR];
    i32x8 a8[S::FP8 ? S::FC : 1], b8[2];
    float sc[2], sr[2];
  } f;

  // Part i of what the products of the kk-th 32 values of k need, in the order
  // in which they need it.
  static constexpr int parts = S::FC + S::FR;
  __device__ __forceinline__ void fetch(int i, uint32_t base, int kk) {
    if (i < S::FC) f.a[kk][i] = cr.get(base + S::BR * kStep, i, kk);
    else f.b[kk][i - S::FC] = rr.get(base, i - S::FC, kk);
  }
  __device__ __forceinline__ void fetch_row(int i, uint32_t base) {
    f.b8[i % 2] = rr.get8(base, i);
    f.sr[i % 2] = read_lds<float>(base + S::scales_at +
                                  ((wr * S::FR + i) * kFrag + lane_id() % 16) * 4);
  }
  __device__ __forceinline__ void fetch_column_scales(uint32_t base) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      f.sc[j] = read_lds<float>(base + S::scales_at + S::scale_slots * 256 + (wc * 2 + j) * 4);
  }

  __device__ __forceinline__ void fetch_first(uint32_t base) {
    if constexpr (!S::FP8) {
#pragma unroll
      for (int i = 0; i < parts; ++i) fetch(i, base, 0);
    } else {
      fetch_row(0, base);
      fetch_column_scales(base);
#pragma unroll
      for (int j = 0; j < S::FC; ++j) f.a8[j] = cr.get8(base + S::BR * kStep, j);
    }
  }

  // Copies of rows that start in the step before the one whose beginning has
  // the others.
  static constexpr int early = S::FP8 ? S::r_copies / 2 : S::r_copies;
  // e4m3: the columns' tile is free as soon as the step has begun, since its
  // fragments stay in registers.
  static constexpr bool columns_first = S::FP8 && S::FR >= 4;

  // One step's products. Before its last part every wave has read the step's
  // tiles (the last fragments are in registers) and the next step's have
  // arrived; then the copies of the step that is `stages` further, which aim()
  // finds, start in their place. They are spread over the products, since a
  // copy holds a wave up while the memory pipeline takes it.
  template <typename A>
  __device__ __forceinline__ void step(uint32_t next, A&& aim) {
    constexpr int products = S::FR * S::FC;
    if constexpr (!S::FP8) {
      each<2>([&](auto half) {
        constexpr int kk = half;
        if constexpr (kk == 1) settle<(S::stages - 2) * S::copies>();
        each<products>([&](auto product) {
          constexpr int m = product, i = m / S::FC, j = m % S::FC;
          // The reads before the barrier are through by then.
          constexpr int slots = kk ? products : (3 * products + 3) / 4;
          if constexpr (m < slots)
            spread<parts, slots, m>([&](auto q) { fetch(q, kk ? next : here, 1 - kk); });
          if constexpr (kk == 0 && m == slots - 1) aim();
          if constexpr (kk == 1)
            spread<S::copies, products, m>([&](auto q) {
              if constexpr (q < S::c_copies) copy_c(q, here);
              else copy_r(q - S::c_copies, here);
            });
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, f.a[kk][j]), __builtin_bit_cast(bf16x8, f.b[kk][i]),
              acc[i][j], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        });
      });
    } else {
      // The matrix instruction without scales of its own (constants of 0 select
      // it); the blocks' multiply its sum over 128 values of k, in 32 bits, two
      // products later, when it is there.
      constexpr int behind = 2;
      f32x4 sum[behind + 1];
      float by[S::FR][2];
      const auto scale = [&](auto product) {
        constexpr int m = product, i = m / S::FC, j = m % S::FC;
#pragma unroll
        for (int v = 0; v < 4; ++v)
          acc[i][j][v] = __builtin_fmaf(sum[m % (behind + 1)][v], by[i][j % 2], acc[i][j][v]);
      };
      each<S::FR>([&](auto fragment) {
        constexpr int i = fragment;
        constexpr bool turned = i == S::FR - 1;
        by[i][0] = f.sr[i % 2] * f.sc[0];
        by[i][1] = f.sr[i % 2] * f.sc[1];
        if constexpr (i == 1 && columns_first)
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
        if constexpr (turned) {
          settle<(S::stages - 2) * S::copies + (columns_first ? S::c_copies : 0)>();
          fetch_column_scales(next);
          if constexpr (S::FR % 2 == 0) fetch_row(0, next);
        } else {
          fetch_row(i + 1, here);
        }
        each<S::FC>([&](auto column) {
          constexpr int j = column, m = i * S::FC + j;
          // The instruction lines up the products of 8 neighbouring codes at their
          // largest exponent and keeps 13 bits below it (seen with 448^2 - 448^2
          // + 8 = 8, + 9 = 8, + 4 = 0); across the eights it adds accurately. The
          // one for 32 codes does the same and takes 11.2 ms where this takes 8.5
          // (2 x 8192 tokens, top-8 of 32, 2048 values to 7168).
          sum[m % (behind + 1)] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              f.a8[j], f.b8[i % 2], f32x4{}, 0, 0, 0, 0, 0, 0);
          if constexpr (turned) f.a8[j] = cr.get8(next + S::BR * kStep, j);
          if constexpr (i == 0) {
            spread<S::r_copies - early, S::FC, j>([&](auto q) { copy_r(early + q, last); });
            if constexpr (j == S::FC - 1) aim();
          }
          if constexpr (columns_first && i >= 1 && i < 3)
            spread<S::c_copies, 2 * S::FC, m - S::FC>([&](auto q) { copy_c(q, here); });
          if constexpr (turned) {
            if constexpr (!columns_first)
              spread<S::c_copies, S::FC, j>([&](auto q) { copy_c(q, here); });
            spread<early, S::FC, j>([&](auto q) { copy_r(q, here); });
          }
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (m >= behind) scale(std::integral_constant<int, m - behind>{});
          __builtin_amdgcn_sched_barrier(0);
        });
      });
      if constexpr (S::FR % 2 != 0) fetch_row(0, next);
      each<behind>([&](auto b) { scale(std::integral_constant<int, products - behind + b>{}); });
    }
  }
};

// Two neighbouring fragments' registers, turned so that a lane holds eight
// neighbouring columns of its row: lanes of odd groups of 16 swap the first
// fragment's values for the second's of the group before. The columns are
// 8 (group / 2) ... of fragment group % 2. Outputs then go out 16 bytes at a
// time and 64 in a row.
__device__ __forceinline__ void eight_columns(const f32x4& a, const f32x4& b, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(a[i]), __float_as_uint(b[i]),
                                                    false, false);
    v[i] = __uint_as_float(x[0]);
    v[4 + i] = __uint_as_float(x[1]);
  }
}
__device__ __forceinline__ int column_of_lane() {
  return lane_id() / 16 % 2 * kFrag + lane_id() / 32 * 8;
}

__device__ __forceinline__ void add8(float (&v)[8], const uint16_t* p) {
  const u32x4 u = *(const u32x4*)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] += bf16_lo(u[i]);
    v[2 * i + 1] += bf16_hi(u[i]);
  }
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *(u32x4*)p = u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                     pack_bf16(v[6], v[7])};
}

// The tile of this workgroup, among `cols` column blocks per block of BR rows;
// false: none is left. The tiles of the groups lie on a line that the eight
// XCDs (workgroup b runs on XCD b % 8) share in equal stretches, so that the
// workgroups beside each other in an L2 read the same rows and weights: a
// group's tiles go by stripes of eight column blocks, row blocks inside.
template <int BR, int THREADS>
__device__ __forceinline__ bool find_tile(const Groups& g, int cols, Where* out) {
  __shared__ int wave_sum[THREADS / kWave];
  __shared__ Where found;
  const int experts = g.N * g.L, tid = threadIdx.x, lane = lane_id(), room = room_of(g, BR);
  const int per = (experts + THREADS - 1) / THREADS;
  const int e0 = tid * per, e1 = e0 + per < experts ? e0 + per : experts;
  int mine = 0;
  for (int e = e0; e < e1; ++e) mine = add_blocks(mine, blocks_of(g, e, BR, room), room);
  int sum = mine, before = 0;  // before: of the threads before this one
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int up = __shfl_up(sum, off);
    if (lane >= off) sum = add_blocks(sum, up, room);
  }
  before = __shfl_up(sum, 1);
  if (lane == 0) before = 0;
  if (lane == kWave - 1) wave_sum[tid / kWave] = sum;
  if (tid == 0) found = Where{0, 0, 0, 0, 0};
  __syncthreads();
  int total = 0;
  for (int w = 0; w < THREADS / kWave; ++w) {
    if (w < tid / kWave) before = add_blocks(before, wave_sum[w], room);
    total = add_blocks(total, wave_sum[w], room);
  }
  const int64_t tiles = (int64_t)total * cols;
  const int64_t stretch = (tiles + 7) / 8;
  const int64_t slot = blockIdx.x / 8, want = (int64_t)(blockIdx.x % 8) * stretch + slot;
  if (slot >= stretch || want >= tiles) return false;
  int64_t left = want - (int64_t)before * cols;
  if (left >= 0 && left < (int64_t)mine * cols) {
    for (int e = e0; e < e1; ++e) {
      const Group gr = group_of(g, e);
      const int blocks = blocks_in(gr.rows, BR);
      if (left >= (int64_t)blocks * cols) {
        left -= (int64_t)blocks * cols;
        continue;
      }
      const RowCol rc = stripe_of((int)left, blocks, cols);
      found = where_of(gr, e, BR, rc.row, rc.col);
      break;
    }
  }
  __syncthreads();
  *out = Where{wave_uniform(found.expert), wave_uniform(found.first), wave_uniform(found.rows),
               wave_uniform(found.at), wave_uniform(found.col)};
  return true;
}

// Workgroups that hold every tile that find_tile can name; a multiple of 8.
inline int64_t tile_grid(const Groups& g, int br, int64_t cols) {
  return (room_of(g, br) * cols + 7) / 8 * 8;
}

// The tiles of a workgroup that takes one after the other. The groups' tiles
// lie on the line one group behind another; `ends` (a number per expert, in LDS):
// row blocks before the end of each expert's.
template <int BR, int THREADS>
struct Line {
  const Groups& g;
  int* ends;
  int experts, cols, taken;  // taken: tiles that the workgroup has had
  int64_t tiles;

  __device__ __forceinline__ Line(const Groups& g, int cols, int* ends)
      : g(g), ends(ends), experts(g.N * g.L), cols(cols), taken(0) {
    __shared__ int wave_sum[THREADS / kWave];
    const int tid = threadIdx.x, lane = lane_id(), room = room_of(g, BR);
    int total = 0;
    for (int e0 = 0; e0 < experts; e0 += THREADS) {
      const int e = e0 + tid;
      int sum = e < experts ? blocks_of(g, e, BR, room) : 0;
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) {
        const int up = __shfl_up(sum, off);
        if (lane >= off) sum = add_blocks(sum, up, room);
      }
      if (lane == kWave - 1) wave_sum[tid / kWave] = sum;
      __syncthreads();
      int all = 0;
      for (int w = 0; w < THREADS / kWave; ++w) {
        if (w < tid / kWave) sum = add_blocks(sum, wave_sum[w], room);
        all = add_blocks(all, wave_sum[w], room);
      }
      if (e < experts) ends[e] = add_blocks(total, sum, room);
      total = add_blocks(total, all, room);
      __syncthreads();
    }
    tiles = (int64_t)wave_uniform(total) * cols;
  }

  // The workgroup's next tile; false: none is left.
  __device__ __forceinline__ bool next(Where* out) {
    const int64_t want = tile_of(taken, tiles, gridDim.x, blockIdx.x);
    if (want < 0) return false;
    ++taken;
    const int block = (int)(want / cols);  // row blocks of whole groups lie before it
    int e = 0;
    for (int e0 = 0; e0 < experts; e0 += kWave)
      e += __popcll(ballot(e0 + lane_id() < experts && ends[e0 + lane_id()] <= block));
    e = wave_uniform(e);
    const Where t = tile_at(g, BR, e, wave_uniform(e > 0 ? ends[e - 1] : 0), want, cols);
    *out = Where{e, wave_uniform(t.first), wave_uniform(t.rows), wave_uniform(t.at),
                 wave_uniform(t.col)};
    return true;
  }
};

// What a kernel with tiles of br x bc takes, in units that compare kernels: a
// CU takes in operands at about 45 GB/s whatever the tile (7168 values by 4096
// columns, 32 x 64 with 64 rows: 36, 32 x 128 with 256: 46, 128 x 128 with 2048:
// 58, 256 x 256 with 2048 and 8192: 49 and 37), so the time goes by the rounds of
// 256 tiles and by the rows and columns that each takes in. The groups are taken
// to have the mean size, if routed and two standard deviations of a random count
// (a group that just passes a tile reads its weights twice: 32 rows on average
// take 3.2 ms in tiles of 32 x 128 and 2.2 to 2.4 in those of 64 x 256). rows: of
// a tile in steps of which the kernel skips rows that are not there.
inline int64_t cost_of(const Groups& g, int br, int rows, int bc, int64_t cols) {
  const int64_t experts = (int64_t)g.N * g.L, groups = experts < g.most ? experts : g.most;
  if (groups == 0) return 0;
  int64_t mean = (g.most + groups - 1) / groups;
  if (g.off) mean += (int64_t)(2.0 * std::sqrt((double)mean));
  const int64_t blocks = (mean + br - 1) / br;
  const int64_t each = (mean + blocks - 1) / blocks;
  const int64_t rounds = (groups * blocks * ((cols + bc - 1) / bc) + 255) / 256;
  return rounds * ((each + rows - 1) / rows * rows + bc);
}

// Workgroups for a line: one per CU, or as many as there are tiles.
inline unsigned line_grid(int64_t tiles) { return (unsigned)(tiles < 256 ? tiles : 256); }

__device__ __forceinline__ uint32_t lds_base(const void* p) {
  return (uint32_t)(uintptr_t)(const lds_u8*)p;
}

}  // namespace ep
