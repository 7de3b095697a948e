// Tiles of matrix products over the experts' groups of rows, shared by the
// grouped product and its backward pass.
//
// A workgroup computes C[r][c] = sum_k R[r][k] Cc[c][k] for BR rows (r) and BC
// columns (c). Both operands go to LDS with copies that pass through no
// registers, 128 bytes of k a step (64 bf16 or 128 e4m3), STAGES steps in
// turn. An operand lies in memory either with k dense (rows of 128 bytes in
// LDS) or with k as its slow axis (64 rows of B values in LDS, read with the
// transposing LDS reads). The 32x32 matrix products are laid out so that a
// lane holds one row r (lane % 32) and four neighbouring columns c at a time:
// register i is column 8 (i / 4) + 4 (lane / 32) + i % 4 of its 32.
//
// Reads past an operand's end give zeros (the buffer's bounds), so k may end
// inside a step. Rows and columns past the end of the tile's group or matrix
// compute what nothing stores.
#pragma once

#include "ep_device.hpp"
#include "ep_kernels.hpp"

namespace ep {

typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kStep = 128;     // bytes of k in a step
constexpr uint32_t kNowhere = 0x80000000u;  // an offset past every buffer's end

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// Bytes [base, base + size) as the buffer instructions take them (raw: 32-bit
// offsets, reads past the end give zeros).
__device__ __forceinline__ u32x4 buffer_of(const uint8_t* base, int64_t size) {
  const uint64_t p = (uint64_t)(uintptr_t)base;
  const int64_t n = size < 0 ? 0 : size < 0x7fffffff ? size : 0x7fffffff;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(p >> 32) & 0xffffu)),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)n), 0x00020000u};
}

// Starts the copy of 16 (or 4) bytes per lane from offset `at` of the buffer
// to LDS, lane l's to `to` + 16 l (4 l). Nothing waits for it but settle().
__device__ __forceinline__ void copy16(const u32x4& from, uint32_t at, uint32_t to) {
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
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
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
  uint32_t at[copies];

  // 16-byte chunks are stored at places that make the reads of a wave meet
  // all banks: eight rows of a dense-k tile, four of a slow-k one.
  static __device__ __forceinline__ int place(int r, int chunk) {
    if constexpr (!T) return chunk ^ (r & 7);
    else if constexpr (B % 128 == 0) return chunk ^ ((r & 3) << 2);
    else return chunk ^ ((r >> 1 & 1) << 2);
  }

  // Offsets of this lane's chunks; row_at(r): byte offset of row r of the tile
  // (dense k) or of row r of k (slow k).
  template <typename F>
  __device__ __forceinline__ void init(F&& row_at) {
    const int wave = threadIdx.x / kWave, lane = lane_id();
#pragma unroll
    for (int i = 0; i < copies; ++i) {
      const int byte = (wave * copies + i) * 1024 + lane * 16;
      const int r = byte / row, chunk = place(r, byte % row / 16);
      at[i] = row_at(r) + chunk * 16;
    }
  }

  // tail: bytes of k that are left, in a dense-k tile's last step.
  __device__ __forceinline__ void load(const u32x4& from, uint32_t to, int tail) const {
    const int wave = wave_uniform(threadIdx.x / kWave), lane = lane_id();
#pragma unroll
    for (int i = 0; i < copies; ++i) {
      uint32_t a = at[i];
      if (!T && tail < kStep) {
        const int byte = (wave * copies + i) * 1024 + lane * 16;
        if (place(byte / row, byte % row / 16) * 16 >= tail) a = kNowhere;
      }
      copy16(from, a, to + (wave * copies + i) * 1024);
    }
  }
};

// Where a lane reads fragments of 32 rows: `first` is the wave's first row.
template <int B, bool T, int F>
struct Reads {
  uint32_t at[T ? F : 4];

  __device__ __forceinline__ Reads(int first) {
    const int lane = lane_id(), half = lane / 32;
    using Op = Operand<B, T, 1>;
    if constexpr (!T) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        at[kk] = (first + lane % 32) * kStep + Op::place(lane, 2 * kk + half) * 16;
    } else {
      // A group of 16 lanes reads 4 rows of k by 16 columns; lane i gets
      // column i of them.
      const int i16 = lane % 16, r = 8 * half + i16 / 4;
#pragma unroll
      for (int f = 0; f < F; ++f)
        at[f] = r * Op::row +
                Op::place(r, (first / 32 + f) * 4 + lane / 16 % 2 * 2 + i16 % 4 / 2) * 16 +
                i16 % 2 * 8;
    }
  }

  // Fragment f of 16 values of k (the kk-th of a step): k = 8 half + j.
  __device__ __forceinline__ s16x8 get(uint32_t base, int f, int kk) const {
    if constexpr (!T) {
      return read_lds<s16x8>(base + at[kk] + f * 32 * kStep);
    } else {
      typedef s16x4 __attribute__((address_space(3))) lds_s16x4;
      constexpr int row = Operand<B, T, 1>::row;
      const uint32_t a = base + at[f] + kk * 16 * row;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)a);
      const s16x4 hi =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(a + 4 * row));
      return s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
  }

  // Fragment f of 64 e4m3 values of k: 32 per lane; both operands take the
  // same ones.
  __device__ __forceinline__ i32x8 get8(uint32_t base, int f, int kk) const {
    static_assert(!T, "e4m3 operands have k dense");
    const u32x4 a = read_lds<u32x4>(base + at[2 * kk] + f * 32 * kStep);
    const u32x4 b = read_lds<u32x4>(base + at[2 * kk + 1] + f * 32 * kStep);
    return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3],
                 (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
  }
};

// WR x WC waves of FR x FC fragments of 32 x 32.
template <int WR_, int FR_, int WC_, int FC_, bool RT_, bool CT_, bool FP8_, int STAGES_>
struct Shape {
  static constexpr int WR = WR_, FR = FR_, WC = WC_, FC = FC_, stages = STAGES_;
  static constexpr bool RT = RT_, CT = CT_, FP8 = FP8_;
  static constexpr int BR = WR * FR * 32, BC = WC * FC * 32, waves = WR * WC;
  static constexpr int threads = waves * kWave;
  // A stage: the two tiles; for e4m3 the scales of BR rows and of BC / 32
  // fragments, and a place for what the waves without scales copy.
  static constexpr int scales_at = (BR + BC) * kStep;
  static constexpr int scale_slots = BR / kWave + (BR % kWave != 0);
  static constexpr int stage_bytes = scales_at + (FP8 ? (scale_slots + 2) * 256 : 0);
  static constexpr int lds_bytes = stage_bytes * stages;
  static constexpr int copies = Operand<BR, RT, waves>::copies + Operand<BC, CT, waves>::copies +
                                (FP8 ? 1 : 0);
  static_assert(!FP8 || waves >= scale_slots + 1, "one copy of scales per wave");
};

// What a workgroup multiplies. Sizes in bytes from the tile's first byte.
struct Pair {
  const uint8_t *r, *c;
  int64_t r_size, c_size;
  int64_t r_step, c_step;  // bytes from one step to the next
  int64_t k_bytes;         // of k in all, as a dense-k operand counts it (2 per value when bf16)
  // e4m3: scales of the rows, [row][k / 128], and of the fragments' blocks.
  const float *rs, *cs;
  int64_t rs_size, cs_size;
};

template <typename S>
struct Tile {
  f32x16 acc[S::FR][S::FC];
  int wr, wc;  // the wave's place

  // r_at, c_at: byte offsets of rows (see Operand); rs_at(row), cs_at(fragment):
  // byte offsets of scales.
  template <typename FR_AT, typename FC_AT, typename RS_AT, typename CS_AT>
  __device__ __forceinline__ void run(const Pair& p, uint32_t lds, FR_AT&& r_at, FC_AT&& c_at,
                                      RS_AT&& rs_at, CS_AT&& cs_at) {
    const int wave = wave_uniform(threadIdx.x / kWave), lane = lane_id();
    wr = wave / S::WC;
    wc = wave % S::WC;
#pragma unroll
    for (int i = 0; i < S::FR; ++i)
#pragma unroll
      for (int j = 0; j < S::FC; ++j) acc[i][j] = f32x16{};
    Operand<S::BR, S::RT, S::waves> ro;
    Operand<S::BC, S::CT, S::waves> co;
    ro.init(r_at);
    co.init(c_at);
    uint32_t scale_at = kNowhere;
    const uint8_t* scale_base = nullptr;
    int64_t scale_size = 0;
    if constexpr (S::FP8) {
      scale_base = wave < S::scale_slots ? (const uint8_t*)p.rs : (const uint8_t*)p.cs;
      scale_size = wave < S::scale_slots ? p.rs_size : p.cs_size;
      if (wave < S::scale_slots) {
        if (wave * kWave + lane < S::BR) scale_at = rs_at(wave * kWave + lane);
      } else if (wave == S::scale_slots && lane < S::BC / 32) {
        scale_at = cs_at(lane);
      }
    }
    const Reads<S::BR, S::RT, S::FR> rr(wr * S::FR * 32);
    const Reads<S::BC, S::CT, S::FC> cr(wc * S::FC * 32);
    const int steps = (int)((p.k_bytes + kStep - 1) / kStep);
    // Steps past the last are copied too, as zeros from an empty buffer: every
    // stage counts the same number of copies.
    const auto start = [&](int s, uint32_t to) {
      const bool there = s < steps;
      const int64_t left = p.k_bytes - (int64_t)s * kStep;
      const int tail = left < kStep ? (int)left : kStep;
      ro.load(buffer_of(p.r + s * p.r_step, there ? p.r_size - s * p.r_step : 0), to, tail);
      co.load(buffer_of(p.c + s * p.c_step, there ? p.c_size - s * p.c_step : 0),
              to + S::BR * kStep, tail);
      if constexpr (S::FP8) {
        const int slot = wave <= S::scale_slots ? wave : S::scale_slots + 1;
        copy4(buffer_of(scale_base + 4 * s, there ? scale_size - 4 * s : 0), scale_at,
              to + S::scales_at + slot * 256);
      }
    };
#pragma unroll
    for (int s = 0; s < S::stages - 1; ++s) start(s, lds + s * S::stage_bytes);
    uint32_t here = lds, next = lds + (S::stages - 1) * S::stage_bytes;
    const uint32_t end = lds + S::lds_bytes;
    for (int s = 0; s < steps; ++s) {
      settle<(S::stages - 2) * S::copies>();
      start(s + S::stages - 1, next);
      step(here, rr, cr);
      here = here + S::stage_bytes == end ? lds : here + S::stage_bytes;
      next = next + S::stage_bytes == end ? lds : next + S::stage_bytes;
    }
    settle<0>();
  }

  __device__ __forceinline__ void step(uint32_t base, const Reads<S::BR, S::RT, S::FR>& rr,
                                       const Reads<S::BC, S::CT, S::FC>& cr) {
    const uint32_t cbase = base + S::BR * kStep;
    if constexpr (!S::FP8) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        s16x8 a[S::FC], b[S::FR];
#pragma unroll
        for (int j = 0; j < S::FC; ++j) a[j] = cr.get(cbase, j, kk);
#pragma unroll
        for (int i = 0; i < S::FR; ++i) b[i] = rr.get(base, i, kk);
#pragma unroll
        for (int i = 0; i < S::FR; ++i)
#pragma unroll
          for (int j = 0; j < S::FC; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                __builtin_bit_cast(bf16x8, a[j]), __builtin_bit_cast(bf16x8, b[i]), acc[i][j], 0, 0,
                0);
      }
    } else {
      const uint32_t sbase = base + S::scales_at;
      i32x8 a[S::FC][2];
      float sc[S::FC];
#pragma unroll
      for (int j = 0; j < S::FC; ++j) {
        a[j][0] = cr.get8(cbase, j, 0);
        a[j][1] = cr.get8(cbase, j, 1);
        sc[j] = read_lds<float>(sbase + S::scale_slots * 256 + (wc * S::FC + j) * 4);
      }
#pragma unroll
      for (int i = 0; i < S::FR; ++i) {
        const i32x8 b0 = rr.get8(base, i, 0), b1 = rr.get8(base, i, 1);
        const float sr = read_lds<float>(sbase + ((wr * S::FR + i) * 32 + lane_id() % 32) * 4);
#pragma unroll
        for (int j = 0; j < S::FC; ++j) {
          // Scales of 2^0 for both operands; the blocks' own multiply the sum
          // over their 128 values of k, in 32 bits.
          f32x16 s = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[j][0], b0, f32x16{}, 0, 0, 0,
                                                                     0x7f7f7f7f, 0, 0x7f7f7f7f);
          s = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[j][1], b1, s, 0, 0, 0, 0x7f7f7f7f,
                                                              0, 0x7f7f7f7f);
          const float f = sr * sc[j];
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][j][v] = __builtin_fmaf(s[v], f, acc[i][j][v]);
        }
      }
    }
  }
};

// Rows [first, first + rows) of the grouped buffers.
struct Group {
  int first, rows;
};

__device__ __forceinline__ Group group_of(const Groups& g, int e) {
  if (!g.off) return Group{(int)(e * g.cap), (int)g.cap};
  const int d = e / g.L, j = e - d * g.L;
  const int32_t* off = g.off + (size_t)d * (g.L + 1) + j;
  const int64_t lo = off[0] < 0 ? 0 : off[0] < g.cap ? off[0] : g.cap;
  const int64_t hi = off[1] < lo ? lo : off[1] < g.cap ? off[1] : g.cap;
  return Group{(int)(d * g.cap + lo), (int)(hi - lo)};
}

// A tile of a group's rows: `rows` of them from the group's `at`-th on, and
// the tile's column block.
struct Where {
  int expert, first, rows, at, col;
};

// The tile of this workgroup, among `cols` column blocks per block of BR rows;
// false: none is left. The tiles of the groups lie on a line that the eight
// XCDs (workgroup b runs on XCD b % 8) share in equal stretches, so that the
// workgroups beside each other in an L2 read the same rows and weights: a
// group's tiles go by stripes of eight column blocks, row blocks inside.
template <int BR, int THREADS>
__device__ __forceinline__ bool find_tile(const Groups& g, int cols, Where* out) {
  __shared__ int wave_sum[THREADS / kWave];
  __shared__ Where found;
  const int experts = g.N * g.L, tid = threadIdx.x, lane = lane_id();
  const int per = (experts + THREADS - 1) / THREADS;
  const int e0 = tid * per, e1 = e0 + per < experts ? e0 + per : experts;
  int mine = 0;
  for (int e = e0; e < e1; ++e) mine += (group_of(g, e).rows + BR - 1) / BR;
  int sum = mine;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int up = __shfl_up(sum, off);
    if (lane >= off) sum += up;
  }
  if (lane == kWave - 1) wave_sum[tid / kWave] = sum;
  __syncthreads();
  int before = sum - mine, total = 0;
  for (int w = 0; w < THREADS / kWave; ++w) {
    if (w < tid / kWave) before += wave_sum[w];
    total += wave_sum[w];
  }
  const int64_t tiles = (int64_t)total * cols;
  const int64_t stretch = (tiles + 7) / 8;
  const int64_t slot = blockIdx.x / 8, want = (int64_t)(blockIdx.x % 8) * stretch + slot;
  if (slot >= stretch || want >= tiles) return false;
  int64_t left = want - (int64_t)before * cols;
  if (left >= 0 && left < (int64_t)mine * cols) {
    for (int e = e0; e < e1; ++e) {
      const Group gr = group_of(g, e);
      const int blocks = (gr.rows + BR - 1) / BR;
      if (left >= (int64_t)blocks * cols) {
        left -= (int64_t)blocks * cols;
        continue;
      }
      const int at = (int)left, stripe = at / (blocks * 8);
      const int wide = cols - stripe * 8 < 8 ? cols - stripe * 8 : 8;
      const int in = at - stripe * blocks * 8, rb = in / wide;
      const int rows = gr.rows - rb * BR < BR ? gr.rows - rb * BR : BR;
      found = Where{e, gr.first + rb * BR, rows, rb * BR, stripe * 8 + in % wide};
      break;
    }
  }
  __syncthreads();
  *out = Where{wave_uniform(found.expert), wave_uniform(found.first), wave_uniform(found.rows),
               wave_uniform(found.at), wave_uniform(found.col)};
  return true;
}

// Workgroups that hold every tile that find_tile can name, given at most
// `most` rows in groups of `experts`; a multiple of 8.
inline int64_t tile_grid(const Groups& g, int br, int64_t cols) {
  const int64_t experts = (int64_t)g.N * g.L;
  int64_t blocks;
  if (!g.off)
    blocks = g.N * ((g.cap + br - 1) / br);
  else
    blocks = g.most / br + (experts < g.most ? experts : g.most);
  return (blocks * cols + 7) / 8 * 8;
}

__device__ __forceinline__ uint32_t lds_base(const void* p) {
  return (uint32_t)(uintptr_t)(const lds_u8*)p;
}

}  // namespace ep
