// Device helpers of the kernels that read or write a paged KV cache: rows of
// new tokens, page lookups and the number formats of the cache.
#pragma once

#include "ep.h"
#include "ep_device.hpp"

namespace ep {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Types by their EP_DTYPE_* code.
template <int DT>
struct Fmt;

template <>
struct Fmt<EP_DTYPE_BF16> {
  typedef __bf16 elem;
  typedef bf16x8 vec8;
  static constexpr int bytes = 2;
};
template <>
struct Fmt<EP_DTYPE_F16> {
  typedef _Float16 elem;
  typedef f16x8 vec8;
  static constexpr int bytes = 2;
};
template <>
struct Fmt<EP_DTYPE_E4M3> {
  static constexpr int bytes = 1;
};

template <typename V, typename S>
__device__ __forceinline__ V as(const S& s) {
  static_assert(sizeof(V) == sizeof(S), "sizes differ");
  return __builtin_bit_cast(V, s);
}

// The nearest e4m3 code of f, saturating at 448; a NaN stays one.
__device__ __forceinline__ float e4m3_range(float f) {
  return f != f ? f : __builtin_amdgcn_fmed3f(f, -448.0f, 448.0f);
}

template <int DT>
__device__ __forceinline__ void store8(uint8_t* p, const float* f) {
  if constexpr (DT == EP_DTYPE_E4M3) {
    u32x2 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int c = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_range(f[4 * i]), e4m3_range(f[4 * i + 1]), 0,
                                              false);
      c = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_range(f[4 * i + 2]), e4m3_range(f[4 * i + 3]), c,
                                          true);
      w[i] = (uint32_t)c;
    }
    *(u32x2*)p = w;
  } else {
    typename Fmt<DT>::vec8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (typename Fmt<DT>::elem)f[i];
    *(u32x4*)p = as<u32x4>(v);
  }
}

template <int DT>
__device__ __forceinline__ float load1(const uint8_t* p) {
  if constexpr (DT == EP_DTYPE_E4M3)
    return __builtin_amdgcn_cvt_f32_fp8((int)*p, 0);
  else
    return (float)*(const typename Fmt<DT>::elem*)p;
}

template <int DT>
__device__ __forceinline__ void store1(uint8_t* p, float f) {
  if constexpr (DT == EP_DTYPE_E4M3)
    *p = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(e4m3_range(f), 0.0f, 0, false);
  else
    *(typename Fmt<DT>::elem*)p = (typename Fmt<DT>::elem)f;
}

// The sequence of row i < n_tokens (every lane of the wave has the same i):
// the last one that starts at or before it, or -1 when the row lies outside
// every sequence. 64 candidates per round; the range shrinks every round, so
// the search ends for any contents of q_off.
__device__ __forceinline__ int seq_of_row(const ep_kv_batch& b, int i) {
  if (!b.q_off) return i < b.n_seqs ? i : -1;
  int lo = 0, hi = b.n_seqs;  // the answer lies in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + kWave - 1) / kWave;
    const int j = lo + lane_id() * step;
    const uint64_t mask = ballot(j < hi && b.q_off[j < hi ? j : lo] <= i);
    if (mask == 0) return -1;
    lo += (kWave - 1 - __builtin_clzll(mask)) * step;
    hi = hi < lo + step ? hi : lo + step;
  }
  if (lo >= b.n_seqs) return -1;
  return b.q_off[lo] <= i && i < b.q_off[lo + 1] ? lo : -1;
}

}  // namespace ep
