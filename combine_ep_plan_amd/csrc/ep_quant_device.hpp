// Block-fp8 quantisation of values in registers, shared by the quantising
// sender and the norm that writes the dispatch's planes.
#pragma once

#include "ep_device.hpp"

namespace ep {

// OCP e4m3fn code of q (|q| <= 448), round to nearest, ties to even. For
// |q| >= 2^-6 with 2^E <= |q| < 2^(E+1): N = rne(|q| * 2^(3-E)) in [8, 16],
// code = (E + 6) * 8 + N (N = 16 carries into the next exponent). Below 2^-6
// (subnormals): code = rne(|q| * 2^9) in [0, 8]. Both scalings are by powers
// of two, so exact.
__device__ __forceinline__ uint32_t f32_to_e4m3(float q) {
  const uint32_t bits = __float_as_uint(q);
  const uint32_t sign = (bits >> 24) & 0x80u;
  const float a = __uint_as_float(bits & 0x7fffffffu);
  uint32_t code;
  if (a < 0.015625f) {
    code = (uint32_t)__builtin_rintf(a * 512.0f);
  } else {
    const int E = (int)((bits >> 23) & 0xffu) - 127;
    const float scaled = a * __uint_as_float((uint32_t)(127 + 3 - E) << 23);
    code = (uint32_t)((E + 6) * 8) + (uint32_t)__builtin_rintf(scaled);
  }
  return sign | code;
}

// Codes and scale of one step (8 values per lane, 16 lanes per block).
//
// Fast path: y = 1 / scale once per block (IEEE division), then per value
// q0 = |x| y and one correction q = q0 + (|x| - scale q0) y (two FMAs; the
// residual is exact), clamped to 448, signed by x, and encoded by the
// hardware conversion, which equals f32_to_e4m3 on every |q| <= 448
// (tests/test_gpu_fp8_convert.py checks every such fp32 value). For a
// bf16 x and a bf16 block amax of at least 2^-96 this q gives the same e4m3
// code as the IEEE quotient x / scale: checked for every such pair (524.8 M
// of them) by tests/test_fp8_reciprocal.py, which runs these same operations
// on the CPU. For a 32-bit x, q is the rounded quotient itself where nothing
// under- or overflows: y is the rounded reciprocal and q0 within two units of
// the quotient, so one exact residual corrects it. Everything else takes the exact path below for the whole wave:
// a smaller nonzero amax, an infinite amax, or a NaN anywhere in the step.
//
// Exact path: amax with NaN left out (a NaN never compares greater; an
// infinite value makes amax and the scale infinite), IEEE division per
// value, the software encoder; a NaN quotient (a NaN value, or an infinite
// one over its infinite scale) is the NaN code 0x7F, kept from the clamp,
// which would turn it into -448.
__device__ __forceinline__ void quantise_values(const float (&v)[8], uint32_t packed[2],
                                                float& scale_out) {
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
  // Over the block's 16 lanes (one DPP row): the maximum of non-negative
  // floats is the maximum of their bit patterns, and a NaN stays the largest.
  uint32_t ab = __float_as_uint(amax);
  ab = max(ab, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)ab, 0xB1, 0xF, 0xF, false));   // lane ^ 1
  ab = max(ab, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)ab, 0x4E, 0xF, 0xF, false));   // lane ^ 2
  ab = max(ab, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)ab, 0x141, 0xF, 0xF, false));  // half-row mirror
  ab = max(ab, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)ab, 0x140, 0xF, 0xF, false));  // row mirror
  amax = __uint_as_float(ab);
  float scale = amax > 0.0f ? amax / 448.0f : 1.0f;
  const float y = 1.0f / scale;
  uint32_t qmax = 0;
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a = fabsf(v[j]);
    const float q0 = a * y;
    const float q1 = __builtin_fmaf(__builtin_fmaf(-scale, q0, a), y, q0);
    qmax = max(qmax, __float_as_uint(q1));
    q[j] = __builtin_copysignf(fminf(q1, 448.0f), v[j]);
  }
  int w0 = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  w0 = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w0, true);
  int w1 = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  w1 = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], w1, true);
  packed[0] = (uint32_t)w0;
  packed[1] = (uint32_t)w1;
  const bool exact = (amax > 0.0f && amax < 0x1p-96f) || !(amax < __builtin_inff()) ||
                     qmax > 0x7f800000u;
  if (ballot(exact)) {  // wave-uniform: the shuffles below need every lane
    amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = fabsf(v[j]);
      amax = a > amax ? a : amax;
    }
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 16));
    scale = amax > 0.0f ? amax / 448.0f : 1.0f;
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float qq = v[j] / scale;
      c[j] = __builtin_isnan(qq) ? 0x7Fu : f32_to_e4m3(fminf(fmaxf(qq, -448.0f), 448.0f));
    }
    packed[0] = c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24);
    packed[1] = c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24);
  }
  scale_out = scale;
}

}  // namespace ep
