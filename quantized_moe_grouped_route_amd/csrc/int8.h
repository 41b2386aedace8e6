// Symmetric 8- and 16-bit codes of fp32 values, shared by the INT8 kernels.
#pragma once

#include "common.h"

namespace moeq {

typedef int v2i_t __attribute__((ext_vector_type(2)));

// Bytes of one row of a gradient's plane: N up to whole 128-value stages.
__host__ __device__ __forceinline__ int plane_pitch(int N) { return (N + 127) / 128 * 128; }

// s = sig(g) = 1 / (1 + exp(-g)) and c = 1 - s = sig(-g), for values of type KIND.
// What is rounded to 16 bits takes the hardware's exp2 of a rounded product and
// its reciprocal: s is then off by up to (8 + 2 |g|) 2^-24 of itself, c by that of
// s: where g leaves fp32's range of exp, at 87, by 1.1e-5, a 45th of f16's half
// step.  f32 keeps its own bits: exp to 1 ulp, of -|g| so that neither s nor c is
// the difference of larger numbers, and a reciprocal made exact to its rounding by
// one Newton step (its argument lies in [1, 2]): 5 * 2^-24 of each.  f32, 4096
// rows of 2 x 14336, us, against the hardware's two instructions: h 137 for 137, h
// and checkpoint 169 for 167, gradient from the checkpoint 212 for 211, from the
// columns 240 for 231; gated product of 4096 rows, 8 x 28672 x 4096, 525 for 508
// (546 with an IEEE division).
struct Sigmoid {
  float s, c;
};
template <int KIND>
__device__ __forceinline__ Sigmoid sigmoid(float g) {
  if constexpr (KIND == OUT_F32) {
    const float e = expf(-__builtin_fabsf(g)), x = 1.0f + e, r = __builtin_amdgcn_rcpf(x);
    const float big = __builtin_fmaf(__builtin_fmaf(-x, r, 1.0f), r, r), small = e * big;
    return g < 0.0f ? Sigmoid{small, big} : Sigmoid{big, small};
  } else {
    const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
    return Sigmoid{s, 1.0f - s};
  }
}
template <int KIND>
__device__ __forceinline__ float silu(float g) {
  return g * sigmoid<KIND>(g).s;
}

// The fp32 value itself, rounded.  It keeps the compiler from merging a product
// with the conversion after it (one rounding where the kernels of other
// schedules and tile sizes make two): a row's bits then never depend on which
// of them computed it.
__device__ __forceinline__ float rounded(float v) {
  asm("" : "+v"(v));
  return v;
}

// Largest magnitude as fp32 bits: as integers, an infinity or NaN is above
// every finite value, so it is never lost in a maximum.
__device__ __forceinline__ u32 amax_bits(const float (&v)[8]) {
  u32 m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ u32 wave_max(u32 m) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = max(m, (u32)__shfl_xor((int)m, o, 64));
  return m;
}

// Scale of symmetric codes up to `top` for values of largest magnitude m, and
// the factor that makes codes of them: each one fp32 division.  m below
// `tiny`: scale 1, codes 0.  m an infinity or NaN: scale NaN, so what is made
// of the codes (then without meaning) shows it.
struct Scale {
  float scale, recip;
};
__device__ __forceinline__ Scale scale_of(u32 m_bits, float top, float tiny) {
  const float m = __uint_as_float(m_bits);
  if (m_bits >= 0x7f800000u) return Scale{__uint_as_float(0x7fc00000u), 0.0f};
  if (m < tiny) return Scale{1.0f, 0.0f};
  return Scale{m / top, top / m};
}
// rne(v * recip) within [-top, top].
__device__ __forceinline__ int code_of(float v, float recip, float top) {
  return (int)fminf(fmaxf(__builtin_rintf(v * recip), -top), top);
}

// int8 codes of 8 values, packed in order.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float recip) {
  u32 w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j >> 2] |= ((u32)code_of(v[j], recip, 127.0f) & 255u) << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}

}  // namespace moeq
