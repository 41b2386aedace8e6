// Loads and stores of 8 consecutive elements of any of the floating types as
// fp32 values (NT: nontemporal).
#pragma once

#include "common.h"

namespace moeq {

template <bool NT>
__device__ __forceinline__ u32x4 ld16_nt(const void* p) {
  if (NT) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  return ld16(p);
}
template <bool NT>
__device__ __forceinline__ void st16_nt(void* p, u32x4 v) {
  if (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
  else st16(p, v);
}

template <int YK, bool NT>
__device__ __forceinline__ void load8(const void* y, int64_t off, float v[8]) {
  if (YK == OUT_F32) {
    const float* p = static_cast<const float*>(y) + off;
    const v4f a = __builtin_bit_cast(v4f, ld16_nt<NT>(p)), b = __builtin_bit_cast(v4f, ld16_nt<NT>(p + 4));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  } else {
    const u32x4 q = ld16_nt<NT>(static_cast<const uint16_t*>(y) + off);
    const u32 w[4] = {q[0], q[1], q[2], q[3]};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (YK == OUT_BF16) {
        v[2 * j] = bf16_bits_to_f32(w[j] & 0xffffu);
        v[2 * j + 1] = bf16_bits_to_f32(w[j] >> 16);
      } else {
        v[2 * j] = f16_bits_to_f32((uint16_t)(w[j] & 0xffffu));
        v[2 * j + 1] = f16_bits_to_f32((uint16_t)(w[j] >> 16));
      }
    }
  }
}

template <int OK, bool NT>
__device__ __forceinline__ void store8(void* out, int64_t off, const float v[8]) {
  if (OK == OUT_F32) {
    float* p = static_cast<float*>(out) + off;
    st16_nt<NT>(p, __builtin_bit_cast(u32x4, v4f{v[0], v[1], v[2], v[3]}));
    st16_nt<NT>(p + 4, __builtin_bit_cast(u32x4, v4f{v[4], v[5], v[6], v[7]}));
  } else {
    u32 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = (u32)OutT<OK>::from(v[2 * j]) | ((u32)OutT<OK>::from(v[2 * j + 1]) << 16);
    st16_nt<NT>(static_cast<uint16_t*>(out) + off, u32x4{w[0], w[1], w[2], w[3]});
  }
}

}  // namespace moeq
