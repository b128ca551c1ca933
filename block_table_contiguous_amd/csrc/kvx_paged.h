// Device helpers shared by the kernels that compute on a paged cache.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvx_attention.h"

namespace kvx {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Element types. Conversions from 32 bits round to nearest even (v_cvt_pk_bf16_f32 and
// v_cvt_pkrtz's exact sibling v_cvt_f16_f32), NaN stays NaN.
struct Bf16 {
  typedef __bf16 T;
  typedef __bf16 V4 __attribute__((ext_vector_type(4)));
  typedef __bf16 V8 __attribute__((ext_vector_type(8)));
};
struct Fp16 {
  typedef _Float16 T;
  typedef _Float16 V4 __attribute__((ext_vector_type(4)));
  typedef _Float16 V8 __attribute__((ext_vector_type(8)));
};

template <class E>
__device__ __forceinline__ f32x8 widen(u32x4 v) {
  return __builtin_convertvector(__builtin_bit_cast(typename E::V8, v), f32x8);
}
template <class E>
__device__ __forceinline__ u32x4 narrow(f32x8 v) {
  return __builtin_bit_cast(u32x4, __builtin_convertvector(v, typename E::V8));
}

// Global-memory accesses: address space 1, so that none becomes a flat instruction.
template <class T>
__device__ __forceinline__ T gload(const void* p) {
  return *(const __attribute__((address_space(1))) T*)p;
}
template <class T>
__device__ __forceinline__ void gstore(void* p, T v) {
  *(__attribute__((address_space(1))) T*)p = v;
}

__device__ __forceinline__ void raise(int32_t* err, int32_t bits) {
  if (err) atomicOr(err, bits);
}

// Division of slots by the block size: a shift where it is a power of two (the usual 16), the
// 32-bit division otherwise.
struct BlockDiv {
  int32_t size, shift;  // shift < 0: not a power of two
};
inline BlockDiv block_div(int32_t size) {
  return {size, (size & (size - 1)) == 0 ? __builtin_ctz((unsigned)size) : -1};
}
__device__ __forceinline__ int32_t block_of(BlockDiv d, int32_t slot) {
  return d.shift >= 0 ? (int32_t)((uint32_t)slot >> d.shift) : (int32_t)((uint32_t)slot / (uint32_t)d.size);
}

}  // namespace kvx
