// half.hpp - 16-bit element types of queries, keys and values (bf16 and f16): eight
// elements per 16-byte word, widened to fp32 and rounded back to nearest-even.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/smcsd.h"

namespace smcsd {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int DT> struct Half;
template <> struct Half<SMCSD_DTYPE_BF16> {
  typedef __bf16 T;
  typedef __bf16 V4 __attribute__((ext_vector_type(4)));
  typedef __bf16 V8 __attribute__((ext_vector_type(8)));
};
template <> struct Half<SMCSD_DTYPE_F16> {
  typedef _Float16 T;
  typedef _Float16 V4 __attribute__((ext_vector_type(4)));
  typedef _Float16 V8 __attribute__((ext_vector_type(8)));
};

template <int DT>
__device__ __forceinline__ f32x8 widen8(uint4 w) {
  return __builtin_convertvector(__builtin_bit_cast(typename Half<DT>::V8, w), f32x8);
}
template <int DT>
__device__ __forceinline__ uint4 narrow8(f32x8 x) {
  return __builtin_bit_cast(uint4, __builtin_convertvector(x, typename Half<DT>::V8));
}

}  // namespace smcsd
