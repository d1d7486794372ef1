// Element types of the row operators (bf16, fp16, fp32), eight values at a time.
#pragma once

#include "common.hpp"

namespace moe {

enum ElemType { T_BF16 = 0, T_FP16 = 1, T_FP32 = 2 };  // moe_dtype

__host__ __device__ constexpr int elem_size(int t) { return t == T_FP32 ? 4 : 2; }

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// 8 consecutive values starting at element i (16-byte aligned), as fp32.
template <int DT>
__device__ __forceinline__ void load8(const void* base, size_t i, float (&v)[8]) {
  if constexpr (DT == T_FP32) {
    const f32x4 a = *(const f32x4*)((const float*)base + i), b = *(const f32x4*)((const float*)base + i + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  } else if constexpr (DT == T_FP16) {
    const f16x8 a = *(const f16x8*)((const _Float16*)base + i);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)a[j];
  } else {
    const u32x4 a = *(const u32x4*)((const uint16_t*)base + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_bits_to_f32(a[j] & 0xffffu);
      v[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
    }
  }
}

// v rounded to the type (to nearest, ties to even) and back.
template <int DT>
__device__ __forceinline__ float round_to(float v) {
  if constexpr (DT == T_FP32) return v;
  else if constexpr (DT == T_FP16) return (float)(_Float16)v;
  else return (float)(__bf16)v;
}

template <int DT>
__device__ __forceinline__ void store8(void* base, size_t i, const float (&v)[8]) {
  if constexpr (DT == T_FP32) {
    *(f32x4*)((float*)base + i) = f32x4{v[0], v[1], v[2], v[3]};
    *(f32x4*)((float*)base + i + 4) = f32x4{v[4], v[5], v[6], v[7]};
  } else if constexpr (DT == T_FP16) {
    f16x8 a;
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = (_Float16)v[j];
    *(f16x8*)((_Float16*)base + i) = a;
  } else {
    bf16x8 a;
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = (__bf16)v[j];
    *(bf16x8*)((uint16_t*)base + i) = a;
  }
}

// the same with the type known at run time only
__device__ __forceinline__ void load8_as(int dt, const void* base, size_t i, float (&v)[8]) {
  if (dt == T_BF16) load8<T_BF16>(base, i, v);
  else if (dt == T_FP16) load8<T_FP16>(base, i, v);
  else load8<T_FP32>(base, i, v);
}

}  // namespace moe
