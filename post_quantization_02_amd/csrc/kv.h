// What the kernels of the 4-bit paged key/value cache share: their operands as
// they see them, and typed loads and stores of eight values.
#pragma once

#include <hip/hip_runtime.h>

#include "kronq_internal.h"
#include "kv_index.h"

namespace kronq {

struct RopeView {
  const float *cos, *sin;
  int64_t ld;
  int positions;
  int half;                // dim / 2; 0: no rotation
  int neighbours;
};

struct HeadsView {
  void* data;
  int64_t row, head;       // strides in elements
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// for LDS that is written in other units than it is read in
typedef uint16_t u16_alias __attribute__((may_alias));
typedef uint32_t u32_alias __attribute__((may_alias));
typedef uint32_t u32x2_alias __attribute__((ext_vector_type(2), may_alias));
typedef uint32_t u32x4_alias __attribute__((ext_vector_type(4), may_alias));
typedef float f32x4_alias __attribute__((ext_vector_type(4), may_alias));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));

struct bf16_t { uint16_t bits; };

__device__ inline uint16_t to_bf16(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }

// eight consecutive values, 16-byte aligned
__device__ inline void load8(const float* p, float* x) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
}
__device__ inline void load8(const bf16_t* p, float* x) {
  const u32x4 a = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(a[i] << 16);
    x[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
  }
}
__device__ inline void load8(const _Float16* p, float* x) {
  const half8_t a = *reinterpret_cast<const half8_t*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (float)a[i];
}

__device__ inline void store8(float* p, const float* x) {
  *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
}
__device__ inline void store8(bf16_t* p, const float* x) {
  u32x4 a;
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = to_bf16(x[2 * i]) | ((uint32_t)to_bf16(x[2 * i + 1]) << 16);
  *reinterpret_cast<u32x4*>(p) = a;
}
__device__ inline void store8(_Float16* p, const float* x) {
  half8_t a;
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = (_Float16)x[i];
  *reinterpret_cast<half8_t*>(p) = a;
}

// four consecutive values, aligned to four
__device__ inline void store4(float* p, const float* x) {
  *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
}
__device__ inline void store4(bf16_t* p, const float* x) {
  *reinterpret_cast<u32x2*>(p) = u32x2{to_bf16(x[0]) | ((uint32_t)to_bf16(x[1]) << 16),
                                       to_bf16(x[2]) | ((uint32_t)to_bf16(x[3]) << 16)};
}
__device__ inline void store4(_Float16* p, const float* x) {
  typedef _Float16 half4 __attribute__((ext_vector_type(4)));
  *reinterpret_cast<half4*>(p) = half4{(_Float16)x[0], (_Float16)x[1], (_Float16)x[2], (_Float16)x[3]};
}

// The value of another lane of a group of eight or sixteen: its partner in step
// `CTRL` of a reduction (DPP: exchanged pairs, halves of four, of eight, of sixteen lanes).
template <int CTRL>
__device__ inline float partner(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ inline double partner(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_mov_dpp((int)b, CTRL, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

}  // namespace kronq
