// 16-bit values and their matrix instructions (gfx950), for the experts' kernels.
#ifndef MRS_HALF_H_
#define MRS_HALF_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));  // any element's address
typedef uint32_t u32x4_f32 __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct BF16 {
  typedef __bf16 T;
  static __device__ __forceinline__ float lo(uint32_t p) { return __uint_as_float(p << 16); }
  static __device__ __forceinline__ float hi(uint32_t p) { return __uint_as_float(p & 0xFFFF0000u); }
  // two FP32 values rounded to nearest even (a NaN stays one), the first in the low half
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
  }
  static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
  }
  static __device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c, false);
  }
};

struct FP16 {
  typedef _Float16 T;
  static __device__ __forceinline__ float lo(uint32_t p) { return (float)__builtin_bit_cast(f16x2, p)[0]; }
  static __device__ __forceinline__ float hi(uint32_t p) { return (float)__builtin_bit_cast(f16x2, p)[1]; }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const f16x2 v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, v);
  }
  static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, a), __builtin_bit_cast(f16x2, b), c, false);
  }
};

// The first n (up to seven) of eight 16-bit values, the others zero.
__device__ __forceinline__ u32x4 load_few(const uint16_t* p, int n) {
  uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) v[i / 2] |= (uint32_t)p[i] << (i % 2 * 16);
  return u32x4{v[0], v[1], v[2], v[3]};
}

// The eight values without the first n (n >= 0), zeros behind them.
__device__ __forceinline__ u32x4 drop(u32x4 v, int n) {
  if (n & 4) v = u32x4{v[2], v[3], 0u, 0u};
  if (n & 2) v = u32x4{v[1], v[2], v[3], 0u};
  if (n & 1) v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
  return n < 8 ? v : u32x4{0u, 0u, 0u, 0u};
}

// Eight consecutive 16-bit values at any element's address, zeros past the first n.
__device__ __forceinline__ u32x4 load8(const uint16_t* p, int n) {
  return n >= 8 ? *reinterpret_cast<const u32x4_any*>(p) : load_few(p, n);
}

// The first n of eight values, at any element's address.
__device__ __forceinline__ void store8(uint16_t* p, u32x4 v, int n) {
  if (n >= 8) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = (uint16_t)(v[i / 2] >> (i % 2 * 16));
  }
}

static inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

#endif  // MRS_HALF_H_
