// Element types of the attention operators: loads to and stores from f32 (not installed).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tq2 {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));

struct F32 {
  typedef float elem;
};
struct F16 {
  typedef _Float16 elem;
};
struct BF16 {
  typedef __bf16 elem;
};
struct E4M3 {
  typedef uint8_t elem;
};

__device__ __forceinline__ f32x4_t load4(F32, const float* p) {
  return *reinterpret_cast<const f32x4_t*>(p);
}
__device__ __forceinline__ f32x4_t load4(F16, const _Float16* p) {
  return __builtin_convertvector(*reinterpret_cast<const f16x4_t*>(p), f32x4_t);
}
__device__ __forceinline__ f32x4_t load4(BF16, const __bf16* p) {
  const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p);
  return f32x4_t{__builtin_bit_cast(float, w[0] << 16), __builtin_bit_cast(float, w[0] & 0xFFFF0000u),
                 __builtin_bit_cast(float, w[1] << 16), __builtin_bit_cast(float, w[1] & 0xFFFF0000u)};
}

// Each rounds to nearest, ties to even.
__device__ __forceinline__ void store4(F32, float* p, f32x4_t x) {
  *reinterpret_cast<f32x4_t*>(p) = x;
}
__device__ __forceinline__ void store4(F16, _Float16* p, f32x4_t x) {
  *reinterpret_cast<f16x4_t*>(p) = __builtin_convertvector(x, f16x4_t);
}
__device__ __forceinline__ void store4(BF16, __bf16* p, f32x4_t x) {
  *reinterpret_cast<bf16x4_t*>(p) = __builtin_convertvector(x, bf16x4_t);
}
// Beyond the largest finite e4m3, 448, values are clamped; NaN stays NaN.
__device__ __forceinline__ float clamp_e4m3(float x) {
  return x > 448.f ? 448.f : (x < -448.f ? -448.f : x);
}
__device__ __forceinline__ void store4(E4M3, uint8_t* p, f32x4_t x) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(x[0]), clamp_e4m3(x[1]), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(x[2]), clamp_e4m3(x[3]), w, true);
  *reinterpret_cast<uint32_t*>(p) = uint32_t(w);
}

}  // namespace tq2
