// What the two attention kernels share (not installed).
#pragma once

#include "tq2_attn_internal.h"
#include "tq2_device.h"
#include "tq2_types.h"

namespace tq2 {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr float kNone = -__builtin_inff();

__device__ __forceinline__ f32x4_t mfma(F16, u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mfma(BF16, u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

__device__ __forceinline__ f32x16_t mfma(F16, u32x4_t a, u32x4_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a),
                                                __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mfma(BF16, u32x4_t a, u32x4_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack2(F16, float a, float b) {
  typedef _Float16 v2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, v2{_Float16(a), _Float16(b)});
}
__device__ __forceinline__ uint32_t pack2(BF16, float a, float b) {
  typedef __bf16 v2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, v2{__bf16(a), __bf16(b)});
}
// What rounding a and b to the type leaves, in the type.
__device__ __forceinline__ uint32_t pack2_rest(F16, float a, float b) {
  return pack2(F16(), a - float(_Float16(a)), b - float(_Float16(b)));
}
__device__ __forceinline__ uint32_t pack2_rest(BF16, float a, float b) {
  return pack2(BF16(), a - float(__bf16(a)), b - float(__bf16(b)));
}

// Two e4m3 codes (half `hi` of the word) as two 16-bit values, exactly.
template <bool hi>
__device__ __forceinline__ uint32_t widen2(F16, uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, hi));
}
template <bool hi>
__device__ __forceinline__ uint32_t widen2(BF16, uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, hi));
}

__device__ __forceinline__ float word(uint32_t w) { return __builtin_bit_cast(float, w); }
__device__ __forceinline__ uint32_t word(float v) { return __builtin_bit_cast(uint32_t, v); }

// v of the lane's place in the lower and upper half of the wave, and in the
// even and odd 16-lane groups.  (A bit cast takes no vector element itself: the
// compiler would read element 0.)
__device__ __forceinline__ float2 halves32(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(word(v), word(v), false, false);
  const uint32_t x = a[0], y = a[1];
  return float2{word(x), word(y)};
}
__device__ __forceinline__ float2 halves16(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(word(v), word(v), false, false);
  const uint32_t x = a[0], y = a[1];
  return float2{word(x), word(y)};
}

// Types of the two products.
template <class Act, class Cache>
struct Kinds {
  typedef F16 QK;
  typedef F16 PV;
};
template <class Cache>
struct Kinds<BF16, Cache> {
  typedef BF16 QK;
  typedef F16 PV;
};
template <>
struct Kinds<BF16, BF16> {
  typedef BF16 QK;
  typedef BF16 PV;
};

// A buffer resource that the compiler keeps in scalar registers.
__device__ __forceinline__ rsrc_t uniform_rsrc(const void* base, uint32_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(at)), hi = __builtin_amdgcn_readfirstlane(uint32_t(at >> 32));
  return make_rsrc(reinterpret_cast<const void*>(uint64_t(hi) << 32 | lo), __builtin_amdgcn_readfirstlane(bytes));
}

}  // namespace tq2
