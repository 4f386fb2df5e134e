// Shared by the attention kernels over a paged cache (attention.hip,
// tokens.hip): 16-bit element types and their matrix products, loads with a
// range, joins of partial results, and the shape of scores.
#pragma once
#include "device.h"
#include "internal.h"

namespace gbb {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// 16-bit element types of q, P and out.
template <int DT> struct Half;
typedef float f32x16 __attribute__((ext_vector_type(16)));
template <> struct Half<GBB_F16> {
  static constexpr int PARTS = 2;   // operands that P is given in
  typedef _Float16 T;
  typedef half8 V8;
  static __device__ __forceinline__ f32x4 mfma(const V8& a, const V8& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mfma32(const V8& a, const V8& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  // two e4m3 bytes (the low or the high pair of w) as two elements, exactly
  template <bool HI> static __device__ __forceinline__ uint32_t widen(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, HI));
  }
};
template <> struct Half<GBB_BF16> {
  static constexpr int PARTS = 3;
  typedef __bf16 T;
  typedef bf16x8 V8;
  static __device__ __forceinline__ f32x4 mfma(const V8& a, const V8& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mfma32(const V8& a, const V8& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  template <bool HI> static __device__ __forceinline__ uint32_t widen(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, HI));
  }
};

// `bytes` of memory from `base`; loads past them give zeros.
typedef __amdgpu_buffer_rsrc_t Span;
__device__ __forceinline__ Span span(const void* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00020000);   // raw bytes
}
// 16 bytes a lane, at byte `at` of s, to LDS at `to` (the same in all lanes)
// plus 16 bytes times the lane.  The compiler does not wait for such a load
// before LDS reads: loads_left<N>() waits until at most the N vector memory
// operations issued last are under way (they complete in order) and
// in_order() keeps the compiler from moving memory operations across it.
__device__ __forceinline__ void to_lds(Span s, int at, uint8_t* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(s, (__attribute__((address_space(3))) void*)to, 16, at, 0, 0, 0);
}
template <int N>
__device__ __forceinline__ void loads_left() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void in_order() { asm volatile("" ::: "memory"); }

// 2^(x - m) with 2^(-inf - -inf) = 0, for joining partial results
__device__ __forceinline__ float rescale(float x, float m) {
  return x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(x - m);
}

// Two floats at device scope.
__device__ __forceinline__ void put(float* p, float x, float y) {
  const uint64_t v = uint64_t(__builtin_bit_cast(uint32_t, y)) << 32 | __builtin_bit_cast(uint32_t, x);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 get(const float* p) {
  const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__builtin_bit_cast(float, uint32_t(v)), __builtin_bit_cast(float, uint32_t(v >> 32)));
}

// The capped score cap tanh(x / cap) in the log2 domain: x comes times
// log2(e), and so does the result; out = cap log2(e), over = 1 / out.  tanh(y) =
// 1 - 2 / (1 + e^2y) loses digits where y is small: its error is below 2^-22 of
// the cap.  Up to kShortCap that is at most 2e-5 of a score's exponential, below a
// hundredth of what rounding an output to 16 bits takes (lse has it in full; the series
// everywhere takes a capped prompt of 8192 from 907 to 1281 us, with two operands of
// P); above, and for single tokens at any cap, arguments below
// 0.35 take the series (its first term left out is below 2^-25 of the result).
constexpr float kShortCap = 80.f;
__device__ __forceinline__ float capped(float x, float over, float out) {
  const float y = x * over, y2 = y * y;
  const float t = __builtin_fmaf(-2.f * out, __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(y * (2.f * kLog2e)) + 1.f), out);
  const float p = y * out * (1.f + y2 * (-1.f / 3.f + y2 * (2.f / 15.f + y2 * (-17.f / 315.f + y2 * (62.f / 2835.f - y2 * (1382.f / 155925.f))))));
  return fabsf(y) < 0.35f ? p : t;
}

}  // namespace gbb
