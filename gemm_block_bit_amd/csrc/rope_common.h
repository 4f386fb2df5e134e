// Shared by the kernels that rotate heads (rope.hip, norm_rope.hip): element
// types, units of a head, angles, and the cache's conversion.
#pragma once
#include "device.h"
#include "internal.h"

namespace gbb {

typedef __bf16 bfloat;

template <int DT> struct Elem;
template <> struct Elem<GBB_F16> { typedef _Float16 T; };
template <> struct Elem<GBB_BF16> { typedef bfloat T; };
template <> struct Elem<GBB_F32> { typedef float T; };

// E elements at an address that the launcher has checked to be a multiple of
// E elements; E = 2 also serves pairs at odd addresses.
template <typename T, int E>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[E]) {
  struct alignas(sizeof(T) * (E == 2 ? 1 : E)) V { T v[E]; };
  const V r = *reinterpret_cast<const V*>(p);
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = float(r.v[i]);
}
template <typename T, int E>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[E]) {
  struct alignas(sizeof(T) * (E == 2 ? 1 : E)) V { T v[E]; };
  V r;
#pragma unroll
  for (int i = 0; i < E; ++i) r.v[i] = T(x[i]);
  *reinterpret_cast<V*>(p) = r;
}

// A head is E-element units: rot / 2 / E units of pairs in the half layout
// (unit u takes elements u E ... and rot/2 + u E ...), rot / E units in the
// interleaved one, then (D - rot) / EC units of EC elements that are copied.
struct Units {
  int pairs, copies;
};
__host__ __device__ __forceinline__ Units units(int D, int rot, int layout, int E, int EC) {
  return {(layout == GBB_ROPE_HALF ? rot / 2 : rot) / E, (D - rot) / EC};
}

// The table entries of unit u of the token's row: E pairs (half) or E / 2.
template <int E, bool HALF>
struct Angles {
  static constexpr int N = HALF ? E : E / 2;
  float c[N], s[N];
  __device__ __forceinline__ void load(const float* row, int u, float sign) {
    const float2* p = reinterpret_cast<const float2*>(row) + u * N;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 a = p[i];
      c[i] = a.x;
      s[i] = a.y * sign;
    }
  }
};

// Eight cache elements from fp32 values.  e4m3: value / scale, clamped to
// the format's range (the conversion itself would make a NaN of what is
// above it) and rounded to nearest even by the hardware conversion.
__device__ __forceinline__ uint32_t e4m3_pair2(const float* x, float scale) {
  float c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v = x[i] / scale;
    c[i] = v > 448.f ? 448.f : v < -448.f ? -448.f : v;   // a NaN passes both
  }
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w, true));
}
template <int CT, int E>
__device__ __forceinline__ void store_cache(void* base, size_t at, const float (&x)[E], float scale) {
  if constexpr (CT == GBB_E4M3) {
    uint8_t* p = static_cast<uint8_t*>(base) + at;
    if constexpr (E == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(e4m3_pair2(x, scale), e4m3_pair2(x + 4, scale));
    } else if constexpr (E == 4) {
      *reinterpret_cast<uint32_t*>(p) = e4m3_pair2(x, scale);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float one[4] = {x[i], 0.f, 0.f, 0.f};
        p[i] = uint8_t(e4m3_pair2(one, scale));
      }
    }
  } else {
    store_vec<typename Elem<CT>::T, E>(static_cast<typename Elem<CT>::T*>(base) + at, x);
  }
}

}  // namespace gbb
