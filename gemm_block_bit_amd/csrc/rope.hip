// Rotary positions: alone (gbb_rope), and on the output of a fused q|k|v
// product with k and v written to a paged cache (gbb_rope_append).
//
// Pair i of a head (x1, x2) is turned by the angle of its token and pair:
//   y1 = x1 c - x2 s,  y2 = x2 c + x1 s,  (c, s) = table[position][i],
// 3 fp32 operations an element against 2 to 8 bytes moved: memory bound.
// The angles come from a table made in 64 bits, so that a position of 10^5
// keeps the accuracy that its product with a frequency in fp32 would lose;
// a token's row of the table (4 rot bytes) is read once per workgroup from
// memory and is small against the token's heads.
//
// Measured, a call among others: 8192 tokens of 64 / 8 heads of 128 (bf16)
// rotated and written to a cache 65 us, 5.2 TB/s; the transpose of 16384 tokens
// of 32 heads of 128 49 us, 5.5 TB/s, with one input and output or with eight
// in turn (2.1 GB, no cache holds them), where a copy of that size takes 50.6
// (5.3 TB/s).  Calls of up to about a hundred tokens take 2.4 to 3.5 us, a
// launch and two dependent reads.
#include <algorithm>

#include "rope_common.h"

namespace gbb {

namespace {

template <int DT, int E, int EC, bool HALF>
__global__ __launch_bounds__(1024) void rope_kernel(RopeArgs a, Units n, int hp, int tp) {
  typedef typename Elem<DT>::T T;
  const int nu = n.pairs + n.copies;
  const int u = threadIdx.x % nu, r = threadIdx.x / nu;
  const int h0 = r % hp, t = blockIdx.x * tp + r / hp;
  if (r / hp >= tp || t >= a.T) return;
  const int pos = a.positions[t];
  const bool there = unsigned(pos) < unsigned(a.n_pos);
  const T* x = static_cast<const T*>(a.x) + t * a.x_token;
  T* y = static_cast<T*>(a.y) + t * a.y_token;
  if (u >= n.pairs) {
    const int d = a.rot + (u - n.pairs) * EC;
    for (int h = blockIdx.y * hp + h0; h < a.H; h += gridDim.y * hp) {
      float v[EC];
      load_vec<T, EC>(x + h * a.x_head + d, v);
#pragma unroll
      for (int i = 0; i < EC; ++i) v[i] = there ? v[i] : 0.f;
      store_vec<T, EC>(y + h * a.y_head + d, v);
    }
    return;
  }
  Angles<E, HALF> g;
  g.load(a.table + size_t(there ? pos : 0) * a.rot, u, a.transpose ? -1.f : 1.f);
  for (int h = blockIdx.y * hp + h0; h < a.H; h += gridDim.y * hp) {
    const T* xh = x + h * a.x_head;
    T* yh = y + h * a.y_head;
    if constexpr (HALF) {
      float p[E], q[E], v[E], w[E];
      load_vec<T, E>(xh + u * E, p);
      load_vec<T, E>(xh + a.rot / 2 + u * E, q);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        v[i] = there ? p[i] * g.c[i] - q[i] * g.s[i] : 0.f;
        w[i] = there ? q[i] * g.c[i] + p[i] * g.s[i] : 0.f;
      }
      store_vec<T, E>(yh + u * E, v);
      store_vec<T, E>(yh + a.rot / 2 + u * E, w);
    } else {
      float p[E], v[E];
      load_vec<T, E>(xh + u * E, p);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        v[2 * i] = there ? p[2 * i] * g.c[i] - p[2 * i + 1] * g.s[i] : 0.f;
        v[2 * i + 1] = there ? p[2 * i + 1] * g.c[i] + p[2 * i] * g.s[i] : 0.f;
      }
      store_vec<T, E>(yh + u * E, v);
    }
  }
}

// The same units over the q, k and v heads of a token; v heads are copied,
// k and v go to the token's slot.  E = 8 where rot allows it, else 2.
template <int DT, int CT, int E, bool HALF>
__global__ __launch_bounds__(1024) void append_kernel(AppendArgs a, gbb_paged_cache c, Units n, int hp, int tp) {
  typedef typename Elem<DT>::T T;
  const int nu = n.pairs + n.copies;
  const int u = threadIdx.x % nu, r = threadIdx.x / nu;
  const int h0 = r % hp, t = blockIdx.x * tp + r / hp;
  if (r / hp >= tp || t >= a.T) return;
  const int D = c.head_dim, Hkv = c.kv_heads, H = a.Hq + 2 * Hkv;
  const int pos = a.positions[t], slot = a.slots[t];
  const bool there = unsigned(pos) < unsigned(a.n_pos) && unsigned(slot) < unsigned(c.num_pages) * unsigned(c.page);
  const T* x = static_cast<const T*>(a.qkv) + t * a.token_stride;
  const bool pair = u < n.pairs;
  const int d0 = !pair ? a.rot + (u - n.pairs) * E : u * E, d1 = a.rot / 2 + u * E;
  Angles<E, HALF> g;
  if (pair) g.load(a.table + size_t(there ? pos : 0) * a.rot, u, 1.f);
  // slots are below 2^31, pages times heads times rows may not be
  const int page = there ? slot / c.page : 0, off = there ? slot % c.page : 0;
  for (int h = blockIdx.y * hp + h0; h < H; h += gridDim.y * hp) {
    const T* xh = x + size_t(h) * D;
    float p[E], q[E];
    load_vec<T, E>(xh + d0, p);
    if (HALF && pair) load_vec<T, E>(xh + d1, q);
    if (pair && h < a.Hq + Hkv) {
      if constexpr (HALF) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float v = p[i] * g.c[i] - q[i] * g.s[i];
          q[i] = q[i] * g.c[i] + p[i] * g.s[i];
          p[i] = v;
        }
      } else {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          const float v = p[2 * i] * g.c[i] - p[2 * i + 1] * g.s[i];
          p[2 * i + 1] = p[2 * i + 1] * g.c[i] + p[2 * i] * g.s[i];
          p[2 * i] = v;
        }
      }
    }
    if (h < a.Hq) {
      T* y = static_cast<T*>(a.q) + (size_t(t) * a.Hq + h) * D;
      if (!there) {
#pragma unroll
        for (int i = 0; i < E; ++i) p[i] = q[i] = 0.f;
      }
      store_vec<T, E>(y + d0, p);
      if (HALF && pair) store_vec<T, E>(y + d1, q);
    } else if (there) {
      const bool key = h < a.Hq + Hkv;
      const int hk = key ? h - a.Hq : h - a.Hq - Hkv;
      const size_t row = (size_t(page) * Hkv + hk) * c.page + off;
      const float* sc = key ? c.k_scale : c.v_scale;
      const float scale = CT == GBB_E4M3 && sc ? sc[hk] : 1.f;
      void* base = key ? c.k : c.v;
      store_cache<CT, E>(base, row * D + d0, p, scale);
      if (HALF && pair) store_cache<CT, E>(base, row * D + d1, q, scale);
      if (key && u == 0) {
        if (c.positions) c.positions[row] = pos;
        if (c.weights) c.weights[row] = 0.f;
      }
    }
  }
}

// Threads and grid for T tokens of H heads of nu units: hp heads and tp
// tokens per workgroup of up to 256 threads (1024 where one head has more
// units), and as many workgroups along the heads as the chip has room for:
// with few tokens every head gets its own, with many a thread keeps its
// angles over several heads.
struct Shape {
  int hp, tp, threads;
  dim3 grid;
};
Shape shape(int T, int H, int nu) {
  Shape s;
  s.hp = nu >= 256 ? 1 : 256 / nu;
  s.tp = 1;
  if (s.hp > H) {
    s.tp = s.hp / H;
    s.hp = H;
  }
  s.threads = s.hp * s.tp * nu;
  const int gx = (T + s.tp - 1) / s.tp, most = (H + s.hp - 1) / s.hp;
  const int gy = std::max(1, std::min(most, 4 * device_compute_units() / gx));
  s.grid = dim3(unsigned(gx), unsigned(gy));
  return s;
}

template <int DT, int E, int EC>
void run_rope(const RopeArgs& a, hipStream_t s) {
  const Units n = units(a.D, a.rot, a.layout, E, EC);
  const Shape g = shape(a.T, a.H, n.pairs + n.copies);
  if (a.layout == GBB_ROPE_HALF)
    start((rope_kernel<DT, E, EC, true>), g.grid, dim3(g.threads), s, a, n, g.hp, g.tp);
  else if constexpr (E > 1)
    start((rope_kernel<DT, E, EC, false>), g.grid, dim3(g.threads), s, a, n, g.hp, g.tp);
}
template <int DT>
void run_widths(const RopeArgs& a, int E, int EC, hipStream_t s) {
  constexpr int W = DT == GBB_F32 ? 4 : 8;   // elements of 16 bytes
  if constexpr (W == 8)
    if (E == 8) return run_rope<DT, 8, 8>(a, s);
  if (E == 4) return EC == 8 && W == 8 ? run_rope<DT, 4, W>(a, s) : run_rope<DT, 4, 4>(a, s);
  if (E == 2) return EC == W ? run_rope<DT, 2, W>(a, s) : EC == 4 ? run_rope<DT, 2, 4>(a, s) : run_rope<DT, 2, 2>(a, s);
  return EC == W ? run_rope<DT, 1, W>(a, s) : EC == 4 ? run_rope<DT, 1, 4>(a, s) : EC == 2 ? run_rope<DT, 1, 2>(a, s) : run_rope<DT, 1, 1>(a, s);
}

template <int DT, int CT>
void run_append(const gbb_paged_cache& c, const AppendArgs& a, hipStream_t s) {
  const bool half = a.layout == GBB_ROPE_HALF;
  const bool wide = (half ? a.rot / 2 : a.rot) % 8 == 0;
  const int E = wide ? 8 : half ? 1 : 2;
  const Units n = units(c.head_dim, a.rot, a.layout, E, E);
  const Shape g = shape(a.T, a.Hq + 2 * c.kv_heads, n.pairs + n.copies);
  if (wide && half)
    start((append_kernel<DT, CT, 8, true>), g.grid, dim3(g.threads), s, a, c, n, g.hp, g.tp);
  else if (wide)
    start((append_kernel<DT, CT, 8, false>), g.grid, dim3(g.threads), s, a, c, n, g.hp, g.tp);
  else if (half)
    start((append_kernel<DT, CT, 1, true>), g.grid, dim3(g.threads), s, a, c, n, g.hp, g.tp);
  else
    start((append_kernel<DT, CT, 2, false>), g.grid, dim3(g.threads), s, a, c, n, g.hp, g.tp);
}

}  // namespace

int launch_rope(const RopeArgs& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int es = a.dtype == GBB_F32 ? 4 : 2;
  const int run = a.layout == GBB_ROPE_HALF ? a.rot / 2 : a.rot;
  // the widest unit (16 bytes at most) that divides the head's parts and
  // that every address and stride is a multiple of
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                        uintptr_t(a.x_token * es) | uintptr_t(a.x_head * es) | uintptr_t(a.y_token * es) |
                        uintptr_t(a.y_head * es);
  const bool half = a.layout == GBB_ROPE_HALF;
  int E = 16 / es;
  while (E > (half ? 1 : 2) && (run % E || all % uintptr_t(E * es))) E /= 2;
  // and the widest copies (16384 tokens of 32 heads of 96, 24
  // rotated in halves: 54 us, 67 with copies as narrow as the pairs)
  const int rest = a.D - a.rot;
  int EC = 16 / es;
  while (EC > E && (rest % EC || (all | uintptr_t(a.rot * es)) % uintptr_t(EC * es))) EC /= 2;
  while (E > (half ? 1 : 2) && (rest % E || uintptr_t(a.rot * es) % uintptr_t(E * es)) && EC <= E) E /= 2, EC = E;
  if (a.dtype == GBB_F32) run_widths<GBB_F32>(a, E, EC, s);
  else if (a.dtype == GBB_BF16) run_widths<GBB_BF16>(a, E, EC, s);
  else run_widths<GBB_F16>(a, E, EC, s);
  return int(hipGetLastError());
}

int launch_append(const gbb_paged_cache& c, const AppendArgs& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.dtype == GBB_F16) {
    if (c.dtype == GBB_E4M3) run_append<GBB_F16, GBB_E4M3>(c, a, s);
    else run_append<GBB_F16, GBB_F16>(c, a, s);
  } else {
    if (c.dtype == GBB_E4M3) run_append<GBB_BF16, GBB_E4M3>(c, a, s);
    else run_append<GBB_BF16, GBB_BF16>(c, a, s);
  }
  return int(hipGetLastError());
}

}  // namespace gbb
