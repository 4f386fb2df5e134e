// Norms of q and k heads with rotary positions in the same pass: alone
// (gbb_norm_rope, and without the norm gbb_rope_axes), its gradient
// (gbb_norm_rope_grad), and on a fused q|k|v output on its way into a paged
// cache (gbb_norm_rope_append).  Positions have one to four axes.
//
// A head x of D elements becomes R(x r w) with r = (mean x^2 + eps)^(-1/2),
// w a weight an element and R the rotation of its first `rot` elements, whose
// pair i turns by the token's position on the axis that section i lies in.
// With g = R^T dy and xh = x r its gradient is
//   dw = sum over tokens and heads of g xh,
//   dx = r (g w - xh mean(g w xh)).
// 5 to 15 operations an element against 4 to 12 bytes moved: memory bound, so
// every element is read once and written once.  A head is spread over the
// lanes that hold it 16 bytes (in halves: twice 16) each, a power of two of
// them, so that its sums are a few lane exchanges and x, dy, angles and
// weights stay in registers from the sums to the store.  Heads too odd or long
// for one unit a lane go through the same steps unit by unit, x from the
// cache the second time.
//
// dw needs a sum over all heads: a workgroup keeps its own over the tokens it
// takes (in registers; fp32, at most some hundred terms each), writes it to
// the workspace, and a second launch adds the workgroups' in their order, so
// it is the same bits each time.
#include <algorithm>

#include "rope_common.h"

namespace gbb {

namespace {

// A token's place in the table: a row an axis.
struct Place {
  int row[4];
  bool there;
};
__device__ __forceinline__ Place place_of(const Rotation& r, int T, int t) {
  Place p;
  p.there = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pos = i < r.axes ? r.positions[size_t(i) * T + t] : 0;
    p.there = p.there && unsigned(pos) < unsigned(r.n_pos);
    p.row[i] = pos;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) p.row[i] = p.there ? p.row[i] : 0;
  return p;
}

// Angles of unit u, each pair's from the row of its own axis.
template <int E, bool HALF>
__device__ __forceinline__ void load_angles(Angles<E, HALF>& g, const Rotation& r, const Place& at, int u, float sign) {
  if (r.axes == 1) {
    g.load(r.table + size_t(at.row[0]) * r.rot, u, sign);
    return;
  }
#pragma unroll
  for (int i = 0; i < Angles<E, HALF>::N; ++i) {
    const int pair = u * Angles<E, HALF>::N + i;
    const int row = pair < r.end[0] ? at.row[0] : pair < r.end[1] ? at.row[1] : pair < r.end[2] ? at.row[2] : at.row[3];
    const float2 a = reinterpret_cast<const float2*>(r.table + size_t(row) * r.rot)[pair];
    g.c[i] = a.x;
    g.s[i] = a.y * sign;
  }
}

// Unit u of a head: N elements from d0 on and, of a pair in halves, N from d1.
template <int E, bool HALF>
struct Unit {
  bool there, pair, two;
  int d0, d1;
  __device__ __forceinline__ Unit(const Units& n, int rot, int u) {
    there = u < n.pairs + n.copies;
    pair = u < n.pairs;
    two = HALF && pair;
    d0 = pair ? u * E : rot + (u - n.pairs) * E;
    d1 = rot / 2 + u * E;
  }
  template <typename T>
  __device__ __forceinline__ void load(const T* x, float (&p)[E], float (&q)[E]) const {
#pragma unroll
    for (int i = 0; i < E; ++i) p[i] = q[i] = 0.f;
    if (there) load_vec<T, E>(x + d0, p);
    if (two) load_vec<T, E>(x + d1, q);
  }
  template <typename T>
  __device__ __forceinline__ void store(T* y, const float (&p)[E], const float (&q)[E]) const {
    if (there) store_vec<T, E>(y + d0, p);
    if (two) store_vec<T, E>(y + d1, q);
  }
  __device__ __forceinline__ void weights(const void* w, bool wide, int dtype, float (&p)[E], float (&q)[E]) const {
    if (!w) {
#pragma unroll
      for (int i = 0; i < E; ++i) p[i] = q[i] = 1.f;
    } else if (wide) {   // fp32
      load(static_cast<const float*>(w), p, q);
    } else if (dtype == GBB_F16) {
      load(static_cast<const _Float16*>(w), p, q);
    } else {
      load(static_cast<const bfloat*>(w), p, q);
    }
  }
};
template <int E, bool HALF>
__device__ __forceinline__ void turn(const Unit<E, HALF>& u, const Angles<E, HALF>& g, float (&p)[E], float (&q)[E]) {
  if (!u.pair) return;
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
template <int E>
__device__ __forceinline__ void clear(float (&p)[E], float (&q)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) p[i] = q[i] = 0.f;
}
// Sum over the `lanes` lanes (a power of two) of a head, the same in each.
__device__ __forceinline__ float over_head(float x, int lanes) {
  for (int i = 1; i < lanes; i *= 2) x += __shfl_xor(x, i);
  return x;
}
template <int E>
__device__ __forceinline__ float dot(const float (&p)[E], const float (&q)[E], const float (&v)[E], const float (&w)[E]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) s += p[i] * v[i];
#pragma unroll
  for (int i = 0; i < E; ++i) s += q[i] * w[i];
  return s;
}

// hp heads and tp tokens a workgroup, `lanes` lanes a head; ONE: every lane
// has one unit, else units l, l + lanes, ...
struct Spread {
  Units n;
  int lanes, hp, tp;
};

template <int DT, int E, bool HALF, bool ONE>
__global__ __launch_bounds__(256) void norm_rope_kernel(NormRopeArgs a, Spread s) {
  typedef typename Elem<DT>::T T;
  typedef Unit<E, HALF> U;
  const int l = threadIdx.x % s.lanes, r = threadIdx.x / s.lanes;
  const int h0 = r % s.hp, t = blockIdx.x * s.tp + r / s.hp;
  if (r / s.hp >= s.tp || t >= a.T) return;
  const Place at = place_of(a.r, a.T, t);
  const float sign = a.transpose ? -1.f : 1.f;
  const U first(s.n, a.r.rot, l);
  Angles<E, HALF> g;
  float w[E], v[E];
  if (ONE && first.pair) load_angles(g, a.r, at, l, sign);
  if (ONE) first.weights(a.weight, a.wide_weight, a.dtype, w, v);
  for (int h = blockIdx.y * s.hp + h0; h < a.H; h += gridDim.y * s.hp) {
    const T* x = static_cast<const T*>(a.x) + t * a.x_token + h * a.x_head;
    T* y = static_cast<T*>(a.y) + t * a.y_token + h * a.y_head;
    float p[E], q[E], scale = 1.f;
    if (ONE) first.load(x, p, q);
    if (a.norm) {
      float ss = 0.f;
      if (ONE) ss = dot(p, q, p, q);
      else for (int u = l; u < s.n.pairs + s.n.copies; u += s.lanes) {
        U(s.n, a.r.rot, u).load(x, p, q);
        ss += dot(p, q, p, q);
      }
      scale = rsqrtf(over_head(ss, s.lanes) / float(a.D) + a.eps);
    }
    for (int u = l; u < s.n.pairs + s.n.copies; u += s.lanes) {
      const U unit = ONE ? first : U(s.n, a.r.rot, u);
      if (!ONE) {
        if (unit.pair) load_angles(g, a.r, at, u, sign);
        unit.weights(a.weight, a.wide_weight, a.dtype, w, v);
        unit.load(x, p, q);
      }
      if (a.norm) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          p[i] = p[i] * scale * w[i];
          q[i] = q[i] * scale * v[i];
        }
      }
      turn(unit, g, p, q);
      if (!at.there) clear(p, q);
      unit.store(y, p, q);
      if (ONE) break;
    }
  }
}

// The same over the q, k and v heads of a token; v heads are copied, k and v
// go to the token's slot.
template <int DT, int CT, int E, bool HALF, bool ONE>
__global__ __launch_bounds__(256) void norm_append_kernel(NormAppendArgs a, gbb_paged_cache c, Spread s) {
  typedef typename Elem<DT>::T T;
  typedef Unit<E, HALF> U;
  const int l = threadIdx.x % s.lanes, r = threadIdx.x / s.lanes;
  const int h0 = r % s.hp, t = blockIdx.x * s.tp + r / s.hp;
  if (r / s.hp >= s.tp || t >= a.T) return;
  const int D = c.head_dim, Hkv = c.kv_heads, H = a.Hq + 2 * Hkv;
  const int slot = a.slots[t];
  Place at = place_of(a.r, a.T, t);
  const bool there = at.there && unsigned(slot) < unsigned(c.num_pages) * unsigned(c.page);
  const U first(s.n, a.r.rot, l);
  Angles<E, HALF> g;
  if (ONE && first.pair) load_angles(g, a.r, at, l, 1.f);
  // slots are below 2^31, pages times heads times rows may not be
  const int page = there ? slot / c.page : 0, off = there ? slot % c.page : 0;
  for (int h = blockIdx.y * s.hp + h0; h < H; h += gridDim.y * s.hp) {
    const T* x = static_cast<const T*>(a.qkv) + t * a.token_stride + size_t(h) * D;
    const bool query = h < a.Hq, value = h >= a.Hq + Hkv;
    float p[E], q[E], scale = 1.f;
    if (ONE) first.load(x, p, q);
    const bool norm = a.norm && !value;
    const void* weight = query ? a.q_weight : a.k_weight;
    if (norm) {   // the same for all lanes of a head
      float ss = 0.f;
      if (ONE) ss = dot(p, q, p, q);
      else for (int u = l; u < s.n.pairs + s.n.copies; u += s.lanes) {
        U(s.n, a.r.rot, u).load(x, p, q);
        ss += dot(p, q, p, q);
      }
      scale = rsqrtf(over_head(ss, s.lanes) / float(D) + a.eps);
    }
    const int hk = value ? h - a.Hq - Hkv : h - a.Hq;
    const size_t row = query ? 0 : (size_t(page) * Hkv + hk) * c.page + off;
    const float* scales = value ? c.v_scale : c.k_scale;
    const float element = CT == GBB_E4M3 && !query && scales ? scales[hk] : 1.f;
    for (int u = l; u < s.n.pairs + s.n.copies; u += s.lanes) {
      const U unit = ONE ? first : U(s.n, a.r.rot, u);
      if (!ONE) {
        if (unit.pair) load_angles(g, a.r, at, u, 1.f);
        unit.load(x, p, q);
      }
      if (norm) {
        float w[E], v[E];
        unit.weights(weight, a.wide_weight, a.dtype, w, v);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          p[i] = p[i] * scale * w[i];
          q[i] = q[i] * scale * v[i];
        }
      }
      if (!value) turn(unit, g, p, q);
      if (query) {
        if (!there) clear(p, q);
        unit.store(static_cast<T*>(a.q) + (size_t(t) * a.Hq + h) * D, p, q);
      } else if (there) {
        void* base = value ? c.v : c.k;
        store_cache<CT, E>(base, row * D + unit.d0, p, element);
        if (unit.two) store_cache<CT, E>(base, row * D + unit.d1, q, element);
        if (!value && u == 0) {
          if (c.positions) c.positions[row] = at.row[0];
          if (c.weights) c.weights[row] = 0.f;
        }
      }
      if (ONE) break;
    }
  }
}

// Sums of a workgroup's heads: rows of D floats of LDS, one for every head it
// holds at once (at most 256 threads x 16 floats).
constexpr int kSumFloats = 4096;

template <int DT, int E, bool HALF, bool ONE>
__global__ __launch_bounds__(256) void norm_rope_grad_kernel(NormRopeGradArgs a, Spread s) {
  typedef typename Elem<DT>::T T;
  typedef Unit<E, HALF> U;
  __shared__ float sums[kSumFloats];
  const int l = threadIdx.x % s.lanes, r = threadIdx.x / s.lanes;
  const int h0 = r % s.hp;
  const bool works = r / s.hp < s.tp;
  const U first(s.n, a.r.rot, l);
  float* mine = sums + r * a.D;
  const int groups = s.hp * s.tp;
  float w[E], v[E], dw[E], dv[E];
  clear(dw, dv);
  if (ONE) first.weights(a.weight, a.wide_weight, a.dtype, w, v);
  if (!ONE && a.partial) {
    for (int i = threadIdx.x; i < groups * a.D; i += blockDim.x) sums[i] = 0.f;
    __syncthreads();
  }
  for (int t = blockIdx.x * s.tp + r / s.hp; works && t < a.T; t += gridDim.x * s.tp) {
    const Place at = place_of(a.r, a.T, t);
    Angles<E, HALF> g;
    if (ONE && first.pair) load_angles(g, a.r, at, l, -1.f);
    for (int h = h0; h < a.H; h += s.hp) {
      const T* x = static_cast<const T*>(a.x) + t * a.x_token + h * a.x_head;
      const T* dy = static_cast<const T*>(a.dy) + t * a.dy_token + h * a.dy_head;
      T* dx = static_cast<T*>(a.dx) + t * a.dx_token + h * a.dx_head;
      float p[E], q[E], dp[E], dq[E];
      float ss = 0.f, gs = 0.f;   // sum x^2, sum g w x
      for (int u = l; u < s.n.pairs + s.n.copies; u += s.lanes) {
        const U unit = ONE ? first : U(s.n, a.r.rot, u);
        if (!ONE) {
          if (unit.pair) load_angles(g, a.r, at, u, -1.f);
          unit.weights(a.weight, a.wide_weight, a.dtype, w, v);
        }
        unit.load(x, p, q);
        unit.load(dy, dp, dq);
        turn(unit, g, dp, dq);
        ss += dot(p, q, p, q);
        float gw[E], gv[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
          gw[i] = dp[i] * w[i];
          gv[i] = dq[i] * v[i];
        }
        gs += dot(p, q, gw, gv);
        if (ONE) break;
      }
      const float scale = rsqrtf(over_head(ss, s.lanes) / float(a.D) + a.eps);
      const float pull = over_head(gs, s.lanes) / float(a.D) * scale * scale;   // mean(g w xh) r
      for (int u = l; u < s.n.pairs + s.n.copies; u += s.lanes) {
        const U unit = ONE ? first : U(s.n, a.r.rot, u);
        if (!ONE) {
          if (unit.pair) load_angles(g, a.r, at, u, -1.f);
          unit.weights(a.weight, a.wide_weight, a.dtype, w, v);
          unit.load(x, p, q);
          unit.load(dy, dp, dq);
          turn(unit, g, dp, dq);
        }
        float op[E], oq[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float xp = p[i] * scale, xq = q[i] * scale;
          if (ONE) {
            dw[i] += at.there ? dp[i] * xp : 0.f;
            dv[i] += at.there ? dq[i] * xq : 0.f;
          } else if (a.partial && at.there) {
            mine[unit.d0 + i] += dp[i] * xp;
            if (unit.two) mine[unit.d1 + i] += dq[i] * xq;
          }
          op[i] = at.there ? scale * (dp[i] * w[i]) - p[i] * scale * pull : 0.f;
          oq[i] = at.there ? scale * (dq[i] * v[i]) - q[i] * scale * pull : 0.f;
        }
        if (a.dx) unit.store(dx, op, oq);
        if (ONE) break;
      }
    }
  }
  if (!a.partial) return;
  if (ONE && works && first.there) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      mine[first.d0 + i] = dw[i];
      if (first.two) mine[first.d1 + i] = dv[i];
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < a.D; d += blockDim.x) {
    float sum = 0.f;
    for (int i = 0; i < groups; ++i) sum += sums[i * a.D + d];
    a.partial[size_t(blockIdx.x) * a.D + d] = sum;
  }
}

// dw[d] = the sum of n rows of D partial sums: 16 columns a workgroup, every
// 16th row a thread.
__global__ __launch_bounds__(256) void weight_grad_kernel(const float* partial, int n, int D, void* dw, int dtype) {
  __shared__ float part[16][17];
  const int d = blockIdx.x * 16 + threadIdx.x % 16, r = threadIdx.x / 16;
  float sum = 0.f;
  if (d < D)
    for (int i = r; i < n; i += 16) sum += partial[size_t(i) * D + d];
  part[r][threadIdx.x % 16] = sum;
  __syncthreads();
  if (r || d >= D) return;
  for (int i = 1; i < 16; ++i) sum += part[i][threadIdx.x];
  if (dtype == GBB_F32) static_cast<float*>(dw)[d] = sum;
  else if (dtype == GBB_F16) static_cast<_Float16*>(dw)[d] = _Float16(sum);
  else static_cast<bfloat*>(dw)[d] = bfloat(sum);
}

// Elements a unit: as many as 16 bytes hold, or fewer where the head's parts,
// an address or a stride are no multiple of that (interleaved pairs take two at
// least, at any address).
int unit_elements(int es, int rot, int D, bool half, uintptr_t bytes, uintptr_t weight, int ws) {
  const int run = half ? rot / 2 : rot, rest = D - rot;
  int E = 16 / es;
  const auto fits = [&] {
    return run % E == 0 && rest % E == 0 && rot % E == 0 && bytes % uintptr_t(E * es) == 0 && weight % uintptr_t(E * ws) == 0;
  };
  while (E > (half ? 1 : 2) && !fits()) E /= 2;
  return E;
}

Spread spread(int H, int D, int rot, int layout, int E, bool& one) {
  Spread s;
  s.n = units(D, rot, layout, E, E);
  const int nu = s.n.pairs + s.n.copies;
  s.lanes = 1;
  while (s.lanes < nu && s.lanes < 64) s.lanes *= 2;
  one = nu <= s.lanes;
  s.hp = std::min(H, 256 / s.lanes);
  s.tp = std::max(1, 256 / s.lanes / s.hp);
  return s;
}

// Workgroups along the heads: as many as the chip has room for (rope.hip).
dim3 grid_of(const Spread& s, int T, int H) {
  const int gx = (T + s.tp - 1) / s.tp, most = (H + s.hp - 1) / s.hp;
  return dim3(unsigned(gx), unsigned(std::max(1, std::min(most, 4 * device_compute_units() / gx))));
}

// f(element type, E) for the dtype and unit of a call.
template <int N> using Const = std::integral_constant<int, N>;
template <typename F>
void with_unit(int dtype, int E, F f) {
  const auto narrow = [&](auto dt) {
    if (E == 4) f(dt, Const<4>());
    else if (E == 2) f(dt, Const<2>());
    else f(dt, Const<1>());
  };
  if (dtype == GBB_F32) narrow(Const<GBB_F32>());
  else if (dtype == GBB_F16) E == 8 ? f(Const<GBB_F16>(), Const<8>()) : narrow(Const<GBB_F16>());
  else E == 8 ? f(Const<GBB_BF16>(), Const<8>()) : narrow(Const<GBB_BF16>());
}

uintptr_t address(const void* p) { return reinterpret_cast<uintptr_t>(p); }

}  // namespace

int launch_norm_rope(const NormRopeArgs& a, void* stream) {
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int es = a.dtype == GBB_F32 ? 4 : 2;
  const bool half = a.r.layout == GBB_ROPE_HALF;
  const int E = unit_elements(es, a.r.rot, a.D, half,
                              address(a.x) | address(a.y) | uintptr_t(es * (a.x_token | a.x_head | a.y_token | a.y_head)),
                              address(a.weight), a.wide_weight ? 4 : 2);
  bool one;
  const Spread s = spread(a.H, a.D, a.r.rot, a.r.layout, E, one);
  const dim3 grid = grid_of(s, a.T, a.H);
  with_unit(a.dtype, E, [&](auto dt, auto e) {
    constexpr int DT = decltype(dt)::value, N = decltype(e)::value;
    if (half) {
      if (one) start((norm_rope_kernel<DT, N, true, true>), grid, dim3(256), st, a, s);
      else start((norm_rope_kernel<DT, N, true, false>), grid, dim3(256), st, a, s);
    } else if constexpr (N > 1) {
      if (one) start((norm_rope_kernel<DT, N, false, true>), grid, dim3(256), st, a, s);
      else start((norm_rope_kernel<DT, N, false, false>), grid, dim3(256), st, a, s);
    }
  });
  return int(hipGetLastError());
}

// Workgroups of the gradient: enough to fill the chip, few enough that each
// sums over many heads.
int norm_rope_grad_rows(int T, int H) {
  return int(std::min<int64_t>(4 * int64_t(device_compute_units()), std::max<int64_t>(1, int64_t(T) * H)));
}

int launch_norm_rope_grad(const NormRopeGradArgs& a, void* dweight, void* stream) {
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int es = a.dtype == GBB_F32 ? 4 : 2;
  const bool half = a.r.layout == GBB_ROPE_HALF;
  const int E = unit_elements(es, a.r.rot, a.D, half,
                              address(a.x) | address(a.dy) | address(a.dx) |
                                  uintptr_t(es * (a.x_token | a.x_head | a.dy_token | a.dy_head | a.dx_token | a.dx_head)),
                              address(a.weight), a.wide_weight ? 4 : 2);
  bool one;
  const Spread s = spread(a.H, a.D, a.r.rot, a.r.layout, E, one);
  const unsigned grid = unsigned(std::min((a.T + s.tp - 1) / s.tp, norm_rope_grad_rows(a.T, a.H)));
  if (grid) with_unit(a.dtype, E, [&](auto dt, auto e) {
    constexpr int DT = decltype(dt)::value, N = decltype(e)::value;
    if (half) {
      if (one) start((norm_rope_grad_kernel<DT, N, true, true>), dim3(grid), dim3(256), st, a, s);
      else start((norm_rope_grad_kernel<DT, N, true, false>), dim3(grid), dim3(256), st, a, s);
    } else if constexpr (N > 1) {
      if (one) start((norm_rope_grad_kernel<DT, N, false, true>), dim3(grid), dim3(256), st, a, s);
      else start((norm_rope_grad_kernel<DT, N, false, false>), dim3(grid), dim3(256), st, a, s);
    }
  });
  if (dweight)
    start(weight_grad_kernel, dim3(unsigned(a.D + 15) / 16), dim3(256), st, static_cast<const float*>(a.partial), int(grid),
          a.D, dweight, a.wide_weight ? int(GBB_F32) : a.dtype);
  return int(hipGetLastError());
}

namespace {
template <int DT, int CT>
void run_norm_append(const gbb_paged_cache& c, const NormAppendArgs& a, int E, bool half, bool one, const Spread& s,
                     dim3 grid, hipStream_t st) {
  if (E == 8 && half) start((norm_append_kernel<DT, CT, 8, true, true>), grid, dim3(256), st, a, c, s);
  else if (E == 8) start((norm_append_kernel<DT, CT, 8, false, true>), grid, dim3(256), st, a, c, s);
  else if (half && one) start((norm_append_kernel<DT, CT, 1, true, true>), grid, dim3(256), st, a, c, s);
  else if (half) start((norm_append_kernel<DT, CT, 1, true, false>), grid, dim3(256), st, a, c, s);
  else if (one) start((norm_append_kernel<DT, CT, 2, false, true>), grid, dim3(256), st, a, c, s);
  else start((norm_append_kernel<DT, CT, 2, false, false>), grid, dim3(256), st, a, c, s);
}
}  // namespace

int launch_norm_append(const gbb_paged_cache& c, const NormAppendArgs& a, void* stream) {
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const bool half = a.r.layout == GBB_ROPE_HALF;
  int E = unit_elements(2, a.r.rot, c.head_dim, half, address(a.qkv), address(a.q_weight) | address(a.k_weight),
                        a.wide_weight ? 4 : 2);
  if (E < 8) E = half ? 1 : 2;
  bool one;
  const Spread s = spread(a.Hq + 2 * c.kv_heads, c.head_dim, a.r.rot, a.r.layout, E, one);
  const dim3 grid = grid_of(s, a.T, a.Hq + 2 * c.kv_heads);
  if (a.dtype == GBB_F16) {
    if (c.dtype == GBB_E4M3) run_norm_append<GBB_F16, GBB_E4M3>(c, a, E, half, one, s, grid, st);
    else run_norm_append<GBB_F16, GBB_F16>(c, a, E, half, one, s, grid, st);
  } else {
    if (c.dtype == GBB_E4M3) run_norm_append<GBB_BF16, GBB_E4M3>(c, a, E, half, one, s, grid, st);
    else run_norm_append<GBB_BF16, GBB_BF16>(c, a, E, half, one, s, grid, st);
  }
  return int(hipGetLastError());
}

}  // namespace gbb
