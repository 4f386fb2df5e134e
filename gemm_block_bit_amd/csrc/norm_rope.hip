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
// takes (in registers; fp32, one chain a lane and element: 22 terms for 16384 x 32
// heads of 128, some 20 000 for the most tokens that a call takes, 2^22 x 64 heads of
// 256), writes it to the workspace, and a second launch adds the workgroups' in their
// order, so it is the same bits each time.
//
// A workgroup takes several tokens, and loads a head's elements and angles while
// the one before is worked on: one token each waits for its place, angles and
// elements in turn (16384 x 32 heads of 128, bf16, with gradients 258 -> 147 us).
//
// Measured: forward 54 us (4.9 TB/s; a copy of its size 50.6), gradient 87 (4.6
// TB/s), 4097 tokens of 64 / 8 heads of 128 into an e4m3 cache 35 (4.7 TB/s).
// Calls of up to about a hundred tokens take a launch and two dependent reads.
#include <algorithm>

#include "rope_common.h"

namespace gbb {

namespace {

// A token's place in the table: a row an axis.
struct Place {
  int row[4];
  bool there;
};
template <bool AXES>
__device__ __forceinline__ Place place_of(const Rotation& r, int T, int t) {
  Place p;
  p.there = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pos = AXES ? i < r.axes ? r.positions[size_t(i) * T + t] : 0 : i == 0 ? r.positions[t] : 0;
    p.there = p.there && unsigned(pos) < unsigned(r.n_pos);
    p.row[i] = pos;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) p.row[i] = p.there ? p.row[i] : 0;
  return p;
}

// Angles of unit u, each pair's from the row of its own axis.  One axis is
// known at compile time: where both ways are there, the compiler loads word by
// word for either (16384 x 32 heads of 128: 84 us, 60 without).
template <bool AXES, int E, bool HALF>
__device__ __forceinline__ void load_angles(Angles<E, HALF>& g, const Rotation& r, const Place& at, int u, float sign) {
  if constexpr (!AXES) {
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

// Unit u of a head: E elements from d0 on and, in the half layout, E from d1:
// the pairs' other halves, or of a copied unit the E elements behind.
template <int E, bool HALF>
struct Unit {
  bool there, pair, two;
  int d0, d1;
  __device__ __forceinline__ Unit(const Units& n, int rot, int u) {
    there = u < n.pairs + n.copies;
    pair = u < n.pairs;
    two = HALF && there;
    d0 = pair ? u * E : rot + (u - n.pairs) * (HALF ? 2 * E : E);
    d1 = pair ? rot / 2 + u * E : d0 + E;
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
#pragma unroll
  for (int i = 0; i < Angles<E, HALF>::N; ++i) {
    float& a = HALF ? p[i] : p[2 * i];
    float& b = HALF ? q[i] : p[2 * i + 1];
    const float v = __builtin_fmaf(a, g.c[i], -(b * g.s[i]));
    b = __builtin_fmaf(b, g.c[i], a * g.s[i]);
    a = v;
  }
}
template <int E>
__device__ __forceinline__ void clear(float (&p)[E], float (&q)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) p[i] = q[i] = 0.f;
}
// Sum over the `lanes` lanes (a power of two) of a head, the same in each:
// lanes exchanged within the vector pipe (LDS would take 100 cycles a step).
template <int CTRL>
__device__ __forceinline__ float moved(float x) {
  const int v = __builtin_bit_cast(int, x);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(v, v, CTRL, 15, 15, false));
}
__device__ __forceinline__ float over_head(float x, int lanes) {
  if (lanes >= 2) x += moved<0xb1>(x);    // lanes 1 0 3 2 of four
  if (lanes >= 4) x += moved<0x4e>(x);    // 2 3 0 1
  if (lanes >= 8) x += moved<0x141>(x);   // eight lanes reversed: the other four, all alike by now
  if (lanes >= 16) x += moved<0x140>(x);  // sixteen reversed
  if (lanes >= 32) x += __shfl_xor(x, 16);
  if (lanes >= 64) x += __shfl_xor(x, 32);
  return x;
}
template <int E>
__device__ __forceinline__ float dot(const float (&p)[E], const float (&q)[E], const float (&v)[E], const float (&w)[E]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) s = __builtin_fmaf(p[i], v[i], s);
#pragma unroll
  for (int i = 0; i < E; ++i) s = __builtin_fmaf(q[i], w[i], s);
  return s;
}
// A unit as memory has it, so that the next one can be under way.
template <typename T, int E>
struct Packed {
  struct alignas(sizeof(T) * (E == 2 ? 1 : E)) V { T v[E]; };
  V p, q;
  template <bool HALF>
  __device__ __forceinline__ void load(const Unit<E, HALF>& u, const T* x) {
    if (u.there) p = *reinterpret_cast<const V*>(x + u.d0);
    if (u.two) q = *reinterpret_cast<const V*>(x + u.d1);
  }
  __device__ __forceinline__ void wide(float (&a)[E], float (&b)[E]) const {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      a[i] = float(p.v[i]);
      b[i] = float(q.v[i]);
    }
  }
};

// hp heads and tp tokens a workgroup, `lanes` lanes a head; ONE: every lane
// has one unit, else units l, l + lanes, ...
struct Spread {
  Units n;
  int lanes, hp, tp;
};

// The heads that a lane group takes, one after the other: a token's, then
// those of the next token that it has.
struct Walk {
  int t, h, first, last, heads, tokens;
  __device__ __forceinline__ Walk(const Spread& s, int H, int r)
      : t(blockIdx.x * s.tp + r / s.hp), h(blockIdx.y * s.hp + r % s.hp), first(h), last(H), heads(gridDim.y * s.hp),
        tokens(gridDim.x * s.tp) {}
  __device__ __forceinline__ bool step() {   // whether that is another token
    h += heads;
    if (h < last) return false;
    h = first;
    t += tokens;
    return true;
  }
};
__device__ __forceinline__ float inverse_root(float squares, int D, float eps) { return rsqrtf(squares * (1.f / float(D)) + eps); }

template <int DT, int E, bool HALF, bool ONE, bool AXES>
__global__ __launch_bounds__(256) void norm_rope_kernel(NormRopeArgs a, Spread s) {
  typedef typename Elem<DT>::T T;
  typedef Unit<E, HALF> U;
  const int l = threadIdx.x % s.lanes, r = threadIdx.x / s.lanes;
  Walk at(s, a.H, r);
  if (r / s.hp >= s.tp || at.t >= a.T || at.h >= a.H) return;
  const float sign = a.transpose ? -1.f : 1.f;
  const U first(s.n, a.r.rot, l);
  const auto x_of = [&](const Walk& w) { return static_cast<const T*>(a.x) + w.t * a.x_token + w.h * a.x_head; };
  const auto y_of = [&](const Walk& w) { return static_cast<T*>(a.y) + w.t * a.y_token + w.h * a.y_head; };
  float w[E], v[E], p[E], q[E];
  Angles<E, HALF> g;
  Place place = place_of<AXES>(a.r, a.T, at.t);
  if constexpr (ONE) {
    // the next head and, of another token, its angles are under way while this
    // one is worked on; a token's place is asked for a token earlier still
    Packed<T, E> x[2] = {};
    Angles<E, HALF> turns[2] = {};
    x[0].load(first, x_of(at));
    first.weights(a.weight, a.wide_weight, a.dtype, w, v);
    if (first.pair) load_angles<AXES>(turns[0], a.r, place, l, sign);
    Place place_next = place_of<AXES>(a.r, a.T, min(at.t + at.tokens, a.T - 1));
    const auto head = [&](int now, int then) {
      Walk next = at;
      const bool moves = next.step();
      const Place here = place;
      if (next.t < a.T) {
        x[then].load(first, x_of(next));
        if (moves) {
          place = place_next;
          if (first.pair) load_angles<AXES>(turns[then], a.r, place, l, sign);
          place_next = place_of<AXES>(a.r, a.T, min(next.t + next.tokens, a.T - 1));
        } else {
          turns[then] = turns[now];
        }
      }
      x[now].wide(p, q);
      if (a.norm) {
        const float scale = inverse_root(over_head(dot(p, q, p, q), s.lanes), a.D, a.eps);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          p[i] = p[i] * scale * w[i];
          q[i] = q[i] * scale * v[i];
        }
      }
      turn(first, turns[now], p, q);
      if (!here.there) clear(p, q);
      first.store(y_of(at), p, q);
      at = next;
    };
    while (at.t < a.T) {
      head(0, 1);
      if (at.t >= a.T) break;
      head(1, 0);
    }
  } else {
    for (; at.t < a.T; place = at.step() && at.t < a.T ? place_of<AXES>(a.r, a.T, at.t) : place) {
      float scale = 1.f;
      if (a.norm) {
        float ss = 0.f;
        for (int u = l; u < s.n.pairs + s.n.copies; u += s.lanes) {
          U(s.n, a.r.rot, u).load(x_of(at), p, q);
          ss += dot(p, q, p, q);
        }
        scale = inverse_root(over_head(ss, s.lanes), a.D, a.eps);
      }
      for (int u = l; u < s.n.pairs + s.n.copies; u += s.lanes) {
        const U unit(s.n, a.r.rot, u);
        if (unit.pair) load_angles<AXES>(g, a.r, place, u, sign);
        unit.weights(a.weight, a.wide_weight, a.dtype, w, v);
        unit.load(x_of(at), p, q);
        if (a.norm) {
#pragma unroll
          for (int i = 0; i < E; ++i) {
            p[i] = p[i] * scale * w[i];
            q[i] = q[i] * scale * v[i];
          }
        }
        turn(unit, g, p, q);
        if (!place.there) clear(p, q);
        unit.store(y_of(at), p, q);
      }
    }
  }
}

// The same over the q, k and v heads of a token; v heads are copied, k and v
// go to the token's slot.
template <int DT, int CT, int E, bool HALF, bool ONE, bool AXES>
__global__ __launch_bounds__(256) void norm_append_kernel(NormAppendArgs a, gbb_paged_cache c, Spread s) {
  typedef typename Elem<DT>::T T;
  typedef Unit<E, HALF> U;
  const int l = threadIdx.x % s.lanes, r = threadIdx.x / s.lanes;
  const int D = c.head_dim, Hkv = c.kv_heads, H = a.Hq + 2 * Hkv;
  Walk at(s, H, r);
  // q's and k's weights, in LDS: loads from memory on the way would wait for the
  // next head's, which were asked for before
  __shared__ __align__(16) float weights[2][256];
  if (a.norm && a.q_weight) {
    for (int d = threadIdx.x; d < 2 * D; d += 256) {
      const void* const from = d < D ? a.q_weight : a.k_weight;
      const int i = d < D ? d : d - D;
      weights[d >= D][i] = a.wide_weight ? static_cast<const float*>(from)[i] : float(static_cast<const T*>(from)[i]);
    }
    __syncthreads();
  }
  if (r / s.hp >= s.tp || at.t >= a.T || at.h >= H) return;
  const U first(s.n, a.r.rot, l);
  const auto x_of = [&](const Walk& w) { return static_cast<const T*>(a.qkv) + w.t * a.token_stride + size_t(w.h) * D; };
  struct Token {
    Place place;
    int slot;
  };
  const auto token_of = [&](int t) { return Token{place_of<AXES>(a.r, a.T, t), a.slots[t]}; };
  float p[E], q[E], w[E], v[E];
  Angles<E, HALF> g;
  // the scale of a head's elements in the cache
  const auto element_of = [&](int h) {
    const float* const scales = CT != GBB_E4M3 || h < a.Hq ? nullptr : h < a.Hq + Hkv ? c.k_scale : c.v_scale;
    return scales ? scales[(h - a.Hq) % Hkv] : 1.f;
  };
  // unit u of head `at` from p and q, the head's inverse root mean square given
  const auto finish = [&](const U& unit, int u, const Token& token, float scale, float element) {
    const bool query = at.h < a.Hq, value = at.h >= a.Hq + Hkv;
    const bool there = token.place.there && unsigned(token.slot) < unsigned(c.num_pages) * unsigned(c.page);
    if (a.norm && !value) {
      unit.load(weights[!query], w, v);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        p[i] = p[i] * scale * w[i];
        q[i] = q[i] * scale * v[i];
      }
    }
    if (!value) turn(unit, g, p, q);
    if (query) {
      if (!there) clear(p, q);
      unit.store(static_cast<T*>(a.q) + (size_t(at.t) * a.Hq + at.h) * D, p, q);
    } else if (there) {
      // slots are below 2^31, pages times heads times rows may not be
      const int hk = value ? at.h - a.Hq - Hkv : at.h - a.Hq;
      const int shift = 31 - __builtin_clz(unsigned(c.page));   // a power of two
      const size_t row = ((size_t(token.slot >> shift) * Hkv + hk) << shift) + (token.slot & (c.page - 1));
      void* base = value ? c.v : c.k;
      if (unit.there) store_cache<CT, E>(base, row * D + unit.d0, p, element);
      if (unit.two) store_cache<CT, E>(base, row * D + unit.d1, q, element);
      if (!value && u == 0) {
        if (c.positions) c.positions[row] = token.place.row[0];
        if (c.weights) c.weights[row] = 0.f;
      }
    }
  };
  Token token = token_of(at.t);
  if constexpr (ONE) {
    Packed<T, E> x = {}, x_next = {};
    x.load(first, x_of(at));
    float element = element_of(at.h), element_next = 1.f;
    if (first.pair) load_angles<AXES>(g, a.r, token.place, l, 1.f);
    Token token_next = token_of(min(at.t + at.tokens, a.T - 1));
    while (at.t < a.T) {
      Walk next = at;
      const bool moves = next.step();
      Angles<E, HALF> g_next;                // not in halves, where a unit's angles take twice
      if (!HALF) g_next = g;                 // the registers (36 us, with them 42 in 4 workgroups a CU)
      const Token here = token;
      if (next.t < a.T) {
        x_next.load(first, x_of(next));
        element_next = element_of(next.h);
        if (moves) {
          token = token_next;
          if (!HALF && first.pair) load_angles<AXES>(g_next, a.r, token.place, l, 1.f);
          token_next = token_of(min(next.t + next.tokens, a.T - 1));
        }
      }
      x.wide(p, q);
      float scale = 1.f;
      if (a.norm && at.h < a.Hq + Hkv) scale = inverse_root(over_head(dot(p, q, p, q), s.lanes), D, a.eps);
      finish(first, l, here, scale, element);
      x = x_next;
      element = element_next;
      if (!HALF) g = g_next;
      else if (moves && next.t < a.T && first.pair) load_angles<AXES>(g, a.r, token.place, l, 1.f);
      at = next;
    }
  } else {
    for (; at.t < a.T; token = at.step() && at.t < a.T ? token_of(at.t) : token) {
      float scale = 1.f;
      if (a.norm && at.h < a.Hq + Hkv) {   // the same for all lanes of a head
        float ss = 0.f;
        for (int u = l; u < s.n.pairs + s.n.copies; u += s.lanes) {
          U(s.n, a.r.rot, u).load(x_of(at), p, q);
          ss += dot(p, q, p, q);
        }
        scale = inverse_root(over_head(ss, s.lanes), D, a.eps);
      }
      for (int u = l; u < s.n.pairs + s.n.copies; u += s.lanes) {
        const U unit(s.n, a.r.rot, u);
        if (unit.pair) load_angles<AXES>(g, a.r, token.place, u, 1.f);
        unit.load(x_of(at), p, q);
        finish(unit, u, token, scale, element_of(at.h));
      }
    }
  }
}

// Sums of a workgroup's heads: rows of D floats of LDS, one for every head it
// holds at once (at most 256 threads x 16 floats).
constexpr int kSumFloats = 4096;

template <int DT, int E, bool HALF, bool ONE, bool AXES>
__global__ __launch_bounds__(256) void norm_rope_grad_kernel(NormRopeGradArgs a, Spread s) {
  typedef typename Elem<DT>::T T;
  typedef Unit<E, HALF> U;
  __shared__ float sums[kSumFloats];
  const int l = threadIdx.x % s.lanes, r = threadIdx.x / s.lanes;
  const bool works = r / s.hp < s.tp;
  const U first(s.n, a.r.rot, l);
  float* mine = sums + r * a.D;
  const int groups = s.hp * s.tp;
  const float share = 1.f / float(a.D);
  float w[E], v[E], p[E], q[E], dp[E], dq[E], dw[E], dv[E];
  clear(dw, dv);
  Angles<E, HALF> g;
  Walk at(s, a.H, r);
  const auto x_of = [&](const Walk& k) { return static_cast<const T*>(a.x) + k.t * a.x_token + k.h * a.x_head; };
  const auto dy_of = [&](const Walk& k) { return static_cast<const T*>(a.dy) + k.t * a.dy_token + k.h * a.dy_head; };
  const auto dx_of = [&](const Walk& k) { return static_cast<T*>(a.dx) + k.t * a.dx_token + k.h * a.dx_head; };
  // dx of a unit from p, q and the turned dp, dq; also its terms of dw
  const auto finish = [&](const U& unit, bool there, float scale, float pull, auto term) {
    float op[E], oq[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float up = p[i] * scale, uq = q[i] * scale;
      term(i, there ? dp[i] * up : 0.f, there ? dq[i] * uq : 0.f);
      op[i] = there ? scale * __builtin_fmaf(dp[i], w[i], -(up * pull)) : 0.f;
      oq[i] = there ? scale * __builtin_fmaf(dq[i], v[i], -(uq * pull)) : 0.f;
    }
    if (a.dx) unit.store(dx_of(at), op, oq);
  };
  // sums of x^2 and of g w x over a unit
  const auto add_sums = [&](float& ss, float& gs) {
    ss += dot(p, q, p, q);
    float gw[E], gv[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      gw[i] = dp[i] * w[i];
      gv[i] = dq[i] * v[i];
    }
    gs += dot(p, q, gw, gv);
  };
  const bool some = works && at.t < a.T && at.h < a.H;
  if constexpr (ONE) {
    if (some) {
      Packed<T, E> x = {}, dy = {}, x_next = {}, dy_next = {};
      x.load(first, x_of(at));
      dy.load(first, dy_of(at));
      first.weights(a.weight, a.wide_weight, a.dtype, w, v);
      Place place = place_of<AXES>(a.r, a.T, at.t);
      if (first.pair) load_angles<AXES>(g, a.r, place, l, -1.f);
      Place place_next = place_of<AXES>(a.r, a.T, min(at.t + at.tokens, a.T - 1));
      while (at.t < a.T) {
        Walk next = at;
        const bool moves = next.step();
        Angles<E, HALF> g_next = g;
        const bool there = place.there;
        if (next.t < a.T) {
          x_next.load(first, x_of(next));
          dy_next.load(first, dy_of(next));
          if (moves) {
            place = place_next;
            if (first.pair) load_angles<AXES>(g_next, a.r, place, l, -1.f);
            place_next = place_of<AXES>(a.r, a.T, min(next.t + next.tokens, a.T - 1));
          }
        }
        x.wide(p, q);
        dy.wide(dp, dq);
        turn(first, g, dp, dq);
        float ss = 0.f, gs = 0.f;
        add_sums(ss, gs);
        const float scale = inverse_root(over_head(ss, s.lanes), a.D, a.eps);
        const float pull = over_head(gs, s.lanes) * share * scale;   // mean(g w xh)
        finish(first, there, scale, pull, [&](int i, float tp, float tq) {
          dw[i] += tp;
          dv[i] += tq;
        });
        x = x_next;
        dy = dy_next;
        g = g_next;
        at = next;
      }
    }
  } else {
    if (a.partial) {
      for (int i = threadIdx.x; i < groups * a.D; i += blockDim.x) sums[i] = 0.f;
      __syncthreads();
    }
    for (; some && at.t < a.T; at.step()) {
      const Place place = place_of<AXES>(a.r, a.T, at.t);
      const auto load = [&](const U& unit, int u) {
        if (unit.pair) load_angles<AXES>(g, a.r, place, u, -1.f);
        unit.weights(a.weight, a.wide_weight, a.dtype, w, v);
        unit.load(x_of(at), p, q);
        unit.load(dy_of(at), dp, dq);
        turn(unit, g, dp, dq);
      };
      float ss = 0.f, gs = 0.f;
      for (int u = l; u < s.n.pairs + s.n.copies; u += s.lanes) {
        load(U(s.n, a.r.rot, u), u);
        add_sums(ss, gs);
      }
      const float scale = inverse_root(over_head(ss, s.lanes), a.D, a.eps);
      const float pull = over_head(gs, s.lanes) * share * scale;
      for (int u = l; u < s.n.pairs + s.n.copies; u += s.lanes) {
        const U unit(s.n, a.r.rot, u);
        load(unit, u);
        finish(unit, place.there, scale, pull, [&](int i, float tp, float tq) {
          if (!a.partial) return;
          mine[unit.d0 + i] += tp;
          if (unit.two) mine[unit.d1 + i] += tq;
        });
      }
    }
  }
  if (!a.partial) return;
  if (ONE && works && first.there) {   // (zeros of a group that had no head)
#pragma unroll
    for (int i = 0; i < E; ++i) {
      mine[first.d0 + i] = dw[i];
      if (first.two) mine[first.d1 + i] = dv[i];
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < a.D; d += blockDim.x) {
    float sum = 0.f;
#pragma unroll 8
    for (int i = 0; i < groups; ++i) sum += sums[i * a.D + d];
    a.partial[size_t(blockIdx.x) * a.D + d] = sum;
  }
}

// dw[d] = the sum of n rows of D partial sums: 8 columns a workgroup, every
// 32nd row a thread, 16 of them under way at once (one by one 1024 rows took 20
// us, mostly waiting).
__global__ __launch_bounds__(256) void weight_grad_kernel(const float* partial, int n, int D, void* dw, int dtype) {
  __shared__ float part[32][9];
  const int c = threadIdx.x % 8, d = blockIdx.x * 8 + c, r = threadIdx.x / 8;
  float sum = 0.f;
  if (d < D)
    for (int i0 = r; i0 < n; i0 += 32 * 16) {
      float x[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) x[u] = i0 + 32 * u < n ? partial[size_t(i0 + 32 * u) * D + d] : 0.f;
#pragma unroll
      for (int u = 0; u < 16; ++u) sum += x[u];
    }
  part[r][c] = sum;
  __syncthreads();
  if (r || d >= D) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) sum += part[i][c];
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
    return run % E == 0 && rest % (half ? 2 * E : E) == 0 && rot % E == 0 && bytes % uintptr_t(E * es) == 0 && weight % uintptr_t(E * ws) == 0;
  };
  while (E > (half ? 1 : 2) && !fits()) E /= 2;
  return E;
}

Spread spread(int H, int D, int rot, int layout, int E, bool& one) {
  Spread s;
  s.n = units(D, rot, layout, E, layout == GBB_ROPE_HALF ? 2 * E : E);
  const int nu = s.n.pairs + s.n.copies;
  s.lanes = 1;
  while (s.lanes < nu && s.lanes < 64) s.lanes *= 2;
  one = nu <= s.lanes;
  s.hp = std::min(H, 256 / s.lanes);
  s.tp = std::max(1, 256 / s.lanes / s.hp);
  return s;
}

// Workgroups: with few tokens along the heads too, as many as the chip has room
// for, with many those that are resident at once: each then takes several
// tokens, one under way while another is worked on.
dim3 grid_of(const Spread& s, int T, int H, int resident) {
  const int gx = std::min((T + s.tp - 1) / s.tp, resident * device_compute_units()), most = (H + s.hp - 1) / s.hp;
  return dim3(unsigned(gx), unsigned(std::max(1, std::min(most, 4 * device_compute_units() / gx))));
}
// Workgroups of 256 threads a CU, by the registers that a unit takes: 16384 x 32
// heads of 128 in halves 54 us in 4 a CU, 56 in 8, interleaved 56 in 8, 57 in 4;
// 4097 tokens into an e4m3 cache 35 in 6, 40 in 8, 41 in 4, in halves 36 in 5, 40 in 4, 39 in 6.
int resident(bool half, int E) { return half && E == 8 ? 4 : 8; }
int appending(bool half, int E) { return half && E == 8 ? 5 : 6; }
// The gradient's, each of which sums over its heads: in halves 87 us in 3 a CU, 92 in
// 8; interleaved 86 in 5, 98 in 3; heads of 96 with 24 rotated 100 in 5, 132 in 3.
constexpr int kMostSummed = 5;
int summed(bool half, int E) { return half && E == 8 ? 3 : kMostSummed; }

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
  const dim3 grid = grid_of(s, a.T, a.H, resident(half, E));
  with_unit(a.dtype, E, [&](auto dt, auto e) {
    constexpr int DT = decltype(dt)::value, N = decltype(e)::value;
    if (half) {
      if (one) a.r.axes > 1 ? start((norm_rope_kernel<DT, N, true, true, true>), grid, dim3(256), st, a, s)
               : start((norm_rope_kernel<DT, N, true, true, false>), grid, dim3(256), st, a, s);
      else a.r.axes > 1 ? start((norm_rope_kernel<DT, N, true, false, true>), grid, dim3(256), st, a, s)
               : start((norm_rope_kernel<DT, N, true, false, false>), grid, dim3(256), st, a, s);
    } else if constexpr (N > 1) {
      if (one) a.r.axes > 1 ? start((norm_rope_kernel<DT, N, false, true, true>), grid, dim3(256), st, a, s)
               : start((norm_rope_kernel<DT, N, false, true, false>), grid, dim3(256), st, a, s);
      else a.r.axes > 1 ? start((norm_rope_kernel<DT, N, false, false, true>), grid, dim3(256), st, a, s)
               : start((norm_rope_kernel<DT, N, false, false, false>), grid, dim3(256), st, a, s);
    }
  });
  return int(hipGetLastError());
}

// Workgroups of the gradient, at most.
int norm_rope_grad_rows(int T, int H) {
  return int(std::min<int64_t>(kMostSummed * int64_t(device_compute_units()), std::max<int64_t>(1, int64_t(T) * H)));
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
  const unsigned grid = unsigned(std::min((a.T + s.tp - 1) / s.tp, summed(half, E) * device_compute_units()));
  if (grid) with_unit(a.dtype, E, [&](auto dt, auto e) {
    constexpr int DT = decltype(dt)::value, N = decltype(e)::value;
    if (half) {
      if (one) a.r.axes > 1 ? start((norm_rope_grad_kernel<DT, N, true, true, true>), dim3(grid), dim3(256), st, a, s)
               : start((norm_rope_grad_kernel<DT, N, true, true, false>), dim3(grid), dim3(256), st, a, s);
      else a.r.axes > 1 ? start((norm_rope_grad_kernel<DT, N, true, false, true>), dim3(grid), dim3(256), st, a, s)
               : start((norm_rope_grad_kernel<DT, N, true, false, false>), dim3(grid), dim3(256), st, a, s);
    } else if constexpr (N > 1) {
      if (one) a.r.axes > 1 ? start((norm_rope_grad_kernel<DT, N, false, true, true>), dim3(grid), dim3(256), st, a, s)
               : start((norm_rope_grad_kernel<DT, N, false, true, false>), dim3(grid), dim3(256), st, a, s);
      else a.r.axes > 1 ? start((norm_rope_grad_kernel<DT, N, false, false, true>), dim3(grid), dim3(256), st, a, s)
               : start((norm_rope_grad_kernel<DT, N, false, false, false>), dim3(grid), dim3(256), st, a, s);
    }
  });
  if (dweight)
    start(weight_grad_kernel, dim3(unsigned(a.D + 7) / 8), dim3(256), st, static_cast<const float*>(a.partial), int(grid),
          a.D, dweight, a.wide_weight ? int(GBB_F32) : a.dtype);
  return int(hipGetLastError());
}

namespace {
template <int DT, int CT, bool AXES>
void run_norm_append_axes(const gbb_paged_cache& c, const NormAppendArgs& a, int E, bool half, bool one, const Spread& s,
                     dim3 grid, hipStream_t st) {
  if (E == 8 && half) start((norm_append_kernel<DT, CT, 8, true, true, AXES>), grid, dim3(256), st, a, c, s);
  else if (E == 8) start((norm_append_kernel<DT, CT, 8, false, true, AXES>), grid, dim3(256), st, a, c, s);
  else if (half && one) start((norm_append_kernel<DT, CT, 1, true, true, AXES>), grid, dim3(256), st, a, c, s);
  else if (half) start((norm_append_kernel<DT, CT, 1, true, false, AXES>), grid, dim3(256), st, a, c, s);
  else if (one) start((norm_append_kernel<DT, CT, 2, false, true, AXES>), grid, dim3(256), st, a, c, s);
  else start((norm_append_kernel<DT, CT, 2, false, false, AXES>), grid, dim3(256), st, a, c, s);
}
template <int DT, int CT>
void run_norm_append(const gbb_paged_cache& c, const NormAppendArgs& a, int E, bool half, bool one, const Spread& s,
                     dim3 grid, hipStream_t st) {
  if (a.r.axes > 1) run_norm_append_axes<DT, CT, true>(c, a, E, half, one, s, grid, st);
  else run_norm_append_axes<DT, CT, false>(c, a, E, half, one, s, grid, st);
}
}  // namespace

int launch_norm_append(const gbb_paged_cache& c, const NormAppendArgs& a, void* stream) {
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const bool half = a.r.layout == GBB_ROPE_HALF;
  int E = unit_elements(2, a.r.rot, c.head_dim, half, address(a.qkv), address(a.q_weight) | address(a.k_weight),
                        a.wide_weight ? 4 : 2);
  if (E < 8) E = half ? 1 : 2;   // (heads whose parts are no multiple of 8 are few: no kernels of their own between)
  bool one;
  const Spread s = spread(a.Hq + 2 * c.kv_heads, c.head_dim, a.r.rot, a.r.layout, E, one);
  const dim3 grid = grid_of(s, a.T, a.Hq + 2 * c.kv_heads, appending(half, E));
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
