// C-ABI entry points of the rotary positions and the paged cache: argument
// checks, workspace sizes and launches.  No allocation, no synchronization.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "internal.h"

using namespace gbb;

namespace {

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

gbb_status device_status(int err, const char* what) {
  const char* msg = device_error_text(err);
  if (!msg) return GBB_OK;
  return fail(GBB_E_DEVICE, "%s: HIP error %d (%s)", what, err, msg);
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const char* x = static_cast<const char*>(a);
  const char* y = static_cast<const char*>(b);
  return x < y + nb && y < x + na;
}

constexpr int kMaxTokens = 1 << 22;    // tokens of a call: grid x threads stays below 2^32
constexpr int64_t kMaxGroups = 1 << 22;  // workgroups of either kind in a launch, for the same reason
constexpr int kMaxHeads = 1 << 14;

gbb_status check_table(const int32_t* positions, const float* table, int n_pos, int D, int rot, int layout) {
  if (!positions || !table) return fail(GBB_E_ARG, "positions and table must not be NULL");
  if (n_pos <= 0) return fail(GBB_E_ARG, "n_pos must be positive (%d)", n_pos);
  if (layout != GBB_ROPE_HALF && layout != GBB_ROPE_INTERLEAVED) return fail(GBB_E_ARG, "unknown layout %d", layout);
  if (rot < 2 || rot % 2 || rot > D) return fail(GBB_E_SHAPE, "rot=%d must be even, at least 2 and at most %d", rot, D);
  if (!aligned(positions, 4) || !aligned(table, 8)) return fail(GBB_E_ALIGN, "positions or table is misaligned");
  return GBB_OK;
}

gbb_status check_cache(const gbb_paged_cache* c) {
  if (!c) return fail(GBB_E_ARG, "cache is NULL");
  if (!c->k || !c->v) return fail(GBB_E_ARG, "the cache's k and v must not be NULL");
  if (c->dtype != GBB_F16 && c->dtype != GBB_BF16 && c->dtype != GBB_E4M3)
    return fail(GBB_E_ARG, "unknown cache dtype %d", c->dtype);
  if (c->dtype != GBB_E4M3 && (c->k_scale || c->v_scale)) return fail(GBB_E_ARG, "only an e4m3 cache has scales");
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128 && c->page != 256)
    return fail(GBB_E_SHAPE, "page must be 16, 32, 64, 128 or 256 (%d)", c->page);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(GBB_E_SHAPE, "head_dim must be 64, 128 or 256 (%d)", c->head_dim);
  if (c->num_pages <= 0 || c->kv_heads <= 0)
    return fail(GBB_E_ARG, "num_pages and kv_heads must be positive (%d, %d)", c->num_pages, c->kv_heads);
  if (c->kv_heads > kMaxHeads) return fail(GBB_E_SHAPE, "kv_heads=%d exceeds %d", c->kv_heads, kMaxHeads);
  if (int64_t(c->num_pages) * c->page > INT_MAX)
    return fail(GBB_E_SHAPE, "num_pages * page must be below 2^31 (%d * %d)", c->num_pages, c->page);
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return fail(GBB_E_ALIGN, "the cache's k and v must be 16-byte aligned");
  if (!aligned(c->weights, 16) || !aligned(c->positions, 16))
    return fail(GBB_E_ALIGN, "the cache's weights and positions must be 16-byte aligned");
  if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return fail(GBB_E_ALIGN, "k_scale or v_scale is misaligned");
  return GBB_OK;
}

// 16-bit inputs that go with the cache's elements.
gbb_status check_dtype(const gbb_paged_cache* c, int dtype) {
  if (dtype != GBB_F16 && dtype != GBB_BF16) return fail(GBB_E_ARG, "dtype must be GBB_F16 or GBB_BF16 (%d)", dtype);
  if (c->dtype != GBB_E4M3 && c->dtype != dtype)
    return fail(GBB_E_ARG, "dtype %d does not go with a cache of dtype %d", dtype, c->dtype);
  return GBB_OK;
}

gbb_status check_heads(const gbb_paged_cache* c, int q_heads) {
  if (q_heads <= 0 || q_heads % c->kv_heads)
    return fail(GBB_E_SHAPE, "q_heads=%d must be a positive multiple of kv_heads=%d", q_heads, c->kv_heads);
  if (q_heads / c->kv_heads > kMaxGroup)
    return fail(GBB_E_SHAPE, "at most %d query heads per kv head (%d / %d)", kMaxGroup, q_heads, c->kv_heads);
  return GBB_OK;
}

gbb_status check_sequences(const gbb_paged_cache* c, int B, const int32_t* block_table, int max_pages,
                           const int32_t* lengths, int max_len) {
  if (B < 0) return fail(GBB_E_ARG, "B must not be negative (%d)", B);
  if (max_len < 1 || max_pages < 1) return fail(GBB_E_ARG, "max_len and max_pages must be positive (%d, %d)", max_len, max_pages);
  if (int64_t(max_len) > int64_t(max_pages) * c->page)
    return fail(GBB_E_SHAPE, "max_len=%d exceeds max_pages * page = %d * %d", max_len, max_pages, c->page);
  if (max_len > INT_MAX - 8192) return fail(GBB_E_SHAPE, "max_len=%d is too large", max_len);
  if (B == 0) return GBB_OK;
  if (!block_table || !lengths) return fail(GBB_E_ARG, "block_table and lengths must not be NULL");
  if (!aligned(block_table, 4) || !aligned(lengths, 4)) return fail(GBB_E_ALIGN, "block_table or lengths is misaligned");
  return GBB_OK;
}

gbb_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!need) return GBB_OK;
  if (!ws) return fail(GBB_E_ARG, "workspace of %zu bytes is required", need);
  if (have < need) return fail(GBB_E_SPACE, "workspace needs %zu bytes, got %zu", need, have);
  if (!aligned(ws, 16)) return fail(GBB_E_ALIGN, "workspace is not 16-byte aligned");
  return GBB_OK;
}

// Shapes alone, for the workspace queries (launch sizes included).
gbb_status check_attend_shape(const gbb_paged_cache* c, int B, int q_heads, int max_len, bool with_weights, int window,
                              AttendPlan& p) {
  gbb_status st = check_cache(c);
  if (st != GBB_OK) return st;
  if ((st = check_heads(c, q_heads)) != GBB_OK) return st;
  if (B < 0 || max_len < 1 || max_len > INT_MAX - 8192) return fail(GBB_E_ARG, "bad B or max_len (%d, %d)", B, max_len);
  if (int64_t(B) * q_heads > kMaxGroups) return fail(GBB_E_SHAPE, "B * q_heads exceeds %d", int(kMaxGroups));
  if (window < 0) return fail(GBB_E_ARG, "window must not be negative (%d)", window);
  if (B) {
    p = attend_plan(*c, B, q_heads, max_len, with_weights, window);
    const int64_t pairs = int64_t(B) * c->kv_heads;
    if (pairs * p.qtiles > kMaxGroups / p.nsplit || pairs > kMaxGroups / (1 + max_len / 256))
      return fail(GBB_E_SHAPE, "B=%d, kv_heads=%d and max_len=%d make too many workgroups", B, c->kv_heads, max_len);
  }
  return GBB_OK;
}

gbb_status check_evict_shape(const gbb_paged_cache* c, int B, int max_len, int budget) {
  const gbb_status st = check_cache(c);
  if (st != GBB_OK) return st;
  if (B < 0 || max_len < 1 || max_len > INT_MAX - 8192) return fail(GBB_E_ARG, "bad B or max_len (%d, %d)", B, max_len);
  if (max_len > kMaxEvictLen) return fail(GBB_E_SHAPE, "max_len=%d exceeds %d", max_len, kMaxEvictLen);
  if (budget < 1) return fail(GBB_E_ARG, "budget must be at least 1 (%d)", budget);
  if (int64_t(B) * c->kv_heads > kMaxGroups / 4 / (1 + max_len / 4096))
    return fail(GBB_E_SHAPE, "B=%d, kv_heads=%d and max_len=%d make too many workgroups", B, c->kv_heads, max_len);
  return GBB_OK;
}

// A view [T][H][D] of memory with strides in elements.
struct View {
  const void* p;
  int64_t token, head;
};
size_t view_bytes(const View& v, int T, int H, int D, size_t es) {
  return (size_t(T - 1) * v.token + size_t(H - 1) * v.head + D) * es;
}
bool same_view(const View& a, const View& b, int T, int H) {
  return a.p == b.p && (T == 1 || a.token == b.token) && (H == 1 || a.head == b.head);
}

gbb_status check_heads_shape(int dtype, int T, int H, int D) {
  if (dtype != GBB_F16 && dtype != GBB_BF16 && dtype != GBB_F32) return fail(GBB_E_ARG, "unknown dtype %d", dtype);
  if (T < 0 || H <= 0 || D <= 0) return fail(GBB_E_ARG, "T, H or D is negative or zero (%d, %d, %d)", T, H, D);
  if (D % 2 || D > 1024) return fail(GBB_E_SHAPE, "D=%d must be even and at most 1024", D);
  if (T > kMaxTokens || H > kMaxHeads) return fail(GBB_E_SHAPE, "T=%d or H=%d exceeds %d, %d", T, H, kMaxTokens, kMaxHeads);
  return GBB_OK;
}

gbb_status check_strides(std::initializer_list<View> views) {
  const int64_t big = int64_t(1) << 40;
  for (const View& v : views)
    if (v.token < 0 || v.head < 0 || v.token > big || v.head > big)
      return fail(GBB_E_ARG, "a stride is negative or above 2^40");
  return GBB_OK;
}

// Memory that a call writes: the rows of y must be memory of their own, a
// token's heads or a head's tokens together; inputs may repeat (broadcast ones).
gbb_status check_rows_apart(const View& y, int T, int H, int D, const char* name) {
  const auto apart = [&](int64_t inner, int ni, int64_t outer, int no) {
    return (ni == 1 || inner >= D) && (no == 1 || outer >= (ni - 1) * inner + D);
  };
  if (!apart(y.head, H, y.token, T) && !apart(y.token, T, y.head, H))
    return fail(GBB_E_SHAPE, "%s's strides %lld, %lld make its heads overlap", name, (long long)y.token, (long long)y.head);
  return GBB_OK;
}

gbb_status check_turned(const View& x, const View& y, int dtype, int T, int H, int D) {
  if (!x.p || !y.p) return fail(GBB_E_ARG, "x and y must not be NULL");
  const size_t es = dtype == GBB_F32 ? 4 : 2;
  if (!aligned(x.p, es) || !aligned(y.p, es)) return fail(GBB_E_ALIGN, "x or y is not aligned to its elements");
  const gbb_status st = check_rows_apart(y, T, H, D, "y");
  if (st != GBB_OK) return st;
  if (!same_view(x, y, T, H) && overlap(x.p, view_bytes(x, T, H, D, es), y.p, view_bytes(y, T, H, D, es)))
    return fail(GBB_E_ARG, "x and y overlap");
  return GBB_OK;
}

// The rotation of a call with axes and sections.
gbb_status rotation_of(const int32_t* positions, int axes, const int* sections, const float* table, int n_pos, int D,
                       int rot, int layout, Rotation& r) {
  const gbb_status st = check_table(positions, table, n_pos, D, rot, layout);
  if (st != GBB_OK) return st;
  if (axes < 1 || axes > GBB_MAX_AXES) return fail(GBB_E_ARG, "axes must be 1 to %d (%d)", GBB_MAX_AXES, axes);
  r = {positions, table, n_pos, rot, layout, axes, {INT_MAX, INT_MAX, INT_MAX}};
  if (axes == 1 && !sections) return GBB_OK;
  if (!sections) return fail(GBB_E_ARG, "sections must not be NULL with %d axes", axes);
  int64_t sum = 0;
  for (int i = 0; i < axes; ++i) {
    if (sections[i] < 0) return fail(GBB_E_ARG, "sections must not be negative (%d)", sections[i]);
    sum += sections[i];
    if (i + 1 < axes) r.end[i] = int(std::min<int64_t>(sum, INT_MAX));
  }
  if (sum != rot / 2) return fail(GBB_E_SHAPE, "sections add up to %lld, not to rot / 2 = %d", (long long)sum, rot / 2);
  return GBB_OK;
}

gbb_status check_norm(const void* weight, int weight_dtype, int dtype, float eps) {
  if (weight && weight_dtype != GBB_F32 && weight_dtype != dtype)
    return fail(GBB_E_ARG, "weight_dtype must be GBB_F32 or that of x (%d)", weight_dtype);
  if (!aligned(weight, weight_dtype == GBB_F32 ? 4 : 2)) return fail(GBB_E_ALIGN, "a weight is not aligned to its elements");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(GBB_E_ARG, "eps must be 0 or more and finite");
  return GBB_OK;
}

}  // namespace

extern "C" gbb_status gbb_rope(const void* x, int64_t x_token, int64_t x_head, void* y, int64_t y_token,
                               int64_t y_head, int dtype, int T, int H, int D, const int32_t* positions,
                               const float* table, int n_pos, int rot, int layout, int transpose, void* stream) {
  const View vx = {x, x_token, x_head}, vy = {y, y_token, y_head};
  gbb_status st = check_heads_shape(dtype, T, H, D);
  if (st != GBB_OK || (st = check_strides({vx, vy})) != GBB_OK) return st;
  if (T == 0) return GBB_OK;
  if ((st = check_table(positions, table, n_pos, D, rot, layout)) != GBB_OK) return st;
  if ((st = check_turned(vx, vy, dtype, T, H, D)) != GBB_OK) return st;
  const RopeArgs a = {x, y, x_token, x_head, y_token, y_head, positions, table, T, H, D, n_pos, rot, layout,
                      transpose, dtype};
  return device_status(launch_rope(a, stream), "rope launch");
}

extern "C" gbb_status gbb_rope_axes(const void* x, int64_t x_token, int64_t x_head, void* y, int64_t y_token,
                                    int64_t y_head, int dtype, int T, int H, int D, const int32_t* positions, int axes,
                                    const int* sections, const float* table, int n_pos, int rot, int layout,
                                    int transpose, void* stream) {
  const View vx = {x, x_token, x_head}, vy = {y, y_token, y_head};
  NormRopeArgs a = {x, y, x_token, x_head, y_token, y_head, nullptr, {}, T, H, D, dtype, 0.f, false, transpose != 0, false};
  gbb_status st = check_heads_shape(dtype, T, H, D);
  if (st != GBB_OK || (st = check_strides({vx, vy})) != GBB_OK) return st;
  if (T == 0) return GBB_OK;
  if ((st = rotation_of(positions, axes, sections, table, n_pos, D, rot, layout, a.r)) != GBB_OK) return st;
  if ((st = check_turned(vx, vy, dtype, T, H, D)) != GBB_OK) return st;
  return device_status(launch_norm_rope(a, stream), "rope launch");
}

extern "C" gbb_status gbb_norm_rope(const void* x, int64_t x_token, int64_t x_head, void* y, int64_t y_token,
                                    int64_t y_head, int dtype, int T, int H, int D, const void* weight,
                                    int weight_dtype, float eps, const int32_t* positions, int axes,
                                    const int* sections, const float* table, int n_pos, int rot, int layout,
                                    void* stream) {
  const View vx = {x, x_token, x_head}, vy = {y, y_token, y_head};
  NormRopeArgs a = {x, y, x_token, x_head, y_token, y_head, weight, {}, T, H, D, dtype, eps, true, false,
                    weight_dtype == GBB_F32};
  gbb_status st = check_heads_shape(dtype, T, H, D);
  if (st != GBB_OK || (st = check_strides({vx, vy})) != GBB_OK) return st;
  if ((st = check_norm(weight, weight_dtype, dtype, eps)) != GBB_OK) return st;
  if (T == 0) return GBB_OK;
  if ((st = rotation_of(positions, axes, sections, table, n_pos, D, rot, layout, a.r)) != GBB_OK) return st;
  if ((st = check_turned(vx, vy, dtype, T, H, D)) != GBB_OK) return st;
  return device_status(launch_norm_rope(a, stream), "norm rope launch");
}

extern "C" size_t gbb_norm_rope_grad_workspace(int T, int H, int D) {
  if (check_heads_shape(GBB_F32, T, H, D) != GBB_OK || T == 0) return 0;
  return size_t(norm_rope_grad_rows(T, H)) * D * sizeof(float);
}

extern "C" gbb_status gbb_norm_rope_grad(const void* x, int64_t x_token, int64_t x_head, const void* dy,
                                         int64_t dy_token, int64_t dy_head, void* dx, int64_t dx_token,
                                         int64_t dx_head, int dtype, int T, int H, int D, const void* weight,
                                         int weight_dtype, float eps, const int32_t* positions, int axes,
                                         const int* sections, const float* table, int n_pos, int rot, int layout,
                                         void* dweight, void* workspace, size_t ws_bytes, void* stream) {
  const View vx = {x, x_token, x_head}, vg = {dy, dy_token, dy_head}, vd = {dx, dx_token, dx_head};
  NormRopeGradArgs a = {x, dy, dx, x_token, x_head, dy_token, dy_head, dx_token, dx_head, weight,
                        dweight ? static_cast<float*>(workspace) : nullptr, {}, T, H, D, dtype, eps,
                        weight_dtype == GBB_F32};
  gbb_status st = check_heads_shape(dtype, T, H, D);
  if (st != GBB_OK || (st = check_strides({vx, vg})) != GBB_OK) return st;
  if (dx && (st = check_strides({vd})) != GBB_OK) return st;
  if ((st = check_norm(weight, weight_dtype, dtype, eps)) != GBB_OK) return st;
  if (dweight && weight_dtype != GBB_F32 && weight_dtype != dtype)
    return fail(GBB_E_ARG, "weight_dtype must be GBB_F32 or that of x (%d)", weight_dtype);
  const size_t es = dtype == GBB_F32 ? 4 : 2, ws = weight_dtype == GBB_F32 ? 4 : 2;
  if (!aligned(dweight, ws)) return fail(GBB_E_ALIGN, "dweight is not aligned to its elements");
  if (!dx && !dweight) return GBB_OK;
  if (T > 0) {
    if ((st = rotation_of(positions, axes, sections, table, n_pos, D, rot, layout, a.r)) != GBB_OK) return st;
    if (!x || !dy) return fail(GBB_E_ARG, "x and dy must not be NULL");
    if (!aligned(x, es) || !aligned(dy, es) || !aligned(dx, es)) return fail(GBB_E_ALIGN, "x, dy or dx is not aligned to its elements");
    if (dx) {
      if ((st = check_rows_apart(vd, T, H, D, "dx")) != GBB_OK) return st;
      const size_t n = view_bytes(vd, T, H, D, es);
      if (overlap(x, view_bytes(vx, T, H, D, es), dx, n) ||
          (!same_view(vg, vd, T, H) && overlap(dy, view_bytes(vg, T, H, D, es), dx, n)))
        return fail(GBB_E_ARG, "dx overlaps x or dy");
    }
    if (dweight && (st = check_workspace(workspace, ws_bytes, gbb_norm_rope_grad_workspace(T, H, D))) != GBB_OK) return st;
  }
  return device_status(launch_norm_rope_grad(a, dweight, stream), "norm rope gradient launch");
}

namespace {

gbb_status check_append(const gbb_paged_cache* cache, const void* qkv, int64_t token_stride, int T, int q_heads,
                        const int32_t* slots, const float* table, const void* q) {
  if (!qkv || !q || !slots) return fail(GBB_E_ARG, "qkv, q and slots must not be NULL");
  const int64_t row = (int64_t(q_heads) + 2 * cache->kv_heads) * cache->head_dim;
  if (token_stride < row || token_stride > (int64_t(1) << 40))
    return fail(GBB_E_SHAPE, "token_stride=%lld is below a token's %lld elements", (long long)token_stride, (long long)row);
  if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(table, 16) || !aligned(slots, 4) || token_stride % 8)
    return fail(GBB_E_ALIGN, "qkv, q and table must be 16-byte aligned and token_stride a multiple of 8");
  if (overlap(qkv, (size_t(T - 1) * token_stride + row) * 2, q, size_t(T) * q_heads * cache->head_dim * 2))
    return fail(GBB_E_ARG, "qkv and q overlap");
  return GBB_OK;
}

}  // namespace

extern "C" gbb_status gbb_rope_append(const gbb_paged_cache* cache, const void* qkv, int64_t token_stride, int dtype,
                                      int T, int q_heads, const int32_t* positions, const int32_t* slots,
                                      const float* table, int n_pos, int rot, int layout, void* q, void* stream) {
  gbb_status st = check_cache(cache);
  if (st != GBB_OK) return st;
  if ((st = check_dtype(cache, dtype)) != GBB_OK || (st = check_heads(cache, q_heads)) != GBB_OK) return st;
  if (T < 0) return fail(GBB_E_ARG, "T must not be negative (%d)", T);
  if (T > kMaxTokens) return fail(GBB_E_SHAPE, "T=%d exceeds %d", T, kMaxTokens);
  if (T == 0) return GBB_OK;
  if ((st = check_table(positions, table, n_pos, cache->head_dim, rot, layout)) != GBB_OK) return st;
  if ((st = check_append(cache, qkv, token_stride, T, q_heads, slots, table, q)) != GBB_OK) return st;
  const AppendArgs a = {qkv, q, token_stride, positions, slots, table, T, q_heads, n_pos, rot, layout, dtype};
  return device_status(launch_append(*cache, a, stream), "rope append launch");
}

extern "C" gbb_status gbb_norm_rope_append(const gbb_paged_cache* cache, const void* qkv, int64_t token_stride,
                                           int dtype, int T, int q_heads, const void* q_weight, const void* k_weight,
                                           int weight_dtype, float eps, const int32_t* positions, int axes,
                                           const int* sections, const int32_t* slots, const float* table, int n_pos,
                                           int rot, int layout, void* q, void* stream) {
  gbb_status st = check_cache(cache);
  if (st != GBB_OK) return st;
  if ((st = check_dtype(cache, dtype)) != GBB_OK || (st = check_heads(cache, q_heads)) != GBB_OK) return st;
  if (T < 0) return fail(GBB_E_ARG, "T must not be negative (%d)", T);
  if (T > kMaxTokens) return fail(GBB_E_SHAPE, "T=%d exceeds %d", T, kMaxTokens);
  if (!q_weight != !k_weight) return fail(GBB_E_ARG, "q_weight and k_weight must both be given or both be NULL");
  if ((st = check_norm(q_weight, weight_dtype, dtype, eps)) != GBB_OK) return st;
  if ((st = check_norm(k_weight, weight_dtype, dtype, eps)) != GBB_OK) return st;
  if (T == 0) return GBB_OK;
  NormAppendArgs a = {qkv, q, token_stride, q_weight, k_weight, slots, {}, T, q_heads, dtype, eps, q_weight != nullptr,
                      weight_dtype == GBB_F32};
  if ((st = rotation_of(positions, axes, sections, table, n_pos, cache->head_dim, rot, layout, a.r)) != GBB_OK) return st;
  if ((st = check_append(cache, qkv, token_stride, T, q_heads, slots, table, q)) != GBB_OK) return st;
  return device_status(launch_norm_append(*cache, a, stream), "norm rope append launch");
}

extern "C" size_t gbb_paged_attention_workspace(const gbb_paged_cache* cache, int B, int q_heads, int max_len,
                                                int with_weights) {
  return gbb_paged_attention_options_workspace(cache, B, q_heads, max_len, with_weights, 0);
}

extern "C" size_t gbb_paged_attention_options_workspace(const gbb_paged_cache* cache, int B, int q_heads, int max_len,
                                                        int with_weights, int window) {
  AttendPlan p;
  if (check_attend_shape(cache, B, q_heads, max_len, with_weights != 0, window, p) != GBB_OK || B == 0) return 0;
  return p.ws_bytes;
}

namespace {

gbb_status check_options(const gbb_attention_options& o, float scale, bool tokens) {
  if (!(o.softcap >= 0.f) || !std::isfinite(o.softcap)) return fail(GBB_E_ARG, "softcap must be 0 or more and finite");
  if (o.softcap > 0.f && (o.softcap < 1e-30f || o.softcap > 1e30f || std::fabs(scale) > 1e30 * double(o.softcap)))
    return fail(GBB_E_ARG, "softcap must be 0, or within 1e-30 of the scale and 1e30");
  if (o.window < 0) return fail(GBB_E_ARG, "window must not be negative (%d)", o.window);
  if (!tokens && (o.first || o.prefix || o.tree)) return fail(GBB_E_ARG, "first, prefix and tree are for several tokens");
  if (o.tree && o.prefix) return fail(GBB_E_ARG, "tree and prefix exclude each other");
  if (o.tree && (o.tree_words < 1 || o.tree_words > kMaxTokens / 32))
    return fail(GBB_E_SHAPE, "tree_words=%d must be at least 1 and at most %d", o.tree_words, kMaxTokens / 32);
  if (!aligned(o.slopes, 4) || !aligned(o.first, 4) || !aligned(o.prefix, 4) || !aligned(o.tree, 4))
    return fail(GBB_E_ALIGN, "slopes, first, prefix or tree is misaligned");
  return GBB_OK;
}

}  // namespace

extern "C" gbb_status gbb_paged_attention(const gbb_paged_cache* cache, const void* q, int64_t q_token, int dtype,
                                          int B, int q_heads, const int32_t* block_table, int max_pages,
                                          const int32_t* lengths, int max_len, float scale, void* out, float* lse,
                                          float* weights_out, void* workspace, size_t ws_bytes, void* stream) {
  return gbb_paged_attention_options(cache, q, q_token, dtype, B, q_heads, block_table, max_pages, lengths, max_len,
                                     scale, nullptr, out, lse, weights_out, workspace, ws_bytes, stream);
}

extern "C" gbb_status gbb_paged_attention_options(const gbb_paged_cache* cache, const void* q, int64_t q_token,
                                                  int dtype, int B, int q_heads, const int32_t* block_table,
                                                  int max_pages, const int32_t* lengths, int max_len, float scale,
                                                  const gbb_attention_options* options, void* out, float* lse,
                                                  float* weights_out, void* workspace, size_t ws_bytes, void* stream) {
  static const gbb_attention_options none = {};
  const gbb_attention_options& o = options ? *options : none;
  AttendPlan p;
  gbb_status st = check_options(o, scale, false);
  if (st != GBB_OK) return st;
  const int window = o.window >= max_len ? 0 : o.window;   // no limit
  if ((st = check_attend_shape(cache, B, q_heads, max_len, weights_out != nullptr, window, p)) != GBB_OK) return st;
  if ((st = check_dtype(cache, dtype)) != GBB_OK) return st;
  if ((st = check_sequences(cache, B, block_table, max_pages, lengths, max_len)) != GBB_OK) return st;
  if (!std::isfinite(scale)) return fail(GBB_E_ARG, "scale must be finite");
  if (B == 0) return GBB_OK;
  if (!q || !out) return fail(GBB_E_ARG, "q and out must not be NULL");
  const int64_t row = int64_t(q_heads) * cache->head_dim;
  if (B > 1 && (q_token < row || q_token > (int64_t(1) << 40)))
    return fail(GBB_E_SHAPE, "q_token=%lld is below a token's %lld elements", (long long)q_token, (long long)row);
  if (!aligned(q, 16) || !aligned(out, 16) || (B > 1 && q_token % 8))
    return fail(GBB_E_ALIGN, "q and out must be 16-byte aligned and q_token a multiple of 8");
  if (!aligned(lse, 4) || !aligned(weights_out, 4)) return fail(GBB_E_ALIGN, "lse or weights_out is misaligned");
  if (weights_out && !cache->weights) return fail(GBB_E_ARG, "weights_out needs a cache with weights");
  const size_t n = size_t(cache->num_pages) * cache->kv_heads * cache->page * 4;
  if (weights_out && weights_out != cache->weights && overlap(weights_out, n, cache->weights, n))
    return fail(GBB_E_ARG, "weights_out overlaps the cache's weights in part");
  if (overlap(q, (size_t(B - 1) * q_token + row) * 2, out, size_t(B) * row * 2)) return fail(GBB_E_ARG, "q and out overlap");
  if ((st = check_workspace(workspace, ws_bytes, p.ws_bytes)) != GBB_OK) return st;
  const AttendArgs a = {q, q_token, block_table, lengths, out, lse, weights_out, static_cast<char*>(workspace), B,
                        q_heads, max_pages, max_len, dtype, scale, o.softcap, o.slopes, window};
  return device_status(launch_attend(*cache, a, p, stream), "paged attention launch");
}

namespace {

// A window that no distance reaches is none.  A token of more than its sequence
// has slots lies up to T before the first, so slots of its prefix up to T further.
int tokens_window(int window, int max_len, int T) { return window >= int64_t(max_len) + T ? 0 : window; }

// Shapes alone, for the workspace query (launch sizes included).
gbb_status check_tokens_shape(const gbb_paged_cache* c, int T, int B, int q_heads, int max_len, int window, int tree_words,
                              TokensPlan& p) {
  gbb_status st = check_cache(c);
  if (st != GBB_OK) return st;
  if ((st = check_heads(c, q_heads)) != GBB_OK) return st;
  if (T < 0 || B < 0 || max_len < 1 || max_len > INT_MAX - 8192)
    return fail(GBB_E_ARG, "bad T, B or max_len (%d, %d, %d)", T, B, max_len);
  if (T > kMaxTokens) return fail(GBB_E_SHAPE, "T=%d exceeds %d", T, kMaxTokens);
  if (window < 0 || tree_words < 0 || tree_words > kMaxTokens / 32)
    return fail(GBB_E_ARG, "bad window or tree_words (%d, %d)", window, tree_words);
  if (T && B) {
    p = tokens_plan(*c, T, B, q_heads, max_len, window, tree_words);
    if (int64_t(p.tiles) * c->kv_heads > kMaxGroups / p.nsplit)
      return fail(GBB_E_SHAPE, "T=%d, B=%d, q_heads=%d and max_len=%d make too many workgroups", T, B, q_heads, max_len);
  }
  return GBB_OK;
}

}  // namespace

extern "C" size_t gbb_paged_attention_tokens_workspace(const gbb_paged_cache* cache, int T, int B, int q_heads,
                                                       int max_len, int window, int tree_words) {
  TokensPlan p;
  if (check_tokens_shape(cache, T, B, q_heads, max_len, tokens_window(window, max_len, T), tree_words, p) != GBB_OK ||
      T == 0 || B == 0)
    return 0;
  return p.ws_bytes;
}

extern "C" gbb_status gbb_paged_attention_tokens(const gbb_paged_cache* cache, const void* q, int64_t q_token,
                                                 int dtype, int T, int B, int q_heads, const int32_t* starts,
                                                 const int32_t* block_table, int max_pages, const int32_t* lengths,
                                                 int max_len, float scale, const gbb_attention_options* options,
                                                 void* out, float* lse, void* workspace, size_t ws_bytes,
                                                 void* stream) {
  static const gbb_attention_options none = {};
  const gbb_attention_options& o = options ? *options : none;
  TokensPlan p;
  gbb_status st = check_options(o, scale, true);
  if (st != GBB_OK) return st;
  const int window = tokens_window(o.window, max_len, T), words = o.tree ? o.tree_words : 0;
  if ((st = check_tokens_shape(cache, T, B, q_heads, max_len, window, words, p)) != GBB_OK) return st;
  if ((st = check_dtype(cache, dtype)) != GBB_OK) return st;
  if ((st = check_sequences(cache, B, block_table, max_pages, lengths, max_len)) != GBB_OK) return st;
  if (!(std::fabs(scale) <= 1e30f)) return fail(GBB_E_ARG, "scale must be within -1e30 and 1e30");
  if (T == 0 || B == 0) return GBB_OK;
  if (!q || !out || !starts) return fail(GBB_E_ARG, "q, out and starts must not be NULL");
  const int64_t row = int64_t(q_heads) * cache->head_dim;
  if (T > 1 && (q_token < row || q_token > (int64_t(1) << 40)))
    return fail(GBB_E_SHAPE, "q_token=%lld is below a token's %lld elements", (long long)q_token, (long long)row);
  if (!aligned(q, 16) || !aligned(out, 16) || (T > 1 && q_token % 8))
    return fail(GBB_E_ALIGN, "q and out must be 16-byte aligned and q_token a multiple of 8");
  if (!aligned(lse, 4) || !aligned(starts, 4)) return fail(GBB_E_ALIGN, "lse or starts is misaligned");
  if (overlap(q, (size_t(T - 1) * (T > 1 ? q_token : 0) + row) * 2, out, size_t(T) * row * 2))
    return fail(GBB_E_ARG, "q and out overlap");
  if ((st = check_workspace(workspace, ws_bytes, p.ws_bytes)) != GBB_OK) return st;
  const TokensArgs a = {q, q_token, starts, block_table, lengths, o.first, o.prefix, o.tree, out, lse,
                        static_cast<char*>(workspace), T, B, q_heads, max_pages, max_len, dtype, words, window, scale,
                        o.softcap, o.slopes};
  return device_status(launch_tokens(*cache, a, p, stream), "paged attention of tokens launch");
}

extern "C" gbb_status gbb_cache_keep(const gbb_paged_cache* cache, int B, const int32_t* block_table, int max_pages,
                                     const int32_t* lengths, const int32_t* drafted, const int32_t* kept, int max_kept,
                                     const int32_t* counts, int32_t* lengths_out, void* stream) {
  gbb_status st = check_cache(cache);
  if (st != GBB_OK) return st;
  if (B < 0 || max_pages < 1 || max_kept < 0) return fail(GBB_E_ARG, "bad B, max_pages or max_kept (%d, %d, %d)", B, max_pages, max_kept);
  if (int64_t(B) * cache->kv_heads > kMaxGroups)
    return fail(GBB_E_SHAPE, "B=%d and kv_heads=%d make too many workgroups", B, cache->kv_heads);
  if (B == 0) return GBB_OK;
  if (!block_table || !lengths || !drafted || !counts || !lengths_out || (max_kept && !kept))
    return fail(GBB_E_ARG, "block_table, lengths, drafted, kept, counts and lengths_out must not be NULL");
  if (!aligned(block_table, 4) || !aligned(lengths, 4) || !aligned(drafted, 4) || !aligned(kept, 4) || !aligned(counts, 4) ||
      !aligned(lengths_out, 4))
    return fail(GBB_E_ALIGN, "block_table, lengths, drafted, kept, counts or lengths_out is misaligned");
  const size_t n = size_t(B) * 4;
  if (overlap(lengths_out, n, lengths, n) || overlap(lengths_out, n, drafted, n) || overlap(lengths_out, n, counts, n) ||
      overlap(lengths_out, n, kept, n * max_kept) || overlap(lengths_out, n, block_table, n * max_pages))
    return fail(GBB_E_ARG, "lengths_out overlaps an input");
  const KeepArgs a = {block_table, lengths, drafted, kept, counts, lengths_out, B, max_pages, max_kept};
  return device_status(launch_keep(*cache, a, stream), "cache keep launch");
}

extern "C" size_t gbb_cache_evict_workspace(const gbb_paged_cache* cache, int B, int max_len, int budget) {
  if (check_evict_shape(cache, B, max_len, budget) != GBB_OK || B == 0) return 0;
  return evict_plan(*cache, B, max_len, budget).ws_bytes;
}

extern "C" gbb_status gbb_cache_evict(const gbb_paged_cache* cache, int B, const int32_t* block_table, int max_pages,
                                      const int32_t* lengths, int max_len, int budget, int recent,
                                      int32_t* lengths_out, float* weights_out, int32_t* positions_out,
                                      void* workspace, size_t ws_bytes, void* stream) {
  gbb_status st = check_evict_shape(cache, B, max_len, budget);
  if (st != GBB_OK) return st;
  if ((st = check_sequences(cache, B, block_table, max_pages, lengths, max_len)) != GBB_OK) return st;
  if (recent < 0 || recent > budget) return fail(GBB_E_ARG, "recent=%d outside [0, budget=%d]", recent, budget);
  if (!cache->weights || !cache->positions) return fail(GBB_E_ARG, "eviction needs a cache with weights and positions");
  if (B == 0) return GBB_OK;
  if (!lengths_out || !weights_out || !positions_out)
    return fail(GBB_E_ARG, "lengths_out, weights_out and positions_out must not be NULL");
  if (!aligned(lengths_out, 4) || !aligned(weights_out, 4) || !aligned(positions_out, 4))
    return fail(GBB_E_ALIGN, "lengths_out, weights_out or positions_out is misaligned");
  if (overlap(lengths, size_t(B) * 4, lengths_out, size_t(B) * 4)) return fail(GBB_E_ARG, "lengths and lengths_out overlap");
  const size_t n = size_t(cache->num_pages) * cache->kv_heads * cache->page * 4;
  if ((weights_out != cache->weights && overlap(weights_out, n, cache->weights, n)) ||
      (positions_out != cache->positions && overlap(positions_out, n, cache->positions, n)))
    return fail(GBB_E_ARG, "weights_out or positions_out overlaps the cache's in part");
  const EvictPlan p = evict_plan(*cache, B, max_len, budget);
  if ((st = check_workspace(workspace, ws_bytes, p.ws_bytes)) != GBB_OK) return st;
  const EvictArgs a = {block_table, lengths, lengths_out, weights_out, positions_out, static_cast<char*>(workspace), B,
                       max_pages, max_len, budget, recent};
  return device_status(launch_evict(*cache, a, p, stream), "cache evict launch");
}
