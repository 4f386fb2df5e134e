// C-ABI entry points of the rotary positions and the paged cache: argument
// checks, workspace sizes and launches.  No allocation, no synchronization.
#include <climits>
#include <cmath>
#include <cstdint>

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
gbb_status check_attend_shape(const gbb_paged_cache* c, int B, int q_heads, int max_len, bool with_weights, AttendPlan& p) {
  gbb_status st = check_cache(c);
  if (st != GBB_OK) return st;
  if ((st = check_heads(c, q_heads)) != GBB_OK) return st;
  if (B < 0 || max_len < 1 || max_len > INT_MAX - 8192) return fail(GBB_E_ARG, "bad B or max_len (%d, %d)", B, max_len);
  if (int64_t(B) * q_heads > kMaxGroups) return fail(GBB_E_SHAPE, "B * q_heads exceeds %d", int(kMaxGroups));
  if (B) {
    p = attend_plan(*c, B, q_heads, max_len, with_weights);
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

}  // namespace

extern "C" gbb_status gbb_rope(const void* x, int64_t x_token, int64_t x_head, void* y, int64_t y_token,
                               int64_t y_head, int dtype, int T, int H, int D, const int32_t* positions,
                               const float* table, int n_pos, int rot, int layout, int transpose, void* stream) {
  if (dtype != GBB_F16 && dtype != GBB_BF16 && dtype != GBB_F32) return fail(GBB_E_ARG, "unknown dtype %d", dtype);
  if (T < 0 || H <= 0 || D <= 0) return fail(GBB_E_ARG, "T, H or D is negative or zero (%d, %d, %d)", T, H, D);
  if (D % 2 || D > 1024) return fail(GBB_E_SHAPE, "D=%d must be even and at most 1024", D);
  if (T > kMaxTokens || H > kMaxHeads) return fail(GBB_E_SHAPE, "T=%d or H=%d exceeds %d, %d", T, H, kMaxTokens, kMaxHeads);
  const int64_t big = int64_t(1) << 40;
  if (x_token < 0 || x_head < 0 || y_token < 0 || y_head < 0 || x_token > big || x_head > big || y_token > big || y_head > big)
    return fail(GBB_E_ARG, "a stride is negative or above 2^40");
  if (T == 0) return GBB_OK;
  const gbb_status st = check_table(positions, table, n_pos, D, rot, layout);
  if (st != GBB_OK) return st;
  if (!x || !y) return fail(GBB_E_ARG, "x and y must not be NULL");
  const size_t es = dtype == GBB_F32 ? 4 : 2;
  if (!aligned(x, es) || !aligned(y, es)) return fail(GBB_E_ALIGN, "x or y is not aligned to its elements");
  // y's rows must be memory of their own, a token's heads or a head's tokens
  // together; x's may repeat (a broadcast input)
  const auto apart = [&](int64_t inner, int ni, int64_t outer, int no) {
    return (ni == 1 || inner >= D) && (no == 1 || outer >= (ni - 1) * inner + D);
  };
  if (!apart(y_head, H, y_token, T) && !apart(y_token, T, y_head, H))
    return fail(GBB_E_SHAPE, "y's strides %lld, %lld make its heads overlap", (long long)y_token, (long long)y_head);
  const size_t nx = (size_t(T - 1) * x_token + size_t(H - 1) * x_head + D) * es;
  const size_t ny = (size_t(T - 1) * y_token + size_t(H - 1) * y_head + D) * es;
  const bool in_place = x == y && (T == 1 || x_token == y_token) && (H == 1 || x_head == y_head);
  if (!in_place && overlap(x, nx, y, ny)) return fail(GBB_E_ARG, "x and y overlap");
  const RopeArgs a = {x, y, x_token, x_head, y_token, y_head, positions, table, T, H, D, n_pos, rot, layout,
                      transpose, dtype};
  return device_status(launch_rope(a, stream), "rope launch");
}

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
  if (!qkv || !q || !slots) return fail(GBB_E_ARG, "qkv, q and slots must not be NULL");
  const int64_t row = (int64_t(q_heads) + 2 * cache->kv_heads) * cache->head_dim;
  if (token_stride < row || token_stride > (int64_t(1) << 40))
    return fail(GBB_E_SHAPE, "token_stride=%lld is below a token's %lld elements", (long long)token_stride, (long long)row);
  if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(table, 16) || !aligned(slots, 4) || token_stride % 8)
    return fail(GBB_E_ALIGN, "qkv, q and table must be 16-byte aligned and token_stride a multiple of 8");
  if (overlap(qkv, (size_t(T - 1) * token_stride + row) * 2, q, size_t(T) * q_heads * cache->head_dim * 2))
    return fail(GBB_E_ARG, "qkv and q overlap");
  const AppendArgs a = {qkv, q, token_stride, positions, slots, table, T, q_heads, n_pos, rot, layout, dtype};
  return device_status(launch_append(*cache, a, stream), "rope append launch");
}

extern "C" size_t gbb_paged_attention_workspace(const gbb_paged_cache* cache, int B, int q_heads, int max_len,
                                                int with_weights) {
  AttendPlan p;
  if (check_attend_shape(cache, B, q_heads, max_len, with_weights != 0, p) != GBB_OK || B == 0) return 0;
  return p.ws_bytes;
}

extern "C" gbb_status gbb_paged_attention(const gbb_paged_cache* cache, const void* q, int64_t q_token, int dtype,
                                          int B, int q_heads, const int32_t* block_table, int max_pages,
                                          const int32_t* lengths, int max_len, float scale, void* out, float* lse,
                                          float* weights_out, void* workspace, size_t ws_bytes, void* stream) {
  AttendPlan p;
  gbb_status st = check_attend_shape(cache, B, q_heads, max_len, weights_out != nullptr, p);
  if (st != GBB_OK) return st;
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
                        q_heads, max_pages, max_len, dtype, scale};
  return device_status(launch_attend(*cache, a, p, stream), "paged attention launch");
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
