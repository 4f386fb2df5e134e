// What is left of drafted tokens in a paged cache (gbb_cache_keep): the kept
// ones of a sequence's newest slots move to the front of them.
//
// Row i of the kept ones goes from slot ctx + kept[i] to slot ctx + i, and kept
// rises, so kept[i] >= i: rows are moved some at a time in their order, all of
// them read before any is written, and no later row's source has been
// overwritten by then.  One workgroup a (sequence, kv head), 16 bytes a thread
// and step; k, v and what is tracked in the same launch.  A call of usual size
// takes 4 bytes moved an element of a few hundred rows: the chain of dependent
// steps (counts, kept ones, pages, rows, writes) is what it takes.
#include <algorithm>

#include "device.h"
#include "internal.h"

namespace gbb {

namespace {

constexpr int kAhead = 4;   // pieces a thread holds at once

__global__ __launch_bounds__(256) void keep_kernel(gbb_paged_cache c, KeepArgs a, int row_bytes) {
  const int hk = blockIdx.x % c.kv_heads, b = blockIdx.x / c.kv_heads;
  const int len = a.lengths[b], n = a.drafted[b], count = a.counts[b];
  const int32_t* kept = a.kept + size_t(b) * a.max_kept;
  const int32_t* table = a.block_table + size_t(b) * a.max_pages;
  const int page = c.page, ctx = len - n;
  bool good = len >= 0 && len <= int64_t(a.max_pages) * page && n >= 0 && n <= len && count >= 0 && count <= n && count <= a.max_kept;
  const auto page_of = [&](int slot) { return table[slot / page]; };
  if (good)
    for (int i = threadIdx.x; i < count; i += 256) {
      const int s = kept[i];
      good = good && s >= 0 && s < n && (i == 0 || s > kept[i - 1]);
      if (good) good = unsigned(page_of(ctx + i)) < unsigned(c.num_pages) && unsigned(page_of(ctx + s)) < unsigned(c.num_pages);
    }
  good = __syncthreads_and(good);
  if (hk == 0 && threadIdx.x == 0) a.lengths_out[b] = good ? ctx + count : len;
  if (!good) return;
  // pieces of a row: k's, v's, then its weight and position
  const int pieces = row_bytes / 16, items = 2 * pieces + 1;
  const int rows = std::max(1, kAhead * 256 / items);
  const auto at = [&](int slot) { return (size_t(page_of(slot)) * c.kv_heads + hk) * page + slot % page; };
  for (int i0 = 0; i0 < count; i0 += rows) {
    const int end = min(count, i0 + rows) - i0;
    u32x4 x[kAhead];
    const auto each = [&](auto f) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int item = threadIdx.x + 256 * u, i = item / items, piece = item % items;
        if (i < end && kept[i0 + i] != i0 + i) f(x[u], i0 + i, piece);
      }
    };
    const auto place = [&](size_t row, int piece) {
      return static_cast<char*>(piece < pieces ? c.k : c.v) + row * row_bytes + (piece < pieces ? piece : piece - pieces) * 16;
    };
    each([&](u32x4& v, int i, int piece) {
      const size_t from = at(ctx + kept[i]);
      if (piece < 2 * pieces) {
        v = ld16(place(from, piece));
      } else {
        if (c.weights) v[0] = __builtin_bit_cast(uint32_t, c.weights[from]);
        if (c.positions) v[1] = uint32_t(c.positions[from]);
      }
    });
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // read before any thread writes
    __syncthreads();
    each([&](u32x4& v, int i, int piece) {
      const size_t to = at(ctx + i);
      if (piece < 2 * pieces) {
        st16(place(to, piece), v);
      } else {
        const uint32_t weight = v[0];
        if (c.weights) c.weights[to] = __builtin_bit_cast(float, weight);
        if (c.positions) c.positions[to] = int32_t(v[1]);
      }
    });
  }
}

}  // namespace

int launch_keep(const gbb_paged_cache& c, const KeepArgs& a, void* stream) {
  const int row_bytes = c.head_dim * (c.dtype == GBB_E4M3 ? 1 : 2);
  start(keep_kernel, dim3(unsigned(a.B) * unsigned(c.kv_heads)), dim3(256), static_cast<hipStream_t>(stream), c, a, row_bytes);
  return int(hipGetLastError());
}

}  // namespace gbb
