// Eviction from a paged cache by accumulated attention weight
// (gbb_cache_evict).
//
// For a (sequence, kv head) with n slots, `budget` of them stay: a selection
// of the budget largest of n 32-bit keys (a weight's bits in an order that
// compares as unsigned, the newest positions above all of them), with ties
// to the lower slot.  Attention over rotated keys does not depend on the
// order of slots, so the kept slots above the new length fill the holes
// below it and nothing else moves: 4 bytes of weight and position in and out
// a slot, and 2 rows read and written a moved slot, are what it takes.
//
// The first launch selects, one workgroup a (sequence, kv head): the key of
// the budget-th slot is found 8 bits at a time from histograms in LDS, then
// one pass in slot order lists holes and the slots that fill them, and
// weights and positions follow.  The second launch moves the rows of k and
// v, over as many workgroups as the rows give.
#include <algorithm>

#include "device.h"
#include "internal.h"

namespace gbb {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;

struct SelectArgs {
  const int32_t* block_table;
  const int32_t* lengths;
  int32_t* lengths_out;
  const float* weights;
  const int32_t* positions;
  float* weights_out;
  int32_t* positions_out;
  int32_t* count;    // [B Hkv] rows to move
  int32_t* dst;      // [B Hkv][most] slots, ascending
  int32_t* src;
  uint32_t* keys;    // [B Hkv][key_stride]
  size_t key_stride, most;
  int Hkv, num_pages, pshift, max_pages, max_len, budget, recent;
};

__device__ __forceinline__ uint32_t rank_of(float w) {
  if (w != w) return 0;
  const uint32_t u = __builtin_bit_cast(uint32_t, w + 0.f);   // -0 ranks as 0
  return u >> 31 ? ~u : u | 0x80000000u;
}

// Sum over the workgroup's threads before this one; total: over all.
__device__ __forceinline__ int scan(int x, int* lds, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = x;
#pragma unroll
  for (int k = 1; k < 64; k *= 2) {
    const int o = __shfl_up(s, k);
    if (lane >= k) s += o;
  }
  if (lane == 63) lds[wave] = s;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int t = lds[w];
    before += w < wave ? t : 0;
    total += t;
  }
  __syncthreads();
  return before + s - x;
}

__global__ __launch_bounds__(kThreads) void select_kernel(SelectArgs a) {
  __shared__ int lds[kWaves];
  __shared__ unsigned hist[256];
  __shared__ unsigned chosen[2];
  const int tid = threadIdx.x, pair = blockIdx.x, hk = pair % a.Hkv, b = pair / a.Hkv;
  const int len = max(0, min(a.lengths[b], a.max_len));
  const int32_t* table = a.block_table + size_t(b) * a.max_pages;
  const int pages = (len + (1 << a.pshift) - 1) >> a.pshift;
  int bad = 0;
  for (int i = tid; i < pages; i += kThreads) bad |= unsigned(table[i]) >= unsigned(a.num_pages);
  bad = __syncthreads_or(bad);
  const int stay = bad ? len : min(len, a.budget);
  if (tid == 0 && hk == 0) a.lengths_out[b] = stay;
  if (tid == 0) a.count[pair] = 0;
  if (bad) return;
  // weights and positions of slot j of this head
  const auto at = [&](int j) {
    return ((size_t(table[j >> a.pshift]) * a.Hkv + hk) << a.pshift) + (j & ((1 << a.pshift) - 1));
  };
  const bool other = a.weights_out != a.weights || a.positions_out != a.positions;
  if (stay == len) {
    if (other)
      for (int j = tid; j < len; j += kThreads) {
        const size_t x = at(j);
        a.weights_out[x] = a.weights[x];
        a.positions_out[x] = a.positions[x];
      }
    return;
  }

  int newest = INT32_MIN;
  for (int j = tid; j < len; j += kThreads) newest = max(newest, a.positions[at(j)]);
#pragma unroll
  for (int k = 1; k < 64; k *= 2) newest = max(newest, __shfl_xor(newest, k));
  if ((tid & 63) == 0) lds[tid >> 6] = newest;
  __syncthreads();
  for (int w = 0; w < kWaves; ++w) newest = max(newest, lds[w]);
  const int64_t old = int64_t(newest) - a.recent;   // positions above it are kept first

  uint32_t* keys = a.keys + size_t(pair) * a.key_stride;
  for (int j = tid; j < len; j += kThreads) {
    const size_t x = at(j);
    keys[j] = int64_t(a.positions[x]) > old ? 0xffffffffu : rank_of(a.weights[x]);
  }

  // the budget-th largest key, and how many equal to it stay
  uint32_t prefix = 0, mask = 0;
  unsigned need = unsigned(a.budget);
  for (int shift = 24; shift >= 0; shift -= 8) {
    __syncthreads();
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int j = tid; j < len; j += kThreads) {
      const uint32_t k = keys[j];
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1u);
    }
    __syncthreads();
    if (tid < 64) {   // lane i: digits 255 - 4 i ... 252 - 4 i
      unsigned n[4], s = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) s += n[k] = hist[255 - 4 * tid - k];
      unsigned upto = s;
#pragma unroll
      for (int k = 1; k < 64; k *= 2) {
        const unsigned o = __shfl_up(upto, k);
        if (tid >= k) upto += o;
      }
      unsigned above = upto - s;
      if (above < need && upto >= need) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (above < need && above + n[k] >= need) {
            chosen[0] = 255 - 4 * tid - k;
            chosen[1] = need - above;
          }
          above += n[k];
        }
      }
    }
    __syncthreads();
    prefix |= chosen[0] << shift;
    need = chosen[1];
    mask |= 255u << shift;
  }

  // in slot order: what stays, the holes below the new length, and the kept
  // slots from it on
  int32_t* dst = a.dst + size_t(pair) * a.most;
  int32_t* src = a.src + size_t(pair) * a.most;
  int equal = 0, holes = 0, fills = 0;
  for (int j0 = 0; j0 < len; j0 += kThreads) {
    const int j = j0 + tid;
    const uint32_t k = j < len ? keys[j] : 0;
    const bool eq = j < len && k == prefix;
    int total;
    const int rank = equal + scan(eq, lds, total);
    equal += total;
    const bool kept = j < len && (k > prefix || (eq && unsigned(rank) < need));
    const bool hole = j < stay && !kept, fill = j >= stay && kept;
    int both;
    const int before = scan(int(hole) | int(fill) << 16, lds, both);
    if (hole) dst[holes + (before & 0xffff)] = j;
    if (fill) src[fills + (before >> 16)] = j;
    holes += both & 0xffff;
    fills += both >> 16;
    if (other && j < stay) {
      const size_t x = at(j);
      a.weights_out[x] = a.weights[x];
      a.positions_out[x] = a.positions[x];
    }
  }
  if (tid == 0) a.count[pair] = holes;
  __syncthreads();
  for (int i = tid; i < holes; i += kThreads) {
    const size_t to = at(dst[i]), from = at(src[i]);
    a.weights_out[to] = a.weights[from];
    a.positions_out[to] = a.positions[from];
  }
  __syncthreads();
  for (int j = stay + tid; j < len; j += kThreads) {
    const size_t x = at(j);
    a.weights_out[x] = 0.f;
    a.positions_out[x] = -1;
  }
}

struct MoveArgs {
  uint8_t* k;
  uint8_t* v;
  const int32_t* block_table;
  const int32_t* count;
  const int32_t* dst;
  const int32_t* src;
  size_t most;
  int Hkv, pshift, max_pages, lshift;   // lshift: log2 of 16-byte pieces a row
};

// 16 bytes of k and of v a thread.  No row is both a source and a target, so
// the order of the moves is free.
__global__ __launch_bounds__(256) void move_kernel(MoveArgs a) {
  const int pair = blockIdx.x, hk = pair % a.Hkv, b = pair / a.Hkv;
  const int n = a.count[pair];
  const int32_t* table = a.block_table + size_t(b) * a.max_pages;
  const int piece = threadIdx.x & ((1 << a.lshift) - 1), per = 256 >> a.lshift;
  const auto at = [&](int j) {
    const size_t row = ((size_t(table[j >> a.pshift]) * a.Hkv + hk) << a.pshift) + (j & ((1 << a.pshift) - 1));
    return ((row << a.lshift) + piece) * 16;
  };
  for (int i = blockIdx.y * per + (threadIdx.x >> a.lshift); i < n; i += gridDim.y * per) {
    const size_t to = at(a.dst[pair * a.most + i]), from = at(a.src[pair * a.most + i]);
    const u32x4 x = ld16(a.k + from), y = ld16(a.v + from);
    st16(a.k + to, x);
    st16(a.v + to, y);
  }
}

size_t up(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

EvictPlan evict_plan(const gbb_paged_cache& c, int B, int max_len, int budget) {
  EvictPlan p;
  const size_t pairs = size_t(B) * c.kv_heads;
  p.key_stride = (size_t(max_len) + 63) & ~size_t(63);
  p.most = size_t(std::max(0, std::min(budget, max_len - budget)));
  p.count_off = 0;
  p.dst_off = up(pairs * 4);
  p.src_off = p.dst_off + up(pairs * p.most * 4);
  p.key_off = p.src_off + up(pairs * p.most * 4);
  p.ws_bytes = p.key_off + up(pairs * p.key_stride * 4);
  return p;
}

int launch_evict(const gbb_paged_cache& c, const EvictArgs& x, const EvictPlan& p, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  SelectArgs a;
  a.block_table = x.block_table;
  a.lengths = x.lengths;
  a.lengths_out = x.lengths_out;
  a.weights = c.weights;
  a.positions = c.positions;
  a.weights_out = x.weights_out;
  a.positions_out = x.positions_out;
  a.count = reinterpret_cast<int32_t*>(x.ws + p.count_off);
  a.dst = reinterpret_cast<int32_t*>(x.ws + p.dst_off);
  a.src = reinterpret_cast<int32_t*>(x.ws + p.src_off);
  a.keys = reinterpret_cast<uint32_t*>(x.ws + p.key_off);
  a.key_stride = p.key_stride;
  a.most = p.most;
  a.Hkv = c.kv_heads;
  a.num_pages = c.num_pages;
  a.pshift = __builtin_ctz(unsigned(c.page));
  a.max_pages = x.max_pages;
  a.max_len = x.max_len;
  a.budget = x.budget;
  a.recent = x.recent;
  const unsigned pairs = unsigned(x.B) * c.kv_heads;
  hipLaunchKernelGGL(select_kernel, dim3(pairs), dim3(kThreads), 0, s, a);
  if (p.most) {
    MoveArgs m;
    m.k = static_cast<uint8_t*>(c.k);
    m.v = static_cast<uint8_t*>(c.v);
    m.block_table = x.block_table;
    m.count = a.count;
    m.dst = a.dst;
    m.src = a.src;
    m.most = p.most;
    m.Hkv = c.kv_heads;
    m.pshift = a.pshift;
    m.max_pages = x.max_pages;
    m.lshift = __builtin_ctz(unsigned(c.head_dim * (c.dtype == GBB_E4M3 ? 1 : 2) / 16));
    const size_t per = 256 >> m.lshift;
    const unsigned gy = unsigned(std::min<size_t>((p.most + per - 1) / per, std::max(1u, 4096u / pairs)));
    hipLaunchKernelGGL(move_kernel, dim3(pairs, gy), dim3(256), 0, s, m);
  }
  return int(hipGetLastError());
}

}  // namespace gbb
