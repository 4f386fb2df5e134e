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
// One workgroup of 16 waves selects for a (sequence, kv head): the threads
// hold the keys in registers, 4 slots to a load (rows above 32768 slots are
// spread over workgroups and launches instead), the budget-th largest is
// found 11 bits at a time from histograms in LDS, and ranks in slot order are
// prefix sums of each thread's counts.  Where few rows can move, as in a
// cache that is one token over its budget, the same workgroup moves them;
// else a second launch moves rows and writes weights and positions over as
// many workgroups as the slots give.
//
// Measured (GPU time): 256 pairs of 2049 slots cut by one 6.7 us, of which
// about 4.5 are the chain of dependent steps in a workgroup (page, load, newest
// position, smallest key, places, move); 16 pairs of 32768 slots of 128
// fp16 elements cut to 4096 34 us: 20 in the selection, where 16 of the 256
// CUs have work (4 of it the row's loads, the rest some 30 instructions a key),
// and 15 in the moves (4 TB/s).
#include <algorithm>
#include <type_traits>

#include "device.h"
#include "internal.h"

namespace gbb {

namespace {

constexpr int kMaxHeld = 32 * 1024;   // slots a row whose keys a workgroup's registers hold
constexpr int kOneByOne = 4;          // slots that are found one by one
constexpr int kFew = 64;               // rows that the selecting workgroup moves itself

struct EvictKernelArgs {
  const int32_t* block_table;
  const int32_t* lengths;
  int32_t* lengths_out;
  const float* weights;
  const int32_t* positions;
  float* weights_out;
  int32_t* positions_out;
  uint8_t* k;
  uint8_t* v;
  int32_t* count;    // [B Hkv] rows to move, -1: the sequence is left as it is
  uint64_t* dst;     // [B Hkv][most] places (Slots), in the order of slots
  uint64_t* src;
  uint32_t* keys;    // [B Hkv][key_stride], for spread rows
  uint8_t* flags;    // [B Hkv][key_stride / 4]: which of 4 slots are kept, a bit each
  size_t key_stride, most;
  int Hkv, num_pages, pshift, max_pages, max_len, budget, recent, lshift;
  bool other;        // weights_out and positions_out are not the cache's own
};

__device__ __forceinline__ uint32_t rank_of(float w) {
  if (w != w) return 0;
  const uint32_t u = __builtin_bit_cast(uint32_t, w + 0.f);   // -0 ranks as 0
  return u >> 31 ? ~u : u | 0x80000000u;
}

// Sum over the workgroup's threads before this one; total: over all.
template <int WAVES>
__device__ __forceinline__ uint32_t scan(uint32_t x, uint32_t* lds, uint32_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t s = x;
#pragma unroll
  for (int k = 1; k < 64; k *= 2) {
    const uint32_t o = __shfl_up(s, k);
    if (lane >= k) s += o;
  }
  if (lane == 63) lds[wave] = s;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const uint32_t t = lds[w];
    before += w < wave ? t : 0;
    total += t;
  }
  __syncthreads();
  return before + s - x;
}

// Where slot j of a (sequence, kv head) is, in slots of the weights and
// positions and in rows of k and v.
struct Slots {
  const int32_t* table;
  int hk, Hkv, pshift;
  __device__ __forceinline__ size_t operator()(int j) const {
    return ((size_t(table[j >> pshift]) * Hkv + hk) << pshift) + (j & ((1 << pshift) - 1));
  }
};

// One move between two places: 16 bytes of k and of v a thread (`piece` of
// the row), and with the first piece its weight and position.  No place is
// both a source and a target, so the order of the moves is free.
__device__ __forceinline__ void move_row(const EvictKernelArgs& a, uint64_t to, uint64_t from, int piece) {
  const size_t x = ((from << a.lshift) + piece) * 16, y = ((to << a.lshift) + piece) * 16;
  const u32x4 kk = ld16(a.k + x), vv = ld16(a.v + x);
  st16(a.k + y, kk);
  st16(a.v + y, vv);
  if (piece == 0) {
    a.weights_out[to] = a.weights[from];
    a.positions_out[to] = a.positions[from];
    a.weights_out[from] = 0.f;
    a.positions_out[from] = -1;
  }
}

// Slot j that does not move: copied to other memory where it stays, cleared
// where it lies above the new length.
__device__ __forceinline__ void settle(const EvictKernelArgs& a, const Slots& at, int j, int stay, bool kept) {
  if (j < stay ? !(a.other && kept) : kept) return;
  const size_t x = at(j);
  a.weights_out[x] = j < stay ? a.weights[x] : 0.f;
  a.positions_out[x] = j < stay ? a.positions[x] : -1;
}

constexpr int kThreads = 1024, kWaves = 16;
constexpr int kBins[3] = {2048, 2048, 1024};   // digits of 11, 11 and 10 bits
constexpr int kShift[3] = {21, 10, 0};
// Words a bin of the first digit has in select_kernel, a lane's by its number:
// weights crowd a few exponents, and additions to one word go one by one (16
// pairs of 32768: 20.1 us; 20.6 with 2 words, 20.9 with 8).
constexpr int kCopies = 4;

// Inclusive sum over the wave's lanes up to this one.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);   // row_shr 1, 2, 4, 8: within 16 lanes
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);   // row_bcast 15 into rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);   // row_bcast 31 into rows 2 and 3
  return x;
}
// The least of the wave's values, in all lanes.
__device__ __forceinline__ uint32_t wave_least(uint32_t x) {
  x = min(x, uint32_t(__builtin_amdgcn_update_dpp(-1, x, 0x111, 0xf, 0xf, false)));
  x = min(x, uint32_t(__builtin_amdgcn_update_dpp(-1, x, 0x112, 0xf, 0xf, false)));
  x = min(x, uint32_t(__builtin_amdgcn_update_dpp(-1, x, 0x114, 0xf, 0xf, false)));
  x = min(x, uint32_t(__builtin_amdgcn_update_dpp(-1, x, 0x118, 0xf, 0xf, false)));
  x = min(x, uint32_t(__builtin_amdgcn_update_dpp(-1, x, 0x142, 0xa, 0xf, false)));
  x = min(x, uint32_t(__builtin_amdgcn_update_dpp(-1, x, 0x143, 0xc, 0xf, false)));
  return uint32_t(__builtin_amdgcn_readlane(int(x), 63));
}
// The largest of the wave's signed values: the order of complements with the
// sign bit as a digit.
__device__ __forceinline__ int wave_largest(int x) { return int(~wave_least(~(uint32_t(x) ^ 0x80000000u)) ^ 0x80000000u); }
__device__ __forceinline__ uint32_t lane_of(uint32_t x, int lane) {
  return uint32_t(__builtin_amdgcn_readlane(int(x), lane));
}

template <int COPIES>
__device__ __forceinline__ uint32_t bin(const uint32_t* hist, int i) {
  uint32_t s = 0;
#pragma unroll
  for (int c = 0; c < COPIES; ++c) s += hist[i * COPIES + c];
  return s;
}

// The digit that holds the need-th largest entry of a histogram, in every
// wave: sums of 16 groups of bins first, then the bins of one group.  After:
// need is the rank within the digit.  Each bin is the sum of COPIES words.
template <int BINS, int COPIES = 1>
__device__ __forceinline__ uint32_t find_digit(const uint32_t* hist, uint32_t* sums, uint32_t& need, int lane, int wave) {
  constexpr int G = BINS / kWaves, N = G / 64;   // bins a group, bins a lane
  uint32_t s = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) s += bin<COPIES>(hist, wave * G + lane * N + i);
  s = wave_scan(s);
  if (lane == 63) sums[wave] = s;
  __syncthreads();
  const uint32_t g = lane < kWaves ? sums[kWaves - 1 - lane] : 0;
  const uint32_t ig = wave_scan(g);
  const int l = __builtin_ctzll(__ballot(ig >= need));
  const int group = kWaves - 1 - l;
  need -= lane_of(ig, l) - lane_of(g, l);
  // lane i: bins from the group's top down
  uint32_t h[N], sum = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) sum += h[i] = bin<COPIES>(hist, group * G + G - 1 - lane * N - i);
  const uint32_t is = wave_scan(sum);
  const int at = __builtin_ctzll(__ballot(is >= need));
  need -= lane_of(is, at) - lane_of(sum, at);
  int i = 0;
#pragma unroll
  for (int k = 0; k + 1 < N; ++k) {
    const uint32_t n = lane_of(h[k], at);
    if (i == k && n < need) {
      need -= n;
      i = k + 1;
    }
  }
  return uint32_t(group * G + G - 1 - at * N - i);
}

// A sequence that is not over its budget, or lacks a page, stays as it is: in
// other memory its weights and positions are copied (if its pages are there).
__device__ __forceinline__ bool missing(const EvictKernelArgs& a, const Slots& at, int len) {
  const int pages = (len + (1 << a.pshift) - 1) >> a.pshift;
  bool bad = false;
  for (int i = threadIdx.x; i < pages; i += kThreads) bad |= unsigned(at.table[i]) >= unsigned(a.num_pages);
  return __syncthreads_or(bad);
}
__device__ __forceinline__ void leave(const EvictKernelArgs& a, const Slots& at, int pair, int hk, int b, int len, bool finish) {
  if (threadIdx.x == 0 && hk == 0) a.lengths_out[b] = len;
  if (threadIdx.x == 0 && !finish) a.count[pair] = -1;
  if (a.other && !missing(a, at, len))
    for (int j = threadIdx.x; j < len; j += kThreads) settle(a, at, j, len, true);
}

// NB: runs of 4 slots a thread, up to 4096 NB slots a row: slot
// 4096 i + 4 tid + e is element e of thread tid's run i (pages hold whole
// runs).  FINISH: this launch moves the rows too (at most kFew).
template <int NB, bool FINISH>
__global__ __launch_bounds__(kThreads) void select_kernel(EvictKernelArgs a) {
  __shared__ __align__(16) uint32_t hist[kCopies * kBins[0] + kBins[1] + kBins[2]];
  __shared__ uint32_t sums[3][kWaves], counts[2][NB * kWaves];
  __shared__ int tops[kWaves];
  __shared__ uint64_t leasts[2][kWaves];
  __shared__ uint64_t few[2][kFew];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int pair = blockIdx.x, hk = pair % a.Hkv, b = pair / a.Hkv;
  const int len = max(0, min(a.lengths[b], a.max_len));
  const int stay = a.budget;
  const Slots at = {a.block_table + size_t(b) * a.max_pages, hk, a.Hkv, a.pshift};
  if (len <= stay) {
    leave(a, at, pair, hk, b, len, FINISH);
    return;
  }
  const bool one_by_one = NB <= 4 && len - stay <= kOneByOne;
  if (!one_by_one)
    for (int i = tid; i < int(sizeof(hist) / 16); i += kThreads) reinterpret_cast<i32x4*>(hist)[i] = i32x4{0, 0, 0, 0};

  static_assert(NB <= 4 || !FINISH, "a launch that finishes holds weights and positions in registers to the end");
  int page[NB];
  f32x4 w[NB];
  i32x4 p[NB];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    page[i] = at.table[min(4096 * i + 4 * tid, len - 1) >> a.pshift];
    const bool out = unsigned(page[i]) >= unsigned(a.num_pages);
    bad |= out;
    page[i] = out ? 0 : page[i];
  }
  const auto place = [&](int i) {   // of run i's first slot
    return ((size_t(page[i]) * a.Hkv + hk) << a.pshift) + (min(4096 * i + 4 * tid, (len - 1) & ~3) & ((1 << a.pshift) - 1));
  };
  const auto slot = [&](int i, int e) { return 4096 * i + 4 * tid + e; };
  // slots of the run i that is loaded that are below the length
  const auto below = [&](int i) { return 4096 * (i + 1) <= len ? 4 : len - min(slot(i, 0), (len - 1) & ~3); };
  int newest = INT32_MIN;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    w[i] = *reinterpret_cast<const f32x4*>(a.weights + place(i));
    p[i] = *reinterpret_cast<const i32x4*>(a.positions + place(i));
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int n = below(i);
#pragma unroll
    for (int e = 0; e < 4; ++e) newest = e < n ? max(newest, p[i][e]) : newest;
  }
  newest = wave_largest(newest);
  if (lane == 0) tops[wave] = newest;
  bad = __syncthreads_or(bad);
  if (tid == 0 && hk == 0) a.lengths_out[b] = bad ? len : stay;
  if (bad) {
    if (tid == 0 && !FINISH) a.count[pair] = -1;
    return;
  }
  newest = wave_largest(tops[lane & (kWaves - 1)]);
  // The distance to the newest position is exact in 32 unsigned bits.  Slots
  // that are not there have the smallest key and come after all that are, so
  // that none of them is among the budget largest.
  uint32_t key[NB][4];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      key[i][e] = uint32_t(newest) - uint32_t(p[i][e]) < uint32_t(a.recent) ? 0xffffffffu : rank_of(w[i][e]);
      if (4096 * (i + 1) > len && slot(i, e) >= len) key[i][e] = 0;
    }

  // Sums of mine[] over the runs before this thread's run i, in slot order.
  const auto before = [&](uint32_t (&mine)[NB], uint32_t* lds, uint32_t (&out)[NB]) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const uint32_t s = wave_scan(mine[i]);
      out[i] = s - mine[i];
      if (lane == 63) lds[i * kWaves + wave] = s;
    }
    __syncthreads();
    uint32_t carry = 0;
#pragma unroll
    for (int c = 0; c < NB * kWaves; c += 64) {   // 4 runs of 16 waves at a time
      const uint32_t v = c + lane < NB * kWaves ? lds[c + lane] : 0, s = wave_scan(v);
#pragma unroll
      for (int i = c / kWaves; i < c / kWaves + 4 && i < NB; ++i) {
        const int l = i * kWaves - c + wave;
        out[i] += carry + lane_of(s, l) - lane_of(v, l);
      }
      carry += lane_of(s, 63);
    }
    return carry;
  };
  uint32_t kept[NB];   // a bit a slot
#pragma unroll
  for (int i = 0; i < NB; ++i) kept[i] = (1u << min(max(len - slot(i, 0), 0), 4)) - 1;
  if (one_by_one) {
    // few to drop: the smallest key, of equal ones the last slot, one by one
    // (256 pairs of 2049 slots cut by 1 or 4: 6.7 and 8.4 us, 9.1 by digits)
    for (int k = 0; k < len - stay; ++k) {
      uint32_t least = ~0u, last = ~0u;   // a key, and the complement of a slot
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (kept[i] >> e & 1) {
            last = key[i][e] <= least ? ~uint32_t(slot(i, e)) : last;
            least = min(least, key[i][e]);
          }
      const auto join = [&] {   // over the lanes
        const uint32_t m = wave_least(least);
        last = wave_least(least == m ? last : ~0u);
        least = m;
      };
      join();
      if (lane == 0) leasts[k & 1][wave] = uint64_t(least) << 32 | last;
      __syncthreads();
      const uint64_t other = leasts[k & 1][lane & (kWaves - 1)];
      least = uint32_t(other >> 32);
      last = uint32_t(other);
      join();
      const int gone = int(~last);
#pragma unroll
      for (int i = 0; i < NB; ++i)
        if (gone >> 2 == slot(i, 0) >> 2) kept[i] &= ~(1u << (gone & 3));
    }
  } else {
    // the budget-th largest key, digit by digit, until all that share the
    // digits so far stay
    uint32_t prefix = 0, mask = 0, need = uint32_t(stay);
    const auto round = [&](auto bins, auto copies, uint32_t* h, uint32_t* s, int shift) {
      constexpr int BINS = decltype(bins)::value, COPIES = decltype(copies)::value;
      constexpr bool FIRST = COPIES > 1;   // all keys are in
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        if (4096 * i >= len) continue;
        uint32_t digit[4];
        bool in[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          in[e] = FIRST || (key[i][e] & mask) == prefix;
          digit[e] = (key[i][e] >> shift) & (BINS - 1);
        }
        const uint32_t first = uint32_t(uniform(int(digit[0])));
        if (__all(in[0] && digit[0] == first)) {
          bool one = true;
#pragma unroll
          for (int e = 1; e < 4; ++e) one = one && in[e] && digit[e] == first;
          if (__all(one)) {
            // one addition for a wave whose keys agree (equal weights, new tokens)
            if (lane == 0) atomicAdd(&h[first * COPIES], 256u);
            continue;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (in[e]) atomicAdd(&h[digit[e] * COPIES + lane % COPIES], 1u);
      }
      __syncthreads();
      const uint32_t d = find_digit<BINS, COPIES>(h, s, need, lane, wave);
      prefix |= d << shift;
      mask |= uint32_t(BINS - 1) << shift;
      return bin<COPIES>(h, int(d)) == need;
    };
    constexpr auto one_copy = std::integral_constant<int, 1>();
    uint32_t* h1 = hist + kCopies * kBins[0];
    bool all = round(std::integral_constant<int, kBins[0]>(), std::integral_constant<int, kCopies>(), hist, sums[0], kShift[0]);
    if (!all) all = round(std::integral_constant<int, kBins[1]>(), one_copy, h1, sums[1], kShift[1]);
    if (!all) all = round(std::integral_constant<int, kBins[2]>(), one_copy, h1 + kBins[1], sums[2], kShift[2]);

#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((key[i][e] & mask) < prefix) kept[i] &= ~(1u << e);
    if (!all) {   // of the keys equal to the last the first `need` stay
      uint32_t n[NB], rank[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        n[i] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) n[i] += key[i][e] == prefix;
      }
      before(n, counts[0], rank);
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key[i][e] == prefix && rank[i]++ >= need) kept[i] &= ~(1u << e);
    }
  }
  // holes below the new length (low half) and what fills them (high half)
  uint32_t n[NB], rank[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const uint32_t low = (1u << min(max(stay - slot(i, 0), 0), 4)) - 1;
    n[i] = __popc(~kept[i] & low) | __popc(kept[i] & ~low) << 16;
  }
  const uint32_t total = before(n, counts[1], rank) & 0xffff;
  uint64_t* dst = FINISH ? few[0] : a.dst + size_t(pair) * a.most;
  uint64_t* src = FINISH ? few[1] : a.src + size_t(pair) * a.most;
  uint8_t* flags = a.flags + size_t(pair) * (a.key_stride / 4);
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int j = slot(i, 0);
    if (j >= len) continue;
    uint32_t hole = rank[i] & 0xffff, fill = rank[i] >> 16;
    const uint64_t x = place(i);
    const uint32_t low4 = (1u << min(max(stay - j, 0), 4)) - 1;
    for (uint32_t m = ~kept[i] & low4; m; m &= m - 1) dst[hole++] = x + __builtin_ctz(m);
    for (uint32_t m = kept[i] & ~low4; m; m &= m - 1) src[fill++] = x + __builtin_ctz(m);
    if constexpr (FINISH) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool k = kept[i] >> e & 1, low = j + e < stay;
        if (low ? a.other && k : j + e < len && !k) {
          a.weights_out[x + e] = low ? w[i][e] : 0.f;
          a.positions_out[x + e] = low ? p[i][e] : -1;
        }
      }
    } else {
      flags[j / 4] = uint8_t(kept[i]);
    }
  }
  if constexpr (FINISH) {
    __syncthreads();
    const int piece = tid & ((1 << a.lshift) - 1), rows = kThreads >> a.lshift;
    for (uint32_t i = tid >> a.lshift; i < total; i += rows) move_row(a, dst[i], src[i], piece);
  } else if (tid == 0) {
    a.count[pair] = int(total);
  }
}

// Rows that registers do not hold are spread over workgroups of 4096 slots
// each (a segment): the same selection in launches that meet in the workspace
// (newest position; keys and first digit; second digit; third digit; places),
// each workgroup summing the segments' histograms for itself.  8 pairs of
// 65536 slots cut to 8192: 59 us, 142 with one workgroup a pair that keeps its
// keys in the workspace.
constexpr int kSegment = 4 * kThreads;
struct Found {
  uint32_t prefix, mask, need, all;   // all: every key that shares the digits so far stays
};
struct SpreadArgs {
  int32_t* newest;    // [B Hkv][segments]
  int32_t* missing;   // [B Hkv][segments]
  uint32_t* above;    // [2][B Hkv][segments] keys above the digits found so far
  Found* found;       // [2][B Hkv] after the first and the second digit
  uint32_t* hist;     // [B Hkv][segments][2048 + 2048 + 1024]
  int segments, pairs;
};
constexpr int kHists = kBins[0] + kBins[1] + kBins[2];

// What a workgroup of a spread launch works on.
struct Segment {
  int pair, seg, hk, b, len, used;   // used: segments below the length
  Slots at;
};
__device__ __forceinline__ Segment segment(const EvictKernelArgs& a, const SpreadArgs& s) {
  Segment g;
  g.seg = int(blockIdx.x) % s.segments;
  g.pair = int(blockIdx.x) / s.segments;
  g.hk = g.pair % a.Hkv;
  g.b = g.pair / a.Hkv;
  g.len = max(0, min(a.lengths[g.b], a.max_len));
  g.used = (g.len + kSegment - 1) / kSegment;
  g.at = {a.block_table + size_t(g.b) * a.max_pages, g.hk, a.Hkv, a.pshift};
  return g;
}
__device__ __forceinline__ bool spread_missing(const SpreadArgs& s, const Segment& g) {
  int bad = 0;
  for (int i = threadIdx.x; i < g.used; i += kThreads) bad |= s.missing[size_t(g.pair) * s.segments + i];
  return __syncthreads_or(bad);
}

__global__ __launch_bounds__(kThreads) void spread_newest_kernel(EvictKernelArgs a, SpreadArgs s) {
  __shared__ int tops[kWaves];
  const Segment g = segment(a, s);
  const int j = g.seg * kSegment + 4 * int(threadIdx.x);
  const bool in = j < g.len;
  const int page = in ? g.at.table[j >> a.pshift] : 0;
  const int bad = __syncthreads_or(unsigned(page) >= unsigned(a.num_pages));
  if (g.seg >= g.used) return;
  int newest = INT32_MIN;
  if (!bad && in) {
    const i32x4 p = *reinterpret_cast<const i32x4*>(a.positions + g.at(j));
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e < g.len) newest = max(newest, p[e]);
  }
#pragma unroll
  for (int k = 1; k < 64; k *= 2) newest = max(newest, __shfl_xor(newest, k));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = newest;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 0; w < kWaves; ++w) newest = max(newest, tops[w]);
    s.newest[size_t(g.pair) * s.segments + g.seg] = newest;
    s.missing[size_t(g.pair) * s.segments + g.seg] = bad;
  }
}

// The digit of `sum` (LDS) that continues f.
template <int ROUND>
__device__ __forceinline__ Found next_digit(Found f, const uint32_t* sum, uint32_t* sums, int lane, int wave) {
  const uint32_t d = find_digit<kBins[ROUND]>(sum, sums, f.need, lane, wave);
  f.prefix |= d << kShift[ROUND];
  f.mask |= uint32_t(kBins[ROUND] - 1) << kShift[ROUND];
  f.all = sum[d] == f.need;
  return f;
}
constexpr int kHistAt[3] = {0, kBins[0], kBins[0] + kBins[1]};
// Sum over a pair's segments of the histogram of digit ROUND, to LDS.
template <int ROUND>
__device__ __forceinline__ void sum_hists(const SpreadArgs& s, const Segment& g, uint32_t* to) {
  const uint32_t* h = s.hist + size_t(g.pair) * s.segments * kHists + kHistAt[ROUND];
  for (int i = threadIdx.x; i < kBins[ROUND]; i += kThreads) {
    uint32_t n = 0;
    for (int k = 0; k < g.used; ++k) n += h[size_t(k) * kHists + i];
    to[i] = n;
  }
  __syncthreads();
}

// Digit ROUND: its segment's histogram, after the digit before it is found.
// The first also makes the keys.
template <int ROUND>
__global__ __launch_bounds__(kThreads) void spread_hist_kernel(EvictKernelArgs a, SpreadArgs s) {
  __shared__ uint32_t hist[kBins[0]], sums[kWaves];
  __shared__ uint32_t over;
  const Segment g = segment(a, s);
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  if (ROUND == 0 && g.len <= a.budget) {
    if (g.seg == 0) leave(a, g.at, g.pair, g.hk, g.b, g.len, false);
    return;
  }
  if (g.len <= a.budget || g.seg >= g.used) return;
  const bool bad = spread_missing(s, g);
  if (ROUND == 0 && g.seg == 0 && tid == 0) {
    if (g.hk == 0) a.lengths_out[g.b] = bad ? g.len : a.budget;
    if (bad) a.count[g.pair] = -1;
  }
  if (bad) return;
  const int j = g.seg * kSegment + 4 * tid;
  uint32_t* keys = a.keys + size_t(g.pair) * a.key_stride;
  uint32_t key[4];
  Found f = {0, 0, uint32_t(a.budget), 0};
  if constexpr (ROUND == 0) {
    int newest = INT32_MIN;
    for (int i = tid; i < g.used; i += kThreads) newest = max(newest, s.newest[size_t(g.pair) * s.segments + i]);
#pragma unroll
    for (int k = 1; k < 64; k *= 2) newest = max(newest, __shfl_xor(newest, k));
    if (lane == 0) sums[wave] = uint32_t(newest);
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) newest = max(newest, int(sums[w]));
    const size_t x = g.at(min(j, (g.len - 1) & ~3));
    const f32x4 w = *reinterpret_cast<const f32x4*>(a.weights + x);
    const i32x4 p = *reinterpret_cast<const i32x4*>(a.positions + x);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      key[e] = uint32_t(newest) - uint32_t(p[e]) < uint32_t(a.recent) ? 0xffffffffu : rank_of(w[e]);
    if (j < g.len) *reinterpret_cast<u32x4*>(keys + j) = u32x4{key[0], key[1], key[2], key[3]};
  } else {
    const u32x4 k = j < g.len ? *reinterpret_cast<const u32x4*>(keys + j) : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e) key[e] = k[e];
    if constexpr (ROUND == 2) f = s.found[g.pair];
    const Found last = f;
    if (!f.all) {
      sum_hists<ROUND - 1>(s, g, hist);
      f = next_digit<ROUND - 1>(f, hist, sums, lane, wave);
      __syncthreads();
    }
    // keys of this segment that the new digit puts above
    uint32_t n = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      n += j + e < g.len && (key[e] & last.mask) == last.prefix && (key[e] & f.mask) > f.prefix;
    if (tid == 0) over = 0;
    __syncthreads();
    const uint32_t w = wave_scan(n);
    if (lane == 63 && w) atomicAdd(&over, w);
    __syncthreads();
    if (tid == 0) {
      s.above[(size_t(ROUND - 1) * s.pairs + g.pair) * s.segments + g.seg] = over;
      if (g.seg == 0) s.found[size_t(ROUND - 1) * s.pairs + g.pair] = f;
    }
    if (f.all) return;
  }
  for (int i = tid; i < kBins[ROUND]; i += kThreads) hist[i] = 0;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const bool in = j + e < g.len && (key[e] & f.mask) == f.prefix;
    const uint32_t digit = (key[e] >> kShift[ROUND]) & (kBins[ROUND] - 1);
    if (__all(in && digit == uint32_t(uniform(int(digit))))) {
      if (lane == 0) atomicAdd(&hist[digit], 64u);
    } else if (in) {
      atomicAdd(&hist[digit], 1u);
    }
  }
  __syncthreads();
  uint32_t* h = s.hist + (size_t(g.pair) * s.segments + g.seg) * kHists + kHistAt[ROUND];
  for (int i = tid; i < kBins[ROUND]; i += kThreads) h[i] = hist[i];
}

// The places to fill and what fills them.
constexpr int kMaxSegments = kMaxEvictLen / kSegment;
__global__ __launch_bounds__(kThreads) void spread_place_kernel(EvictKernelArgs a, SpreadArgs s) {
  __shared__ uint32_t hist[kBins[2]], sums[kWaves], lds[kWaves];
  __shared__ uint32_t seg_kept[kMaxSegments], seg_equal[kMaxSegments];
  const Segment g = segment(a, s);
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  if (g.len <= a.budget || g.seg >= g.used) return;
  if (spread_missing(s, g)) return;
  const int stay = a.budget;
  const Found f0 = s.found[g.pair], f1 = s.found[s.pairs + g.pair];
  Found f = f1;
  const int round = f0.all ? 0 : f1.all ? 1 : 2;   // the digit that decides
  if (round == 2) {
    sum_hists<2>(s, g, hist);
    f = next_digit<2>(f, hist, sums, lane, wave);
    __syncthreads();
  }
  // per segment: keys above the deciding prefix, and keys with it
  const int shift = kShift[round], bins = kBins[round];
  const uint32_t digit = (f.prefix >> shift) & uint32_t(bins - 1);
  for (int k = wave; k < g.used; k += kWaves) {
    const uint32_t* h = s.hist + (size_t(g.pair) * s.segments + k) * kHists + kHistAt[round];
    uint32_t n = 0;
    if (round == 2)
      for (int i = lane; i < bins; i += 64) n += uint32_t(i) > digit ? h[i] : 0;
    n = lane_of(wave_scan(n), 63);
    if (lane == 0) {
      n += s.above[size_t(g.pair) * s.segments + k];
      if (round > 0) n += s.above[(size_t(s.pairs) + g.pair) * s.segments + k];
      seg_kept[k] = n;
      seg_equal[k] = h[digit];
    }
  }
  __syncthreads();
  if (tid == 0) {   // prefix sums in the order of segments: equal keys, then kept ones
    uint32_t eq = 0;
    for (int k = 0; k < g.used; ++k) {
      const uint32_t e = seg_equal[k];
      seg_kept[k] += eq < f.need ? min(f.need - eq, e) : 0;
      seg_equal[k] = eq;
      eq += e;
    }
    uint32_t n = 0;
    for (int k = 0; k < g.used; ++k) {
      const uint32_t e = seg_kept[k];
      seg_kept[k] = n;
      n += e;
    }
  }
  __syncthreads();
  // a bit a slot of this thread's four in a segment
  const uint32_t* keys = a.keys + size_t(g.pair) * a.key_stride;
  const auto kept_in = [&](int seg) {
    const int j = seg * kSegment + 4 * tid;
    const u32x4 k = j < g.len ? *reinterpret_cast<const u32x4*>(keys + j) : u32x4{0, 0, 0, 0};
    uint32_t equal = 0, bits = 0, total;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      equal += j + e < g.len && (k[e] & f.mask) == f.prefix;
      bits |= uint32_t(j + e < g.len && (k[e] & f.mask) >= f.prefix) << e;
    }
    uint32_t rank = seg_equal[seg] + scan<kWaves>(equal, lds, total);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e < g.len && (k[e] & f.mask) == f.prefix && rank++ >= f.need) bits &= ~(1u << e);
    return bits;
  };
  const auto low_bits = [&](int seg) { return (1u << min(max(stay - seg * kSegment - 4 * tid, 0), 4)) - 1; };
  // kept slots below the new length: those before the segment that it cuts,
  // and that segment's own
  const int cut = stay / kSegment;
  uint32_t total;
  scan<kWaves>(uint32_t(__popc(kept_in(cut) & low_bits(cut))), lds, total);
  const uint32_t kept_low = seg_kept[cut] + total;

  const uint32_t kept = kept_in(g.seg), low = low_bits(g.seg);
  const uint32_t before = seg_kept[g.seg] + scan<kWaves>(uint32_t(__popc(kept)), lds, total);   // kept slots before j
  const int j = g.seg * kSegment + 4 * tid;
  if (g.seg == 0 && tid == 0) a.count[g.pair] = stay - int(kept_low);
  if (j >= g.len) return;
  a.flags[size_t(g.pair) * (a.key_stride / 4) + j / 4] = uint8_t(kept);
  const uint64_t x = g.at(j);
  uint64_t* dst = a.dst + size_t(g.pair) * a.most;
  uint64_t* src = a.src + size_t(g.pair) * a.most;
  // a hole's rank is the slots before it less the kept ones, a fill's the
  // kept ones before it less those that lie low
  uint32_t hole = uint32_t(j) - before, fill = before + uint32_t(__popc(kept & low)) - kept_low;
  for (uint32_t m = ~kept & low; m; m &= m - 1) dst[hole++] = x + __builtin_ctz(m);
  for (uint32_t m = kept & ~low; m; m &= m - 1) src[fill++] = x + __builtin_ctz(m);
}

__global__ __launch_bounds__(256) void move_kernel(EvictKernelArgs a) {
  const int pair = blockIdx.x, hk = pair % a.Hkv, b = pair / a.Hkv;
  const int n = a.count[pair];
  if (n < 0) return;
  const Slots at = {a.block_table + size_t(b) * a.max_pages, hk, a.Hkv, a.pshift};
  const int piece = threadIdx.x & ((1 << a.lshift) - 1), per = 256 >> a.lshift;
  const uint64_t* dst = a.dst + size_t(pair) * a.most;
  const uint64_t* src = a.src + size_t(pair) * a.most;
  for (int i = blockIdx.y * per + (threadIdx.x >> a.lshift); i < n; i += gridDim.y * per)
    move_row(a, dst[i], src[i], piece);
  const int len = min(a.lengths[b], a.max_len);
  const uint8_t* flags = a.flags + size_t(pair) * (a.key_stride / 4);
  for (int j = (a.other ? 0 : a.budget & ~255) + blockIdx.y * 256 + threadIdx.x; j < len; j += gridDim.y * 256)
    settle(a, at, j, a.budget, flags[j >> 2] >> (j & 3) & 1);
}

size_t up(size_t n) { return (n + 255) & ~size_t(255); }

template <int NB>
void run_select(const EvictKernelArgs& a, unsigned pairs, bool finish, hipStream_t s) {
  if constexpr (NB <= 4)
    if (finish) {
      start((select_kernel<NB, true>), dim3(pairs), dim3(kThreads), s, a);
      return;
    }
  start((select_kernel<NB, false>), dim3(pairs), dim3(kThreads), s, a);
}

}  // namespace

EvictPlan evict_plan(const gbb_paged_cache& c, int B, int max_len, int budget) {
  EvictPlan p;
  const size_t pairs = size_t(B) * c.kv_heads;
  p.key_stride = (size_t(max_len) + 63) & ~size_t(63);
  p.most = size_t(std::max(0, std::min(budget, max_len - budget)));
  p.count_off = 0;
  p.dst_off = up(pairs * 4);
  p.src_off = p.dst_off + up(pairs * p.most * 8);
  p.flag_off = p.src_off + up(pairs * p.most * 8);
  p.key_off = p.flag_off + up(pairs * (p.key_stride / 4));
  // (held rows are faster up to where registers end, however few they are: 16
  // pairs of 32768 slots 32 us, spread 50)
  p.spread = max_len > kMaxHeld;
  p.segments = (max_len + kSegment - 1) / kSegment;
  const size_t segs = pairs * p.segments;
  p.seg_off = p.key_off + (p.spread ? up(pairs * p.key_stride * 4) : 0);
  p.found_off = p.seg_off + (p.spread ? up(segs * 4 * 4) : 0);   // newest, missing, two counts
  p.hist_off = p.found_off + (p.spread ? up(pairs * 2 * sizeof(Found)) : 0);
  p.ws_bytes = p.hist_off + (p.spread ? up(segs * kHists * 4) : 0);
  return p;
}

int launch_evict(const gbb_paged_cache& c, const EvictArgs& x, const EvictPlan& p, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  EvictKernelArgs a;
  a.block_table = x.block_table;
  a.lengths = x.lengths;
  a.lengths_out = x.lengths_out;
  a.weights = c.weights;
  a.positions = c.positions;
  a.weights_out = x.weights_out;
  a.positions_out = x.positions_out;
  a.k = static_cast<uint8_t*>(c.k);
  a.v = static_cast<uint8_t*>(c.v);
  a.count = reinterpret_cast<int32_t*>(x.ws + p.count_off);
  a.dst = reinterpret_cast<uint64_t*>(x.ws + p.dst_off);
  a.src = reinterpret_cast<uint64_t*>(x.ws + p.src_off);
  a.keys = reinterpret_cast<uint32_t*>(x.ws + p.key_off);
  a.flags = reinterpret_cast<uint8_t*>(x.ws + p.flag_off);
  a.key_stride = p.key_stride;
  a.most = p.most;
  a.Hkv = c.kv_heads;
  a.num_pages = c.num_pages;
  a.pshift = __builtin_ctz(unsigned(c.page));
  a.max_pages = x.max_pages;
  a.max_len = x.max_len;
  a.budget = x.budget;
  a.recent = x.recent;
  a.lshift = __builtin_ctz(unsigned(c.head_dim * (c.dtype == GBB_E4M3 ? 1 : 2) / 16));
  a.other = x.weights_out != c.weights || x.positions_out != c.positions;
  const unsigned pairs = unsigned(x.B) * c.kv_heads;
  const bool finish = !p.spread && p.most <= size_t(kFew) && x.max_len <= 16384;
  if (p.spread) {
    SpreadArgs g;
    const size_t segs = size_t(pairs) * p.segments;
    g.newest = reinterpret_cast<int32_t*>(x.ws + p.seg_off);
    g.missing = g.newest + segs;
    g.above = reinterpret_cast<uint32_t*>(g.missing + segs);
    g.found = reinterpret_cast<Found*>(x.ws + p.found_off);
    g.hist = reinterpret_cast<uint32_t*>(x.ws + p.hist_off);
    g.segments = p.segments;
    g.pairs = int(pairs);
    const dim3 grid(static_cast<unsigned>(segs)), block(kThreads);
    start(spread_newest_kernel, grid, block, s, a, g);
    start((spread_hist_kernel<0>), grid, block, s, a, g);
    start((spread_hist_kernel<1>), grid, block, s, a, g);
    start((spread_hist_kernel<2>), grid, block, s, a, g);
    start(spread_place_kernel, grid, block, s, a, g);
  } else if (x.max_len <= 4096) {
    run_select<1>(a, pairs, finish, s);
  } else if (x.max_len <= 8192) {
    run_select<2>(a, pairs, finish, s);
  } else if (x.max_len <= 16384) {
    run_select<4>(a, pairs, finish, s);
  } else {
    run_select<8>(a, pairs, finish, s);
  }
  if (!finish) {
    const size_t per = 256 >> a.lshift;
    const size_t most = std::max((p.most + per - 1) / per, (size_t(x.max_len) + 255) / 256);
    const unsigned gy = unsigned(std::min<size_t>(most, std::max(1u, 4096u / pairs)));
    start(move_kernel, dim3(pairs, gy), dim3(256), s, a);
  }
  return int(hipGetLastError());
}

}  // namespace gbb
