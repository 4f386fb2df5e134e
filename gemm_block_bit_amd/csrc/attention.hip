// Attention of one new token per sequence over a paged cache
// (gbb_paged_attention), split over the cache's length and joined.
//
// For a kv head with G query heads the work is two thin products and a
// softmax, o = softmax(scale q K^T) V with q [G][D]: 4 G D operations a slot
// against 2 D elements read, so with G <= 16 the cache's bytes bound it and
// the matrix cores, at 16 query rows a tile, have room to spare (8 to 15 % of
// the cycles; vector instructions 17 to 34 %).  A workgroup has at most 16 query
// heads: where a kv head has more, its K and V are read once for every 16.
//
// A workgroup takes one run of `chunk` slots of one (sequence, kv head); its
// waves take tiles of 32 slots in turn, one pass with the running maximum:
//  - S^T = K q^T: the A operand of a 16x16x32 MFMA is 16 slots x 32 elements
//    of K, a row a lane.  K is loaded with whole rows over neighbouring lanes
//    straight into LDS of the wave's own, and read back a row a lane.
//    The result has lane c + 16 g holding query head c, slots 4 g ... 4 g + 3.
//  - O^T = V^T P: the contraction runs over slots, and which slot a k index
//    stands for is free as long as both operands agree.  So P's registers
//    are the B operand as they are, and a lane of the A operand needs
//    elements of V at the slots 4 g ... 4 g + 3: it loads 16 bytes of those
//    four rows (16 lanes side by side take a whole row) and byte permutes
//    within the lane pair them up.  Output row c of tile j is element
//    EV c + j of the head.
//  - the running maximum is per query head, hence the same in the 4 lanes
//    that share c (two lane exchanges a tile); sums stay per lane to the end.
//  - loads have the rows that take part as their range, so that rows past the
//    length read as zeros whatever their memory holds.
// The next tile's K is under way while this one's product is formed, its V
// while the next scores are; every wait counts the loads behind it.
//
// P is rounded to 16 bits for the matrix cores; what the rounding drops is
// multiplied too, as further operands: one for fp16, which then carries 22
// bits of P (its exponential's argument is good to 21), two for bf16, which
// carries all 24 (17 with one: a value that the others nearly cancel loses
// its digits).  So the output's own rounding is what is left.
// exp2 is taken 14 powers above the running maximum's 0, so that fp16 keeps
// small probabilities out of its subnormals; the sums carry the same factor.
// e4m3 elements widen to 16 bits exactly; their scales go into the scores'
// scale and the output.
//
// The partial results of a sequence with several runs (maximum, sum and
// unnormalised output, fp32) go to the workspace, and the last workgroup of a
// sequence to arrive joins them in the order of the runs; where there are too
// many, and with weights, a second launch does, to the same bits.  With
// weights the scores are stored too (fp32), and exp(s - max) / sum is added
// over the kv head's query heads, one thread a slot, without atomics.
//
// Scores may be capped, biased by distance or cut to a window (OPT, kernels of
// their own, so that plain calls keep theirs): a cap is an exponential and a
// reciprocal a score more, a bias one multiply-add, and a window moves the first
// slot of the runs, so that what lies before it is not read.
//
// Measured: 32 sequences of up to 8192 slots (64 / 8 heads of 128, bf16,
// 523 MB) 103 us, 5.1 TB/s; 2 of 131072 (32 / 8, e4m3, 537 MB) 100 us, 5.4
// TB/s; a plain read kernel reaches 5.2 to 5.5 TB/s here.  1 of 1000 slots (32
// / 8, fp16) 7 us, a chain of dependent steps: launch, page, K and V, scores,
// the joins in the workgroup and over the runs; with a bias 9.1 a call, eager.
// 32 of up to 16384 with a cap and a window of 4096 (64 / 8, bf16, 464 MB) 92 us.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "attention_common.h"

namespace gbb {

namespace {

constexpr float kShift = 14.f;   // see above: 2^14 < 65504
constexpr int kMaxJoin = 64;     // runs that the last workgroup of a sequence joins itself
constexpr int kMaxArrived = GBB_ATTENTION_COUNTERS / 4;   // counters of such sequences, at the workspace's start
constexpr int kMaxChunk = 4096;  // two page entries of a tile a lane: 32 tiles x 4 waves x 32 slots

// N pieces of 16 bytes from LDS, at the byte offsets at[] plus OFF, awaited.
// Written out because the compiler, where it sees the reads, awaits every
// vector memory load before them, V's among them.
template <int OFF> __device__ __forceinline__ void from_lds(u32x4 (&x)[1], const uint32_t (&at)[1]) {
  asm volatile("ds_read_b128 %0, %1 offset:%2\n\ts_waitcnt lgkmcnt(0)" : "=&v"(x[0]) : "v"(at[0]), "n"(OFF) : "memory");
}
template <int OFF> __device__ __forceinline__ void from_lds(u32x4 (&x)[2], const uint32_t (&at)[2]) {
  asm volatile("ds_read_b128 %0, %2 offset:%4\n\tds_read_b128 %1, %3 offset:%4\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(x[0]), "=&v"(x[1])
               : "v"(at[0]), "v"(at[1]), "n"(OFF)
               : "memory");
}
template <int OFF> __device__ __forceinline__ void from_lds(u32x4 (&x)[4], const uint32_t (&at)[4]) {
  asm volatile("ds_read_b128 %0, %4 offset:%8\n\tds_read_b128 %1, %5 offset:%8\n\t"
               "ds_read_b128 %2, %6 offset:%8\n\tds_read_b128 %3, %7 offset:%8\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
               : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(OFF)
               : "memory");
}
template <int OFF> __device__ __forceinline__ void from_lds(u32x4 (&x)[8], const uint32_t (&at)[8]) {
  asm volatile("ds_read_b128 %0, %8 offset:%16\n\tds_read_b128 %1, %9 offset:%16\n\t"
               "ds_read_b128 %2, %10 offset:%16\n\tds_read_b128 %3, %11 offset:%16\n\t"
               "ds_read_b128 %4, %12 offset:%16\n\tds_read_b128 %5, %13 offset:%16\n\t"
               "ds_read_b128 %6, %14 offset:%16\n\tds_read_b128 %7, %15 offset:%16\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
               : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "v"(at[4]), "v"(at[5]), "v"(at[6]), "v"(at[7]), "n"(OFF)
               : "memory");
}

struct SplitArgs {
  const void* q;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* lengths;
  const float* weights;
  float* weights_out;
  void* out;
  float* lse;
  unsigned* arrived;  // [B][Hkv][qtiles] runs of a sequence that are done, 0 between calls; NULL: join_kernel joins
  float2* ml;       // [B][Hkv][nsplit][G] maximum (log2 domain) and sum
  float* o;         // [B][Hkv][nsplit][G][D]
  float* scores;    // [B][Hkv][G][score_stride], log2 domain
  size_t score_stride;
  int64_t q_token;
  bool joins;       // no second launch
  int B, Hq, Hkv, G, qtiles, num_pages, pshift, max_pages, max_len, chunk, nsplit;
  float scale;      // scale * log2(e)
  // OPT: a cap (times log2(e); 0: none), slopes [Hq] of a bias by distance or
  // NULL, and how many of the newest slots take part (0: all)
  float cap;
  const float* slopes;
  int window;
};

__device__ __forceinline__ int length_of(const SplitArgs& a, int b) {
  return max(0, min(a.lengths[b], a.max_len));
}
// The first slot that takes part, and where the runs of a sequence start: a
// tile's 16 slots lie in one page.
__device__ __forceinline__ int low_of(const SplitArgs& a, int len) { return a.window ? max(0, len - a.window) : 0; }
__device__ __forceinline__ int base_of(int low) { return low & ~15; }

// Waves of a workgroup: 4, or 8 (WIDE) for calls with so few runs that a
// workgroup should have a CU to itself.
constexpr int waves(bool wide) { return wide ? 8 : 4; }

// weights_out = weights + sum over the kv head's query heads of
// 2^(score - ref) inv, for the slots j ... j + 3, j + STEP ... below len (a
// page holds whole groups of 4).  Slots below low have no score: what is read
// in its place is not used.
template <int STEP>
__device__ __forceinline__ void add_weights(const SplitArgs& a, int b, int hk, int low, int len, int j, const float* ref,
                                            const float* inv) {
  for (; j < len; j += STEP) {
    const int p = a.block_table[size_t(b) * a.max_pages + (j >> a.pshift)];
    const float* s = a.scores + (size_t(b) * a.Hq + size_t(hk) * a.G) * a.score_stride + j;
    constexpr int AHEAD = 8;
    f32x4 x[AHEAD];
    const auto fetch = [&](int q0) {
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) x[u] = *reinterpret_cast<const f32x4*>(s + min(q0 + u, a.G - 1) * a.score_stride);
    };
    fetch(0);
    const bool there = unsigned(p) < unsigned(a.num_pages);
    const size_t at = ((size_t(there ? p : 0) * a.Hkv + hk) << a.pshift) + (j & ((1 << a.pshift) - 1));
    const f32x4 old = *reinterpret_cast<const f32x4*>(a.weights + at);
    f32x4 w = {0, 0, 0, 0};
    for (int q0 = 0; q0 < a.G; q0 += AHEAD) {
      if (q0) fetch(q0);
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        if (q0 + u < a.G)
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] += __builtin_amdgcn_exp2f(x[u][k] - ref[q0 + u]) * inv[q0 + u];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (there && j + k < len) a.weights_out[at + k] = j + k < low ? old[k] : old[k] + w[k];
  }
}

template <int DT, int CT, int D, bool WT, bool WIDE, bool OPT>
__global__ __launch_bounds__(64 * waves(WIDE), WIDE || D == 256 ? 2 : D == 128 ? 3 : 4) void split_kernel(SplitArgs a) {
  typedef Half<DT> H;
  constexpr int NW = waves(WIDE), THREADS = 64 * NW;
  typedef typename H::V8 V8;
  constexpr bool F8 = CT == GBB_E4M3;
  constexpr int ES = F8 ? 1 : 2, ROW = D * ES;
  constexpr int KP = ROW / 64;                       // 16-byte loads a lane and 16 slots of K
  constexpr int VB = ROW / 16 < 16 ? ROW / 16 : 16;  // bytes a lane loads at once of a row of V
  constexpr int VW = VB / 4, NV = ROW / 16 / VB, EV = VB / ES;
  constexpr int NT = D / 16;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int c = lane & 15, g4 = lane >> 4;
  int id = blockIdx.x;
  // (divisions are done in vector registers; what follows addresses memory by
  // scalar ones)
  const int qt = uniform(id % a.qtiles);
  id /= a.qtiles;
  const int hk = uniform(id % a.Hkv);
  id /= a.Hkv;
  const int b = uniform(id % a.B), sp = uniform(id / a.B);
  const int rows = min(16, a.G - 16 * qt);           // query heads of this tile
  const int hq0 = hk * a.G + 16 * qt;
  // (with a window the runs follow from the length)
  const int low = OPT ? uniform(low_of(a, a.window ? length_of(a, b) : 0)) : 0;
  const int base = OPT ? base_of(low) : 0;
  const int k0 = base + sp * a.chunk;
  // lane 2 i + s: the page of 16-slot half s of this wave's tile i, looked up
  // before the length is known (the table has max_len's entries)
  const int key = k0 + 32 * (wave + NW * (lane >> 1)) + 16 * (lane & 1);
  int page = a.block_table[size_t(b) * a.max_pages + (min(key, a.max_len - 1) >> a.pshift)];
  // rows past the last query head repeat it: their results are not used
  u32x4 qw[D / 32];
#pragma unroll
  for (int kc = 0; kc < D / 32; ++kc) {
    const int d = F8 ? 64 * (kc >> 1) + 16 * g4 + 8 * (kc & 1) : 32 * kc + 8 * g4;
    qw[kc] = ld16(static_cast<const uint16_t*>(a.q) + b * a.q_token + size_t(hq0 + min(c, rows - 1)) * D + d);
  }
  in_order();
  const int len = uniform(length_of(a, b));
  if (k0 >= len) {
    if (sp == 0) {                                   // an empty sequence
      for (int i = threadIdx.x; i < rows * D; i += THREADS)
        static_cast<typename H::T*>(a.out)[(size_t(b) * a.Hq + hq0) * D + i] = typename H::T(0.f);
      if (a.lse && threadIdx.x < rows) a.lse[size_t(b) * a.Hq + hq0 + threadIdx.x] = -INFINITY;
    }
    return;
  }
  const int k1 = min(len, k0 + a.chunk);
  const int ntile = (k1 - k0 + 31) >> 5;
  const int n = (ntile - wave + NW - 1) / NW;        // tiles of this wave: wave, wave + NW, ...
  if (key >= k1 || unsigned(page) >= unsigned(a.num_pages)) page = -1;
  V8 qf[D / 32];
#pragma unroll
  for (int kc = 0; kc < D / 32; ++kc) {
    asm volatile("" : "+v"(qw[kc]));   // awaited here, with the page, and not in the loop with its loads
    qf[kc] = __builtin_bit_cast(V8, qw[kc]);
  }
  const float scale = F8 && a.k_scale ? a.scale * a.k_scale[hk] : a.scale;
  const float over = OPT && a.cap > 0.f ? 1.f / a.cap : 0.f;
  const float slope = OPT && a.slopes ? a.slopes[hq0 + min(c, rows - 1)] * kLog2e : 0.f;

  // 32 rows of K a wave, and in the end the waves' outputs
  constexpr int OROW = D + 4, OWN = 16 * OROW * 4 > 32 * ROW ? 16 * OROW * 4 : 32 * ROW;
  __shared__ __align__(16) uint8_t lds[NW * OWN];
  uint8_t* mine = lds + wave * OWN;
  const auto so = [&](int w, int q, int d) -> float& { return reinterpret_cast<float*>(lds + w * OWN)[q * OROW + d]; };
  f32x4 o[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) o[i] = f32x4{0, 0, 0, 0};
  float m = -INFINITY, l = 0.f;
  const int pmask = (1 << a.pshift) - 1;
  const size_t page_bytes = (size_t(1) << a.pshift) * ROW;

  // K goes through LDS, in memory of the wave's own: it is loaded there
  // directly with neighbouring lanes on a row (a load with a row a lane asks
  // for 64 separate lines and takes four times as long to issue) and read
  // back a row a lane.  The load writes lane by lane, so lane l is given the
  // piece (16 bytes) that makes piece p of row r land at p ^ swizzle(r),
  // which spreads the 16 rows that lanes read at once over all banks.
  constexpr int LPR = ROW / 16, RPI = 64 / LPR;      // lanes a row, rows an instruction
  constexpr auto swizzle = [](int r) { return (ROW >= 256 ? r : r / (256 / ROW)) & (LPR < 16 ? LPR - 1 : 15); };
  // The rows of 16-slot half s of tile i that take part: a page holds whole
  // halves, and rows past the length or of a page that is not there read as
  // zeros, whatever their memory holds.
  const auto rows_at = [&](const uint8_t* base, int i, int s) {
    const int p = __builtin_amdgcn_readlane(page, 2 * i + s);
    const int key = k0 + 32 * (wave + NW * i) + 16 * s;
    const size_t off = (size_t(max(p, 0)) * a.Hkv + hk) * page_bytes + size_t(key & pmask) * ROW;
    return span(base + off, uniform(p < 0 ? 0 : max(0, min(k1 - key, 16)) * ROW));
  };
  uint32_t vr[2][4][NV][VW];
  const auto load_k = [&](int i) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const Span rows = rows_at(a.k, i, s);
#pragma unroll
      for (int j = 0; j < KP; ++j) {
        const int r = j * RPI + lane / LPR;
        to_lds(rows, r * ROW + ((lane % LPR) ^ swizzle(r)) * 16, mine + s * 16 * ROW + j * 1024);
      }
    }
  };
  const auto load_v = [&](int i) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const Span rows = rows_at(a.v, i, s);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int u = 0; u < NV; ++u) {
          int at = (4 * g4 + r) * ROW + u * 256 + c * VB;
          // slots before the window read as zeros: at a weight of 0 a NaN there would reach the output
          if (OPT && k0 + 32 * (wave + NW * i) + 16 * s + 4 * g4 + r < low) at = INT_MAX;
          if constexpr (VW == 4) {
            const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(rows, at, 0, 0);
#pragma unroll
            for (int w = 0; w < 4; ++w) vr[s][r][u][w] = x[w];
          } else if constexpr (VW == 2) {
            const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(rows, at, 0, 0);
            vr[s][r][u][0] = x[0];
            vr[s][r][u][1] = x[1];
          } else {
            vr[s][r][u][0] = __builtin_amdgcn_raw_buffer_load_b32(rows, at, 0, 0);
          }
        }
    }
  };
  uint32_t k_at[KP];   // this lane's pieces of row c in LDS
#pragma unroll
  for (int j = 0; j < KP; ++j)
    k_at[j] = uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)mine)) +
              c * ROW + ((4 * j + g4) ^ swizzle(c)) * 16;
  // NEXT: there is a next tile, whose K is loaded.  Known at compile time so
  // that the waits for V can count the loads behind it.
  const auto compute = [&](int i, auto NEXT) {
    const int key0 = k0 + 32 * (wave + NW * i);
    f32x4 s[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      s[e] = f32x4{0, 0, 0, 0};
      u32x4 kk[KP];
      if (e == 0) from_lds<0>(kk, k_at);
      else from_lds<16 * ROW>(kk, k_at);
#pragma unroll
      for (int j = 0; j < KP; ++j) {
        if constexpr (F8) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t w0 = kk[j][2 * h], w1 = kk[j][2 * h + 1];
            const u32x4 x = {H::template widen<false>(w0), H::template widen<true>(w0),
                             H::template widen<false>(w1), H::template widen<true>(w1)};
            s[e] = H::mfma(__builtin_bit_cast(V8, x), qf[2 * j + h], s[e]);
          }
        } else {
          s[e] = H::mfma(__builtin_bit_cast(V8, kk[j]), qf[j], s[e]);
        }
      }
      s[e] *= scale;
      if constexpr (OPT) {
        if (a.cap > 0.f) {
#pragma unroll
          for (int r = 0; r < 4; ++r) s[e][r] = capped(s[e][r], over, a.cap);
        }
        if (a.slopes) {
#pragma unroll
          for (int r = 0; r < 4; ++r) s[e][r] -= slope * float(len - 1 - (key0 + 16 * e + 4 * g4 + r));
        }
      }
    }
    if constexpr (decltype(NEXT)::value) {
      in_order();
      load_k(i + 1);
      in_order();
    }
    // slots of a tile that the length or a missing page cuts
    const int p0 = __builtin_amdgcn_readlane(page, 2 * i), p1 = __builtin_amdgcn_readlane(page, 2 * i + 1);
    if (key0 + 32 > k1 || (p0 | p1) < 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          s[e][r] = key0 + 16 * e + 4 * g4 + r >= k1 || (e ? p1 : p0) < 0 ? -INFINITY : s[e][r];
    }
    if (OPT && key0 < low) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r) s[e][r] = key0 + 16 * e + 4 * g4 + r < low ? -INFINITY : s[e][r];
    }
    if constexpr (WT) {
      if (c < rows) {
        float* sc = a.scores + (size_t(b) * a.Hq + hq0 + c) * a.score_stride + key0 + 4 * g4;
        *reinterpret_cast<f32x4*>(sc) = s[0];
        *reinterpret_cast<f32x4*>(sc + 16) = s[1];
      }
    }
    float mx = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                     fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    if (__any(mx > m)) {
      const float mn = fmaxf(m, mx), f = rescale(m, mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int j = 0; j < NT; ++j) o[j] *= f;
    }
    const float ref = m == -INFINITY ? 0.f : m - kShift;
    V8 part[H::PARTS];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float p = __builtin_amdgcn_exp2f(s[e][r] - ref);
        l += p;
#pragma unroll
        for (int i = 0; i < H::PARTS; ++i) {
          const typename H::T h = typename H::T(p);
          part[i][4 * e + r] = h;
          p -= float(h);   // exact
        }
      }
    auto product = [&](int tile, const u32x4& x) {
#pragma unroll
      for (int i = 0; i < H::PARTS; ++i) o[tile] = H::mfma(__builtin_bit_cast(V8, x), part[i], o[tile]);
    };
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        // word w of the four rows of both halves: elements EV c + (w's) of them
        if constexpr (F8) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t sel = h ? 0x07030602u : 0x05010400u;   // (a, b) -> a0 b0 a1 b1 of two rows' words
            uint32_t x[2][2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int r = 0; r < 2; ++r)
                x[e][r] = __builtin_amdgcn_perm(vr[e][2 * r + 1][u][w], vr[e][2 * r][u][w], sel);
            product(u * EV + 4 * w + 2 * h,
                    u32x4{H::template widen<false>(x[0][0]), H::template widen<false>(x[0][1]),
                          H::template widen<false>(x[1][0]), H::template widen<false>(x[1][1])});
            product(u * EV + 4 * w + 2 * h + 1,
                    u32x4{H::template widen<true>(x[0][0]), H::template widen<true>(x[0][1]),
                          H::template widen<true>(x[1][0]), H::template widen<true>(x[1][1])});
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t sel = h ? 0x07060302u : 0x05040100u;
            product(u * EV + 2 * w + h,
                    u32x4{__builtin_amdgcn_perm(vr[0][1][u][w], vr[0][0][u][w], sel),
                          __builtin_amdgcn_perm(vr[0][3][u][w], vr[0][2][u][w], sel),
                          __builtin_amdgcn_perm(vr[1][1][u][w], vr[1][0][u][w], sel),
                          __builtin_amdgcn_perm(vr[1][3][u][w], vr[1][2][u][w], sel)});
          }
        }
      }
  };
  // the next tile's K is loaded once this one's scores are there, its V once
  // this one's product is
  if (n > 0) {
    load_k(0);
    in_order();
    load_v(0);
  }
  const auto await_k = [&](int i) {
    // younger than this tile's K are its V's 8 NV loads and, with weights, the
    // last tile's two stores of scores
    if (WT && i) loads_left<8 * NV + 2>();
    else loads_left<8 * NV>();
  };
  for (int i = 0; i + 1 < n; ++i) {
    await_k(i);
    compute(i, std::true_type());
    in_order();
    load_v(i + 1);
  }
  if (n > 0) {
    await_k(n - 1);
    compute(n - 1, std::false_type());
  }

  // join the waves
  __shared__ float sm[NW][16], sl[NW][16];
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (g4 == 0) {
    sm[wave][c] = m;
    sl[wave][c] = l;
  }
  if (c < rows) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) so(wave, c, (t / EV) * 16 * EV + EV * (4 * g4 + r) + t % EV) = o[t][r];
  }
  __syncthreads();
  const bool whole = len - base <= a.chunk;
  const float vs = F8 && a.v_scale ? a.v_scale[hk] : 1.f;
  typedef typename H::T V2 __attribute__((ext_vector_type(2)));
  // out and lse from the joined sums of a head; with weights also what is
  // taken off its scores and one over its sum
  __shared__ float ref[16], inv[16];
  const auto finish = [&](int q, int d, float m, float l, float o0, float o1) {
    const size_t head = size_t(b) * a.Hq + hq0 + q;
    const float f0 = l == 0.f ? 0.f : o0 / l * vs, f1 = l == 0.f ? 0.f : o1 / l * vs;
    *reinterpret_cast<V2*>(static_cast<typename H::T*>(a.out) + head * D + d) = V2{typename H::T(f0), typename H::T(f1)};
    if (d == 0) {
      if (a.lse) a.lse[head] = l == 0.f ? -INFINITY : (m - kShift + __builtin_amdgcn_logf(l)) * kLn2;
      if (WT) {
        ref[q] = m == -INFINITY ? 0.f : m - kShift;
        inv[q] = l == 0.f ? 0.f : 1.f / l;
      }
    }
  };
  const size_t row0 = (size_t(b * a.Hkv + hk) * a.nsplit + sp) * a.G + 16 * qt;
  for (int i = threadIdx.x; i < rows * (D / 2); i += THREADS) {
    const int q = i / (D / 2), d = 2 * (i % (D / 2));
    float mm = sm[0][q];
#pragma unroll
    for (int w = 1; w < NW; ++w) mm = fmaxf(mm, sm[w][q]);
    float ll = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = rescale(sm[w][q], mm);
      ll += f * sl[w][q];
      o0 += f * so(w, q, d);
      o1 += f * so(w, q, d + 1);
    }
    if (whole) {
      finish(q, d, mm, ll, o0, o1);
      if (WT && d == 0) a.ml[row0 + q] = make_float2(mm, ll);
    } else {
      put(a.o + (row0 + q) * D + d, o0, o1);
      if (d == 0) put(reinterpret_cast<float*>(a.ml + row0 + q), mm, ll);
    }
  }
  if (whole) {
    if (WT && a.joins) {
      loads_left<0>();   // the waves' scores are written
      __syncthreads();
      add_weights<4 * THREADS>(a, b, hk, low, len, 4 * threadIdx.x, ref, inv);
    }
    return;
  }
  if (!a.arrived) return;

  // The workgroup that is the last of its sequence to get here joins all
  // runs, in their order whichever it is.  Partial results are written and
  // read at device scope (past the caches of the XCDs, which do not see each
  // other's), every wave awaits its writes before the count, and no
  // workgroup waits for another.  The order of the partial results and the
  // count so rests on that wait and on the reads' scope, not on the count's
  // own order: a release and an acquire there write back and invalidate the
  // whole XCD's L2 once a run (32 ragged 107 -> 125 us, 2 of 131072 103 -> 115,
  // 1 of 1000 7.1 -> 7.4), for memory that nothing here keeps in it.
  __shared__ unsigned count;
  loads_left<0>();
  __syncthreads();
  unsigned* arrived = a.arrived + (b * a.Hkv + hk) * a.qtiles + qt;
  if (threadIdx.x == 0) count = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  const int ns = (len - base + a.chunk - 1) / a.chunk;
  if (count != unsigned(ns - 1)) return;
  if (threadIdx.x == 0) __hip_atomic_store(arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const size_t first = size_t(b * a.Hkv + hk) * a.nsplit * a.G + 16 * qt;   // row of run 0
  float* factor = reinterpret_cast<float*>(lds);   // [kMaxJoin][16], then the joined maxima and sums
  float* joined = factor + kMaxJoin * 16;
  for (int q = wave; q < rows; q += NW) {
    static_assert(kMaxJoin <= 64, "a run a lane");
    float2 e = make_float2(-INFINITY, 0.f);
    if (lane < ns) e = get(reinterpret_cast<const float*>(a.ml + first + size_t(lane) * a.G + q));
    float mm = e.x;
#pragma unroll
    for (int x = 1; x < 64; x *= 2) mm = fmaxf(mm, __shfl_xor(mm, x));
    const float f = rescale(e.x, mm);
    float ll = f * e.y;
#pragma unroll
    for (int x = 1; x < 64; x *= 2) ll += __shfl_xor(ll, x);
    if (lane < kMaxJoin) factor[lane * 16 + q] = f;
    if (lane == 0) {
      joined[2 * q] = mm;
      joined[2 * q + 1] = ll;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 2); i += THREADS) {
    const int q = i / (D / 2), d = 2 * (i % (D / 2));
    const float* o = a.o + (first + q) * D + d;
    float o0 = 0.f, o1 = 0.f;
    for (int s0 = 0; s0 < ns; s0 += 8) {
      float2 x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = get(o + size_t(min(s0 + u, ns - 1)) * a.G * D);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (s0 + u < ns) {
          const float f = factor[(s0 + u) * 16 + q];
          o0 += f * x[u].x;
          o1 += f * x[u].y;
        }
    }
    finish(q, d, joined[2 * q], joined[2 * q + 1], o0, o1);
  }
}

// Maximum and sum of a query head over its ns runs, the same in all 64 lanes.
// e: lane i's run i, loaded before ns was known (first_runs).
__device__ __forceinline__ float2 first_runs(const float2* ml, const SplitArgs& a, int lane) {
  return ml[size_t(min(lane, a.nsplit - 1)) * a.G];
}
__device__ __forceinline__ float2 join_sums(float2 e, const float2* ml, int ns, int G, int lane) {
  if (lane >= ns) e = make_float2(-INFINITY, 0.f);
  float mm = e.x, ll = 0.f;
  for (int i = lane + 64; i < ns; i += 64) mm = fmaxf(mm, ml[size_t(i) * G].x);
#pragma unroll
  for (int x = 1; x < 64; x *= 2) mm = fmaxf(mm, __shfl_xor(mm, x));
  ll = rescale(e.x, mm) * e.y;
  for (int i = lane + 64; i < ns; i += 64) {
    const float2 f = ml[size_t(i) * G];
    ll += rescale(f.x, mm) * f.y;
  }
#pragma unroll
  for (int x = 1; x < 64; x *= 2) ll += __shfl_xor(ll, x);
  return make_float2(mm, ll);
}

// Joins the runs of every (sequence, query head), 256 / D to a workgroup and
// an element a thread, in the first `joining` workgroups; the others (with
// weights) take 1024 slots of a (sequence, kv head) each.  A launch of few
// short loads: what counts is that the loads do not wait for each other, so
// those of the first runs are issued before the length is known (the
// workspace has them for all nsplit runs).  The sums go run by run, as in
// split_kernel, and so to the same bits.
constexpr int kJoinSlots = 1024;
template <int DT, bool F8, int D, bool WT>
__global__ __launch_bounds__(256) void join_kernel(SplitArgs a, int joining) {
  typedef Half<DT> H;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  if (int(blockIdx.x) < joining) {
    const int head = uniform(int(blockIdx.x) * (256 / D) + int(threadIdx.x) / D), d = threadIdx.x % D;
    if (head >= a.B * a.Hq) return;
    const int hq = head % a.Hq, b = head / a.Hq;
    const int hk = hq / a.G, q = hq % a.G;
    const size_t row = size_t(b * a.Hkv + hk) * a.nsplit * a.G + q;
    const float2* ml = a.ml + row;
    constexpr int AHEAD = 16;
    const float* o = a.o + row * D + d;
    const size_t step = size_t(a.G) * D;
    float x[AHEAD], m[AHEAD];
    const auto fetch = [&](int i0) {
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int i = min(i0 + u, a.nsplit - 1);
        x[u] = o[i * step];
        m[u] = ml[size_t(i) * a.G].x;
      }
    };
    fetch(0);
    const float2 first = first_runs(ml, a, lane);
    in_order();
    const int len = length_of(a, b), span = len - base_of(low_of(a, len));
    if (span <= a.chunk) return;
    const int ns = (span + a.chunk - 1) / a.chunk;
    const float2 e = join_sums(first, ml, ns, a.G, lane);
    float acc = 0.f;
    for (int i0 = 0; i0 < ns; i0 += AHEAD) {
      if (i0) fetch(i0);
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        if (i0 + u < ns) acc += rescale(m[u], e.x) * x[u];
    }
    const float vs = F8 && a.v_scale ? a.v_scale[hk] : 1.f;
    static_cast<typename H::T*>(a.out)[size_t(head) * D + d] = typename H::T(e.y == 0.f ? 0.f : acc / e.y * vs);
    if (d == 0 && a.lse) a.lse[head] = e.y == 0.f ? -INFINITY : (e.x - kShift + __builtin_amdgcn_logf(e.y)) * kLn2;
    return;
  }
  if constexpr (WT) {
    const int nb = (a.max_len + kJoinSlots - 1) / kJoinSlots;
    int id = blockIdx.x - joining;
    const int j0 = (id % nb) * kJoinSlots;
    id /= nb;
    const int hk = id % a.Hkv, b = id / a.Hkv;
    const float2* ml = a.ml + size_t(b * a.Hkv + hk) * a.nsplit * a.G;
    const float2 first = first_runs(ml + min(wave, a.G - 1), a, lane);
    in_order();
    const int len = length_of(a, b);
    if (j0 >= len) return;
    // per query head: what is taken off a score, and one over the sum
    __shared__ float ref[kMaxGroup], inv[kMaxGroup];
    const int low = low_of(a, len), ns = (len - base_of(low) + a.chunk - 1) / a.chunk;
    for (int q = wave; q < a.G; q += 4) {
      const float2 e = join_sums(q == wave ? first : first_runs(ml + q, a, lane), ml + q, ns, a.G, lane);
      if (lane == 0) {
        ref[q] = e.x == -INFINITY ? 0.f : e.x - kShift;
        inv[q] = e.y == 0.f ? 0.f : 1.f / e.y;
      }
    }
    __syncthreads();
    add_weights<kJoinSlots>(a, b, hk, low, min(len, j0 + kJoinSlots), j0 + 4 * threadIdx.x, ref, inv);
  }
}

template <int DT, int CT, int D, bool WT, bool OPT>
void run_split(const SplitArgs& a, bool wide, hipStream_t s) {
  const unsigned grid = unsigned(a.B) * a.Hkv * a.qtiles * a.nsplit;
  if (wide) start((split_kernel<DT, CT, D, WT, true, OPT>), dim3(grid), dim3(64 * waves(true)), s, a);
  else start((split_kernel<DT, CT, D, WT, false, OPT>), dim3(grid), dim3(256), s, a);
}

template <int DT, int CT, int D>
void run(const SplitArgs& a, bool wide, bool wt, hipStream_t s) {
  const bool opt = a.cap > 0.f || a.slopes || a.window;
  if (wt && opt) run_split<DT, CT, D, true, true>(a, wide, s);
  else if (wt) run_split<DT, CT, D, true, false>(a, wide, s);
  else if (opt) run_split<DT, CT, D, false, true>(a, wide, s);
  else run_split<DT, CT, D, false, false>(a, wide, s);
  if (a.joins) return;
  const int heads = a.nsplit == 1 ? 0 : (a.B * a.Hq + 256 / D - 1) / (256 / D);
  constexpr bool F8 = CT == GBB_E4M3;
  if (wt) {
    const unsigned more = unsigned(a.B) * a.Hkv * unsigned((a.max_len + kJoinSlots - 1) / kJoinSlots);
    start((join_kernel<DT, F8, D, true>), dim3(unsigned(heads) + more), dim3(256), s, a, heads);
  } else if (heads) {
    start((join_kernel<DT, F8, D, false>), dim3(unsigned(heads)), dim3(256), s, a, heads);
  }
}
template <int DT, int CT>
void run_dim(const SplitArgs& a, int D, bool wide, bool wt, hipStream_t s) {
  if (D == 64) run<DT, CT, 64>(a, wide, wt, s);
  else if (D == 128) run<DT, CT, 128>(a, wide, wt, s);
  else run<DT, CT, 256>(a, wide, wt, s);
}

size_t up(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

AttendPlan attend_plan(const gbb_paged_cache& c, int B, int Hq, int most, bool with_weights, int window) {
  AttendPlan p;
  // slots of a sequence that take part, from the one that its runs start at
  const int max_len = window ? int(std::min<int64_t>(most, int64_t(window) + 15)) : most;
  const int G = Hq / c.kv_heads;
  p.qtiles = (G + 15) / 16;
  const int64_t pairs = int64_t(B) * c.kv_heads * p.qtiles;
  // Runs.  A run costs about 1.5 us of a CU beside its bytes and its partial
  // results have to be joined, and few CUs read faster each.  So contexts stay
  // whole where they are short and where the (sequence, kv head) pairs alone
  // keep the chip busy: one for every CU up to 4096 slots (256 pairs of 4000: 93
  // us whole, 97 and 100 in runs of 2048 and 1024), three for five CUs up to
  // 2048 of up to 128 elements (160 pairs of 2000: 32 us, 41 in 1024; of up to
  // 2000: 21, 18.5 in 1024), three for eight up to 1024 (96 of 1000: 12 and
  // 13.5 in 256; of up to 1000: 11 and 12; with 256 elements 28.5, 26.3 in 256,
  // and of up to 1000 17.5 to 19 and 20.6).  Lengths are known on the GPU only, so a
  // rule takes what is better for equal and ragged ones together.
  // Else the longest run that makes three for five CUs (24 pairs of 8000: 20 us
  // in 192 runs of 1024, 24 in 512; 8 of 60000: 48 in 240 of 2048, 53 in 1024;
  // 8 of 32768: 31 in 256 of 1024, 33 in 128 of 2048, 48 in 64 of 4096; 100 of 1500:
  // 17.2 in 200 of 1024, 21.6 in 512, but of up to 1500 13.6 to 14.1 and 12.5).  It
  // has at most 2048 slots, and those one for every CU, so that ragged lengths
  // balance (32 ragged of up to 8192: 105 us, 114 in 4096; 80 pairs of up to
  // 5000: 21 in 1024, 25 in 240 of 2048), but above 16384 there are runs enough
  // for that (2 of 131072: 99 us in 4096, 102 in 2048; 9 ragged pairs of up to
  // 107545: 34 to 38 and 40); and below 1024 at most 16 runs are made (4 pairs
  // of 16 query heads and 8192 slots: 14 us in 512, 22 in 128).
  // Eight waves a workgroup where it has work for them (1152 ragged pairs of
  // up to 2047 slots: 63 against 69 us), four for short runs (2048 pairs of
  // 256: 51 against 58 us).
  const int64_t cus = device_compute_units();
  int chunk = kMaxChunk;
  if (max_len <= 512 || (pairs >= cus && max_len <= kMaxChunk) || (8 * pairs >= 3 * cus && max_len <= 1024) ||
      (5 * pairs >= 3 * cus && max_len <= 2048 && c.head_dim < 256)) {
    p.wide = pairs < cus || max_len >= 1024;
  } else {
    const bool few = max_len <= 16384;   // runs for a sequence
    if (few) chunk = 2048;
    const int least = max_len <= 128 * 16 ? 128 : max_len <= 256 * 16 ? 256 : max_len <= 512 * 16 ? 512 : 1024;
    const auto enough = [&] {
      const int64_t runs = pairs * ((max_len + chunk - 1) / chunk);
      return few && chunk == 2048 ? runs >= cus : 5 * runs >= 3 * cus;
    };
    while (chunk > least && !enough()) chunk /= 2;
    p.wide = chunk >= 512;
  }
  p.chunk = chunk;
  p.nsplit = std::max(1, (max_len + chunk - 1) / chunk);
  const size_t rows = size_t(B) * Hq * p.nsplit;
  p.score_stride = (size_t(most) + (window ? 47 : 31)) & ~size_t(31);   // (a window's tiles may start 16 slots off)
  const bool parts = p.nsplit > 1;
  // One launch where the last workgroup of a sequence can join its runs.  With
  // weights, where there are none to join and a workgroup has all query heads
  // of its kv head: a second launch finds the scores of all runs without
  // their having to be written past the caches (16 ragged of up to 4097: 40
  // us, 44 with the scores at device scope and one launch).
  p.joins = with_weights ? !parts && p.qtiles == 1 : !parts || (p.nsplit <= kMaxJoin && pairs <= kMaxArrived);
  p.ml_off = parts || with_weights ? kMaxArrived * sizeof(unsigned) : 0;   // nothing else lies on the counters
  p.o_off = p.ml_off + (parts || with_weights ? up(rows * sizeof(float2)) : 0);
  p.s_off = p.o_off + (parts ? up(rows * c.head_dim * sizeof(float)) : 0);
  p.ws_bytes = p.s_off + (with_weights ? up(size_t(B) * Hq * p.score_stride * sizeof(float)) : 0);
  return p;
}

int launch_attend(const gbb_paged_cache& c, const AttendArgs& x, const AttendPlan& p, void* stream) {
  SplitArgs a;
  a.q = x.q;
  a.k = static_cast<const uint8_t*>(c.k);
  a.v = static_cast<const uint8_t*>(c.v);
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.block_table = x.block_table;
  a.lengths = x.lengths;
  a.weights = c.weights;
  a.weights_out = x.weights_out;
  a.out = x.out;
  a.lse = x.lse;
  a.joins = p.joins;
  a.arrived = p.joins && p.nsplit > 1 ? reinterpret_cast<unsigned*>(x.ws) : nullptr;
  a.ml = reinterpret_cast<float2*>(x.ws + p.ml_off);
  a.o = reinterpret_cast<float*>(x.ws + p.o_off);
  a.scores = reinterpret_cast<float*>(x.ws + p.s_off);
  a.score_stride = p.score_stride;
  a.q_token = x.q_token;
  a.B = x.B;
  a.Hq = x.Hq;
  a.Hkv = c.kv_heads;
  a.G = x.Hq / c.kv_heads;
  a.qtiles = p.qtiles;
  a.num_pages = c.num_pages;
  a.pshift = __builtin_ctz(unsigned(c.page));
  a.max_pages = x.max_pages;
  a.max_len = x.max_len;
  a.chunk = p.chunk;
  a.nsplit = p.nsplit;
  a.scale = x.scale * kLog2e;
  a.cap = x.softcap * kLog2e;
  a.slopes = x.slopes;
  a.window = x.window;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool wt = x.weights_out != nullptr;
  if (x.dtype == GBB_F16) {
    if (c.dtype == GBB_E4M3) run_dim<GBB_F16, GBB_E4M3>(a, c.head_dim, p.wide, wt, s);
    else run_dim<GBB_F16, GBB_F16>(a, c.head_dim, p.wide, wt, s);
  } else {
    if (c.dtype == GBB_E4M3) run_dim<GBB_BF16, GBB_E4M3>(a, c.head_dim, p.wide, wt, s);
    else run_dim<GBB_BF16, GBB_BF16>(a, c.head_dim, p.wide, wt, s);
  }
  return int(hipGetLastError());
}

}  // namespace gbb
