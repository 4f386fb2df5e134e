// Attention of several new tokens per sequence over a paged cache
// (gbb_paged_attention_tokens): prompts, chunks of them, and trees of drafted
// tokens, with capped or biased scores and masks.
//
// A row is a (token, query head) of one kv head, tokens outermost, so that the
// G query heads of a kv head and neighbouring tokens share K and V.  A
// workgroup takes 32 rows a wave and a run of `chunk` slots, one pass with the
// running maximum; its waves share tiles of BN slots of K and V in LDS:
//  - S^T = K q^T: the A operand of a 32x32x16 MFMA is 32 slots x 16 elements of
//    K, a slot a lane; the result has lane c + 32 h holding row c, slots 8 (i /
//    4) + 4 h + i % 4 in register i.
//  - O^T = V^T P: which slot a k index stands for is free as long as both
//    operands agree, so P's registers are the B operand as they are, and the A
//    operand needs, a lane, one element of V at four slots in a row, twice:
//    what a transposing LDS read gives (16 lanes read 4 slots of 16 elements,
//    each gets an element's 4 slots).
//  - a row's maximum and sum lie in the two lanes that share it: one lane swap
//    a tile for the maximum, one at the end for the sum.
//  - 16-bit tiles go from memory straight to LDS, e4m3 ones to registers and
//    from there, widened, to LDS; either while the tile before is worked on, in
//    two buffers, so that a tile takes one barrier.  Pieces of 16 bytes are
//    permuted within a row so that lanes that read together hit different
//    banks.  Memory past a row's range, and pages that are not there, read as
//    zeros, whatever they hold.
//  - what a row sees of a tile is a 64-bit mask.  A tile that all rows of a wave
//    see whole takes none, one that none sees is passed over.
//
// With n rows the work is 4 D operations a visible slot and row against 2 D
// elements of K and V a slot: matrix bound from some 100 rows on, by the bytes
// of the cache below that.  Beside the products every score costs an
// exponential, a maximum, a sum and a conversion in the vector pipes, which
// take about as long as its share of the products at D = 128, and a cap another
// exponential and a reciprocal; the tiles' reads from LDS (each wave reads all
// of K and V) come third.  Measured, 32 query over 8 kv heads of 128, bf16, a
// prompt of 8192 tokens (550e9 operations, 456 us at the rate of a large
// product): 584 to 612 us, with a bias 670 to 710, with a cap 717 to 754; as many
// heads of 64 (275e9) 346 to 364, 16 over 4 of 256 (550e9) 867 to 873, 32 over 8 of
// 256 1720; e4m3 592 to 629.  Through registers and LDS writes the plain one took
// 621, with waits before every load to LDS 780.
//
// P is rounded to 16 bits for the matrix cores, once where a sequence has more
// than 128 rows, so that the products bound the call (a second operand for what the
// rounding drops takes a third as long again): an output is off by at most
// half a step of its type relative to sum p |v|, beside its own rounding.  The
// sum that divides the output, and makes lse, is of P before that, in fp32.
// With fewer rows the cache's bytes and the steps that wait for each other bound the
// call, and P is given in two operands (22 bits in fp16, 16 in bf16).
//
// Where there are few row tiles the slots are split over workgroups; partial
// results (maximum, sum, unnormalised output, fp32) go to the workspace, and
// the last workgroup of a row tile, or where there are more runs a second
// launch, joins them in the order of the runs, so the result is the same bits
// each time.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <utility>

#include "attention_common.h"

namespace gbb {

namespace {

constexpr int kMaxJoin = 64;     // runs of a row tile
constexpr int kMaxArrived = GBB_ATTENTION_COUNTERS / 4;   // counters of row tiles with several runs
// Probabilities are 2^(score - ref).  ref is moved to kShift below a row's
// maximum when they would pass 2^kLimit: seldom after the first tiles, and
// each move costs a pass over the output.  fp16 (below 65504) so keeps those
// down to 2^-20 of the maximum out of its subnormals; a smaller one is off by
// 2^-31 of the maximum's at most.
constexpr float kShift = 6.f, kLimit = 15.f;

typedef int16_t i16x4 __attribute__((ext_vector_type(4)));

// What the second launch has to know of a row tile and kv head.
struct Note { int t0, r0, rows, runs; };       // its sequence's first token and rows, its own first row

struct Args {
  const void* q;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* starts;
  const int32_t* block_table;
  const int32_t* lengths;
  const int32_t* first;
  const int32_t* prefix;
  const uint32_t* tree;
  const float* slopes;
  void* out;
  float* lse;
  unsigned* arrived;   // [row tile][Hkv] runs that are done, 0 between calls
  float2* ml;          // [row tile][Hkv][nsplit][rows] ref (below) and sum
  float* o;            // [row tile][Hkv][nsplit][rows * D], in the order of the lanes that hold them
  Note* notes;         // [row tile][Hkv] where a second launch joins the runs, else NULL
  int64_t q_token;
  int T, B, Hq, Hkv, G, num_pages, pshift, max_pages, max_len, chunk, nsplit, tiles, tree_words, window;
  float scale, cap;    // times log2(e)
  bool negative;       // the scale's sign, taken into q
};

// Slots per tile: K and V of it take 16 KiB of LDS each at D = 128 and four waves.
constexpr int tile_slots(int D, int NW) { return D == 256 || NW < 4 ? 32 : 64; }

__device__ __forceinline__ int wave_min(int x) {
#pragma unroll
  for (int i = 1; i < 32; i *= 2) x = min(x, __shfl_xor(x, i));
  return x;
}
__device__ __forceinline__ int wave_max(int x) {
#pragma unroll
  for (int i = 1; i < 32; i *= 2) x = max(x, __shfl_xor(x, i));
  return x;
}
// n ones from bit 0 on, all or none where n is outside a word
__device__ __forceinline__ uint64_t below(int n) { return n <= 0 ? 0 : n >= 64 ? ~uint64_t(0) : (uint64_t(1) << n) - 1; }
// Both lanes' values of a row.
__device__ __forceinline__ float2 both(float x) {
  const uint32_t bits = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);
  const uint32_t r0 = r[0], r1 = r[1];   // (a bit_cast of r[1] itself would take r[0])
  return make_float2(__builtin_bit_cast(float, r0), __builtin_bit_cast(float, r1));
}
__device__ __forceinline__ float row_max(float x) {
  const float2 r = both(x);
  return fmaxf(r.x, r.y);
}
__device__ __forceinline__ float row_sum(float x) {
  const float2 r = both(x);
  return r.x + r.y;
}

// f(0), f(1), ... as compile-time constants
template <int... I, typename F>
__device__ __forceinline__ void unrolled(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void unrolled(F f) {
  unrolled(std::make_integer_sequence<int, N>(), f);
}

// Operands from LDS, awaited.  Written out because the compiler, where it sees
// the reads, awaits every load to LDS before them, the next tile's among them.
// Four pieces of 16 bytes at the offset OFF from four addresses;
template <int OFF>
__device__ __forceinline__ void read4(u32x4 (&x)[4], const uint32_t* at) {
  asm volatile("ds_read_b128 %0, %4 offset:%8\n\tds_read_b128 %1, %5 offset:%8\n\t"
               "ds_read_b128 %2, %6 offset:%8\n\tds_read_b128 %3, %7 offset:%8\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
               : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(OFF)
               : "memory");
}
// transposed, four slots from OFF on and four from OFF + STEP on, of two or four
// pieces: 16 lanes read 4 slots of 16 elements, and each gets an element of the four.
template <int OFF, int STEP>
__device__ __forceinline__ void read_turned(u32x4 (&x)[2], const uint32_t* at) {
  u32x2 y[4];
  asm volatile("ds_read_b64_tr_b16 %0, %4 offset:%6\n\tds_read_b64_tr_b16 %1, %4 offset:%7\n\t"
               "ds_read_b64_tr_b16 %2, %5 offset:%6\n\tds_read_b64_tr_b16 %3, %5 offset:%7\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(y[0]), "=&v"(y[1]), "=&v"(y[2]), "=&v"(y[3])
               : "v"(at[0]), "v"(at[1]), "n"(OFF), "n"(OFF + STEP)
               : "memory");
#pragma unroll
  for (int i = 0; i < 2; ++i) x[i] = __builtin_shufflevector(y[2 * i], y[2 * i + 1], 0, 1, 2, 3);
}
template <int OFF, int STEP>
__device__ __forceinline__ void read_turned(u32x4 (&x)[4], const uint32_t* at) {
  u32x2 y[8];
  asm volatile("ds_read_b64_tr_b16 %0, %8 offset:%12\n\tds_read_b64_tr_b16 %1, %8 offset:%13\n\t"
               "ds_read_b64_tr_b16 %2, %9 offset:%12\n\tds_read_b64_tr_b16 %3, %9 offset:%13\n\t"
               "ds_read_b64_tr_b16 %4, %10 offset:%12\n\tds_read_b64_tr_b16 %5, %10 offset:%13\n\t"
               "ds_read_b64_tr_b16 %6, %11 offset:%12\n\tds_read_b64_tr_b16 %7, %11 offset:%13\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(y[0]), "=&v"(y[1]), "=&v"(y[2]), "=&v"(y[3]), "=&v"(y[4]), "=&v"(y[5]), "=&v"(y[6]), "=&v"(y[7])
               : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(OFF), "n"(OFF + STEP)
               : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __builtin_shufflevector(y[2 * i], y[2 * i + 1], 0, 1, 2, 3);
}

// The kernel's arguments, read again where this is called: what is not needed
// in the loop over tiles would fill the scalar registers there.
typedef __attribute__((address_space(4))) const Args* LateArgs;
__device__ __forceinline__ LateArgs late_args() {
  uintptr_t p = reinterpret_cast<uintptr_t>(__builtin_amdgcn_kernarg_segment_ptr());
  asm volatile("" : "+s"(p));
  return reinterpret_cast<LateArgs>(p);
}

template <int DT, int CT, int D, int NW, int PARTS, bool TREE>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void tokens_kernel(Args a) {
  typedef Half<DT> H;
  typedef typename H::T T;
  typedef typename H::V8 V8;
  constexpr bool F8 = CT == GBB_E4M3;
  constexpr int THREADS = 64 * NW, ROWS = 32 * NW, BN = tile_slots(D, NW);
  constexpr int ROW = 2 * D;                  // bytes of a slot in LDS
  constexpr int GROW = F8 ? D : 2 * D;        // and in memory
  constexpr int LPR = GROW / 16;              // lanes that load a slot
  constexpr int RPI = 64 / LPR;               // slots a wave's load takes
  constexpr int NL = BN / (NW * RPI);         // loads a lane of a tile of K or V
  constexpr int PIECES = ROW / 16;
  constexpr int KC = D / 16, NT = D / 32, NE = BN / 32;
  constexpr int KA = KC < 8 ? KC : 8, VA = NT < 4 ? NT : 4;   // pieces of 256 bytes of a slot (beyond, 256 bytes on)
  static_assert(NL >= 1 && RPI <= 16, "a load stays within 16 slots");
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int c = lane & 31, h = lane >> 5;

  int id = blockIdx.x;
  const int hk = uniform(id % a.Hkv);
  id /= a.Hkv;
  const int w = uniform(id % a.tiles), sp = uniform(id / a.tiles);
  // the sequence whose row tile number w of the call is, 64 sequences at a time
  const auto start_of = [&](int b) { return max(0, min(a.starts[b], a.T)); };
  int b = -1, tile = 0, before = 0, ntiles = 0, t0 = 0, n = 0, len = 0, shared = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    // all that is known of a sequence in one step
    const int i = min(b0 + lane, a.B - 1);
    const int from = start_of(i), slots = a.lengths[i], prefix = a.prefix ? a.prefix[i] : 0;
    const int tokens = b0 + lane < a.B ? max(0, start_of(i + 1) - from) : 0;
    const int mine = (tokens * a.G + ROWS - 1) / ROWS;
    int sum = mine;
#pragma unroll
    for (int i = 1; i < 64; i *= 2) {
      const int x = __shfl_up(sum, i);
      if (lane >= i) sum += x;
    }
    const uint64_t past = __ballot(w < before + sum);
    if (past) {
      const int at = __builtin_ctzll(past);
      b = b0 + at;
      ntiles = __builtin_amdgcn_readlane(mine, at);
      tile = w - (before + __builtin_amdgcn_readlane(sum, at) - ntiles);
      t0 = __builtin_amdgcn_readlane(from, at);
      n = __builtin_amdgcn_readlane(tokens, at);
      len = max(0, min(__builtin_amdgcn_readlane(slots, at), a.max_len));
      shared = __builtin_amdgcn_readlane(prefix, at);
      break;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  // for the second launch: how many runs there are to join
  const auto tell = [&](int t0, int r0, int rows, int runs) {
    Note* const notes = late_args()->notes;
    if (notes && sp == 0 && threadIdx.x == 0) notes[w * a.Hkv + hk] = Note{t0, r0, rows, runs};
  };
  if (b < 0) {
    tell(0, 0, 0, 0);
    return;
  }
  b = uniform(b);
  t0 = uniform(t0);
  n = uniform(n);
  len = uniform(len);
  const int ctx = len - n;                     // may be negative
  const int rows_all = n * a.G;
  const int r0 = uniform(ntiles - 1 - tile) * ROWS;   // the last tokens first: they see most
  const int row = r0 + 32 * wave + c;
  const bool real = row < rows_all;
  const int token = real ? row / a.G : 0, hq = hk * a.G + (real ? row - token * a.G : 0);
  const int t = t0 + token;
  // q, the B operand: row c, elements 16 kc + 8 h ...; and the first pages of the
  // run, where it is known by now that they will be asked for (else of no use)
  u32x4 qw[KC];
#pragma unroll
  for (int kc = 0; kc < KC; ++kc) {
    qw[kc] = u32x4{0, 0, 0, 0};
    if (real) qw[kc] = ld16(static_cast<const uint16_t*>(a.q) + int64_t(t) * a.q_token + size_t(hq) * D + 16 * kc + 8 * h);
  }
  const auto page_of = [&](int slot) {
    const LateArgs x = late_args();
    return x->block_table[size_t(b) * x->max_pages + (min(slot, x->max_len - 1) >> x->pshift)];
  };
  const bool from_zero = !a.first && !a.window;
  const int early = page_of(min(int64_t(sp) * a.chunk, int64_t(a.max_len)) + 16 * lane);
  in_order();

  // What a row sees: slots [lo, hi), and with a tree those of [ctx, len) whose
  // bit is set, from `first` on and less than `window` away.  place: where
  // distances to slots before the new ones count from.
  int lo = 0, hi, place = ctx + token, first = 0, drafted = 0;
  // word i of the row's tree, without bits that do not count
  const auto tree_word = [&](int i) {
    if (i < 0 || i >= a.tree_words) return 0u;
    return a.tree[size_t(t) * a.tree_words + i] & uint32_t(below(n - 32 * i));
  };
  if (a.first) first = max(0, a.first[t]);
  if constexpr (TREE) {
    for (int i0 = 0; i0 < a.tree_words; i0 += 4) {
      uint32_t x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = tree_word(i0 + u);
#pragma unroll
      for (int u = 0; u < 4; ++u) drafted += __popc(x[u]);
    }
    place = ctx + drafted - 1;
    hi = ctx;
  } else {
    hi = place + 1;
    if (a.prefix) hi = max(hi, shared);
    if (a.window) hi = int(min(int64_t(hi), int64_t(place) + a.window));
    hi = min(hi, len);
  }
  if (a.window) lo = int(max(int64_t(0), int64_t(place) - a.window + 1));
  lo = max(lo, first);
  if (!real) lo = INT_MAX, hi = 0;
  const int top = TREE && real ? ctx + min(n, 32 * a.tree_words) : hi;         // one past the last slot it may see
  const int bottom = TREE && real ? max(first, min(lo, max(0, ctx))) : lo;     // and the first
  const bool some = top > bottom;
  const int lo_wave = uniform(wave_min(some ? bottom : INT_MAX)), hi_wave = uniform(wave_max(some ? top : 0));
  const int lo_all = uniform(wave_max(real ? lo : 0)), hi_all = uniform(wave_min(real ? hi : INT_MAX));   // all its rows see these
  __shared__ int range[2 * NW];
  if (lane == 0) {
    range[2 * wave] = lo_wave;
    range[2 * wave + 1] = hi_wave;
  }
  __syncthreads();
  int k_low = range[0], k_high = range[1];
#pragma unroll
  for (int i = 1; i < NW; ++i) {
    k_low = min(k_low, range[2 * i]);
    k_high = max(k_high, range[2 * i + 1]);
  }
  k_low = uniform(k_low);
  k_high = uniform(k_high);
  if (k_low >= k_high) {                       // no row sees a slot
    if (sp == 0 && real) {
      const size_t head = size_t(t) * a.Hq + hq;
      for (int d = 8 * h; d < D; d += 16) st16(static_cast<T*>(a.out) + head * D + d, u32x4{0, 0, 0, 0});
      if (a.lse && h == 0) a.lse[head] = -INFINITY;
    }
    tell(0, 0, 0, 0);
    return;
  }
  k_low &= ~15;
  // (nsplit runs reach over max_len slots from 0 on: from k_low on they may end past 2^31)
  if (int64_t(sp) * a.chunk >= k_high - k_low) return;
  const int k0 = k_low + sp * a.chunk;
  // what is needed after the tiles
  __shared__ int saved[4];
  if (threadIdx.x == 0) {
    saved[0] = t0;
    saved[1] = r0;
    saved[2] = rows_all;
    saved[3] = (k_high - k_low - 1) / a.chunk + 1;
  }
  tell(t0, r0, rows_all, (k_high - k_low - 1) / a.chunk + 1);
  const int k1 = k0 + min(k_high - k0, a.chunk);
  const int nt = (k1 - k0 + BN - 1) / BN;

  V8 qf[KC];
#pragma unroll
  for (int kc = 0; kc < KC; ++kc) qf[kc] = __builtin_bit_cast(V8, a.negative ? qw[kc] ^ 0x80008000u : qw[kc]);
  const float scale = F8 && a.k_scale ? a.scale * a.k_scale[hk] : a.scale;
  const float over = a.cap > 0.f ? 1.f / a.cap : 0.f;
  const float slope = a.slopes ? a.slopes[hq] * kLog2e : 0.f;
  enum { PLAIN, SHORT_CAP, BIAS, OTHER };
  const int shape = a.cap > 0.f ? a.slopes || a.cap > kShortCap * kLog2e ? OTHER : SHORT_CAP : a.slopes ? BIAS : PLAIN;
  // slots up to this are behind every row of the wave (of a tree: before all new ones)
  const int place_low = uniform(min(wave_min(real ? place : INT_MAX), TREE ? ctx - 1 : INT_MAX));

  // two tiles of K, then two of V
  constexpr int TILE = BN * ROW;
  __shared__ __align__(1024) uint8_t lds[4 * TILE];
  // Piece p (16 bytes) of slot r lies at p ^ swizzle(r): a slot a lane for K (8
  // lanes together hit 8 pieces), 4 slots of two pieces for V.
  constexpr int KS = PIECES < 16 ? PIECES - 1 : 15, VS = PIECES < 16 ? PIECES / 2 - 1 : 7;
  const auto k_swizzle = [](int r) { return r & KS; };
  const auto v_swizzle = [](int r) { return 2 * (r & VS); };

  // Where 64 groups of 16 slots lie, a group a lane: bytes from the cache's
  // start, bytes that take part (none of a page that is not there), and a bit
  // for every page that should be there and is not.
  // (bytes from the cache's start of a slot of page p)
  const auto place_of_slot = [&](int p, int slot) {
    const LateArgs x = late_args();
    return ((size_t(p) * x->Hkv + hk) << x->pshift) * GROW + size_t(slot & ((1 << x->pshift) - 1)) * GROW;
  };
  int off_lo, off_hi, bytes;
  uint64_t missing;
  const auto locate = [&](int first_slot, int p) {
    const int key = first_slot + 16 * lane;
    const bool used = key < k1, there = used && unsigned(p) < unsigned(late_args()->num_pages);
    const size_t off = there ? place_of_slot(p, key) : 0;
    off_lo = int(uint32_t(off));
    off_hi = int(uint32_t(off >> 32));
    bytes = there ? min(k1 - key, 16) * GROW : 0;
    missing = __ballot(used && !there);
  };
  constexpr int TPP = 1024 / BN;               // tiles of 64 groups
  // Starts tile i on its way: 16-bit elements straight to LDS (a load writes its
  // lanes side by side, so each is given the piece that belongs there), e4m3 ones
  // to registers, to be widened.  Returns a bit for every missing group.
  u32x4 kr[F8 ? NL : 1], vr[F8 ? NL : 1];
  const auto fetch = [&](int i) {
    if (i % TPP == 0) locate(k0 + i * BN, i == 0 && from_zero ? early : page_of(k0 + i * BN + 16 * lane));
    const int group = (i % TPP) * (BN / 16);
    // load j of the wave takes slots from STEP j + first on: within 16 of them that
    // the compiler can tell where `first` adds nothing across them
    constexpr int STEP = NW * RPI;
    static_assert(STEP % 16 == 0 || 16 % STEP == 0, "a load's 16 slots follow from j and the wave apart");
    const int first = wave * RPI, row = first % 16 + lane / LPR, p = lane % LPR;
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const int g = group + j * STEP / 16 + (STEP > 16 ? first / 16 : 0), r = j * STEP % 16 + row;
        const uint64_t off = __builtin_bit_cast(uint64_t, u32x2{uint32_t(__builtin_amdgcn_readlane(off_lo, g)),
                                                                uint32_t(__builtin_amdgcn_readlane(off_hi, g))});
        const Span from = span((v ? a.v : a.k) + off, __builtin_amdgcn_readlane(bytes, g));
        if constexpr (F8) (v ? vr : kr)[j] = __builtin_amdgcn_raw_buffer_load_b128(from, r * GROW + p * 16, 0, 0);
        else to_lds(from, r * GROW + (p ^ (v ? v_swizzle(r) : k_swizzle(r))) * 16,
                    lds + (2 * v + (i & 1)) * TILE + first * ROW + j * STEP * ROW);
      }
    return uniform(uint32_t(missing >> group) & ((1u << (BN / 16)) - 1));
  };
  const auto widened = [&](const u32x4 (&x)[F8 ? NL : 1], uint8_t* to, auto swizzle) {
    if constexpr (F8) {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const int r = (j * NW + wave) * RPI + lane / LPR, p = lane % LPR;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t w0 = x[j][2 * e], w1 = x[j][2 * e + 1];
          st16(to + r * ROW + ((2 * p + e) ^ swizzle(r)) * 16,
               u32x4{H::template widen<false>(w0), H::template widen<true>(w0),
                     H::template widen<false>(w1), H::template widen<true>(w1)});
        }
      }
    }
  };
  // tile i from the registers to LDS (e4m3)
  const auto widen_tile = [&](int i) {
    widened(kr, lds + (i & 1) * TILE, k_swizzle);
    widened(vr, lds + (2 + (i & 1)) * TILE, v_swizzle);
  };
  // V may hold infinities or NaN.  In the products they become NaN at a weight of
  // 0 (of rows that do not see the slot, or whose weight rounds to 0), and at one
  // given in two operands, of which the second is 0 or negative.  So a workgroup
  // whose output is not finite after its tiles, which is rare, goes over them
  // again with care: such elements are left out of the product, and what they do to
  // the rows that see them is found by products with 1 in the place of infinities of
  // each sign and of NaN.
  constexpr uint32_t EXP = DT == GBB_F16 ? 0x7c00u : 0x7f80u, ONE = DT == GBB_F16 ? 0x3c00u : 0x3f80u;
  const auto elements = [](u32x4 x, auto f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f(x[i] & 0xffffu) | f(x[i] >> 16) << 16;
    return x;
  };
  __shared__ int odd_tile;                     // the last tile that has such elements
  __shared__ bool again;                       // the tiles are gone over again
  // f of every 16 bytes of V's tile i, in place where f says so
  const auto each_piece = [&](int i, auto f) {
#pragma unroll 1
    for (int at = 16 * threadIdx.x; at < TILE; at += 16 * THREADS) {
      uint8_t* const p = lds + (2 + (i & 1)) * TILE + at;
      u32x4 x = ld16(p);
      if (f(x)) st16(p, x);
    }
  };
  const auto clean = [&](int i) {
    each_piece(i, [&](u32x4& x) {
      bool odd = false;
      x = elements(x, [&](uint32_t e) {
        const bool bad = (e & EXP) == EXP;
        odd |= bad;
        return bad ? 0u : e;
      });
      if (odd) odd_tile = i;
      return odd;
    });
    __syncthreads();
  };

  // This lane's addresses in LDS: K's slot c, V's slots 4 h + (lane % 16) / 4.
  // Other pieces of the slot differ in bits that the permutation leaves to an xor.
  const uint32_t lds_at = uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));
  const uint32_t k_at = lds_at + c * ROW + (h ^ k_swizzle(c)) * 16;
  const int v_slot = 4 * h + ((lane & 15) >> 2);
  const uint32_t v_at = lds_at + 2 * TILE + v_slot * ROW +
                        ((2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ v_swizzle(v_slot)) * 16 + 8 * (lane & 1);
  constexpr int VG = NT < 4 ? NT : 4;          // pieces of V that are read at once
  // product(j, operand) for V's elements 32 j ... of the slots 16 s ... of a tile
  const auto each_v = [&](const uint32_t (&at)[VA], auto S, auto product) {
    unrolled<NT / VG>([&](auto G) {
      u32x4 x[VG];
      read_turned<decltype(S)::value * 16 * ROW + decltype(G)::value * 256, 8 * ROW>(x, at);
#pragma unroll
      for (int u = 0; u < VG; ++u) product(decltype(G)::value * VG + u, __builtin_bit_cast(V8, x[u]));
    });
  };

  f32x16 o[NT];
  float ref, l;
  bool careful = false;
  if (threadIdx.x == 0) again = false;
#pragma unroll 1
  for (;;) {
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    ref = -FLT_MAX;
    l = 0.f;

    if (threadIdx.x == 0) odd_tile = -1;
    uint32_t holes_next = fetch(0);
#pragma unroll 1
    for (int i = 0; i < nt; ++i) {
      // tile i is in LDS for all waves, and all are done with the one before
      if (F8) widen_tile(i);
      else loads_left<0>();
      __syncthreads();
      if (careful) clean(i);
      const uint32_t holes = holes_next;
      if (i + 1 < nt) holes_next = fetch(i + 1);
      const int key0 = k0 + i * BN, buffer = (i & 1) * TILE;
      const bool works = key0 < hi_wave && key0 + BN > lo_wave;
      uint32_t v_pieces[VA];
#pragma unroll
      for (int u = 0; u < VA; ++u) v_pieces[u] = (v_at + buffer) ^ (u * 64);
      f32x16 s[NE];
      if (works) {
        uint32_t k_pieces[KA];
#pragma unroll
        for (int u = 0; u < KA; ++u) k_pieces[u] = (k_at + buffer) ^ (u * 32);
        unrolled<NE>([&](auto E) {
          constexpr int e = decltype(E)::value;
          s[e] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
          unrolled<KC / 4>([&](auto G) {
            constexpr int kc = 4 * decltype(G)::value;
            u32x4 x[4];
            read4<e * 32 * ROW + kc / KA * 256>(x, k_pieces + kc % KA);
#pragma unroll
            for (int u = 0; u < 4; ++u) s[e] = H::mfma32(__builtin_bit_cast(V8, x[u]), qf[kc + u], s[e]);
          });
        });
      }
      V8 part[PARTS][BN / 16];
      if (works) {
        // slot of register r of s[e]: key + 32 e + 8 (r / 4) + r % 4
        const int key = key0 + 4 * h;
        const auto slot = [](int e, int r) { return 32 * e + 8 * (r / 4) + r % 4; };
        // scores are s times unit plus offset
        float unit = scale, offset = 0.f;
        const bool whole = key0 >= lo_all && key0 + BN <= min(hi_all, k1) && !holes;
        // With a tree: bit j of the slot key0 + j that is a new token which the row's
        // tree has, and how many of those lie behind the tile.
        const bool branches = TREE && key0 + BN > ctx;
        uint64_t bits = 0;
        int beyond = 0;
        if (branches && real) {
          const int from = key0 - ctx, i0 = from >> 5, end = from + BN;   // end above 0
          uint32_t x[3];
#pragma unroll
          for (int u = 0; u < 3; ++u) x[u] = tree_word(i0 + u);
          const uint64_t low = uint64_t(x[1]) << 32 | x[0], high = uint64_t(x[2]) << 32 | x[1];
          const int shift = from & 31;
          bits = (low >> shift & 0xffffffffu) | (high >> shift) << 32;
          if (BN == 32) bits &= 0xffffffffu;
          beyond = drafted;
          for (int i = 0; 32 * i < end; ++i) beyond -= __popc(tree_word(i) & uint32_t(below(end - 32 * i)));
        }
        // (The usual shapes each in one branch of their own: where branches follow
        // each other the scores are copied in those that are not taken, 64 and more
        // registers a tile.)
        const auto cap_short = [&](float x) {    // tanh(x / cap) / 2 - 1 / 2 = -1 / (1 + e^(2 x / cap))
          return __builtin_amdgcn_rcpf(-1.f - __builtin_amdgcn_exp2f(x * (scale * over * (2.f * kLog2e))));
        };
        if (shape == SHORT_CAP) {
          unit = 2.f * a.cap;
          offset = a.cap;
#pragma unroll
          for (int e = 0; e < NE; ++e)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[e][r] = cap_short(s[e][r]);
        } else if (shape == BIAS && key0 + BN <= place_low + 1) {   // no slot lies ahead of a row
          const float base = -slope * float(place - key);
          unit = 1.f;
#pragma unroll
          for (int e = 0; e < NE; ++e)
#pragma unroll
            for (int r = 0; r < 16; ++r)
              s[e][r] = __builtin_fmaf(s[e][r], scale, __builtin_fmaf(slope, float(slot(e, r)), base));
        } else if (shape != PLAIN) {
          unit = 1.f;
          if (a.cap > kShortCap * kLog2e) {
#pragma unroll
            for (int e = 0; e < NE; ++e)
#pragma unroll
              for (int r = 0; r < 16; ++r) s[e][r] = capped(s[e][r] * scale, over, a.cap);
          } else if (a.cap > 0.f) {
#pragma unroll
            for (int e = 0; e < NE; ++e)
#pragma unroll
              for (int r = 0; r < 16; ++r) s[e][r] = __builtin_fmaf(2.f * a.cap, cap_short(s[e][r]), a.cap);
          } else {
#pragma unroll
            for (int e = 0; e < NE; ++e) s[e] *= scale;
          }
          if (a.slopes) {
            const float from = float(place - key);
#pragma unroll
            for (int e = 0; e < NE; ++e)
#pragma unroll
              for (int r = 0; r < 16; ++r) {
                float far = fabsf(from - float(slot(e, r)));
                if (branches && key + slot(e, r) >= ctx)
                  far = float(beyond + __popcll(bits >> (4 * h) >> slot(e, r) >> 1));
                s[e][r] = __builtin_fmaf(-slope, far, s[e][r]);
              }
          }
        }
        if (!whole) {
          // bit j: the row sees the slot key0 + j
          uint64_t seen = below(min(hi, k1) - key0) & ~below(lo - key0);
          if (branches) {
            uint64_t x = bits;
            if (a.window)   // the nearest ones: those with fewer behind them
              for (int more = beyond + __popcll(x) - a.window; more > 0 && x; --more) x &= x - 1;
            seen |= x & below(k1 - key0) & ~below(first - key0);
          }
          if (holes) {
#pragma unroll
            for (int g = 0; g < BN / 16; ++g)
              if (holes >> g & 1u) seen &= ~(uint64_t(0xffff) << (16 * g));
          }
          seen >>= 4 * h;
          const uint32_t part[2] = {uint32_t(seen), uint32_t(seen >> 32)};
#pragma unroll
          for (int e = 0; e < NE; ++e)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[e][r] = part[e] >> slot(0, r) & 1u ? s[e][r] : -INFINITY;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < NE; ++e)
#pragma unroll
          for (int r = 0; r < 16; r += 2) mx = fmaxf(fmaxf(s[e][r], s[e][r + 1]), mx);
        mx = __builtin_fmaf(row_max(mx), unit, offset);
        if (__any(mx > ref + kLimit)) {
          const float to = mx > ref + kLimit ? mx - kShift : ref, f = __builtin_amdgcn_exp2f(ref - to);
          ref = to;
          l *= f;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (careful && f == 0.f)           // what an infinity added so far has no weight any more
              o[j] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
            o[j] *= f;
          }
        }
        const float under = offset - ref;
        // 16 slots at a time, so that exponentials are taken while the products
        // of those before are formed
        unrolled<BN / 16>([&](auto S) {
          constexpr int t = decltype(S)::value;
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t / 2][8 * (t % 2) + r], unit, under));
            l += p;
#pragma unroll
            for (int x = 0; x < PARTS; ++x) {
              const T y = T(p);
              part[x][t][r] = y;
              p -= float(y);   // exact
            }
          }
          each_v(v_pieces, S, [&](int j, const V8& x) {
#pragma unroll
            for (int u = 0; u < PARTS; ++u) o[j] = H::mfma32(x, part[u][t], o[j]);
          });
        });
      }
      if (careful && uniform(odd_tile) == i) {
        // rare: infinities of either sign, from V as memory has it
        const int p = page_of(key0 + 16 * min(lane, BN / 16 - 1));
#pragma unroll 1
        for (int negative = 0; negative < 2; ++negative) {
          __syncthreads();
#pragma unroll 1
          for (int r = wave * 16; r < BN; r += 16 * NW) {        // 16 slots of a page a wave
            const int page = __builtin_amdgcn_readlane(p, r >> 4), slot = key0 + r;
            const bool there = unsigned(page) < unsigned(late_args()->num_pages);
            const size_t off = place_of_slot(there ? page : 0, slot);
            const Span from = span(a.v + off, uniform(there ? max(0, min(k1 - slot, 16)) * GROW : 0));
#pragma unroll 1
            for (int q = lane; q < 16 * (D / 8); q += 64) {      // a piece of 8 elements a lane
              const int row = q / (D / 8), piece = q % (D / 8);
              u32x4 x;
              if constexpr (F8) {
                const u32x2 y = __builtin_amdgcn_raw_buffer_load_b64(from, row * GROW + piece * 8, 0, 0);
                x = u32x4{H::template widen<false>(y[0]), H::template widen<true>(y[0]),
                          H::template widen<false>(y[1]), H::template widen<true>(y[1])};
              } else {
                x = __builtin_amdgcn_raw_buffer_load_b128(from, row * GROW + piece * 16, 0, 0);
              }
              x = elements(x, [=](uint32_t e) {   // 1 where an element is an infinity of that sign or NaN
                return (e & EXP) == EXP && ((e & 0x7fffu) != EXP || int(e >> 15) == negative) ? ONE : 0u;
              });
              st16(lds + 2 * TILE + buffer + (r + row) * ROW + (piece ^ v_swizzle(r + row)) * 16, x);
            }
          }
          __syncthreads();
          if (works) {
#pragma unroll
            for (int j0 = 0; j0 < NT; j0 += VG) {
              f32x16 hit[VG];
#pragma unroll
              for (int j = 0; j < VG; ++j) hit[j] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
              unrolled<BN / 16>([&](auto S) {
                each_v(v_pieces, S, [&](int j, const V8& x) {
                  if (j >= j0 && j < j0 + VG) hit[j - j0] = H::mfma32(x, part[0][decltype(S)::value], hit[j - j0]);
                });
              });
#pragma unroll
              for (int j = 0; j < VG; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                  if (hit[j][r] > 0.f) o[j0 + j][r] += negative ? -INFINITY : INFINITY;
            }
          }
        }
      }
    }

    if (careful) break;
    f32x4 odd = {0, 0, 0, 0};                    // 0, or NaN where an output is not finite
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) odd[r % 4] = __builtin_fmaf(o[j][r], 0.f, odd[r % 4]);
    if (__any(odd[0] + odd[1] + odd[2] + odd[3] != 0.f)) again = true;
    __syncthreads();                             // all are done with the tiles
    careful = uniform(again);
    if (!careful) break;
  }

  l = row_sum(l);
  const LateArgs x = late_args();
  const int ns = uniform(saved[3]);
  const int last_row = uniform(saved[1]) + 32 * wave + c;
  const bool writes = last_row < uniform(saved[2]);
  // out and lse of this lane's row from the output's pieces (4 elements each)
  const float vscale = F8 && x->v_scale ? x->v_scale[hk] : 1.f;
  const auto finish = [&](float ref, float l) {
    if (!writes) return;
    const int G = x->G, token = last_row / G;
    const size_t head = size_t(uniform(saved[0]) + token) * x->Hq + hk * G + (last_row - token * G);
    const float f = l == 0.f ? 0.f : vscale / l;
    typedef T V4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        V4 y;
#pragma unroll
        for (int u = 0; u < 4; ++u) y[u] = T(l == 0.f ? 0.f : o[j][r + u] * f);
        *reinterpret_cast<V4*>(static_cast<T*>(x->out) + head * D + 32 * j + 8 * (r / 4) + 4 * h) = y;
      }
    if (x->lse && h == 0) x->lse[head] = l == 0.f ? -INFINITY : (ref + __builtin_amdgcn_logf(l)) * kLn2;
  };
  if (ns == 1) {
    finish(ref, l);
    return;
  }

  // Partial results, as the lanes hold them: piece by piece, 16 bytes a lane.
  // At device scope and awaited before the count (as in attention.hip, where
  // the reasons stand); the last workgroup joins them in the order of the runs.
  const int tile_of_call = uniform(int(blockIdx.x) / x->Hkv % x->tiles), run = uniform(int(blockIdx.x) / x->Hkv / x->tiles);
  const size_t run0 = (size_t(tile_of_call) * x->Hkv + hk) * x->nsplit;
  constexpr int DEVICE = 16;                   // the cache policy of device scope
  const auto run_at = [&](int s) { return span(x->o + (run0 + s) * (ROWS * D), ROWS * D * 4); };
  const auto ml_at = [&](int s) { return reinterpret_cast<float*>(x->ml + (run0 + s) * ROWS + 32 * wave + c); };
  const int at = (wave * (4 * NT) * 64 + lane) * 16;
  if (writes) {
    const Span to = run_at(run);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const f32x4 y = {o[j][r], o[j][r + 1], o[j][r + 2], o[j][r + 3]};
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), to, at + (4 * j + r / 4) * 1024, 0, DEVICE);
      }
    if (h == 0) put(ml_at(run), ref, l);
  }
  if (x->notes) return;
  __shared__ unsigned count;
  loads_left<0>();
  __syncthreads();
  unsigned* arrived = x->arrived + tile_of_call * x->Hkv + hk;
  if (threadIdx.x == 0) count = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (count != unsigned(ns - 1)) return;
  if (threadIdx.x == 0) __hip_atomic_store(arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (!writes) return;
  constexpr int AHEAD = 2;                     // runs whose pieces are under way at once
  u32x4 pieces[AHEAD][4 * NT];
  float2 e[AHEAD];
  const auto take = [&](int s0) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const Span from = run_at(min(s0 + u, ns - 1));
      e[u] = get(ml_at(min(s0 + u, ns - 1)));
#pragma unroll
      for (int i = 0; i < 4 * NT; ++i) pieces[u][i] = __builtin_amdgcn_raw_buffer_load_b128(from, at + i * 1024, 0, DEVICE);
    }
  };
  float high = -FLT_MAX;
  for (int s0 = 0; s0 < ns; s0 += 16) {
    float y[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) y[u] = get(ml_at(min(s0 + u, ns - 1))).x;
    if (s0 == 0) take(0);
#pragma unroll
    for (int u = 0; u < 16; ++u) high = fmaxf(high, y[u]);
  }
  l = 0.f;
#pragma unroll
  for (int j = 0; j < NT; ++j) o[j] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
  for (int s0 = 0; s0 < ns; s0 += AHEAD) {
    if (s0) take(s0);
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (s0 + u < ns) {
        const float f = __builtin_amdgcn_exp2f(e[u].x - high);
        l += f * e[u].y;
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) {
          const f32x4 y = __builtin_bit_cast(f32x4, pieces[u][i]);
#pragma unroll
          for (int r = 0; r < 4; ++r)          // (an infinity at a weight of 0 is none)
            o[i / 4][4 * (i % 4) + r] = __builtin_fmaf(f, f == 0.f ? 0.f : y[r], o[i / 4][4 * (i % 4) + r]);
        }
      }
  }
  finish(high, l);
}

// The join in a launch of its own: a workgroup of one wave takes 32 elements of 32
// rows of a row tile and kv head.  The same sums in the same order.
constexpr int kBatch = 8;        // runs under way at once
template <int DT, int D>
__global__ __launch_bounds__(64) void join_kernel(Args a, int rows) {
  typedef typename Half<DT>::T T;
  constexpr int NT = D / 32;
  const int lane = threadIdx.x, j = blockIdx.x % NT, c = lane & 31, h = lane >> 5;
  const int slices = rows / 32, part = blockIdx.x / NT % slices, group = blockIdx.x / NT / slices, hk = group % a.Hkv;
  const Note note = a.notes[group];
  const int ns = uniform(note.runs);
  if (ns < 2) return;                          // its workgroup has written the output
  const int row = note.r0 + 32 * part + c;
  if (row >= note.rows) return;
  const float2* const ml = a.ml + size_t(group) * a.nsplit * rows + 32 * part + c;
  const float* const o = a.o + size_t(group) * a.nsplit * rows * D + (part * (4 * NT) + 4 * j) * 256 + 4 * lane;
  f32x4 pieces[kBatch][4];
  float2 e[kBatch];
  const auto take = [&](int s0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int s = min(s0 + u, ns - 1);
      e[u] = ml[size_t(s) * rows];
#pragma unroll
      for (int i = 0; i < 4; ++i) pieces[u][i] = *reinterpret_cast<const f32x4*>(o + size_t(s) * rows * D + 256 * i);
    }
  };
  float high = -FLT_MAX;
  for (int s0 = 0; s0 < ns; s0 += 16) {
    float y[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) y[u] = ml[size_t(min(s0 + u, ns - 1)) * rows].x;
    if (s0 == 0) take(0);
#pragma unroll
    for (int u = 0; u < 16; ++u) high = fmaxf(high, y[u]);
  }
  float l = 0.f, sum[16] = {};
  for (int s0 = 0; s0 < ns; s0 += kBatch) {
    if (s0) take(s0);
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (s0 + u < ns) {
        const float f = __builtin_amdgcn_exp2f(e[u].x - high);
        l += f * e[u].y;
#pragma unroll
        for (int i = 0; i < 16; ++i)           // (an infinity at a weight of 0 is none)
          sum[i] = __builtin_fmaf(f, f == 0.f ? 0.f : pieces[u][i / 4][i % 4], sum[i]);
      }
  }
  const int token = row / a.G;
  const size_t head = size_t(note.t0 + token) * a.Hq + hk * a.G + (row - token * a.G);
  const float f = l == 0.f ? 0.f : (a.v_scale ? a.v_scale[hk] : 1.f) / l;
  typedef T V4 __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int r = 0; r < 16; r += 4) {
    V4 y;
#pragma unroll
    for (int u = 0; u < 4; ++u) y[u] = T(l == 0.f ? 0.f : sum[r + u] * f);
    *reinterpret_cast<V4*>(static_cast<T*>(a.out) + head * D + 32 * j + 8 * (r / 4) + 4 * h) = y;
  }
  if (a.lse && h == 0 && j == 0) a.lse[head] = l == 0.f ? -INFINITY : (high + __builtin_amdgcn_logf(l)) * kLn2;
}

size_t up(size_t n) { return (n + 255) & ~size_t(255); }

template <int DT, int CT, int D, bool TREE>
void run_waves(const Args& a, const TokensPlan& p, unsigned grid, hipStream_t s) {
  if (p.waves == 2) start((tokens_kernel<DT, CT, D, 2, 2, TREE>), dim3(grid), dim3(128), s, a);
  else if (p.parts == 2) start((tokens_kernel<DT, CT, D, 4, 2, TREE>), dim3(grid), dim3(256), s, a);
  else start((tokens_kernel<DT, CT, D, 4, 1, TREE>), dim3(grid), dim3(256), s, a);
}
template <int DT, int CT, int D>
void run(const Args& a, const TokensPlan& p, unsigned grid, hipStream_t s) {
  if (a.tree) run_waves<DT, CT, D, true>(a, p, grid, s);
  else run_waves<DT, CT, D, false>(a, p, grid, s);
}
template <int DT, int CT>
void run_dim(const Args& a, int D, const TokensPlan& p, unsigned grid, hipStream_t s) {
  if (D == 64) run<DT, CT, 64>(a, p, grid, s);
  else if (D == 128) run<DT, CT, 128>(a, p, grid, s);
  else run<DT, CT, 256>(a, p, grid, s);
}
template <int DT>
void run_join(const Args& a, int D, int rows, hipStream_t s) {
  const dim3 grid(unsigned(a.tiles) * unsigned(a.Hkv) * unsigned(rows / 32) * unsigned(D / 32));
  if (D == 64) start((join_kernel<DT, 64>), grid, dim3(64), s, a, rows);
  else if (D == 128) start((join_kernel<DT, 128>), grid, dim3(64), s, a, rows);
  else start((join_kernel<DT, 256>), grid, dim3(64), s, a, rows);
}

}  // namespace

TokensPlan tokens_plan(const gbb_paged_cache& c, int T, int B, int Hq, int max_len, int window, int tree_words) {
  TokensPlan p;
  const int G = Hq / c.kv_heads;
  const int64_t rows = int64_t(T) * G;         // of a kv head
  const int64_t cus = device_compute_units();
  // Two waves a workgroup where a sequence has few rows and there are sequences
  // enough for the cache's bytes to bound the call (32 ragged of up to 8192
  // slots, 8 tokens of 32 / 8 heads each: 130 us, 146 with four; with few, four
  // stage a tile in half the time: 1 of 4000, 2 tokens: 29 and 23.5).
  p.waves = rows <= int64_t(64) * B && 2 * int64_t(B) * c.kv_heads >= cus ? 2 : 4;
  // Operands of P: one where the products bound the call.  A slot's K and V are 4 D
  // bytes in 16 bits, and a row takes 4 D operations, 6 D with two operands: up to 128
  // rows, a row tile, are 192 operations a byte, where this card's rates balance at 236.
  // (With two a tree of 25 behind 4000, 32 / 8 heads, takes 24.4 us, 23.1 with one, and 2
  // tokens behind 4000 20 and 18.3: there verifying a draft has the bits of decoding
  // it.  A prompt of 8192 takes 768 with two and 584 with one, 16 trees of 64 347 and 276.)
  p.parts = rows <= int64_t(128) * B ? 2 : 1;
  p.rows = 32 * p.waves;
  p.tiles = int(std::min<int64_t>(rows / p.rows + B, INT_MAX));
  // slots from the first to the last that a row tile may see
  int64_t most = max_len;
  if (window && tree_words) most = std::min<int64_t>(most, int64_t(window) + 32 * int64_t(tree_words) + 15);
  else if (window) most = std::min<int64_t>(most, 2 * int64_t(window) + p.rows + 15);
  else most = most + 15;
  // Runs.  Two workgroups a CU are resident; a run costs some 10 us beside its
  // slots (1.3 us a tile of 64), and 0.6 in the join by the last workgroup.  With
  // fewer row tiles than that: as many runs as make four a CU, or three where there
  // are several sequences (some of p.tiles are empty then, and some tiles short), of
  // 256 to 2048 slots, which a second launch joins, on more CUs but some 4 us later: a
  // tree of 25 behind 4000 takes 22.5 us in runs of 256, 24 in 192, 28 in runs of 384
  // that the last workgroup joins; 64 tokens behind 65536 take 121, 136 with three a
  // CU, 143 joined by the last; 4 sequences of 300 tokens behind up to 4000 each 52, 59
  // with four a CU, 66 joined by the last (all with one operand of P).
  // Where that makes one or two runs, of at least 384, and no second launch (256
  // tokens 14, 17 with one).  With more tiles, a single sequence's balance by
  // themselves, since those that see most start first; those of several may be of
  // any length: runs of up to 4096 (32 trees of 64, 32 / 8 heads, bf16, behind up to
  // 16384: 332 us, whole 443; behind 8192 each 399 and 371).
  const int64_t groups = int64_t(p.tiles) * c.kv_heads;
  int64_t chunk = most;
  bool second = false;
  if (groups <= kMaxArrived) {
    if (groups < 2 * cus) {
      chunk = std::min<int64_t>(2048, std::max<int64_t>(256, most * groups / ((B > 1 ? 3 : 4) * cus)));
      second = most > 2 * chunk;
      if (!second) chunk = std::max<int64_t>(384, chunk);
    } else if (B > 1) {
      chunk = 4096;
    }
    // at most 64 runs a tile and 16 workgroups a CU (the workspace has 64 KiB
    // for each at 128 elements)
    chunk = std::max({chunk, (most + kMaxJoin - 1) / kMaxJoin, most * groups / (16 * cus)});
    const int64_t runs = (most + chunk - 1) / chunk;   // of one size
    chunk = (most + runs - 1) / runs;
  }
  p.chunk = int(std::min<int64_t>((chunk + 63) & ~int64_t(63), INT_MAX & ~63));
  p.nsplit = int(std::max<int64_t>(1, (most + p.chunk - 1) / p.chunk));
  const size_t parts = p.nsplit > 1 ? size_t(groups) * p.nsplit * p.rows : 0;
  p.second = second && p.nsplit > 1;
  p.notes_off = parts ? GBB_ATTENTION_COUNTERS : 0;
  p.ml_off = p.notes_off + (p.second ? up(groups * sizeof(Note)) : 0);
  p.o_off = p.ml_off + up(parts * sizeof(float2));
  p.ws_bytes = p.o_off + up(parts * c.head_dim * sizeof(float));
  return p;
}

int launch_tokens(const gbb_paged_cache& c, const TokensArgs& x, const TokensPlan& p, void* stream) {
  Args a;
  a.q = x.q;
  a.k = static_cast<const uint8_t*>(c.k);
  a.v = static_cast<const uint8_t*>(c.v);
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.starts = x.starts;
  a.block_table = x.block_table;
  a.lengths = x.lengths;
  a.first = x.first;
  a.prefix = x.prefix;
  a.tree = x.tree;
  a.slopes = x.slopes;
  a.out = x.out;
  a.lse = x.lse;
  a.arrived = reinterpret_cast<unsigned*>(x.ws);
  a.ml = reinterpret_cast<float2*>(x.ws + p.ml_off);
  a.o = reinterpret_cast<float*>(x.ws + p.o_off);
  a.notes = p.second ? reinterpret_cast<Note*>(x.ws + p.notes_off) : nullptr;
  a.q_token = x.q_token;
  a.T = x.T;
  a.B = x.B;
  a.Hq = x.Hq;
  a.Hkv = c.kv_heads;
  a.G = x.Hq / c.kv_heads;
  a.num_pages = c.num_pages;
  a.pshift = __builtin_ctz(unsigned(c.page));
  a.max_pages = x.max_pages;
  a.max_len = x.max_len;
  a.chunk = p.chunk;
  a.nsplit = p.nsplit;
  a.tiles = p.tiles;
  a.tree_words = x.tree ? x.tree_words : 0;
  a.window = x.window;
  // a maximum of scaled scores is the scaled maximum for a scale above 0
  // (1e-30 gives the exponentials that 0 does, and keeps 0 * inf out)
  a.scale = std::max(std::fabs(x.scale), 1e-30f) * kLog2e;
  a.negative = x.scale < 0.f;
  a.cap = x.softcap * kLog2e;
  const unsigned grid = unsigned(p.tiles) * unsigned(c.kv_heads) * unsigned(p.nsplit);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (x.dtype == GBB_F16) {
    if (c.dtype == GBB_E4M3) run_dim<GBB_F16, GBB_E4M3>(a, c.head_dim, p, grid, s);
    else run_dim<GBB_F16, GBB_F16>(a, c.head_dim, p, grid, s);
  } else {
    if (c.dtype == GBB_E4M3) run_dim<GBB_BF16, GBB_E4M3>(a, c.head_dim, p, grid, s);
    else run_dim<GBB_BF16, GBB_BF16>(a, c.head_dim, p, grid, s);
  }
  if (p.second) {
    if (c.dtype != GBB_E4M3) a.v_scale = nullptr;
    if (x.dtype == GBB_F16) run_join<GBB_F16>(a, c.head_dim, p.rows, s);
    else run_join<GBB_BF16>(a, c.head_dim, p.rows, s);
  }
  return int(hipGetLastError());
}

}  // namespace gbb
