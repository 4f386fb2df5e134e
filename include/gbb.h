/*
 * gbb -- fused dequantize-and-multiply GEMV/GEMM over weight-only quantized
 * LLM layers, for AMD Instinct MI355X (gfx950).
 *
 * Two weight formats:
 *
 *  1. Block format.  The weight matrix W [N out][K in] is cut into blocks of
 *     64 output rows x 128 input columns; every block has one bitwidth
 *     b in {1,2,3,4,6,8} ("ScaleBITS: Scalable Bitwidth Search for
 *     Hardware-Aligned Mixed-Precision LLMs", explainer page, section 1.2.2
 *     "hardware-aligned block partition" and section 4.2 for the bitwidth set).
 *     Each (row, 128-column group) has an fp16 scale s and zero z; codes are
 *     q = clamp(rint(w / s) + z, 0, 2^b - 1) and dequantize as (q - z) * s
 *     ("MixLLM: LLM Quantization with Global Mixed-precision between
 *     Output-features and Highly-efficient System Design", section 2.1).
 *
 *  2. Output-feature mixed format ("W4.4A8", MixLLM page, sections 3.1.1 and
 *     3.3): a set of salient output rows is quantized 8-bit symmetric, the
 *     other rows 4-bit asymmetric, both with group 128, and multiplied with
 *     8-bit symmetric activations by a two-step dequantization: an integer
 *     product per group, then the two scales.
 *
 * Conventions for every entry point:
 *  - Matrices are row-major.  fp16 values are passed as their 16-bit patterns
 *    (uint16_t).  y = x . W^T: x is [M][K], y is [M][N].
 *  - "host" pointers are CPU memory; "device" pointers are GPU memory of the
 *    current HIP device (hipMalloc or a torch tensor).  The caller owns every
 *    buffer.  `stream` is a hipStream_t (NULL = the default stream).
 *  - Device entry points only validate arguments and enqueue kernels on
 *    `stream`; they never allocate, never synchronize and return before the
 *    work finishes.  Faults inside kernels are not reported by the call.
 *  - Nothing throws, aborts or prints.  A negative status is an error; the
 *    text of the last error of the calling thread is gbb_last_error().
 *  - Device pointers must be 16-byte aligned; x and y must not overlap.
 */
#ifndef GBB_H
#define GBB_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int gbb_status;

enum {
  GBB_OK = 0,
  GBB_E_ARG = -1,     /* null pointer, non-positive size, bad flag or option */
  GBB_E_SHAPE = -2,   /* N % 64 != 0 or K % 128 != 0 (block format), or bad row set */
  GBB_E_BITS = -3,    /* a bitwidth outside {1,2,3,4,6,8}, or a bad given zero */
  GBB_E_ALIGN = -4,   /* a device pointer that is not 16-byte aligned */
  GBB_E_SPACE = -5,   /* an output or workspace capacity that is too small */
  GBB_E_FORMAT = -6,  /* an image header that does not match the arguments */
  GBB_E_DEVICE = -7   /* a HIP runtime or launch error */
};

/* Text of the last non-OK status returned to this thread ("" if none). */
const char* gbb_last_error(void);

/* Library version: 10000 * major + 100 * minor + patch. */
int gbb_version(void);

/* ======================================================================== */
/* Block format                                                             */
/* ======================================================================== */

/* Byte size of the packed image for an N x K matrix with the per-block
 * bitwidth map `bits` (host, uint8 [N/64][K/128], block-row major): the
 * block-wise storage with a small per-block bitwidth record of the ScaleBITS
 * explainer page, section 3.2, in the layout of layout.h.  The size
 * is a 64-byte header, then 256-byte aligned sections: one byte per block,
 * 4 * (blocks + 1) bytes of offsets, 256 bytes of scale/zero per block and
 * 64 * 128 * b / 8 = 1024 * b bytes of codes per block.  Returns 0 on a bad
 * argument (see gbb_last_error). */
size_t gbb_packed_bytes(const uint8_t* bits, int N, int K);

#define GBB_PACK_GIVEN_SZ 1u  /* use the caller's scale/zero instead of min/max */

/* Quantize and pack (host, synchronous, deterministic; may use several CPU
 * threads).
 *   W      host fp16 [N][K].
 *   bits   host uint8 [N/64][K/128], each in {1,2,3,4,6,8}.
 *   scale, zero  host fp16 [N][K/128].  Without GBB_PACK_GIVEN_SZ they are
 *          outputs (may be NULL): per (row, group) s = fp16((max - min) /
 *          (2^b - 1)) and z = clamp(rint(-min / s), 0, 2^b - 1), decisions in
 *          fp64, round-half-even (MixLLM page, section 2.1, with min/max
 *          ranges).  With GBB_PACK_GIVEN_SZ they are inputs (e.g. scales from
 *          a clipping search): s must be finite and > 0, z an integer in
 *          [0, 2^b - 1].
 *   image  host output of gbb_packed_bytes(bits, N, K) bytes (image_cap).
 * Codes q = clamp(rint(w / s) + z, 0, 2^b - 1).  The image can be copied to
 * the device as is and shared by any number of streams. */
gbb_status gbb_pack_blocks(const uint16_t* W, int N, int K, const uint8_t* bits,
                           uint16_t* scale, uint16_t* zero, unsigned flags,
                           void* image, size_t image_cap);

/* Offline bitwidth allocation (host, synchronous, deterministic): one
 * bitwidth from {1,2,3,4,6,8} per 64x128 block with a mean of at most
 * target_bits, by the batched greedy of the ScaleBITS explainer page
 * (section 2.2: gamma * nblk blocks per round, gamma = 0.05 there; section
 * 4.2: the bitwidth set and the 3-bit start).  The pages' gradient
 * sensitivity needs a model and calibration data; here block i's cost at
 * bitwidth b is S_i * e_i(b), S_i = sum |w| over the block, e_i(b) = sum
 * (w - w')^2 under gbb_pack_blocks' quantizer.  Rounds lower the cheapest
 * blocks while over budget, raise the most beneficial ones that fit while
 * under it, then trade the most beneficial raises for the cheapest
 * lowerings that pay for them while that lowers the summed cost; ties go to
 * the lower block index.
 *   W            fp16 [N][K], finite; N % 64 == 0, K % 128 == 0.
 *   target_bits  mean bitwidth budget in [1, 8].
 *   gamma        fraction of the blocks moved per round, in (0, 1].
 *   bits         host output [N/64][K/128], row-major.
 * Errors: GBB_E_ARG (NULL, non-finite W, target or gamma out of range),
 * GBB_E_SHAPE. */
gbb_status gbb_allocate_bits(const uint16_t* W, int N, int K, double target_bits, double gamma,
                             uint8_t* bits);

/* Bidirectional channel reordering (ScaleBITS explainer page, section
 * 1.2.1) with |W| as the sensitivity: rows and columns by descending L1
 * norm (exact), ties to the lower index.  Packing W[row_order][:, col_order]
 * gathers the large weights in the top-left blocks; the caller permutes the
 * activations (x[:, col_order]) and un-permutes the outputs accordingly.
 *   W          fp16 [N][K], finite, any N, K > 0.
 *   row_order  host output [N] (a permutation of 0 ... N-1).
 *   col_order  host output [K].
 * Errors: GBB_E_ARG. */
gbb_status gbb_channel_order(const uint16_t* W, int N, int K, int32_t* row_order, int32_t* col_order);

/* Check a host copy of an image header against N and K (GBB_E_FORMAT): the
 * block-wise storage of the ScaleBITS explainer page, section 3.2 (version 1,
 * 64x128 blocks) or its 64x64 variant of section 4.2 (version 2). */
gbb_status gbb_check_image(const void* image, size_t image_bytes, int N, int K);

/* Workspace bytes gbb_gemm_mixed_w needs for (N, K, M) (the fused product of
 * the ScaleBITS explainer page, section 3.2, when its K range is split over
 * workgroups); may be 0.  On the decode route, when K is split across
 * workgroups, it is M * N * 12 (per output element an int64 fixed-point and
 * an fp32 accumulator), or for 17 <= M <= 32 on matrices of at least 2^26
 * weights (two block rows per workgroup) fp32 partials, segments * M * N * 4
 * bytes, summed in segment order by a second launch; for batches run as
 * 32-token chunks, that of the largest chunk; a smaller workspace is an
 * error.  On the prefill route it is
 * the fp32 partials of the K split described under
 * gbb_gemm_mixed_w_path_workspace, and a smaller workspace only shortens the
 * split.  The workspace must be zero-filled once before its first use; every
 * call leaves it zero-filled again.  Calls that run at the same time need
 * separate workspaces. */
size_t gbb_gemm_mixed_w_workspace(int N, int K, int M);
/* The same for gbb_gemm_mixed_w_path with a given path (0 equals
 * gbb_gemm_mixed_w_workspace).  For the prefill kernel (path 2, or path 0
 * when it takes the batch) the workspace holds the K split: when the tile
 * grid of 128 tokens x 512 rows fills at most half of the compute units,
 * each tile's K range is cut into up to 16 segments of at least 1024
 * columns, whose fp32 partials live in the workspace (segments * M * N * 4
 * bytes) until a second launch of the same call adds them in segment order
 * and clears them.  A prefill call whose
 * workspace is smaller (or NULL) takes as many segments as fit, down to
 * none; it never fails for lack of workspace. */
size_t gbb_gemm_mixed_w_path_workspace(int N, int K, int M, int path);

/* y = x . dequant(W)^T over a packed block image (ScaleBITS explainer page,
 * section 3.2: the weight is dequantized inside the matrix product, one
 * bitwidth per 64x128 block).
 *   image  device copy of gbb_pack_blocks' output for this N, K.
 *   x      device fp16 [M][K];  y device fp16 [M][N] (fp32 accumulation,
 *          round-to-nearest-even at the end).
 *   M >= 1.  M <= 32 runs the decode kernels (weights streamed once, matrix
 *   cores for the dot products).  Larger M runs the tiled prefill kernel,
 *   with its K range split into segments when its grid of 128-token x
 *   512-row tiles is small (see gbb_gemm_mixed_w_path_workspace), or the
 *   decode kernels in 32-token chunks, one launch each, when the chunks are
 *   few against the prefill grid: chunks x max(CUs / 4, split prefill
 *   workgroups) <= 3/4 of the device's compute units, a ragged last chunk
 *   counted as half.
 *   workspace/ws_bytes  device memory of gbb_gemm_mixed_w_workspace(N, K, M)
 *          bytes (NULL allowed when that is 0).  On the prefill route the
 *          number of K segments follows ws_bytes, and with it the order of
 *          the fp32 sums: for one ws_bytes the result is the same on every
 *          call, across sizes it may differ in the last bits.
 * Errors: GBB_E_ARG (NULL image/x/y, N or K <= 0, M < 0, x and y overlap,
 * missing workspace), GBB_E_SHAPE (N % 64, K % 128, N or K above 2^20, or
 * M * K >= 2^31 on the prefill kernel), GBB_E_ALIGN, GBB_E_SPACE (workspace
 * too small), GBB_E_DEVICE (launch failed).  M == 0 does nothing. */
gbb_status gbb_gemm_mixed_w(const void* image, int N, int K, const uint16_t* x,
                            uint16_t* y, int M, void* workspace, size_t ws_bytes,
                            void* stream);

/* Allocation-free variant of gbb_gemm_mixed_w, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.  Same arguments (without the workspace),
 * checks and kernels as gbb_gemm_mixed_w; the split-K accumulators live in a
 * fixed array of GBB_NOALLOC_SCRATCH_BYTES of device memory that the library
 * holds on each GPU it runs on, from the first call on that GPU until the
 * process ends.  That first call also zero-fills the array on `stream`
 * (again on later calls while the fills so far were recorded under stream
 * capture); every call leaves it zero.  All calls on one GPU share that
 * GPU's array, so calls that may overlap on one GPU (several streams or
 * threads, graphs replayed concurrently) race and give wrong results.  The
 * call allocates and frees nothing.
 * The prefill route's K split takes as many segments as the array holds, so
 * the result equals gbb_gemm_mixed_w's with ws_bytes =
 * GBB_NOALLOC_SCRATCH_BYTES.
 * Errors: those of gbb_gemm_mixed_w; GBB_E_SPACE when the decode route
 * needs more than GBB_NOALLOC_SCRATCH_BYTES of workspace (no shape the block
 * entry points accept needs more than 12 MiB);
 * GBB_E_DEVICE when the array's address cannot be obtained. */
#define GBB_NOALLOC_SCRATCH_BYTES (16u << 20)
gbb_status gbb_gemm_mixed_w_noalloc(const void* image, int N, int K, const uint16_t* x,
                                    uint16_t* y, int M, void* stream);

/* Grouped products: n (1 ... 32) independent block GEMMs y[i] = x[i] .
 * dequant(W_i)^T with one M, for products that do not depend on each other
 * (the concurrent sub-problems of the MixLLM page, section 3.3; the
 * per-bitwidth execution plan of the ScaleBITS explainer page, section 3.2).
 * For M <= 16 all of them run as ONE launch of the decode kernels: problem
 * i's workgroups follow problem i-1's in a single grid, so small products
 * share the GPU instead of paying a launch and a ramp each.  For larger M
 * the problems run one after another, as gbb_gemm_mixed_w runs them.
 *   images[i]  device image of N[i] x K[i] (gbb_pack_blocks).
 *   x[i], y[i] device fp16 [M][K[i]] and [M][N[i]]; no y may overlap another
 *              problem's x or y.
 *   workspace  device memory of gbb_gemm_mixed_w_batched_workspace(n, N, K,
 *              M) bytes (NULL allowed when that is 0), zero-filled once
 *              before first use; every call leaves it zero-filled.
 * Errors: GBB_E_ARG (n outside 1 ... 32, NULL arrays, missing workspace),
 * those of gbb_gemm_mixed_w for each problem (with its index in the
 * message), GBB_E_SPACE, GBB_E_DEVICE. */
size_t gbb_gemm_mixed_w_batched_workspace(int n, const int* N, const int* K, int M);
gbb_status gbb_gemm_mixed_w_batched(int n, const void* const* images, const int* N, const int* K,
                                    const uint16_t* const* x, uint16_t* const* y, int M,
                                    void* workspace, size_t ws_bytes, void* stream);

/* Whole-layer execution (ScaleBITS explainer page, section 3.2: an execution
 * plan generated for a given bit configuration; MixLLM page, section 3.3:
 * the kernels of a step replayed from a captured graph).  Captures n
 * gbb_gemm_mixed_w calls, in order, into one HIP graph: call i multiplies
 * x[i] (device fp16 [M][K[i]]) by images[i] (device, N[i] x K[i]) into y[i]
 * (device fp16 [M][N[i]]).  Every pointer is recorded as is and must stay
 * valid, with the same shapes, for the graph's life; each call is checked as
 * gbb_gemm_mixed_w checks it, and the first failing call's status is
 * returned.  The calls share one workspace (device, zero-filled once before
 * the first launch, ws_bytes >= the largest gbb_gemm_mixed_w_workspace of
 * the calls); they run one after the other and leave it zero-filled, so
 * launches of the graph on one stream may follow each other, but launches
 * that may run at the same time need graphs with separate workspaces.  Host
 * call; captures on a stream of its own (default priority), allocates only
 * the graph.  On success *out owns the graph.
 * Errors: GBB_E_ARG (NULL, n < 1, M < 1), those of gbb_gemm_mixed_w,
 * GBB_E_DEVICE (capture or instantiation failed). */
typedef struct gbb_graph gbb_graph;
gbb_status gbb_graph_create(int n, const void* const* images, const int* N, const int* K,
                            const uint16_t* const* x, uint16_t* const* y, int M,
                            void* workspace, size_t ws_bytes, gbb_graph** out);

/* Launch a captured graph on `stream` (asynchronous). */
gbb_status gbb_graph_launch(const gbb_graph* g, void* stream);

/* Free a graph (NULL is allowed).  The caller makes sure no launch of it is
 * still running. */
gbb_status gbb_graph_destroy(gbb_graph* g);

/* Same as gbb_gemm_mixed_w with the kernel chosen by `path`: 0 = automatic,
 * 1 = decode kernel (requires M <= 32), 2 = prefill kernel.  For tests. */
gbb_status gbb_gemm_mixed_w_path(const void* image, int N, int K, const uint16_t* x,
                                 uint16_t* y, int M, void* workspace, size_t ws_bytes,
                                 int path, void* stream);

/* Debug exports over a device image, for bit-exactness tests.
 *   gbb_unpack_codes: q device uint8 [N][K], the codes read back from the
 *   block-wise storage (ScaleBITS explainer page, section 3.2).
 *   gbb_dequant: the affine dequantization of the MixLLM page, section 2.1:
 *   w32 device fp32 [N][K] = (q - z) * s (exact), and/or w16
 *   device fp16 [N][K] = its round-to-nearest-even (either may be NULL). */
gbb_status gbb_unpack_codes(const void* image, int N, int K, uint8_t* q, void* stream);
gbb_status gbb_dequant(const void* image, int N, int K, float* w32, uint16_t* w16,
                       void* stream);

/* ------------------------------------------------------------------------ */
/* 64x64 blocks (the other GPU block size of the ScaleBITS explainer page,  */
/* section 4.2): 64 output rows x 64 input columns per block, one bitwidth  */
/* per block, scale/zero per (row, 64-column group).  The image is version  */
/* 2 of the block image: 512 * b bytes of codes per block.  Each call below */
/* is its 64x128 counterpart's with K a multiple of 64 and bits [N/64][K/64].*/
/* ------------------------------------------------------------------------ */
size_t gbb_packed_bytes_64x64(const uint8_t* bits, int N, int K);
gbb_status gbb_pack_blocks_64x64(const uint16_t* W, int N, int K, const uint8_t* bits,
                                 uint16_t* scale, uint16_t* zero, unsigned flags,
                                 void* image, size_t image_cap);
/* y = x . dequant(W)^T over a version-2 image, with the arguments, layout,
 * workspace rules and errors of gbb_gemm_mixed_w / gbb_gemm_mixed_w_path
 * (K % 64 == 0).  M <= 32 runs the 64x64 decode kernels; larger M runs the
 * 64x64 prefill kernel (M * K < 2^31; K split into segments of at least
 * 1024 columns as for 64x128 blocks), or the decode kernels in 32-token
 * chunks under the same rule as for 64x128 blocks.  path: 0 that choice, 1 the decode
 * kernel (M <= 32), 2 the prefill kernel. */
size_t gbb_gemm_mixed_w_64x64_workspace(int N, int K, int M);
gbb_status gbb_gemm_mixed_w_64x64(const void* image, int N, int K, const uint16_t* x,
                                  uint16_t* y, int M, void* workspace, size_t ws_bytes,
                                  void* stream);
size_t gbb_gemm_mixed_w_64x64_path_workspace(int N, int K, int M, int path);
gbb_status gbb_gemm_mixed_w_64x64_path(const void* image, int N, int K, const uint16_t* x,
                                       uint16_t* y, int M, void* workspace, size_t ws_bytes,
                                       int path, void* stream);
gbb_status gbb_unpack_codes_64x64(const void* image, int N, int K, uint8_t* q, void* stream);
gbb_status gbb_dequant_64x64(const void* image, int N, int K, float* w32, uint16_t* w16,
                             void* stream);

/* ======================================================================== */
/* Output-feature mixed format, W8 (symmetric) / W4 (asymmetric) x A8       */
/* ======================================================================== */

/* Byte size of the W4/W8 image for N x K with n8 8-bit rows (0 on error):
 * the output-feature mixed format of the MixLLM page, sections 3.1.1 and
 * 3.1.2, pre-packed as in section 3.3. */
size_t gbb_w48_packed_bytes(int N, int K, int n8);

/* Quantize and pack (host, synchronous, deterministic).
 *   W      host fp16 [N][K], K % 128 == 0.
 *   rows8  host int32 [n8], strictly ascending output rows that get 8-bit
 *          symmetric codes (s = fp16(max|w| / 127), q = clamp(rint(w / s),
 *          -127, 127)); every other row gets 4-bit asymmetric codes as in
 *          gbb_pack_blocks (MixLLM page, sections 3.1.1 and 3.1.2).
 *   scale  host fp16 [N][K/128] output in original row order (may be NULL).
 *   zero   host uint8 [N][K/128] output, 0 for 8-bit rows (may be NULL).
 *   image  host output of gbb_w48_packed_bytes(N, K, n8) bytes. */
gbb_status gbb_pack_w48(const uint16_t* W, int N, int K, const int32_t* rows8, int n8,
                        uint16_t* scale, uint8_t* zero, void* image, size_t image_cap);

/* 8-bit symmetric activation quantization (MixLLM page, section 3.1.2):
 * per token (ga == K) or per group of 128 columns (ga == 128).  Decisions in
 * fp32: s = fp16(max|x| / 127) (1 if the group is all zero),
 * xq = clamp(rint(x / s), -127, 127).
 *   x  device fp16 [M][K];  xq device int8 [M][K];  xs device fp16 [M][K/ga]. */
gbb_status gbb_quant_act_i8(const uint16_t* x, int M, int K, int ga, int8_t* xq,
                            uint16_t* xs, void* stream);

/* y = dequant(xq) . dequant(W)^T by two-step dequantization (MixLLM page,
 * section 3.3): per 128-group an exact int32 product xq . (q - z) on the int8
 * matrix cores, then scaled by s_a * s_w and accumulated in fp32; each output
 * is written straight to its original row (fused scatter).
 *   image  device copy of gbb_pack_w48's output.
 *   xq, xs as produced by gbb_quant_act_i8 with the same ga (K or 128).
 *   y      device fp16 [M][N]. */
gbb_status gbb_gemm_w48a8(const void* image, int N, int K, int n8, const int8_t* xq,
                          const uint16_t* xs, int ga, uint16_t* y, int M, void* stream);

/* Workspace bytes for gbb_gemm_w48a8_split (0 when the call does not split
 * K, or on invalid arguments): the fp32 partial sums of the K split,
 * segments x M x padded rows x 4 bytes (M at most 64, the tokens of one pass,
 * on the streaming kernel; padded rows: each of the two row sets rounded up
 * to a multiple of 16). */
size_t gbb_gemm_w48a8_workspace(int N, int K, int n8, int M, int ga);

/* gbb_gemm_w48a8 with a caller workspace, for batches on matrices with few
 * output rows per compute unit (MixLLM page, section 3.3: the same
 * two-step product over a K range cut into segments).  The streaming kernel
 * (M <= 64 per pass; per-token activation scales, or per-group ones over an
 * even number of groups with xs 4-byte aligned) splits K where its 64-row
 * blocks, an 8-bit one counted twice, number at most 3/4 of the compute
 * units; it then streams 128-row blocks, and each one's 128-column groups
 * are cut into up to 16 segments of at least 8 groups, an 8-bit row block
 * into twice as many as a 4-bit one, so that every workgroup streams about
 * the same bytes.  The tile
 * kernel (larger M) splits K where its token tiles x row blocks fill at most
 * half of its resident workgroups, a 4-bit row block (twice the rows)
 * counted twice and cut into twice the segments.  Each segment writes its
 * fp32 sum of s_w-scaled group products (with per-group activation scales,
 * of s_a s_w-scaled ones) for every output to the workspace; a second
 * launch adds the segments in order, multiplies by the per-token s_a,
 * rounds to fp16, writes each output to its original row and clears the
 * workspace.  With a workspace smaller than gbb_gemm_w48a8_workspace(N, K,
 * n8, M, ga) (or NULL) the call takes as many segments as fit, down to none
 * (then it equals gbb_gemm_w48a8).  The segment counts fix the order of the
 * fp32 sums: for one ws_bytes the result is the same on every call.
 *   workspace/ws_bytes  device memory, 16-byte aligned, zero-filled before
 *          its first use (every call leaves it zero); calls that may overlap
 *          need separate workspaces.
 * Errors: those of gbb_gemm_w48a8; GBB_E_ALIGN for a misaligned workspace. */
gbb_status gbb_gemm_w48a8_split(const void* image, int N, int K, int n8, const int8_t* xq,
                                const uint16_t* xs, int ga, uint16_t* y, int M, void* workspace,
                                size_t ws_bytes, void* stream);

/* Debug export of the first step of the two-step dequantization (MixLLM
 * page, section 3.3: per group an exact integer product of the int8
 * activations and the int8 weight codes (q - z), before any scale):
 * acc[m][n][g] = sum over group g of xq[m][k] * (q[n][k] - z[n][g]) for every
 * original row n (device int32 [M][N][K/128]), for bit-exact tests.  The call
 * runs the kernel gbb_gemm_w48a8 runs for the same M and ga (K or 128), with
 * that kernel's scaling step replaced by a store of the group sums, so the
 * integers checked are those the product path forms (where the product
 * kernel starts a group's sums from the constant 0x4B400000 so that the
 * result reads as a float, its integers are these plus that constant); the
 * streaming kernel runs with the K segments that gbb_gemm_w48a8_split takes
 * with a full workspace.  Errors as gbb_gemm_w48a8. */
gbb_status gbb_w48_group_acc(const void* image, int N, int K, int n8, const int8_t* xq, int ga,
                             int32_t* acc, int M, void* stream);

/* ======================================================================== */
/* The rest of a decoding step's attention: rotary positions, a paged       */
/* key-value cache, attention of one new token over it, and eviction        */
/* ======================================================================== */

/* Element types (the values of every `dtype` argument below). */
enum {
  GBB_F16 = 0,    /* IEEE binary16 */
  GBB_BF16 = 1,   /* bfloat16 */
  GBB_F32 = 2,    /* IEEE binary32 (gbb_rope only) */
  GBB_E4M3 = 3    /* OCP 8-bit e4m3 without infinities, largest 448 (caches only) */
};

/* How a rotated head pairs its first `rot` elements. */
enum {
  GBB_ROPE_HALF = 0,          /* (i, i + rot/2) */
  GBB_ROPE_INTERLEAVED = 1    /* (2i, 2i + 1) */
};

/* Scalings of the rotary frequencies f_i = base^(-2i/rot) for contexts
 * longer than the model's own (F = factor, L = original_len). */
enum {
  GBB_ROPE_PLAIN = 0,    /* f_i */
  GBB_ROPE_LINEAR = 1,   /* f_i / F */
  GBB_ROPE_BANDS = 2,    /* by the wave length w = 2 pi / f_i: f_i where w < L / high, f_i / F where
                            w > L / low, else (1 - t) f_i / F + t f_i with t = (L / w - low) / (high - low) */
  GBB_ROPE_YARN = 3      /* by the pair's index ("YaRN: Efficient Context Window Extension of Large Language
                            Models"): with d(r) = rot ln(L / (2 pi r)) / (2 ln base), a = max(floor(d(high)), 0),
                            b = min(ceil(d(low)), rot - 1) and t = clamp((i - a) / max(b - a, 0.001), 0, 1):
                            (1 - t) f_i + t f_i / F */
};

typedef struct {
  int kind;              /* GBB_ROPE_PLAIN ... GBB_ROPE_YARN */
  double factor;         /* F >= 1; ignored by PLAIN */
  double original_len;   /* L > 0; BANDS and YARN */
  double low, high;      /* BANDS: 0 < low < high (wave lengths per L); YARN: turns per L, 0 < low < high */
  double attention;      /* multiplies every cos and sin (1: none); finite and not 0 */
} gbb_rope_scaling;

/* Table of rotations (host, synchronous, may use several CPU threads):
 * table[p][i] = (cos(p f_i), sin(p f_i)) * attention for p < n_pos and
 * i < rot/2, each computed in double and rounded once; float
 * [n_pos][rot/2][2].  scaling NULL is PLAIN with attention 1.
 * Errors: GBB_E_ARG (NULL, rot odd or not positive, n_pos <= 0, base not
 * above 1, a scaling outside the ranges above). */
gbb_status gbb_rope_table(int rot, int n_pos, double base, const gbb_rope_scaling* scaling, float* table);

/* Rotary positions: for every token t < T and head h < H, pair i of the
 * head's first `rot` elements (x1, x2) becomes (x1 c - x2 s, x2 c + x1 s)
 * with (c, s) = table[positions[t]][i], in fp32 and rounded once; elements
 * rot ... D - 1 are copied.  transpose != 0 takes -s for s: the transposed
 * map, which is the gradient with respect to x of a call without it (and,
 * for a table with attention 1, its inverse).
 *   x, y       device, `dtype` GBB_F16, GBB_BF16 or GBB_F32: element d of
 *              head h of token t is at t * token stride + h * head stride
 *              + d (strides in elements, 16-byte alignment not required;
 *              tokens or heads may be the outer dimension, and x's strides
 *              may be 0).  y == x with equal strides works in place;
 *              otherwise x and y must not overlap.
 *   positions  device int32 [T]; table device float [n_pos][rot/2][2].  A
 *              token whose position is outside [0, n_pos) is padding: its
 *              y is zero.
 * T = 0 is a no-op.  Errors: GBB_E_ARG, GBB_E_SHAPE (D odd or above 1024,
 * rot odd, below 2 or above D, heads of y that overlap), GBB_E_ALIGN
 * (a pointer that is not aligned to its element), GBB_E_DEVICE. */
gbb_status gbb_rope(const void* x, int64_t x_token, int64_t x_head, void* y, int64_t y_token, int64_t y_head,
                    int dtype, int T, int H, int D, const int32_t* positions, const float* table, int n_pos,
                    int rot, int layout, int transpose, void* stream);

/* A paged cache of keys and values.  Slot s is token s % page of page
 * s / page.  All pointers are device memory that the caller owns; k, v,
 * weights and positions are 16-byte aligned. */
typedef struct {
  void* k;                /* [num_pages][kv_heads][page][head_dim], dtype */
  void* v;                /* the same shape and dtype */
  const float* k_scale;   /* [kv_heads], GBB_E4M3 only: an element stands for its value times this */
  const float* v_scale;   /* (NULL: 1; finite and above 0, which is not checked) */
  float* weights;         /* [num_pages][kv_heads][page] attention weight that a slot gathered, or NULL */
  int32_t* positions;     /* [num_pages][kv_heads][page] position of a slot's token, or NULL */
  int dtype;              /* GBB_F16, GBB_BF16 or GBB_E4M3 */
  int num_pages;          /* num_pages * page < 2^31 */
  int page;               /* 16, 32, 64, 128 or 256 tokens */
  int kv_heads;
  int head_dim;           /* 64, 128 or 256 */
} gbb_paged_cache;

/* Rotary positions of a fused q|k|v product's output, with k and v written
 * to the cache in the same pass.
 *   qkv        device [T][token_stride], dtype GBB_F16 or GBB_BF16: q_heads
 *              query heads, then the cache's kv_heads key heads, then as
 *              many value heads, head_dim elements each.
 *   positions, table, n_pos, rot, layout  as gbb_rope.
 *   slots      device int32 [T]: the cache slot of each token.  Two tokens
 *              of a call must not name the same slot.
 *   q          device [T][q_heads][head_dim]: the rotated query heads.
 *   cache      k (rotated) and v; its dtype is that of qkv, or GBB_E4M3:
 *              then an element is value / scale (fp32), clamped to +-448
 *              and rounded to nearest even.  A NaN stays one.
 *              Where the cache has them, positions[slot] = the token's
 *              position and weights[slot] = 0 for every kv head.
 * A token whose position is outside [0, n_pos) or whose slot is outside the
 * cache is padding: its q is zero and it is not written to the cache.
 * T = 0 is a no-op.  Errors: GBB_E_ARG, GBB_E_SHAPE, GBB_E_ALIGN (qkv, q,
 * k, v and table 16-byte aligned, token_stride a multiple of 8),
 * GBB_E_DEVICE. */
gbb_status gbb_rope_append(const gbb_paged_cache* cache, const void* qkv, int64_t token_stride, int dtype, int T,
                           int q_heads, const int32_t* positions, const int32_t* slots, const float* table,
                           int n_pos, int rot, int layout, void* q, void* stream);

/* Bytes of workspace of gbb_paged_attention (0 on a bad argument or where
 * none is needed).  Its first GBB_ATTENTION_COUNTERS bytes (all of it, if it
 * is smaller) must be zero before its first use: with other contents outputs
 * stay unwritten, without an error.  Every call leaves it ready for the next
 * one of any size, but not zero: it must not be shared with calls that want a
 * zero workspace (gbb_gemm_*), with gbb_cache_evict, which leaves it in any
 * state, or with a call that may run at the same time. */
#define GBB_ATTENTION_COUNTERS 16384
size_t gbb_paged_attention_workspace(const gbb_paged_cache* cache, int B, int q_heads, int max_len, int with_weights);

/* Attention of one new token per sequence over the cache:
 * for query head h of sequence b, with kv head h / (q_heads / kv_heads) and
 * s_j = scale * (q . k_j) over the slots j < lengths[b] of the sequence,
 * out = sum_j p_j v_j, p_j = exp(s_j) / sum_j exp(s_j); fp32 sums, one
 * rounding of out.  A sequence of length 0 gives zeros (so does a head
 * whose scores are all -inf).  Memory past the length is never used, so it
 * may hold anything, NaN included.  An infinity of v among the slots may come
 * out as NaN (weights go into the product in two or three parts).
 *   q, out     device [B][q_heads][head_dim] of `dtype` (GBB_F16 or
 *              GBB_BF16; the cache's dtype or a GBB_E4M3 cache); sequence b
 *              of q is at b * q_token elements.
 *   block_table device int32 [B][max_pages]: slot j of sequence b is token
 *              j % page of page block_table[b][j / page].  An entry outside
 *              [0, num_pages) is a page that is not there: its slots take no
 *              part.
 *   lengths    device int32 [B], at most max_len (larger ones are taken as
 *              max_len, negative ones as 0).
 *   max_len    an upper bound on the lengths, at most max_pages * page.  The
 *              split over the length is planned for it.
 *   lse        NULL, or device float [B][q_heads]: log(sum_j exp(s_j)), -inf
 *              for an empty sequence: what joining the outputs over parts of
 *              a context takes.
 *   weights_out NULL, or like the cache's weights (which must be there, and
 *              may be the same memory, but not overlap it in part): for every slot j < lengths[b] the
 *              cache's weight plus the sum of p_j over the kv head's query
 *              heads.  Other slots are not written.  No atomics: results do
 *              not depend on the order of execution.  Two sequences of a
 *              call must not share a page then.
 *   workspace  16-byte aligned, of gbb_paged_attention_workspace bytes.
 * B = 0 is a no-op.  Errors: GBB_E_ARG, GBB_E_SHAPE, GBB_E_ALIGN,
 * GBB_E_SPACE, GBB_E_DEVICE. */
gbb_status gbb_paged_attention(const gbb_paged_cache* cache, const void* q, int64_t q_token, int dtype, int B,
                               int q_heads, const int32_t* block_table, int max_pages, const int32_t* lengths,
                               int max_len, float scale, void* out, float* lse, float* weights_out,
                               void* workspace, size_t ws_bytes, void* stream);

/* Bytes of workspace of gbb_cache_evict (0 on a bad argument).  Its contents
 * need no initialisation.  Calls that may run at the same time need separate
 * workspaces. */
size_t gbb_cache_evict_workspace(const gbb_paged_cache* cache, int B, int max_len, int budget);

/* Eviction by accumulated attention weight.  For every sequence b and kv
 * head with lengths[b] > budget, `budget` of the first lengths[b] slots are
 * kept: first those whose position is above (the largest position among
 * them) - recent, then those of the largest weight (a NaN ranks below
 * everything, -0 as 0); ties go to the lower slot.  Kept slots below budget
 * stay where they are; the i-th dropped slot below budget takes k, v, weight
 * and position of the i-th kept slot from budget on.  So slots are in no
 * order afterwards, which attention over rotated keys does not need, and no
 * more rows move than have to.
 *   lengths_out device int32 [B], not overlapping lengths: min(lengths[b],
 *              budget).
 *   weights_out, positions_out  like the cache's weights and positions
 *              (both must be there), and may be the same memory; in other
 *              memory, all slots below lengths[b] are written.  Slots from
 *              the new length up to lengths[b] get weight 0 and position -1.
 *   0 <= recent <= budget, 1 <= budget, 1 <= max_len <= max_pages * page,
 *   max_len <= 2^21.
 * k and v change in place.  Two sequences must not share a page.  A sequence
 * with an entry outside [0, num_pages) among its pages is left as it is.
 * B = 0 is a no-op.  Errors: GBB_E_ARG, GBB_E_SHAPE, GBB_E_ALIGN,
 * GBB_E_SPACE, GBB_E_DEVICE. */
gbb_status gbb_cache_evict(const gbb_paged_cache* cache, int B, const int32_t* block_table, int max_pages,
                           const int32_t* lengths, int max_len, int budget, int recent, int32_t* lengths_out,
                           float* weights_out, int32_t* positions_out, void* workspace, size_t ws_bytes,
                           void* stream);

/* ======================================================================== */
/* Norms of heads, positions of several axes, and attention of prompts and  */
/* drafted tokens over the paged cache                                      */
/* ======================================================================== */

/* Rotations of one to four axes.  Where a call takes `axes` and `sections`,
 * positions is device int32 [axes][T] and pair i of the rot/2 pairs turns by
 * the token's position on axis a, the first with i < sections[0] + ... +
 * sections[a]: (c, s) = table[positions[a][t]][i].  sections is a host array of
 * `axes` counts, 0 or more, whose sum is rot/2 (NULL with one axis).  A token
 * with a position outside [0, n_pos) on any axis is padding. */
#define GBB_MAX_AXES 4

/* gbb_rope with positions of several axes: every argument as there. */
gbb_status gbb_rope_axes(const void* x, int64_t x_token, int64_t x_head, void* y, int64_t y_token, int64_t y_head,
                         int dtype, int T, int H, int D, const int32_t* positions, int axes, const int* sections,
                         const float* table, int n_pos, int rot, int layout, int transpose, void* stream);

/* Norm of every head and its rotation in one pass: y = R(x r w) with r =
 * (mean x^2 + eps)^(-1/2) over the head's D elements, w = weight and R the
 * rotation of gbb_rope (R does not change the elements from rot on); fp32,
 * one rounding of y.
 *   x, y       device, as gbb_rope (in place too); padding tokens give zeros.
 *   weight     device [D] of weight_dtype, which is GBB_F32 or `dtype`; NULL: ones.
 *   eps        0 or more, finite.
 * T = 0 is a no-op.  Errors: those of gbb_rope. */
gbb_status gbb_norm_rope(const void* x, int64_t x_token, int64_t x_head, void* y, int64_t y_token, int64_t y_head,
                         int dtype, int T, int H, int D, const void* weight, int weight_dtype, float eps,
                         const int32_t* positions, int axes, const int* sections, const float* table, int n_pos,
                         int rot, int layout, void* stream);

/* Its gradient: with g = R^T dy and u = x r,
 *   dx = r (g w - u mean(g w u)),  dweight = sum over tokens and heads of g u;
 * fp32 sums in an order that only the sizes set, one rounding.  Padding
 * tokens have dx 0 and no part in dweight.
 *   x, dy, dx  device, of `dtype`, strides as gbb_rope's x (x, dy) and y
 *              (dx).  dx may be NULL, or dy with equal strides; otherwise it
 *              must not overlap x or dy.
 *   dweight    device [D] of weight_dtype, or NULL.  T = 0 makes it 0.
 *   workspace  device, 16-byte aligned, gbb_norm_rope_grad_workspace bytes
 *              where dweight is given; its contents need no initialisation.
 * Errors: those of gbb_rope, GBB_E_SPACE. */
size_t gbb_norm_rope_grad_workspace(int T, int H, int D);
gbb_status gbb_norm_rope_grad(const void* x, int64_t x_token, int64_t x_head, const void* dy, int64_t dy_token,
                              int64_t dy_head, void* dx, int64_t dx_token, int64_t dx_head, int dtype, int T, int H,
                              int D, const void* weight, int weight_dtype, float eps, const int32_t* positions,
                              int axes, const int* sections, const float* table, int n_pos, int rot, int layout,
                              void* dweight, void* workspace, size_t ws_bytes, void* stream);

/* gbb_rope_append with norms of the q and k heads before their rotation (as
 * gbb_norm_rope, over head_dim elements) and positions of several axes.
 *   q_weight, k_weight  device [head_dim] of weight_dtype (GBB_F32 or
 *              `dtype`); both NULL: no norms.
 * The cache's positions, where it has them, are those of the first axis. */
gbb_status gbb_norm_rope_append(const gbb_paged_cache* cache, const void* qkv, int64_t token_stride, int dtype, int T,
                                int q_heads, const void* q_weight, const void* k_weight, int weight_dtype, float eps,
                                const int32_t* positions, int axes, const int* sections, const int32_t* slots,
                                const float* table, int n_pos, int rot, int layout, void* q, void* stream);

/* What shapes the scores s = scale * (q . k) of attention, and what is seen. */
typedef struct {
  float softcap;          /* above 0: s becomes softcap * tanh(s / softcap); 0: none.  Of 1e-30 to 1e30, and of
                             1e-30 |scale| or more */
  const float* slopes;    /* device [q_heads], or NULL: then s (capped) minus slopes[head] * distance */
  int window;             /* above 0: only slots at a distance below it are seen; 0: no such limit */
  /* the rest for gbb_paged_attention_tokens alone: */
  const int32_t* first;   /* device [T], or NULL: token t sees no slot before first[t] (packed documents, padding) */
  const int32_t* prefix;  /* device [B], or NULL: the slots below prefix[b] are seen by all of b's tokens */
  const uint32_t* tree;   /* device [T][tree_words], or NULL: bit j of token t's row: it sees new token j */
  int tree_words;
} gbb_attention_options;

/* gbb_paged_attention with a cap, a bias by distance or a window: the token
 * is that of slot lengths[b] - 1, and the distance of slot j is lengths[b] - 1
 * - j.  Slots that are not seen have no weight (weights_out holds the cache's
 * there) and may hold anything.  options NULL is gbb_paged_attention. */
size_t gbb_paged_attention_options_workspace(const gbb_paged_cache* cache, int B, int q_heads, int max_len,
                                             int with_weights, int window);
gbb_status gbb_paged_attention_options(const gbb_paged_cache* cache, const void* q, int64_t q_token, int dtype, int B,
                                       int q_heads, const int32_t* block_table, int max_pages, const int32_t* lengths,
                                       int max_len, float scale, const gbb_attention_options* options, void* out,
                                       float* lse, float* weights_out, void* workspace, size_t ws_bytes, void* stream);

/* Attention of several new tokens per sequence over the cache that holds
 * them already: prompts, chunks of them, trees of drafted tokens.
 * Sequence b has the tokens starts[b] ... starts[b + 1] - 1, n_b of them, in
 * the last n_b of its lengths[b] slots: token starts[b] + i has slot p =
 * lengths[b] - n_b + i.  It sees slot j < lengths[b] of a page that is there if
 *   without a tree: j <= p, or j < prefix[b];
 *   with a tree: j < lengths[b] - n_b, or bit j - (lengths[b] - n_b) of its
 *     row of the tree is set (bits from n_b on do not count);
 *   and j >= first[t], and the distance of j is below the window.
 * The distance is |p - j| without a tree; with one it is counted along the
 * tree: the number of new tokens that it sees (by the tree alone) behind slot j
 * if that is a new token's, else lengths[b] - n_b - 1 - j plus the number of
 * all new tokens that it sees.
 * out and lse as gbb_paged_attention, for every token; a row that sees nothing
 * gives zeros and -inf.  A slot that a token does not see may hold anything,
 * NaN included; one that it sees with a weight that rounds to 0 counts as such.
 *   q, out     device [T][q_heads][head_dim] of `dtype` (as
 *              gbb_paged_attention); token t of q is at t * q_token elements.
 *   starts     device int32 [B + 1], rising, within [0, T] (values outside
 *              are taken as the nearer end, a falling pair as no tokens).
 *              Tokens outside all sequences are not read, and their outputs
 *              not written.
 *   block_table, lengths, max_len  as gbb_paged_attention.
 *   scale      of -1e30 to 1e30.
 *   options    NULL, or what shapes and masks the scores; tree and prefix
 *              exclude each other.
 *   workspace  16-byte aligned, of gbb_paged_attention_tokens_workspace bytes
 *              (for the same options' window and tree_words, 0 without a
 *              tree); to be had and shared as that of gbb_paged_attention.
 * Sums, maxima and lse are fp32.  Probabilities are rounded to `dtype` once
 * where T * q_heads / kv_heads is above 128 B (an output is then off by up to
 * half a step of `dtype` relative to sum p |v|, beside its own rounding), and
 * carry twice its bits in other calls.  A capped score, and so lse, is off by up
 * to 2^-21 of a softcap of up to 80, whatever the score's size.
 * T = 0 or B = 0 is a no-op.  Results do not depend on the order of execution.
 * Errors: GBB_E_ARG, GBB_E_SHAPE, GBB_E_ALIGN, GBB_E_SPACE, GBB_E_DEVICE. */
size_t gbb_paged_attention_tokens_workspace(const gbb_paged_cache* cache, int T, int B, int q_heads, int max_len,
                                            int window, int tree_words);
gbb_status gbb_paged_attention_tokens(const gbb_paged_cache* cache, const void* q, int64_t q_token, int dtype, int T,
                                      int B, int q_heads, const int32_t* starts, const int32_t* block_table,
                                      int max_pages, const int32_t* lengths, int max_len, float scale,
                                      const gbb_attention_options* options, void* out, float* lse, void* workspace,
                                      size_t ws_bytes, void* stream);

/* Keeps some of a sequence's newest slots, in their order: of the last
 * drafted[b] of lengths[b] slots those numbered kept[b][i], i < counts[b], move
 * to the first counts[b] places of them, with their weights and positions where
 * the cache has them, for every kv head.  The slots behind are left as they are.
 *   drafted, counts  device int32 [B]; kept device int32 [B][max_kept],
 *              rising, within [0, drafted[b]).
 *   lengths_out device int32 [B], not overlapping any input: lengths[b] -
 *              drafted[b] + counts[b].
 * A sequence with numbers outside these ranges, or with a missing page among
 * the slots that it moves between, is left as it is, its length too.  Two
 * sequences must not share a page among these slots.
 * B = 0 is a no-op.  Errors: GBB_E_ARG, GBB_E_SHAPE, GBB_E_ALIGN, GBB_E_DEVICE. */
gbb_status gbb_cache_keep(const gbb_paged_cache* cache, int B, const int32_t* block_table, int max_pages,
                          const int32_t* lengths, const int32_t* drafted, const int32_t* kept, int max_kept,
                          const int32_t* counts, int32_t* lengths_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GBB_H */
