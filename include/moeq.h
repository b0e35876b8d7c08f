/*
 * moeq.h - C ABI of the MI355X (gfx950) block-quantized routed-MoE library.
 *
 * The library computes the routed-expert projection of a DeepSeek-V4-Flash-shaped
 * MoE layer (DeepSeek-V4-Flash W4A16-FP8 model card, "Architecture & precision",
 * base-model table: 256 routed experts, top-6, hidden 4096, 43 layers) with expert
 * weights in block-quantized formats, on one GPU:
 *
 *   for token t routed to experts e_k with route weights w_k (k < top_k):
 *     h_k = silu(G_e x_t) * (U_e x_t),   y_t = sum_k w_k * (D_e h_k)
 *
 * At decode (few tokens) each projection streams the routed experts' weights:
 * MXFP4 and NVFP4 gate/up and MXFP4 down feed the FP4 codes straight into the
 * block-scaled matrix instruction, and the Q2_K down its 2-bit codes as FP8
 * operands of the same instruction; IQ2_XXS and the remaining shapes decode on the
 * VALU (dequantize + GEMV). Up to 8 tokens (4 for NVFP4 gate/up; Q2_K down below
 * 1.06 pairs per touched expert) these kernels run over every (token, slot) pair
 * with no routing step; beyond, each routed expert is read once per step for all
 * of its tokens (MXFP4, the NVFP4 gate/up and the Q2_K down on the block-scaled
 * instruction, Q2_K's sub-block scale and min folded into the FP8 operand; IQ2_XXS
 * gate/up and down decoding once per 16-token tile for the bf16 matrix
 * instruction). At prefill with MXFP4 weights it is a token-grouped GEMM
 * on the block-scaled FP4 matrix instructions, with activations quantised to
 * MXFP8 (fp4 weights times E4M3 activations: DeepSeekv4 Flash for 1x Spark forum
 * thread, second post). The decode paths agree with the exact layer to the
 * documented tolerance, the prefill path with the same layer on MXFP8
 * activations; which path runs depends only on formats, shapes, T and
 * alignment, never on the data. INT4 projections (codes as exact operands of the bf16
 * or fp16 matrix instruction, group scales on fp32 sums) run pair by pair while that
 * reads few weights twice, and grouped by expert beyond.
 *
 * Conventions for every entry point:
 *  - Pointers named *_host are host memory; every other buffer pointer is device
 *    memory on the current HIP device, owned and allocated by the caller. The
 *    library never allocates, frees or synchronises on the forward path and keeps
 *    no global state; launches are asynchronous on `stream` (a hipStream_t passed
 *    as void*, NULL = the default stream) and may be captured into a HIP graph.
 *  - Arguments are checked on the host before any launch; a check that fails
 *    returns a negative MOEQ_E_* code and launches nothing. MOEQ_E_HIP reports a
 *    launch error. Faults inside kernels follow HIP semantics (reported at the
 *    next synchronisation). Expert ids outside [0, n_experts) never cause an
 *    out-of-bounds access: the pair is skipped (its outputs are zero) and
 *    MOEQ_DEVERR_EXPERT_ID is set in the workspace's device error word.
 *  - Element order: rows are output features, cols are input features (the
 *    contraction axis); all matrices are row-major.
 */
#ifndef MOEQ_H_
#define MOEQ_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOEQ_ABI_VERSION 2

/* ------------------------------------------------------------------ formats
 * Device layout of one expert tensor [rows, cols] (the `data` and `scales`
 * planes of moeq_weight; experts are expert_stride / scale_expert_stride bytes
 * apart):
 *
 * MOEQ_FMT_MXFP4 - e2m1 elements, one e8m0 scale per 32 along cols (REAP K180
 *   Mixed NVFP4 card, lossless MXFP4 -> NVFP4 conversion section; 4.25 bits per
 *   weight in the 1x Spark forum thread, first post).
 *   data: u8 [rows][cols/2], element 2j in the low nibble of byte j.
 *   scales: u8 [rows][cols/32] e8m0 codes; weight = e2m1 * 2^(E-127), E=255 NaN.
 * MOEQ_FMT_NVFP4 - e2m1 elements, one e4m3 scale per 16, one fp32 scale_2 per
 *   expert tensor (same card, "Why this mix?": 4.50 bits per weight).
 *   data: as MXFP4. scales: u8 [rows][cols/16] e4m3fn codes.
 *   scale2: fp32 [n_experts]. weight = e2m1 * e4m3 * scale_2.
 * MOEQ_FMT_Q2_K - ggml 256-weight superblocks, 84 bytes (2.625 bits per weight;
 *   IQ2_XXS + Q2_K + FP8 hybrid card, format table). Stored as two planes so
 *   every load is aligned; moeq_pack_ggml converts from the contiguous block.
 *   data: u8 [rows][cols/256][64] = the block's qs bytes.
 *   scales: u8 [rows][cols/256][20] = the block's 16 scale bytes, then d and
 *   dmin (fp16, little-endian).
 *   weight i of a superblock: j = i/16, h = i/128, r = i%128,
 *   q = (qs[32h + r%32] >> 2*(r/32)) & 3,
 *   w = d * (sc[j] & 15) * q - dmin * (sc[j] >> 4).
 * MOEQ_FMT_IQ2_XXS - ggml 256-weight superblocks, 66 bytes (2.0625 bits per
 *   weight; same table). Two planes:
 *   data: u8 [rows][cols/256][64] = 8 sub-blocks of (u32 a0, u32 a1).
 *   scales: fp16 d [rows][cols/256].
 *   grid: u8 [256][8] device codebook (an input: any values 0..255).
 *   weight 32b + 8l + j: db = d * (0.5 + (a1 >> 28)) / 4,
 *   g = grid[(a0 >> 8l) & 255][j], c = (a1 >> 7l) & 127,
 *   mask = c | parity(c) << 7, w = (mask >> j & 1 ? -1 : 1) * db * g.
 * MOEQ_FMT_FP8_B128 - E4M3 weights with one UE8M0 scale per 128x128 tile (IQ2_XXS
 *   + Q2_K + FP8 hybrid card, format table; W4A16-FP8 card, FP8 block 128x128).
 *   data: u8 [rows][cols] e4m3fn codes. scales: u8 [rows/128][cols/128].
 *
 * MOEQ_FMT_INT8 - 8-bit integers with one fp32 scale per row (output channel);
 *   moeq_linear_int8, moeq_linear_int8_dynamic, moeq_dequant and the shared expert
 *   of moeq_moe_forward only (elsewhere MOEQ_E_FMT). data: i8 [rows][cols], cols a
 *   multiple of 16; scales: fp32 [rows]; weight = code * scale (codes -128..127).
 *
 * MOEQ_FMT_INT4_G32 / _G64 / _G128 - 4-bit integers with a scale per group of 32, 64 or
 *   128 along cols: weight = scale2 * s * (q - 8), q 0..15. MOEQ_FMT_INT4Z_*: with a zero
 *   point per group, weight = scale2 * s * (q - z), z 0..255. For layers, moeq_linear_int4
 *   and moeq_dequant. Any rows (up to 2^23); cols a multiple of the group (up to 2^20).
 *   Made by moeq_pack_int4 from row-major codes, in the order of the matrix instruction's
 *   operand, in tiles of 16 rows x 128 cols; rows and cols past the end are padding with
 *   scale 0. tile = (r/16) * ceil(cols/128) + c/128.
 *   data: 1024 bytes at tile * 1024; lane n + 16g of the tile holds row n in four words
 *   j = 0..3 at 16 (n + 16g) + 4j: cols 32j + 8g + 0..7 of the tile, col 2p in bits 4p of
 *   the word, col 2p + 1 in bits 16 + 4p.
 *   scales: fp16 [tile][16][128/G]; then, for INT4Z, the zero points u8 [tile][16][128/G].
 *   16-byte aligned, as is scale_expert_stride. scale2: fp32 [n_experts], a power of two.
 *
 * Dense-linear formats (moeq_linear and moeq_dequant only; a layer using one is
 * refused with MOEQ_E_FMT):
 * MOEQ_FMT_FP8_B32 - E4M3 weights with one UE8M0 scale per 32x32 tile, the dense
 *   FP8 weights of DeepSeek-V4.1 (DeepSeek-V4.1-Flash mixed-Q2 GGUF card, Recipe:
 *   V4.1 uses 32x32 E8M0 block scales, V4 128x128; reading one as the other
 *   rescales every weight). data: u8 [rows][cols]; scales: u8 [rows/32][cols/32].
 * MOEQ_FMT_MXFP8 - E4M3 elements with one e8m0 scale per 32 along cols (8.25 bits
 *   per weight), the checkpoint's format for attention, shared experts and the head
 *   (DeepSeekv4 Flash for 1x Spark forum thread, first post).
 *   data: u8 [rows][cols]; scales: u8 [rows][cols/32]; weight = e4m3 * 2^(E-127).
 * MOEQ_FMT_MXFP8_TILED - the same bytes pre-stored in the order of the block-scaled
 *   matrix instruction's operand (same thread, second post: MXFP8 weights stored
 *   in the matrix engine's layout so that nothing is repacked at run time); rows a
 *   multiple of 16, cols of 512. Made from MOEQ_FMT_MXFP8 by moeq_mxfp8_to_tiled.
 *   data: per tile of 16 rows x 128 cols (tile = (r/16) * (cols/128) + c/128),
 *   2048 bytes at tile * 2048; lane L = n + 16g of the tile holds the 32 bytes at
 *   32 L: row n, cols 16g + [0, 16) then 64 + 16g + [0, 16) of the tile.
 *   scales: per group of 16 rows x 512 cols (group = (r/16) * (cols/512) +
 *   c/512), 256 bytes; byte 4 L + j = e8m0 of row n, 32-block 4j + g of the group.
 */
#define MOEQ_FMT_MXFP4 1
#define MOEQ_FMT_NVFP4 2
#define MOEQ_FMT_Q2_K 3
#define MOEQ_FMT_IQ2_XXS 4
#define MOEQ_FMT_FP8_B128 5
#define MOEQ_FMT_MXFP8 6
#define MOEQ_FMT_FP8_B32 7
#define MOEQ_FMT_MXFP8_TILED 8
#define MOEQ_FMT_INT8 9
#define MOEQ_FMT_INT4_G32 10
#define MOEQ_FMT_INT4_G64 11
#define MOEQ_FMT_INT4_G128 12
#define MOEQ_FMT_INT4Z_G32 13
#define MOEQ_FMT_INT4Z_G64 14
#define MOEQ_FMT_INT4Z_G128 15

/* Types of the outputs that come in more than one. */
#define MOEQ_OUT_F32 0
#define MOEQ_OUT_BF16 1

/* ------------------------------------------------------------------ status */
#define MOEQ_OK 0
#define MOEQ_E_INVAL -1     /* null pointer, negative count, bad argument */
#define MOEQ_E_FMT -2       /* unknown format, or a format the entry point does not take */
#define MOEQ_E_ALIGN -3     /* pointer or stride not aligned as documented */
#define MOEQ_E_SHAPE -4     /* shape the format or the kernels cannot hold */
#define MOEQ_E_WORKSPACE -5 /* workspace missing or smaller than moeq_workspace_bytes */
#define MOEQ_E_HIP -6       /* a HIP call or kernel launch failed */
#define MOEQ_E_LOSSY -7     /* MXFP4 -> NVFP4 cannot be exact (span > 17 or NaN scale) */
#define MOEQ_E_SCRATCH -8   /* moeq_expert_forward_noalloc: the call needs more than the scratch holds */

/* Bits of the device error word (first 4 bytes of a workspace). */
#define MOEQ_DEVERR_EXPERT_ID 1u /* an expert id was outside [0, n_experts) */

/* ------------------------------------------------------------------ descriptors
 * Read on the host only, during the call. */
typedef struct moeq_weight {
  int fmt;                    /* MOEQ_FMT_* */
  int rows;                   /* output features */
  int cols;                   /* input features */
  int n_experts;              /* experts stored expert-major */
  const void* data;           /* 16-byte aligned */
  size_t expert_stride;       /* bytes between experts in data, multiple of 16 */
  const void* scales;         /* 4-byte aligned */
  size_t scale_expert_stride; /* bytes between experts in scales, multiple of 4 */
  const float* scale2;        /* NVFP4, INT4: fp32 [n_experts]; else ignored */
  const uint8_t* grid;        /* IQ2_XXS: u8 [256][8]; else ignored */
} moeq_weight;

typedef struct moeq_layer {
  int hidden;    /* H: gate/up cols, down rows */
  int inter;     /* I: gate/up rows, down cols */
  int n_experts; /* E */
  int top_k;     /* K, 1..16 */
  moeq_weight gate, up, down;
} moeq_layer;

/* ------------------------------------------------------------------ sizes */
int moeq_abi_version(void);
const char* moeq_status_string(int status);

/* Bytes of plane 0 (data) or plane 1 (scales) of one expert tensor [rows, cols];
 * 0 for an invalid format, plane or shape. cols must be a multiple of the format's
 * block: 32 MXFP4, 16 NVFP4, 256 Q2_K and IQ2_XXS, 128 FP8_B128 (rows too), 16 INT8, the
 * group of INT4. */
size_t moeq_plane_bytes(int fmt, int rows, int cols, int plane);

/* Total bytes of one expert tensor, both planes plus NVFP4's and INT4's 4-byte scale2. The
 * algorithmic bytes per weight equal the format's bits per weight / 8. */
size_t moeq_packed_bytes(int fmt, int rows, int cols);

/* ------------------------------------------------------------------ host utilities */

/* Repack contiguous ggml blocks (Q2_K: 84 B, IQ2_XXS: 66 B per 256 weights, rows x
 * cols/256 blocks row-major) into the two device planes, in host memory. */
int moeq_pack_ggml(int fmt, const void* blocks_host, int rows, int cols, void* data_host, void* scales_host);

/* Device version over n tensors stored back to back (block bytes, data and scale
 * planes each contiguous per tensor). */
int moeq_pack_ggml_device(int fmt, const void* blocks, int rows, int cols, int n, void* data, void* scales,
                          void* stream);

/* Lossless MXFP4 -> NVFP4 re-encode of one tensor in host memory (REAP K180 Mixed
 * NVFP4 card, conversion section and "How It Was Built" step 3): nibbles copied,
 * e8m0 per 32 -> e4m3 per 16 with scale_2 = 2^(Emax-135), e4m3 = 2^(E-Emax+8).
 * MOEQ_E_LOSSY if Emax - Emin > 17 or a code is 255; outputs are then untouched. */
int moeq_mxfp4_to_nvfp4(const uint8_t* nib_host, const uint8_t* e8m0_host, int rows, int cols, uint8_t* nib_out_host,
                        uint8_t* e4m3_out_host, float* scale2_out_host);

/* Row-major MXFP8 (MOEQ_FMT_MXFP8) -> the pre-stored operand order
 * (MOEQ_FMT_MXFP8_TILED) for n tensors stored back to back in device memory
 * (data planes rows * cols bytes apart, scale planes rows * cols / 32). rows a
 * multiple of 16 and cols of 512 (MOEQ_E_SHAPE otherwise); data and tdata 16-byte
 * aligned, tscales 4-byte aligned; outputs must not overlap inputs. Asynchronous
 * on `stream`. */
int moeq_mxfp8_to_tiled(const void* data, const void* scales, int rows, int cols, int n, void* tdata, void* tscales,
                        void* stream);

/* Device versions of the MXFP4 <-> NVFP4 re-encodes (REAP K180 Mixed NVFP4 card,
 * conversion section and "How It Was Built" step 3; the rule is the host one above),
 * for n tensors [rows][cols] stored back to back in device memory: nibbles rows *
 * cols / 2 bytes apart, e8m0 planes rows * cols / 32, e4m3 planes rows * cols / 16,
 * one scale_2 per tensor. status (device, u32 [n]) receives 0 for a tensor
 * converted exactly and 1 for one that cannot be (MXFP4 -> NVFP4: exponent span
 * above 17 or a NaN scale; NVFP4 -> MXFP4: the two 16-halves of a block differ or
 * their scale times scale_2 is not a power of two 2^k, -127 <= k <= 127), whose
 * outputs are then left untouched. nib_out may equal nib (converted in place);
 * the scale planes must not overlap. Nibble planes 16-byte aligned. Asynchronous on
 * `stream`. */
int moeq_mxfp4_to_nvfp4_device(const uint8_t* nib, const uint8_t* e8m0, int rows, int cols, int n, uint8_t* nib_out,
                               uint8_t* e4m3_out, float* scale2_out, uint32_t* status, void* stream);
int moeq_nvfp4_to_mxfp4_device(const uint8_t* nib, const uint8_t* e4m3, const float* scale2, int rows, int cols, int n,
                               uint8_t* nib_out, uint8_t* e8m0_out, uint32_t* status, void* stream);

/* ------------------------------------------------------------------ kernels */

/* Dequantise expert `expert` of w to fp32 [rows][cols]. The value is the format's
 * exact weight rounded once to fp32 (exact for MXFP4, IQ2_XXS, FP8_B128). */
int moeq_dequant(const moeq_weight* w, int expert, float* out, void* stream);

/* Workspace bytes needed by moeq_expert_forward / the stage entry points for T
 * tokens. The workspace must be zero-filled once before first use (or passed to
 * moeq_workspace_init); its first 4 bytes hold the sticky device error word. */
size_t moeq_workspace_bytes(const moeq_layer* L, int T);
int moeq_workspace_init(void* ws, size_t ws_bytes, void* stream);

/* y[T][H] (fp32, overwritten) of the routed layer for x[T][H] (bf16), expert ids
 * ids[T][K] (int32) and route weights rw[T][K] (fp32, applied after down as given).
 * Decode path (any format: the stage kernels below) below T = 128 tokens. From
 * T = 128, each MXFP4 projection that meets the prefill stages' shape and
 * alignment conditions (below) runs the W4A8 prefill GEMM instead (gate/up on x
 * quantised to MXFP8; down on h quantised to MXFP8), whatever the format of the
 * other projection: a layer mixing IQ2_XXS (or Q2_K) and MXFP4 projections takes
 * the W4A8 GEMM for its MXFP4 projection and the grouped decode kernels for the
 * other (1x Spark forum thread, second post: one grouped GEMM per projection).
 * T == 0 is a no-op. x, y 16-byte aligned. */
int moeq_expert_forward(const moeq_layer* L, const void* x, const int32_t* ids, const float* rw, int T, float* y,
                        void* ws, size_t ws_bytes, void* stream);

/* moeq_expert_forward without a caller workspace, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc). It runs the same kernels on the same path,
 * with their scratch (routing, h, partials, MXFP8 buffers) in a fixed device
 * array inside the library: MOEQ_NOALLOC_SCRATCH_BYTES per GPU, held until the
 * process ends, its address taken once per device on the first call. No call
 * allocates or frees anything. A call whose moeq_workspace_bytes(L, T) exceeds
 * the scratch returns MOEQ_E_SCRATCH before any launch (at hidden 4096,
 * intermediate 2048, 256 experts, top-6: up to T = 227 tokens on the decode path;
 * an all-MXFP4 layer takes the prefill path from T = 128, up to T = 204). Every call on a GPU shares that GPU's scratch: calls
 * that overlap on one GPU (two streams, or two threads) race and must be
 * serialised by the caller; nothing in the scratch has to start at zero.
 * dev_err (device memory, 4-byte aligned, may be NULL) receives the
 * MOEQ_DEVERR_* bits by OR; with NULL they go to a word nobody reads. Other
 * arguments, checks and outputs as moeq_expert_forward. */
#define MOEQ_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
int moeq_expert_forward_noalloc(const moeq_layer* L, const void* x, const int32_t* ids, const float* rw, int T,
                                float* y, uint32_t* dev_err, void* stream);

/* Stages of the decode path, for tests and timing (moeq_expert_forward runs them
 * in order). moeq_route groups the T*K (token, slot) pairs by expert into the
 * workspace (needed before the other two when T > 1). moeq_gate_up writes
 * h[T][K][I] (fp32) = silu(G x) * (U x) per pair. moeq_down writes y[T][H].
 * x, h, y 16-byte aligned. */
int moeq_route(const moeq_layer* L, const int32_t* ids, int T, void* ws, size_t ws_bytes, void* stream);
int moeq_gate_up(const moeq_layer* L, const void* x, const int32_t* ids, int T, float* h, void* ws, size_t ws_bytes,
                 void* stream);
int moeq_down(const moeq_layer* L, const float* h, const int32_t* ids, const float* rw, int T, float* y, void* ws,
              size_t ws_bytes, void* stream);

/* moeq_gate_up with its kernel launched so that start_event / stop_event (two
 * hipEvent_t created with timing, passed as void*) record the kernel's own start
 * and end, for timing that excludes queue gaps (of the product, where a launch before it
 * prepares the tokens). Same arguments and outputs. T == 0 records nothing. */
int moeq_gate_up_timed(const moeq_layer* L, const void* x, const int32_t* ids, int T, float* h, void* ws,
                       size_t ws_bytes, void* stream, void* start_event, void* stop_event);

/* Stages of the W4A8 prefill path, one per projection (its weights MXFP4, else
 * MOEQ_E_FMT; the other projection may be in any format; hidden and inter
 * multiples of 256; the stage's weight scale planes and their expert stride
 * 8-byte aligned, else MOEQ_E_ALIGN; moeq_route first, on the same workspace).
 * moeq_prefill_gate_up: xq/xs = MXFP8 x (codes u8 [T][H], 16-byte aligned; e8m0
 *   u8 [T][H/32], 8-byte aligned) -> hq/hs = MXFP8 h (codes u8 [T*K][I], e8m0 u8
 *   [T*K][I/32]); h_f32 (may be NULL) receives h before quantisation, fp32 [T*K][I].
 * moeq_prefill_down: hq/hs (same alignment as xq/xs) -> y[T][H] (16-byte
 *   aligned); T >= 2.
 * MOEQ_E_FMT for other formats, MOEQ_E_SHAPE for other shapes. */
int moeq_prefill_gate_up(const moeq_layer* L, const uint8_t* xq, const uint8_t* xs, const int32_t* ids, int T,
                         float* h_f32, uint8_t* hq, uint8_t* hs, void* ws, size_t ws_bytes, void* stream);
int moeq_prefill_down(const moeq_layer* L, const uint8_t* hq, const uint8_t* hs, const int32_t* ids, const float* rw,
                      int T, float* y, void* ws, size_t ws_bytes, void* stream);

/* Dense block-quantized linear y[T][rows] = W_expert x[T][cols] (fp32 out). Any
 * format but INT8 (moeq_linear_int8); FP8_B128 is the dense-layer format (IQ2_XXS +
 * Q2_K + FP8 hybrid card).
 * MXFP8, MXFP8_TILED and FP8_B32 run on the block-scaled FP8 matrix instruction
 * for every T (the weights' e8m0 scale is the instruction's scale; x enters as
 * two E4M3 terms per value with e8m0 scales per 32, exact to 2^-21.8 of each
 * 32-block's maximum): rows a multiple of 16 (FP8_B32: 32), cols a multiple of
 * 128 (MXFP8_TILED: 512) and at most 8192, else MOEQ_E_SHAPE.
 * x bf16 [T][cols], 16-byte aligned; y fp32 [T][rows], 4-byte aligned; both
 * caller-owned, y overwritten. FP8_B128 with T >= 2 and cols a multiple of 256
 * runs on the bf16 matrix instruction (E4M3 codes exact in bf16, block scale
 * applied to each 128-wide K tile's fp32 partial); otherwise one GEMV pass per
 * token group, which needs cols / (weights per 16-byte chunk) <= 256 (MOEQ_E_SHAPE
 * beyond). Asynchronous on `stream`. */
int moeq_linear(const moeq_weight* w, int expert, const void* x, int T, float* y, void* stream);

/* MXFP8 quantisation of rows of K values (K a multiple of 32): per 32 consecutive
 * values, e8m0 code E = clamp(e + 127, 0, 254) with 2^e the smallest power of two
 * keeping max|v| / 2^e <= 448 (e = p-9 if the frexp mantissa of max|v| is <= 0.875,
 * else p-8; all-zero block: E = 0, codes 0); codes = E4M3FN round-to-nearest-even of
 * v / 2^(E-127), saturating, sign kept (1x Spark forum thread, second post: E4M3
 * activations with a dynamic scale; the 32-wide block and the non-clipping scale
 * rule are this library's reading). moeq_quantize_mxfp8 takes bf16 input x [T][K]
 * (the prefill activations), moeq_quantize_mxfp8_f32 fp32 (the intermediate h).
 * x and q 16-byte aligned, caller-owned device memory; q u8 [T][K] and e8m0 u8
 * [T][K/32] overwritten. MOEQ_E_SHAPE if K is not a positive multiple of 32. */
int moeq_quantize_mxfp8(const void* x, int T, int K, uint8_t* q, uint8_t* e8m0, void* stream);
int moeq_quantize_mxfp8_f32(const float* x, int T, int K, uint8_t* q, uint8_t* e8m0, void* stream);

/* ------------------------------------------------------------------ 8-bit integers */

/* Codes and scale of every token for the INT8 linears: s = fl32(max |x| / 127), q =
 * round-half-even(fl32(x / s)) clamped to +-127, in fp32 with correctly rounded
 * divisions. A token of zeros gives s = 0 and codes 0; one that holds an infinity or a
 * NaN gives s = NaN and codes 0 (its outputs are NaN). x [T][K] bf16 (fp32 in the _f32
 * form) and q i8 [T][K] 16-byte aligned, scale fp32 [T]; q and scale overwritten.
 * MOEQ_E_SHAPE unless K is a multiple of 16, 16 .. 65536. T == 0 is a no-op. */
int moeq_quantize_int8(const void* x, int T, int K, int8_t* q, float* scale, void* stream);
int moeq_quantize_int8_f32(const float* x, int T, int K, int8_t* q, float* scale, void* stream);

/* y[t][r] = xs[t] * scale[r] * sum_k xq[t][k] W[r][k] (+ bias[r]) for expert `expert`
 * of an MOEQ_FMT_INT8 weight. The sum is exact (int32; cols at most 65536, any codes);
 * the scales and the bias are applied in fp32. xq i8 [T][cols], 16-byte aligned; xs
 * fp32 [T]; bias fp32 [rows] or NULL; y [T][rows] overwritten, fp32 (MOEQ_OUT_F32) or
 * bf16 rounded to nearest even (MOEQ_OUT_BF16), aligned to its element. Any T; rows
 * up to 2^23 (MOEQ_E_SHAPE beyond); T == 0 is a no-op. The same inputs give the same
 * bits whatever the batch they are part of. */
int moeq_linear_int8(const moeq_weight* w, int expert, const int8_t* xq, const float* xs, int T, const float* bias,
                     int out_type, void* y, void* stream);

/* The same product from bf16 tokens x [T][cols] (16-byte aligned), quantised as by
 * moeq_quantize_int8 within the call. ws: at least
 * moeq_linear_int8_workspace_bytes(T, cols) bytes, 256-byte aligned, contents
 * arbitrary, not shared with an overlapping call. For a few tokens (T <= 16, and T
 * rounded up to a power of two times cols <= 65536) it is one launch that stores no
 * codes: ws may then be NULL. */
size_t moeq_linear_int8_workspace_bytes(int T, int cols);
int moeq_linear_int8_dynamic(const moeq_weight* w, int expert, const void* x, int T, const float* bias, int out_type,
                             void* y, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ 4-bit integers */

/* Types of the scales that moeq_pack_int4 takes. */
#define MOEQ_SCALE_F16 0
#define MOEQ_SCALE_BF16 1

/* Row-major INT4 tensors to the planes of MOEQ_FMT_INT4*, for n tensors back to back in
 * device memory: codes u8 [n][rows][cols/2] (the even column in the low half of its byte),
 * scales [n][rows][cols/G] fp16 or bf16 (any sign), zeros u8 [n][rows][cols/G] for the
 * formats with zero points and NULL for the others. data, scales_out (moeq_plane_bytes
 * apart) and scale2 fp32 [n] are overwritten. scale2 is the power of two that brings the
 * tensor's largest finite |scale| into [64, 128); stored scales are exact unless they are
 * below 2^-20 of the largest, where they are rounded to 2^-31 of it. Infinite and NaN
 * scales stay what they are. data and scales_out 16-byte aligned; outputs must not overlap
 * inputs. Asynchronous on `stream`; n == 0 is a no-op. */
int moeq_pack_int4(int fmt, const void* codes, const void* scales, int scale_type, const uint8_t* zeros, int rows, int cols,
                   int n, void* data, void* scales_out, float* scale2, void* stream);

/* y[t][r] = sum_k W[r][k] x[t][k] (+ bias[r]) for expert `expert` of an INT4 weight. Sums of
 * exact products in fp32, scales applied to each group's sum, one rounding to the output type;
 * beyond 16 tokens a value keeps all its bits down to 2^-31 of its token's largest and is rounded
 * by up to 2^-39 of that largest below. The kernel depends on shapes alone; out_type decides
 * nothing but the last rounding.
 * x bf16 [T][cols], 16-byte aligned; bias fp32 [rows] or NULL; y [T][rows] overwritten, fp32
 * or bf16 (MOEQ_OUT_*), aligned to its element. A token that holds an infinity or a NaN
 * gives NaN, and nobody else's outputs change. Partial sums of an output have to stay inside
 * fp32's range; up to 16 tokens also a group's sum of (16 + q) x, which |x| < 2^112 ensures.
 * ws: moeq_linear_int4_workspace_bytes(T, cols) bytes, 256-byte aligned, contents arbitrary, not
 * shared with an overlapping call; NULL for up to 16 tokens. Any T; T == 0 is a no-op. */
size_t moeq_linear_int4_workspace_bytes(int T, int cols);
int moeq_linear_int4(const moeq_weight* w, int expert, const void* x, int T, const float* bias, int out_type, void* y, void* ws,
                     size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ router, whole layer */

/* Scores s of the logits z: softmax over the experts, 1 / (1 + e^-z), or
 * sqrt(log(1 + e^z)). */
#define MOEQ_SCORE_SOFTMAX 0
#define MOEQ_SCORE_SIGMOID 1
#define MOEQ_SCORE_SQRT_SOFTPLUS 2

typedef struct moeq_router {
  int hidden;         /* H, a multiple of 8, at most 65536 */
  int n_experts;      /* E, 1..1024 */
  int top_k;          /* K, 1..16, at most E */
  int scoring;        /* MOEQ_SCORE_* */
  int normalize;      /* != 0: the K chosen scores are divided by their sum */
  float scale;        /* factor of the route weights */
  const void* weight; /* bf16 [E][H], 16-byte aligned */
  const float* bias;  /* fp32 [E], added to the scores for the choice only, or NULL */
} moeq_router;

/* The shared expert beside the routed ones: three MOEQ_FMT_INT8 tensors (expert 0 of
 * each), gate and up [inter][hidden], down [hidden][inter]; inter a multiple of 16. */
typedef struct moeq_shared {
  int inter;
  moeq_weight gate, up, down;
} moeq_shared;

/* The K experts with the largest s + bias of every token, in falling order (ties: the
 * lower id first; a NaN counts below every number; softmax without a bias: in the
 * order of the logits), and their weights s * scale, or
 * s / (sum of the K) * scale. The logits W x are sums of exact products in fp64, and so
 * are scores, sums and denominators at every T: neither the choice nor the weights
 * depend on an order of summation beyond fp64's. x bf16 [T][H], 16-byte aligned; ids
 * int32 [T][K] (always distinct and inside [0, E)) and rw fp32 [T][K] overwritten:
 * what moeq_expert_forward takes. A sum of 0 gives weights 0. ws:
 * moeq_router_workspace_bytes(R, T) bytes, 256-byte aligned, zero-filled once before
 * first use (or passed to moeq_workspace_init), not shared with an overlapping call
 * (calls on one stream do not overlap if no other thread queues launches between
 * theirs). Any T; T == 0 is a no-op. */
size_t moeq_router_workspace_bytes(const moeq_router* R, int T);
int moeq_router_topk(const moeq_router* R, const void* x, int T, int32_t* ids, float* rw, void* ws, size_t ws_bytes,
                     void* stream);

/* The same with the experts in n_groups groups of equal size (experts e of group
 * e / (n_experts / n_groups)), of which every token takes top_groups before it takes its
 * experts inside them. A group's merit is the sum of its two largest s + bias (one, if it
 * has one expert) or its largest, in fp64; ties go to the lower group; a NaN counts as
 * minus infinity. Softmax scores count with their denominators over all experts, so do
 * route weights. n_groups at most 64, a divisor of n_experts; top_k at most the experts of
 * top_groups groups. G == NULL, n_groups == 1 or top_groups == n_groups:
 * moeq_router_topk. Same workspace. */
#define MOEQ_GROUP_TOP2 0
#define MOEQ_GROUP_MAX 1
typedef struct moeq_router_groups {
  int n_groups;
  int top_groups;
  int score; /* MOEQ_GROUP_* */
} moeq_router_groups;
int moeq_router_topk_groups(const moeq_router* R, const moeq_router_groups* G, const void* x, int T, int32_t* ids, float* rw,
                            void* ws, size_t ws_bytes, void* stream);

/* The whole layer for x[T][H] (bf16): y = bf16(routed + shared), with the routed
 * experts of moeq_router_topk as moeq_expert_forward computes them (so from 128 tokens
 * on an MXFP4 projection takes its activations as MXFP8, which moves the routed part by
 * 3 to 5 % of its RMS; fewer tokens and other formats' are not rounded to 8 bits) and
 * the shared expert Ds (silu(Gs x) * (Us x)) on the INT8 linears: x and the intermediate
 * h (fp32) quantised per token as by moeq_quantize_int8, sums in fp32, one rounding to
 * bf16 at the end. S may be NULL (no shared expert). R and L agree on hidden,
 * n_experts and top_k. ids and rw (int32 / fp32 [T][K]) receive the routing, or NULL.
 * ws: moeq_moe_workspace_bytes bytes, 256-byte aligned, zero-filled once before first
 * use (or passed to moeq_workspace_init), not shared with an overlapping call; its
 * first 4 bytes hold the device error word. x, y 16-byte aligned. Any T; made for a
 * few tokens. T == 0 is a no-op. */
size_t moeq_moe_workspace_bytes(const moeq_layer* L, const moeq_router* R, const moeq_shared* S, int T);
int moeq_moe_forward(const moeq_layer* L, const moeq_router* R, const moeq_shared* S, const void* x, int T, void* y,
                     int32_t* ids, float* rw, void* ws, size_t ws_bytes, void* stream);

/* moeq_moe_forward with the router of moeq_router_topk_groups. Same workspace. */
int moeq_moe_forward_groups(const moeq_layer* L, const moeq_router* R, const moeq_router_groups* G, const moeq_shared* S,
                            const void* x, int T, void* y, int32_t* ids, float* rw, void* ws, size_t ws_bytes, void* stream);

/* Synchronise `stream`, then read (and with clear != 0, zero) the device error word. */
int moeq_check_device_error(void* ws, void* stream, uint32_t* err_host, int clear);

#ifdef __cplusplus
}
#endif

#endif /* MOEQ_H_ */
