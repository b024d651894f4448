/*
 * pqmoe.h -- C ABI of the block-scaled quantizer and MoE grouped-GEMM
 * library for AMD Instinct MI355X (gfx950).
 *
 * The library implements the data-parallel core of the low-precision RL
 * precision contract described in:
 *   [BW] "Towards Blackwell-Native 8-bit and 4-bit RL"
 *   [MT] "miniTE technical report: stable training and efficient
 *        implementation of native NVFP4 RL"
 *   [PR] "PR #2396 report: docs: refresh MXFP8 and NVFP4 RL guide"
 *
 * Conventions for every entry point
 * ---------------------------------
 *  - Pointers named d_* or documented as "device" are device pointers (HBM);
 *    the caller owns every buffer.  The library never allocates, frees or
 *    synchronizes; all work is enqueued on `stream` (NULL = the null stream)
 *    and returns before it runs.
 *  - bf16 tensors are passed as 16-bit bit patterns (uint16_t).  Inputs must
 *    be finite; NaN and infinity are outside the contract.
 *  - Shapes are row-major.  `ld` is the row stride of an input in elements.
 *  - Argument errors are reported synchronously, before anything is
 *    enqueued: PQM_ERR_NULL (a required pointer is NULL), PQM_ERR_SHAPE
 *    (a size is negative or not a multiple of the block length),
 *    PQM_ERR_ALIGN (a vector-loaded pointer or stride is not 16-byte
 *    aligned), PQM_ERR_ENUM (unknown format/kind/dtype), PQM_ERR_WORKSPACE
 *    (workspace too small).  A failed launch returns PQM_ERR_HIP.
 *  - Results are deterministic: the same inputs give bitwise identical
 *    outputs on every run (fixed reduction order, no split-K atomics),
 *    following the deterministic-mode rule of [MT] 4.5.
 *  - Zero-sized inputs (rows == 0, or an empty group) are legal and enqueue
 *    nothing for the empty part.
 */
#ifndef PQMOE_H
#define PQMOE_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pqm_status {
    PQM_OK = 0,
    PQM_ERR_NULL = 1,
    PQM_ERR_SHAPE = 2,
    PQM_ERR_ALIGN = 3,
    PQM_ERR_ENUM = 4,
    PQM_ERR_WORKSPACE = 5,
    PQM_ERR_HIP = 6
} pqm_status;

typedef enum pqm_format {
    PQM_FMT_BF16 = 0,  /* plain bf16 operands */
    PQM_FMT_MXFP8 = 1, /* E4M3 data, one E8M0 scale per 32 along the row */
    PQM_FMT_NVFP4 = 2, /* packed E2M1, one E4M3 scale per 16, FP32 outer */
    PQM_FMT_FP8_BLOCK = 3 /* E4M3, FP32 scale per 1x128 tile / 128x128 block */
} pqm_format;

typedef enum pqm_gemm_kind {
    PQM_GEMM_FPROP = 0, /* Y[m,:] = A[m,:] . B_g^T,  B [G, N, K]          */
    PQM_GEMM_DGRAD = 1, /* Y[m,:] = A[m,:] . B_g,    B [G, K, N] (bf16)   */
    PQM_GEMM_WGRAD = 2  /* Y_g = A_g^T . B_g over the group's rows (bf16) */
} pqm_gemm_kind;

typedef enum pqm_dtype {
    PQM_OUT_BF16 = 0,
    PQM_OUT_FP32 = 1
} pqm_dtype;

/* Human-readable name of a status code (static string, never NULL). */
const char *pqm_status_string(pqm_status s);

/* Version of the ABI described by this header. */
int pqm_abi_version(void);

/*
 * MXFP8 quantization ([BW] Format background: MXFP8; Recipe 1: training).
 *
 * Each 1x32 block of E4M3 values shares one E8M0 (power of two) scale,
 * rounded up so the block maximum is never clipped: the scale is 2^e with
 * e the smallest integer for which max|x| <= 448 * 2^e (e >= -127; an
 * all-zero block gets e = -127).  Elements are x / 2^e rounded to the
 * nearest E4M3 value, ties to even; a negative input that rounds to zero
 * keeps its sign (0x80).
 *
 * Row-wise and column-wise copies are both quantized independently from
 * the bf16 input in the same pass (never one from the other):
 *   x       [rows, cols] bf16, row stride ld elements           (device)
 *   q_row   [rows, cols]       E4M3 bytes, 1x32 blocks along rows  (device)
 *   s_row   [rows, cols/32]    E8M0 bytes                          (device)
 *   q_colT  [cols, rows]       E4M3 bytes of the 32x1 blocks down each
 *                              column, stored transposed so each block is
 *                              contiguous                          (device)
 *   s_colT  [cols, rows/32]    E8M0 bytes                          (device)
 * Either output pair may be NULL to skip that copy, not both.
 * Requires cols % 32 == 0; rows % 32 == 0 when the column copy is asked
 * for; fewer than 2^31 tiles of 128 x 128 (PQM_ERR_SHAPE otherwise); x,
 * q_row, q_colT and ld 16-byte aligned (ld % 8 == 0); s_row and s_colT
 * 4-byte aligned (PQM_ERR_ALIGN otherwise).
 */
pqm_status pqm_quantize_mxfp8(const uint16_t *x, int64_t rows, int64_t cols,
                              int64_t ld, uint8_t *q_row, uint8_t *s_row,
                              uint8_t *q_colT, uint8_t *s_colT,
                              hipStream_t stream);

/*
 * NVFP4 quantization with an online FP32 outer scale ([BW] Format
 * background: NVFP4; Recipe 2: per-token activation scaling, gate/up
 * pairing; [MT] 2.2 decode x^ = q s_b s_g; [MT] 5.6 gs = gamax / 2688).
 *
 * Rows are split into scope groups of `rows_per_scale` consecutive rows;
 * each group has one FP32 outer scale s_g:
 *   rows_per_scale = 1    per token (the activation recipe): one fused pass
 *                         reads each row once and writes all three outputs;
 *   rows_per_scale = R_e  one scale per expert tensor; for fused gate/up
 *                         weights [gate; up] of R_e rows this is the joint
 *                         option: gate and up share one outer scale.
 * For a group with absolute maximum A:
 *   s_g   = A / 2688 rounded once to binary32 (2688 = 6 * 448);
 *   s_b   = nearest E4M3 to a_b / (6 s_g) for each 1x16 block with block
 *           maximum a_b, ties to even, saturating at 448 (0 if s_g == 0);
 *   q     = nearest E2M1 to x / (s_b s_g), ties to even, saturating at 6
 *           (+-0 if s_b == 0); all quotients are exact, not approximated.
 * Outputs (device):
 *   q        [rows, cols/2]  packed E2M1, element 2j in the low nibble
 *   s_block  [rows, cols/16] E4M3 bytes
 *   s_outer  [rows / rows_per_scale] binary32 decode scales s_g
 * Requires cols % 16 == 0, cols <= 16384, rows < 2^31, rows % rows_per_scale
 * == 0, x and ld 16-byte aligned, q 8-byte aligned, s_outer 4-byte aligned
 * (PQM_ERR_SHAPE / PQM_ERR_ALIGN otherwise).  When rows_per_scale > 1 the group maximum is reduced across
 * workgroups through `workspace` (device, >= pqm_quantize_nvfp4_workspace
 * bytes, 4-byte aligned; contents on entry are ignored); it may be NULL
 * when rows_per_scale == 1.
 */
pqm_status pqm_quantize_nvfp4_per_token(const uint16_t *x, int64_t rows,
                                        int64_t cols, int64_t ld,
                                        int64_t rows_per_scale, uint8_t *q,
                                        uint8_t *s_block, float *s_outer,
                                        void *workspace,
                                        size_t workspace_bytes,
                                        hipStream_t stream);

/* Workspace bytes pqm_quantize_nvfp4_per_token needs for these sizes. */
size_t pqm_quantize_nvfp4_workspace(int64_t rows, int64_t cols,
                                    int64_t rows_per_scale);

/*
 * Block-scaled FP8 in the DeepSeek-V3 style ([BW] Why Blackwell-native
 * recipes: 128x128 weight blocks and 1x128 activation tiles, an FP32 scale
 * per block computed online and applied around the matrix core; [PR] Choose
 * a precision: FP8 block-wise, 128x128, FP32 scales).
 *
 * Blocks of block_rows x 128 (block_rows = 1: activation tiles; 128: weight
 * blocks).  For a block with absolute maximum A:
 *   s = A / 448 rounded once to binary32;
 *   q = nearest E4M3 to the exact quotient x / s, ties to even, saturating
 *       at 448 (the block maximum encodes to +-448); A = 0 gives s = 0 and
 *       q = +-0 (a negative input keeps its sign: 0x80).
 *   x [rows, cols] bf16, row stride ld elements                  (device)
 *   q [rows, cols] E4M3 bytes                                    (device)
 *   s [rows / block_rows, cols / 128] binary32                   (device)
 * Requires block_rows 1 or 128, cols % 128 == 0, rows % block_rows == 0,
 * fewer than 2^31 workgroups (PQM_ERR_SHAPE); x and ld 16-byte aligned,
 * q 8-byte and s 4-byte aligned (PQM_ERR_ALIGN).
 */
pqm_status pqm_quantize_fp8_block(const uint16_t *x, int64_t rows, int64_t cols, int64_t ld,
                                  int64_t block_rows, uint8_t *q, float *s,
                                  hipStream_t stream);

/*
 * Dequantize to bf16 for the dequantized-backward mode ([BW]
 * High-precision and dequantized backward: the backward GEMMs run in BF16
 * on the BF16 dequantization of the exact forward operands).
 *
 * y = the exact decoded value rounded once to the nearest bf16 (ties to
 * even; values beyond bf16 range become +-inf):
 *   PQM_FMT_MXFP8: q [rows, cols] E4M3, s_block [rows, cols/32] E8M0,
 *                  s_outer unused (may be NULL);  y = q * 2^(s - 127)
 *   PQM_FMT_NVFP4: q [rows, cols/2] packed E2M1, s_block [rows, cols/16]
 *                  E4M3, s_outer [rows / rows_per_scale] binary32;
 *                  y = q * s_b * s_g
 * y [rows, cols] bf16 (device).  The orientation of y is that of q: a
 * column-wise (transposed) MXFP8 copy dequantizes to the transpose.
 * Requires cols % 32 == 0 (MXFP8) or cols % 16 == 0 (NVFP4).
 */
pqm_status pqm_dequantize(pqm_format fmt, const uint8_t *q,
                          const uint8_t *s_block, const float *s_outer,
                          int64_t rows, int64_t cols, int64_t rows_per_scale,
                          uint16_t *y, hipStream_t stream);

/*
 * Grouped GEMM over routed experts ([MT] 5.2: one contiguous buffer with
 * expert offsets handed to a dense grouped GEMM, metadata on the device,
 * empty experts handled inside; [MT] 5.4: ACC = block-scaled GEMM(A, B),
 * ACC *= alpha_a[m] (* alpha_b)).
 *
 * offsets [G+1] int64 (device): group g owns rows offsets[g] ..
 * offsets[g+1]-1 of A; offsets[0] = 0, non-decreasing, offsets[G] <=
 * M_total (rows from offsets[G] on are neither read nor written).  Empty
 * groups are legal.  Values outside this contract are undefined behaviour.
 *
 *   PQM_GEMM_FPROP (all formats):   Y[m, n] = sum_k A[m, k] B_g[n, k]
 *       A [M_total, K] and B [G, N, K], both with K contiguous;
 *       Y [M_total, N].
 *   PQM_GEMM_DGRAD (PQM_FMT_BF16):  Y[m, n] = sum_k A[m, k] B_g[k, n]
 *       A [M_total, K], B [G, K, N] (N contiguous); Y [M_total, N].
 *   PQM_GEMM_WGRAD (PQM_FMT_BF16):  Y_g[n, k] = sum_{m in g} A[m, n] B[m, k]
 *       A [M_total, N], B [M_total, K]; Y [G, N, K] (zero for empty g).
 *   PQM_GEMM_DGRAD (PQM_FMT_MXFP8): the same Y, with the contraction
 *       blocks of B_g running along k ([BW] MXFP8 training: backward GEMMs
 *       read the column-wise copies): a = row-wise MXFP8 of A [M_total, K];
 *       b / b_scale = the column-wise copy (q_colT [N, G*K], s_colT
 *       [N, G*K/32]) that pqm_quantize_mxfp8 makes of the stacked B [G*K, N];
 *       expert g uses its columns g*K .. g*K+K-1.  K % 128 == 0, K <= 2048,
 *       G*K*256 + K < 2^32.
 *   PQM_GEMM_WGRAD (PQM_FMT_MXFP8): the same Y_g from the column-wise
 *       copies of both operands: a / a_scale = q_colT [N, M_total] /
 *       s_colT [N, M_total/32] of A, b / b_scale = q_colT [K, M_total] /
 *       s_colT [K, M_total/32] of B.  Every offsets[g] must be a multiple
 *       of 32 (each expert's rows padded to whole 32-row blocks, padding
 *       rows zero), else the result is undefined (reads stay in bounds).
 *       M_total % 32 == 0, M_total*256 + 4096 < 2^32; any N, K.
 *
 * Operand encodings (all device):
 *   PQM_FMT_BF16:  a, b bf16; scales and outer scales unused (NULL).
 *   PQM_FMT_MXFP8: a = E4M3 [M_total, K], a_scale = E8M0 [M_total, K/32];
 *                  b = E4M3 [G, N, K], b_scale = E8M0 [G, N, K/32].
 *   PQM_FMT_NVFP4: a = packed E2M1 [M_total, K/2], a_scale = E4M3
 *                  [M_total, K/16], a_outer = binary32 [M_total] (per
 *                  token); b = packed E2M1 [G, N, K/2], b_scale = E4M3
 *                  [G, N, K/16], b_outer = binary32 [(G*N) /
 *                  b_rows_per_scale] (b_rows_per_scale = N: one scale per
 *                  expert, e.g. joint gate/up).
 *   PQM_FMT_FP8_BLOCK (FPROP only; [BW] Why Blackwell-native recipes: the
 *                  DeepSeek-V3 design, FP32 scales applied around the
 *                  matrix core): a = E4M3 [M_total, K] with a_outer =
 *                  binary32 [M_total, K/128] (1x128 tiles); b = E4M3
 *                  [G, N, K] with b_outer = binary32 [G*N/128, K/128]
 *                  (128x128 blocks), as pqm_quantize_fp8_block makes them;
 *                  a_scale, b_scale unused.  Y[m, n] = sum over 128-K
 *                  blocks kb of a_outer[m, kb] b_outer[n/128, kb] times the
 *                  block's sum of E4M3 products.  K % 128 == 0, K <= 8192,
 *                  N % 128 == 0.
 * a, b and out 16-byte aligned, offsets 8-byte aligned, MXFP8 scale arrays
 * and block-FP8 scales 4-byte aligned (PQM_ERR_ALIGN otherwise).
 * The products use the exact operand values; accumulation is binary32 and
 * the outer scales are applied to the binary32 accumulator.
 * out: Y in bf16 (rounded once) or binary32 per out_dtype.
 * K % 32 == 0 (MXFP8 FPROP / DGRAD), K % 16 == 0 (NVFP4), K % 8 and
 * N % 8 == 0 (BF16); BF16 WGRAD needs N % 8 == 0 and K % 8 == 0; NVFP4 and
 * block FP8 are FPROP only (PQM_ERR_ENUM otherwise).
 * workspace (device, optional): pqm_moe_grouped_gemm_workspace_size(fmt,
 * kind) bytes, 4-byte aligned, contents irrelevant; the call overwrites
 * them, so calls that may run at the same time need separate workspaces.
 * Only the MXFP8 weight gradient uses one today (a tile counter: with it the
 * tiles, heaviest experts first, go to whichever workgroup is free; without
 * it they are dealt in a fixed order, same results either way).  NULL / 0,
 * or a buffer that is too small or misaligned, means no workspace.
 * bias (device, optional; FPROP only, else PQM_ERR_ENUM; 4-byte aligned):
 * binary32 [G, N], the forward epilogue's additive term ([MT] 5.4: the
 * accumulator times the outer scales, plus bias): Y_g[m, n] = alpha
 * x accumulator + bias[g, n] in binary32 (NVFP4: the product and the sum
 * in binary64, rounded once to binary32), then the output rounding.  NULL:
 * no bias.
 * An empty contraction (K == 0) makes FPROP / DGRAD write zeros (with a
 * bias: each routed row's bias row) to rows 0 .. offsets[G]-1 and read no
 * operand; operand, scale and outer-scale pointers are required (non-NULL)
 * only when M_total, N and K are all positive, and out only when Y has
 * elements.
 */
pqm_status pqm_moe_grouped_gemm(pqm_format fmt, pqm_gemm_kind kind,
                                const void *a, const uint8_t *a_scale,
                                const float *a_outer, const void *b,
                                const uint8_t *b_scale, const float *b_outer,
                                int64_t b_rows_per_scale, const float *bias,
                                const int64_t *offsets, int64_t G,
                                int64_t M_total, int64_t N, int64_t K,
                                void *out, pqm_dtype out_dtype,
                                void *workspace, size_t workspace_bytes,
                                hipStream_t stream);

/* Workspace bytes pqm_moe_grouped_gemm can use for (fmt, kind): 4 for the
 * MXFP8 weight gradient, 0 otherwise (host only, no device work). */
size_t pqm_moe_grouped_gemm_workspace_size(pqm_format fmt, pqm_gemm_kind kind);

/*
 * The NVFP4 down projection with online amax compensation ([MT] 5.6, the
 * single-pass fusion study): the activation P is consumed in 128-wide K-tiles
 * before each row's full maximum is known.  Per row, a running maximum
 * gamax = max(|P| over the tiles so far); tile i is encoded under
 * gs = binary32(gamax / 2688) exactly as pqm_quantize_nvfp4_per_token
 * encodes a row of maximum gamax (1x16 E4M3 block scales, E2M1 codes), its
 * block-scaled product with W2 (without gs) is dO_i, and the accumulator
 * moves to the new scale: O = O (gs_prev / gs) + dO_i, gs_prev = gs.  While
 * gamax is zero the tile adds nothing and gs_prev stays.  Y = O gs_prev
 * alpha_W2(n); an all-zero row gives zero.  The encodings depend on when the
 * row's maximum arrives, so Y can differ from the two-pass path (whole-row
 * per-token encoding, then pqm_moe_grouped_gemm NVFP4) by the quantization
 * difference, while the compensation itself is exact up to rounding.
 *   p        bf16 [M_total, K], routed rows grouped by offsets;
 *   w_q      packed E2M1 [G, N, K/2], w_scale E4M3 [G, N, K/16] (4-byte
 *            aligned), w_outer binary32 [(G*N) / w_rows_per_scale];
 *   out      [M_total, N] bf16 (rounded once) or binary32 per out_dtype;
 *            rows 0 .. offsets[G]-1 written;
 *   gs_out   (optional, binary32 [M_total]) each row's final gs;
 *   q_out, sb_out (optional, both or neither; [M_total, K/2] and
 *            [M_total, K/16]) the codes and block scales P was encoded
 *            with, tile by tile.
 * Accumulation is binary32; gs_prev / gs is one binary32 division.
 * K must be a positive multiple of 256 and w_rows_per_scale >= 1 dividing
 * G*N (PQM_ERR_SHAPE); p, w_q, out, q_out 16-byte aligned, offsets 8-byte,
 * w_scale and gs_out 4-byte (PQM_ERR_ALIGN).  The caller owns every buffer;
 * nothing is allocated.
 */
pqm_status pqm_moe_fc2_online_nvfp4(const uint16_t *p, const uint8_t *w_q,
                                    const uint8_t *w_scale, const float *w_outer,
                                    int64_t w_rows_per_scale, const int64_t *offsets,
                                    int64_t G, int64_t M_total, int64_t N, int64_t K,
                                    void *out, pqm_dtype out_dtype, float *gs_out,
                                    uint8_t *q_out, uint8_t *sb_out, hipStream_t stream);

/*
 * The same online-amax FC2 ([MT] 5.6) split into two kernels.  A row's encoding
 * depends on its K-tiles only, not on the output column, so the first kernel
 * encodes every routed row once.  The second is the NVFP4 grouped GEMM
 * on those codes, which moves its accumulator rows by the stored ratios
 * before each K-tile.  The codes, block scales and gs are those of
 * pqm_moe_fc2_online_nvfp4, and so is Y bit for bit: the same accumulation
 * order and the same epilogue.  The one-kernel entry point encodes P again
 * in every 256-column tile.
 *   p, w_q, w_scale, w_outer, offsets, out, out_dtype: as
 *            pqm_moe_fc2_online_nvfp4;
 *   gs_out   binary32 [M_total], each row's final gs (written);
 *   q_out, sb_out [M_total, K/2] and [M_total, K/16], the codes and block
 *            scales P was encoded with (written, then read by the GEMM);
 *   ratio_out binary32 [M_total, K/128], each tile's gs_prev / gs (1 when
 *            the row's maximum did not grow; written, then read).
 * Rows 0 .. offsets[G]-1 of every output are written.  All four buffers
 * are required (PQM_ERR_NULL).  K is a positive multiple of 256 and at most
 * 4096 (PQM_ERR_SHAPE).  p, w_q, out and q_out must be 16-byte aligned,
 * offsets 8-byte, and w_scale, sb_out, gs_out and ratio_out 4-byte
 * (PQM_ERR_ALIGN).  The caller owns every buffer; nothing is allocated.
 */
pqm_status pqm_moe_fc2_online_nvfp4_split(const uint16_t *p, const uint8_t *w_q,
                                          const uint8_t *w_scale, const float *w_outer,
                                          int64_t w_rows_per_scale, const int64_t *offsets,
                                          int64_t G, int64_t M_total, int64_t N, int64_t K,
                                          void *out, pqm_dtype out_dtype, float *gs_out,
                                          uint8_t *q_out, uint8_t *sb_out, float *ratio_out,
                                          hipStream_t stream);

/*
 * The MXFP8 gate_up grouped GEMM with its activation fused into the
 * epilogue ([MT] 5.3-5.4: D = act(gate, up) x prob is produced where C is,
 * and quantized for the down GEMM without another pass; C is not written):
 *   C_g = A . B_g^T as pqm_moe_grouped_gemm FPROP (MXFP8, bf16 output),
 *   D   = pqm_swiglu_prob(C, prob, src),  (q, s) = row-wise MXFP8 of D,
 * with the same bytes as those three calls.  A [M_total, K] E4M3 + a_scale
 * [M_total, K/32]; B [G, 2 inter, K] E4M3 (rows 0..inter-1 gate, then up)
 * + b_scale [G, 2 inter, K/32]; prob / src as pqm_swiglu_prob; q [M_total,
 * inter] E4M3 and s [M_total, inter/32] E8M0 (device).
 * Requires inter % 128 == 0, K % 128 == 0, K <= 2048 (PQM_ERR_SHAPE); a, b,
 * q 16-byte aligned, the scale arrays 4-byte aligned (PQM_ERR_ALIGN).
 */
pqm_status pqm_moe_gemm_swiglu_quantize_mxfp8(const uint8_t *a, const uint8_t *a_scale,
                                              const uint8_t *b, const uint8_t *b_scale,
                                              const int64_t *offsets, int64_t G,
                                              int64_t M_total, int64_t inter, int64_t K,
                                              const float *prob, const int32_t *src,
                                              uint8_t *q, uint8_t *s, hipStream_t stream);

/*
 * MoE glue around the grouped GEMM ([MT] 5.2: quantized rows are placed in
 * one contiguous buffer with offsets marking the expert boundaries, built
 * on the device; [MT] 5.4: D = act(gate, up) x prob; [BW] Fine-grained
 * precision control: routed outputs go through a high-precision weighted
 * reduction).
 */

/*
 * Stable counting sort of token -> expert assignments.
 *   topk_ids  [tokens, k] int32 expert ids in [0, num_experts)   (device)
 *   shared_expert  0, or 1 to append one more group (index num_experts)
 *             holding every token in order, for an always-active shared
 *             expert run through the same grouped GEMM
 *   offsets   [num_experts + 1 + shared_expert] int64: group e owns
 *             positions offsets[e] .. offsets[e+1]-1              (device)
 *   src_row   [tokens * (k + shared_expert)] int32: the assignment index
 *             t*k + j stored at each position (tokens*k + t for the shared
 *             expert's row of token t); within an expert, flat order is
 *             kept                                               (device)
 *   token     [same] int32: the token of each position           (device)
 *   slot      [tokens, k] int32: position of assignment (t, j)   (device)
 *   workspace >= pqm_moe_route_workspace(...) bytes (0 when tokens == 0;
 *             may then be NULL), 8-byte aligned.
 * num_experts <= 4096, tokens * (k + 1) < 2^31.  Ids outside
 * [0, num_experts) are undefined behaviour.
 */
size_t pqm_moe_route_workspace(int64_t tokens, int64_t k, int64_t num_experts);
pqm_status pqm_moe_route(const int32_t *topk_ids, int64_t tokens, int64_t k,
                         int64_t num_experts, int shared_expert, int64_t *offsets,
                         int32_t *src_row, int32_t *token, int32_t *slot,
                         void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * pqm_moe_route without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation): the same kernels and the same outputs
 * as pqm_moe_route, with the (chunk, expert) counts and expert totals kept
 * in a scratch array of PQM_ROUTE_NOALLOC_SCRATCH_BYTES that the library
 * holds on each GPU it runs on until the process ends.  The call allocates
 * and frees nothing.  Requires pqm_moe_route_workspace(tokens, k,
 * num_experts) <= PQM_ROUTE_NOALLOC_SCRATCH_BYTES, i.e. about
 * ceil(tokens k / 256) num_experts 4 + num_experts 8 bytes (PQM_ERR_WORKSPACE
 * otherwise; 65536 tokens x top-8 over 256 experts need 2 MiB, 4096 tokens x
 * top-8 over 256 experts 130 KiB); other arguments and errors as
 * pqm_moe_route; PQM_ERR_HIP if the scratch address cannot be obtained.
 * All calls on one GPU share its scratch array: calls that overlap in time
 * on one GPU (different streams, or host threads) race and must be
 * serialized by the caller; calls in stream order are safe.
 */
#define PQM_ROUTE_NOALLOC_SCRATCH_BYTES ((size_t)4 << 20)
pqm_status pqm_moe_route_noalloc(const int32_t *topk_ids, int64_t tokens, int64_t k,
                                 int64_t num_experts, int shared_expert, int64_t *offsets,
                                 int32_t *src_row, int32_t *token, int32_t *slot,
                                 hipStream_t stream);

/*
 * Row gather: out row i = src row (index[i] / divisor), rows of row_bytes
 * bytes (quantized data, scale bytes or FP32 token scales).  With
 * index = token from pqm_moe_route (divisor 1) this places each token's
 * already-quantized row at its expert-sorted positions: per-row blocks run
 * along K, so gathering quantized rows gives the same bytes as quantizing
 * gathered rows.  index entries must be < src_rows * divisor.
 */
pqm_status pqm_moe_gather_rows(const void *src, int64_t src_rows, int64_t row_bytes,
                               const int32_t *index, int64_t n, int64_t divisor,
                               void *out, hipStream_t stream);

/*
 * Per-expert padding to whole blocks of `align` rows ([MT] 5.3: the
 * permuted FC1 activation is padded before it is quantized; [BW] MXFP8
 * training: the column-wise copies have 32 x 1 blocks down each column, so
 * with align = 32 no block holds two experts' tokens):
 *   padded_offsets[0] = 0, padded_offsets[g+1] = padded_offsets[g] +
 *       ceil(n_g / align) * align,  n_g = offsets[g+1] - offsets[g];
 *   out row padded_offsets[g] + j = src row offsets[g] + j for j < n_g;
 *   every other row of out (the padding, and rows from padded_offsets[G]
 *   to out_rows) is zero.
 *   src [src_rows, row_bytes], out [out_rows, row_bytes]        (device)
 *   offsets, padded_offsets [G+1] int64                         (device)
 * Requires align >= 1, row_bytes % 16 == 0, out_rows >= src_rows + G *
 * (align - 1) (room for any offsets; PQM_ERR_SHAPE otherwise); src and out
 * 16-byte aligned, the offset arrays 8-byte aligned (PQM_ERR_ALIGN).
 * offsets must satisfy the pqm_moe_grouped_gemm contract with offsets[G]
 * <= src_rows.
 */
pqm_status pqm_moe_pad_rows(const void *src, int64_t src_rows, int64_t row_bytes,
                            const int64_t *offsets, int64_t G, int64_t align,
                            int64_t *padded_offsets, void *out, int64_t out_rows,
                            hipStream_t stream);

/*
 * Weighted SwiGLU: d[m, j] = bf16( silu(g) * u * p ) with g = c[m, j],
 * u = c[m, inter + j] (c = [gate | up], bf16 [rows, 2*inter]),
 * silu(z) = z / (1 + exp(-z)), p = prob[src[m]] (prob binary32 indexed by
 * assignment, i.e. src_row from pqm_moe_route; with a shared expert prob
 * holds tokens*k + tokens entries, the last tokens of them 1.0; src may be
 * NULL to index prob by m).  Binary32 math with the hardware exponential
 * and reciprocal (about 1 ulp each before the bf16 rounding); for g <= -64
 * the value is formed as (g u p) e^g with power-of-two range scaling, so
 * that neither e^-g nor e^g leaves the binary32 normal range.
 * d bf16 [rows, inter]; inter % 8 == 0.
 */
pqm_status pqm_swiglu_prob(const uint16_t *c, const float *prob, const int32_t *src,
                           int64_t rows, int64_t inter, uint16_t *d, hipStream_t stream);

/*
 * The weighted SwiGLU above fused with the row-wise MXFP8 quantization of
 * its output, the FC2 operand ([MT] 5.3-5.4: the activation of the FC1
 * output, times the router probability, is quantized for the down GEMM
 * without a separate pass over D; [BW] Format background: MXFP8).
 *   q [rows, inter] E4M3 and s [rows, inter / 32] E8M0 equal
 *   pqm_quantize_mxfp8 (row-wise) of the d that pqm_swiglu_prob returns;
 *   d (bf16 [rows, inter]) is also written when non-NULL.
 * Requires inter % 32 == 0 (PQM_ERR_SHAPE), c and d 16-byte aligned, q
 * 8-byte aligned (PQM_ERR_ALIGN); c, prob, q, s non-NULL (PQM_ERR_NULL).
 */
pqm_status pqm_swiglu_prob_quantize_mxfp8(const uint16_t *c, const float *prob,
                                          const int32_t *src, int64_t rows, int64_t inter,
                                          uint16_t *d, uint8_t *q, uint8_t *s,
                                          hipStream_t stream);

/*
 * The weighted SwiGLU above fused with the per-token NVFP4 quantization of
 * its output, the FC2 operand of the NVFP4 recipe ([MT] 5.3-5.4: the
 * activation times the router probability is quantized where it is
 * produced, the per-token amax taken in the same pass, so D is neither
 * written nor read back; [BW] Recipe 2: per-token activation scaling):
 *   q [rows, inter / 2] packed E2M1, s_block [rows, inter / 16] E4M3 and
 *   s_outer [rows] binary32 equal pqm_quantize_nvfp4_per_token (one scale
 *   per row) of the d that pqm_swiglu_prob returns; d (bf16 [rows, inter])
 *   is also written when non-NULL.
 * Requires inter % 16 == 0, inter <= 16384, rows < 2^31 (PQM_ERR_SHAPE);
 * c and d 16-byte aligned, q 8-byte and s_outer 4-byte aligned
 * (PQM_ERR_ALIGN); c, prob, q, s_block, s_outer non-NULL (PQM_ERR_NULL).
 */
pqm_status pqm_swiglu_prob_quantize_nvfp4(const uint16_t *c, const float *prob,
                                          const int32_t *src, int64_t rows, int64_t inter,
                                          uint16_t *d, uint8_t *q, uint8_t *s_block,
                                          float *s_outer, hipStream_t stream);

/*
 * Opt-in check of an offsets array against the grouped-GEMM contract ([MT]
 * 5.2: experts' rows in one contiguous buffer described by offsets on the
 * device); the GEMMs and the glue never check it themselves, since a bad
 * array is undefined behaviour there.  Scans i = 0 .. G and writes, on the
 * stream, to result (device, 2 x int32): result[0] = the first failing check
 * at the smallest failing index (0: the array is valid), result[1] = that
 * index (-1 when valid).  Checks at index i, in this order:
 *   PQM_OFFSETS_FIRST_NOT_ZERO  i == 0 and offsets[0] != 0
 *   PQM_OFFSETS_DECREASING      i < G and offsets[i + 1] < offsets[i]
 *   PQM_OFFSETS_MISALIGNED      offsets[i] % align != 0 (align = 32 for the
 *                               MXFP8 weight gradient's padded groups, else 1)
 *   PQM_OFFSETS_PAST_END        i == G and offsets[G] > M_total
 * G >= 0, M_total >= 0, align >= 1 (PQM_ERR_SHAPE); offsets 8-byte and result
 * 4-byte aligned (PQM_ERR_ALIGN), both non-NULL (PQM_ERR_NULL).  Reads
 * offsets[0 .. G]; one workgroup.
 */
#define PQM_OFFSETS_FIRST_NOT_ZERO 1
#define PQM_OFFSETS_DECREASING 2
#define PQM_OFFSETS_MISALIGNED 3
#define PQM_OFFSETS_PAST_END 4
pqm_status pqm_validate_offsets(const int64_t *offsets, int64_t G, int64_t M_total,
                                int64_t align, int32_t *result, hipStream_t stream);

/*
 * Combine: out[t, n] = bf16( sum_j y_rows[slot[t, j], n] + shared[t, n] ),
 * summed in binary32 in j order (shared may be NULL).  y_rows, shared, out
 * bf16 with N contiguous; N % 8 == 0.
 */
pqm_status pqm_moe_combine(const uint16_t *y_rows, const int32_t *slot,
                           const uint16_t *shared, int64_t tokens, int64_t k, int64_t N,
                           uint16_t *out, hipStream_t stream);

/*
 * RMS norm with the residual's addition, and the row-wise MXFP8 encoding of
 * its output: the activation in front of an expert layer, normalised and
 * quantized where it is produced ([BW] Format background: MXFP8; [MT] 5.3: an
 * operand is quantized without another pass over it).  Per row:
 *   sum = bf16(x + residual), added in binary32   (residual NULL: sum = x)
 *   rstd = 1 / sqrt(mean(sum^2) + eps)
 *   y = bf16(sum rstd weight)
 *   q, s = pqm_quantize_mxfp8 (row-wise) of y, the same bytes
 *   x [rows, cols] bf16, row stride ldx; residual likewise with ldr (device)
 *   weight [cols] in weight_dtype (bf16 or binary32)                (device)
 *   sum, y [rows, cols] bf16; q [rows, cols] E4M3; s [rows, cols/32] E8M0;
 *   rstd [rows] binary32, for the backward pass                     (device)
 * sum, y and rstd may be NULL, and so may the pair q, s; one of y and q is
 * required (PQM_ERR_NULL).  sum may be the memory of x or of residual, whose
 * row stride must then be cols (PQM_ERR_SHAPE), and is updated in place; no
 * other output may overlap an input.  The sum and the root are binary64, and y
 * is the nearest bf16 value of the product; rows whose squares leave binary32
 * (values from about 2^63 on) are handled, and so are subnormal values.  A sum
 * or a y beyond bf16 is an infinity; an infinity in sum makes the row's rstd 0
 * and y 0, NaN in its own place; a NaN in sum makes the row's rstd and y NaN.
 * Requires cols % 8 == 0 (% 32 with q, s), cols <= 16384, rows < 2^31,
 * ldx, ldr >= cols, 2^-100 <= eps < infinity (PQM_ERR_SHAPE); x, residual,
 * weight, sum, y and the strides 16-byte aligned, q 8-byte, rstd 4-byte
 * (PQM_ERR_ALIGN).
 */
pqm_status pqm_rmsnorm_quantize_mxfp8(const uint16_t *x, int64_t ldx, const uint16_t *residual,
                                      int64_t ldr, const void *weight, pqm_dtype weight_dtype,
                                      int64_t rows, int64_t cols, float eps, uint16_t *sum,
                                      uint16_t *y, uint8_t *q, uint8_t *s, float *rstd,
                                      hipStream_t stream);

/*
 * Gradients of that norm, straight through the rounding and the encoding:
 * with g = dy weight and h = x rstd (x: the `sum` of the forward call),
 *   dx = bf16(rstd (g - h mean(g h)) + d_sum)   per row: the gradient of x
 *        and of residual alike; d_sum (bf16 [rows, cols], may be NULL) is the
 *        gradient that reaches sum past the norm;
 *   dweight[c] = sum over rows of dy h, binary32, in a fixed order.
 * dy, x, d_sum, dx bf16 [rows, cols] contiguous, rstd binary32 [rows],
 * dweight binary32 [cols] (device).  dx may be the memory of d_sum, and no
 * other output may overlap an input.  workspace (device, 16-byte aligned,
 * contents irrelevant): pqm_rmsnorm_backward_workspace bytes; calls that may
 * run at the same time need separate ones.  rows == 0 writes dweight = 0.
 * Requires cols % 8 == 0, cols <= 16384, rows < 2^31 (PQM_ERR_SHAPE); dy, x,
 * weight, d_sum, dx 16-byte aligned (PQM_ERR_ALIGN).
 */
pqm_status pqm_rmsnorm_backward(const uint16_t *dy, const uint16_t *x, const void *weight,
                                pqm_dtype weight_dtype, const float *rstd, const uint16_t *d_sum,
                                int64_t rows, int64_t cols, uint16_t *dx, float *dweight,
                                void *workspace, size_t workspace_bytes, hipStream_t stream);
size_t pqm_rmsnorm_backward_workspace(int64_t rows, int64_t cols);

/*
 * The router's gate: the k experts of each token, their probabilities, and
 * the balance loss that keeps the experts' loads alike (the topk_ids and prob
 * that pqm_moe_route and pqm_swiglu_prob take).
 *   v = softmax(z) or sigmoid(z) of a token's logits z; p = v / sum(v)
 *   topk_ids[t, j]: the expert of the j-th largest logit, equal logits in the
 *       order of their index;
 *   prob[t, j] = scale v_j / sum of the chosen v  (renormalize 1), or
 *       scale v_j (renormalize 0);
 *   counts[e] = valid tokens that chose e, counts[E] = their number Tv;
 *   prob_sum[e] = sum of p over the valid tokens;
 *   loss = loss_coef E sum_e (counts[e] / (k Tv)) (prob_sum[e] / Tv), 0 when
 *       no token is valid.
 *   logits [tokens, E] bf16 or binary32 (logits_dtype); topk_ids int32 and
 *   prob binary32 [tokens, k]; counts int32 [E + 1], prob_sum binary32 [E],
 *   loss binary32 [1]                                               (device)
 * mask (device, uint8 [tokens], NULL: all valid): the logits of a token with
 * mask 0 are not read; its prob is 0, it takes no part in counts, prob_sum or
 * loss, and its ids are (t k + j) mod E, so that padding loads every expert
 * alike in pqm_moe_route.  A logit of -inf closes an expert to a token
 * (chosen last, prob 0; a row of -inf alone gives prob 0, as do chosen sigmoid
 * scores that all vanish in binary32, z below about -87).  A NaN logit ranks
 * first; it (with softmax also +inf) makes its token's prob, and with it prob_sum
 * and loss, NaN; the ids stay in [0, E).  The arithmetic is binary32.
 * counts, prob_sum and loss go together: all NULL skips the loss, and
 * workspace is then not needed.  workspace (device, 4-byte aligned, contents
 * irrelevant): pqm_moe_gate_workspace bytes; calls that may run at the same
 * time need separate ones.
 * Requires 1 <= k <= 16, k <= num_experts <= 1024, tokens (k + 1) < 2^31
 * (PQM_ERR_SHAPE); logits aligned to their element (PQM_ERR_ALIGN);
 * renormalize 0 or 1 (PQM_ERR_ENUM).
 */
typedef enum pqm_score {
    PQM_SCORE_SOFTMAX = 0,
    PQM_SCORE_SIGMOID = 1
} pqm_score;
pqm_status pqm_moe_gate(const void *logits, pqm_dtype logits_dtype, const uint8_t *mask,
                        int64_t tokens, int64_t num_experts, int64_t k, pqm_score score,
                        int renormalize, float scale, int32_t *topk_ids, float *prob,
                        float loss_coef, int32_t *counts, float *prob_sum, float *loss,
                        void *workspace, size_t workspace_bytes, hipStream_t stream);
size_t pqm_moe_gate_workspace(int64_t tokens, int64_t num_experts);

/*
 * Gradient of the gate with respect to its logits: d_prob (binary32
 * [tokens, k], NULL: none) through the chosen probabilities and d_loss
 * (binary32 [1] on the device) through the loss.  The choice and the counts
 * are held fixed; counts is the forward call's [E + 1], and counts and d_loss
 * go together (both NULL: no loss).  The other arguments are the forward
 * call's.  d_logits [tokens, E] in d_logits_dtype (rounded once), zero for
 * masked tokens, NaN for a token whose prob is; it may not overlap logits.
 * topk_ids may hold any experts (an id twice adds up); ids outside [0, E) add
 * nothing.  Same limits and errors.
 */
pqm_status pqm_moe_gate_backward(const void *logits, pqm_dtype logits_dtype, const uint8_t *mask,
                                 int64_t tokens, int64_t num_experts, int64_t k, pqm_score score,
                                 int renormalize, float scale, const int32_t *topk_ids,
                                 const float *d_prob, float loss_coef, const int32_t *counts,
                                 const float *d_loss, void *d_logits, pqm_dtype d_logits_dtype,
                                 hipStream_t stream);

/*
 * The experts' products for a few routed rows (decode): bf16 activations
 * times NVFP4 weights ([BW] Format background: NVFP4; [MT] 2.2 decode), with
 * neither routing nor activation quantization before it.  Row r belongs to
 * expert e = ids[r]:
 *   out[r, n] = s_g sum_k x[r / divisor, k] q[e, n, k] s_b[e, n, k / 16]
 *   x bf16 [ceil(rows / divisor), K] contiguous; ids int32 [rows]   (device)
 *   w_q [G, N, K/2], w_scale [G, N, K/16], w_outer [G N / w_rows_per_scale]
 *       as pqm_quantize_nvfp4_per_token makes them                  (device)
 *   out [rows, N] bf16 (rounded once) or binary32 per out_dtype     (device)
 * With topk_ids [T, k] as ids: divisor = k for the first projection (x holds
 * the tokens), 1 for the second (x holds one row per assignment).  Any order
 * and any repetition of ids is legal; a row whose id lies outside [0, G) gives
 * zeros.  Sums are binary32, the outer scale is applied to the sum.  The
 * weights are exact; so are x's values down to 2^-31 of the largest of their
 * row, and smaller ones are off by less than 2^-38 of that largest value (large
 * calls hold x in scaled binary16).  A row's result depends on its own x and
 * on the call's sizes alone.  Nothing may overlap out.  The weights are read
 * again for each 16 rows of an expert: from about 32 rows an expert on,
 * pqm_moe_route and pqm_moe_grouped_gemm are faster.
 * Requires rows <= 4096 (more: pqm_moe_route and pqm_moe_grouped_gemm),
 * 1 <= divisor <= 4096, 1 <= G <= 4096, N <= 2^20, K % 32 == 0, 32 <= K <=
 * 2^20, w_rows_per_scale >= 1 dividing G N (PQM_ERR_SHAPE); x, w_q and out
 * 16-byte aligned, the others 4-byte (PQM_ERR_ALIGN).
 */
pqm_status pqm_moe_gemv_nvfp4(const uint16_t *x, const int32_t *ids, int64_t rows, int64_t divisor,
                              const uint8_t *w_q, const uint8_t *w_scale, const float *w_outer,
                              int64_t w_rows_per_scale, int64_t G, int64_t N, int64_t K, void *out,
                              pqm_dtype out_dtype, hipStream_t stream);

/*
 * The same for the gate_up projection, with the weighted SwiGLU in its
 * epilogue: w_q [G, 2 inter, K/2] (gate rows, then up rows), prob binary32
 * [rows], d bf16 [rows, inter] = bf16(silu(gate) up prob[r]).  gate and up
 * stay in binary32 (pqm_swiglu_prob takes them rounded to bf16).
 */
pqm_status pqm_moe_gemv_swiglu_nvfp4(const uint16_t *x, const int32_t *ids, const float *prob,
                                     int64_t rows, int64_t divisor, const uint8_t *w_q,
                                     const uint8_t *w_scale, const float *w_outer,
                                     int64_t w_rows_per_scale, int64_t G, int64_t inter, int64_t K,
                                     uint16_t *d, hipStream_t stream);

/*
 * A whole expert layer for a few tokens (decode), from the residual stream on,
 * in one call: what pqm_rmsnorm_quantize_mxfp8 (without its encoding), the
 * router's product, pqm_moe_gate, the two few-row products and pqm_moe_combine
 * do one after the other.
 *   h = bf16(x + residual)                       (residual NULL: h = x)
 *   y = bf16(h rstd norm_w), the nearest bf16 values, rstd as there
 *   z = y gate_w^T; topk_ids, prob: pqm_moe_gate of z (score, renormalize, scale)
 *   d[t, j] = bf16(silu(g) u prob[t, j]), (g, u) = y[t] W1_e^T, e = topk_ids[t, j]
 *   out[t] = bf16(sum_j d[t, j] W2_e^T), summed in binary32
 * With shared_expert 1 the weights have one expert more, number E, which every
 * token meets with prob 1 as row j = k; it is not among topk_ids.
 *   x, residual, h, y, out [tokens, hidden] bf16; norm_w [hidden] in norm_dtype
 *   (bf16 or binary32); gate_w [E, hidden] bf16; topk_ids int32 and prob
 *   binary32 [tokens, k]; d [tokens, k + shared_expert, inter] bf16  (device)
 *   w1_q [G, 2 inter, hidden / 2] (gate rows, then up rows), w1_scale
 *   [G, 2 inter, hidden / 16], w1_outer [G], w2_q [G, hidden, inter / 2],
 *   w2_scale [G, hidden, inter / 16], w2_outer [G], G = E + shared_expert, as
 *   pqm_quantize_nvfp4_per_token makes them with one outer scale per expert
 * The logits are sums of exact products, in binary64 over partial sums of 32,
 * so that two close ones keep their order; they are rounded to binary32.  d and
 * out are sums in binary32.  The weights are exact in their products; so are y and
 * d down to 2^-31 of the largest value of their row, and smaller values are off by
 * less than 2^-38 of it (they may enter in scaled binary16).  A NaN in a token's
 * row makes that token's results NaN and no other's.  The last bits of d and out may depend on
 * how many tokens and which experts a call has, never on the run.
 * workspace (device, 16-byte aligned, contents irrelevant):
 * pqm_moe_decode_nvfp4_workspace bytes; calls that may run at the same time
 * need separate ones.  No output may overlap an input or another output.
 * Requires tokens <= 64, hidden and inter multiples of 32 in 32 .. 16384,
 * 1 <= k <= 16, k <= E <= 1024, 2^-100 <= eps < infinity (PQM_ERR_SHAPE);
 * shared_expert and renormalize 0 or 1 (PQM_ERR_ENUM); bf16 tensors, norm_w,
 * w1_q and w2_q 16-byte aligned, the others 4-byte (PQM_ERR_ALIGN).
 */
pqm_status pqm_moe_decode_nvfp4(const uint16_t *x, const uint16_t *residual, const void *norm_w,
                                pqm_dtype norm_dtype, float eps, const uint16_t *gate_w,
                                int64_t tokens, int64_t hidden, int64_t inter, int64_t num_experts,
                                int64_t k, int shared_expert, pqm_score score, int renormalize,
                                float scale, const uint8_t *w1_q, const uint8_t *w1_scale,
                                const float *w1_outer, const uint8_t *w2_q,
                                const uint8_t *w2_scale, const float *w2_outer, uint16_t *h,
                                uint16_t *y, int32_t *topk_ids, float *prob, uint16_t *d,
                                uint16_t *out, void *workspace, size_t workspace_bytes,
                                hipStream_t stream);
size_t pqm_moe_decode_nvfp4_workspace(int64_t tokens, int64_t hidden, int64_t inter,
                                      int64_t num_experts, int64_t k, int shared_expert);

/*
 * Dense products of bf16 operands (a router, an output head, any projection
 * that is not an expert's), with what follows them in the same pass:
 *   z = x W^T + bias,   y = act(z) + residual
 *   x [M, K] bf16, row stride ldx; w [N, K] bf16 contiguous          (device)
 *   bias [N] binary32, may be NULL; residual [M, N] bf16, row stride ldr,
 *       may be NULL                                                  (device)
 *   y [M, N] bf16 (rounded once) or binary32 per y_dtype; z [M, N] bf16, for
 *       the backward pass, may be NULL                               (device)
 * act: PQM_ACT_NONE, PQM_ACT_SILU z / (1 + e^-z), or PQM_ACT_GELU
 * z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2.  Sums are binary32 and the
 * activation takes z before its rounding.  A NaN or an infinity of x or of
 * residual reaches its own row of y, one of w or bias its own column.  bf16 y
 * may be the memory of residual, with ldr == N (PQM_ERR_SHAPE); nothing else
 * may overlap an output.  workspace (device, 16-byte aligned, contents
 * irrelevant): pqm_linear_workspace bytes, 0 for many sizes; calls that may run
 * at the same time need separate ones.  A row's sums depend on the sizes alone
 * besides its own values.
 * Requires K % 8 == 0, 8 <= K <= 2^22, 0 <= N <= 2^22, M < 2^29 with fewer than
 * 2^24 tiles of 128 x 128 and M (N + K) <= 2^40, K <= ldx <= 2^22,
 * N <= ldr <= 2^22 (PQM_ERR_SHAPE); x, w, y, z and ldx aligned to 16 bytes,
 * bias 4, residual 2 (PQM_ERR_ALIGN).  Beyond a few rows N and ldr of whole 8
 * and a residual aligned to 16 bytes are faster (8190 x 4096 x 2048 141 us, 4095
 * outputs 203; with everything in the epilogue 168 and 402).
 */
typedef enum pqm_act {
    PQM_ACT_NONE = 0,
    PQM_ACT_SILU = 1,
    PQM_ACT_GELU = 2
} pqm_act;
pqm_status pqm_linear(const uint16_t *x, int64_t ldx, const uint16_t *w, const float *bias,
                      pqm_act act, const uint16_t *residual, int64_t ldr, int64_t M, int64_t N,
                      int64_t K, void *y, pqm_dtype y_dtype, uint16_t *z, void *workspace,
                      size_t workspace_bytes, hipStream_t stream);
size_t pqm_linear_workspace(int64_t M, int64_t N, int64_t K);

/*
 * Gradients of that product (the residual's is dy itself):
 *   dz = bf16(dy act'(z)), the nearest value, the operand of the products; without an
 *        activation it is dy, and z and dz are not used
 *   dx = bf16(dz W + d_x), d_x (bf16 [M, K], row stride ldd, may be NULL): a
 *        gradient that reaches x past this product
 *   dw [N, K] = dz^T x and dbias [N] = sum of dz's rows, binary32, each sum in a
 *        fixed order
 * dy [M, N] bf16, row stride lddy; z and dz bf16 [M, N], dx bf16 [M, K],
 * contiguous.  dx, dw, dbias may be NULL, but not all three; x is read for dw
 * only, w for dx only.  dx may be the memory of d_x, with ldd == K, and dz that
 * of z; nothing else may overlap an output.  M == 0 writes dw = 0, dbias = 0.
 * workspace as above, of pqm_linear_backward_workspace bytes.
 * Requires the sizes above, M <= 2^29 - 32, fewer than 2^24 tiles of 128 x 128 of
 * dx and of dw too, N >= 8, N % 8 == 0, N <= lddy <= 2^22,
 * K <= ldx, ldd <= 2^22 (PQM_ERR_SHAPE); all tensors, lddy and ldx aligned to
 * 16 bytes, d_x to 2 (PQM_ERR_ALIGN).
 */
pqm_status pqm_linear_backward(const uint16_t *dy, int64_t lddy, const uint16_t *x, int64_t ldx,
                               const uint16_t *w, pqm_act act, const uint16_t *z,
                               const uint16_t *d_x, int64_t ldd, int64_t M, int64_t N, int64_t K,
                               uint16_t *dz, uint16_t *dx, float *dw, float *dbias,
                               void *workspace, size_t workspace_bytes, hipStream_t stream);
size_t pqm_linear_backward_workspace(int64_t M, int64_t N, int64_t K);

/*
 * What a policy's logits say of given tokens: the log probabilities that
 * rollout and training are compared by ([MT] 4.5; one formula on both sides),
 * the entropy of each row, and its best alternatives.
 * With x a row of logits, M its largest, u_i = (x_i - M) / temperature,
 * S = sum e^u:
 *   logprob = u_id - log S,   entropy = log S - (sum e^u u) / S,
 *   stats = (M, log S), for the backward pass; M / temperature + log S is the
 *       row's log-sum-exp,
 *   top_ids, top_logprob: the top_n largest logits, equal ones in the order of
 *       their index, and their log probabilities
 *   logits [tokens, vocab] bf16 or binary32 (logits_dtype), row stride ld; ids
 *   int32 [tokens]; logprob, entropy [tokens], stats [tokens, 2], top_logprob
 *   [tokens, top_n] binary32; top_ids int32 [tokens, top_n]        (device)
 * ids may be NULL, then logprob has to be; a row whose id lies outside
 * [0, vocab) is left out: its logits are not read, its results are 0 and its
 * top_ids -1.  logprob, entropy, stats may be NULL (one result is required).
 * A logit of -inf is a token that cannot come; a row of -inf alone has
 * logprob -inf, entropy 0, stats (-inf, 0).  A NaN or +inf makes the row's
 * results NaN (M apart); a NaN ranks first.  The arithmetic is binary32; a row's
 * results depend on tokens, vocab and top_n besides its own values, which decide
 * the order of its sums: between calls of other sizes their last bits may differ,
 * between runs or by the row's place they do not.
 * workspace (device, 8-byte aligned, contents irrelevant):
 * pqm_token_logprobs_workspace bytes, 0 where a row is one workgroup's; calls
 * that may run at the same time need separate ones.
 * Requires 1 <= vocab <= 2^30, vocab <= ld <= 2^30, tokens * ceil(vocab / 8192) < 2^24,
 * 0 <= top_n <= 32, top_n <= vocab, 2^-60 <= temperature <= 2^60
 * (PQM_ERR_SHAPE); tensors aligned to their element (PQM_ERR_ALIGN).
 */
pqm_status pqm_token_logprobs(const void *logits, pqm_dtype logits_dtype, int64_t ld,
                              const int32_t *ids, int64_t tokens, int64_t vocab, float temperature,
                              float *logprob, float *entropy, float *stats, int32_t *top_ids,
                              float *top_logprob, int64_t top_n, void *workspace,
                              size_t workspace_bytes, hipStream_t stream);
size_t pqm_token_logprobs_workspace(int64_t tokens, int64_t vocab, int64_t top_n);

/*
 * Gradient with respect to the logits, for the gradients d_logprob and
 * d_entropy (binary32 [tokens], either may be NULL) of the two:
 *   d_i = (d_logprob ([i = id] - p_i) - d_entropy p_i (log p_i + entropy))
 *         / temperature
 * rounded once to d_logits_dtype; zero in rows that are left out and in rows
 * of -inf alone.  stats and entropy (needed with d_entropy) are the forward
 * call's, the other arguments too.  d_logits [tokens, vocab], row stride ldd,
 * may be the memory of logits, with the same type and stride (PQM_ERR_SHAPE),
 * and may not overlap it otherwise.  ids may be NULL with d_logprob NULL.
 * Same limits and errors; ldd as ld.
 */
pqm_status pqm_token_logprobs_backward(const void *logits, pqm_dtype logits_dtype, int64_t ld,
                                       const int32_t *ids, int64_t tokens, int64_t vocab,
                                       float temperature, const float *stats,
                                       const float *entropy, const float *d_logprob,
                                       const float *d_entropy, void *d_logits,
                                       pqm_dtype d_logits_dtype, int64_t ldd,
                                       hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PQMOE_H */
