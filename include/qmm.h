/*
 * qmm.h -- matrix multiply against GGUF block-quantized weights on AMD
 * MI355X (gfx950).  C ABI: plain pointers and sizes, no framework types.
 *
 * The operation (all entry points):  y[m][n] = sum_k x[m][k] * w[n][k]
 *   W  the weight matrix, N rows of K elements.  Each row is K / block_elems
 *      consecutive GGUF blocks and rows are stored back to back, so row n
 *      starts at byte n * qmm_row_bytes(kind, K).  ("One output row's blocks
 *      are contiguous": redgpu/Vulkore examples/llm/quant_test.cpp, the fused
 *      dequant-matvec section; ferrox-cuda 0.21.0 mul_mm.rs, BODY_SRC and
 *      validate_shape.)  Any byte alignment of W is accepted.
 *   x  activations, row-major [M][K], f32 or f16 (QMM_F32 / QMM_F16), aligned
 *      to their element size.
 *   y  output, row-major [M][N] f32 (y[m * N + n]; ferrox-cuda mul_mm.rs,
 *      BODY_SRC, writes dst[token * n_rows + row]).  Overwritten, never
 *      accumulated into.
 * Each weight element w[n][k] is decoded from its block by its kind's rule:
 * scale * code + bias for the affine kinds, scale * table[code] for the
 * codebook kinds (ferrox-cuda 0.20.0 mul_mm_kinds/codebook.rs, module docs).
 *
 * Numerics.  Accumulation is in f32 and at most one factor of each product
 * is rounded, once, to f16 (relative error <= 2^-11).  The decode GEMV keeps
 * every weight exact (an exact f16 integer times an f32 scale) and, on its
 * matrix-core path, rounds f32 activations once to f16.  The prefill GEMM
 * rounds each decoded weight once to f16 and, for f32 activations, splits
 * each activation into two f16 parts so that the activation stays exact to
 * about 2^-22.  Results satisfy |y - y_exact| <= 1e-3 * sum_k |w||x| + 1e-6
 * per element.  Activations are taken in f16 on the matrix-core paths (the
 * GEMV at M <= 8 for every kind but Q2_K, Q3_K and Q5_K, qmm_moe, the GEMM),
 * so an f32 activation must lie within the f16 range, |x| <= 65504; a larger
 * one overflows to infinity there.  qmm_moe_ffn scales its intermediate
 * activations into that range itself.
 *
 * Ownership and asynchrony.  The caller owns every buffer; the library never
 * allocates device memory.  W, x and ids are read only.  Calls that take a
 * `stream` (a hipStream_t; NULL is the default stream) enqueue their kernels
 * there and return without synchronizing; a fault inside a kernel surfaces at
 * the caller's next synchronization.
 *
 * Errors.  Shape and argument errors are returned before anything is
 * launched, checked in this order: empty shape -> unsupported kind -> K not a
 * whole number of blocks -> K > 2^30 or N > INT32_MAX -> bad dtype -> null
 * pointer, misaligned activation or out-of-range M -> workspace too small.  A refused call computes nothing
 * (ferrox-cuda mul_mm.rs: kind_by_name and MulMmUnsupported -- a kind or
 * shape the kernel cannot do must be refused by name, never computed some
 * other way).  A failed launch returns QMM_ERR_HIP.  qmm_last_error() gives
 * the calling thread's most recent message.
 */
#ifndef QMM_H
#define QMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The eleven kinds, by GGUF type id (ferrox-cuda mul_mm.rs, KINDS; MXFP4 is
 * ggml type tag 39 per codebook.rs, the MXFP4 row). */
enum qmm_kind {
    QMM_Q4_0 = 2,    /*  18 B /  32: f16 d, 16 B nibbles; d*(q-8)               */
    QMM_Q5_0 = 6,    /*  22 B /  32: f16 d, u32 qh, 16 B nibbles; d*(q-16)      */
    QMM_Q8_0 = 8,    /*  34 B /  32: f16 d, 32 int8; d*q                        */
    QMM_Q2_K = 10,   /*  84 B / 256: 16 scale/min bytes, 64 B 2-bit, d, dmin    */
    QMM_Q3_K = 11,   /* 110 B / 256: 32 B hmask, 64 B 2-bit, 12 B scales, d    */
    QMM_Q4_K = 12,   /* 144 B / 256: d, dmin, 12 B 6-bit scales/mins, 128 B     */
    QMM_Q5_K = 13,   /* 176 B / 256: d, dmin, 12 B scales/mins, 32 B qh, 128 B  */
    QMM_Q6_K = 14,   /* 210 B / 256: 128 B ql, 64 B qh, 16 int8 scales, d       */
    QMM_IQ4_NL = 20, /*  18 B /  32: f16 d, 16 B codes into a 16-entry table    */
    QMM_IQ4_XS = 23, /* 136 B / 256: d, scales_h, scales_l[4], 128 B codes      */
    QMM_MXFP4 = 39   /*  17 B /  32: E8M0 scale byte, 16 B of E2M1 codes        */
};

enum qmm_dtype { QMM_F32 = 0, QMM_F16 = 1 };

enum qmm_status {
    QMM_OK = 0,
    QMM_ERR_EMPTY_SHAPE = 1,          /* a zero dimension: nothing to launch   */
    QMM_ERR_UNSUPPORTED_KIND = 2,     /* not one of the eleven kinds           */
    QMM_ERR_K_NOT_BLOCK_ALIGNED = 3,  /* K is not a whole number of blocks     */
    QMM_ERR_BAD_DTYPE = 4,            /* activation dtype not QMM_F32/QMM_F16  */
    QMM_ERR_BAD_ARG = 5,              /* null/misaligned pointer, bad M, ids   */
    QMM_ERR_HIP = 6,                  /* a HIP launch failed                   */
    QMM_ERR_WORKSPACE = 7             /* workspace missing or too small        */
};

/* Largest M the decode GEMV takes in one call. */
#define QMM_GEMV_MAX_M 8

/* Decode GEMV, M = 1: y[N] = W . x[K], f32 x, on the default stream.
 * ferrox-cuda mul_mm.rs worth_a_gemm: one token is a matvec. */
int qmm_gemv(int kind, const void *W, const float *x, float *y, int64_t N, int64_t K);

/* Decode GEMV, 1 <= M <= QMM_GEMV_MAX_M tokens, f32 or f16 x, on `stream`.
 * The few-token product below the GEMM threshold of ferrox-cuda mul_mm.rs
 * (worth_a_gemm: a batch that small stays on the matvec arm) and the
 * one-row-per-output decode matvec of inferencelayer cublas_prefill.rs (the
 * q4_0 GEMV family, y[row] = sum over blocks of scale * code . x).
 * Every weight is decoded exactly; f32 x may be rounded once to f16;
 * products accumulate in f32. */
int qmm_gemv_ex(int kind, const void *W, const void *x, int x_dtype, float *y,
                int64_t M, int64_t N, int64_t K, void *stream);

/* Prefill GEMM: C[M][N] = A[M][K] . W^T with f16 A, on the default stream.
 * Weight tiles are decoded to f16 and multiplied on the matrix cores with f32
 * accumulation (inferencelayer cublas_prefill.rs, CublasPrefill::gemm: f16
 * in, f32 accumulate, y = x . W^T).  A decoded weight beyond the f16 range
 * (|w| > 65504) becomes an infinity; the decode GEMV and qmm_moe keep every
 * weight exact instead. */
int qmm_gemm(int kind, const void *W, const void *A, float *C, int64_t M, int64_t N, int64_t K);

/* Prefill GEMM for any M >= 1 with f32 or f16 A, on `stream`: the same
 * contract (inferencelayer cublas_prefill.rs, CublasPrefill::gemm: y = x . W^T,
 * beta 0, f32 accumulate), and ferrox-cuda mul_mm.rs's batched product
 * (BODY_SRC: every token of the batch against every row, dst[token * n_rows
 * + row]).  f32 A is split into two f16 parts (see Numerics above). */
int qmm_gemm_ex(int kind, const void *W, const void *A, int a_dtype, float *C,
                int64_t M, int64_t N, int64_t K, void *stream);

/* Either path, chosen by the number of tokens as ferrox-cuda mul_mm.rs
 * worth_a_gemm chooses between its matvec arm and its GEMM: the GEMV for
 * M <= QMM_GEMV_MAX_M, the GEMM above.  Numerics and errors as the path
 * taken. */
int qmm_matmul(int kind, const void *W, const void *A, int a_dtype, float *C,
               int64_t M, int64_t N, int64_t K, void *stream);

/* Routed SiLU-gated expert FFN with a weighted top-k combine (model
 * semantics beyond the pages, which stop at the routed expert products of
 * qmm_moe).  W_gu holds E experts of 2 * N_ff rows of K elements (rows
 * [0, N_ff) are the gate, [N_ff, 2 N_ff) the up projection); W_d holds E
 * experts of K rows of N_ff elements; both in the layout of qmm_moe.  For
 * token t and slot s with e = ids[t][s] in [0, E):
 *   h = silu(W_gate[e] . X[t]) * (W_up[e] . X[t]),  silu(v) = v / (1 + e^-v)
 *   Y[t] = sum over such slots of topk_w[t][s] * (W_d[e] . h)
 * X is [M][K] f32 or f16; topk_w is [M][topk] f32; Y is [M][K] f32, 16-byte
 * aligned, overwritten.  Slots whose id lies outside [0, E) add nothing.
 * The products run as qmm_moe (each within 1e-3 sum|w||x| + 1e-6), h and
 * the combine in f32; each pair's h is divided by a power of two that
 * brings max|h| to 2^14 or below before the down product (whose matrix-core
 * path takes f16 activations), and the combine multiplies it back, exactly.
 * The sum over slots runs in a fixed order (the same call gives the same
 * bits).  With fewer than four pairs per expert on average (M * topk < 4 E),
 * whole k-blocks (N_ff, K multiples of 256), topk <= 64 and a kind with a
 * matrix-core decoder over the layout given (repacked: as qmm_gemv_packed;
 * native: Q2_K, Q3_K, Q4_K, Q5_K, Q6_K), the FFN runs in two launches:
 * gate/up with the SiLU-product in its epilogue, then down with the combine
 * in its epilogue.
 * workspace: qmm_moe_ffn_workspace_bytes(E, M, topk, N_ff, K) bytes,
 * 256-byte aligned, overwritten; calls sharing it must not overlap.  Errors as qmm_moe, with both matrices' shapes checked (gate/up
 * first) and a NULL topk_w or misaligned Y as QMM_ERR_BAD_ARG. */
int qmm_moe_ffn(int kind, const void *W_gu, const void *W_d, int64_t E, const int32_t *ids,
                const float *topk_w, int64_t topk, const void *X, int x_dtype, float *Y,
                int64_t M, int64_t N_ff, int64_t K, void *workspace, size_t workspace_bytes,
                void *stream);
/* qmm_moe_ffn over repacked experts: P_gu holds E experts' gate/up records
 * (expert e at e * qmm_packed_bytes(kind, 2 N_ff, K)), P_d their down
 * records (at e * qmm_packed_bytes(kind, K, N_ff)), each from qmm_repack of
 * that expert's rows; both 16-byte aligned.  Kinds as qmm_gemv_packed; K
 * and N_ff multiples of 256; M * topk * max(K, N_ff) below 2^31.  Semantics,
 * numerics, workspace and the remaining errors as qmm_moe_ffn. */
int qmm_moe_ffn_packed(int kind, const void *P_gu, const void *P_d, int64_t E, const int32_t *ids,
                       const float *topk_w, int64_t topk, const void *X, int x_dtype, float *Y,
                       int64_t M, int64_t N_ff, int64_t K, void *workspace, size_t workspace_bytes,
                       void *stream);
/* Workspace of qmm_moe_ffn: the routing words of qmm_moe plus f32 gate/up,
 * h, per-slot down outputs and per-pair scales; 0 for a non-positive
 * argument. */
size_t qmm_moe_ffn_workspace_bytes(int64_t E, int64_t M, int64_t topk, int64_t N_ff, int64_t K);

/* Prefill GEMM for MXFP4 weights on the scaled FP8 x FP4 matrix cores, a
 * separately toleranced variant of qmm_gemm_ex for kind QMM_MXFP4 only (the
 * block: an E8M0 scale byte and 32 E2M1 codes; codebook.rs, the MXFP4 row).
 * The weight blocks go to the matrix cores as they are stored; W must be
 * 16-byte aligned, and its rows are fetched as aligned 16-byte pieces, so the
 * last piece may cover up to 12 bytes past the end of W (never past its
 * 16-byte granule, hence never onto another page).  A (f32 or f16,
 * [M][K]) is first quantized into `workspace` to two MX FP8 terms: per row
 * and 32-element block, hi = E4M3(a / 2^e1) with 2^e1 the smallest power of
 * two with max|a| / 2^e1 <= 448, and lo = E4M3(r / 2^e2) of the residual
 * r = a - 2^e1 hi on its own such scale, both rounded to nearest even; the
 * matrix cores multiply both terms by the weights into one f32 sum.  The
 * two roundings (|a - 2^e1 hi - 2^e2 lo| <= 2^-8 |a|, plus 2^(e1 - 14) where
 * hi is subnormal) are the only difference from the exact product besides
 * f32 accumulation, so |C - exact| <= about 2^-8 . sum|w||a|; blocks whose
 * elements are E4M3 values times one power of two come through exactly.
 * Workspace layout (bytes; Mp = M rounded up to 64, rows past M are zero
 * codes with scale byte 0): hi codes [Mp][K], lo codes [Mp][K], hi scale
 * bytes e1 + 127 [Mp][K/32], lo scale bytes e2 + 127 [Mp][K/32]; within
 * each 32-element block the code at position p is element p / 2 (p even)
 * or 16 + p / 2 (p odd), the order of the MXFP4 nibbles.
 * K a multiple of 128 runs the scaled path; any other K runs qmm_gemm_ex's
 * f16 GEMM.  workspace is device memory of at least
 * qmm_gemm_mx_workspace_bytes(M, K) bytes at 16-byte alignment, overwritten by
 * the call; calls that share it must not overlap.  Errors: kinds other than
 * MXFP4 give QMM_ERR_UNSUPPORTED_KIND, a short workspace QMM_ERR_WORKSPACE,
 * M > 65535 * 64 or more than 2^31 - 8 tiles of 64 x 128 QMM_ERR_BAD_ARG,
 * the rest as qmm_gemm_ex. */
int qmm_gemm_mx(int kind, const void *W, const void *A, int a_dtype, float *C,
                int64_t M, int64_t N, int64_t K, void *workspace, size_t workspace_bytes,
                void *stream);
/* Bytes of workspace qmm_gemm_mx needs: M rounded up to 64, times
 * 2 * K * 33 / 32; 0 for M <= 0, K <= 0 or K not a multiple of 32. */
size_t qmm_gemm_mx_workspace_bytes(int64_t M, int64_t K);

/* Routed expert products, every expert in one grouped launch (plus a small
 * routing prologue when an expert may receive several pairs).  No page
 * defines this operation: the pages name expert routing only as model
 * context (ferrox-cuda 0.20.0 codebook.rs, the MXFP4 row: gpt-oss expert
 * weights; inferencelayer cublas_prefill.rs, the Qwen3-30B-A3B decode
 * estimate).  It is the batched/expert product of a 128-expert top-8
 * mixture with per-pair semantics and nothing more (no gating weights, no
 * combine).  W holds E experts of N rows each, back to back: expert
 * e's row n starts at byte (e * N + n) * qmm_row_bytes(kind, K).
 * ids is [M][topk] int32 in [0, E).  For token t and slot s with
 * e = ids[t][s]:  Y[t][s][:] = W_e . x, where x is X[t] when x_per_slot is 0
 * (X is [M][K]) and X[t][s] when it is 1 (X is [M][topk][K]).  Y is
 * [M][topk][N] f32.  A pair whose id lies outside [0, E) is skipped and its Y
 * row is left as it was; W is never read outside its E experts.
 * workspace is device memory of at least
 * qmm_moe_workspace_bytes(E, M, topk) bytes, overwritten by the call; calls
 * that share a workspace must not overlap. */
int qmm_moe(int kind, const void *W, int64_t E, const int32_t *ids, int64_t topk,
            const void *X, int x_dtype, int x_per_slot, float *Y,
            int64_t M, int64_t N, int64_t K, void *workspace, size_t workspace_bytes,
            void *stream);
size_t qmm_moe_workspace_bytes(int64_t E, int64_t M, int64_t topk);

/* Load-time repack (Vulkore quant_test.cpp, section 4, "repacked fast
 * path": weights are transformed once when loaded so the decode matvec reads
 * aligned planes; values rebuilt from the repacked bytes must equal the
 * native dequantization bit for bit).  The layout is this library's: rows
 * in tiles of 16 (the last padded with zero rows), K in k-blocks of 256
 * elements; tile t and k-block b form one record of 16 * B bytes at
 * (t * K/256 + b) * 16 * B, B being one row's k-block in native bytes (144
 * for Q4_0, IQ4_NL, Q4_K; 136 for MXFP4, IQ4_XS; 176 Q5_0, Q5_K; 272 Q8_0;
 * 210 Q6_K; 84 Q2_K; 110 Q3_K).  A record holds exactly the bytes of its sixteen native row pieces,
 * permuted: first lane sections of 1024 bytes (16-byte slot 16 G + j holds
 * the code bytes that lane j + 16 G of a wave decodes for row j), then row
 * sections (per row: its scales and headers).  The per-kind byte tables are
 * in qmm_repack.hip.
 *
 * Kinds: all eleven (Q4_0, Q5_0, Q8_0, IQ4_NL, MXFP4, IQ4_XS, Q2_K, Q3_K,
 * Q4_K, Q5_K, Q6_K).  Size in bytes of
 * the repacked tensor of N rows of K elements: qmm_packed_bytes (-1 for any
 * other kind, K not a multiple of 256, or N <= 0). */
int64_t qmm_packed_bytes(int kind, int64_t N, int64_t K);

/* Repack N native rows W (byte-aligned, N * qmm_row_bytes(kind, K) bytes)
 * into P (qmm_packed_bytes(kind, N, K) bytes, 16-byte aligned, overwritten)
 * on `stream`.  Errors: the shape checks of qmm_gemv_ex, then a kind without
 * a repacked layout (QMM_ERR_UNSUPPORTED_KIND), K not a multiple of 256
 * (QMM_ERR_K_NOT_BLOCK_ALIGNED), NULL or misaligned pointers
 * (QMM_ERR_BAD_ARG). */
int qmm_repack(int kind, const void *W, void *P, int64_t N, int64_t K, void *stream);

/* Decode GEMV over repacked weights P (from qmm_repack with the same kind,
 * N and K): y[M][N] = x[M][K] . W^T, 1 <= M <= QMM_GEMV_MAX_M, f32 or f16
 * x, on `stream`; the numerics of qmm_gemv_ex (exact weights, x rounded once
 * to f16, f32 accumulation).  Errors as qmm_repack, plus those of
 * qmm_gemv_ex for x, y and M, and M * K >= 2^31 (QMM_ERR_BAD_ARG). */
int qmm_gemv_packed(int kind, const void *P, const void *x, int x_dtype, float *y,
                    int64_t M, int64_t N, int64_t K, void *stream);

/* Matmul over repacked weights, any M: C[M][N] = A[M][K] . W^T with W given
 * as its qmm_repack records P (16-byte aligned).  This is the prefill-GEMM
 * contract of inferencelayer cublas_prefill.rs (CublasPrefill::gemm: a
 * batch of M tokens against one weight matrix, f32 output, beta = 0) over
 * the repacked fast path of Vulkore quant_test.cpp, section 4.  M <=
 * QMM_GEMV_MAX_M runs qmm_gemv_packed; larger M runs the prefill GEMM over
 * the records, which takes Q8_0, Q4_0, Q5_0, IQ4_NL, MXFP4 and IQ4_XS (other
 * kinds give QMM_ERR_UNSUPPORTED_KIND there).  A is [M][K] f32 or f16, C
 * [M][N] f32, overwritten.  Numerics of the GEMM: each weight rounded once
 * to f16 (the f16 product of the code and the block scale; IQ4_XS instead
 * multiplies each 32-element group's product by its exact f32 scale
 * d * (ls - 32), so its weights are not rounded), f16 activations exact, f32
 * activations split into two
 * f16 halves (hi = RN_f16(a), lo = RN_f16(a - hi)) that are both multiplied,
 * f32 accumulation in a fixed order (deterministic):
 * |C - exact| <= 1e-3 . sum|w||a| + 1e-6; as in qmm_gemm_ex, a weight beyond
 * the f16 range (|w| > 65504) becomes an infinity.  Errors: as qmm_gemv_packed for
 * kind, K, dtype and pointers (without its M limit), M * K >= 2^31
 * QMM_ERR_BAD_ARG; above QMM_GEMV_MAX_M tokens also packed bytes >= 2^31 or
 * A bytes (M * K * 2 for f16, * 4 for f32) >= 2^31 QMM_ERR_BAD_ARG. */
int qmm_matmul_packed(int kind, const void *P, const void *A, int a_dtype, float *C,
                      int64_t M, int64_t N, int64_t K, void *stream);

/* Routed expert products (as qmm_moe) over repacked experts: P holds E
 * experts, expert e's records (qmm_repack of its N rows) at byte
 * e * qmm_packed_bytes(kind, N, K).  Kinds and K as qmm_gemv_packed; every
 * pair runs on the matrix cores, so M * topk * K must stay below 2^31.
 * Semantics, workspace and the remaining errors as qmm_moe. */
int qmm_moe_packed(int kind, const void *P, int64_t E, const int32_t *ids, int64_t topk,
                   const void *X, int x_dtype, int x_per_slot, float *Y,
                   int64_t M, int64_t N, int64_t K, void *workspace, size_t workspace_bytes,
                   void *stream);

/* Largest M * K of qmm_gemv_i8 (its per-block scales and code sums are
 * staged in 64 KiB of LDS). */
#define QMM_GEMV_I8_MAX_MK 262144

/* Decode GEMV with integer activations, a separately toleranced variant of
 * qmm_gemv_packed for repacked Q8_0, Q4_0, Q5_0, IQ4_NL or MXFP4 weights,
 * whose codes, table values or doubled E2M1 values are integers that fit in
 * int8 (the integer dot-product
 * path that the ferrox-cuda mul_mm page names and leaves out).  x (f32 or
 * f16, [M][K], finite) is first quantized into `workspace`, per token and
 * 32-element block: amax = max |x|, d = amax / 127 and x / d each rounded to
 * f32 (correctly rounded), then q = x / d rounded to the nearest integer,
 * ties to even (|q| <= 127: cut there where a subnormal d makes x / d larger); a
 * block with d = 0 has q = 0.  Then
 *   y[t][n] = sum over blocks b of d_w[n][b] d[t][b] (sum_i w_i q_i)
 * with each block's integer dot product exact (Q4_0 as code - 8, Q5_0 as
 * code - 16, IQ4_NL as the table value, MXFP4 as twice its E2M1 value with
 * half the block scale) and the scaling and accumulation in
 * f32: for K <= 32768, y is within 2e-5 * sum |w| |d q| + 1e-6 of the exact
 * product with the rebuilt activations d q (the f32 accumulation adds about
 * K * 2^-31 of that sum beyond), and those lie within d / 2 of x.
 * Workspace (qmm_gemv_i8_workspace_bytes(M, K) bytes, 256-byte aligned,
 * overwritten; calls sharing it must not overlap): the codes [M][K] int8,
 * each block's 32 codes in the lane order of the weight codes (Q8_0: element
 * order; the others: position 8G + e holds element 4G + e for e < 4
 * and 16 + 4G + e - 4 otherwise, G = 0..3); at the next multiple of 256
 * bytes the scales d [M][K/32] f32; at the next, the code sums [M][K/32]
 * int32.  1 <= M <= QMM_GEMV_MAX_M and M * K <= QMM_GEMV_I8_MAX_MK.  Errors:
 * as qmm_gemv_packed, other kinds QMM_ERR_UNSUPPORTED_KIND, a larger M * K
 * QMM_ERR_BAD_ARG, a missing, short or misaligned workspace
 * QMM_ERR_WORKSPACE. */
int qmm_gemv_i8(int kind, const void *P, const void *x, int x_dtype, float *y,
                int64_t M, int64_t N, int64_t K, void *workspace, size_t workspace_bytes,
                void *stream);
/* Bytes of workspace qmm_gemv_i8 needs; 0 for M <= 0, K <= 0 or K not a
 * multiple of 32. */
size_t qmm_gemv_i8_workspace_bytes(int64_t M, int64_t K);

/* Bytes of the device scratch that qmm_gemv_i8_noalloc uses on each GPU:
 * qmm_gemv_i8_workspace_bytes at the largest M * K. */
#define QMM_GEMV_I8_SCRATCH_BYTES 327680

/* qmm_gemv_i8 without a workspace argument, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc.  It calls no allocating routine;
 * the quantized activations go to a scratch of QMM_GEMV_I8_SCRATCH_BYTES
 * that the library holds in each GPU's memory (a static device array, in
 * place from library load until the process ends; its address on the
 * current device is looked up on the first call there).  Same kernels,
 * arguments, numerics and results bit for bit as qmm_gemv_i8.  Nothing in
 * the scratch needs to start at zero: every call writes all it reads, and
 * the scratch keeps the last call's contents.  Calls that overlap on one
 * GPU (two streams, or two host threads) race on the scratch and must be
 * serialized by the caller; calls on different GPUs do not share it.
 * Errors: as qmm_gemv_i8 without its workspace checks (M * K above
 * QMM_GEMV_I8_MAX_MK, whose workspace would exceed the scratch, gives
 * QMM_ERR_BAD_ARG), and QMM_ERR_HIP when the scratch cannot be located on
 * the current device. */
int qmm_gemv_i8_noalloc(int kind, const void *P, const void *x, int x_dtype, float *y,
                        int64_t M, int64_t N, int64_t K, void *stream);

/* ------------------------------------------------------------------------
 * Products with an epilogue: what a layer does with a projection's sums before
 * anything else reads them.  Model semantics beyond the pages, like
 * qmm_moe_ffn.
 *   out[m][n] = act(sum_k A[m][k] w[n][k] + bias[n]) * mul[m][n] + residual[m][n]
 * with act one of
 *   QMM_ACT_NONE       v
 *   QMM_ACT_RELU       max(v, 0)
 *   QMM_ACT_SILU       v / (1 + e^-v)
 *   QMM_ACT_GELU       v (1 + erf(v / sqrt 2)) / 2
 *   QMM_ACT_GELU_TANH  v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2
 * A NULL bias, mul or residual leaves its step out; mul and residual are
 * [M][N], f32 or f16, with row strides in elements (>= N), bias is [N] f32.  A
 * gated FFN is act(x . W_gate^T) into g, then mul = g in the product with W_up.
 * out is f32 or f16 with a row stride; it may be mul or residual itself (same
 * type and stride), and overlaps nothing else.  The sum is held to the plain entry
 * points' accuracy, the epilogue is in f32 (activations within 2^-20 relative of
 * their value at the f32 sum with its bias, or within 2^-126 where that value is
 * below f32's normal range), and the result is rounded once to out's type: an f16
 * out beyond 65504 is an infinity.
 * --------------------------------------------------------------------- */
enum qmm_act { QMM_ACT_NONE = 0, QMM_ACT_RELU = 1, QMM_ACT_SILU = 2, QMM_ACT_GELU = 3, QMM_ACT_GELU_TANH = 4 };
typedef struct qmm_epilogue {
    const float *bias;
    const void *mul;
    const void *residual;
    int64_t mul_stride;
    int64_t residual_stride;
    int act;
    int mul_dtype;
    int residual_dtype;
} qmm_epilogue;

/* qmm_matmul with an epilogue (ep NULL: none).  A of more than QMM_GEMV_MAX_M tokens
 * is 16-byte aligned.  The sum is the GEMV's (f32 A rounded once to f16, weights
 * exact) up to QMM_GEMV_MAX_M tokens, and beyond them while the 16 x 16 tiles of
 * [M][N] are few: K a multiple of 256 up to 2^20 and at most seven tiles a compute
 * unit (four over native IQ4_XS rows), on 256 units 112 tokens at N = 4096 and 7168
 * at N = 64.  Otherwise it is the GEMM's (weights rounded once to f16, f32 A in two
 * f16 parts, as qmm_matmul takes any M above QMM_GEMV_MAX_M).  Some of these sizes
 * decode the weights once into the workspace, to f16 as the GEMM rounds them, with
 * f32 activations' two parts beside them, and multiply from there:
 * qmm_matmul_ep_workspace_bytes gives its size, 0 where none is used.  It is device
 * memory, 256-byte aligned, overwritten; calls sharing it must not overlap.  Errors as
 * qmm_matmul, with the dtypes of out, mul and residual beside A's, a stride below N,
 * an unknown act or a misaligned operand as QMM_ERR_BAD_ARG, and last a short
 * workspace as QMM_ERR_WORKSPACE. */
int qmm_matmul_ep(int kind, const void *W, const void *A, int a_dtype, const qmm_epilogue *ep, void *out,
                  int out_dtype, int64_t out_stride, int64_t M, int64_t N, int64_t K, void *workspace,
                  size_t workspace_bytes, void *stream);
/* qmm_matmul_packed with an epilogue and that workspace, at any M for every kind
 * (those that qmm_matmul_packed's GEMM does not take, and records of 2^31 bytes and
 * more, go through the workspace: K up to 2^20 there); errors as both. */
int qmm_matmul_packed_ep(int kind, const void *P, const void *A, int a_dtype, const qmm_epilogue *ep, void *out,
                         int out_dtype, int64_t out_stride, int64_t M, int64_t N, int64_t K, void *workspace,
                         size_t workspace_bytes, void *stream);
/* Bytes of workspace of qmm_matmul_ep (packed 0) and qmm_matmul_packed_ep (packed
 * 1) on the current device; 0 also for shapes, kinds and dtypes that they refuse. */
size_t qmm_matmul_ep_workspace_bytes(int kind, int packed, int64_t M, int64_t N, int64_t K, int a_dtype);

/* The product of qmm_gemv_i8 over activations that are quantized already (by
 * qmm_rmsnorm_q8, for this kind of weights), with an epilogue: codes [M][K]
 * int8, 16-byte aligned, scales and code_sums [M][K / 32].  Kinds, sizes (M <=
 * QMM_GEMV_MAX_M, M * K <= QMM_GEMV_I8_MAX_MK), numerics and errors as
 * qmm_gemv_i8 and qmm_matmul_ep.  More rows than M are taken by more calls: row
 * t's codes start at t * K, its scales and sums at t * K / 32. */
int qmm_gemv_q8(int kind, const void *P, const int8_t *codes, const float *scales, const int32_t *code_sums,
                const qmm_epilogue *ep, void *out, int out_dtype, int64_t out_stride, int64_t M, int64_t N, int64_t K,
                void *stream);

/* Root-mean-square norm of [T][H][D] rows (H packed rows of D elements at t *
 * stride: the heads of a projection, or H = 1), with the residual's addition:
 *   h = x + residual, rounded to f32 (residual NULL: x)
 *   y = h / sqrt(mean(h^2) + eps) * weight    (weight [D] f32, or NULL: 1)
 * sum (if not NULL) receives h in the residual's type, y is f32 or f16.  Each of
 * x and residual is f32 or f16.  The mean and y are computed in 64 bits and y is
 * rounded to f32, then to f16: within 2^-24 relative (f16: 2^-11 + 2^-24, and
 * 2^-25 absolute below its normal range).  A row of zeros with eps = 0 gives
 * zeros.  An infinity in a row gives NaN at its place and zeros elsewhere, a NaN
 * gives a row of NaN.  sum and y may each be x or residual itself (same type and
 * stride) but not each other; other overlaps are not allowed.
 * Errors: a zero dimension, dtypes, then QMM_ERR_BAD_ARG: D > 32768, H > 65536, T *
 * H * D > 2^40 or T * H >= 2^31, eps negative or not finite, sum without residual,
 * sum equal to y, pointers, alignment to the elements, strides below H * D. */
int qmm_rmsnorm(const void *x, int x_dtype, int64_t x_stride, const void *residual, int residual_dtype,
                int64_t residual_stride, const float *weight, float eps, void *sum, int64_t sum_stride, void *y,
                int y_dtype, int64_t y_stride, int64_t T, int64_t H, int64_t D, void *stream);
/* qmm_rmsnorm of [T][D] rows with y in 8 bits, as qmm_gemv_i8 quantizes the f32
 * y (bit for bit; a block with an infinity or NaN gets a NaN for its scale): codes
 * [T][D] in the lane order of the weights of `kind`, scales and code_sums [T][D /
 * 32], all contiguous, codes 16-byte aligned.  They overlap no operand.  Errors as
 * qmm_rmsnorm, with unsupported kinds (those of qmm_gemv_i8) and D not a multiple
 * of 32 before the dtypes. */
int qmm_rmsnorm_q8(int kind, const void *x, int x_dtype, int64_t x_stride, const void *residual, int residual_dtype,
                   int64_t residual_stride, const float *weight, float eps, void *sum, int64_t sum_stride,
                   int8_t *codes, float *scales, int32_t *code_sums, int64_t T, int64_t D, void *stream);

/* The choice of experts for qmm_moe, qmm_moe_ffn: per token t, from its logits
 * l_e (f32 or f16, row stride in elements),
 *   s_e = e^(l_e) / sum_j e^(l_j)   (QMM_ROUTE_SOFTMAX), or
 *   s_e = 1 / (1 + e^(-l_e))        (QMM_ROUTE_SIGMOID)
 *   c_e = s_e + bias[e]             (bias [E] f32, or NULL: c_e = s_e)
 * With n_group > 1 the experts lie in n_group groups of E / n_group; a group's
 * value is the sum of its group_top (1 or 2) largest c, and only the topk_group
 * groups of the largest values keep their experts.  The topk largest c that are
 * left are chosen, in their order; equal ones (groups too) go by the lowest
 * index.  ids [M][topk] int32 gets their numbers and weights [M][topk] f32 their
 * s_e, divided by the chosen ones' sum if normalize is 1, times scale.
 * An expert whose logit or c is NaN or minus infinity is never chosen and has no
 * part in the softmax; a row that runs out of experts, and every row t with
 * slots[t] < 0 (slots [M] int32, or NULL: none; the padding tokens of
 * qmm_kv_append) gets ids of -1, which qmm_moe skips, and weights of 0.
 * Numerics: the choice is that of 64-bit scores (without a bias, and with
 * group_top = 1, that of the logits themselves), so neighbours that f32 cannot
 * tell apart keep their order; weights are within 2^-20 relative, also where
 * every chosen score vanishes.
 * Errors: a zero dimension, dtype, then QMM_ERR_BAD_ARG: E > 4096, topk > 64 or
 * above the topk_group * E / n_group experts that can be left, n_group > 64, E
 * not a multiple of it, topk_group outside [1, n_group], group_top not 1 or 2, an
 * unknown score, normalize not 0 or 1, scale not finite, M >= 2^31, pointers,
 * alignment, a stride below E. */
enum qmm_route_score { QMM_ROUTE_SOFTMAX = 0, QMM_ROUTE_SIGMOID = 1 };
int qmm_moe_route(const void *logits, int dtype, int64_t stride, const float *bias, int64_t M, int64_t E,
                  int64_t topk, int score, int64_t n_group, int64_t topk_group, int group_top, int normalize,
                  float scale, const int32_t *slots, int32_t *ids, float *weights, void *stream);

/* Dequantize n_elems consecutive elements (whole blocks) of W to f32 on
 * `stream`: the GPU dequantization that redgpu/Vulkore quant_test.cpp checks
 * bit for bit against its CPU references (its dequant_q8_0 / _q5_0 / _q4_k /
 * _q6_k kernels, the per-kind dequant test), and ferrox-cuda mul_mm.rs's
 * dequant_twin, one block's elements to f32 by the kind's rule.  Every value
 * is the f32 rounding of the exact value, evaluated scale first with IEEE
 * signed zeros (so MXFP4 code 8 gives -0.0; codebook.rs, the E2M1 table).
 * Errors: as qmm_gemv_ex's kind check, then n_elems not a whole number of
 * blocks (QMM_ERR_K_NOT_BLOCK_ALIGNED), NULL pointers (QMM_ERR_BAD_ARG). */
int qmm_dequant(int kind, const void *W, float *out, int64_t n_elems, void *stream);

/* ------------------------------------------------------------------------
 * The attention side of a decode step: rotary positions, a paged key/value
 * cache held in block formats, and attention of one new token per sequence
 * over it.  Model semantics beyond the pages, like qmm_moe_ffn; these are the
 * operators between the projections that the products above compute.
 *
 * The cache of a layer is two arrays of pages, one for keys and one for
 * values, each page holding page_size tokens of n_kv heads of head_dim
 * elements in one of three kinds (the two arrays may differ):
 *   QMM_CACHE_F16   2 bytes an element, rounded to nearest (|x| <= 65504)
 *   QMM_Q8_0        32-element blocks, value d * c, c in [-127, 127]:
 *                   d = the smallest f16 >= max|x| / 127 (at most 65504),
 *                   c = RNE(x / d)
 *   QMM_Q4_0        value d * (c - 8), c in [0, 15]: |d| = the smallest f16 >=
 *                   max|x| / 8 with the sign that makes the largest element
 *                   (the positive one at a tie) code 0, c = RNE(x / d) + 8,
 *                   at most 15
 * with f32 quotients; |value - x| <= |d| / 2 except where a Q4_0 code was cut
 * to 15 (up to |d|).  A block holding an infinity or a NaN reads back as NaN.
 * page_size is a multiple of 32 (at most 65536) and head_dim one of 64, 96,
 * 128, 192, 256.  A page is qmm_kv_page_bytes(...) bytes, 16-byte aligned, and
 * holds [n_kv][page_size / 32] groups of 32 tokens; a group is its codes
 * followed by its f16 scales (none for F16) as [head_dim / 32][32 tokens].
 * The codes of block b (elements 32b + c) of the group's token r (base =
 * b * 2048 bytes for F16, 1024 Q8_0, 512 Q4_0; i = 4 (r / 8) + r % 4,
 * m = (r / 4) % 2, integer division):
 *   keys    F16   half  at ((4m + c/8) * 16 + i) * 16 + 2 (c % 8)
 *           Q8_0  c+128 at ((16 (c/8) + i) * 2 + m) * 8 + c % 8
 *           Q4_0  byte  at ((16 (c%16/4) + i) * 2 + m) * 4 + c % 4, elements
 *                 below 16 in the low nibble
 *   values  F16   half  at ((4 (c/16) + r/8) * 16 + c % 16) * 16 + 2 (r % 8)
 *           Q8_0  c+128 at ((16 (r/8) + c % 16) * 2 + c/16) * 8 + r % 8
 *           Q4_0  byte  at (16 (r/8) + c % 16) * 8 + r % 8, same nibbles
 * A page need not be initialized: bytes of tokens that no call has written
 * are never given weight, whatever they hold.
 *
 * A slot names a token's place: slot = page * page_size + offset, int32,
 * with n_pages * page_size below 2^31.  A slot outside [0, n_pages *
 * page_size) marks a token to skip (padding): nothing is written for it, and
 * it reads as zeros.  Two tokens of one call must
 * not name the same slot (that slot's contents are then unspecified).
 *
 * Row strides are in elements: row t of a [T][H][head_dim] operand starts at
 * t * stride, its heads packed (stride >= H * head_dim), so that the q, k and
 * v parts of one projection's output need no copies.
 * --------------------------------------------------------------------- */
#define QMM_CACHE_F16 1
int64_t qmm_kv_page_bytes(int kind, int64_t page_size, int64_t n_kv, int64_t head_dim); /* -1: refused */

/* How the pairs of the rotated part of a head lie: (i, i + n_rot/2) or
 * (2i, 2i + 1). */
enum qmm_rope_layout { QMM_ROPE_HALF = 0, QMM_ROPE_INTERLEAVED = 1 };

/* Angles per position of the n_rot / 2 pairs, on the HOST (no GPU work; the
 * caller copies them to the device once): freqs[i] = base^(-2i / n_rot),
 * divided by factors[i] if factors is not NULL (the per-pair factors some
 * GGUF files carry), then for factor > 1
 *   orig_ctx = 0   divided by factor (positions interpolated linearly);
 *   orig_ctx > 0   YaRN: with dim(n) = n_rot ln(orig_ctx / (2 pi n)) /
 *                  (2 ln base), low = max(floor(dim(beta_fast)), 0), high =
 *                  min(ceil(dim(beta_slow)), n_rot - 1) and ramp = clamp((i -
 *                  low) / max(high - low, 0.001), 0, 1), the mean of freqs[i]
 *                  (weight 1 - ramp) and freqs[i] / factor (ramp).
 * *mscale (if not NULL) becomes 0.1 ln(factor) + 1 for YaRN, else 1.
 * Errors: n_rot <= 0 QMM_ERR_EMPTY_SHAPE; odd n_rot, NULL freqs, base <= 1,
 * factor < 1 (or not finite), negative orig_ctx, YaRN without beta_fast >
 * beta_slow > 0, or one of factors zero or not finite QMM_ERR_BAD_ARG. */
int qmm_rope_freqs(double *freqs, float *mscale, int64_t n_rot, double base, const float *factors, double factor,
                   int64_t orig_ctx, double beta_fast, double beta_slow);

/* Rotary positions: y = x with, in every head of row t, pair (a, b) number i
 * turned by phi = pos[t] * freqs[i] (freqs: n_rot / 2 f64 on the device):
 *   y_a = mscale (x_a cos phi - x_b sin phi)
 *   y_b = mscale (x_a sin phi + x_b cos phi);
 * elements n_rot .. head_dim - 1 are copied.  mscale cos and mscale sin are
 * computed in 64 bits, so far positions lose nothing, and rounded once to f32, as
 * are the products (within 2^-22 mscale (|x_a| + |x_b|), before the rounding to
 * f16).  x is [T][H][head_dim] f32 or f16, y f32 or f16, head_dim and n_rot even, n_rot <= head_dim.  y may be x itself
 * (same stride and type); any other overlap is not allowed.
 * Errors: a zero dimension, dtype, then pointers, alignment, strides, layout,
 * n_rot and T * H * head_dim > 2^32 as QMM_ERR_BAD_ARG. */
int qmm_rope(const double *freqs, int64_t n_rot, int layout, float mscale, const int32_t *pos, const void *x,
             int x_dtype, int64_t x_stride, void *y, int y_dtype, int64_t y_stride, int64_t T, int64_t H,
             int64_t head_dim, void *stream);

/* Writes T tokens' keys and values ([T][n_kv][head_dim], both of `dtype`) into
 * the cache at their slots.  Errors: a zero dimension, unsupported kinds,
 * head_dim not a multiple of 32 (QMM_ERR_K_NOT_BLOCK_ALIGNED), dtype, then
 * QMM_ERR_BAD_ARG for any other head_dim or page_size, n_kv > 1024, T * n_kv *
 * head_dim >= 2^31, NULL or misaligned pointers and short strides. */
int qmm_kv_write(int k_kind, int v_kind, void *k_pages, void *v_pages, int64_t n_pages, int64_t page_size,
                 int64_t n_kv, int64_t head_dim, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                 int dtype, const int32_t *slots, int64_t T, void *stream);

/* qmm_rope on q and k and qmm_kv_write of the rotated k and of v, in one
 * launch: what a decode step does between the projections and the
 * attention.  q is [T][n_q][head_dim] of `dtype`, q_out of q_out_dtype (it may
 * be q itself, as in qmm_rope); the rotated k is quantized from f32.  Tokens
 * with a skipped slot still get their q rows.  Errors as qmm_kv_write (with T *
 * (n_q + n_kv) * head_dim below 2^31) and qmm_rope. */
int qmm_kv_append(const double *freqs, int64_t n_rot, int layout, float mscale, const int32_t *pos, const void *q,
                  int64_t q_stride, int64_t n_q, void *q_out, int q_out_dtype, int64_t q_out_stride, int k_kind,
                  int v_kind, void *k_pages, void *v_pages, int64_t n_pages, int64_t page_size, int64_t n_kv,
                  int64_t head_dim, const void *k, int64_t k_stride, const void *v, int64_t v_stride, int dtype,
                  const int32_t *slots, int64_t T, void *stream);

/* Reads T tokens back: k_out and v_out [T][n_kv][head_dim], contiguous, f32
 * (exact) or f16 (the value rounded once).  Errors as qmm_kv_write. */
int qmm_kv_read(int k_kind, int v_kind, const void *k_pages, const void *v_pages, int64_t n_pages, int64_t page_size,
                int64_t n_kv, int64_t head_dim, const int32_t *slots, int64_t T, void *k_out, void *v_out, int dtype,
                void *stream);

/* Attention of one new token per sequence: for sequence b and query head h,
 * with key head h / (n_q / n_kv),
 *   s_t = scale * q . k_t,  out = sum_t e^{s_t} v_t / (sum_t e^{s_t} + e^{sinks[h]})
 * over the tokens max(0, len - window) <= t < len, len = seq_lens[b] (window 0:
 * all of them; sinks NULL: no such term).  Token t lies in page
 * block_table[b * max_pages + t / page_size] at offset t % page_size.  The new
 * token's own key and value are part of the cache (qmm_kv_append first).  q is
 * [B][n_q][head_dim] f32 or f16 with a row stride, out [B][n_q][head_dim],
 * contiguous, of the same type; out may be q itself where q is contiguous, and
 * overlaps nothing else.  A sequence without tokens (length 0 or
 * below) gives zeros; lengths are cut to max_pages * page_size; tokens whose
 * page number lies outside [0, n_pages) count as absent.
 * Numerics: keys and values are exact (codes as integers, block scales in
 * f32 or folded into the weight); scores, softmax and sums are f32.  f16 q is
 * exact (beside quantized keys down to 2^-35 of the head's largest element) and
 * the weights, times the value's block scale, are rounded once to f16; f32 q is
 * carried as two f16 terms (2^-21 of an element, or 2^-39 of the head's largest),
 * and weights as f32.  With w_t the exact weights,
 *   |out - exact| <= (r + 2 max_t e_t) sum_t w_t |v_t| + a  (+ f16 out's rounding)
 * where r = 2^-11 + 2^-18 for f16 and 2^-18 for f32, and e_t = c (scale * sum
 * over 32-element blocks of (sum |q| + 2^-13 max |q| of the whole head) (max
 * |k_t|) + max |s| + 40) with c = 2^-17 for f16 and 2^-20 for f32 bounds a
 * score's error.  a is 0 for f32
 * (weights below 2^-100 of the largest may count as 0); for f16 it is what f16
 * weights lose far below the strongest, 2^-39 M sum_t |c_t|, with c_t the code
 * of the value (F16: the value itself) and M the largest product of a weight
 * and a block scale (F16: 1) of two tokens with the same t / 8: it counts in
 * elements that are empty in all strong tokens and in blocks far smaller than
 * the others of their head, where a caller for whom they matter takes f32 q.
 * The bound holds at every length: long sums carry what they round off.  The
 * order of every sum is fixed: a call repeated gives the same bits.
 * n_q is a multiple of n_kv.  workspace: qmm_attn_decode_workspace_bytes(B,
 * n_q, n_kv, head_dim) bytes, 16-byte aligned, overwritten (it need not be
 * initialized); calls sharing it must not overlap.  Nothing depends on the
 * host's knowledge of the lengths, so a captured call replays with others.
 * Errors: a zero dimension, kinds and head_dim as qmm_kv_write, dtype, then
 * QMM_ERR_BAD_ARG (n_q not a multiple of n_kv, B * n_q > 2^23, max_pages *
 * page_size >= 2^31, scale not finite, window < 0, pointers, alignment, stride), then QMM_ERR_WORKSPACE. */
int qmm_attn_decode(int k_kind, int v_kind, const void *k_pages, const void *v_pages, int64_t n_pages,
                    int64_t page_size, int64_t n_kv, int64_t head_dim, const void *q, int dtype, int64_t q_stride,
                    int64_t n_q, const int32_t *block_table, int64_t max_pages, const int32_t *seq_lens, int64_t B,
                    float scale, int64_t window, const float *sinks, void *out, void *workspace,
                    size_t workspace_bytes, void *stream);
/* 0 for a non-positive argument, n_q not a multiple of n_kv or sizes
 * qmm_attn_decode refuses. */
size_t qmm_attn_decode_workspace_bytes(int64_t B, int64_t n_q, int64_t n_kv, int64_t head_dim);

/* Geometry and names.  qmm_row_bytes is the expected row length of
 * ferrox-cuda mul_mm.rs validate_shape ((K / block_elems) * block_bytes),
 * -1 for a bad kind or K not a whole number of blocks.  qmm_block_geometry
 * gives a kind's block_bytes and block_elems, the two geometry columns of
 * mul_mm.rs's KINDS rows (QMM_OK, or QMM_ERR_UNSUPPORTED_KIND with the
 * outputs untouched).  qmm_kind_from_name is mul_mm.rs's kind_by_name over
 * the GGUF quant names ("Q4_0", "MXFP4", ...): -1 where kind_by_name gives
 * None, so a caller must fall back and say so.  qmm_kind_name is its
 * inverse (NULL for an unsupported kind).  qmm_status_string names a
 * status; qmm_last_error gives the calling thread's most recent message
 * (the refused check, in the order of validate_shape, or the HIP error). */
int64_t qmm_row_bytes(int kind, int64_t K);
int qmm_block_geometry(int kind, int *block_bytes, int *block_elems);
int qmm_kind_from_name(const char *gguf_name);
const char *qmm_kind_name(int kind);
const char *qmm_status_string(int status);
const char *qmm_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* QMM_H */
