/*
 * qblk.h -- C ABI of libqblk: 4-bit block quantization of weight matrices and
 * the fused dequantize-and-multiply that streams the blocks, for AMD Instinct
 * MI355X (gfx950).
 *
 * Formats (all little-endian, no padding: the packed bytes are the storage
 * format itself):
 *
 *   QBLK_Q4_0        32 weights in 18 bytes (4.5 bit/weight):
 *                      [d: fp16][qs: 16 bytes]
 *                    byte qs[j] holds the 4-bit code of weight j in its low
 *                    nibble and of weight j+16 in its high nibble; a weight is
 *                    d * (code - 8).
 *                    ("GGUF 量化内幕 第4章 Q4_0" (sxkj888.cn), sections 4.1.2,
 *                    4.2.1, 4.2.2, 4.3.)
 *
 *   QBLK_SB4         super-block of 256 weights in 138 bytes (4.3125 bit/weight):
 *                      [S: fp16][sc: 8 x int8][qs: 8 x 16 bytes]
 *                    eight Q4_0-style sub-blocks of 32 whose fp16 scales are
 *                    themselves quantized to INT8 in [-127, 127] under the fp16
 *                    super-scale S = max(scale)/127; a weight of sub-block j is
 *                    (S * sc[j]) * (code - 8).
 *                    ("GGUF K-quants" blog (hugo-blog-2v1.pages.dev), section
 *                    "套娃": the super-block, steps 1-5 and the storage table.)
 *
 *   QBLK_SB4_AFFINE  affine super-block of 256 weights in 148 bytes (4.625 b/w):
 *                      [Ss: fp16][Sa: fp16][sc: 8 x int8][ac: 8 x int8][qs: 128]
 *                    per sub-block scale (max-min)/15 and offset min with codes
 *                    0..15; scales and offsets are each INT8-quantized under
 *                    their own fp16 super-scale; a weight is
 *                    (Ss * sc[j]) * code + (Sa * ac[j]).
 *                    (Same blog, section "套娃": Type 1 blocks also carry an
 *                    offset whose fp16 value is compressed to INT8.)
 *
 *   QBLK_Q4_K        super-block of 256 weights in 144 bytes (4.5 bit/weight):
 *                      [d: fp16][dmin: fp16][f: 12 bytes][qs: 8 x 16 bytes]
 *                    per 32-weight sub-block j a 6-bit scale s_j and a 6-bit
 *                    min m_j; field i of the sixteen 6-bit fields (s_0..s_7,
 *                    then m_0..m_7) sits at bits 6i..6i+5 of f read as one
 *                    little-endian integer; codes 0..15 stored as in Q4_0;
 *                    a weight is (d * s_j) * code - dmin * m_j.
 *                    (Q4_0 chapter, section 4.6, which names the 6-bit
 *                    packing without describing it: the field order is this
 *                    library's.)
 *
 *   QBLK_W4G128      groups of 128 weights along a row, one fp16 scale each
 *                    (66 bytes per group, 4.125 bit/weight), stored as two
 *                    planes: first the codes, k/2 bytes per row (byte j of
 *                    group g holds weight 128g+j in its low nibble and weight
 *                    128g+64+j in its high nibble, codes stored +8), then the
 *                    scales, k/128 fp16 values per row.  Symmetric: scale
 *                    d = absmax/7, a weight is d * (code - 8).  Products take
 *                    8-bit activations (qblk_quantize_act_i8, qblk_gemm_w4a8).
 *                    (TurboQuant W4A8 article (codechina.net), sections 2.1
 *                    and 2.2; the layout is this library's, the page gives
 *                    none.)
 *
 * Matrices are dense row-major.  A packed matrix of rows x k weights stores row
 * r, block b at byte (r * k/E + b) * B, with E weights and B bytes per block
 * (QBLK_W4G128: the two planes above, rows * k/E * B bytes in all).
 *
 * Quantization rule (the same for all formats; both the codes and the INT8
 * or 6-bit scales are computed against the scale the block STORES, decoded
 * back from fp16): code = clamp(round_half_away(v / s), lo, hi), with IEEE
 * fp32 division, a zero scale giving code 0 (Q4_0/Type 0: stored code 8),
 * fp16 rounding to nearest even with subnormals kept.  Q4_0 uses s = absmax/7
 * per 32 weights.  The GPU library reproduces the CPU definition bit for bit.
 *
 * Conventions for every entry point:
 *   - Pointers to data are DEVICE pointers owned by the caller; the library
 *     allocates nothing and keeps no mutable state, so calls are reentrant.
 *   - Work is enqueued on `stream` (a hipStream_t; NULL = the null stream) and
 *     the call returns without waiting.  Device faults surface at the caller's
 *     next synchronization.
 *   - Arguments are checked on the host before any launch; on error nothing is
 *     launched and nothing is written.  A failed launch returns
 *     QBLK_ERR_LAUNCH.
 *   - Data pointers must be 16-byte aligned (QBLK_ERR_ALIGN); the fp32
 *     per-token scale arrays of the 8-bit activations only 4-byte aligned.
 *   - k must be a multiple of the format's block size (QBLK_ERR_SHAPE);
 *     rows/m/n/k may be 0 (an empty product writes zeros to y when m, n > 0).
 *   - rows, m, n and k must each stay below 2^31, and a packed matrix below
 *     2^40 bytes (QBLK_ERR_SHAPE); qblk_gemm and qblk_gemm_w4a8 take at most
 *     m = 2^28 rows (QBLK_ERR_SHAPE).  A call whose grid would exceed the
 *     2^32 - 1 threads one launch can hold (the quantizers, dequant, the
 *     activation quantizer and the batch-1 products at very large sizes)
 *     is run as several launches in stream order.
 *   - Inputs must be finite; non-finite inputs give unspecified results.
 *     A block whose scale overflows fp16 (|w| > 7 * 65504 for Q4_0 and
 *     Type 0, a 32-weight range above 15 * 65504 for Type 1) is stored with an
 *     infinite scale; that is well defined for Q4_0 but not for super-blocks.
 */
#ifndef QBLK_H
#define QBLK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  QBLK_Q4_0 = 0,       /* 32 weights, 18 bytes  */
  QBLK_SB4 = 1,        /* 256 weights, 138 bytes */
  QBLK_SB4_AFFINE = 2, /* 256 weights, 148 bytes */
  QBLK_Q4_K = 3,       /* 256 weights, 144 bytes */
  QBLK_W4G128 = 4      /* 128 weights, 66 bytes (two planes) */
} qblk_format_t;

typedef enum {
  QBLK_F32 = 0,  /* IEEE binary32 */
  QBLK_F16 = 1,  /* IEEE binary16 */
  QBLK_BF16 = 2  /* bfloat16      */
} qblk_dtype_t;

typedef enum {
  QBLK_OK = 0,
  QBLK_ERR_NULL = 1,        /* a required pointer is NULL               */
  QBLK_ERR_SHAPE = 2,       /* negative/too large size, k not a multiple */
  QBLK_ERR_DTYPE = 3,       /* element type not accepted by this call   */
  QBLK_ERR_ALIGN = 4,       /* a data pointer is not 16-byte aligned    */
  QBLK_ERR_UNSUPPORTED = 5, /* format/type combination not implemented  */
  QBLK_ERR_LAUNCH = 6,      /* the kernel launch failed                 */
  QBLK_ERR_FORMAT = 7,      /* unknown format                           */
  QBLK_ERR_WORKSPACE = 8    /* the workspace is smaller than the call needs */
} qblk_status_t;

typedef void* qblk_stream_t; /* hipStream_t */

/* One product of qblk_gemv_batch: y (m fp32) = W x with W (m x k) in blocks
 * and x (k elements); device pointers owned by the caller. */
typedef struct {
  const void* blocks;
  int64_t m;
  const void* x;
  float* y;
} qblk_gemv_item_t;

/* Most products one qblk_gemv_batch call takes. */
#define QBLK_GEMV_BATCH_MAX 32

/* Geometry.  qblk_block_bytes/elems return 0 for an unknown format;
 * qblk_packed_bytes returns 0 if k is not a multiple of the block size or a
 * size is negative. */
size_t qblk_block_bytes(qblk_format_t fmt);
int qblk_block_elems(qblk_format_t fmt);
size_t qblk_packed_bytes(qblk_format_t fmt, int64_t rows, int64_t k);

/* Quantize w (rows x k, element type wt in {F32, F16, BF16}, read exactly as
 * fp32 values) into Q4_0 blocks (qblk_packed_bytes(QBLK_Q4_0, rows, k) bytes).
 * Q4_0 chapter section 4.1.1 gives the absmax/7 scale; sections 4.1.2-4.2.2
 * the layout and the +8 code offset. */
qblk_status_t qblk_quantize_q4_0(const void* w, qblk_dtype_t wt, int64_t rows,
                                 int64_t k, void* blocks, qblk_stream_t stream);

/* Quantize w into super-blocks: affine = 0 gives QBLK_SB4 (Type 0), affine = 1
 * gives QBLK_SB4_AFFINE (Type 1).  K-quants blog, section "套娃", steps 1-4
 * for the INT8 sub-scales (and offsets). */
qblk_status_t qblk_quantize_sb4(const void* w, qblk_dtype_t wt, int64_t rows,
                                int64_t k, int affine, void* blocks,
                                qblk_stream_t stream);

/* Quantize w (element type F32, F16 or BF16) into QBLK_Q4_K super-blocks.
 * Q4_0 chapter, section 4.6 gives the form y = d*s_j*q - dmin*m_j; the steps
 * it leaves open are taken as: sub-block range lo = min(0, min w), hi = max w;
 * first-level scale (hi - lo)/15 and min -lo in fp32; d = fp16(max scale/63),
 * dmin = fp16(max min/63); s_j, m_j = clamp(round_half_away(v / stored), 0, 63);
 * codes clamp(round_half_away((w + dmin*m_j) / (d*s_j)), 0, 15) with the
 * rebuilt (exact fp32) d*s_j and dmin*m_j. */
qblk_status_t qblk_quantize_q4_k(const void* w, qblk_dtype_t wt, int64_t rows,
                                 int64_t k, void* blocks, qblk_stream_t stream);

/* Quantize w (element type F32, F16 or BF16, k a multiple of 128) into
 * QBLK_W4G128 groups: per row, each group of 128 weights takes the scale
 * d = fp16(max|w| / 7) and codes clamp(round_half_away(w / d), -8, 7) + 8
 * against the stored d (TurboQuant article, section 2.1: per-row symmetric
 * groups of 128, scale from the group's own maximum, 4-bit integers). */
qblk_status_t qblk_quantize_w4g128(const void* w, qblk_dtype_t wt, int64_t rows,
                                   int64_t k, void* blocks, qblk_stream_t stream);

/* 8-bit activations (TurboQuant article, section 2.2, which leaves the
 * activation scaling open): for each of the n rows (tokens) of x (n x k,
 * type xt, k a multiple of 8), one symmetric scale s = max|x| / 127 kept in
 * fp32 (scale[t], n floats) and codes xq = clamp(round_half_away(x / s),
 * -127, 127) (n x k int8, row-major); a zero row gives s = 0 and codes 0. */
qblk_status_t qblk_quantize_act_i8(const void* x, qblk_dtype_t xt, int64_t n,
                                   int64_t k, int8_t* xq, float* scale,
                                   qblk_stream_t stream);

/* W4A8 product Y = X W^T with W (m x k) in QBLK_W4G128 and X given as the
 * int8 codes xq (n x k) and token scales (n floats) of
 * qblk_quantize_act_i8: Y[t,i] = scale[t] * sum_g d[i,g] *
 * sum_{k in g} (code - 8) * xq[t,k], Y n x m fp32 row-major.  The integer
 * sums are exact; Y is within 2e-5 * sum_k |W[i,k] * scale[t] * xq[t,k]| of
 * the exact product of the rebuilt weights and activations.  n = 1 runs a
 * batch-1 kernel (k <= 16384); otherwise int8 matrix cores, with the k range
 * split over the grid (partial sums added into Y, zeroed first by this call)
 * when m*n is small.  qblk_gemv and qblk_gemm return QBLK_ERR_UNSUPPORTED
 * for QBLK_W4G128. */
qblk_status_t qblk_gemm_w4a8(const void* blocks, int64_t m, int64_t k,
                             const int8_t* xq, const float* scale, int64_t n,
                             float* y, qblk_stream_t stream);

/* Q4_0 quantization as the Q4_0 chapter's section 4.4 prints it: the signed
 * value of largest magnitude divided by -8 is the scale, codes are
 * min(15, trunc(w * (1/d) + 8.5)) with the fp32 reciprocal.  Input F32 only
 * (QBLK_ERR_DTYPE otherwise).  Output layout as QBLK_Q4_0. */
qblk_status_t qblk_quantize_q4_0_ref(const void* w, qblk_dtype_t wt,
                                     int64_t rows, int64_t k, void* blocks,
                                     qblk_stream_t stream);

/* Rebuild the weights from blocks into out (rows x k, type ot in {F32, F16,
 * BF16}).  F32 output is the fp32 value of the format's formula (Q4_0
 * chapter section 4.3 for Q4_0; K-quants blog step 5 for the super-blocks;
 * chapter section 4.6 for Q4_K, one rounding of the exact product minus the
 * exact min); F16/BF16 outputs are that value rounded to nearest even. */
qblk_status_t qblk_dequant(qblk_format_t fmt, const void* blocks, int64_t rows,
                           int64_t k, void* out, qblk_dtype_t ot,
                           qblk_stream_t stream);

/* Batch-1 product y = W x for W (m x k) in blocks: x has k elements of type xt
 * in {F32, F16, BF16}; y has m fp32 elements.  Products are formed from the
 * exact codes and x, accumulated in fp32; the result is within
 * 2e-5 * sum_k |W[i,k] x[k]| of the exact sum of the rebuilt weights times x. */
qblk_status_t qblk_gemv(qblk_format_t fmt, const void* blocks, int64_t m,
                        int64_t k, const void* x, qblk_dtype_t xt, float* y,
                        qblk_stream_t stream);

/* Several batch-1 products that share the format, k and the type of x, in
 * one launch: items[i].y = W_i x_i for i < count (count <= 32, the items
 * read during the call only).  Each product is the one qblk_gemv computes,
 * with the same bound; a layer's matrices of equal k (a transformer's q, k, v
 * and o projections, or gate and up) then share one grid instead of paying a
 * kernel boundary each.  Items with m = 0 are skipped; argument errors in any
 * item are returned before any launch.  fp16 x with k <= 12288 runs as one
 * launch; other x types or longer rows run one launch per item. */
qblk_status_t qblk_gemv_batch(qblk_format_t fmt, int64_t k, qblk_dtype_t xt,
                              const qblk_gemv_item_t* items, int count,
                              qblk_stream_t stream);

/* Small-batch product Y = X W^T: X is n x k row-major (token-major) of type xt,
 * Y is n x m row-major fp32.  All four formats run on the bf16 matrix cores
 * with xt = BF16; F32/F16 activations, and Q4_0 with k % 256 != 0, return
 * QBLK_ERR_UNSUPPORTED.  Same error bound as qblk_gemv, per output element.
 * When k spans many groups and m*n is small the k range is split over the
 * grid and partial sums are added into Y (zeroed first by this call), so the
 * summation order, not the bound, varies between tilings and between runs
 * (qblk_set_deterministic turns the split off). */
qblk_status_t qblk_gemm(qblk_format_t fmt, const void* blocks, int64_t m,
                        int64_t k, const void* x, qblk_dtype_t xt, int64_t n,
                        float* y, qblk_stream_t stream);

/* Reproducible products.  With on != 0, qblk_gemm and qblk_gemm_w4a8 never
 * split the k range over workgroups: every output is summed by one
 * workgroup in a fixed order, so identical inputs and sizes give bitwise
 * identical Y on the same device, run after run (split sums are added into
 * Y with fp32 atomics, whose order varies).  Slower where the split paid: few
 * tokens, or few rows with a long k.  The setting is process-wide, applies to
 * calls made after it, and is off at load.  Always returns QBLK_OK.  (Not an
 * operation of the pages: a property of this implementation's sums.) */
qblk_status_t qblk_set_deterministic(int on);

/* 1 when reproducible products are on (qblk_set_deterministic), else 0. */
int qblk_deterministic(void);

/* ------------------------------------------------------------------------
 * 8-bit floating point with a scale for each block of 128: the format for the
 * matrices that 4 bits are too few for (dense feed-forward layers, shared
 * experts, the output head).  Codes are OCP e4m3 (4 exponent bits, 3 mantissa
 * bits, largest value 448, no infinities), one byte each, row-major; a scale
 * covers 128 x 128 weights (wscale[r/128][c/128], ceil(rows/128) x k/128
 * fp32), or 128 columns of one token (xscale[t][c/128], n x k/128 fp32).
 * Rule: scale = max|v| / 448 in fp32; code = e4m3(clamp(v / scale, +-448)),
 * round to nearest even, both divisions IEEE fp32; a zero scale gives code 0.
 * A NaN makes the scale of its block NaN, and so what the block enters; with an
 * infinity the scale is infinite, its own code NaN and the others' 0.
 * k must be a multiple of 128, a product's matrix at most 2^26 rows of at most
 * 2^24 columns (QBLK_ERR_SHAPE).
 *
 * The products: Y[t,r] = sum_g xscale[t,g] wscale[r/128,g] *
 * (sum over the 128 columns of g of code * code), Y n x m row-major of type
 * yt in {F32, F16, BF16}, one rounding at the end.  Sums over groups are fp32
 * in a fixed order, so equal inputs give bitwise equal outputs.  The sum inside
 * a group is exact to fp32 rounding too up to 64 tokens, and for F32 results
 * at any number.  F16 and BF16 results of more than 64 tokens are formed by
 * the fp8 matrix instructions, which drop of the products of 8 neighbouring
 * columns what lies below 2^-13 of the largest: 1.4e-5 of the result in the
 * 2-norm on normal data, 7e-5 with channels 1000 times the others, and up to
 * 7 * 2^-13 of the largest product of each 8 columns in a single result.  The two
 * scales are multiplied first, in fp32: a group counts as long as xscale * wscale
 * is a normal number (about 1e-38 to 3e38).
 *
 * Workspaces (also of the calls below) are device memory owned by the caller,
 * 16-byte aligned, of at least the bytes that the call's _workspace function
 * gives (0: none needed, NULL is fine; it also gives 0 for sizes the call
 * rejects).  They hold no state between calls and may be shared by calls on
 * the same stream. */

/* Quantize w (rows x k, type wt in {F32, F16, BF16}). */
qblk_status_t qblk_quantize_f8(const void* w, qblk_dtype_t wt, int64_t rows,
                               int64_t k, uint8_t* codes, float* scale,
                               qblk_stream_t stream);

/* Quantize the n rows (tokens) of x (n x k, type xt). */
qblk_status_t qblk_quantize_act_f8(const void* x, qblk_dtype_t xt, int64_t n,
                                   int64_t k, uint8_t* xq, float* scale,
                                   qblk_stream_t stream);

/* Y = X W^T with W (m x k) and X (n x k) given as codes and scales (several
 * products of one X then share its quantization). */
size_t qblk_gemm_f8_workspace(int64_t m, int64_t k, int64_t n);
qblk_status_t qblk_gemm_f8(const uint8_t* w, const float* wscale, int64_t m,
                           int64_t k, const uint8_t* xq, const float* xscale,
                           int64_t n, void* y, qblk_dtype_t yt,
                           void* workspace, size_t workspace_bytes,
                           qblk_stream_t stream);

/* The same with X given as values of type xt, quantized by the call by the
 * rule of qblk_quantize_act_f8. */
size_t qblk_linear_f8_workspace(int64_t m, int64_t k, int64_t n);
qblk_status_t qblk_linear_f8(const uint8_t* w, const float* wscale, int64_t m,
                             int64_t k, const void* x, qblk_dtype_t xt,
                             int64_t n, void* y, qblk_dtype_t yt,
                             void* workspace, size_t workspace_bytes,
                             qblk_stream_t stream);

/* A gated feed-forward layer: H = silu(Wg X) * (Wu X) in fp32, Y = W2 H, with X
 * and H quantized per token and 128 columns.  w13 is (2*inter) x hidden, the
 * inter rows of Wg before those of Wu; w2 is hidden x inter; hidden and inter
 * are multiples of 128; X and Y are n x hidden.  silu(v) = v / (1 + exp(-v)).
 * The sums of the first product use the fp8 matrix instructions for BF16
 * results of more than 64 tokens only, because the codes of H turn on them: they
 * move 1e-3 (normal data) to 2.3e-3 (channels 1000 times the others) of the result
 * in the 2-norm, beside the 1.7e-3 of rounding to BF16. */
size_t qblk_ffn_f8_workspace(int64_t hidden, int64_t inter, int64_t n);
qblk_status_t qblk_ffn_f8(const uint8_t* w13, const float* s13,
                          const uint8_t* w2, const float* s2, int64_t hidden,
                          int64_t inter, const void* x, qblk_dtype_t xt,
                          int64_t n, void* y, qblk_dtype_t yt,
                          void* workspace, size_t workspace_bytes,
                          qblk_stream_t stream);

/* A mixture-of-experts layer for a few tokens, out of packed 4-bit experts:
 *
 *   Y[t] = sum_j weights[t,j] * D_e (silu(G_e X[t]) * (U_e X[t])),  e = ids[t,j]
 *
 * gate_up holds experts x (2*inter) rows of hidden weights (per expert the
 * inter rows of G before those of U), down experts x hidden rows of inter
 * weights, both packed in fmt (QBLK_Q4_0, QBLK_SB4, QBLK_SB4_AFFINE or
 * QBLK_Q4_K; hidden and inter multiples of its block, at most 2^19).  X is
 * n x hidden of type xt in {F16, BF16}, Y n x hidden of type yt.
 *
 * Routing.  With logits (n x experts fp32) the call chooses each token's
 * top_k experts itself, in descending order of the logit, equal logits in
 * order of the expert, and writes ids (n x top_k) and weights: the softmax of
 * the logits over the chosen experts (renorm != 0) or over all of them
 * (renorm = 0), times weight_scale.  A logit of -infinity or NaN takes its
 * expert out; where fewer than top_k are left the remaining ids are -1 with
 * weight 0, and a token with none gets Y = 0.  (+infinity counts as the
 * largest finite value.)  With logits = NULL, ids and weights are inputs from
 * a router of the caller's, taken as they are (renorm and weight_scale are not
 * looked at); ids outside [0, experts) contribute nothing.
 *
 * Products are formed from the exact codes and 16-bit activations, sums are
 * fp32, the intermediate keeps 16 mantissa bits; the order of the sums is fixed,
 * so equal inputs give bitwise equal outputs.  Each token depends on its own
 * row of X and its own experts only.  experts <= 512, top_k <= 32.  Tokens
 * beyond 1024/top_k run as further launches; from some hundred tokens on,
 * one matrix product per expert is the better tool.  ids, weights and Y are
 * written when n and hidden are positive (for inter = 0 only Y, as zeros). */
typedef struct {
  int fmt; /* a qblk_format_t; plain ints, so that any value can be refused */
  int64_t n, hidden, inter;
  int experts, top_k;
  const void* x;
  int xt; /* a qblk_dtype_t */
  const float* logits; /* or NULL */
  int renorm;
  float weight_scale;
  const void* gate_up;
  const void* down;
  int32_t* ids;   /* n x top_k: written with logits, else read */
  float* weights; /* n x top_k: likewise */
  void* y;
  int yt; /* a qblk_dtype_t */
  void* workspace;
  size_t workspace_bytes;
} qblk_moe_t;

size_t qblk_moe_workspace(const qblk_moe_t* args); /* reads the sizes and fmt only */
qblk_status_t qblk_moe(const qblk_moe_t* args, qblk_stream_t stream);

/* ------------------------------------------------------------------------
 * OCP microscaling (MX): 32 neighbouring values of a row under one power of two,
 * kept as the byte e + 127 (e8m0; 255: every value of the block is NaN).  Rows
 * of k values, k a multiple of 32: codes row-major, scales rows x k/32 bytes.
 *
 *   QBLK_ACT_MXFP4   e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives), two
 *                    to a byte: column 2j in the low half of byte j, k/2 bytes a row
 *   QBLK_ACT_MXFP8   e4m3, a byte each
 *
 * Rule: e = floor(log2(max|v|)) - 2 (MXFP4) or - 8 (MXFP8), at least -127 (a block
 * of zeros: -127); code = the element nearest to v / 2^e, halves to the even code,
 * beyond the largest element (6 or 448) that one; all exact, so equal inputs give
 * equal bytes everywhere.  A NaN or an infinity in a block makes its scale 255
 * and its codes 0.
 *
 * The products: Y[t,r] = sum_c W[r,c] X[t,c] with W (m x k) in MXFP4 and X
 * (n x k) in either, an element being code * 2^e; Y n x m row-major of type yt in
 * {F32, F16, BF16}, one rounding at the end, sums in fp32 in a fixed order (equal
 * inputs, equal bits).  With MXFP4 activations, and with MXFP8 ones and F32
 * results, sums are exact to fp32 rounding.  F16 and BF16 results of MXFP8
 * activations are formed by the 8-bit matrix instructions, which drop of the
 * products of 8 neighbouring columns what lies below 2^-13 of the largest.  A token
 * with a NaN block has NaN results, and so has a row of W with one.  With MXFP8
 * and F32 elements are taken as bf16 numbers: multiples of 2^-133 (others, of
 * blocks under the lowest scales, may move by that much) below 2^128 (all that the
 * quantizers make; others are infinite).
 * m at most 2^26, k at most 2^23 (QBLK_ERR_SHAPE).
 *
 * Codes are 16-byte aligned, the scales' bytes at any address; workspaces as for
 * the 8-bit products above. */
typedef enum {
  QBLK_ACT_NONE = -1, /* qblk_rmsnorm only: no codes */
  QBLK_ACT_F8 = 0,    /* e4m3, fp32 scale per 128 columns (qblk_quantize_act_f8) */
  QBLK_ACT_I8 = 1,    /* int8, fp32 scale per row (qblk_quantize_act_i8) */
  QBLK_ACT_MXFP8 = 2,
  QBLK_ACT_MXFP4 = 3
} qblk_act_t;

/* Quantize v (rows x k, type vt in {F32, F16, BF16}); elem is one of the two MX
 * formats (QBLK_ERR_FORMAT otherwise, as everywhere below). */
qblk_status_t qblk_quantize_mx(const void* v, qblk_dtype_t vt, int64_t rows,
                               int64_t k, qblk_act_t elem, void* codes,
                               uint8_t* scale, qblk_stream_t stream);

/* The values that codes and scales stand for, rounded once to type ot. */
qblk_status_t qblk_dequant_mx(const void* codes, const uint8_t* scale,
                              qblk_act_t elem, int64_t rows, int64_t k,
                              void* out, qblk_dtype_t ot, qblk_stream_t stream);

/* Y = X W^T from the codes and scales of both. */
size_t qblk_gemm_mxfp4_workspace(int64_t m, int64_t k, int64_t n,
                                 qblk_act_t act);
qblk_status_t qblk_gemm_mxfp4(const uint8_t* w, const uint8_t* wscale,
                              int64_t m, int64_t k, const void* xq,
                              const uint8_t* xscale, qblk_act_t act, int64_t n,
                              void* y, qblk_dtype_t yt, void* workspace,
                              size_t workspace_bytes, qblk_stream_t stream);

/* The same with X given as values of type xt, quantized to `act` by the call. */
size_t qblk_linear_mxfp4_workspace(int64_t m, int64_t k, int64_t n,
                                   qblk_act_t act);
qblk_status_t qblk_linear_mxfp4(const uint8_t* w, const uint8_t* wscale,
                                int64_t m, int64_t k, const void* x,
                                qblk_dtype_t xt, qblk_act_t act, int64_t n,
                                void* y, qblk_dtype_t yt, void* workspace,
                                size_t workspace_bytes, qblk_stream_t stream);

/* Root-mean-square norm of n rows (tokens) of `hidden` values, with the codes that
 * a product reads:
 *
 *   t = x + residual, rounded to the type xt (t = x where residual is NULL)
 *   y = t * (1 / sqrt(mean(t^2) + eps)) * weight     in fp32
 *
 * total: t (n x hidden of type xt), written where residual is given; it may be the
 * same memory as x or as residual.  y: the normed values rounded to xt, or NULL.
 * codes and scale: y quantized by the rule and in the layout of `act` (hidden a
 * multiple of 128 for QBLK_ACT_F8, of 32 for the MX formats, of 8 for
 * QBLK_ACT_I8 and QBLK_ACT_NONE), from the fp32 values.  Other outputs must not
 * overlap any input or one another.  weight has `hidden` values of type wt in
 * {F32, F16, BF16}; eps >= 0 (QBLK_ERR_SHAPE).  Squares are fp32: |t| and |t * weight|
 * have to stay below 1.8e19, and with eps = 0 a row's root mean square above 1e-18; a row
 * of zeros with eps = 0 gives NaN.  A row's results do not depend on the rows beside it.
 * hidden at most 2^24. */
typedef struct {
  int64_t n, hidden;
  const void* x;
  const void* residual; /* or NULL */
  int xt;               /* a qblk_dtype_t; plain ints, so that any value can be refused */
  const void* weight;
  int wt; /* a qblk_dtype_t */
  float eps;
  int act; /* a qblk_act_t */
  void* codes;
  void* scale;
  void* total;
  void* y;
} qblk_rmsnorm_t;

qblk_status_t qblk_rmsnorm(const qblk_rmsnorm_t* args, qblk_stream_t stream);

/* Static English text for a status code (never NULL). */
const char* qblk_status_string(qblk_status_t st);

/* Library version as "major.minor.patch" (static string). */
const char* qblk_version(void);

#ifdef __cplusplus
}
#endif
#endif /* QBLK_H */
