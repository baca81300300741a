/*
 * qk.h -- C ABI of the GB300 (sm_103a) quantised-weight GEMV / GEMM library.
 *
 * The library multiplies GGUF block-quantised weights by fp32 activations,
 * decoding every block inside the multiply.  That is what the nurllama
 * runtime does with weight types it has a device kernel for: their GGUF bytes
 * go to the device unchanged and each block is decoded inside the matmul
 * (nurllama 0.18.1 API reference, model.nu), through its quantised matvec
 * dispatch `lk_matvec_q ks gt wd xd yd rows cols batch` (same page,
 * kernels.nu).  One entry point per weight format; there is no
 * type dispatch and no host fallback.
 *
 * Operation (every entry point):
 *   y[b][r] = sum_{c < K} W[row_offset + r][c] * x[b][c]
 * with W row-major, the column index fastest: row r of W starts at element
 * r*K (the layout contract of kernels.nu).
 *
 * Block formats (the pages name them, the bytes follow the GGUF layouts):
 *   Q8_0 : 34-byte blocks of 32 weights: fp16 d, then 32 int8 q;  w = d*q.
 *   Q4_K : 144-byte super-blocks of 256 weights: fp16 d, fp16 dmin, 12 bytes
 *          of packed 6-bit sub-block scales sc and mins m (8 sub-blocks of
 *          32), 128 bytes of 4-bit quants q;  w = d*sc*q - dmin*m.
 *   A row holds ceil(K / 32) (Q8_0) or ceil(K / 256) (Q4_K, Q6_K) whole
 *   blocks; columns >= K inside a row's last block are ignored.  In
 *   strict-blocks mode (qk_set_strict_blocks) a K that is not a whole number
 *   of blocks is refused instead (QK_ERR_BAD_DIM).
 *
 * Row addressing: `w` points at the first byte of the whole tensor, and a call
 * uses rows [row_offset, row_offset + rows).  Row r starts at byte
 * r * row_bytes with row_bytes = blocks_per_row * block_bytes.  This is how
 * the parts of a fused tensor are addressed (in nurllama too a weight is a
 * device pointer with a row count and the parts of a fused tensor are ranges
 * of its rows: nurllama README, "What it runs", phi3), and how one expert of
 * a 3-D expert tensor [E][rows_e][K] is addressed: row_offset = e*rows_e + r0.
 *
 * Ownership and execution: every pointer is a device pointer owned by the
 * caller; the library allocates and frees nothing per call and keeps no
 * per-call state.  Calls are asynchronous on `stream` (NULL = the legacy
 * default stream) and never synchronise.
 *
 * Errors: argument errors are detected on the host before any launch and
 * leave every output untouched; a failed launch returns QK_ERR_CUDA.  Device
 * waits are bounded: a kernel whose wait runs out records the fact in a
 * device error word and returns early (its outputs are then unspecified);
 * qk_device_error() reads and clears that word.
 */
#ifndef QK_H
#define QK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st *qk_stream_t;

typedef enum {
    QK_OK = 0,
    QK_ERR_NULL = 1,        /* a required pointer is NULL                              */
    QK_ERR_BAD_DIM = 2,     /* rows/N/M <= 0, K <= 0, row_offset < 0, ldy too small;
                               strict-blocks mode: K not a whole number of blocks      */
    QK_ERR_ALIGN = 3,       /* w, x or y misaligned (see each call)                     */
    QK_ERR_BATCH = 4,       /* GEMV batch outside [1, QK_MAX_BATCH]                     */
    QK_ERR_CUDA = 5,        /* a CUDA runtime call or launch failed                     */
    QK_ERR_TIMEOUT = 6,     /* a bounded device wait ran out (from qk_device_error)     */
    QK_ERR_WORKSPACE = 7,   /* workspace NULL, misaligned or smaller than required      */
    QK_ERR_TOO_LARGE = 8,   /* a size exceeds what the kernels support (see each call)  */
    QK_ERR_BAD_INDEX = 9,   /* an index read from device memory was out of range        */
                            /* (from qk_device_error; see qmatvec_experts_*)             */
    QK_ERR_TYPE = 10        /* an element type is none of qk_dtype                       */
} qk_status;

/* Element types of the attention operators' queries, keys, values and outputs. */
typedef enum { QK_F32 = 0, QK_F16 = 1, QK_BF16 = 2 } qk_dtype;

#define QK_MAX_BATCH 8

/*
 * Q8_0 GEMV, batch 1..8: y[b*ldy + r] = sum_{c<K} W[row_offset + r][c] * x[b*K + c].
 *   w      device, raw Q8_0 block bytes of the whole tensor; 2-byte aligned.
 *   x      device fp32 [batch][K], row stride K; 4-byte aligned.
 *   y      device fp32 [batch][ldy]; writes y[b*ldy + r] for r < rows only;
 *          4-byte aligned.  ldy == 0 means ldy = rows.
 *   K      columns, any K >= 1.  A launch keeps its activation rows (about
 *          4.1 to 4.6 bytes a column each, K rounded up to the block size) in
 *          shared memory next to at least one staged tile of weight rows; a
 *          batch whose activations do not fit in the device's shared memory
 *          per block is computed by several launches of fewer batch rows
 *          (each batch row's result is the same as in a call of that size).
 *          A K for which one activation row does not fit (above about 48000
 *          on GB300) returns QK_ERR_TOO_LARGE before any launch.
 * Accuracy (every GEMV entry point; the tests check these bounds).  The
 * arithmetic is fp32 and a result differs from the exact dot product by at
 * most 1e-5 * S + 1e-6 + A, per element, where
 *   S = sum_c |x[b][c]| * (the magnitudes of the terms the weight is made
 *       of): |w| for Q8_0, |d*sc*q| + |dmin*m| for Q4_K and
 *       |d*scale*q| + 32*|d*scale| for Q6_K.  The kernels sum a Q4_K or Q6_K
 *       weight's two terms separately, so this is sum|w*x| unless the terms
 *       of the weights nearly cancel (then S is the larger);
 *   A is the term of the activation encoding, 0 where x is used as fp32:
 *     - Batch 1 holds each 32-column group of x as 24-bit integers that
 *       share one binary exponent: that of the group's largest magnitude
 *       or, when the largest is at least 2^3 times (in binary exponent)
 *       every other value of the group, that of the second largest, the
 *       largest value then being carried exactly on its own.  A value of
 *       x is thus held within 2^-20 times the second largest magnitude of
 *       its group (the largest within 2^-22 of itself), and
 *       A = 2^-20 * sum_groups (second largest |x| of the group) *
 *                   (sum |w| over the group's columns).
 *       A single outlier per group, at any magnitude, therefore costs
 *       nothing, and A is far inside 1e-5 * S unless a row's weights sit
 *       mostly on values much smaller than their group's second largest
 *       (for instance two values 2^20 times the rest in one group, meeting
 *       zero weights).
 *     - Batch 2..8 takes one of two forms.  Q8_0 with K a multiple of 128
 *       (K up to 4096) and Q4_K (K up to 4864) take the tensor-core form
 *       when the call has at least 128 rows per SM of the device (19456
 *       rows on 152 SMs) and, for Q4_K, batch 4..8; other calls take the
 *       fp32 form, for which A = 0.  The tensor-core form applies the same
 *       rule for a lone outlier (carried exactly), then holds each 32-column
 *       group of a batch row as two fp16 pieces of x scaled by the power of
 *       two that puts the group's largest remaining magnitude M in
 *       [2^14, 2^15) ([2^10, 2^11) for the high-nibble groups of Q4_K): a
 *       value is held within 2^-24 of itself or within 2^-39 (2^-35) * M,
 *       whichever is more (M taken as at least 2^-100), so
 *       A = 2^-35 * sum_groups M * (sum |w| over the group's columns).  Each form's arithmetic for a row depends on K
 *       only: row ranges of a tensor give the bits of the whole call when
 *       both take the same form.
 *   NaN and infinities in x give non-finite results.
 */
int qmatvec_q8_0(const void *w, int64_t row_offset, int64_t rows, int64_t K,
                 const float *x, int batch, float *y, int64_t ldy, qk_stream_t stream);

/*
 * Q4_K GEMV, batch 1..8.  Same contract as qmatvec_q8_0, with w 16-byte
 * aligned (144-byte super-blocks keep every row 16-byte aligned).
 */
int qmatvec_q4_k(const void *w, int64_t row_offset, int64_t rows, int64_t K,
                 const float *x, int batch, float *y, int64_t ldy, qk_stream_t stream);

/*
 * Q6_K GEMV, batch 1..8.  Same contract as qmatvec_q8_0 (w 2-byte aligned:
 * 210-byte super-blocks).  Q6_K is the format of lm_head / ffn_down in the
 * Q4_K_M files people download (their output weight is Q4_K or Q6_K:
 * nx_f32_llm_v4.nx source, lm_head binder comment; kernel `mv_q6_k`,
 * nurllama 0.18.1 API reference, kernels.nu).  Block reading (GGUF):
 * ql[128] | qh[64] | scales[16] int8 | fp16 d per 256 weights; weight i of
 * half n = i/128 (cc = i%128, t = cc/32, l = cc%32) takes its low 4 bits
 * from ql[64n + l + 32*(t%2)] (low nibble if t < 2, else high) and its high
 * 2 bits from (qh[32n + l] >> 2t) & 3;  w = d * scales[i/16] * (q - 32).
 */
int qmatvec_q6_k(const void *w, int64_t row_offset, int64_t rows, int64_t K,
                 const float *x, int batch, float *y, int64_t ldy, qk_stream_t stream);

/*
 * Fused gate/up GEMV with the SwiGLU product, batch 1..8:
 *   g = sum_{c<K} W[gate_offset + p][c] * x[b*K + c]
 *   u = sum_{c<K} W[up_offset + p][c]   * x[b*K + c]
 *   h[b*ldh + p] = silu(g) * u,   silu(z) = z / (1 + e^-z),   for p < F.
 * The SwiGLU of the llama FFN (nurllama README, "What it runs") as silumul
 * g <- silu(g) * u (nurllama 0.18.1 API reference, kernels.nu `lk_silumul`),
 * folded into the matvec as loom's decode matvecs fuse it (loom-port-llm
 * SKILL.md, "Kernel inventory").  Gate and up rows may be row
 * ranges of one fused tensor (phi3's ffn_up: gate_offset 0, up_offset F;
 * nurllama README, "What it runs"), or of two tensors passed as one
 * allocation with the offsets between them.
 *   w            device block bytes holding both row ranges; alignment as the
 *                plain GEMV of the format (Q8_0 2 bytes, Q4_K 16 bytes).
 *   gate_offset, up_offset  first gate / up row (>= 0), in rows of K columns.
 *   x            device fp32 [batch][K];  h  device fp32 [batch][ldh], ldh == 0
 *                means ldh = F; only h[b*ldh + p] for p < F is written.
 * g and u are computed exactly as the plain GEMV's rows (each within the
 * plain GEMV's accuracy bound, see qmatvec_q8_0); silu uses CUDA's expf and its
 * fast division (within 2 ulp; a denominator past 2^126 gives a zero of z's
 * sign, the limit).  Errors: as the plain
 * GEMV; a negative up_offset is QK_ERR_BAD_DIM.
 */
int qmatvec_swiglu_q8_0(const void *w, int64_t gate_offset, int64_t up_offset, int64_t F, int64_t K,
                        const float *x, int batch, float *h, int64_t ldh, qk_stream_t stream);
int qmatvec_swiglu_q4_k(const void *w, int64_t gate_offset, int64_t up_offset, int64_t F, int64_t K,
                        const float *x, int batch, float *h, int64_t ldh, qk_stream_t stream);
int qmatvec_swiglu_q6_k(const void *w, int64_t gate_offset, int64_t up_offset, int64_t F, int64_t K,
                        const float *x, int batch, float *h, int64_t ldh, qk_stream_t stream);

/*
 * Batched expert GEMV over n_assign expert assignments:
 *   y[a*ldy + r] = sum_{c<K} W[expert_ids[a]*rows + r][c] * x[(a / xk)*K + c]
 * for a < n_assign and r < rows: nurllama's batched expert matvec, one call
 * for every assignment, output row a taken from expert expid_dev[a] with
 * input row a/xk (nurllama 0.18.1 API reference, kernels.nu
 * `lk_matvec_experts`); the experts of a projection live in one 3-D tensor
 * [n_experts][rows][K] evaluated as row ranges (nurllama README, "What it
 * runs", llada2).
 *   w           device block bytes of the whole expert tensor (alignment as
 *               the plain GEMV of the format).
 *   x           device fp32 [ceil(n_assign / xk)][K]; xk >= 1 assignments per
 *               input row (e.g. the experts chosen per token).
 *   expert_ids  device int32 [n_assign], 4-byte aligned; it may be written by
 *               the kernel just before this call on the same stream (the
 *               kernel reads it after the previous kernel completes).
 *   y           device fp32 [n_assign][ldy], ldy == 0 means ldy = rows.
 * An id outside [0, n_experts) is not dereferenced: that assignment's rows
 * are set to NaN and qk_device_error() reports QK_ERR_BAD_INDEX.  Error
 * bound as the plain GEMV at batch 1 (see qmatvec_q8_0).
 */
int qmatvec_experts_q8_0(const void *w, int64_t n_experts, int64_t rows, int64_t K, const float *x, int xk,
                         const int32_t *expert_ids, int64_t n_assign, float *y, int64_t ldy, qk_stream_t stream);
int qmatvec_experts_q4_k(const void *w, int64_t n_experts, int64_t rows, int64_t K, const float *x, int xk,
                         const int32_t *expert_ids, int64_t n_assign, float *y, int64_t ldy, qk_stream_t stream);
int qmatvec_experts_q6_k(const void *w, int64_t n_experts, int64_t rows, int64_t K, const float *x, int xk,
                         const int32_t *expert_ids, int64_t n_assign, float *y, int64_t ldy, qk_stream_t stream);

/*
 * Q4_K prefill GEMM on the tensor cores:
 *   y[m*ldy + n] = sum_{c<K} bf16(W[row_offset + n][c]) * bf16(x[m*K + c])
 * for m < M tokens and n < N weight rows, accumulated in fp32.  Each weight
 * is decoded to fp32 (w = d*sc*q - dmin*m) and rounded to bf16, each
 * activation is rounded to bf16 (round to nearest even).  This is the
 * batched (prefill) form of the matvec: the chunked prefill multiplies a
 * whole chunk of positions at once, so a chunk reads each weight only once
 * (nurllama 0.18.1 API reference, model.nu).
 *   w          device Q4_K block bytes of the whole tensor; 16-byte aligned.
 *   x          device fp32 [M][K], row stride K; 4-byte aligned.
 *   y          device fp32 [M][ldy]; writes y[m*ldy + n] for n < N only.
 *              ldy == 0 means ldy = N.
 *   workspace  device scratch of at least qgemm_q4_k_workspace_bytes(M, N, K)
 *              bytes, 256-byte aligned, owned by the caller (it receives the
 *              bf16 copy of x; its contents on return are unspecified).
 * Error bound: |y - exact| <= 1e-2 * sum|w*x| + 1e-6 per element (two bf16
 * roundings); the tests also check it against the bf16-rounded product.
 */
int qgemm_q4_k(const void *w, int64_t row_offset, int64_t N, int64_t K, const float *x, int64_t M,
               float *y, int64_t ldy, void *workspace, size_t workspace_bytes, qk_stream_t stream);

/*
 * Accumulating form of qgemm_q4_k: y[m*ldy + n] += sum_k bf16(W[row_offset+n][k]) * bf16(x[m*K + k]),
 * the acc mode of loom's prefill GEMMs (they come in store, acc and swiglu
 * modes: loom-port-llm SKILL.md, "What the starter generates", gen_gemm.py): the
 * product lands on what y holds (e.g. the residual stream).  Same arguments,
 * errors and bound as qgemm_q4_k, plus one fp32 rounding of the final add.
 */
int qgemm_q4_k_acc(const void *w, int64_t row_offset, int64_t N, int64_t K, const float *x, int64_t M,
                   float *y, int64_t ldy, void *workspace, size_t workspace_bytes, qk_stream_t stream);

/*
 * SwiGLU form of the prefill GEMM (loom's "swiglu" mode, same source): for
 * m < M and p < F
 *   g = sum_k bf16(W[gate_offset + p][k]) * bf16(x[m*K + k])
 *   u = sum_k bf16(W[up_offset + p][k])   * bf16(x[m*K + k])
 *   h[m*ldh + p] = silu(g) * u,   silu(z) = z / (1 + e^-z)  (CUDA expf, fast division as above),
 * g and u accumulated in fp32 on the tensor cores exactly as qgemm_q4_k's
 * outputs.  Gate and up are row ranges of one Q4_K tensor (or of one
 * allocation holding both); gate_offset, up_offset >= 0.  Workspace and
 * errors as qgemm_q4_k (ldh == 0 means ldh = F).
 */
int qgemm_swiglu_q4_k(const void *w, int64_t gate_offset, int64_t up_offset, int64_t F, int64_t K, const float *x,
                      int64_t M, float *h, int64_t ldh, void *workspace, size_t workspace_bytes, qk_stream_t stream);

/*
 * Q8_0 forms of the prefill GEMM (loom's prefill GEMM formats include q8_0,
 * loom-port-llm SKILL.md, "What the starter generates", gen_gemm.py): the same
 * three modes with Q8_0 weights (w = d*q, rounded to bf16), w 2-byte aligned
 * (34-byte blocks); arguments, workspace, errors and bounds as the Q4_K forms.
 */
int qgemm_q8_0(const void *w, int64_t row_offset, int64_t N, int64_t K, const float *x, int64_t M,
               float *y, int64_t ldy, void *workspace, size_t workspace_bytes, qk_stream_t stream);
int qgemm_q8_0_acc(const void *w, int64_t row_offset, int64_t N, int64_t K, const float *x, int64_t M,
                   float *y, int64_t ldy, void *workspace, size_t workspace_bytes, qk_stream_t stream);
int qgemm_swiglu_q8_0(const void *w, int64_t gate_offset, int64_t up_offset, int64_t F, int64_t K, const float *x,
                      int64_t M, float *h, int64_t ldh, void *workspace, size_t workspace_bytes, qk_stream_t stream);

/* Workspace bytes the prefill GEMMs need for M tokens and K columns (N unused). */
size_t qgemm_q4_k_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * qgemm_q4_k for callers that cannot allocate device memory -- for example a
 * plugin inside an inference engine that owns every device allocation, or
 * code that must not allocate once running -- and so cannot pass the
 * workspace qgemm_q4_k needs.  The pages have no counterpart of this call;
 * it exists for such callers only.
 * Same operation, arguments and results as qgemm_q4_k, without the
 * workspace: the scratch is a fixed array of QK_NOALLOC_SCRATCH_BYTES inside
 * the library, held by every GPU that loads the library until the process
 * exits.  No call allocates or frees memory.
 *   Sizes: M * round_up(K, 8) * 2 + 256 must not exceed
 *   QK_NOALLOC_SCRATCH_BYTES, else QK_ERR_TOO_LARGE (before any launch).
 *   The first call on a device looks up the array's device address; make
 *   it before any stream capture.
 *   All calls share the array: calls that overlap on the GPU (for example on
 *   two streams at once) race on it and give undefined results.
 */
#define QK_NOALLOC_SCRATCH_BYTES (8u << 20)
int qgemm_q4_k_noalloc(const void *w, int64_t row_offset, int64_t N, int64_t K, const float *x, int64_t M,
                       float *y, int64_t ldy, qk_stream_t stream);

/* ------------------------------------------------------------------------
 * Attention operators: what a decode step or a prompt chunk does between its
 * QKV product and its output product (the rope and attention steps of the
 * decode loop, nurllama 0.18.1 API reference, kernels.nu `lk_rope`,
 * `lk_attn`; QK-norm, rotation and cache store in one kernel and split
 * decode attention, loom-port-llm SKILL.md, "Kernel inventory").  The
 * key/value cache is held in 4 bits.
 *
 * Rotation table: fp32 [n_pos][rot/2][2], (cos, sin) of each position's
 * angles; qk_rope_table fills one.  rot (even, <= head_dim) channels at the
 * start of a head rotate, the others pass.  Pair i of a head is channels
 * (i, i + rot/2), or (2i, 2i + 1) with interleaved != 0 (the two layouts of
 * nurllama's `rope_neox` and `rope`), and (a, b) becomes
 * (a*cos - b*sin, a*sin + b*cos).  rot == 0: no rotation (table may be NULL).
 *
 * Norm: n_j = x_j * weight_j / sqrt(mean_j(x_j^2) + eps) over a head's
 * channels, before the rotation; weight NULL: no norm.
 *
 * The arithmetic is fp32 whatever the element types, with one rounding to
 * the output's type.
 */

/*
 * Fills table[p][i] = amplitude * (cos, sin)(p * f_i) for p < n_pos,
 * i < rot/2.  f_i is the angle of one position:
 *   e_i = base^(-2i/rot) / freq_factors[i]   (freq_factors NULL: 1)
 *   f_i = e_i * freq_scale                   where orig_ctx == 0, else
 *   f_i = e_i * (freq_scale * (1 - m_i) + m_i),
 *   m_i = 1 - clamp((i - lo) / max(hi - lo, 0.001), 0, 1),
 *   lo = max(0, floor(dim(beta_fast))), hi = min(rot - 1, ceil(dim(beta_slow))),
 *   dim(t) = rot * ln(orig_ctx / (2*pi*t)) / (2 * ln(base)):
 * position interpolation (freq_scale = 1/s), per-frequency factors (the
 * rope_freqs tensor of GGUF files) and the ramp between interpolated and
 * kept frequencies of Peng et al., "YaRN", 2023 (its attention temperature
 * goes into `amplitude`).  Angles are formed and reduced in 64 bits, so a
 * table of any length is within 4e-7 * amplitude of the exact values.
 *   table         device, 8-byte aligned; freq_factors device fp32 [rot/2] or NULL.
 * QK_ERR_BAD_DIM: n_pos or rot <= 0, rot odd, base <= 1, freq_scale <= 0,
 * orig_ctx < 0, or (with orig_ctx > 0) a beta <= 0.
 */
int qk_rope_table(float *table, int64_t n_pos, int rot, double base, double freq_scale, const float *freq_factors,
                  int64_t orig_ctx, double beta_fast, double beta_slow, double amplitude, qk_stream_t stream);

/*
 * Norm and rotation of T rows of n_q_heads query heads followed by n_k_heads
 * key heads of head_dim channels (as the QKV product writes them), in one
 * pass: query heads use q_weight, key heads k_weight.
 *   x, y        device, element types x_type / y_type, aligned to their
 *               element; rows ldx / ldy elements apart (0: heads * head_dim).
 *               y may be x (with the same stride and type).
 *   head_dim    even, 2..512;  n_q_heads + n_k_heads >= 1.
 *   weights     device fp32 [head_dim], 4-byte aligned, or NULL.
 *   positions   device int32 [T]; the rows of a token whose position is
 *               outside [0, n_pos) become NaN and qk_device_error() reports
 *               QK_ERR_BAD_INDEX.  Not read when rot == 0 (may be NULL).
 * T == 0 is a call that does nothing.
 */
int qk_norm_rope(const void *x, int64_t ldx, int x_type, int n_q_heads, int n_k_heads, int head_dim,
                 const float *q_weight, const float *k_weight, float eps, const float *table, int64_t n_pos, int rot,
                 int interleaved, const int32_t *positions, int64_t T, void *y, int64_t ldy, int y_type,
                 qk_stream_t stream);

/*
 * A paged key/value cache in 4 bits, owned by the caller.  The device buffer
 * is [n_pages][n_kv_heads][page_tokens / 16] blocks of 18 * head_dim bytes,
 * 16-byte aligned: QK_KV_Q4_BYTES in all.  Slot s is token s % page_tokens
 * of page s / page_tokens.
 *   head_dim     64, 96, 128 or 256;  page_tokens a multiple of 16, 16..1024.
 * A value is d * (n - 8): the scale d is fp16(m / -8), m the value of largest
 * magnitude of 32 neighbouring channels (the positive one of a tie; |d| is
 * held to 65504), and the nibble n = clamp(floor(x / d + 8.5), 0, 15), 8
 * where d is 0: in fp32, the quotient and the sum each rounded, wherever the
 * rows lie.  A group that holds a NaN or an infinity gets a NaN scale.
 *
 * Block (16 tokens of one head; G = head_dim/32 scale groups, Gp = 4 where G
 * is a multiple of 4 and else G):
 *   key nibbles    [G/Gp][row 16][c 4][Gp] 32-bit words: nibble i of a word is
 *                  channel 32*group + 8*c + i; row 8h + 2a + b is token 4a + 2h + b
 *   value nibbles  [G/Gp][u 2][r 8][c 4][Gp] 32-bit words: nibble 4b + j of a
 *                  word is channel 32*group + 4*r + j of token 4c + 2u + b
 *   key scales     [token 16][G] fp16;   value scales [token 16][G] fp16
 * so that the words a thread reads are the operand fragments of the tensor
 * cores' products over the block.
 */
typedef struct {
    void *pages;
    int64_t n_pages;
    int n_kv_heads, head_dim, page_tokens;
} qk_kv_cache_q4;
#define QK_KV_Q4_BYTES(n_pages, n_kv_heads, page_tokens, head_dim) \
    ((int64_t)(n_pages) * (n_kv_heads) * ((page_tokens) / 16) * 18 * (head_dim))

/*
 * Norm and rotation of T tokens' queries and keys as qk_norm_rope, with the
 * keys and values stored into the cache: token t goes to slots[t].
 *   q, k, v     device rows of n_q_heads, cache->n_kv_heads and
 *               cache->n_kv_heads heads, all of element type `type`, ldq, ldk,
 *               ldv elements apart (0: packed); q may be NULL (then q_out is
 *               not written).
 *   slots       device int64 [T], 8-byte aligned.  A negative slot stores
 *               nothing (a padded token; its q_out row is written).  A slot
 *               beyond the cache stores nothing and reports QK_ERR_BAD_INDEX.
 *               Two tokens of a call in one slot: either may be left there.
 *   positions   as qk_norm_rope; a bad one makes the token's q_out NaN and
 *               its stored key NaN.
 *   q_out       device rows of n_q_heads heads of type q_out_type; may be q
 *               (with the same stride and type).
 */
int qk_kv_append_q4(const qk_kv_cache_q4 *cache, const void *q, int64_t ldq, int n_q_heads, const void *k, int64_t ldk,
                    const void *v, int64_t ldv, int type, const float *q_weight, const float *k_weight, float eps,
                    const float *table, int64_t n_pos, int rot, int interleaved, const int32_t *positions,
                    const int64_t *slots, int64_t T, void *q_out, int64_t ldqo, int q_out_type, qk_stream_t stream);

/*
 * Reads slots back as values: k[t], v[t] (rows of n_kv_heads heads of type
 * `type`, ldk / ldv elements apart, 0: packed) are what the cache holds at
 * slots[t]; k or v may be NULL.  Rows of a negative slot become 0, of a slot
 * beyond the cache NaN (QK_ERR_BAD_INDEX from qk_device_error()).
 */
int qk_kv_read_q4(const qk_kv_cache_q4 *cache, const int64_t *slots, int64_t T, void *k, int64_t ldk, void *v,
                  int64_t ldv, int type, qk_stream_t stream);

/*
 * Attention of T query rows over the cache, grouped heads (query head h
 * reads key/value head h / (n_q_heads / n_kv_heads)):
 *   out[t][h] = sum_j p_j * V_j,  p = softmax_j(scale * q[t][h] . K_j)
 * over the keys j of the row's sequence with j <= pos, j < lens[b] and, with
 * window > 0, j > pos - window; pos = lens[b] - n_b + i for query i of the
 * sequence's n_b.  A row that sees no key is 0.
 *   q, out      device rows of n_q_heads heads, ldq / ldo elements apart (0:
 *               packed), element types q_type / out_type.
 *   page_table  device int32 [B][ld_pages]: page page_table[b][j / page_tokens]
 *               holds key j; max_pages (<= ld_pages; 0: ld_pages) entries a
 *               row are readable, those past a sequence's length are not read.
 *   lens        device int32 [B], the sequences' lengths, the new tokens'
 *               keys among them; 0 is a sequence with no keys.
 *   q_start     device int32 [B + 1]: sequence b's queries are rows
 *               [q_start[b], q_start[b+1]), at most max_q of them.  NULL: each
 *               has max_q, and T == B * max_q.
 *   max_len     an upper bound of lens that the call's split of the keys is
 *               sized by (0: max_pages * page_tokens).  Longer sequences are
 *               computed all the same.
 *   scale       finite.
 *   workspace   NULL, or device scratch, 256-byte aligned, that was filled
 *               with zeros once before its first use; every call leaves its
 *               counters zero again.  Calls that may overlap on the GPU need
 *               one each.  With one, the keys of long sequences are split
 *               over more thread blocks, as far as workspace_bytes allow;
 *               qk_attn_q4_workspace_bytes() gives what the call can use.
 * A page outside [0, n_pages), a length above max_pages * page_tokens or
 * below 0, or a q_start out of order, beyond T or with more than max_q rows
 * reports QK_ERR_BAD_INDEX from qk_device_error() without any access out of
 * range.  A bad page makes the sequence's rows that see its keys NaN (and
 * may make its other rows NaN); a bad length or q_start makes every row of
 * the sequence NaN, as far as q_start names rows inside [0, T).
 * A group of 32 values whose scale is not finite makes its channels NaN in
 * the rows that see the key, and in chunks (below) those rows whole.
 * Rows of out that no sequence has (before q_start[0], from q_start[B] on)
 * are not written.
 * Accuracy: sums and the softmax are fp32 whatever the types.  With fp32
 * queries every product is formed from the exact 4-bit values, 22-bit
 * probabilities, and queries of 22 bits below the row's largest channel; with
 * fp16 queries in chunks (more than 32 rows a sequence and key/value head,
 * head_dim <= 128) likewise, the queries exact.  Else with 16-bit queries the
 * probabilities are rounded to fp16 (2^-11), and in bf16 chunks the cache's
 * values too.  The scales of a head's groups and tokens may differ by 2^20
 * without loss.
 * T == 0 or B == 0 is a call that does nothing.
 */
int qk_attn_q4(const qk_kv_cache_q4 *cache, const void *q, int64_t ldq, int q_type, int n_q_heads,
               const int32_t *page_table, int64_t ld_pages, int64_t max_pages, const int32_t *lens,
               const int32_t *q_start, int64_t B, int64_t T, int64_t max_q, int64_t max_len, float scale,
               int64_t window, void *out, int64_t ldo, int out_type, void *workspace, size_t workspace_bytes,
               qk_stream_t stream);

/* Workspace bytes that a qk_attn_q4 call of these sizes can make use of; max_len 0: of any length. */
size_t qk_attn_q4_workspace_bytes(int64_t B, int n_q_heads, int n_kv_heads, int head_dim, int64_t max_q,
                                  int64_t max_len);

/* ------------------------------------------------------------------------
 * Beside the products: routing to experts and the experts' feed-forward
 * products (nurllama 0.18.1 API reference, kernels.nu `moe_route`,
 * `moe_scatter`; loom-port-llm SKILL.md, gen_moe.py), and low-rank adapters
 * (its LoRA fine-tunes).  Sums are fp32 whatever the element types, with one
 * rounding to the output's type.
 */

/* Expert scores of a token's logits z: softmax(z) over all experts, or 1 / (1 + e^-z) of each. */
typedef enum { QK_SOFTMAX = 0, QK_SIGMOID = 1 } qk_score;

/*
 * Routing of T tokens: ids[t][j], weights[t][j] for j < top_k.
 *   p = the scores;  c = p + bias (bias device fp32 [n_experts], or NULL: p).
 *   Groups: the experts are n_groups runs of n_experts / n_groups; a group
 *   counts as the sum of its group_top (1 or 2) largest c, and the top_groups
 *   best groups stay (top_groups == n_groups: all).
 *   ids: the top_k experts of largest c in them, largest first.  The lower
 *   index wins a tie, of groups too.
 *   weights: p[ids], over their sum with renorm != 0, times scale.
 * The choice is that of the exact formulas: neighbours that 32-bit scores
 * leave undecided are compared in 64 bits; without a bias (and with
 * group_top 1, where groups count) the logits are compared.  Weights are
 * within 1.2e-6 of themselves, or 2^-126 times scale.
 * A logit of -infinity has score 0.  A token none of whose chosen experts has
 * a score gets weights of 0.  A token with a NaN among its logits or the
 * biases, or (softmax) a logit of +infinity, gets ids 0..top_k-1 and NaN
 * weights.
 *   logits      device rows of n_experts elements of `type`, ld apart (0: packed).
 *   ids, weights  device int32 and fp32 [T][top_k].
 * n_experts <= 1024, top_k <= 32, n_groups <= 32 (else QK_ERR_TOO_LARGE);
 * top_k <= top_groups * n_experts / n_groups.  T == 0 does nothing.
 */
int qk_moe_route(const void *logits, int64_t ld, int type, int64_t T, int n_experts, int top_k, int score,
                 const float *bias, int n_groups, int top_groups, int group_top, int renorm, float scale, int32_t *ids,
                 float *weights, qk_stream_t stream);

/* Block formats of expert tensors. */
typedef enum { QK_Q8_0 = 0, QK_Q4_K = 1, QK_Q6_K = 2 } qk_format;

/*
 * The experts' rows of one projection: expert e's row r is row
 * row_offset + e * expert_rows + r of w (expert_rows 0: the call's row
 * count).  A 3-D expert tensor has row_offset 0 and expert_rows 0; the halves
 * of a fused gate-and-up tensor [E][2F][K] have row_offset 0 and F, and
 * expert_rows 2F.  w's alignment as the format's GEMV.
 */
typedef struct {
    const void *w;
    int format;
    int64_t row_offset, expert_rows;
} qk_expert_weights;

/*
 * The experts' feed-forward products of T tokens:
 *   y[t] = sum_{j < top_k} weights[t][j] * down_e h,
 *   h = silu(gate_e x[t]) * (up_e x[t]),   e = ids[t][j],
 * gate and up [F][K] (one format), down [N][F].  An expert's weights are
 * read once for up to 128 of its tokens, or for 16 where the batch has few such
 * experts; for each of its tokens where a call has 24 assignments or fewer and
 * K and F are 8192 at most.  ids may be in any order and repeat; a negative id
 * adds nothing (a token with none left gets 0).  An id past the last makes the
 * token's row NaN and qk_device_error() reports QK_ERR_BAD_INDEX.
 *   x, y        device rows of K and N elements of x_type / y_type, ldx / ldy
 *               apart (0: packed), aligned to their element.  y may overlap x,
 *               whose rows are all read before one of y is written, and nothing
 *               else.
 *   ids, weights  device int32 and fp32 [T][top_k].
 *   workspace   device scratch, 256-byte aligned, of at least
 *               qk_moe_ffn_workspace_bytes() bytes; its contents need not be
 *               kept or set.  Calls that may overlap need one each.
 * Accuracy: sums are fp32 (Q4_K's two each, of scales times quants and of
 * minima).  Activations (x, and h) are held to 2^-22 of themselves or 2^-39 of
 * their row's largest with fp32 x or y; else to 2^-11 or 2^-39 (one fp16 below a
 * power of two of the row's own, so bf16 values are exact above 2^-28 of it); in
 * calls of up to 24 assignments (as above) in fp32, whatever the types, to
 * 2^-138.  Weights are exact in calls of fewer than 16 tokens.  In others those
 * of an expert with 16 tokens or more, and of any other where the counts of the
 * whole batch make it cheaper, are held to 2^-22 of themselves and 2^-24 of what
 * they are made of (scale times quant, and minimum), or 2^-29 of the largest that
 * their row's scales allow; with bf16 x and y to 2^-11 of themselves and of what
 * they are made of, or that 2^-29.  A token's low bits can so differ with the
 * batch it is in.
 * A NaN or an infinity in a row of x makes that token's y not finite, and no other's.
 * n_experts <= 1024; K, F, N <= 2^24; T * top_k <= 2^28.  T == 0 does nothing.
 */
int qk_moe_ffn(const qk_expert_weights *gate, const qk_expert_weights *up, const qk_expert_weights *down,
               int64_t n_experts, int64_t K, int64_t F, int64_t N, const void *x, int64_t ldx, int x_type, int64_t T,
               const int32_t *ids, const float *weights, int top_k, void *y, int64_t ldy, int y_type, void *workspace,
               size_t workspace_bytes, qk_stream_t stream);

/* Workspace bytes of qk_moe_ffn calls of up to these sizes, whatever the formats and types (0: no call has them). */
size_t qk_moe_ffn_workspace_bytes(int64_t T, int top_k, int64_t n_experts, int64_t K, int64_t F, int64_t N);

/*
 * Low-rank adapters beside a projection's output y:
 *   out[t] = y[t] + scales[a] * B[a] (A[a] x[t]),   a = ids[t].
 *   x           device rows of K elements of x_type, ldx apart (0: packed).
 *   A, B        device [n_adapters][rank][K] and [n_adapters][N][rank] of
 *               w_type; a smaller adapter is padded with zero ranks.
 *   ids         device int32 [T]; a negative id: out[t] = y[t].  One past the
 *               last makes the row NaN (QK_ERR_BAD_INDEX from qk_device_error()).
 *   scales      device fp32 [n_adapters], or NULL: 1.
 *   y, out      device rows of N elements of y_type, ldy / ldo apart (0:
 *               packed); out may be y (with the same stride, if there is more
 *               than one row) and must not overlap x.
 * Tokens of one adapter may lie anywhere; neighbouring ones share its reads.
 * Both products are fp32 sums of operands that are exact in 16 bits and held
 * to 22 bits in fp32.  So is A x in between, but to 2^-17 of itself with bf16
 * adapters and outputs.
 *   workspace   NULL, or device scratch, 256-byte aligned, whose contents need
 *               not be kept or set; calls that may overlap need one each.
 *               With qk_lora_workspace_bytes() of it, calls of many tokens,
 *               of 16-bit operands or of high ranks take two launches instead
 *               of one, which is faster.
 * rank <= 256; K, N <= 2^24; T <= 2^26.  T == 0 does nothing.
 */
int qk_lora(const void *x, int64_t ldx, int x_type, int64_t T, int64_t K, const void *A, const void *B, int w_type,
            int64_t n_adapters, int rank, int64_t N, const int32_t *ids, const float *scales, const void *y,
            int64_t ldy, void *out, int64_t ldo, int y_type, void *workspace, size_t workspace_bytes,
            qk_stream_t stream);

/* Workspace bytes that a qk_lora call of T tokens can make use of (0: none). */
size_t qk_lora_workspace_bytes(int64_t T, int rank);

/*
 * Bytes of one row of a tensor with K columns: ceil(K/32)*34 (Q8_0),
 * ceil(K/256)*144 (Q4_K) or ceil(K/256)*210 (Q6_K).
 */
int64_t qk_row_bytes_q8_0(int64_t K);
int64_t qk_row_bytes_q4_k(int64_t K);
int64_t qk_row_bytes_q6_k(int64_t K);

/* Human-readable name of a status code (static string, never NULL). */
const char *qk_status_string(int status);

/*
 * Reads and clears the device error word of the current device after
 * synchronising `stream`: QK_OK, QK_ERR_TIMEOUT (a bounded wait ran out),
 * QK_ERR_BAD_INDEX (an expert id was out of range) or QK_ERR_CUDA (the
 * synchronisation itself failed).  Meant for tests and
 * debugging; the compute calls never synchronise.
 */
int qk_device_error(qk_stream_t stream);

/*
 * Upper bound, in nanoseconds, of every device-side wait of later launches
 * (default 2e9).  Returns the previous value.  Tests shorten it.
 */
uint64_t qk_set_wait_limit_ns(uint64_t ns);

/*
 * Programmatic dependent launch for later calls (default off; returns the
 * previous setting).  When on, a call may be scheduled while the kernel just
 * before it in the stream is still running: it starts streaming its weights
 * at once and waits for that kernel (griddepcontrol.wait) only before it
 * reads x and writes y.  So the weights of a call must not be written by
 * the kernel directly before it in the stream; x and y keep full stream
 * order.  Meant for decode loops whose weights are loaded once.
 */
int qk_set_programmatic_launch(int enable);

/*
 * Strict-blocks mode for later calls (returns the previous setting).  Off by
 * default, where any K >= 1 is accepted and a row's last block may be
 * partly used; on, every compute call whose K is not a multiple of its
 * format's block (32 columns for Q8_0, 256 for Q4_K and Q6_K) returns
 * QK_ERR_BAD_DIM before any launch.  The library starts with it on when the
 * environment holds QK_STRICT=1 at load time.  A GGUF row always holds whole
 * blocks (nurllama README, "What it runs"); the mode is for callers that want
 * such shapes rejected rather than read with an unused tail.
 */
int qk_set_strict_blocks(int enable);

/* Library version, major*10000 + minor*100 + patch. */
int qk_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QK_H */
