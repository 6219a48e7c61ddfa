/*
 * bi.h - batch-invariant verify pass for GB300 (sm_103a), C ABI.
 *
 * The library computes the linear layers of an LLM decode or speculative
 * verify pass (M = 1 .. K+1 tokens against a large int8 weight matrix) so that
 * every output row is bitwise identical whatever M is and whatever else shares
 * the pass; with them the LM-head argmax, greedy verification, a block-scaled
 * variant of the linear and the verify queries' split-KV attention, each with
 * the same guarantee.  Greedy speculative decoding then keeps exactly the target's own
 * argmax ("why speculative decoding changed my output", introduction: the
 * guarantee needs a position's logits inside a batch to equal its logits
 * decoded alone).
 *
 * Arithmetic (W8A8 as in "Deterministic LLM Inference Across GPU Kernels:
 * Power-of-Two INT8 Quantization Scales and the Limits of Tolerance-Based
 * Conformance", Abstract, Fig. 1, Table II):
 *   s_a[m]   = absmax_k |x[m,k]| / 127  (IEEE fp32 division; 1 if absmax = 0)
 *   q[m,k]   = clamp(rne(x[m,k] / s_a[m]), -127, 127)
 *   acc[m,n] = sum_k q[m,k] * W[n,k]       exact in int32 (K * 127^2 < 2^31)
 *   y[m,n]   = bf16_rne((float(acc) * s_a[m]) * s_w[n])
 * The integer sum is exact and independent of summation order ("The Integer
 * Alibi", abstract), so the kernels may split K in any way; the epilogue is
 * fixed element by element.  Hence rows do not depend on M.
 *
 * Conventions for every entry point:
 *  - Pointers are DEVICE pointers, allocated and owned by the caller; the
 *    library allocates nothing and keeps no pointer after returning.
 *  - bf16 values are passed as their uint16_t bit patterns.
 *  - Matrices are row-major: x [M, ldx] (ldx >= K), q [M, K], W [N, K]
 *    (K contiguous), y / logits [M, N].
 *  - Work is enqueued on `stream` (NULL = legacy default stream) and the call
 *    returns without waiting.  Calls are reentrant; calls that may run
 *    concurrently on the device must not share output or workspace buffers.
 *  - Arguments are validated on the host before anything is launched; an
 *    invalid call returns an error status and enqueues nothing.  No call
 *    aborts, throws, or writes to stderr.
 *  - Shape limits: 1 <= M <= 65535, 1 <= N <= 2^31-1, 16 <= K, K % 16 == 0,
 *    K * 127^2 < 2^31 (K <= 133144).  Base pointers of x, q and w_q must be
 *    16-byte aligned, and ldx % 8 == 0 (16-byte aligned rows).
 */
#ifndef BI_H
#define BI_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define BI_API __attribute__((visibility("default")))
#else
#define BI_API
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st *bi_stream_t;

typedef enum {
    BI_OK = 0,
    BI_ERR_INVALID_ARG = 1, /* null pointer, bad shape, ldx < K, K % 16 != 0 */
    BI_ERR_ALIGNMENT = 2,   /* a base pointer or row stride not 16-byte aligned */
    BI_ERR_INT32_BOUND = 3, /* K * 127^2 >= 2^31: the int32 sum could overflow */
    BI_ERR_WORKSPACE = 4,   /* workspace null or smaller than the queried size */
    BI_ERR_UNSUPPORTED = 5, /* no usable sm_103a device, or a feature missing */
    BI_ERR_TIMEOUT = 6,     /* a kernel gave up a bounded wait (see bi_workspace_status) */
    BI_ERR_CUDA = 7         /* a CUDA runtime/driver call failed */
} bi_status;

/* Flags for the calls that take `flags`. */
enum {
    /* Programmatic dependent launch.  The call may begin while the kernel
     * that precedes it on `stream` is still running: it waits for that kernel
     * before reading any of its inputs except the weight codes w_q, which it
     * may start streaming early, and it lets the next kernel on the stream
     * launch early in the same way.  Use it only when w_q is not written by
     * the immediately preceding kernel (weights are constants of the model).
     * Results are bitwise identical with and without the flag. */
    BI_FLAG_PDL = 1u
};

/* Human-readable name of a status (static string, never NULL). */
BI_API const char *bi_status_string(bi_status s);

/*
 * Per-token activation quantisation.
 *   x    bf16 [M, ldx], first K columns used (read only)
 *   q    int8 [M, K] out, s_a fp32 [M] out
 * s_a[m] = absmax/127 by IEEE division (1 for an all-zero row); q by IEEE
 * division x/s_a, round-to-nearest-even, clamp to [-127, 127].  Subnormal
 * inputs are honoured (no flush to zero).  With BI_FLAG_PDL the kernel waits
 * for the preceding kernel before reading x.
 */
BI_API bi_status bi_quantize_act(const uint16_t *x, int64_t ldx, int M, int K,
                          int8_t *q, float *s_a, unsigned flags, bi_stream_t stream);

/*
 * Chained verify pass: the two elementwise steps between a layer's linears,
 * each fused with the activation quantisation of the linear that reads it.
 * A decode/verify pass chains its linears through the residual stream ("why
 * speculative decoding changed my output", "the mat-vec kernel"; "My
 * speculative decoder got slower", "The physics"); the pages print no layer
 * body, so the steps are this library's reading, both exact roundings of
 * fp32 operations on bf16 values (fp32 has enough bits that an fp32 add or
 * multiply of two bf16 values, then bf16 rounding, equals one rounding of
 * the exact result):
 *
 * bi_residual_quantize: the residual update after the o and down projections.
 *   h    bf16 [M, K] (row stride K), read and written in place
 *   y    bf16 [M, ldy], first K columns added (read only; must not overlap h)
 *   h'   = bf16_rne(h + y)  (fp32 add);  e = floor(log2 max_k |h'[m, k]|),
 *          0 for an all-zero row;  h = bf16_rne(h' * 2^-e)
 *   q, s_a = bi_quantize_act of the new h (the power-of-two rescale keeps a
 *          deep stack finite and changes no code: per-row absmax quantisation
 *          is exactly invariant to scaling a row by a power of two)
 *
 * bi_relu_mul_quantize: the gated MLP product feeding the down projection.
 *   gu   bf16 [M, ldgu] (ldgu >= 2K): gate g = gu[:, 0:K], up u = gu[:, K:2K]
 *        (the output of one packed gate/up linear), read only
 *   m    = bf16_rne(relu(g) * u), relu(g) = g if g > 0 else +0 (fp32 multiply)
 *   q, s_a = bi_quantize_act of m;  m_out bf16 [M, K] (row stride K) receives
 *          m unless it is NULL (it must not overlap gu)
 *
 * Both: 16-byte aligned h, y, gu, m_out and q; row strides multiples of 8
 * elements; K % 16 == 0.  One CTA per row; with BI_FLAG_PDL the kernel waits
 * for the preceding kernel before reading.
 */
BI_API bi_status bi_residual_quantize(uint16_t *h, const uint16_t *y, int64_t ldy, int M, int K,
                                      int8_t *q, float *s_a, unsigned flags, bi_stream_t stream);
BI_API bi_status bi_relu_mul_quantize(const uint16_t *gu, int64_t ldgu, int M, int K, int8_t *q, float *s_a,
                                      uint16_t *m_out, unsigned flags, bi_stream_t stream);

/*
 * Checkpoint-style per-output-channel weight quantisation (offline, not part
 * of the verify pass): the same rule as bi_quantize_act applied to each row of
 * an fp32 matrix.
 *   w    fp32 [N, ldw] (ldw >= K, ldw % 4 == 0, 16-byte aligned), read only
 *   w_q  int8 [N, K] out, s_w fp32 [N] out
 */
BI_API bi_status bi_quantize_weight(const float *w, int64_t ldw, int N, int K,
                             int8_t *w_q, float *s_w, bi_stream_t stream);

/*
 * Power-of-two scale requantisation ("Deterministic LLM Inference ...",
 * Abstract and Fig. 1: every weight scale is moved to its nearest power of
 * two and the codes are requantised to it, not merely relabelled).
 *   s'   = 2^round(log2 s_w[n])   (nearest in the log domain; never a tie)
 *   w_q' = clamp(rne(w_q * s_w[n] / s'), -127, 127), computed exactly
 * A scale whose power of two would exceed fp32 is held at 2^127; rows whose
 * scale is not a positive finite number are copied unchanged.  Outputs may
 * alias the inputs exactly (w_q_out == w_q, s_w_out == s_w) for an in-place
 * update; partial overlap is not allowed.
 */
BI_API bi_status bi_requant_pow2(const int8_t *w_q, const float *s_w, int N, int K,
                          int8_t *w_q_out, float *s_w_out, bi_stream_t stream);

/*
 * Workspace bytes needed by bi_linear_w8a8 for this shape (> 0).  The
 * workspace holds split-K partial sums, their counters and a status word.  It
 * must be zero-filled before its first use (cudaMemset); every call that
 * completes leaves it zero-filled again, so one workspace can serve a whole
 * sequence of calls on one stream.  For M > 16 it is larger: about 12.6 MB
 * for the int32 partial sums of prefill tiles split along K to fill the GPU's
 * last wave (scratch: every call overwrites what it reads) and their counters
 * (zero between calls).  For M > 256 it also holds 2 * (M + N) * K bytes
 * (each part rounded up to 256) for exact f16 copies of q and w_q that the
 * tensor cores read by TMA (scratch).  A smaller workspace still works for
 * M > 16, with the same results: without the f16 room the kernel converts
 * the codes in its tile loop (slower above 256 tokens), and with only the
 * M <= 16 size it also runs without the split.
 */
BI_API size_t bi_linear_workspace_size(int M, int N, int K);

/*
 * y = the W8A8 linear layer above.
 *   q    int8 [M, K], s_a fp32 [M]          (from bi_quantize_act)
 *   w_q  int8 [N, K], s_w fp32 [N]          (per-output-channel codes/scales)
 *   y    bf16 [M, N] out (row stride N)
 *   ws   workspace of ws_bytes >= bi_linear_workspace_size(M, N, K)
 * M <= 16 runs the weight-streaming kernel (TMA-staged int8 weight tiles,
 * int8 tensor-core dot products, int32 partial sums reduced exactly across
 * CTAs); larger M runs the tiled prefill kernel.  Both give the same bits for
 * every row.  Any outputs that do not fit bf16 become +-Inf by round to
 * nearest even.
 */
BI_API bi_status bi_linear_w8a8(const int8_t *q, const float *s_a, int M, int K,
                         const int8_t *w_q, const float *s_w, int N,
                         uint16_t *y, void *ws, size_t ws_bytes,
                         unsigned flags, bi_stream_t stream);

/* Workspace bytes needed by bi_lmhead_argmax (same zero-fill rule). */
BI_API size_t bi_lmhead_workspace_size(int M, int N, int K);

/*
 * Greedy LM head: the logits of bi_linear_w8a8 (optionally written to
 * `logits`, bf16 [M, N]) and, per row, argmax[m] = the lowest n whose bf16
 * logit is the row maximum, logits compared as real numbers (-0 == +0).
 * ("My speculative decoder got slower", "We're nowhere near SOL": a head that
 * computes only the winning token; "Why the decoders disagreed?": bf16 logits
 * do tie.)  M <= 16.
 *   logits  bf16 [M, N] out, or NULL to skip writing them
 *   argmax  int32 [M] out
 */
BI_API bi_status bi_lmhead_argmax(const int8_t *q, const float *s_a, int M, int K,
                           const int8_t *w_q, const float *s_w, int N,
                           uint16_t *logits, int32_t *argmax,
                           void *ws, size_t ws_bytes, unsigned flags, bi_stream_t stream);

/*
 * Device-side status of a workspace: waits for `stream`, reads the status word
 * that kernels set when a bounded wait gives up, clears it, and returns BI_OK
 * or BI_ERR_TIMEOUT (or BI_ERR_CUDA if the stream itself reports an error).
 * After BI_ERR_TIMEOUT the workspace must be zero-filled again before reuse.
 * For workspaces of linear calls, programs and bi_attention_kv4.
 */
BI_API bi_status bi_workspace_status(void *ws, size_t ws_bytes, bi_stream_t stream);

/*
 * Greedy verification of a verify pass, the step after the LM head.  Greedy
 * speculative decoding keeps exactly the tokens plain greedy decoding would
 * produce ("why speculative decoding changed my output", introduction; "My
 * speculative decoder got slower", "Speculative decoding (SD)").  The pass
 * ran the target on the last accepted token followed by the drafted tokens
 * d_1 .. d_{M-1}; argmax[i] is the target's choice after input i.
 *   argmax int32 [M] (from bi_lmhead_argmax), draft int32 [M - 1] (NULL when
 *   M == 1), out int32 [2] receives L = the length of the longest prefix with
 *   argmax[i] == draft[i], and argmax[L] (the correction, or the bonus token
 *   when all M - 1 drafts are accepted).  Device pointers, 4-byte aligned.
 * One warp; M <= 65535.  In a program, the same result is produced by an
 * LM-head op whose `draft` and `accept` fields are set, in the CTA that
 * finishes the argmax.
 */
BI_API bi_status bi_greedy_verify(const int32_t *argmax, const int32_t *draft, int M, int32_t *out,
                                  bi_stream_t stream);

/*
 * Test of the failure path: launches one thread that waits, with the same
 * bounded wait the kernels use, on a barrier phase that nothing completes.
 * After the wait limit (2 s of GPU time) it gives up and sets the status
 * word of `ws` (a linear workspace, >= bi_linear_workspace_size(1, 1, 16)
 * bytes), so that bi_workspace_status then returns BI_ERR_TIMEOUT.  With
 * ws = NULL (ws_bytes ignored) the status word is that of the fixed scratch
 * of bi_linear_w8a8_noalloc, read back by bi_linear_w8a8_noalloc_status.
 * Nothing faults or hangs; the context stays usable.
 */
BI_API bi_status bi_selftest_wait_timeout(void *ws, size_t ws_bytes, bi_stream_t stream);

/*
 * Block-scaled variant: the mat-vec of "why speculative decoding changed my
 * output", section "the mat-vec kernel" (q6_k-style weight blocks of 256,
 * int8 activation blocks of 32, integer products per block, fp32 per-block
 * scale-and-add in an order fixed for every number of tokens).  The pages
 * print no storage layout or quantiser; this library's are:
 *
 * Weights, K % 256 == 0.  Super-blocks of 256 = 16 sub-blocks of 16; code
 * c in [-32, 31], int8 sub-scale sc per sub-block, fp32 scale d per
 * super-block; w ~ c * (d * sc).  Per row n:
 *   ql [K/2]  low 4 bits of c + 32, element k in byte k/2, bits 4 (k & 1)
 *   qh [K/4]  high 2 bits of c + 32, element k in byte k/4, bits 2 (k & 3)
 *   sc [K/16], d [K/256]
 * Quantiser, per super-block: t_j = absmax_j / 31 (IEEE fp32 division);
 * d = max_j t_j / 127 (1 if all zero); sc_j = clamp(rne(t_j / d), 0, 127);
 * e_j = d * sc_j (fp32); c = clamp(rne(w / e_j), -32, 31), 0 where e_j = 0.
 *   w  fp32 [N, K] (row stride ldw >= K, ldw % 4 == 0), device.
 *   ql, qh, sc, d  device outputs, row-major as above (16-byte aligned; d 4).
 * Returns BI_ERR_INVALID_ARG for K not a positive multiple of 256.
 */
BI_API bi_status bi_quantize_weight_q6(const float *w, int64_t ldw, int N, int K, uint8_t *ql, uint8_t *qh,
                                       int8_t *sc, float *d, bi_stream_t stream);

/*
 * Activation blocks of 32 for the block-scaled linear: the per-token rule of
 * bi_quantize_act applied to each block of 32 (d_a = absmax / 127, 1 for an
 * all-zero block; q = clamp(rne(x / d_a), -127, 127), IEEE division).
 *   x    bf16 [M, K] (row stride ldx >= K), K % 32 == 0
 *   q    int8 [M, K] out;  d_a  fp32 [M, K/32] out (4-byte aligned)
 */
BI_API bi_status bi_quantize_act_blocks(const uint16_t *x, int64_t ldx, int M, int K, int8_t *q, float *d_a,
                                        bi_stream_t stream);

/*
 * y = the block-scaled linear, fp32 [M, N] (row stride N), 1 <= M <= 16.
 * For token m and row n, 32-block b (of K/32) of super-block s = b / 8 holds
 * sub-blocks j = 2b and 2b + 1:
 *   isum_b = sc_j * sum(c * q) over its first 16 elements
 *          + sc_(j+1) * sum over the next 16               (exact integer)
 *   v_b    = ((float)isum_b * d_a[m][b]) * d[n][s]          (fp32, RNE)
 * Partial l (l = 0 .. 31) adds v_l, v_(l+32), v_(l+64), ... in that order
 * starting from +0; then, for offsets 16, 8, 4, 2, 1, every partial becomes
 * p[l] + p[l xor offset]; y[m][n] = p[0].  The order depends on K only, so
 * every row is bitwise the same for any M and any other rows in the pass.
 *   q, d_a  from bi_quantize_act_blocks (q rows 16-byte aligned)
 *   ql, qh, sc, d  from bi_quantize_weight_q6
 *   flags   BI_FLAG_PDL or 0
 */
BI_API bi_status bi_linear_q6(const int8_t *q, const float *d_a, int M, int K, const uint8_t *ql, const uint8_t *qh,
                              const int8_t *sc, const float *d, int N, float *y, unsigned flags, bi_stream_t stream);

/*
 * Split-KV attention of a verify pass, batch-invariant ("My speculative
 * decoder got slower", split-KV attention in 256-token chunks with a merge;
 * "why speculative decoding changed my output", "attention").  Query m
 * (0 .. M-1) attends to cache positions 0 .. T0 + m; query head h reads kv
 * head h / (Hq / Hkv).  Per query, head and chunk c (positions 256c ..
 * 256c + 255 of those), fp32, every operation rounded once:
 *   s_t = (sum over d in order of q_d k_td, from +0) * scale
 *   mx  = max s_t,  p_t = e(s_t - mx),  l = sum of p_t in position order,
 *   a_d = sum of p_t v_td in position order;
 * then over the query's chunks in order: mx* = max mx_c, w_c = e(mx_c - mx*),
 * L = sum w_c l_c, o_d = bf16_rne((sum w_c a_cd) / L).  e(x) for x <= 0:
 * t = x log2(e) (fp32 constant 0x3FB8AA3B); 0 if t < -126; else n = rne(t),
 * f = t - n, 2^f by the degree-6 Taylor polynomial of e^(f ln 2) in Horner
 * form with c_0 = 1, c_k = (c_(k-1) ln 2) / k (ln 2 = 0x3F317218), times 2^n.
 * Every step acc <- acc + x * y is one fused multiply-add.  A query's result
 * depends only on its own positions: the same bits for any M, for any T0
 * that leaves it the same cache positions, alone or in a batch.
 *   q      bf16 [M, Hq, D]          k, v  bf16 [S, Hkv, D]
 *   o      bf16 [M, Hq, D] out      D = 64 or 128; Hq % Hkv == 0; T0 + M <= S
 *   ws     device workspace of at least bi_attention_workspace_size(M, Hq,
 *          D, T0) bytes (null when that size is 0); its contents need no
 *          initialisation and are overwritten.
 * Device pointers, all 16-byte aligned; M <= 4096, Hq <= 65535, T0 + M <=
 * 2^20 positions, M * Hq / Hkv <= 65535 * 32.
 * One or two launches on `stream` (the second merges when the last query
 * covers more than one chunk).  Returns BI_ERR_INVALID_ARG for a null
 * pointer or an out-of-range size, BI_ERR_ALIGNMENT, BI_ERR_WORKSPACE.
 */
BI_API size_t bi_attention_workspace_size(int M, int Hq, int D, int T0);
BI_API bi_status bi_attention_verify(const uint16_t *q, const uint16_t *k, const uint16_t *v, int M, int Hq, int Hkv,
                                     int D, int T0, int S, float scale, uint16_t *o, void *ws, size_t ws_bytes,
                                     bi_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Decoder-step operators: what stands between the linears of a decode or
 * verify step when it serves a model with normalised layers, rotary positions
 * and a shared cache.  Like everything above, a row's result does not depend
 * on the rows beside it: the same bits for any M, T, B and any other sequences
 * in the call.
 * ---------------------------------------------------------------------------
 *
 * bi_rmsnorm_quantize: the residual's addition, the root-mean-square norm and
 * the activation quantisation of the linear that reads it.  Per row, fp32:
 *   h'  = bf16_rne(h + y)                 (h itself when y is NULL)
 *   t_k = h'_k * w_k                      (exact: two bf16 factors)
 *   r   = 1 / sqrt(sum_k h'_k^2 / K + eps)
 *   a   = max_k |t_k|;  st = a / 127 (IEEE division)
 *   q_k = clamp(rne(t_k / st), -127, 127);  s_a = st * r
 * An all-zero t gives q = 0 and s_a = 1.  The normalised row is t * r, and
 * per-row absmax quantisation is invariant to a row's factor, so the codes are
 * those of the normalised row, without the rounding of r in them; r's sum is
 * taken in an order that depends on K alone.
 *   h    bf16 [M, ldh], read only;  y bf16 [M, ldy], read only, or NULL
 *   w    bf16 [K], the norm's weight;  eps >= 0
 *   h_out bf16 [M, ldo] receives h'; it may be h (ldo == ldh) but not overlap
 *        it otherwise.  Given exactly when y is given.
 *   q    int8 [M, K] out, s_a fp32 [M] out, for bi_linear_w8a8
 * 16-byte aligned h, y, w, h_out and q; row strides multiples of 8 elements;
 * K as for bi_quantize_act.  Products t and the sum of squares must be finite
 * in fp32.  With BI_FLAG_PDL the kernel waits for the preceding kernel first.
 */
BI_API bi_status bi_rmsnorm_quantize(const uint16_t *h, int64_t ldh, const uint16_t *y, int64_t ldy, const uint16_t *w,
                                     float eps, int M, int K, uint16_t *h_out, int64_t ldo, int8_t *q, float *s_a,
                                     unsigned flags, bi_stream_t stream);

/*
 * A paged key/value cache held in 4 bits.  Page p of the pool starts at byte
 * p * page_stride and holds page_size positions of every kv head; the block of
 * kv head g starts bi_kv4_block_bytes(page_size, D) * g bytes into its page.
 * Every 64 consecutive elements of a head's key (or value) at one position
 * form a group with a scale s and a minimum z, both bf16, and 4-bit codes:
 *   z = min x;  s = bf16_rne((max x - min x) / 15)  (fp32, IEEE division)
 *   c = clamp(rne((x - z) / s), 0, 15)  (fp32, IEEE division; 0 when s = 0)
 *   the value held is z + s * c.
 * x are bf16 values, so z is exact, and s is 0 or at least |z| / 4096, which a
 * cache filled in another way has to keep to.  x and max x - min x have to be
 * finite in fp32: other values give codes and parameters without meaning, in
 * their own group (a value group whose s or z is not finite leaves no finite
 * element of that group to the attention's rows that see its position, and
 * touches no other row or group).
 * Values whose s lies outside 2^-110 .. 2^118 lose precision in the attention.
 * Inside a block, P = page_size, G = D / 64, all words little-endian:
 *   keys       [P][4 segments][G][2 words], position-major: element d of a key
 *              is in segment (d % 64) / 16, group d / 64, word (d % 16) / 8,
 *              nibble (d % 8) / 2 + 4 (d % 2);
 *   values     [P / 2][8 segments][G][2 words], after P D / 2 bytes: positions
 *              2 i and 2 i + 1 share words, the even one in the low half;
 *              element d is in segment (d % 64) / 8, group d / 64, word
 *              (d % 8) / 4, nibble d % 4 of its half;
 *   parameters [P][2][G] words, after P D bytes: s in the low and z in the
 *              high half, keys then values.
 * The order of the nibbles is that of tensor-core fragments, so that the
 * attention needs one AND for two codes.
 */
typedef struct {
    void *pool;          /* device, 16-byte aligned */
    int64_t page_stride; /* bytes, a multiple of 16, >= Hkv * bi_kv4_block_bytes(page_size, D) */
    int num_pages;
    int page_size;       /* positions a page: 16, 32, 64 or 128 */
    int Hkv;             /* kv heads, 1 .. 1024 */
    int D;               /* head size, 64 or 128 */
} bi_kv4_cache;

/*
 * A batch of sequences with new tokens, as the append, the gather and the
 * attention read it.  Token rows cu_q[b] .. cu_q[b + 1] - 1 are the newest of
 * sequence b: the last of them is at position kv_len[b] - 1.  Position p of
 * sequence b is kept in page pages[b * ld_pages + p / page_size] of the pool,
 * at p % page_size.  The arrays are read on the device, so a captured graph
 * can be replayed with other lengths and pages; T, max_q and max_kv are bounds
 * that the host knows.  Rows from T on are not touched.  Tokens of a sequence
 * past max_q, or at a position from max_kv on, are left out: their key and value
 * are not written, their q, attention and gathered values are zeros.  Positions
 * whose page index lies outside the table, or whose page is not in 0 ..
 * num_pages - 1, are not written, not attended to, and gathered as zeros; the
 * q of a token at such a position is rotated, and its attention goes over the
 * positions that have pages.  Token rows from cu_q[B] on belong to no sequence:
 * their outputs are not touched.
 */
typedef struct {
    const int32_t *cu_q;   /* [B + 1], non-decreasing, cu_q[0] = 0 */
    const int32_t *kv_len; /* [B], new tokens included */
    const int32_t *pages;  /* [B, ld_pages] */
    int64_t ld_pages;
    int B;                 /* sequences, 1 .. 65535 */
    int T;                 /* rows of the token arrays, 1 .. 2^20 */
    int max_q;             /* most new tokens of a sequence, 1 .. 65535 */
    int max_kv;            /* longest sequence, 1 .. 2^22 */
} bi_kv4_batch;

/* Bytes of one kv head of one page; 0 for a page size or head size that is not supported. */
BI_API size_t bi_kv4_block_bytes(int page_size, int D);

/*
 * Table of rotations: rope[p][i] = (cos, sin)(p * inv_freq[i]) * amp as fp32
 * pairs, p < n_pos, i < n_freq, the angle and its functions in fp64.  Long
 * contexts scale inv_freq (interpolation by a common factor or per frequency)
 * and amp (the amplitude that goes with it); both are the caller's.
 *   inv_freq  fp64 [n_freq], device;  rope fp32 [n_pos, n_freq, 2] out, 8-byte aligned
 */
BI_API bi_status bi_rope_table(const double *inv_freq, int n_freq, float amp, int n_pos, float *rope,
                               bi_stream_t stream);

/*
 * New tokens' heads: optional RMS norm of every q and k head, rotation, q out
 * in bf16, k and v appended to the cache.  Per head x[D] of q or k, fp32, every
 * operation rounded once:
 *   norm (q_norm / k_norm given): n_d = (x_d * r) * w_d,
 *        r = 1 / sqrt(S / D + eps), S = the squares added as halves (d and
 *        d + D / 2), then neighbours, then halves again down to one;
 *   rotation of the first `rot` elements by rope[position]: a pair (a, b)
 *        becomes (a c - b s, b c + a s); pair i is (i, i + rot / 2) with
 *        BI_ROPE_HALF and (2 i, 2 i + 1) with BI_ROPE_INTERLEAVED;
 *   bf16_rne; k and v (v as given) are then quantised as bi_kv4_cache says.
 * A token at a negative position, or at one from n_pos on, has q_out 0 and is
 * not appended either.
 *   q  bf16, row t and head h at q + t ldq + h D, Hq heads (read only)
 *   k, v  bf16, rows of Hkv heads with strides ldk, ldv
 *        (the three may be parts of one packed projection output)
 *   rope  fp32 [n_pos, rot / 2, 2];  rot 0 .. D, a multiple of 8 (of 4 with
 *        BI_ROPE_INTERLEAVED)
 *   q_norm, k_norm  bf16 [D] or NULL;  eps >= 0
 *   q_out bf16 [T, Hq, D], must not overlap the inputs
 * 16-byte aligned pointers; strides multiples of 8 elements.  Hq, Hkv <= 1024.
 * With BI_FLAG_PDL the kernel waits for the preceding kernel first.
 */
enum { BI_ROPE_HALF = 0, BI_ROPE_INTERLEAVED = 1 };
BI_API bi_status bi_rope_append_kv4(const uint16_t *q, int64_t ldq, int Hq, const uint16_t *k, int64_t ldk,
                                    const uint16_t *v, int64_t ldv, const uint16_t *q_norm, const uint16_t *k_norm,
                                    float eps, const float *rope, int n_pos, int rot, int layout, uint16_t *q_out,
                                    const bi_kv4_cache *cache, const bi_kv4_batch *batch, unsigned flags,
                                    bi_stream_t stream);

/*
 * The cached keys and values of the batch's token rows, as bf16_rne(z + s c):
 * what an append wrote, or, with cu_q counting whole sequences, a cached prefix.
 *   k_out, v_out  bf16 [T, Hkv, D] out, 16-byte aligned, not overlapping.
 */
BI_API bi_status bi_kv4_gather(const bi_kv4_cache *cache, const bi_kv4_batch *batch, uint16_t *k_out, uint16_t *v_out,
                               bi_stream_t stream);

/*
 * Attention of the batch's new tokens over the 4-bit cache.  The token at
 * position p of sequence b sees that sequence's positions 0 .. p; q head h
 * reads kv head h / (Hq / Hkv):
 *   o = sum_j softmax_j(scale q . k_j) v_j  over the values held.
 * A token that sees no position (a sequence of length 0) has o = 0.
 *   q  bf16, row t at q + t ldq, head h at h D (ldq >= Hq D, a multiple of 8)
 *   o  bf16 [T, Hq, D] out, must not overlap q
 *   scale  positive and finite;  max_q * (Hq / Hkv) <= 2^22
 *   ws  workspace of at least bi_attention_kv4_workspace_size(...) bytes,
 *       16-byte aligned, zero-filled before its first use; every call that
 *       completes leaves it ready for the next.  Its layout depends on no
 *       argument, so one workspace of the largest size serves calls of any
 *       shape on one stream.  It overlaps neither q nor o.  Its size is the
 *       counters' (about 2 MB) and, where max_kv is above 2048, 4 (D + 4) bytes for
 *       each of T Hq ceil(max_kv / 2048) results: 0.55 GB for 8192 tokens of 32
 *       heads of 128 at 8192 positions, 8.9 GB at 131072; long prompts go in
 *       parts of fewer tokens.  A copy that does not arrive within the wait limit
 *       is reported by bi_workspace_status as BI_ERR_TIMEOUT.
 * Scores, softmax sums and outputs are fp32; the products run on the tensor
 * cores with the codes exact and q exact but for elements 2^-24 below its
 * head's largest (scale times that one below 2^115), and the weights in f16 with
 * 11 bits, always: outputs differ from fp32 weights' by up to 2^-10 of the mean
 * |v| under them, beside the bf16 of the result (2^-8).  A query's result
 * depends on its own positions only.
 */
BI_API size_t bi_attention_kv4_workspace_size(int Hq, const bi_kv4_cache *cache, const bi_kv4_batch *batch);
BI_API bi_status bi_attention_kv4(const uint16_t *q, int64_t ldq, int Hq, const bi_kv4_cache *cache,
                                  const bi_kv4_batch *batch, float scale, uint16_t *o, void *ws, size_t ws_bytes,
                                  unsigned flags, bi_stream_t stream);

/*
 * Rules applied to logits before the argmax or a sampler reads them.  Row m of
 * M, element v, fp32, every operation rounded once, in this order:
 *   x = logits[m][v]
 *   if v is in the row's history:    x = x > 0 ? x / repetition : x * repetition
 *   if it is there c > 0 times as a generated token:
 *                                    x = (x - frequency * c) - presence
 *   if the row has a bias for v:     x = x + bias
 *   if the row's mask forbids v:     x = -inf
 * out[m][v] = x, and argmax[m] = the lowest v with the largest x (NaN counts as
 * -inf), or -1 when every x is -inf: nothing is allowed.
 * The history of row m is ids[begin[m]] .. ids[end[m] - 1]; those from mid[m] on
 * are generated, the others the prompt's.  Rows of one verify pass share ids
 * and differ in `end`.  Ids outside 0 .. V - 1 are ignored.
 */
typedef struct {
    const int32_t *ids;        /* all rows' histories, or NULL: none */
    const int32_t *begin, *mid, *end; /* [M] each, given with ids */
    const float *repetition;   /* [M], > 0, or NULL: 1 */
    const float *presence;     /* [M] or NULL: 0 */
    const float *frequency;    /* [M] or NULL: 0 */
    const int32_t *bias_ids;   /* [M, n_bias] or NULL; of equal ids in a row the last applies */
    const float *bias;         /* [M, n_bias], given with bias_ids */
    int n_bias;                /* 0 .. 65535 */
    const uint32_t *mask;      /* [M, ld_mask] words, bit v % 32 of word v / 32 set = allowed; or NULL: all */
    int64_t ld_mask;           /* >= ceil(V / 32) */
} bi_logits_rules;

/*
 *   logits  bf16 [M, ldl] (read only), ldl >= V
 *   out     fp32 [M, ldo], ldo >= V, or NULL;  argmax int32 [M] or NULL (not
 *           both NULL)
 *   ws      workspace of at least bi_logits_workspace_size(M) bytes, 16-byte
 *           aligned, zero-filled before its first use; every call that completes
 *           leaves it zero-filled
 * out, argmax and ws overlap neither one another nor anything that is read.
 * 1 <= M <= 65535, 1 <= V <= 2^24.  Logits rows may start anywhere on 2 bytes,
 * out rows on 4; rows on 16 bytes are faster.
 */
BI_API size_t bi_logits_workspace_size(int M);
BI_API bi_status bi_logits_process(const uint16_t *logits, int64_t ldl, int M, int V, const bi_logits_rules *rules,
                                   float *out, int64_t ldo, int32_t *argmax, void *ws, size_t ws_bytes, unsigned flags,
                                   bi_stream_t stream);

/*
 * e4m3 linears: activations in 8-bit floating point (1 sign, 4 exponent and 3
 * fraction bits, largest 448, no infinities) with an fp32 scale for each 128
 * elements of a row, weights with one for each block of 128 x 128.  Blocks at
 * the end of a row or column may be short; KB = ceil(K / 128), NB = ceil(N / 128).
 * K is a multiple of 16, 16 .. 2^20; codes are passed as their bytes.
 *
 * Quantisation, every operation rounded once:
 *   s = amax / 448 over the block, or 1 where that is 0
 *   q = e4m3(x / s): fp32 division, round to nearest even, 448 at most
 * x is bf16, or the fp32 gated product act(g) * u of packed rows gate|up:
 * relu(g) = g > 0 ? g : 0, silu(g) = g / (1 + exp(-g)) with a relative error
 * below (|g| + 8) 2^-23 for g >= -131; below that, where it is 2^-181 and less, it
 * may be 0.  A block with an infinity or a NaN has that as its scale and NaN in its
 * codes, so that it shows in its own row alone.
 *   x   bf16 [M, ldx], first K columns (2 K behind a gate) read, 16-byte aligned, ldx % 8 == 0
 *   q   e4m3 [M, K] out, 16-byte aligned;  s_a fp32 [M, KB] out;  1 <= M <= 2^20, M KB < 2^31
 * Outputs overlap neither each other nor the input.  With BI_FLAG_PDL the kernel
 * waits for the preceding kernel first.
 */
enum { BI_GATE_RELU = 0, BI_GATE_SILU = 1 };
BI_API bi_status bi_quantize_act_f8(const uint16_t *x, int64_t ldx, int M, int K, uint8_t *q, float *s_a, unsigned flags,
                                    bi_stream_t stream);
BI_API bi_status bi_gated_quantize_f8(const uint16_t *gu, int64_t ldgu, int M, int K, int gate, uint8_t *q, float *s_a,
                                      unsigned flags, bi_stream_t stream);

/*
 * The weights' format from fp32, by the same rule over blocks of 128 x 128.
 *   w    fp32 [N, ldw], first K columns, 16-byte aligned, ldw % 4 == 0;  1 <= N <= 2^24
 *   w_q  e4m3 [N, K] out, 16-byte aligned;  s_w fp32 [NB, KB] out
 */
BI_API bi_status bi_quantize_weight_f8(const float *w, int64_t ldw, int N, int K, uint8_t *w_q, float *s_w,
                                       bi_stream_t stream);

/*
 * The linear: y[m, n] = bf16_rne(acc) with acc = 0 and then, for the blocks b of
 * K in order,
 *   acc = fma(d, s_a[m, b] * s_w[n / 128, b], acc)   (product and fma in fp32)
 * where d is the tensor cores' fp32 sum of the block's products of codes, added
 * in the same way whatever M, N and the call are: a row's bits depend on that row
 * and the weights alone.
 *   q, s_a  as above, q 16-byte aligned;  w e4m3 [N, K], 16-byte aligned;  s_w fp32 [NB, KB]
 *   y   bf16 [M, N] out (on 2 bytes);  1 <= M <= 2^20, 1 <= N <= 2^24
 *   ws  workspace of at least bi_f8_workspace_size() bytes, 16-byte aligned,
 *       zero-filled before its first use.  It holds a status alone (a wait that
 *       gives up is reported by bi_workspace_status as BI_ERR_TIMEOUT), so that
 *       calls that overlap may share one.
 * y and ws overlap neither each other nor an input.
 *
 * bi_linear_f8_grouped: rows that belong to experts with weights of their own.
 * Expert e has rows offsets[e] .. offsets[e + 1] - 1 of y:
 *   y[r] = the linear of row src[r] of q (row r where src is NULL) and w[e].
 *   q, s_a   q_rows rows, q_rows >= R where src is NULL;  1 <= q_rows, R <= 2^20
 *   src      int32 [R] or NULL; a row that it sends outside 0 .. q_rows - 1 is 0
 *   offsets  int32 [E + 1], non-decreasing, read on the device (a captured graph
 *            may be replayed with other offsets).  Rows of y before offsets[0] and
 *            from offsets[E] on are left as they were.  An offset below the one
 *            before it counts as that one, one above R as R.
 *   w        e4m3 [E, N, K];  s_w fp32 [E, NB, KB];  1 <= E <= 1024, E N < 2^31
 * R and E decide how the work is split, not what a row's bits are.
 */
BI_API size_t bi_f8_workspace_size(void);
BI_API bi_status bi_linear_f8(const uint8_t *q, const float *s_a, int M, int K, const uint8_t *w, const float *s_w, int N,
                              uint16_t *y, void *ws, size_t ws_bytes, unsigned flags, bi_stream_t stream);
BI_API bi_status bi_linear_f8_grouped(const uint8_t *q, const float *s_a, int q_rows, int K, const int32_t *src, int R,
                                      const int32_t *offsets, int E, const uint8_t *w, const float *s_w, int N, uint16_t *y,
                                      void *ws, size_t ws_bytes, unsigned flags, bi_stream_t stream);

/*
 * A router's selection, and the order of rows by expert that the grouped linear
 * reads.  Token m takes the k experts with the largest logits, in that order, the
 * lowest id first among equals.  A logit of -inf (or NaN) is never taken: where
 * fewer than k are left, ids are -1 and weights 0.  +inf counts as the largest
 * finite value.  Weights, fp32:
 *   BI_ROUTE_SOFTMAX  p = exp(x - max) / sum over all experts (over the taken ones with renorm)
 *   BI_ROUTE_SIGMOID  p = 1 / (1 + exp(-x)), divided by the taken ones' sum with renorm
 *   weights = p * scale
 * Slot m k + j of expert e has a row; rows are in the order of experts, then slots:
 *   logits   fp32 or bf16 (`type`) [M, ldl], ldl >= E, read only
 *   ids      int32 [M, k] out;  weights fp32 [M, k] out
 *   offsets  int32 [E + 1] out: first row of each expert, and the number of rows
 *   src      int32 [M k] out: token of each row, -1 from offsets[E] on
 *   pos      int32 [M, k] out: row of each slot, -1 for an id of -1
 *   ws       workspace of at least bi_moe_route_workspace_size(M, E) bytes, 16-byte
 *            aligned, scratch: calls that may overlap must not share one
 * 1 <= M <= 65535, 1 <= E <= 1024, 1 <= k <= min(E, 32), scale finite.  Outputs and
 * workspace overlap neither one another nor the logits.  More than 2^20 slots are more
 * rows than the quantisers and the grouped linear take: such a prompt goes in parts, each
 * with a routing of its own, and has the same bits.
 */
enum { BI_TYPE_F32 = 0, BI_TYPE_BF16 = 1 };
enum { BI_ROUTE_SOFTMAX = 0, BI_ROUTE_SIGMOID = 1 };
BI_API size_t bi_moe_route_workspace_size(int M, int E);
BI_API bi_status bi_moe_route(const void *logits, int64_t ldl, int type, int M, int E, int k, int score, int renorm,
                              float scale, int32_t *ids, float *weights, int32_t *offsets, int32_t *src, int32_t *pos,
                              void *ws, size_t ws_bytes, unsigned flags, bi_stream_t stream);

/*
 * The weighted sum of the experts' rows: acc = 0, then acc = fma(weights[m, j],
 * rows[pos[m, j], n], acc) in the order of j, y[m, n] = bf16_rne(base[m, n] + acc).
 * A slot whose pos lies outside 0 .. R - 1 is left out, whatever its weight.
 *   rows bf16 [R, N];  pos int32, weights fp32 [M, k];  base bf16 [M, N] or NULL: 0
 *   y    bf16 [M, N] out; it may be base, and overlaps nothing else
 * 1 <= M <= 65535, 1 <= k <= 32, 1 <= R <= 2^21, 1 <= N <= 2^24.  Rows on 2 bytes;
 * on 16 with N a multiple of 8 they are faster.
 */
BI_API bi_status bi_moe_combine(const uint16_t *rows, int R, const int32_t *pos, const float *weights, int M, int k, int N,
                                const uint16_t *base, uint16_t *y, unsigned flags, bi_stream_t stream);

/*
 * Bandwidth probes, for measurement only: the device's own read-only and copy
 * ceilings with 16-byte streaming loads (8 in flight per thread) over a grid
 * of four 512-thread CTAs per SM.  A weight stream only reads, so the
 * read-only ceiling is the one it is measured against.
 *   bi_probe_read: reads `bytes` of `buf` once; *out (device, 8-byte aligned)
 *     = the xor of all its 64-bit words (a check that every byte was read).
 *   bi_probe_copy: dst = src, `bytes` bytes; src and dst must not overlap.
 * Device pointers, 16-byte aligned; bytes a positive multiple of 16.
 * Returns BI_ERR_INVALID_ARG or BI_ERR_ALIGNMENT for bad arguments.
 */
BI_API bi_status bi_probe_read(const void *buf, size_t bytes, unsigned long long *out, bi_stream_t stream);
BI_API bi_status bi_probe_copy(const void *src, void *dst, size_t bytes, bi_stream_t stream);

/*
 * Exhaustive check of the quotient the verify-pass executor quantises with.
 * Codes are clamp(rne(v / s), -127, 127) with v / s an IEEE fp32 division
 * (the per-token absmax quantisation of the W8A8 page, "Quantization").  The
 * executor forms v / s from r = RN(1/s) by one fused-multiply-add correction
 * instead of dividing.  This runs, for every positive finite bf16 row maximum
 * amax (scale s = RN(amax / 127) >= 2^-64) and every bf16 v with |v| <= amax
 * (about 0.99e9 pairs), that quotient and the IEEE division, and counts the
 * pairs whose codes differ or whose quotients differ at |v / s| >= 2^-8
 * (smaller quotients have code 0 either way).
 *   out  device, 8-byte aligned, 3 x uint64, overwritten: [0] pairs checked,
 *        [1] mismatches, [2] one mismatching pair (amax bits << 16 | v bits)
 *        or 0.  Read it after the stream completes.
 * Returns BI_ERR_INVALID_ARG for a null or misaligned `out`.
 */
BI_API bi_status bi_selftest_quotient(unsigned long long *out, bi_stream_t stream);

/*
 * Verify-pass executor: a program of ops run by one persistent kernel.
 *
 * A decode or verify pass is a chain of small dependent steps (quantise an
 * activation, stream a weight matrix, ...).  Launched one call at a time each
 * step pays a launch, a ramp to full memory bandwidth and a tail, which for
 * the smaller projections cost more than the weight read itself.  A program
 * runs all of them in one cooperative launch (two CTAs per SM): op i starts
 * only after every op before it has completed on the whole GPU (a grid-wide
 * barrier), so an op may read anything earlier ops wrote, while the weight
 * tiles of the ops ahead keep streaming into shared memory across the
 * barriers (weights never depend on earlier ops).  Every op gives exactly
 * the bits of the corresponding single call.
 *
 * Build once, run many times: bi_program_build validates the ops, encodes
 * the TMA descriptors and copies the program (bi_program_bytes(n_ops) bytes,
 * caller-allocated device memory, 128-byte aligned) synchronously; the
 * program refers to the ops' buffers by address, so their contents may
 * change between runs but not their addresses.  bi_program_run is one
 * asynchronous launch on `stream` (capturable in a CUDA graph once the
 * program is built); `max_tokens` is the largest M of the program's linear
 * and LM-head ops (1..16) and must be the value the program was built for.
 * The workspace follows the zero-fill rule of bi_linear_workspace_size.
 * A mismatched program or max_tokens is reported by bi_workspace_status as
 * BI_ERR_INVALID_ARG; a bounded wait that gives up as BI_ERR_TIMEOUT.
 */
typedef enum {
    BI_OP_QUANTIZE_ACT = 1, /* x, ldx, M, K -> q, s_a        (bi_quantize_act)  */
    BI_OP_LINEAR = 2,       /* q, s_a, M, K, w_q, s_w, N -> y (bi_linear_w8a8, M <= 16) */
    BI_OP_LMHEAD = 3,       /* ... -> y (logits, may be NULL), argmax (bi_lmhead_argmax) */
    BI_OP_RESIDUAL_QUANT = 4, /* y = h [M, K] in/out, x = addend (ldx), M, K -> q, s_a
                                 (bi_residual_quantize) */
    BI_OP_RELU_MUL_QUANT = 5  /* x = packed gate|up [M, ldx >= 2K], M, K -> q, s_a,
                                 y = m or NULL (bi_relu_mul_quantize) */
} bi_op_kind;

typedef struct {
    int kind;               /* bi_op_kind */
    int M, N, K;            /* N unused by the three quantising kinds */
    const uint16_t *x;      /* quantising kinds: input rows (see above) */
    int64_t ldx;
    int8_t *q;              /* quantise: output; linear / head: input */
    float *s_a;             /* quantise: output; linear / head: input */
    const int8_t *w_q;      /* linear / head weights [N, K] */
    const float *s_w;       /* [N] */
    uint16_t *y;            /* linear: output [M, N]; head: logits or NULL;
                               residual: the stream h; relu-mul: m or NULL */
    int32_t *argmax;        /* head: output [M] */
    const int32_t *draft;   /* head, optional: drafted tokens [M - 1] (see bi_greedy_verify) */
    int32_t *accept;        /* head, optional: [2] accepted count and next token, or NULL */
} bi_op;

BI_API size_t bi_program_bytes(int n_ops);
BI_API size_t bi_program_workspace_size(void);
BI_API bi_status bi_program_build(const bi_op *ops, int n_ops, void *program, size_t program_bytes);
BI_API bi_status bi_program_run(const void *program, int max_tokens, void *ws, size_t ws_bytes,
                                bi_stream_t stream);

/*
 * bi_linear_w8a8 for callers that cannot allocate device memory.
 *
 * No counterpart in the papers: this is a deployment variant.  Some callers
 * cannot call cudaMalloc or any allocating routine: code running inside a
 * custom allocator or memory-pool callback, plugins that their host framework
 * hands only input and output pointers, and processes that must not grow
 * their device memory after start-up.  This entry point allocates nothing.
 * The weight-streaming kernel's scratch (split-K partial sums, their
 * counters, a status word) is a fixed array of BI_NOALLOC_SCRATCH_BYTES
 * inside the library, present on every GPU that loads the library until the
 * process exits.  The caller still passes all inputs and outputs.
 *
 *   Arguments, layouts, results and the errors found before any launch are
 *   those of bi_linear_w8a8; there is no workspace argument.
 *   M must be <= BI_NOALLOC_MAX_M (the most the fixed scratch holds); larger
 *   M returns BI_ERR_UNSUPPORTED without launching anything.
 *   The first call on each device (and the first after the device's context
 *   was replaced, for instance by cudaDeviceReset) looks up the scratch
 *   array's device address with that device current; make that first call
 *   before any stream capture.
 *   Every call shares the one array.  The kernel leaves the scratch's counters
 *   and partial sums at zero when it completes, so a call launches with no
 *   clearing (BI_FLAG_PDL keeps its effect).  Calls that may overlap on the
 *   GPU (other streams, other host threads) race on the array and must not
 *   be issued; calls in order on one stream are fine.
 *   A wait inside the kernel that gives up (after 2 s) is recorded in the
 *   scratch's status word and leaves y partly written; later calls are then
 *   not reliable until bi_linear_w8a8_noalloc_status has reported it.
 *   Results are bitwise identical to bi_linear_w8a8.
 *
 * bi_linear_w8a8_noalloc_status: waits for `stream`, then reads the status
 * word of the scratch on the current device: BI_OK, or BI_ERR_TIMEOUT if a
 * wait of an earlier call (or of bi_selftest_wait_timeout with a NULL
 * workspace) gave up.  After a timeout it restores the whole scratch to zero,
 * so that the next call is reliable again.  Allocates nothing.
 */
#define BI_NOALLOC_MAX_M 16
#define BI_NOALLOC_SCRATCH_BYTES 2164992
BI_API bi_status bi_linear_w8a8_noalloc(const int8_t *q, const float *s_a, int M, int K,
                                        const int8_t *w_q, const float *s_w, int N,
                                        uint16_t *y, unsigned flags, bi_stream_t stream);
BI_API bi_status bi_linear_w8a8_noalloc_status(bi_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BI_H */
