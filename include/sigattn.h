/*
 * sigattn — padding-aware bidirectional sigmoid self-attention on NVIDIA B200
 * (sm_100a).  C ABI of libsigattn.so.
 *
 * The operation (gist.science summary of "Better Models, Faster Training:
 * Sigmoid Attention for single-cell Foundation Models", section 2.A, and the
 * paper.rainbus.top summary of the same paper, method steps (1)-(5)):
 *
 *   S  = alpha * Q K^T + b                        per sample z and head h
 *   P  = sigma(S) with P[i, j] = 0 for keys j >= n_k(z)   (the "-inf" mask)
 *   O  = P V, and O[i, :] = 0 for query rows i >= n_q(z)
 *   dS = P (1 - P) (dO V^T)          (padded query rows carry no gradient)
 *   dQ = alpha dS K,  dK = alpha dS^T Q,  dV = P^T dO
 *
 * sigma is the logistic function 1 / (1 + e^-x); there is no row
 * normalisation.  The backward recomputes P (method step (5)); it needs
 * neither O nor any saved statistic.
 *
 * Layout of every tensor argument: [Z][L][H][D], contiguous, row-major:
 * element (z, l, h, d) at ((z * L + l) * H + h) * D + d.  Z = batch, L =
 * padded length, H = heads, D = head dimension.  Base pointers must be
 * 16-byte aligned (every pointer PyTorch allocates is).
 *
 * Sequence lengths are int32[Z] arrays in DEVICE memory (n_q and n_k may
 * differ).  They are read by the kernels, not by the host.  Values outside
 * [0, L] are clamped on the device and flag SIGATTN_ERR_SEQLEN_RANGE in the
 * device status word (see sigattn_last_device_status).
 *
 * Ownership: the caller owns and allocates every buffer; calls allocate
 * no device memory per call.  The library lazily allocates, once per device,
 * a small device status buffer that lives until process exit.  In host
 * memory it caches the TMA tensor maps it encodes, keyed by (base address,
 * Z, L, H, D), which is all a map depends on (at most 1024, then the cache is
 * emptied).
 *
 * CUDA graphs: the compute calls (not sigattn_fwd_bwd_host) can be captured
 * after a first call on the device; a replay reads the lengths and tensors
 * from the captured addresses again.
 *
 * Asynchrony: every compute call enqueues its kernels on `stream` (a
 * cudaStream_t passed as void*; NULL = the legacy default stream) and
 * returns without synchronising.  The return code covers argument
 * validation and launch errors only; errors detected on the device (bounded
 * waits that ran out, clamped lengths) accumulate in the device status word.
 *
 * Precision: SIGATTN_BF16 inputs/outputs run on the tcgen05 tensor cores
 * with fp32 accumulation in tensor memory (P and dS are rounded to bf16
 * before their second matmul).  SIGATTN_FP32 runs an fp32 CUDA-core path
 * meant for accuracy checks, not speed.
 */
#ifndef SIGATTN_H
#define SIGATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SIGATTN_OK = 0,
    SIGATTN_ERR_INVALID_ARG = 1,          /* null pointer, non-positive size, ... */
    SIGATTN_ERR_UNSUPPORTED_HEADDIM = 2,  /* D not in {64, 128} */
    SIGATTN_ERR_UNSUPPORTED_DTYPE = 3,
    SIGATTN_ERR_UNSUPPORTED_DEVICE = 4,   /* bf16 path needs compute capability 10.0 */
    SIGATTN_ERR_MISALIGNED = 5,           /* a base pointer is not 16-byte aligned */
    SIGATTN_ERR_CUDA = 6,                 /* a CUDA runtime/driver call failed */
    SIGATTN_ERR_TIMEOUT = 7,              /* device: a bounded wait ran out */
    SIGATTN_ERR_SEQLEN_RANGE = 8,         /* device: a length was outside [0, L] */
    SIGATTN_ERR_TOO_LARGE = 9,            /* a size exceeds a fixed limit */
    SIGATTN_ERR_PAGE_RANGE = 10           /* device: a page number was outside [0, pages) */
} sigattn_status;

typedef enum {
    SIGATTN_BF16 = 0,
    SIGATTN_FP32 = 1
} sigattn_dtype;

/* How the bf16 kernels evaluate sigma in registers.
 * SIGATTN_SIGMOID_TANH: sigma(x) = 0.5 tanh(x / 2) + 0.5 with the hardware
 *   tanh.approx.f32 (paper.rainbus.top summary, method step (3)); one MUFU
 *   operation per score.
 * SIGATTN_SIGMOID_EXP: u = e^-|x| with one hardware ex2.approx, then
 *   g = 1/(1+u) by a degree-4 minimax polynomial on the FMA pipe (relative
 *   error < 3.4e-4) and sigma = g (x >= 0) or u g (x < 0); one MUFU
 *   operation per score and relative accuracy in both tails.
 * The fp32 path always uses the exact library expf. */
typedef enum {
    SIGATTN_SIGMOID_TANH = 0,
    SIGATTN_SIGMOID_EXP = 1
} sigattn_sigmoid_mode;

/* Forward: O = [i < n_q] * sum_{j < n_k} sigma(alpha q_i . k_j + b) v_j.
 * q, k, v: [Z][L][H][D] inputs (device, read only).  o: [Z][L][H][D] output
 * (device); every element is written, padded query rows as exact zeros.
 * D in {64, 128}; any L >= 1 (partial tiles are masked); Z, H >= 1.
 * Errors: SIGATTN_ERR_INVALID_ARG, _UNSUPPORTED_HEADDIM, _UNSUPPORTED_DTYPE,
 * _UNSUPPORTED_DEVICE, _MISALIGNED, _CUDA.  On error nothing is launched. */
sigattn_status sigattn_fwd(const void *q, const void *k, const void *v, void *o,
                           const int32_t *seqlens_q, const int32_t *seqlens_k,
                           int Z, int L, int H, int D, float alpha, float bias,
                           sigattn_dtype dtype, void *stream);

/* Backward: given dout = dL/dO, writes dq, dk, dv (each [Z][L][H][D],
 * device, fully written; rows at or beyond n_q (dq) or n_k (dk, dv) are exact
 * zeros).  dout rows at or beyond n_q are ignored.  Launches a dQ kernel and
 * a dK/dV kernel on `stream`; neither uses atomics.  Same errors as
 * sigattn_fwd. */
sigattn_status sigattn_bwd(const void *q, const void *k, const void *v, const void *dout,
                           void *dq, void *dk, void *dv,
                           const int32_t *seqlens_q, const int32_t *seqlens_k,
                           int Z, int L, int H, int D, float alpha, float bias,
                           sigattn_dtype dtype, void *stream);

/* The two halves of sigattn_bwd, for callers that want to run them on
 * separate streams (they only read q, k, v, dout and write disjoint
 * outputs) or time them apart.  sigattn_bwd_dq writes dq; sigattn_bwd_dkdv
 * writes dk and dv.  Arguments, layout and errors as sigattn_bwd. */
sigattn_status sigattn_bwd_dq(const void *q, const void *k, const void *v, const void *dout,
                              void *dq, const int32_t *seqlens_q, const int32_t *seqlens_k,
                              int Z, int L, int H, int D, float alpha, float bias,
                              sigattn_dtype dtype, void *stream);
sigattn_status sigattn_bwd_dkdv(const void *q, const void *k, const void *v, const void *dout,
                                void *dk, void *dv, const int32_t *seqlens_q,
                                const int32_t *seqlens_k, int Z, int L, int H, int D,
                                float alpha, float bias, sigattn_dtype dtype, void *stream);

/* Queries and keys of different padded lengths: q, dout, o, dq are
 * [Z][Lq][H][D]; k, v, dk, dv are [Z][Lk][H][D]; n_q <= Lq and n_k <= Lk.
 * This is the shape of one rank's work when a sequence is split across GPUs
 * (context parallelism): its slice of queries against every key, and dK, dV
 * contributions of its queries to every key, which the ranks then add up.
 * Since sigma needs no row normalisation, those contributions are plain sums
 * (the operation as in sigattn_fwd / sigattn_bwd, gist.science summary,
 * section 2.A).  Lq = Lk gives exactly sigattn_fwd / sigattn_bwd.
 * Errors as sigattn_fwd / sigattn_bwd, plus SIGATTN_ERR_INVALID_ARG when
 * exactly one of Lq, Lk is zero (both zero, or Z or H zero: nothing to do). */
sigattn_status sigattn_fwd_rect(const void *q, const void *k, const void *v, void *o,
                                const int32_t *seqlens_q, const int32_t *seqlens_k, int Z, int Lq,
                                int Lk, int H, int D, float alpha, float bias, sigattn_dtype dtype,
                                void *stream);
sigattn_status sigattn_bwd_rect(const void *q, const void *k, const void *v, const void *dout,
                                void *dq, void *dk, void *dv, const int32_t *seqlens_q,
                                const int32_t *seqlens_k, int Z, int Lq, int Lk, int H, int D,
                                float alpha, float bias, sigattn_dtype dtype, void *stream);

/* Forward and backward of a batch held in HOST memory, with the transfers
 * overlapped.  The batch is cut into units of one sample and a group of heads
 * (about 16 units in all, so that the first copy in and the last copy out,
 * which nothing overlaps, are short, but never less than 8 MB per tensor of a
 * unit, so that whole samples stay whole when they are small; the first and
 * the last group are then halved, as nothing overlaps their copies).
 * Per unit, its rows of q, k, v, dout (host, [Z][L][H][D]) are copied into a
 * compact device slot on a library-owned copy stream while earlier units
 * compute; the forward and the backward of the unit run on one of two
 * library-owned compute streams (consecutive units alternate, so one unit's
 * last wave overlaps the next unit's first); its o, dq, dk, dv rows go back to
 * the host tensors on a second copy stream while later units compute.  The
 * results equal sigattn_fwd + sigattn_bwd on the same data bit for bit (every
 * (sample, head) pair is computed on its own by the same kernels).
 * host_seqlens_q / host_seqlens_k: int32[Z] in host memory, checked and read
 * on the host during the call (values outside [0, L] are
 * SIGATTN_ERR_INVALID_ARG); they may be reused as soon as it returns.
 * workspace: caller-owned device memory of at least
 * sigattn_fwd_bwd_host_workspace_bytes(Z, L, H, D, dtype) bytes, 256-byte
 * aligned (three unit slots of the eight tensors plus their lengths).
 * The transfers overlap the compute only when the host buffers are pinned
 * (page-locked); pageable buffers work but serialise the copies.  Returns when
 * all work is enqueued; it is complete once `stream` has passed it (the
 * pipeline's streams start after the work already on `stream`).  The streams
 * are created on the first call on each device and kept; calls on one device
 * must not overlap each other (they share those streams).
 * Errors as sigattn_bwd, plus SIGATTN_ERR_INVALID_ARG for a missing or small
 * workspace and SIGATTN_ERR_MISALIGNED for a misaligned one. */
sigattn_status sigattn_fwd_bwd_host(const void *q, const void *k, const void *v, const void *dout,
                                    void *o, void *dq, void *dk, void *dv,
                                    const int32_t *host_seqlens_q, const int32_t *host_seqlens_k,
                                    int Z, int L, int H, int D, float alpha, float bias,
                                    sigattn_dtype dtype, void *workspace, size_t workspace_bytes,
                                    void *stream);
size_t sigattn_fwd_bwd_host_workspace_bytes(int Z, int L, int H, int D, sigattn_dtype dtype);

/* Per-sample bias and its gradient.
 *
 * The pages set the bias to b = -log(n) (paperlayer.ai summary, section 3,
 * background on sigmoid attention; gist.science summary, section 2.A, bias
 * term) and note that this choice was never swept (paper.rainbus.top summary,
 * limitations).  These calls take one bias per sample, so b_z = -ln n_z or a
 * learned value can be used, and return the bias gradient
 *     db_z = sum over heads h and valid (i < n_q, j < n_k) of dS_zhij,
 * since x = alpha q.k + b_z.  For one bias shared by all samples, sum db over z.
 *
 * sigattn_fwd_bias: as sigattn_fwd, with `bias` a device float[Z] (not NULL
 * when Z > 0) in place of the scalar.
 *
 * sigattn_bwd_bias: as sigattn_bwd, with `bias` a device float[Z].  `dbias`,
 * if not NULL, is a device float[Z] that receives db; it is computed from the
 * fp32 dS values of the dQ pass, summed per dQ work unit and then per sample
 * in a fixed order (the result does not depend on scheduling).  That needs a
 * caller-owned device `workspace` of at least
 * sigattn_dbias_workspace_bytes(Z, L, H, dtype) bytes, 4-byte aligned, which
 * the call overwrites (its contents on entry do not matter).  With dbias NULL
 * the workspace is not used and may be NULL.
 * Errors: SIGATTN_ERR_INVALID_ARG when bias is NULL, or dbias is set and the
 * workspace is missing, too small or misaligned; otherwise as sigattn_bwd. */
sigattn_status sigattn_fwd_bias(const void *q, const void *k, const void *v, void *o,
                                const int32_t *seqlens_q, const int32_t *seqlens_k, int Z, int L,
                                int H, int D, float alpha, const float *bias, sigattn_dtype dtype,
                                void *stream);
sigattn_status sigattn_bwd_bias(const void *q, const void *k, const void *v, const void *dout,
                                void *dq, void *dk, void *dv, const int32_t *seqlens_q,
                                const int32_t *seqlens_k, int Z, int L, int H, int D, float alpha,
                                const float *bias, float *dbias, void *workspace,
                                size_t workspace_bytes, sigattn_dtype dtype, void *stream);
/* The pages' per-sample bias b_z = -ln n_z (paperlayer.ai summary, section 3;
 * gist.science summary, section 2.A), for sigattn_fwd_bias / sigattn_bwd_bias:
 * seqlens is a device int32[Z] (typically seqlens_k), bias a device float[Z]
 * that receives -logf(n_z), or 0 where n_z <= 1.  Asynchronous on `stream`.
 * Errors: SIGATTN_ERR_INVALID_ARG for Z < 0 or a NULL pointer with Z > 0,
 * SIGATTN_ERR_CUDA for a launch failure. */
sigattn_status sigattn_log_length_bias(const int32_t *seqlens, int Z, float *bias, void *stream);

/* Bytes of device workspace sigattn_bwd_bias needs to return dbias (0 for an
 * empty problem): one float per dQ work unit (bf16: per 128-row query tile
 * and head; fp32: per query row and head) of every sample. */
size_t sigattn_dbias_workspace_bytes(int Z, int L, int H, sigattn_dtype dtype);

/* Masked attention: spans, a cap on the scores, a bias that falls with distance,
 * and heads that share keys.
 *
 *   x_ij = cap tanh(alpha q_i . k_j / cap) - slopes[h] |i - j| + b
 *          (cap = 0: alpha q_i . k_j - slopes[h] |i - j| + b)
 *   P_ij = sigma(x_ij) where lo_i <= j < hi_i, j < n and i < n; 0 elsewhere
 *   O    = P V
 *
 * Query i and key j are positions of one padded row of L places with n true
 * tokens.  q, dout, o, dq: [Z][L][H][D]; k, v, dk, dv: [Z][L][Hk][D] with H a
 * multiple of Hk: query head h reads key head h / (H / Hk), and dk, dv are the
 * sums over the query heads that read them.
 *
 * seqlens: device int32[Z], the true lengths n (clamped and flagged as in
 * sigattn_fwd).  spans: device int32[Z][L][2], {lo, hi} of each row, or NULL
 * for rows that see all n keys; any values are allowed (they are clipped to
 * [0, n), and a row with lo >= hi sees nothing: its O and dQ are exact zeros and
 * it adds nothing to dK, dV).  One interval a row covers causal, prefix, document
 * and window masks (sigattn_mask_spans makes those), and key tiles outside the
 * intervals of a tile's rows are neither loaded nor computed; spans that scatter
 * within 128 neighbouring rows give the same results but skip less.
 * bias_z: device float[Z], one bias per sample, or NULL for the scalar bias.
 * cap: 0, or a positive finite number.  slopes: device float[H], or NULL.
 *
 * Rows at or beyond n may hold anything, NaN included: they are never read into
 * a result.  Within a sample a masked key or query must still be finite (it is
 * multiplied by a weight of zero).  What a key or query holds does not change a
 * bit of the rows that do not see it in SIGATTN_SIGMOID_EXP mode and in fp32.  In
 * SIGATTN_SIGMOID_TANH mode one form of the score function is chosen for 32
 * neighbouring rows and the keys that all of them see (queries and keys changed
 * round in dK, dV), so the last bits of a row may depend on the queries (keys) of the
 * 31 beside it; keys outside its span, other documents and padding still have no say.
 *
 * The same call gives the same bits every time.  Between calls of other shapes the
 * order of the fp32 sums may differ: a batch with few tiles splits each tile's keys
 * or queries over up to four blocks, whose sums are added in order.
 *
 * Outputs must not overlap inputs (the kernels of one call run side by side).
 * sigattn_bwd_span writes dq, dk, dv in full and needs neither O nor any saved
 * statistic.  Its workspace (device memory, 16-byte aligned, at least
 * sigattn_bwd_span_workspace_bytes(Z, L, dtype) bytes; 0 for fp32) is
 * overwritten; calls that may overlap, captured graphs included, need one each.
 * Errors: SIGATTN_ERR_INVALID_ARG (also: H not a multiple of Hk or H = 0 with
 * Hk > 0, a negative or non-finite cap, a missing or small workspace), _UNSUPPORTED_HEADDIM,
 * _UNSUPPORTED_DTYPE, _UNSUPPORTED_DEVICE, _MISALIGNED (also: spans not 8-byte
 * aligned), _TOO_LARGE (fp32: 2^31 groups of four rows), _CUDA.  On error nothing is
 * launched. */
sigattn_status sigattn_fwd_span(const void *q, const void *k, const void *v, void *o,
                                const int32_t *seqlens, const int32_t *spans, int Z, int L, int H,
                                int Hk, int D, float alpha, float bias, const float *bias_z,
                                float cap, const float *slopes, sigattn_dtype dtype, void *stream);
sigattn_status sigattn_bwd_span(const void *q, const void *k, const void *v, const void *dout,
                                void *dq, void *dk, void *dv, const int32_t *seqlens,
                                const int32_t *spans, int Z, int L, int H, int Hk, int D, float alpha,
                                float bias, const float *bias_z, float cap, const float *slopes,
                                void *workspace, size_t workspace_bytes, sigattn_dtype dtype,
                                void *stream);
size_t sigattn_bwd_span_workspace_bytes(int Z, int L, sigattn_dtype dtype);

/* Writes the spans of the usual masks, int32[Z][L][2] on the device.  Row i of a
 * sample of n tokens starts from [0, n), or, with docs (device int32[Z][L], a
 * document id per token), from the run of equal ids around i; then
 *   causal:   hi = min(hi, i + 1)
 *   prefix:   (device int32[Z], with causal) hi = min(end, max(i + 1, start +
 *             prefix[z])): the first prefix[z] tokens of the sample, or of each
 *             document, are seen by all its rows
 *   window:   (> 0, not with prefix) lo = max(lo, i - window + 1), and without
 *             causal hi = min(hi, i + window)
 * Rows at or beyond n, and rows that see nothing, get {0, 0}.  prefix and docs
 * may be NULL.  Errors: SIGATTN_ERR_INVALID_ARG, _MISALIGNED, _CUDA. */
sigattn_status sigattn_mask_spans(const int32_t *seqlens, const int32_t *prefix, const int32_t *docs,
                                  int causal, int window, int Z, int L, int32_t *spans,
                                  void *stream);

/* A paged cache of keys and values, and attention against it.
 *
 * k_pages, v_pages: [pages][page_size][Hk][D], page_size 16, 32, 64, 128 or 256.
 * page_table: device int32[Z][max_pages]; place at of sample z is row at %
 * page_size of page page_table[z][at / page_size].  Entries that no place of a
 * call reaches may hold anything.  A page number outside [0, pages) is flagged
 * (SIGATTN_ERR_PAGE_RANGE in the device status word): nothing is written there,
 * and reading it counts as keys that weigh zero.  Pages may be shared by
 * samples for reading; writing one place twice in a call leaves either value.
 *
 * sigattn_cache_append writes seqlens_new[z] <= L tokens of k, v ([Z][L][Hk][D])
 * behind the cache_lens[z] places that sample z has, and lens_out[z] =
 * cache_lens[z] + seqlens_new[z] (device int32[Z]; may be cache_lens itself when
 * L = 1, and must not overlap the lengths, prefix_len or other outputs otherwise).  Keys are rotated on the way, and so are the queries q
 * ([Z][L][H][D] -> q_out, which may be q and overlaps no input otherwise; both
 * NULL and H = 0 for none; rows of padding are written as zeros): token l has position p = prefix_len[0] +
 * cache_lens[z] + l, and pair i of the first rot entries of each head turns by
 * p inv_freq[i] (angles in 64 bits),
 *     (a, b) -> (a cos - b sin, b cos + a sin),
 * the pairs being entries (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved.
 * rot: 0 (no rotation) or a multiple of 16 up to D; inv_freq: device
 * float[rot / 2].  prefix_len: device int32[1] (a shared prefix before the
 * sample's own places), or NULL for 0.  Places beyond max_pages * page_size are
 * not written; that, and lengths outside their range, are flagged
 * (SIGATTN_ERR_SEQLEN_RANGE) and clamped.  No place but the new tokens' is
 * touched.
 *
 * sigattn_fwd_paged: queries q, output o [Z][L][H][D] (o may be q, and overlaps no
 * input otherwise); seqlens_q[z] <= L of them
 * are sample z's last tokens, and seqlens_k[z] >= seqlens_q[z] its own tokens in
 * the cache, theirs included.  Query l, at own place i = seqlens_k - seqlens_q + l,
 * sees its own places up to i and, with a prefix, all prefix_len[0] places of
 * the pages prefix_table (device int32[prefix_pages]).  In bf16 these are read once
 * per key head for up to 256 rows (tokens times query heads) of the batch together, and
 * not once a sample; the fp32 path, made for accuracy, reads all keys for each row.
 * Scores as in sigattn_fwd_span, |i - j| being the distance
 * between positions (the prefix comes first).  Padded query rows are written as
 * exact zeros; cache places that no query sees may hold anything, NaN included.
 * workspace (device, 16-byte aligned, sigattn_fwd_paged_workspace_bytes bytes,
 * 0 for fp32) is overwritten; calls that may overlap, captured graphs included,
 * need one each.  Results do not depend on scheduling; the last bits of a row may
 * depend on the other rows of the batch.  Z is at most SIGATTN_PAGED_MAX_Z.
 *
 * Errors of both: SIGATTN_ERR_INVALID_ARG (sigattn_cache_append: also L = 0;
 * sigattn_fwd_paged: also pages = 0), _UNSUPPORTED_HEADDIM,
 * _UNSUPPORTED_DTYPE, _UNSUPPORTED_DEVICE, _MISALIGNED, _TOO_LARGE (2^31 places,
 * tokens, rows or, over all samples of sigattn_fwd_paged, 64-place tiles; 65536
 * heads; sigattn_fwd_paged: tokens that make 65536 pairs of row tiles, of 128 / (H /
 * Hk) tokens each), _CUDA.  On error nothing is launched. */
#define SIGATTN_PAGED_MAX_Z 4096
sigattn_status sigattn_cache_append(const void *k, const void *v, const void *q, void *q_out,
                                    void *k_pages, void *v_pages, const int32_t *page_table,
                                    const int32_t *cache_lens, const int32_t *seqlens_new,
                                    const int32_t *prefix_len, int32_t *lens_out, int Z, int L,
                                    int H, int Hk, int D, int pages, int page_size, int max_pages,
                                    const float *inv_freq, int rot, int interleaved,
                                    sigattn_dtype dtype, void *stream);
sigattn_status sigattn_fwd_paged(const void *q, const void *k_pages, const void *v_pages, void *o,
                                 const int32_t *page_table, const int32_t *seqlens_k,
                                 const int32_t *seqlens_q, const int32_t *prefix_table,
                                 const int32_t *prefix_len, int Z, int L, int H, int Hk, int D,
                                 int pages, int page_size, int max_pages, int prefix_pages,
                                 float alpha, float bias, const float *bias_z, float cap,
                                 const float *slopes, void *workspace, size_t workspace_bytes,
                                 sigattn_dtype dtype, void *stream);
size_t sigattn_fwd_paged_workspace_bytes(int Z, int L, int H, int Hk, int D, sigattn_dtype dtype);

/* Selects how later bf16 calls in this process evaluate sigma (process-wide,
 * default SIGATTN_SIGMOID_TANH, the pages' form; see sigattn_sigmoid_mode).  Returns
 * SIGATTN_ERR_INVALID_ARG for an unknown mode.
 *
 * Accuracy against the fp64 definition grows worse with L in TANH mode: with
 * b = -ln L most scores sit in sigma's left tail, where 0.5 + 0.5 tanh(x/2)
 * cancels (relative error of sigma up to 1.4% for x in [-12, -8]).  Measured
 * L1 relative error of the outputs on B200 (sampled rows, tanh mode): <= 3.4e-3
 * at L = 16384, 4.6e-3 to 4.8e-3 at L = 65536, against a bf16 bar of 5e-3;
 * EXP mode stays near 2.3e-3 at every L.  Use EXP for sequences longer than
 * about 32K, or wherever the left tail must be accurate. */
sigattn_status sigattn_set_sigmoid_mode(sigattn_sigmoid_mode mode);
sigattn_sigmoid_mode sigattn_get_sigmoid_mode(void);

/* Evaluates the kernels' own device sigma routine for `mode` on n fp32
 * values: y[i] = sigma(x[i]) and, if dy != NULL, dy[i] = sigma'(x[i]) as
 * the backward kernels form it.  x, y, dy are device arrays of n floats.
 * Used to measure the error of the in-register sigma against fp64. */
sigattn_status sigattn_sigmoid_eval(const float *x, float *y, float *dy, int64_t n,
                                    sigattn_sigmoid_mode mode, void *stream);

/* Reads and clears the current device's status word: synchronises `stream`
 * and returns SIGATTN_OK or the first device-side error recorded since the
 * last call (SIGATTN_ERR_TIMEOUT, SIGATTN_ERR_SEQLEN_RANGE or
 * SIGATTN_ERR_PAGE_RANGE). */
sigattn_status sigattn_last_device_status(void *stream);

/* Bound, in nanoseconds, on every wait inside the bf16 kernels (default
 * 4e9, at least 1e6, else SIGATTN_ERR_INVALID_ARG).  A wait that runs out
 * records SIGATTN_ERR_TIMEOUT, the kernel abandons its work, waits (with the
 * same bound) for the tile loads and MMAs it has in flight, frees its tensor
 * memory and exits. */
sigattn_status sigattn_set_wait_timeout_ns(uint64_t ns);

/* Launches a one-CTA kernel whose only job is to wait on a barrier that
 * nothing signals, bounded by timeout_ns; it must return with
 * SIGATTN_ERR_TIMEOUT recorded in the status word and leave the context
 * usable.  Exercises the failure path of the bounded waits. */
sigattn_status sigattn_selftest_wait_timeout(uint64_t timeout_ns, void *stream);

/* Forward for callers that must not allocate device memory.
 *
 * No counterpart in the paper; this is a deployment convenience.  Some
 * callers cannot call cudaMalloc at the time they run attention: code running
 * inside a framework whose caching allocator owns all device memory (a
 * cudaMalloc behind its back can fail or fragment the pool it manages), or a
 * service that reserves its memory at start-up and forbids allocation on the
 * request path (an allocation there can stall or fail under load).  Such
 * callers often also have the per-sample lengths only on the host.  This entry point
 * computes exactly what sigattn_fwd computes, with the same kernel, but takes
 * seqlens_q / seqlens_k as HOST int32[Z] arrays and never allocates: the
 * lengths and the kernel's device status word live in a fixed array in the
 * library's own device memory (a file-scope __device__ array, loaded with
 * the module, present on every GPU that loads the library until exit).
 *
 * Limits and behaviour:
 *  - Z <= SIGATTN_NOALLOC_MAX_Z (8192), else SIGATTN_ERR_TOO_LARGE and
 *    nothing is launched.  Lengths are checked on the host: any value
 *    outside [0, L] returns SIGATTN_ERR_SEQLEN_RANGE before any launch.
 *  - The host arrays are read during the call: their values reach the
 *    device as kernel arguments (up to 480 samples per small launch), so
 *    they may be reused or freed as soon as the call returns, pageable or
 *    pinned alike.
 *  - The first call on a device looks up the array's device address
 *    (cudaGetSymbolAddress); make that first call before any stream capture.
 *  - Every call shares the one array, and it keeps the last call's contents
 *    (the status word is cleared at the start of each call): calls whose
 *    work overlaps on the GPU (different streams, or devices driven from
 *    several threads at once) race on it and must be serialised by the
 *    caller.  A wait that runs out inside the kernel is recorded in that
 *    array's status word only; sigattn_last_device_status does not see it.
 * Other arguments, layout and errors as sigattn_fwd. */
#define SIGATTN_NOALLOC_MAX_Z 8192
sigattn_status sigattn_fwd_noalloc(const void *q, const void *k, const void *v, void *o,
                                   const int32_t *host_seqlens_q, const int32_t *host_seqlens_k,
                                   int Z, int L, int H, int D, float alpha, float bias,
                                   sigattn_dtype dtype, void *stream);

/* Text of the CUDA error behind the most recent SIGATTN_ERR_CUDA returned
 * by any call in this process (static string; "no error" if none). */
const char *sigattn_last_cuda_error(void);

/* Human-readable name of a status code (static string). */
const char *sigattn_status_string(sigattn_status s);

/* Order in which the bf16 kernels start the samples of a batch: blocks are
 * dispatched in grid order, and the block of grid position z works on the
 * sample of rank z by decreasing work, ties by increasing index, so the
 * samples with the most tiles start first and the short ones fill in behind
 * them.  A sample's work is its key length n_k (forward, dQ kernel) or its
 * query length n_q (dK/dV kernel), and 0 when its other length is 0.  For
 * Z > 64 the kernels keep the index order.
 *
 * This host function applies the same rule: work is host int32[Z], order
 * (host int32[Z], written) receives the sample index for each rank.  It runs
 * no device code.  Returns SIGATTN_ERR_INVALID_ARG for a NULL pointer or
 * Z < 0. */
sigattn_status sigattn_launch_order(const int32_t *work, int Z, int32_t *order);

/* Library version, major * 10000 + minor * 100 + patch. */
int sigattn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SIGATTN_H */
