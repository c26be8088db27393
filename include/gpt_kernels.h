/*
 * gpt_kernels.h - per-step entry points of the GB300 GPT library.
 *
 * Each call runs ONE step of the forward pass (the same kernels gpt_forward
 * launches) on caller-owned device buffers, so that every step can be checked
 * on its own against the definitions it implements. All pointers are device
 * pointers, 16-byte aligned; all calls are stream-ordered and asynchronous.
 * Device-side errors (out-of-range ids, expired waits) are recorded in an error
 * word of the current device, which gptk_status() reads and clears with that
 * device current.
 *
 * dtype selects the arithmetic: 0 = fp32 SIMT kernels (fp32 operands),
 * 1 = bf16 operands on the tcgen05 tensor-core kernels with fp32 accumulation.
 */
#ifndef GPT_GB300_KERNELS_H
#define GPT_GB300_KERNELS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* GEMM epilogues */
enum {
  GPTK_EPI_BIAS = 0,        /* out = A W^T + bias, stored in dtype (bf16 or fp32) */
  GPTK_EPI_BIAS_GELU = 1,   /* out = gelu_tanh(A W^T + bias) ("第 25 章" §25.3) */
  GPTK_EPI_BIAS_RESID = 2,  /* out (fp32) += A W^T + bias: the residual add (§25.1) */
  GPTK_EPI_F32 = 3          /* out (fp32) = A W^T (+ bias if non-NULL) */
};

/*
 * out[M,N] = epilogue(A[M,K] . W[N,K]^T + bias[N]).
 * A and W are row-major in dtype (nn.Linear orientation, §25.5); bias fp32
 * [N] or NULL; out row-major with row stride N. K and N must be multiples of
 * 8 on the bf16 path (16-byte TMA row strides). Where the bf16 tiles would not
 * fill whole waves of the GPU and K >= 1536, epilogues 0-2 split tiles along K
 * between two CTAs (stream-K, fixed summation order: results do not depend on
 * timing); their fp32 partial tiles and flags are allocated on the stream
 * (stream-ordered allocator) and freed there after the launch.
 */
int gptk_gemm(const void* A, const void* W, const float* bias, void* out, int32_t M, int32_t N,
              int32_t K, int32_t epilogue, int32_t dtype, void* stream);

/*
 * The bf16 products on pairs of CTAs: clusters of two whose tcgen05.mma.cta_group::2 computes
 * 256 x 256 tiles, each CTA staging 128 rows of A and 128 of the tile's W rows per K step.
 * The epilogues of gptk_gemm: GPTK_EPI_BIAS and GPTK_EPI_BIAS_GELU (out bf16), GPTK_EPI_BIAS_RESID
 * (out fp32 += A W^T + bias, the residual add), GPTK_EPI_F32 (out fp32 = A W^T + bias). A and W
 * bf16 row-major [M,K] and [N,K], K and N multiples of 8, 16-byte aligned pointers; bias fp32 [N]
 * or NULL; out row-major [M, N]. ksplit <= 1: whole tiles,
 * or stream-K (as gptk_gemm, workspace on the stream) where whole tiles would leave a part-idle
 * last wave and K >= 1536; ksplit > 1 (GPTK_EPI_BIAS_RESID only): each tile's K range is cut
 * into ksplit slices whose partial products are added into out separately (bias must be NULL;
 * the order of those fp32 additions varies between runs). GPT_ECONFIG if clusters of two with
 * this kernel's shared memory cannot be resident on the device.
 */
int gptk_gemm_pair(const void* A, const void* W, const float* bias, void* out, int32_t M, int32_t N,
                   int32_t K, int32_t epilogue, int32_t ksplit, void* stream);

/*
 * Causal self-attention of one layer ("第 25 章" §25.2).
 * qkv: [B, T, 3C] in dtype (Q, K, U thirds; head h = columns [hD, (h+1)D) of each);
 * y:   [B, T, C] in dtype, heads merged. C = H*D; bf16 path: D in {32, 64}.
 */
int gptk_attention(const void* qkv, void* y, int32_t B, int32_t T, int32_t H, int32_t D,
                   int32_t dtype, void* stream);

/*
 * gptk_attention on the bf16 path that also writes, for every query row, the base-2
 * log-sum-exp of its scaled scores: lse2[(b H + h) T + t] = log2 sum_{s <= t} 2^(q_t . k_s log2(e) / sqrt(D))
 * (fp32, [B*H*T]); the softmax normaliser of "第 25 章" §25.2 that the derivative below reuses.
 */
int gptk_attention_lse(const void* qkv, void* y, float* lse2, int32_t B, int32_t T, int32_t H, int32_t D,
                       void* stream);

/*
 * Derivative of the causal self-attention of one layer (bf16 path; the chain rule through the
 * definitions of §25.2, as the training loop of "预训练一个 Mini GPT" needs it): from qkv [B, T, 3C],
 * the output y [B, T, C] and lse2 of gptk_attention_lse, and dy [B, T, C] (the loss gradient with
 * respect to y), writes dqkv [B, T, 3C] bf16: dQ, dK and dU in the thirds of qkv's layout. D in {32, 64};
 * all four bf16 arrays 16-byte aligned. Its fp32 dQ accumulator (B*T*C*4 bytes) and Dsum scratch are
 * allocated on the stream and freed there after the launches.
 */
int gptk_attention_bwd(const void* qkv, const void* y, const void* dy, const float* lse2, void* dqkv, int32_t B,
                       int32_t T, int32_t H, int32_t D, void* stream);

/*
 * Sliding-window attention with sinks (bf16; the source pages attend to the whole past, §25.2: a window at least as
 * long as the sequence gives that): query t sees key s if s <= t and (t - s < window or s < sinks), window >= 1.
 * qkv [B, T, (H + 2 Hkv) D]: a token's H queries, Hkv keys, Hkv values (Q, K, U thirds where Hkv = H); query head h
 * reads key head h / (H / Hkv). y [B, T, H D], heads merged; lse2 fp32 [B, H, T] or NULL: each row's base-2
 * log-sum-exp of its seen scaled scores, as for gptk_attention_lse. fp32 scores and sums; the probabilities are
 * rounded to bf16 for the product with the values. A sequence shorter than T is padded behind its end (rows of finite
 * numbers): no real token sees the padding. A value that is not finite makes the outputs of the queries that see it NaN,
 * and may make those of others of its tile of 128 tokens and the tiles that read it so. y overlaps no input. D in {32, 64},
 * H a multiple of Hkv, 16-byte aligned arrays (GPT_ECONFIG otherwise), T < 2^30, B T < 2^31, rows of less than 2^30
 * elements.
 */
int gptk_attention_window(const void* qkv, void* y, float* lse2, int32_t B, int32_t T, int32_t H, int32_t Hkv, int32_t D,
                          int32_t window, int32_t sinks, void* stream);

/*
 * Its derivative: from qkv, y and lse2 of gptk_attention_window (the same window and sinks) and dy [B, T, H D], writes
 * dqkv [B, T, (H + 2 Hkv) D]: dQ, and dK and dU summed over the H / Hkv query heads of a key head. Rows behind a
 * padded sequence's end take no part where their dy is zero. dqkv overlaps no input. Scratch (4 B T H D bytes, 1,024 B H
 * for each 128 rows of T or part of them, and 1,024 D for each part of a key tile that several CTAs share, a few hundred at
 * most) is taken on the stream from a pool that the library keeps; make a process's first call on a device before any
 * stream capture. dQ's fp32 additions come in an order that varies between runs.
 */
int gptk_attention_window_bwd(const void* qkv, const void* y, const void* dy, const float* lse2, void* dqkv, int32_t B,
                              int32_t T, int32_t H, int32_t Hkv, int32_t D, int32_t window, int32_t sinks, void* stream);

/*
 * LayerNorm over rows of x [M, C] fp32 ("预训练一个 Mini GPT" 第4步; "GPT-1 学习笔记" §3.2):
 * out (dtype) = (x - mean)/sqrt(var + eps) * g + b; out_f32 (fp32, may alias x, may be NULL)
 * receives the same values in fp32. C must be a multiple of 8 and at most 2048.
 */
int gptk_layernorm(const float* x, const float* g, const float* b, void* out, float* out_f32,
                   int32_t M, int32_t C, float eps, int32_t dtype, void* stream);

/*
 * x[b,t,:] = E[ids[b,t],:] + P[t,:] as fp32 [B*T, C] ("第 25 章" §25.1).
 * wte [V, C] and wpe [>=T, C] in dtype.
 */
int gptk_embed(const int32_t* ids, const void* wte, const void* wpe, float* x, int32_t B,
               int32_t T, int32_t C, int32_t V, int32_t dtype, void* stream);

/*
 * Tied head + per-row cross-entropy: nll[m] = logsumexp_j(h_m . E_j) - h_m . E_{targets[m]}
 * ("第 25 章" §25.4, "预训练一个 Mini GPT" 第6步). h [M, C] and wte [V, C] in dtype;
 * nll fp32 [M]; logits fp32 [M, V] or NULL (written only when non-NULL).
 * The bf16 path allocates its partial-logsumexp scratch on the stream.
 */
int gptk_lmhead_ce(const void* h, const void* wte, const int32_t* targets, float* nll,
                   float* logits, int32_t M, int32_t V, int32_t C, int32_t dtype, void* stream);

/*
 * gptk_lmhead_ce without any device allocation (bf16 path only; the source
 * pages have no counterpart: this is an operational variant of the step
 * above). For callers that cannot allocate device memory while they run: a
 * server whose memory budget is fixed at start-up, a framework whose caching
 * allocator already holds the free memory, or a loop that cannot take the
 * synchronisation an allocation may cause. The scratch lives in a fixed
 * library array of 2,097,152 floats (8 MiB) that every GPU loading the library
 * keeps until the process exits; the call returns GPT_EINVAL when
 * M * (2 * ceil(V / 256) + 1) exceeds it (e.g. at most 5,309 rows for V = 50257).
 * The first call on each device looks up that array's device address (with the
 * device current); make that first call before any stream capture. All calls
 * share the array, so calls whose GPU work overlaps race; order them on one
 * stream. The looked-up address is kept for the life of the process: do not
 * use this entry after a reset of the device (cudaDeviceReset or a destroyed
 * and recreated primary context), which invalidates it. d_err: caller-owned
 * device int that receives a nonzero code (and keeps the first one) if a target
 * is outside [0, V) or a bounded wait expired; the nll of a row whose target is
 * out of range is then unspecified, the other rows are still correct. With
 * d_err NULL such errors are not reported anywhere. nll as in gptk_lmhead_ce.
 * No logits.
 */
int gptk_lmhead_ce_noalloc(const void* h, const void* wte, const int32_t* targets, float* nll,
                           int32_t M, int32_t V, int32_t C, int32_t* d_err, void* stream);

/*
 * Paged key/value cache (bf16, D in {32, 64}): the cached keys and values of many sequences of different lengths in
 * one pool of pages. The source pages describe the cache of a single sequence ("预训练一个 Mini GPT", the sections on
 * the KV cache); pages, the window and the eviction below are this library's extension of it.
 *   pool    [pages][2][Hkv][page][D] bf16: per page the rows of every key head's keys, then of their values
 *   weight  [pages][Hkv][page] fp32 or NULL: per cached row and key head, the attention weight it has received
 *   table   [B][max_pages] int32: row r of sequence b lies in page table[b][r / page] at slot r % page
 * page is a power of two, 8..256. H query heads share Hkv key heads (H a multiple of Hkv): query head h reads key
 * head h / (H / Hkv), H / Hkv <= 128 for the attention. A token's qkv row holds H D queries, Hkv D keys, Hkv D values,
 * as the output of one product (less than 2^30 elements).
 * All arrays are device memory of the current device, pool, qkv and y 16-byte aligned. B <= 8192, max_pages * page <=
 * 2^31 - 4096.
 * GPT_EINVAL: null pointers or sizes; GPT_ECONFIG: D, H % Hkv or alignment. Checked on the device: a page number
 * outside [0, pages) or a row past max_pages * page is neither read nor written, and gptk_status() then returns
 * GPT_EPAGE (what the call wrote for that sequence is unspecified).
 *
 * gptk_paged_store: rows start[b] + t of sequence b take the keys and values of qkv[b][t] ([B, T, (H + 2 Hkv) D])
 * for t < count[b]; their weights become 0. start NULL: 0; count NULL: T (more than T counts as T, less than 0 as 0).
 * No two of the stored rows may share a place.
 */
int gptk_paged_store(const void* qkv, void* pool, float* weight, const int32_t* table, const int32_t* start,
                     const int32_t* count, int32_t B, int32_t T, int32_t H, int32_t Hkv, int32_t D, int32_t pages,
                     int32_t page, int32_t max_pages, void* stream);

/*
 * Attention of one new token per sequence over its cached rows. Sequence b holds rows 0..lens[b]-1; its new token,
 * qkv[b] ([B, (H + 2 Hkv) D]), becomes row n = lens[b] (key and value are stored there), and its queries see the
 * rows r <= n with n - r < window or r < sinks (window 0: all of them):
 *   y[b, h] = sum_r a_r u_r,  a = softmax(q_h . k_r / sqrt(D))     bf16 [B, H D]
 *   lse2[b, h] = log2 sum_r 2^(q_h . k_r log2(e) / sqrt(D))         fp32 [B, H], NULL: not wanted
 *   weight(r, key head) += the sum of a_r over the head's H / Hkv queries (r < n); = that sum for row n
 * lens[b] < 0: no sequence; row b of the outputs, the cache and the weights stay as they were (qkv[b] and the entries of
 * table[b] may be read, and count for nothing). B max_pages page / 32 < 2^31, and times Hkv <= 2^40 (GPT_EINVAL otherwise).
 * The window counts cached rows. An eviction numbers the rows that it keeps anew, so a window over such a cache reaches
 * further back in the text than over a whole one.
 * Scratch (none where the table, or the window and sinks, hold few rows; else about 10 MB and 4 B (H + 1) bytes at most,
 * and with weights 4 B H bytes for each row that the table, or the window and sinks, have room for, whatever the lengths)
 * is taken on the stream from a pool that the library keeps; make a process's first call on a device before any stream
 * capture. The caller counts lens up (one cache per layer shares one lens). Sequences may share the pages of rows below
 * their own; the new rows' pages are their own. fp32 scores and sums; the probabilities enter the product with the values
 * in two bf16 parts (2^-16 of each at most is lost). A NaN in sight makes the outputs and weights of its queries NaN, and
 * so do scores that are all -inf (products past fp32's range; lse2 is -inf then). y overlaps no input.
 */
int gptk_paged_attention(const void* qkv, void* pool, float* weight, const int32_t* table, const int32_t* lens, void* y,
                         float* lse2, int32_t B, int32_t H, int32_t Hkv, int32_t D, int32_t pages, int32_t page,
                         int32_t max_pages, int32_t window, int32_t sinks, void* stream);

/*
 * Eviction by summed attention weight, for every sequence and key head by itself: of rows 0..lens[b]-1 keeps the
 * first `sinks`, the last `recent`, and between them the rows of the largest weight, budget rows in all (every row
 * where lens[b] <= budget; sinks + recent <= budget <= 2^31 - 4096). Equal weights, as after a store alone, which sets
 * them to 0: the lowest rows are kept; a NaN weight counts as the smallest. The kept rows, their weights with them, become
 * rows 0.. of dst_table [B][dst_max_pages] in their order; kept[b][head][i] (int32 [B, Hkv, budget]) is the row that row i
 * was, -1 behind the last; new_lens[b] = min(lens[b], budget) (lens[b] itself where it is negative; new_lens must not be
 * lens). dst_table either is `table`, or starts every sequence with the same pages (in place), or names pages that no
 * sequence of `table` holds, each once; the old rows then stay as they were. In place no page may be held by two sequences.
 */
int gptk_paged_evict(void* pool, float* weight, const int32_t* table, const int32_t* lens, const int32_t* dst_table,
                     int32_t* new_lens, int32_t* kept, int32_t B, int32_t Hkv, int32_t D, int32_t pages, int32_t page,
                     int32_t max_pages, int32_t dst_max_pages, int32_t budget, int32_t sinks, int32_t recent,
                     void* stream);

/* Deterministic mean of nll[0..M) into *loss (device fp32). */
int gptk_mean(const float* nll, int32_t M, float* loss, void* stream);

/*
 * Gives memory of the current device's scratch pool back to the device, down to `keep` bytes. The pool serves the calls
 * above whose comments name it and keeps what they have freed, so that the next call does not map it anew; the largest
 * call's scratch therefore stays with the process until this is called. Only memory of calls that have been waited for
 * is given back (synchronise first); a captured graph's scratch is the graph's own. GPT_OK also where there is no pool.
 */
int gptk_scratch_trim(uint64_t keep);

/* Synchronise the stream, then read and clear the current device's per-step error word. */
int gptk_status(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GPT_GB300_KERNELS_H */
