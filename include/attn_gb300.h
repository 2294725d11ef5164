/*
 * attn_gb300.h -- C ABI of the GB300 (sm_103a) exact-attention library.
 *
 * Exact scaled-dot-product attention computed the
 * FlashAttention way (K/V streamed in tiles past a resident Q tile, running
 * max m and normaliser l, accumulator rescaled by exp(m_old - m_new), the
 * score matrix never written to memory):
 *
 *   attn_fwd / attn_fwd_kvlen -- prefill forward, causal or not, emitting O
 *       and the per-row log-sum-exp.  The method: NanoInfer README ("Flash
 *       Attention v1/v2" bullets and the naive-vs-flash paragraph);
 *       gpu-inference blog, section 02 (online softmax, rescale by
 *       exp(m_old - m_new), log-sum-exp saved, causal mask combined with the
 *       padding mask before the softmax); llm-kernel-lib README, kernel 1
 *       (causal tile skipping); Kernel-Inference-Engine README, the tile-loop
 *       flowchart (Q tile held, K/V tiles streamed, normalise and store).
 *
 *   attn_bwd -- the backward of the prefill forward (dQ, dK, dV from the
 *       saved log-sum-exp; gpu-inference blog, section 02).
 *
 *   paged_attn_decode -- one query token per sequence attending over a KV
 *       cache split into fixed-size pages reached through a page table; the
 *       result equals that of a contiguous cache (inference-kernel-cookbook
 *       README, recipes 02 "KV Cache" and 03 "Paged Attention").  Long
 *       contexts are split into chunks whose partial (m, l, O) are merged by
 *       their log-sum-exp weights in a second pass.
 *
 * Definition computed (per batch b, head h, query row i):
 *   J     = { j < Nkv : j < kv_len[b] and (not causal or j <= i + Nkv - Nq) }
 *   s_j   = scale * <q_i, k_j>
 *   O_i   = sum_J exp(s_j - m) v_j / sum_J exp(s_j - m),   m = max_J s_j
 *   LSE_i = m + ln(sum_J exp(s_j - m))        (natural log, of the scaled scores)
 *   A row with no valid key gets O_i = 0 and LSE_i = -inf.
 *   Causal alignment is bottom-right: with Nq < Nkv the queries are the last
 *   Nq positions of the key sequence.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller, contiguous
 *     row-major.  bf16 tensors are passed as void* (storage of __nv_bfloat16).
 *     Every tensor pointer must be 16-byte aligned.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *     stream).  The library never allocates device memory, never copies
 *     between host and device and never synchronises the stream.
 *   - Host-side checks happen before any launch; on error nothing is launched
 *     and the outputs are untouched.
 *   - Device-resident lengths (kv_lens, ctx_lens, page_table) are not read on
 *     the host.  The kernels clamp lengths to [0, capacity] and treat a page id
 *     outside [0, num_pages) as an unmapped page that holds no token (its keys
 *     are skipped, on every paged entry point alike), so bad values give wrong
 *     numbers, never out-of-bounds accesses.
 *   - Every wait inside a kernel is bounded.  A wait that runs out records
 *     ATTN_ERR_DEVICE_TIMEOUT in a device status word and in a host-visible flag
 *     of that device, and the kernel exits cleanly.  The flag is reported without
 *     synchronising: once it is set, every later call that would launch work on
 *     that device returns ATTN_ERR_DEVICE_TIMEOUT and launches nothing, and
 *     attn_last_device_status() returns it, until attn_check_device_status()
 *     clears it.  (A kernel still running when a call is made has not reported
 *     yet; attn_check_device_status() synchronises first.)
 *   - The first call on each device does a one-time set-up with that device
 *     current: a check of the architecture, the lookup of the status word, the
 *     page-locking of the library's static page of host flags (once per process)
 *     and one small synchronous copy into the status word.  Make that first call
 *     before any stream capture.
 *   - Supported: head dim d in {32, 64, 80, 96, 128} for every entry point
 *     (prefill, decode, KV cache, backward); page_size 16.
 */
#ifndef ATTN_GB300_H
#define ATTN_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t. */
typedef struct CUstream_st *attn_stream_t;

typedef enum {
    ATTN_OK = 0,
    ATTN_ERR_INVALID_ARG = 1,     /* null pointer, non-positive size, size overflow */
    ATTN_ERR_UNSUPPORTED = 2,     /* head dim not supported by the call, page_size != 16, no sm_103 device */
    ATTN_ERR_MISALIGNED = 3,      /* a tensor pointer not 16-byte aligned */
    ATTN_ERR_WORKSPACE = 4,       /* workspace missing, misaligned or too small */
    ATTN_ERR_CUDA = 5,            /* a CUDA runtime/driver call or launch failed */
    ATTN_ERR_DEVICE_TIMEOUT = 6,  /* a bounded in-kernel wait ran out (see attn_check_device_status) */
    ATTN_ERR_SCRATCH_LIMIT = 7    /* paged_attn_decode_noalloc: sizes need more than its fixed scratch */
} attn_status_t;

/*
 * Prefill forward.
 *   q   [B, H, Nq,  d] bf16      k, v [B, H, Nkv, d] bf16
 *   o   [B, H, Nq,  d] bf16 (written, round-to-nearest-even from fp32)
 *   lse [B, H, Nq]     fp32 (written; may be NULL to skip)
 *   causal: 0 or 1 (bottom-right aligned).  scale: multiplier of q.k (e.g. 1/sqrt(d)).
 * Returns ATTN_OK or an attn_status_t error code.
 */
int attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
             int B, int H, int Nq, int Nkv, int d, int causal, float scale,
             attn_stream_t stream);

/*
 * Prefill forward with per-sequence key padding: key j of sequence b is valid
 * only if j < kv_lens[b] (device int32 [B]; NULL means every key is valid).
 * The padding mask applies to every query row and is ANDed with the causal
 * mask.  Other arguments as attn_fwd.
 */
int attn_fwd_kvlen(const void *q, const void *k, const void *v, void *o, float *lse,
                   int B, int H, int Nq, int Nkv, int d, int causal, float scale,
                   const int32_t *kv_lens, attn_stream_t stream);

/*
 * Prefill forward with grouped-query (or multi-query) attention: Hq query heads
 * share Hkv key/value heads, query head h reading key/value head h / (Hq / Hkv)
 * (the MHA / GQA / MQA variants compared in the llm-kernel-lib README's
 * attention ablation).  q, o [B, Hq, Nq, d]; k, v [B, Hkv, Nkv, d]; lse
 * [B, Hq, Nq]; Hq % Hkv == 0 (else ATTN_ERR_INVALID_ARG).  Hkv == Hq is
 * attn_fwd_kvlen.  Other arguments as attn_fwd_kvlen.
 */
int attn_fwd_gqa(const void *q, const void *k, const void *v, void *o, float *lse,
                 int B, int Hq, int Hkv, int Nq, int Nkv, int d, int causal, float scale,
                 const int32_t *kv_lens, attn_stream_t stream);

/*
 * Prefill forward with modified scores and an interval of visible keys per query.  With p_i = i + Nkv -
 * Nq the position of query i among the keys (bottom-right alignment, as the causal mask's):
 *     s_ij = cap tanh(scale <q_i, k_j> / cap) - slope[h] |p_i - j|       (softcap cap > 0)
 *     s_ij = scale <q_i, k_j> - slope[h] |p_i - j|                       (softcap 0: no cap)
 *     J    = { j : key_begin[b, i] <= j < key_end[b, i], 0 <= j < kv_lens[b], j <= p_i if causal }
 * and O, LSE as in attn_fwd_gqa over these scores and keys (no visible key: O = 0, LSE = -inf).
 *   softcap       0, or positive; it and scale / softcap at most 2^100
 *   alibi_slopes  [Hq] fp32 (device), finite; NULL: no distance bias.  With slopes, scale >= 2^-100.  Scores and
 *                 LSE are fp32: a score below its range counts as a key that is not seen, one above it gives NaN
 *   key_begin, key_end [B, Nq] int32 (device): any values, clamped; NULL: 0 and Nkv
 * The intervals say documents packed into a row (begin and end of the query's document), a prefix that
 * every query sees (key_end = max(p_i + 1, prefix), causal 0), a window (key_begin = p_i - window + 1)
 * and their combinations; key tiles that no row of a query tile sees are not visited.  Rows of k and v
 * past kv_lens[b] may hold anything; those below it must be finite.  Other arguments as attn_fwd_gqa.
 */
int attn_fwd_scoremod(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq, int Hkv,
                      int Nq, int Nkv, int d, int causal, float scale, float softcap, const float *alibi_slopes,
                      const int32_t *key_begin, const int32_t *key_end, const int32_t *kv_lens,
                      attn_stream_t stream);

/*
 * Bytes of device workspace paged_attn_decode needs for these sizes (0 on
 * invalid sizes).  The caller allocates it (16-byte aligned) and may reuse it
 * across calls on the same stream; calls that overlap on the GPU need
 * separate workspaces.  The size depends on the page table's capacity,
 * max_pages_per_seq * page_size tokens, because the split grid covers every
 * position the table can address.
 */
size_t paged_attn_decode_workspace_size(int B, int H, int d, int max_pages_per_seq,
                                        int page_size);

/*
 * The same size stated by the longest context: max_ctx_len tokens in 16-token
 * pages, i.e. paged_attn_decode_workspace_size(B, H, d, ceil(max_ctx_len / 16),
 * 16).  Pass the capacity of the table the decode will get (max_pages_per_seq *
 * 16), which is at least the longest context.
 */
size_t paged_attn_decode_workspace_size_ctx(int B, int H, int d, int max_ctx_len);

/*
 * Workspace of paged_attn_decode_gqa and paged_attn_decode_fp8 for H query heads
 * over Hkv cache heads.  Groups of two or more query heads run longer splits
 * (1024 tokens instead of 512) and need about half the multi-head size; the
 * multi-head size is always enough.
 */
size_t paged_attn_decode_gqa_workspace_size(int B, int H, int Hkv, int d, int max_pages_per_seq,
                                            int page_size);

/*
 * Paged-KV decode: one query per sequence over its cached tokens.
 *   q          [B, H, d] bf16
 *   k_pages    [num_pages, H, page_size, d] bf16 (one page of one head is a
 *   v_pages     contiguous page_size x d block)
 *   page_table [B, max_pages_per_seq] int32: physical page of logical page p of
 *              sequence b; token t of b is slot t % page_size of page
 *              page_table[b][t / page_size]
 *   ctx_lens   [B] int32: number of cached tokens of each sequence (the query
 *              attends to all of them; clamped to [0, max_pages_per_seq*page_size])
 *   o          [B, H, d] bf16 (written)      lse [B, H] fp32 (written; may be NULL)
 *   workspace  device scratch of at least paged_attn_decode_workspace_size() bytes
 */
int paged_attn_decode(const void *q, const void *k_pages, const void *v_pages,
                      const int32_t *page_table, const int32_t *ctx_lens, int page_size,
                      void *o, float *lse, int B, int H, int d, int max_pages_per_seq,
                      int num_pages, float scale, void *workspace, size_t workspace_bytes,
                      attn_stream_t stream);

/*
 * Paged decode with grouped-query attention: the cache has Hkv heads
 * (k_pages, v_pages [num_pages, Hkv, page_size, d]) shared by the H query heads
 * (q, o [B, H, d]; lse [B, H]); query head h reads cache head h / (H / Hkv), and
 * each cache page is read once for all the query heads that share it.  H % Hkv
 * must be 0.  The workspace is sized by paged_attn_decode_gqa_workspace_size(B,
 * H, Hkv, ...) with H the number of query heads.  Other arguments as
 * paged_attn_decode.
 */
int paged_attn_decode_gqa(const void *q, const void *k_pages, const void *v_pages,
                          const int32_t *page_table, const int32_t *ctx_lens, int page_size,
                          void *o, float *lse, int B, int H, int Hkv, int d, int max_pages_per_seq,
                          int num_pages, float scale, void *workspace, size_t workspace_bytes,
                          attn_stream_t stream);

/*
 * Paged decode with modified scores (paged_attn_decode_gqa with the modification of attn_fwd_scoremod for
 * one query at position ctx_lens[b] - 1, the length clamped to the table's capacity as there):
 *     s_j = cap tanh(scale <q, k_j> / cap) - slope[h] (ctx_lens[b] - 1 - j)      (softcap cap > 0)
 *     s_j = scale <q, k_j> - slope[h] (ctx_lens[b] - 1 - j)                      (softcap 0)
 * over the cached tokens key_begin[b] <= j < ctx_lens[b].
 *   softcap 0, or positive; alibi_slopes [H] fp32 (finite) or NULL; key_begin [B] int32 (clamped) or NULL.
 *     Bounds as in attn_fwd_scoremod, of scale * k_scale in place of scale over an e4m3 cache
 *   workspace: at least paged_attn_decode_scoremod_workspace_size(...) bytes, 16-byte aligned
 *   max_pages_per_seq: the work is cut by the table's width, since the lengths are on the device; a table much wider
 *     than the contexts costs time (2 short sequences: 4.5 us at up to 2048 columns, 11 at 8192) and workspace
 * Pages wholly before key_begin are not read, and slots of the first page before it may hold anything.
 * A sequence that sees no token gets O = 0 and LSE = -inf.  Other arguments as paged_attn_decode_gqa;
 * _fp8: over an e4m3 cache, as paged_attn_decode_fp8.
 */
size_t paged_attn_decode_scoremod_workspace_size(int B, int H, int Hkv, int d, int max_pages_per_seq,
                                                 int page_size);

int paged_attn_decode_scoremod(const void *q, const void *k_pages, const void *v_pages,
                               const int32_t *page_table, const int32_t *ctx_lens, int page_size, void *o,
                               float *lse, int B, int H, int Hkv, int d, int max_pages_per_seq, int num_pages,
                               float scale, float softcap, const float *alibi_slopes, const int32_t *key_begin,
                               void *workspace, size_t workspace_bytes, attn_stream_t stream);

int paged_attn_decode_scoremod_fp8(const void *q, const void *k_pages, const void *v_pages, float k_scale,
                                   float v_scale, const int32_t *page_table, const int32_t *ctx_lens,
                                   int page_size, void *o, float *lse, int B, int H, int Hkv, int d,
                                   int max_pages_per_seq, int num_pages, float scale, float softcap,
                                   const float *alibi_slopes, const int32_t *key_begin, void *workspace,
                                   size_t workspace_bytes, attn_stream_t stream);

/*
 * Paged decode of a batch whose groups of sequences share their first pages (samples of one prompt, users
 * behind one system prompt or document): paged_attn_decode_gqa, with the shared pages read once per group
 * (or once per sequence, from L2, where that is faster: small batches).
 *   group_size    the batch is B / group_size groups of consecutive sequences (B % group_size == 0); pad a
 *                 shorter group with sequences of ctx_lens 0
 *   shared_pages  [B / group_size] int32 (device, clamped to [0, max_pages_per_seq]): the first
 *                 shared_pages[g] entries of page_table are the same for every sequence of group g, and
 *                 are read from the row of its FIRST sequence (b = g * group_size); those entries of its
 *                 other rows are not read
 * Sequence b still attends to its first ctx_lens[b] tokens, which may end inside the shared pages.  The
 * later pages of each sequence are its own.  The work is cut by the table's width here too (4 samples of 576
 * tokens: 5.2 us at up to 512 columns, 15.5 from 2048 on).  Unmapped ids, empty sequences, o and lse as in
 * paged_attn_decode_gqa.  workspace: at least paged_attn_decode_shared_workspace_size(...) bytes, 16-byte
 * aligned.  _fp8: over an e4m3 cache, as paged_attn_decode_fp8.
 */
size_t paged_attn_decode_shared_workspace_size(int B, int H, int Hkv, int d, int max_pages_per_seq,
                                               int group_size, int page_size);

int paged_attn_decode_shared(const void *q, const void *k_pages, const void *v_pages,
                             const int32_t *page_table, const int32_t *ctx_lens, const int32_t *shared_pages,
                             int group_size, int page_size, void *o, float *lse, int B, int H, int Hkv, int d,
                             int max_pages_per_seq, int num_pages, float scale, void *workspace,
                             size_t workspace_bytes, attn_stream_t stream);

int paged_attn_decode_shared_fp8(const void *q, const void *k_pages, const void *v_pages, float k_scale,
                                 float v_scale, const int32_t *page_table, const int32_t *ctx_lens,
                                 const int32_t *shared_pages, int group_size, int page_size, void *o, float *lse,
                                 int B, int H, int Hkv, int d, int max_pages_per_seq, int num_pages, float scale,
                                 void *workspace, size_t workspace_bytes, attn_stream_t stream);

/*
 * Chunked prefill over the paged KV cache (a prefill step writing into, then
 * attending over, a KV cache kept in pages: inference-kernel-cookbook README,
 * recipes 02 and 03).  Sequence b holds ctx_lens[b] tokens (device int32 [B],
 * clamped to [0, max_pages_per_seq * page_size]) in its pages; the Nq queries
 * q[b, :, i] are its LAST Nq positions (ctx_lens[b] - Nq + i), so with causal = 1
 * query i sees keys j <= i + ctx_lens[b] - Nq (bottom-right), and every query sees
 * only keys j < ctx_lens[b].  The new tokens' K/V must already be in the pages
 * (paged_kv_append).
 *   q, o [B, H, Nq, d] bf16; lse [B, H, Nq] fp32 (may be NULL)
 *   k_pages, v_pages [num_pages, Hkv, page_size, d] bf16; page_table [B, max_pages_per_seq]
 *   H % Hkv == 0 (grouped-query heads as attn_fwd_gqa); page_size 16; d in {32, 64, 80, 96, 128}.
 * A page id outside [0, num_pages) is an unmapped page, as in decode: the positions
 * it covers hold no token (their keys are masked out; the other positions keep their
 * places, so the causal alignment is unchanged), and a query that sees no mapped key
 * gets O = 0 and LSE = -inf.  Slots of the last page past ctx_lens[b] may hold anything.
 * Runs on the same tcgen05 pipeline as attn_fwd, with each 128-key tile gathered page by
 * page through TMA.
 */
int paged_attn_prefill(const void *q, const void *k_pages, const void *v_pages,
                       const int32_t *page_table, const int32_t *ctx_lens, int page_size,
                       void *o, float *lse, int B, int H, int Hkv, int Nq, int d,
                       int max_pages_per_seq, int num_pages, int causal, float scale,
                       attn_stream_t stream);

/*
 * Appends the K/V of Nnew new tokens to the paged cache: token t of sequence b
 * goes to position p = start_pos[b] + t, i.e. page page_table[b][p / page_size],
 * slot p % page_size, for every key/value head.
 *   k_new, v_new [B, Hkv, Nnew, d] bf16; k_pages, v_pages [num_pages, Hkv, page_size, d]
 *   start_pos [B] int32 (device; tokens already in the cache before this append)
 * Positions past max_pages_per_seq * page_size and page ids outside [0, num_pages)
 * are skipped (nothing written).  The caller reserves the pages in the table.
 */
int paged_kv_append(const void *k_new, const void *v_new, void *k_pages, void *v_pages,
                    const int32_t *page_table, const int32_t *start_pos, int page_size,
                    int B, int Hkv, int Nnew, int d, int max_pages_per_seq, int num_pages,
                    attn_stream_t stream);

/*
 * paged_kv_append with rotary position embedding on the way: the new tokens' queries and keys are
 * rotated to their positions, keys and values go to the pages, the rotated queries to q_out.  Token t
 * of sequence b sits at position p = max(start_pos[b], 0) + t.  The first rope_dim dims of a query or
 * key row are rope_dim / 2 pairs (x, y) -- dims (i, i + rope_dim / 2), or (2i, 2i + 1) when
 * interleaved is 1 -- and
 *     x' = x cos[p][i] - y sin[p][i],   y' = y cos[p][i] + x sin[p][i];
 * the other dims and the values are copied.  Computed in fp32 and rounded once.
 *   q [B, H, Nnew, d], k_new, v_new [B, Hkv, Nnew, d] bf16; *_strides: HOST arrays of three strides
 *     {batch, head, token} in elements (the last dim is contiguous), non-negative multiples of 8, so
 *     views of a fused [B, Nnew, (H + 2 Hkv) d] projection need no copy; NULL means contiguous
 *   q and q_out may both be NULL (keys and values only; H is then ignored)
 *   q_out [B, H, Nnew, d] bf16, contiguous; may be q itself if q is contiguous, else must not
 *     overlap an input
 *   cos_sin [max_pos, rope_dim] fp32: row p holds cos of its rope_dim / 2 pairs, then their sin
 *   rope_dim: a multiple of 16, at most d
 *   start_pos [B] int32; new_lens [B] int32 (may be NULL: Nnew each): tokens t >= new_lens[b] are
 *     padding.  Of padding, and of tokens at positions >= max_pos, nothing is written at all.
 * Keys and values of positions past the page table's capacity and of page ids outside [0, num_pages)
 * are skipped as in paged_kv_append; their queries are still rotated.  Two tokens of one call must
 * not map to the same page slot.  d in {32, 64, 80, 96, 128}, page_size 16.
 * paged_kv_append_rope_fp8: into an e4m3 cache (see below), the rotated fp32 key times 1 / k_scale
 * rounded once to e4m3.
 */
int paged_kv_append_rope(const void *q, const int64_t *q_strides, const void *k_new, const int64_t *k_strides,
                         const void *v_new, const int64_t *v_strides, void *q_out, void *k_pages, void *v_pages,
                         const float *cos_sin, int rope_dim, int max_pos, int interleaved,
                         const int32_t *page_table, const int32_t *start_pos, const int32_t *new_lens,
                         int page_size, int B, int H, int Hkv, int Nnew, int d, int max_pages_per_seq,
                         int num_pages, attn_stream_t stream);

int paged_kv_append_rope_fp8(const void *q, const int64_t *q_strides, const void *k_new, const int64_t *k_strides,
                             const void *v_new, const int64_t *v_strides, void *q_out, void *k_pages, void *v_pages,
                             float k_scale, float v_scale, const float *cos_sin, int rope_dim, int max_pos,
                             int interleaved, const int32_t *page_table, const int32_t *start_pos,
                             const int32_t *new_lens, int page_size, int B, int H, int Hkv, int Nnew, int d,
                             int max_pages_per_seq, int num_pages, attn_stream_t stream);

/*
 * FP8 KV cache.  The NanoInfer README's roadmap names FP8 e4m3 storage (cuda_fp8.h
 * __nv_fp8_e4m3) as the successor of INT8 with the quantisation math unchanged;
 * here it is the storage of the paged KV cache, which halves the bytes a decode
 * step reads.  A cache tensor holds E4M3 codes (1 sign, 4 exponent bits with bias
 * 7, 3 mantissa bits, no infinities, largest finite 448) with one scale per
 * tensor:  value = e4m3(code) * scale.  Conversion from bf16:
 *   code = e4m3 nearest-even rounding of fp32(x) * fp32(1 / scale), saturating at
 *          +-448 (1 / scale is computed in fp32 on the host).
 *
 * paged_attn_prefill_fp8: paged_attn_prefill over an e4m3 cache (k_pages, v_pages
 *   [num_pages, Hkv, page_size, d] uint8 codes; k_scale, v_scale > 0 and finite): the
 *   chunked prefill of a serving loop that keeps its cache in e4m3.  q, o, lse, the
 *   table, the masks and the result are as in paged_attn_prefill, for the dequantised
 *   cache.  The codes are widened exactly to f16 in shared memory and both products run
 *   in f16 with fp32 accumulation: each query row is rounded to f16 after a power-of-two
 *   factor of its own, which keeps it below 2^15 and its largest value from 2^-7 on (exact
 *   but for values under f16's normal range, off by 2^-18 of the row's largest at most).
 *   The key scale multiplies the scores and the value scale the output.
 * paged_attn_decode_fp8: paged_attn_decode_gqa over an e4m3 cache (k_pages,
 *   v_pages [num_pages, Hkv, page_size, d] uint8 codes; k_scale, v_scale > 0
 *   and finite).  q, o, lse, the table, the workspace and the result are as in
 *   paged_attn_decode_gqa, for the dequantised cache.  The codes are widened exactly
 *   to f16 or fp32; where the products run on tensor cores they run in f16 with fp32
 *   accumulation, the query rounded to f16 after a power-of-two factor as above.
 * kv_quantize_fp8: n contiguous bf16 elements of src -> n codes in dst (n a
 *   multiple of 8; both 16-byte aligned).  Converts a whole bf16 page pool.
 * paged_kv_append_fp8: paged_kv_append into an e4m3 cache, converting each new
 *   element with the tensor's scale.
 */
int paged_attn_decode_fp8(const void *q, const void *k_pages, const void *v_pages, float k_scale,
                          float v_scale, const int32_t *page_table, const int32_t *ctx_lens,
                          int page_size, void *o, float *lse, int B, int H, int Hkv, int d,
                          int max_pages_per_seq, int num_pages, float scale, void *workspace,
                          size_t workspace_bytes, attn_stream_t stream);

int paged_attn_prefill_fp8(const void *q, const void *k_pages, const void *v_pages, float k_scale,
                           float v_scale, const int32_t *page_table, const int32_t *ctx_lens,
                           int page_size, void *o, float *lse, int B, int H, int Hkv, int Nq, int d,
                           int max_pages_per_seq, int num_pages, int causal, float scale,
                           attn_stream_t stream);

int kv_quantize_fp8(const void *src, void *dst, size_t n, float scale, attn_stream_t stream);

int paged_kv_append_fp8(const void *k_new, const void *v_new, void *k_pages, void *v_pages,
                        float k_scale, float v_scale, const int32_t *page_table,
                        const int32_t *start_pos, int page_size, int B, int Hkv, int Nnew, int d,
                        int max_pages_per_seq, int num_pages, attn_stream_t stream);

/*
 * 4-bit KV cache.  A value is e2m1(code) * e4m3(block scale) * the tensor's scale: a 4-bit code (1 sign, 2 exponent bits
 * of bias 1, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) and one e4m3 scale per block of 16 dims of a token.  k_pages,
 * v_pages are [num_pages, Hkv, 9 d] bytes; the 9 d bytes of a page of a head are, with token t of 0 .. 15 and dim x,
 *   keys    the code of (t, x) in byte t d / 2 + x / 2, low nibble for even x; the scale of (t, block j) in byte
 *           8 d + t d / 16 + j
 *   values  with q = (t mod 8) / 2 and h = t / 8, the code of (t, x) in byte 128 (x / 16) + 32 q + 16 h + x mod 16, low nibble
 *           for even t; the scale of (t, block j) in byte 8 d + q d / 4 + 4 j + 2 h + t mod 2
 * (all divisions whole).  k_scale, v_scale lie in [1e-37, 1e37].  d and page_size as everywhere.
 *
 * paged_kv_append_fp4: new tokens into such a cache, optionally rotated on the way.  cos_sin NULL: keys and values as they
 *   are (q must be NULL).  Else as paged_kv_append_rope (positions NULL: token t turns by row start_pos[b] + t) or as
 *   paged_kv_append_rope_axes (positions [n_axes, B, Nnew]).  With u = fp32(x * fp32(1 / scale)) of a block (x in fp32,
 *   after the rotation): the block scale is e4m3(fp32(max |u| * fp32(1/6))), nearest-even and at most 448, a code is
 *   e2m1(fp32(u / block scale)), nearest-even and at most 6, and 0 in a block whose scale is 0.  Inputs must be finite.
 *   Tokens at positions 2m and 2m + 1 share bytes: no two sequences of a call may write to the same page.
 * paged_kv_unpack_fp4: pages page_ids[i] (n of them, device) as bf16, k_out and v_out [n, Hkv, 16, d]: fp32(code * block
 *   scale) * scale, rounded to bf16.  An id outside [0, num_pages) leaves out[i] as it was.  With a table of the places i
 *   paged_attn_prefill attends over the result: the chunked prefill over a 4-bit cache.
 * paged_attn_decode_fp4: paged_attn_decode_scoremod over such a cache (softcap 0, alibi_slopes and key_begin NULL: the plain
 *   decode).  The codes are widened exactly to f16, both products run in f16 with fp32 accumulation (each query rounded to
 *   f16 after a power of two of its own, the weights to f16: by 2^-11 of each, under 2^-21 of
 *   the row's largest by 2^-32 of that).  Slots that a query does not see may hold anything.
 *   scale * k_scale lies in [1e-37, 1e37] too.
 *   workspace: at least paged_attn_decode_fp4_workspace_size(...) bytes.
 */
size_t paged_attn_decode_fp4_workspace_size(int B, int H, int Hkv, int d, int max_pages_per_seq, int page_size);

int paged_attn_decode_fp4(const void *q, const void *k_pages, const void *v_pages, float k_scale, float v_scale,
                          const int32_t *page_table, const int32_t *ctx_lens, int page_size, void *o, float *lse, int B,
                          int H, int Hkv, int d, int max_pages_per_seq, int num_pages, float scale, float softcap,
                          const float *alibi_slopes, const int32_t *key_begin, void *workspace, size_t workspace_bytes,
                          attn_stream_t stream);

int paged_kv_append_fp4(const void *q, const int64_t *q_strides, const void *k_new, const int64_t *k_strides,
                        const void *v_new, const int64_t *v_strides, void *q_out, void *k_pages, void *v_pages,
                        float k_scale, float v_scale, const float *cos_sin, int rope_dim, int max_pos, int interleaved,
                        const int32_t *positions, int n_axes, const uint8_t *pair_axis, const int32_t *page_table,
                        const int32_t *start_pos, const int32_t *new_lens, int page_size, int B, int H, int Hkv, int Nnew,
                        int d, int max_pages_per_seq, int num_pages, attn_stream_t stream);

int paged_kv_unpack_fp4(const void *k_pages, const void *v_pages, float k_scale, float v_scale, const int32_t *page_ids,
                        int n, void *k_out, void *v_out, int page_size, int Hkv, int d, int num_pages,
                        attn_stream_t stream);

/*
 * Rotary positions with several axes (time, height and width of an image's or a video's tokens; equal ones for text).
 *   positions  [n_axes, B, N] int32 (device), n_axes 1 to 4
 *   pair_axis  HOST array of rope_dim / 2 entries < n_axes: pair i of a token turns by column i of row
 *              positions[pair_axis[i]][b][t] of cos_sin, so sections of the pairs, axes taken in turn, and frequencies that
 *              start again for each axis are all a matter of this array and the table's columns
 * and the pairs, cos_sin, rope_dim and interleaved as in paged_kv_append_rope.
 *
 * paged_kv_append_rope_axes(_fp8): paged_kv_append_rope with such positions; start_pos says only where in the cache the
 *   tokens go.  Of a token with a position outside [0, max_pos) nothing is written.
 * attn_rope_axes: the rotation alone.  q [B, H, N, d], k [B, Hkv, N, d] (k and k_out may both be NULL; Hkv is then ignored)
 *   and their outputs are bf16 views with contiguous rows, *_strides as in paged_kv_append_rope; an output may be its input
 *   (the same strides), and must else not overlap an input or the other output.  An output whose own rows overlap (a stride of
 *   0, or one that does not step past what the smaller ones reach) is refused.  positions_batch: B, or 1 for positions [n_axes, 1, N] that all
 *   sequences share.  A token with a position outside [0, max_pos) gives zeros.
 * attn_rope_axes_bwd: its gradient: dq, dk are those of the outputs, q_out and k_out get those of q and k (the transposed
 *   rotation; zeros for tokens outside the table).
 */
int paged_kv_append_rope_axes(const void *q, const int64_t *q_strides, const void *k_new, const int64_t *k_strides,
                              const void *v_new, const int64_t *v_strides, void *q_out, void *k_pages, void *v_pages,
                              const float *cos_sin, int rope_dim, int max_pos, int interleaved, const int32_t *positions,
                              int n_axes, const uint8_t *pair_axis, const int32_t *page_table, const int32_t *start_pos,
                              const int32_t *new_lens, int page_size, int B, int H, int Hkv, int Nnew, int d,
                              int max_pages_per_seq, int num_pages, attn_stream_t stream);

int paged_kv_append_rope_axes_fp8(const void *q, const int64_t *q_strides, const void *k_new, const int64_t *k_strides,
                                  const void *v_new, const int64_t *v_strides, void *q_out, void *k_pages, void *v_pages,
                                  float k_scale, float v_scale, const float *cos_sin, int rope_dim, int max_pos,
                                  int interleaved, const int32_t *positions, int n_axes, const uint8_t *pair_axis,
                                  const int32_t *page_table, const int32_t *start_pos, const int32_t *new_lens,
                                  int page_size, int B, int H, int Hkv, int Nnew, int d, int max_pages_per_seq,
                                  int num_pages, attn_stream_t stream);

int attn_rope_axes(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides, const float *cos_sin,
                   int rope_dim, int max_pos, int interleaved, const int32_t *positions, int n_axes, int positions_batch,
                   const uint8_t *pair_axis, void *q_out, const int64_t *q_out_strides, void *k_out,
                   const int64_t *k_out_strides, int B, int H, int Hkv, int N, int d, attn_stream_t stream);

int attn_rope_axes_bwd(const void *dq, const int64_t *dq_strides, const void *dk, const int64_t *dk_strides,
                       const float *cos_sin, int rope_dim, int max_pos, int interleaved, const int32_t *positions,
                       int n_axes, int positions_batch, const uint8_t *pair_axis, void *q_out, const int64_t *q_out_strides,
                       void *k_out, const int64_t *k_out_strides, int B, int H, int Hkv, int N, int d,
                       attn_stream_t stream);

/*
 * Page tables and reference counts of a cache, on the device throughout: no call reads them on the host, so all may be
 * captured into a graph.
 *   page_table [B, max_pages_per_seq], ctx_lens [B] int32 as everywhere; entries outside [0, num_pages) (-1) name no page
 *   ref_counts [num_pages] int32: how many entries of the table name each page (a caller may add its own).  A page is free
 *              iff its count is not positive.
 * A table has at most 2^30 entries, a pool at most 2^30 pages.
 * Which page goes where follows from the order of rows and page numbers alone.  Outputs must not overlap inputs but where it
 * says that an output may be its input.
 *
 * paged_kv_fork: row b of the result continues row parents[b] of the table (b < B_out, parents [B_out] int32): the entries of
 *   its ceil(ctx_lens / 16) pages, the others -1; parents[b] == b keeps the whole row as it is, parents[b] outside [0, B)
 *   gives an empty one.  A row of the table that no row continues is thereby freed.  ref_counts_out (may be ref_counts): the
 *   counts plus the new table's entries less the old one's.
 * paged_kv_reserve: makes the entries that cover positions ctx_lens[b] .. ctx_lens[b] + new_lens[b] - 1 the row's own: an
 *   entry that names no page gets a free one, and so does one whose page has a count over 1 at the call's start (it is
 *   shared).  So of S rows that share a page and all write into it each gets one of its own, and the shared one is left with
 *   S counts less (free, if no one else holds it): what a row needs does not hang on whether another row is served.  Free
 *   pages are given out in ascending order, to rows and entries in ascending order.  A row that needs more
 *   pages than rows before it leave, or more entries than the table has, is left as it is; the former rows' needs count for
 *   the rows after them, the latter's do not.
 *     reserved [B]: new_lens[b] if the row can take its tokens, else 0 (and 0 where new_lens[b] <= 0), which is what the
 *       append takes as new_lens
 *     src_pages, dst_pages [B]: where ctx_lens[b] ends inside a page that was shared, that page and the row's new one, into
 *       which paged_kv_copy_pages is to copy it; else -1
 *     page_table_out, ref_counts_out (may be the inputs); counts 16-byte aligned
 *     workspace: at least paged_kv_reserve_workspace_size(B, num_pages) bytes, 16-byte aligned
 * paged_kv_compact: with L live pages (count positive), moves those at ids >= L, in order, to the free ids < L, in order.
 *   src_pages, dst_pages [num_pages]: the moves, then -1; count [1]: how many.  page_table_out (may be page_table) names
 *   the pages' new places, and -1 where an entry names no live page; ref_counts_out (not ref_counts) their counts, both
 *   counts 16-byte aligned.  workspace: at least paged_kv_compact_workspace_size(num_pages) bytes, 16-byte aligned.
 * paged_kv_copy_pages: page dst_pages[i] of each pool becomes a copy of page src_pages[i], for i < n and, if count (device
 *   [1], may be NULL) is given, i < count[0].  pools: HOST array of n_pools device pointers, each to num_pages pages of
 *   page_bytes contiguous bytes (a multiple of 16; keys and values of every layer).  Pairs with an id outside the pool are
 *   skipped.  No page may be the destination of two pairs, or the destination of one and the source of another.
 */
int paged_kv_fork(const int32_t *page_table, const int32_t *ctx_lens, const int32_t *parents, const int32_t *ref_counts,
                  int32_t *page_table_out, int32_t *ctx_lens_out, int32_t *ref_counts_out, int page_size, int B, int B_out,
                  int max_pages_per_seq, int num_pages, attn_stream_t stream);

size_t paged_kv_reserve_workspace_size(int B, int num_pages);

int paged_kv_reserve(const int32_t *page_table, const int32_t *ctx_lens, const int32_t *new_lens,
                     const int32_t *ref_counts, int32_t *page_table_out, int32_t *ref_counts_out, int32_t *reserved,
                     int32_t *src_pages, int32_t *dst_pages, int page_size, int B, int max_pages_per_seq, int num_pages,
                     void *workspace, size_t workspace_bytes, attn_stream_t stream);

size_t paged_kv_compact_workspace_size(int num_pages);

int paged_kv_compact(const int32_t *page_table, const int32_t *ref_counts, int32_t *page_table_out,
                     int32_t *ref_counts_out, int32_t *src_pages, int32_t *dst_pages, int32_t *count, int B,
                     int max_pages_per_seq, int num_pages, void *workspace, size_t workspace_bytes, attn_stream_t stream);

int paged_kv_copy_pages(void *const *pools, int n_pools, size_t page_bytes, const int32_t *src_pages,
                        const int32_t *dst_pages, const int32_t *count, int n, int num_pages, attn_stream_t stream);

/*
 * Backward of attn_fwd_gqa: gradients of the loss with respect to q, k and v
 * given its gradient dout with respect to the forward output.  The method
 * (gpu-inference blog, section 02 "FlashAttention-2 in Triton"): the
 * probabilities are recomputed tile by tile from the forward's log-sum-exp
 * instead of being stored, and the work is three kernels -- the row term
 * D_i = dO_i . O_i, a dK/dV kernel and a dQ kernel.  With P_ij = exp(s_ij -
 * LSE_i) on the valid keys (0 elsewhere), dP = dO V^T and dS = P * (dP - D):
 *   dV = P^T dO,   dK = scale dS^T Q,   dQ = scale dS K;
 * for grouped-query heads dK and dV of a key/value head sum over the query
 * heads that read it.  A row with no valid key contributes nothing.
 *   q, o, dout, dq [B, Hq, Nq, d] bf16    k, v, dk, dv [B, Hkv, Nkv, d] bf16
 *   lse [B, Hq, Nq] fp32: the forward's log-sum-exp (natural log), required
 *   o: the forward's output for these inputs (used only for D)
 *   kv_lens, causal, scale, Hq % Hkv == 0: exactly as in the forward call
 *   workspace: device scratch of at least attn_bwd_workspace_size(B, Hq, Nq)
 *       bytes, 16-byte aligned; it holds D [B, Hq, Nq] fp32 when the call ends.
 * dq, dk and dv are fully written (rows past a sequence's key length get zero
 * dk/dv).  Products run on bf16 operands with fp32 accumulation: P and dS are
 * rounded to bf16 before they multiply dO, Q and K.  d in {32, 64, 80, 96, 128}.
 */
size_t attn_bwd_workspace_size(int B, int Hq, int Nq);

int attn_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
             const void *dout, void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int Nq,
             int Nkv, int d, int causal, float scale, const int32_t *kv_lens, void *workspace,
             size_t workspace_bytes, attn_stream_t stream);

/*
 * Backward of attn_fwd_scoremod: as attn_bwd for the modified scores.  With t_ij = tanh(scale <q_i, k_j> /
 * cap) the gradient of the modified score, dS = P * (dP - D), times 1 - t_ij^2 is that of scale <q_i, k_j>:
 *     dV = P^T dO,   dK = scale (dS (1 - t^2))^T Q,   dQ = scale (dS (1 - t^2)) K
 * (without the cap the factor is 1; the slopes and the intervals get no gradient).
 *   lse, o: attn_fwd_scoremod's for the same inputs and modification; dout finite.  The weights are exp(s - LSE)
 *     with LSE in fp32: a row whose |LSE| passes 2^16 (steep slopes, no key near the query) has gradients off by
 *     |LSE| 2^-24 of themselves and more
 *   workspace: at least attn_bwd_scoremod_workspace_size(B, Hq, Hkv, Nq, Nkv, d) bytes, 16-byte aligned
 * Rows of k and v past kv_lens[b] may hold anything; dk and dv get zeros there.  Other arguments as
 * attn_bwd and attn_fwd_scoremod.
 */
size_t attn_bwd_scoremod_workspace_size(int B, int Hq, int Hkv, int Nq, int Nkv, int d);

int attn_bwd_scoremod(const void *q, const void *k, const void *v, const void *o, const float *lse,
                      const void *dout, void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int Nq, int Nkv,
                      int d, int causal, float scale, float softcap, const float *alibi_slopes,
                      const int32_t *key_begin, const int32_t *key_end, const int32_t *kv_lens, void *workspace,
                      size_t workspace_bytes, attn_stream_t stream);

/*
 * paged_attn_decode for callers that cannot allocate device memory.  The pages
 * describe no such variant; it exists for callers such as code running inside
 * a memory pool or allocator callback (where a nested cudaMalloc is not
 * allowed), serving loops that must not block on the allocator or risk an
 * out-of-memory failure in the middle of a step, and hosts that can only pass
 * the input and output buffers they already own.
 *
 * Arguments, layouts and results are those of paged_attn_decode without the
 * workspace: the chunk partials live in a fixed 12 MiB array inside the
 * library's device memory (every GPU that loads the library holds it until the
 * process exits).  Sizes whose workspace (paged_attn_decode_workspace_size)
 * exceeds 12 MiB are rejected with ATTN_ERR_SCRATCH_LIMIT before anything is
 * launched.  No call allocates or frees memory.
 *
 * The first call on each device looks up the array's device address (with that
 * device current); make that first call before any stream capture.  All calls
 * share the one array: calls that may overlap on the GPU (other streams, other
 * host threads) race on it and must be ordered by the caller.  A call that
 * completes normally writes every part of the array it later reads, so what an
 * earlier call left there does not reach its result.  A call whose bounded wait
 * runs out (ATTN_ERR_DEVICE_TIMEOUT) is different: the split that gave up does
 * not write its partial, and the merge may then read an earlier call's partial
 * from the array, so that call's O and LSE are invalid (as the status says).
 */
int paged_attn_decode_noalloc(const void *q, const void *k_pages, const void *v_pages,
                              const int32_t *page_table, const int32_t *ctx_lens, int page_size,
                              void *o, float *lse, int B, int H, int d, int max_pages_per_seq,
                              int num_pages, float scale, attn_stream_t stream);

/*
 * Synchronises `stream`, then returns and clears the current device's status
 * (the device word and the host-visible flag): ATTN_OK,
 * ATTN_ERR_DEVICE_TIMEOUT if a kernel's bounded wait ran out since the last
 * check, or ATTN_ERR_CUDA if the synchronisation itself failed.  After it the
 * other entry points launch work again.
 */
int attn_check_device_status(attn_stream_t stream);

/*
 * The current device's host-visible timeout flag, read without synchronising
 * and without clearing it: ATTN_ERR_DEVICE_TIMEOUT if a kernel that has already
 * reached its timeout path recorded one since the last attn_check_device_status(),
 * else ATTN_OK.  The same condition makes the launching entry points return
 * ATTN_ERR_DEVICE_TIMEOUT.  (The op sequence of the Kernel-Inference-Engine
 * README reads the error state right after a launch, with no host round trip;
 * this is that check for the asynchronous in-kernel timeouts.)
 */
int attn_last_device_status(void);

/*
 * Self-test of the failure detection: launches one block whose only thread waits
 * on an mbarrier that nothing arrives on.  The wait gives up after its limit
 * (about two seconds), records ATTN_ERR_DEVICE_TIMEOUT in the device status word
 * and the kernel returns normally, so the CUDA context stays usable.  The next
 * attn_check_device_status() on this stream returns ATTN_ERR_DEVICE_TIMEOUT.
 * Returns ATTN_OK if the launch succeeded.
 */
int attn_selftest_bounded_wait(attn_stream_t stream);

/* Static, human-readable text for a status code. */
const char *attn_status_string(int status);

/* Library version as "major.minor.patch" (static string). */
const char *attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_GB300_H */
