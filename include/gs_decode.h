/*
 * gs_decode.h -- C ABI of the decode operators for GB300 (sm_103a): a paged key-value
 * cache, attention of one new token over it, and guided logits.
 *
 * A token generator is guided like a diffusion model: two branches of every sample
 * (uncond and cond) give two outputs, pred = uncond + s (cond - uncond), with s from the
 * bucket table (gs_bucket_plan; [BCG] sections 2-4).  Here the outputs are logits, and
 * each branch keeps a cache of its keys and values.  One step of a batch is
 *   gs_pages_extend        room for the new token of every branch (once a step),
 *   gs_paged_attention     per layer: store the new token's K and V, attend over the cache,
 *   gs_guided_logits       the two branches' logits -> the next token.
 * gs_pages_fork starts the uncond branch (or further samples) from a shared prompt,
 * gs_pages_free returns finished branches' pages, gs_pages_compact makes a pool dense,
 * gs_kv_write stores prompts.  All state (tables, lengths, counts) is on the device:
 * no call reads it on the host, so a step can be captured in a CUDA graph and replayed.
 *
 * Conventions are those of gs.h: the caller owns every buffer, nothing is allocated and
 * nothing synchronises; work goes on the caller's stream; argument errors are returned
 * before any launch; what only the device can see is OR-ed into an optional status word.
 * Every kernel is launched with programmatic dependent launch and waits for the stream's
 * earlier work before it touches memory.  Calls that share a cache or a workspace are
 * ordered by the caller (one stream, or events).
 */
#ifndef GS_DECODE_H
#define GS_DECODE_H

#include "gs.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits of the device status word beside gs.h's (uint32, zeroed by the caller). */
#define GS_DEV_NO_PAGE   16u  /* no free page (or no table column) was left: that sequence
                                 was not served                                          */
#define GS_DEV_BAD_SEQ   32u  /* a sequence id, length, page id or layer position outside its
                                 range, or a sequence listed where it must not be: skipped */
#define GS_DEV_EMPTY_ROW 64u  /* every logit of a row is masked: its token is -1           */

/* Largest number of sequences of a cache, and of entries of one call's list. */
#define GS_MAX_SEQS 8192

/* ------------------------------------------------------------------------ */
/* The cache.                                                                */
/* ------------------------------------------------------------------------ */

/*
 * A paged key-value cache in caller-owned device memory.  Sequence s holds lens[s] tokens;
 * token t is row t % page of page table[s][t / page].  refs[p] counts the sequences that
 * hold page p; a page of count 0 is free.  A partly filled page is held by one sequence
 * only (gs_pages_fork copies it), so an append never writes to a shared page.
 * To start: lens and refs all 0 (table entries past a sequence's pages are never read).
 * K and V have the same strides (in elements; dim has stride 1).
 */
typedef struct gs_kv_cache {
    int32_t dtype;              /* GS_DTYPE_*                                             */
    int32_t layers, pages;      /* >= 1                                                   */
    int32_t kv_heads, page;     /* >= 1; page = tokens a page holds; layers * kv_heads <=
                                   2^30                                                   */
    int32_t dim;                /* head dimension: dim * element size a multiple of 16
                                   bytes, dim <= 256                                      */
    void*   k;                  /* device, 16-byte aligned                                */
    void*   v;
    int64_t layer_stride, page_stride, head_stride, token_stride;
                                /* each a multiple of 16 bytes; no two (layer, page, head,
                                   token) rows overlap                                    */
    int32_t seqs, cols;         /* sequences (<= GS_MAX_SEQS); pages a sequence can hold
                                   (cols * page <= 2^30)                                  */
    int32_t* table;             /* device int32[seqs][cols]                               */
    int32_t* lens;              /* device int32[seqs]                                     */
    int32_t* refs;              /* device int32[pages]                                    */
    uint32_t* dev_status;       /* device uint32 or NULL: GS_DEV_* bits OR-ed in          */
    void*    workspace;         /* device, gs_pages_workspace bytes, 16-byte aligned, all 0
                                   before its first use: it keeps which sequences the last
                                   gs_pages_extend refused (descriptions that share a table
                                   share it too)                                          */
    int64_t  workspace_bytes;
} gs_kv_cache;

/* Bytes of workspace the page calls of this cache need (from its sizes alone; pointers are
   not looked at).  Errors: GS_ERR_INVALID_ARG (NULL, sizes < 1), GS_ERR_UNSUPPORTED. */
gs_status gs_pages_workspace(const gs_kv_cache* cache, int64_t* bytes);

/*
 * gs_pages_extend -- room for add[i] more tokens of sequence seq[i]: takes the pages that
 * the longer sequences need and adds to their lengths.  Free pages are taken lowest number
 * first, in the order of the list.  Entry i is served when the needs of all entries up to
 * and including it fit the free pages (an entry that needs none always is) and its row of the
 * table; else it is left as it is, GS_DEV_NO_PAGE is set, and nothing is stored for the
 * sequence (gs_kv_write, the append of gs_paged_attention) until an extension by one token or
 * more is served, it is freed or forked onto, or its length is another.  An id outside the cache, a negative add and the second
 * listing of a sequence are skipped (GS_DEV_BAD_SEQ).
 *
 * seq: device int32[n].  add: device int32[n], or NULL (one token each).
 * Errors: GS_ERR_INVALID_ARG (NULL pointers, sizes, workspace too small), GS_ERR_UNSUPPORTED
 * (alignment, strides, dim, n or seqs over GS_MAX_SEQS), GS_ERR_CUDA.  n = 0 does nothing.
 * The same errors hold for the calls below.
 */
gs_status gs_pages_extend(const gs_kv_cache* cache, const int32_t* seq, const int32_t* add,
                          int32_t n, gs_stream stream);

/*
 * gs_pages_fork -- sequence dst[i] becomes a copy of src[i]: it releases the pages it holds,
 * shares src's full pages and, where src's last page is partly filled, takes a free page
 * (lowest number first, in the order of the list; pages released by this call count) and
 * copies the filled rows of every layer into it.  Where no page is left, dst[i] is empty
 * (length 0) and GS_DEV_NO_PAGE is set.  A sequence may be the src of several pairs.  A
 * sequence named in dst twice, or in dst and in src, is refused for the later pair and for
 * the pair that reads it (GS_DEV_BAD_SEQ).  Table columns past dst's pages are set to -1.
 */
gs_status gs_pages_fork(const gs_kv_cache* cache, const int32_t* src, const int32_t* dst,
                        int32_t n, gs_stream stream);

/* gs_pages_free -- the listed sequences release their pages: table entries -1, length 0.
   A sequence listed twice is freed once.  seq: device int32[n]. */
gs_status gs_pages_free(const gs_kv_cache* cache, const int32_t* seq, int32_t n,
                        gs_stream stream);

/*
 * gs_pages_compact -- make a pool dense: with n pages held, the k-th lowest free page below
 * n takes over the contents, count and table entries of the k-th highest held page (k and v
 * are moved in place; each page moves at most once).  Afterwards pages 0 .. n-1 are held.
 *
 * table_out: device int32[seqs][cols]; may be cache->table.
 * refs_out:  device int32[pages]; may be cache->refs.
 * live_out:  device int32[1] or NULL: n.
 */
gs_status gs_pages_compact(const gs_kv_cache* cache, int32_t* table_out, int32_t* refs_out,
                           int32_t* live_out, gs_stream stream);

/*
 * gs_kv_write -- store the K and V of new tokens in one layer: rows start[i] .. start[i+1]-1
 * of k and v are the last start[i+1] - start[i] tokens of sequence seq[i] (after
 * gs_pages_extend).  Rows that would lie before the sequence's first token or in a page that
 * other sequences share, and rows outside 0 .. tokens-1, are skipped (GS_DEV_BAD_SEQ), as are
 * the rows of a sequence whose last extension was refused (GS_DEV_NO_PAGE).  tokens = 0 does
 * nothing.
 *
 * k, v: device, storage dtype, [tokens][kv_heads][dim] with the strides given (elements;
 * dim has stride 1; any alignment).  seq: device int32[n].  start: device int32[n+1], rising.
 */
gs_status gs_kv_write(const gs_kv_cache* cache, int32_t layer, const void* k, const void* v,
                      int64_t token_stride, int64_t head_stride, int32_t tokens,
                      const int32_t* seq, const int32_t* start, int32_t n, gs_stream stream);

/* ------------------------------------------------------------------------ */
/* Attention of one new token.                                               */
/* ------------------------------------------------------------------------ */

typedef struct gs_paged_attention_args {
    const gs_kv_cache* cache;   /* its workspace is used where k_new is given             */
    int32_t layer;
    int32_t batch;              /* query rows (<= GS_MAX_SEQS)                             */
    const int32_t* seq;         /* device int32[batch]: row b reads sequence seq[b] (rows
                                   that append name different sequences); NULL = row b
                                   reads sequence b                                       */
    int32_t q_heads;            /* a multiple of kv_heads: query head h reads kv head
                                   h / (q_heads / kv_heads)                               */
    const void* q;              /* device, cache dtype, [batch][q_heads][dim]             */
    int64_t q_batch_stride, q_head_stride;
    const void* k_new;          /* device, cache dtype, [batch][kv_heads][dim], or NULL:   */
    const void* v_new;          /* stored at the sequence's last position (lens - 1) and
                                   attended to from there; both or neither.  Where that
                                   position is not the new token's (its extension was
                                   refused, the length was cut, or the page is shared or
                                   outside the pool), nothing is stored and the row attends
                                   over what the cache holds                              */
    int64_t new_batch_stride, new_head_stride;
    float   scale;              /* of the scores (usually dim ** -0.5); finite            */
    int32_t window;             /* 0: every position; else the last `window` ...          */
    int32_t sinks;              /* ... and the first `sinks` positions                    */
    void*   out;                /* device, cache dtype, [batch][q_heads][dim]             */
    int64_t out_batch_stride, out_head_stride;
    float*  lse;                /* device float[batch][q_heads] or NULL                   */
    void*   workspace;          /* device, gs_paged_attention_workspace bytes, 16-byte
                                   aligned; its first batch * q_heads int32 words are 0
                                   before its first use (the rest may hold anything); a
                                   call leaves it ready for calls of the same sizes
                                   (batch, heads, dim, dtype, cols, page, window, sinks) -
                                   zero those words again before one of others            */
    int64_t workspace_bytes;
} gs_paged_attention_args;

gs_status gs_paged_attention_workspace(const gs_paged_attention_args* args, int64_t* bytes);

/*
 * gs_paged_attention -- one query token a row over the visible positions j of its sequence
 * (0 <= j < lens; with a window: j < sinks or j >= lens - window):
 *   s_j = scale * q . k_j,  m = max_j s_j,  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),
 *   lse = m + ln sum_j e^(s_j - m).
 * Sums, maxima and the output's accumulator are fp32; for 16-bit caches the weights
 * e^(s_j - m) enter the product with V as a sum of two 16-bit numbers.  A row of length 0
 * gives out = 0 and lse = -inf.  Rows of a page past the sequence's length are never used,
 * whatever they hold.  Results do not depend on the grid's timing: the parts of a split
 * sequence are joined in their order.
 * Device-found: GS_DEV_BAD_SEQ (a sequence id outside the cache: as length 0; a page id
 * outside the pool: its rows read as zeros; a length past the table: cut, and no new token
 * stored; a new token whose page other sequences share), GS_DEV_NO_PAGE (a new token whose extension was refused).
 * Errors: as the page calls', and GS_ERR_INVALID_ARG for q_heads not a multiple of kv_heads,
 * layer outside the cache, k_new without v_new, window or sinks < 0, sinks without window,
 * a scale that is not finite; GS_ERR_UNSUPPORTED also where batch * q_heads * cols * page / 32
 * passes 2^31.
 */
gs_status gs_paged_attention(const gs_paged_attention_args* args, gs_stream stream);

/* ------------------------------------------------------------------------ */
/* Guided logits.                                                            */
/* ------------------------------------------------------------------------ */

typedef struct gs_guided_logits_args {
    int32_t batch, vocab;       /* >= 1 (batch <= GS_MAX_SEQS)                             */
    int32_t dtype;              /* GS_DTYPE_*: of uncond and cond                         */
    const void* uncond;         /* device [batch][vocab] or NULL (unguided, or every scale
                                   is 1)                                                  */
    const void* cond;           /* device [batch][vocab]                                  */
    int64_t row_stride;         /* elements between rows of uncond and of cond, >= vocab  */
    const int32_t* step_idx;    /* device int32[batch] or NULL (= step)                    */
    int32_t step;
    const float* scale_lut;     /* device float[n_lut] or NULL (= cfg)                    */
    int32_t n_lut;
    float cfg;
    const float* bias;          /* device float[.][vocab] or NULL                         */
    int64_t bias_stride;        /* elements between rows; 0 = one row for all             */
    const int32_t* tokens;      /* device int32[batch][tokens_stride] or NULL: history     */
    int64_t tokens_stride;      /* >= 0, <= 2^30: entries a row holds                      */
    const int32_t* tokens_len;  /* device int32[batch]: prompt and output tokens in a row;
                                   entries outside 0 .. vocab-1 are passed over           */
    const int32_t* prompt_len;  /* device int32[batch] or NULL (= 0)                      */
    const float* repetition;    /* device float[batch] or NULL (= 1), > 0                 */
    const float* frequency;     /* device float[batch] or NULL (= 0)                      */
    const float* presence;      /* device float[batch] or NULL (= 0)                      */
    const float* temperature;   /* device float[batch] or NULL (= 1); <= 0: greedy         */
    const uint32_t* mask;       /* device uint32[.][ceil(vocab/32)] or NULL: bit v % 32 of
                                   word v / 32 allows token v                             */
    int64_t mask_stride;        /* words between rows; 0 = one row for all                */
    const uint8_t* mask_present;/* device uint8[batch] or NULL: rows with 0 are not masked */
    const float* noise;         /* device float[.][vocab] or NULL: added to the logits the
                                   token is chosen by (Gumbel noise draws from softmax(z));
                                   not for greedy rows                                    */
    int64_t noise_stride;
    float*   out;               /* device float[batch][out_stride] or NULL: z             */
    int64_t  out_stride;        /* >= vocab                                               */
    int32_t* token;             /* device int32[batch] or NULL                            */
    float*   logprob;           /* device float[batch] or NULL: z[token] - ln sum e^z     */
    uint32_t* dev_status;
    void*    workspace;         /* device, gs_guided_logits_workspace bytes, 16-byte
                                   aligned; its first batch int32 words are 0 before its
                                   first use (the rest may hold anything); a call leaves
                                   it ready for calls of the same batch, vocab, dtype and
                                   streams given - zero those words again before one of
                                   others                                                 */
    int64_t  workspace_bytes;
} gs_guided_logits_args;

gs_status gs_guided_logits_workspace(const gs_guided_logits_args* args, int64_t* bytes);

/*
 * gs_guided_logits -- for every row b and token v, in fp32:
 *   z = fma(s, cond, (1 - s) * uncond)   s = scale_lut[step_idx[b]] (or cfg), as in
 *                                        gs_guided_step; cond where uncond is -inf, -inf
 *                                        where cond is; z = cond exactly at s = 1 (uncond is
 *                                        then not read) or without uncond
 *   z = z + bias
 *   z = z > 0 ? z * (1 / repetition) : z * repetition    for tokens of the history (the
 *                                        reciprocal rounded; z / repetition for repetitions
 *                                        outside 2^-40 .. 2^40, where it could overflow)
 *   z = z - (frequency * count + presence)               for tokens said count > 0 times
 *                                        in the output part of the history
 *   z = z / temperature                                  (temperature > 0; correctly rounded)
 *   z = -inf                                             where the mask forbids v
 * token = the lowest index of the largest z (+ noise); NaN is never chosen.  A row with no
 * z above -inf gives token -1, logprob -inf and GS_DEV_EMPTY_ROW.
 * A row whose step index is outside the table (GS_DEV_STEP_RANGE) or that needs the
 * missing uncond (scale not 1: GS_DEV_NEED_UNCOND) is not written, but for its token (-1).
 * Errors: GS_ERR_INVALID_ARG (NULL cond, sizes, strides, unknown dtype, tokens without
 * tokens_len, no output at all, workspace too small, step outside the table),
 * GS_ERR_UNSUPPORTED (batch over GS_MAX_SEQS, vocab over 2^28, tokens_stride over 2^30),
 * GS_ERR_CUDA.  No output may overlap an input or another output.
 */
gs_status gs_guided_logits(const gs_guided_logits_args* args, gs_stream stream);

/* The status of a device status word of these calls: GS_ERR_INVALID_ARG for GS_DEV_BAD_SEQ,
   GS_ERR_CAPACITY for GS_DEV_NO_PAGE, GS_ERR_UNSUPPORTED for GS_DEV_EMPTY_ROW, else
   gs_status_from_word. */
gs_status gs_decode_status_from_word(uint32_t word);

#ifdef __cplusplus
}
#endif

#endif /* GS_DECODE_H */
