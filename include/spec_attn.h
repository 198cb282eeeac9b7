/*
 * spec_attn.h -- the target pass's cache and attention, next to the
 * verification step of spec_verify.h (same library, same conventions:
 * device pointers, caller-owned memory, nothing allocated or synchronised,
 * work enqueued on `stream`, argument errors returned at once as a negative
 * status with nothing enqueued).
 *
 * One target pass scores the k + 1 chain positions, or the N nodes of a
 * candidate tree, of every sequence ("3.5 Speculative Decoding"
 * (llm-learning-path), "Tree verification": each node attends to the context
 * and to its own ancestors).  Per layer a user's program
 *   1. writes the new tokens' keys and values into the cache
 *      (spec_kv_append),
 *   2. attends from the new tokens to the cache (spec_attn_tree, or
 *      spec_attn_shared when the batch continues one long prefix) under the
 *      mask and positions of spec_verify_tree_mask,
 *   3. after spec_verify_tree / spec_verify_tree_sample, writes the accepted
 *      path's nodes again, now at consecutive positions (spec_kv_append with
 *      rows = out_path).
 *
 * The cache
 *   Keys and values live in pages of `page` positions.  A page holds, for
 *   every key/value head, `page` consecutive rows of D elements:
 *   k, v [num_pages, Hkv, page, D].  A sequence's page table lists the pages
 *   of its positions 0..page-1, page..2*page-1, ...
 *   SPEC_BF16: elements as they are.
 *   SPEC_E4M3: one byte per element and, per position and head, a signed
 *   exponent k_exp, v_exp [num_pages, Hkv, page]: the element is
 *   byte * 2^exponent.  The exponent of a row x is the smallest e with
 *   max |x| <= 448 * 2^e, clamped to [-120, 120] (0 for a row of zeros); a
 *   NaN or infinite element is stored as the NaN byte and takes no part in
 *   the maximum.  Powers of two keep the scaling and the reading back
 *   exact, so the one rounding is the byte's own (nearest, ties to even).
 *   An exponent outside [-120, 120], which no append writes, counts as the
 *   nearer end.  A page id outside [0, num_pages) in a table is never followed.
 */
#ifndef SPEC_ATTN_H
#define SPEC_ATTN_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Cache storage: SPEC_BF16 (spec_verify.h) or */
enum { SPEC_E4M3 = 2 };

/* Data-error bit of the attention workspace's error word: a length outside
 * [0, table_width * page] or a page id outside [0, num_pages) among the
 * pages a sequence needs.  That sequence's outputs are NaN. */
enum { SPEC_DATA_PAGE_RANGE = 1 << 7 };

/* An internal wait of the attention kernel ran out (its waits are bounded):
 * the call's outputs are undefined. */
enum { SPEC_DATA_STALL = 1 << 8 };

typedef struct spec_kv_cache {
    void *k, *v;            /* [num_pages, Hkv, page, D], 16-byte aligned     */
    int8_t *k_exp, *v_exp;  /* [num_pages, Hkv, page], 4-byte aligned
                               (SPEC_E4M3; ignored for SPEC_BF16)            */
    int num_pages;          /* >= 1                                          */
    int Hkv;                /* key/value heads, 1..1024                      */
    int page;               /* 16, 32, 64 or 128 positions                   */
    int D;                  /* 64 or 128 elements a head                     */
    int dtype;              /* SPEC_BF16 or SPEC_E4M3                        */
} spec_kv_cache;

/*
 * Write M new tokens per sequence into the cache: entry t of sequence b goes
 * to position starts[b] + t and takes token r = rows[b][t] of k and v (r = t
 * where rows is NULL).  Skipped, without touching the cache: a negative
 * position (left padding) or one past the table, a page id outside
 * [0, num_pages), an r outside [0, N) (spec_verify_tree's out_path pads with
 * -1).  Two entries that name one position of one page race.
 *
 * Arguments
 *   cache         see above (host struct, read during the call)
 *   page_table    [B, table_width] int32, device
 *   starts        [B] int32, device
 *   k, v          [B, N, Hkv, D] dtype, device: Hkv * D contiguous elements
 *                 a token, consecutive tokens (across sequences too) at
 *                 token_stride elements
 *   token_stride  >= Hkv * D, or 0 for Hkv * D; a multiple of 8
 *   rows          [B, M] int32, device, or NULL (then M = N)
 *   dtype         SPEC_F32 or SPEC_BF16: type of k and v, 16-byte aligned
 *   B, N, M >= 0
 */
int spec_kv_append(const spec_kv_cache *cache, const int32_t *page_table, int table_width,
                   const int32_t *starts, const void *k, const void *v, int64_t token_stride,
                   const int32_t *rows, int B, int N, int M, int dtype, spec_stream_t stream);

/*
 * Read M consecutive positions per sequence back: out_k, out_v
 * [B, M, Hkv, D] get position starts[b] + t; zeros where the position or its
 * page id is out of range.  dtype SPEC_F32 (exact) or SPEC_BF16 (exact for
 * either storage: a byte times a power of two fits bf16).  Either output
 * may be NULL.
 */
int spec_kv_read(const spec_kv_cache *cache, const int32_t *page_table, int table_width,
                 const int32_t *starts, void *out_k, void *out_v, int B, int M, int dtype,
                 spec_stream_t stream);

/* Workspace bytes of spec_attn_tree and spec_attn_shared for B sequences of N
 * new tokens (any cache lengths). */
int spec_attn_workspace_size(int B, int N, int Hq, int Hkv, int D, size_t *bytes);

/*
 * Attention of N new tokens per sequence to the cache.  lens[b] counts
 * sequence b's cached positions, the new tokens included: new token n is
 * position lens[b] - N + n (written by spec_kv_append before).  For query
 * head h of key/value head h / (Hq / Hkv), new token i and position j:
 *   s_ij = scale * q_i . k_j
 *   cap > 0:      s_ij = cap * tanh(s_ij / cap)
 *   slopes:       s_ij -= slopes[h] * (pos_i - pos_j)
 *   seen_ij:      a context position (before the new tokens) always; a new
 *                 token j where mask[b][i][j] != 0, or j <= i without a mask;
 *                 and only pos_i - pos_j < window if window > 0
 *   out_i  = sum_seen e^s_ij v_j / sum_seen e^s_ij
 *   lse_i  = ln sum_seen e^s_ij
 * A token that sees nothing gets zeros and lse -inf; an unseen position adds
 * nothing whatever its key and value hold.  Scores, sums and the output's
 * accumulation are fp32; the softmax weights are rounded to bf16 for the product
 * with the values, whatever the cache's type (an e4m3 cache's values are exact in
 * bf16; its products q . k take the query to 2^-18 of its largest element).
 * Results do not depend on timing: calls with the same inputs give
 * the same bits.
 *
 * Arguments
 *   cache, page_table, table_width, lens [B] int32: as above; the table of a
 *                sequence covers its lens[b] positions
 *   q            [B, N, Hq, D] bf16, device, 16-byte aligned, consecutive
 *                tokens at q_stride elements (0: Hq * D; a multiple of 8)
 *   mask         [B, N, N] uint8, device, or NULL (a chain)
 *   pos          [B, N] int32, device, or NULL: position indices of the new
 *                tokens for the bias and the window (spec_verify_tree_mask's
 *                out_pos); NULL: their cache positions.  A context position's
 *                index is its place in the sequence.
 *   slopes       [Hq] fp32, device, or NULL
 *   B >= 0, 1 <= N <= SPEC_MAX_TREE_NODES, Hq a multiple of Hkv
 *   scale        finite; cap >= 0 and finite (0: none, as 2^64 and more are);
 *                window >= 0 (0: none)
 *   dtype        type of q and out: SPEC_BF16
 *   out          [B, N, Hq, D] bf16, device, contiguous, 16-byte aligned
 *   out_lse      [B, N, Hq] fp32, device, or NULL
 *   workspace    >= spec_attn_workspace_size(...) bytes, 16-byte aligned, its
 *                first 4 bytes (the error word) zeroed before first use, the
 *                rest in any state.  One workspace per call in flight, and
 *                not a verification call's: its counters would be lost
 */
int spec_attn_tree(const spec_kv_cache *cache, const int32_t *page_table, int table_width,
                   const int32_t *lens, const void *q, int64_t q_stride, const uint8_t *mask,
                   const int32_t *pos, const float *slopes, int B, int N, int Hq, float scale,
                   float cap, int window, int dtype, void *out, float *out_lse, void *workspace,
                   size_t workspace_bytes, spec_stream_t stream);

/*
 * The same where all sequences continue one prefix of shared_len positions,
 * held once: the pages of shared_table [ceil(shared_len / page)] int32,
 * device.  page_table and lens describe what follows: position j of a
 * sequence's own cache is position shared_len + j of the sequence.  The
 * prefix's keys and values are read once for the whole batch, not once per
 * sequence.  shared_len >= 0; a bad page id in shared_table fails every
 * sequence.  With a window, what of the prefix no row reaches is not read, in
 * whole blocks of 128 positions, and its page ids are not looked at.
 */
int spec_attn_shared(const spec_kv_cache *cache, const int32_t *shared_table, int shared_len,
                     const int32_t *page_table, int table_width, const int32_t *lens,
                     const void *q, int64_t q_stride, const uint8_t *mask, const int32_t *pos,
                     const float *slopes, int B, int N, int Hq, float scale, float cap, int window,
                     int dtype, void *out, float *out_lse, void *workspace,
                     size_t workspace_bytes, spec_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_ATTN_H */
