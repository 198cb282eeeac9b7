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

/*
 * Rotary positions.  A head's `rot` elements from element `first` on are rot / 2
 * pairs; pair i of a token at position index p is turned by the angle
 * p * theta_i and multiplied by `amplitude`:
 *   (u, v) -> amplitude (u cos - v sin, v cos + u sin)
 * SPEC_ROPE_HALF: pair i is elements (i, i + rot / 2) of the part;
 * SPEC_ROPE_INTERLEAVED: (2 i, 2 i + 1).  The head's other elements stay.
 * Angles are held as fractions of a turn in 64-bit fixed point: a frequency is the
 * integer nearest to 2^64 theta_i / (2 pi), its product with p modulo 2^64 is exact,
 * so that the angle is at most 2^-65 |p| of a turn off (2^-34 at the farthest
 * position, less than fp32 holds).  Positions are any int32.
 */
enum { SPEC_ROPE_HALF = 0, SPEC_ROPE_INTERLEAVED = 1 };

/* How frequencies theta_i = base^(-2 i / rot) are scaled for contexts longer
 * than `original` by `factor`:
 *   SPEC_ROPE_PLAIN   not at all
 *   SPEC_ROPE_LINEAR  theta / factor
 *   SPEC_ROPE_TURNS   theta (w + (1 - w) / factor), w = (t - low) / (high - low)
 *                     clamped to [0, 1], t = original theta / (2 pi): the turns
 *                     that the pair makes in the original context
 *   SPEC_ROPE_INDEX   the same with w = 1 - (i - a) / max(b - a, 1/1000) clamped,
 *                     a = max(0, floor(at(high))), b = min(rot - 1, ceil(at(low))),
 *                     at(t) = rot ln(original / (2 pi t)) / (2 ln base): the pair
 *                     that makes t turns there */
enum { SPEC_ROPE_PLAIN = 0, SPEC_ROPE_LINEAR = 1, SPEC_ROPE_TURNS = 2, SPEC_ROPE_INDEX = 3 };

/*
 * The frequencies, computed on the host into freqs [rot / 2] (HOST memory; copy
 * them to the device for the calls below).  rot: a multiple of 16, 16..1024;
 * base > 1, at most 1e30; factor >= 1 (unread for SPEC_ROPE_PLAIN); original,
 * low and high only for the last two: original >= 1, 0 < low < high, each at
 * most 1e30.  All finite.
 */
int spec_rope_freqs(int rot, double base, int scaling, double factor, double original, double low,
                    double high, uint64_t *freqs);

/*
 * Rotary positions of B * N tokens of H heads of D elements.
 *   x, out       [B, N, H, D] dtype, device, 16-byte aligned; consecutive tokens
 *                (across sequences too) at x_stride / out_stride elements (0: H * D;
 *                at least that, a multiple of 8), a token's heads contiguous.
 *                out may be x, with the same stride (then only the turned part is
 *                written); otherwise they do not overlap (SPEC_ERR_SHAPE)
 *   freqs        [rot / 2], device, 16-byte aligned
 *   pos          [B, N] int32, device
 *   D, rot, first  multiples of 16: 16 <= D <= 1024, first + rot <= D
 *   amplitude    finite; a negative angle (`inverse` != 0) takes the turn back
 *   layout       SPEC_ROPE_HALF or SPEC_ROPE_INTERLEAVED
 *   dtype        SPEC_F32 or SPEC_BF16 (computed in fp32, rounded once)
 */
int spec_rope(const void *x, int64_t x_stride, void *out, int64_t out_stride, const uint64_t *freqs,
              int rot, int first, float amplitude, int layout, int inverse, const int32_t *pos,
              int B, int N, int H, int D, int dtype, spec_stream_t stream);

/*
 * spec_kv_append with the keys rotated on the way: token r of sequence b is
 * turned (its first `rot` elements a head) to position index pos[b][r], then
 * written as spec_kv_append writes it (an e4m3 cache takes the turned values
 * unrounded).  Without pos the index is the cache position.  The values are
 * written as they are.
 * With q, the same tokens' queries are rotated in the same launch: out_q gets
 * token n of q at index pos[b][n], or starts[b] + n.
 *   pos          [B, N] int32, device, or NULL
 *   freqs, rot, amplitude, layout  as for spec_rope; rot <= D
 *   q, out_q     [B, N, Hq, D] dtype, device, as x and out of spec_rope, or both
 *                NULL; with `rows` NULL only (SPEC_ERR_PARAM).  out_q does not
 *                overlap k or v
 * Other arguments as for spec_kv_append.
 */
int spec_kv_append_rope(const spec_kv_cache *cache, const int32_t *page_table, int table_width,
                        const int32_t *starts, const void *k, const void *v, int64_t token_stride,
                        const int32_t *rows, const int32_t *pos, const uint64_t *freqs, int rot,
                        float amplitude, int layout, const void *q, int64_t q_stride, void *out_q,
                        int64_t out_q_stride, int B, int N, int M, int Hq, int dtype,
                        spec_stream_t stream);

/*
 * A latent cache: one row of C + R bf16 elements a position, shared by all
 * heads.  The first C are the latent vector, values and the keys' first part at
 * once; the R after them are the keys' rotary part.  Pages and tables as above.
 */
typedef struct spec_latent_cache {
    void *data;     /* [num_pages, page, C + R] bf16, 16-byte aligned          */
    int num_pages;  /* >= 1                                                    */
    int page;       /* 16, 32, 64 or 128 positions                             */
    int C;          /* 128, 256 or 512                                         */
    int R;          /* 64                                                      */
} spec_latent_cache;

/*
 * Write M new tokens per sequence into a latent cache: positions, rows and what
 * is skipped as in spec_kv_append.  c [B, N, C] and r [B, N, R] dtype, device,
 * 16-byte aligned, tokens at c_stride and r_stride elements (0: C, R; at least
 * that, multiples of 8: both may be parts of one projection).  r is rotated
 * (all R elements) to pos[b][r], or to the cache position without pos; freqs
 * NULL: r as it is (pos is then ignored).
 */
int spec_latent_append(const spec_latent_cache *cache, const int32_t *page_table, int table_width,
                       const int32_t *starts, const void *c, int64_t c_stride, const void *r,
                       int64_t r_stride, const int32_t *rows, const int32_t *pos,
                       const uint64_t *freqs, float amplitude, int layout, int B, int N, int M,
                       int dtype, spec_stream_t stream);

/* Workspace bytes of spec_latent_attn for B sequences of N new tokens and H
 * heads (any cache lengths; its sizes, its limits). */
int spec_latent_workspace_size(int B, int N, int H, int C, size_t *bytes);

/*
 * Attention of N new tokens per sequence to a latent cache, in the absorbed
 * form: every head's query comes with its own key projection multiplied in
 * (C elements) and its rotary part (R elements, rotated), so that all heads
 * read one row (c_j, r_j) a position.  For token i, head h, position j:
 *   s_ij  = scale * q_ih . (c_j, r_j)
 *   out_ih = sum_seen e^s_ij c_j / sum_seen e^s_ij     (C elements: the head's value
 *                                        projection is applied by the caller)
 *   lse_ih = ln sum_seen e^s_ij
 * seen as in spec_attn_tree: the context always, new token j where
 * mask[b][i][j] != 0, or j <= i without a mask.  A token that sees nothing gets
 * zeros and lse -inf; an unseen position adds nothing whatever it holds.  A latent
 * element that is not finite and seen is NaN in the result (its score is not finite
 * either), whatever else the row sees.
 * Scores, sums and accumulators are fp32, the softmax weights are rounded to
 * bf16 for the product with the latents.  Calls with the same inputs give the
 * same bits.
 *   lens         [B] int32, device: cached positions, the new tokens included
 *   q            [B, N, H, C + R] bf16, device, 16-byte aligned, tokens at
 *                q_stride elements (0: H * (C + R); a multiple of 8)
 *   mask         [B, N, N] uint8, device, or NULL (a chain)
 *   1 <= N <= SPEC_MAX_TREE_NODES, 1 <= H <= 1024, B * N * H <= 2^30; scale finite
 *   out          [B, N, H, C] bf16, device, contiguous, 16-byte aligned
 *   out_lse      [B, N, H] fp32, device, or NULL
 *   workspace    >= spec_latent_workspace_size(...) bytes, as for spec_attn_tree
 * A length outside [0, table_width * page] or a bad page id fails its sequence:
 * outputs NaN, SPEC_DATA_PAGE_RANGE in the workspace's error word.
 */
int spec_latent_attn(const spec_latent_cache *cache, const int32_t *page_table, int table_width,
                     const int32_t *lens, const void *q, int64_t q_stride, const uint8_t *mask,
                     int B, int N, int H, float scale, void *out, float *out_lse, void *workspace,
                     size_t workspace_bytes, spec_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_ATTN_H */
