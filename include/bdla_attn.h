/*
 * bdla_attn.h — the softmax layer that stands beside the linear attention of
 * bdla.h in a hybrid stack: norm and rotation of queries and keys, causal
 * softmax attention with grouped heads over packed documents, the paged cache
 * of its keys and values (norm, rotation and append also in one call), and
 * attention of a sequence's newest tokens over that cache.
 *
 * Conventions are those of bdla.h: device pointers owned by the caller, no
 * allocation and no synchronisation inside a call, every call ordered on
 * `stream`, host-detectable errors returned before any launch, errors found
 * on the device recorded in the status word at the start of `ws`
 * (bdla_read_device_status), the first 256 bytes of a workspace zeroed once by
 * its owner.  Calls that share a workspace must be ordered by one stream.
 * Tensors are bf16, contiguous and 16-byte aligned unless said otherwise.
 */
#ifndef BDLA_ATTN_H
#define BDLA_ATTN_H

#include "bdla.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int B;    /* documents (fixed-length calls), sequences (cache calls), or 1 (packed documents) */
    int T;    /* tokens per document, total packed tokens, or new tokens per sequence */
    int Hq;   /* query heads, a multiple of Hk: query head h reads key head h / (Hq / Hk) */
    int Hk;   /* key and value heads */
    int d;    /* width of queries, keys and values: 64 or 128 */
} bdla_attn_dims;

/*
 * RMS norm of every query and key head with the position rotation in the same
 * pass.  For each token and head, with x the head's d features:
 *     n = x / sqrt(mean(x^2) + eps),   y = n o w
 * (w = wq for queries, wk for keys, fp32 [d]), and the first `rotary`
 * features of y are rotated in pairs (a, b) by the angle
 * pos * base^(-2 i / rotary) of pair i: (a cos - b sin, b cos + a sin).
 * Pair i is (y[i], y[i + rotary/2]), or (y[2i], y[2i + 1]) if `interleaved`.
 * rotary is 0 (no rotation) or a multiple of 16 up to d.  The angle is taken
 * from an exact product of the position with a 64-bit binary fraction of a
 * turn, so far positions lose nothing.  An L2 norm (the keys of the linear
 * attention) is eps = 0 or tiny with w = 1/sqrt(d); with eps = 0 a head of zeros
 * gives NaN.  Squares are summed in fp32: a mean square above its range gives 0.
 *   q, k      bf16 [B, T, Hq | Hk, d] with strides: element strides of a
 *             token and of a head, multiples of 8 (so that they may be views
 *             of one fused projection); features contiguous; rows of a batch
 *             follow each other (batch stride = T * token stride)
 *   positions int32 [B, T], or NULL: the token's index in its document
 *   cu_seqlens int32 [n_docs + 1] (B = 1), or NULL for fixed-length rows; read
 *             only when positions is NULL, and not checked here
 *   qn, kn    bf16 [B, T, Hq | Hk, d] contiguous
 * The gradient takes dqn, dkn (bf16 or fp32, contiguous) and writes dq, dk
 * (bf16, contiguous) and dwq, dwk (fp32 [d], summed over tokens and heads in
 * an order that depends on the sizes alone).
 */
typedef struct {
    const void *q, *k;
    int64_t q_token, q_head, k_token, k_head;   /* element strides */
    const float *wq, *wk;
    const int32_t *positions;
    const int32_t *cu_seqlens;
    double base;
    float eps;
    int rotary;
    int interleaved;
    int n_docs;
} bdla_qk_norm_args;
bdla_status bdla_qk_norm(bdla_qk_norm_args a, void *qn, void *kn, bdla_attn_dims d, void *stream);
bdla_status bdla_qk_norm_bwd(bdla_qk_norm_args a, const void *dqn, const void *dkn, bdla_dtype g_dtype, void *dq,
                             void *dk, float *dwq, float *dwk, bdla_attn_dims d, void *ws, size_t ws_bytes,
                             void *stream);

/*
 * Causal softmax attention of whole documents.  For token i of a document and
 * query head h, over the tokens j <= i of the same document:
 *     s_ij = scale q_i . k_j,   p_ij = e^{s_ij - lse_i},   o_i = sum_j p_ij v_j
 *     lse_i = log sum_j e^{s_ij}
 *   q, o, dO, dq   bf16 [B, T, Hq, d];   k, v, dk, dv  bf16 [B, T, Hk, d]
 *   lse            fp32 [Hq, B*T] (head-major)
 * Documents are the B rows, or packed (B = 1, device int32 cu_seqlens
 * [n_docs + 1] as in bdla.h).  scale > 0.  The gradient is
 *     delta_i = dO_i . o_i,   ds_ij = p_ij (dO_i . v_j - delta_i),
 *     dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i,   dv_j = sum_i p_ij dO_i
 * at the o and lse that it is handed: the forward's, or those joined with what
 * the call does not see (a sink in the denominator, other keys).  For delta it
 * may take its own fp32 sum of p dO . v where that lies within the rounding of
 * o, and weights over their sum where that sum is 1 within 2^-8.  dk and dv are
 * summed over the query heads of their key head in a fixed order, so the same
 * inputs give the same bits.  Infinities and NaN in one document do not reach
 * another.  Within a document they reach what sees them and, since a masked
 * weight is a factor of 0, may reach other rows of the same 128 queries or keys.
 */
bdla_status bdla_attn_fwd(const void *q, const void *k, const void *v, const int32_t *cu_seqlens, int n_docs,
                          float scale, void *o, float *lse, bdla_attn_dims d, void *ws, size_t ws_bytes,
                          void *stream);
bdla_status bdla_attn_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                          const void *dO, const int32_t *cu_seqlens, int n_docs, float scale, void *dq, void *dk,
                          void *dv, bdla_attn_dims d, void *ws, size_t ws_bytes, void *stream);

/*
 * A paged cache of keys and values.  Page p holds the rows of `page`
 * consecutive positions; position t of sequence b is row t % page of page
 * pages[b][t / page].  n_pages * page is at most 2^31 - 1, and so is (nearly)
 * max_pages * page (BDLA_ERR_TOO_LARGE).
 */
typedef struct {
    void *k, *v;            /* bf16 [n_pages, page, Hk, d] */
    const int32_t *pages;   /* [B, max_pages]; entries past a sequence's need are not read */
    const int32_t *lens;    /* [B] tokens in the cache before the new ones */
    int n_pages;
    int page;               /* tokens per page, 1 .. 65536 */
    int max_pages;          /* width of the page table */
} bdla_cache;

/*
 * Writes new rows into the cache: for j < counts[b] (all T where counts is
 * NULL), position lens[b] + j of sequence b takes row rows[b][j] (row j where
 * rows is NULL) of k and v, bf16 [B, T, Hk, d].  With rows and counts this
 * also compacts a verified tree of drafts: the accepted drafts, in order, move
 * to the positions that follow the context.  lens is not changed.  Sequences
 * that share a page (after a fork) must not both write into it: copy it first.
 * The source rows must not lie in the cache that is written.  A row whose
 * position lies past the page table, whose page lies outside the cache, or
 * whose source lies outside 0 .. T - 1 is not written and recorded as
 * BDLA_ERR_DEVICE, and so is a count outside 0 .. T.
 */
bdla_status bdla_cache_append(const void *k, const void *v, bdla_cache c, const int32_t *rows,
                              const int32_t *counts, bdla_attn_dims d, void *ws, size_t ws_bytes, void *stream);

/*
 * bdla_qk_norm and bdla_cache_append in one launch, with their bits: queries
 * normed and rotated to qn, keys normed and rotated into the cache, values into
 * the cache.  A token's position is its place in the cache (lens[b] + j for the
 * j-th new token of sequence b) unless `a` gives positions.
 *   a        as for bdla_qk_norm; q NULL: keys and values alone (wq and qn may
 *            be NULL, d.Hq is not looked at).  With cu_seqlens (B = 1, n_docs
 *            sequences) the tokens of all sequences are packed, as many of each
 *            as there happen to be (prompts and single tokens in one call)
 *   v        bf16 [B, T, Hk, d] with element strides of a token and of a head,
 *            multiples of 8, as q and k
 *   rows, counts   as for bdla_cache_append (NULL for packed tokens,
 *            BDLA_ERR_UNSUPPORTED): place j takes the keys and values of row
 *            rows[b][j], at that place's position, or at positions[b][rows[b][j]]
 *            where positions are given.  They say nothing about queries: all T
 *            are normed, row j at place j
 *   qn       bf16 [B, T, Hq, d] contiguous
 * lens is not changed; what bdla_cache_append records as BDLA_ERR_DEVICE and does
 * not write is treated so here too, and so are malformed cu_seqlens and the
 * tokens that they give to no sequence.  Neither q, k nor v may lie in the cache.
 */
bdla_status bdla_qk_norm_append(bdla_qk_norm_args a, const void *v, int64_t v_token, int64_t v_head, bdla_cache c,
                                const int32_t *rows, const int32_t *counts, void *qn, bdla_attn_dims d, void *ws,
                                size_t ws_bytes, void *stream);

/*
 * Softmax attention of a sequence's T newest tokens (1 .. 64), whose keys and
 * values are already in the cache at positions lens[b] .. lens[b] + T - 1.
 * Every new token sees the lens[b] positions before them, and of the new ones
 * those whose bit is set in its mask: tree[b][i] bit j (uint64) for token j;
 * NULL means the tokens j <= i (T = 1: plain decoding).  A token that sees
 * nothing gets o = 0 and lse = -inf.
 *   q, o   bf16 [B, T, Hq, d];   lse  fp32 [B, T, Hq]
 * What lies in the cache outside the positions that a sequence's new tokens
 * see is not read, whatever its bits; a value that one of them sees and that is
 * not finite may reach the others, whose weight of 0 it is multiplied by.
 * Positions past the page table, pages outside the cache and negative lens are
 * recorded as BDLA_ERR_DEVICE and not seen.
 */
bdla_status bdla_attn_cached(const void *q, bdla_cache c, const uint64_t *tree, float scale, void *o, float *lse,
                             bdla_attn_dims d, void *ws, size_t ws_bytes, void *stream);

/*
 * bdla_attn_cached for a batch in which groups of sequences share the positions
 * that they begin with (a system prompt, several samples of one prompt): what a
 * group shares is read once for all of its sequences.  The result is that of
 * bdla_attn_cached up to rounding.
 *   cu_groups  device int32 [n_groups + 1], 0 <= cu[0] <= cu[1] .. <= B: group g
 *              is the sequences cu[g] .. cu[g + 1] - 1 (sequences outside all
 *              groups share nothing; groups may be empty)
 *   shared     device int32 [n_groups]: positions that the group's sequences share:
 *              the first shared[g] positions of all of them lie in the same pages,
 *              and each of their tables names those.  They are read as the table
 *              of the group's first sequence says, or, where reading them once
 *              would not pay (bdla_set_share_least), as each sequence's own does.
 *              What goes beyond the shortest committed context of a group's
 *              sequences (lens) is not counted as shared
 * n_groups is 1 .. 65535, T 1 .. 64.  Both arrays may change between replays of a
 * captured call, as lens and the tables may.  Malformed cu_groups (then no
 * sequence shares anything) and negative shared[g] are recorded as
 * BDLA_ERR_DEVICE, and so is what bdla_attn_cached records.  Sizes whose counts
 * pass 32 bits are BDLA_ERR_TOO_LARGE.  Finding out what to join and joining it take
 * 5 to 10 us (more for batches of trees), so where little is shared bdla_attn_cached
 * is the quicker call.  The workspace has room for the sums of any lengths and groups:
 * up to 4 fp32 rows of d + 2 for each of the B T Hq rows, and up to 66 MB beside them.
 */
bdla_status bdla_attn_shared(const void *q, bdla_cache c, const int32_t *cu_groups, const int32_t *shared, int n_groups,
                             const uint64_t *tree, float scale, void *o, float *lse, bdla_attn_dims d, void *ws,
                             size_t ws_bytes, void *stream);

/* Bytes of workspace of the calls above (0 on invalid sizes).  n_docs as for
 * bdla_workspace_bytes, the groups of a BDLA_ATTN_SHARED; max_keys is max_pages *
 * page of a BDLA_ATTN_CACHED or BDLA_ATTN_SHARED. */
enum { BDLA_ATTN_FWD = 0, BDLA_ATTN_BWD = 1, BDLA_ATTN_NORM_BWD = 2, BDLA_ATTN_APPEND = 3, BDLA_ATTN_CACHED = 4,
       BDLA_ATTN_SHARED = 5 };
size_t bdla_workspace_bytes_attn(int op, bdla_attn_dims d, int n_docs, int64_t max_keys);

#ifdef __cplusplus
}
#endif

#endif /* BDLA_ATTN_H */
