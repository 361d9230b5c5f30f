/*
 * gdnattn.h -- C ABI of the softmax-attention layers beside the GDN layers in
 * libgdnreplay (sm_103a), under speculative decoding: a paged key/value cache, the
 * step that fills it, the attention of a block of drafted tokens over it, and what
 * accepting or forking does to it.
 *
 * A decode step of one attention layer is
 *     gdn_attn_stage   norms of queries and keys per head and the position rotation;
 *                      the rotated keys and the values go to the draft's cache rows;
 *     gdn_attn_verify  attention of the T drafted tokens (a chain or a tree) over the
 *                      committed rows and, along the tree, each other;
 * and, once per step for all layers,
 *     gdn_attn_accept  the accepted path's rows moved to the front of the draft's rows,
 *                      and the new lengths.  A chain moves nothing: its rollback is the
 *                      length alone, as for the recurrent layers (gdnreplay.h).
 * gdn_pages_reserve / fork / copy / release keep the pages: a device-resident free list
 * and a reference count for each page, so that forked sequences share their full pages.
 *
 * Conventions as in gdnreplay.h: device pointers, host structs read during the call
 * only, no allocation, no synchronisation, no global state, 0 or a negative GDN_ERR_*
 * code from host validation, device faults OR-ed into a status word.  Calls on one
 * cache must be stream-ordered.
 */
#ifndef GDNATTN_H
#define GDNATTN_H

#include <stdint.h>

#include "gdnreplay.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_STATUS_BAD_PAGE   64   /* a block-table entry, a copy pair or a free-list entry that the
                                      call needs is outside [0, n_page), the entry is not one of the
                                      sequence's own (n_owned), or a page was released more
                                      often than it was shared; see each call */
#define GDN_STATUS_BAD_POS   128   /* a rotation position outside [0, max_pos); the token is skipped */
#define GDN_STATUS_BAD_TREE  256   /* a parent not in [-1, t) or an accepted path that is not strictly
                                      increasing in [0, T); the sequence is skipped */
#define GDN_STATUS_NO_PAGES  512   /* the free list ran out; the sequence is skipped */

/*
 * The cache of n_layer attention layers and the pages' bookkeeping, which all layers share
 * (row-major, innermost last, dense):
 *   k, v         dtype  [n_layer, n_page, Hkv, page, d]   16-byte aligned
 *   block_table  int32  [n_slot, max_pages]  pages of a sequence in order of position
 *   seq_len      int32  [n_slot]             committed tokens
 *   n_owned      int32  [n_slot]             entries of the block table that are in use
 *   ref          int32  [n_page]             sequences that hold the page; 0 = free
 *   free_list    int32  [n_page]             the free pages are its first free_count entries;
 *   free_count   int32  [1]                  pages are taken from the end
 * Token p of a sequence sits in row p % page of page block_table[slot][p / page].  The
 * attention calls use k, v, block_table, seq_len and n_owned; the other pointers may then be
 * NULL, and n_owned too where the caller keeps the pages by means of its own.  Entries of a block-table
 * row from n_owned on say nothing: a release leaves its ids there, and a reserve or fork that finds no
 * free page does not replace them.  The attention calls therefore use none of them: a token
 * that would lie there is one without a page (GDN_STATUS_BAD_PAGE).
 */
typedef struct {
    int32_t n_slot;     /* sequence slots, >= 0 */
    int32_t max_pages;  /* block-table entries per slot, 1..2^18; max_pages * page <= 2^24 */
    int32_t n_page;     /* pages, >= 1; n_page * Hkv * page < 2^31 */
    int32_t page;       /* tokens per page: 16, 32, 64 or 128 */
    int32_t n_layer;    /* 1..32767 */
    int32_t Hkv;        /* key/value heads, 1..128 */
    int32_t d;          /* head dim: 64, 128 or 256 */
    int32_t dtype;      /* GDN_DTYPE_BF16 or GDN_DTYPE_F32 (q, k, v and out too) */
    void *k, *v;
    int32_t *block_table, *seq_len, *n_owned, *ref, *free_list, *free_count;
} gdn_page_cache;

/* One block of drafted tokens.  Row t of sequence b is in use when t < draft_len[b]
 * (draft_len NULL: every row). */
typedef struct {
    int32_t B;          /* sequences in this call, 0..65535 */
    int32_t T;          /* rows per sequence: 1..64; gdn_attn_stage: 1..2^20, B * T <= 2^30 */
    int32_t Hq;         /* query heads, a multiple of Hkv, Hq / Hkv <= 64; head h reads key head
                           h / (Hq / Hkv) */
    float   scale;      /* score scale, normally 1/sqrt(d) */
    int32_t flags;      /* GDN_FLAG_TEST_EXPIRE or 0 */
} gdn_attn_dims;

#define GDN_ROPE_HALF  0    /* pairs (i, i + rot/2) */
#define GDN_ROPE_PAIRS 1    /* pairs (2i, 2i + 1) */

/* Norm and rotation.  Strides count elements between a tensor's rows (tokens); the
 * heads of a token are dense, so q, k and v may be views of one projection's output. */
typedef struct {
    int32_t rot;        /* rotated dims of each head: a multiple of 16, 0..d */
    int32_t style;      /* GDN_ROPE_HALF or GDN_ROPE_PAIRS */
    int32_t max_pos;    /* rows of cos_sin, >= 1 */
    float   eps;        /* >= 0 */
    int64_t q_stride, k_stride, v_stride;   /* >= Hq d, Hkv d, Hkv d; multiples of 16 bytes */
} gdn_rope_dims;

/*
 * gdn_attn_stage -- for every row t < draft_len[b] in use and every head of q and k:
 *     r = 1 / sqrt(mean_i(x_i^2) + eps),  y_i = x_i r w_i  (w = q_weight or k_weight),
 * then the first rot dims turned by the position's angles, (a, b) -> (a cos - b sin,
 * b cos + a sin).  Queries go to q_out; keys, and v unchanged, go to the cache row of
 * token seq_len[slot] + t.  Rows not in use: q_out 0, nothing staged.  Arithmetic in
 * fp32, rounded once to dtype.
 *   q [B, T, Hq, d], k, v [B, T, Hkv, d] dtype (token strides in gdn_rope_dims; 16-byte
 *   aligned);  q_weight, k_weight fp32 [d];  cos_sin fp32 [max_pos, rot]: rot/2 cosines,
 *   then rot/2 sines (NULL when rot is 0), these three 16-byte aligned;  pos int32 [B, T] rotation positions, NULL =
 *   seq_len + t;  q_out dtype [B, T, Hq, d] dense.
 * GDN_STATUS_BAD_SLOT, _BAD_LEN (seq_len or draft_len out of range) and _NO_ROOM (seq_len +
 * draft_len > max_pages * page): the sequence is skipped, q_out included; _BAD_POS: the
 * token is treated as not in use; _BAD_PAGE: the token's key and value are not staged.
 */
int gdn_attn_stage(const gdn_page_cache *cache, int32_t layer, const gdn_attn_dims *dims,
                   const gdn_rope_dims *rope, const int32_t *state_idx, const int32_t *draft_len,
                   const void *q, const void *k, const void *v, const int32_t *pos,
                   const float *q_weight, const float *k_weight, const float *cos_sin,
                   void *q_out, int32_t *status, cudaStream_t stream);

/*
 * gdn_tree_build -- from parent int32 [B, T] (parent[t] < t; -1: a root, which follows the
 * committed tokens) the ancestors of each token and its rotation position:
 *   tree uint64 [B, T]: bit u set when u is t or an ancestor of t;
 *   pos  int32  [B, T]: seq_len[slot] + the number of t's ancestors (may be NULL).
 * Rows not in use: tree 0, pos seq_len.  T <= 64.
 */
int gdn_tree_build(const gdn_page_cache *cache, const gdn_attn_dims *dims, const int32_t *state_idx,
                   const int32_t *draft_len, const int32_t *parent, uint64_t *tree, int32_t *pos,
                   int32_t *status, cudaStream_t stream);

/*
 * gdn_attn_verify -- for row t < draft_len[b] and query head h, over the visible tokens j
 * (all committed ones, and draft token u where bit u of tree[b][t] is set; tree NULL: u <= t;
 * bits at or past draft_len[b] are ignored):
 *     s_j = scale q_t . k_j,   out = sum_j e^{s_j} v_j / sum_j e^{s_j},   lse = ln sum_j e^{s_j}.
 * A row that sees no token, or is not in use, gets out 0 and lse -inf.  What an unseen token's
 * rows hold (NaN and infinity included) has no effect.  A drafted token's infinite or NaN value is added as it
 * is to the rows that see it; a committed one's leaves infinity or NaN in its column (bf16: the weight's
 * second term may turn an infinity into NaN).  The draft's keys and values are read from the cache
 * (gdn_attn_stage).
 *   q, out dtype [B, T, Hq, d] (16-byte aligned);  lse fp32 [B, T, Hq] or NULL;
 *   tree uint64 [B, T] or NULL;  workspace: workspace_bytes >= gdn_attn_workspace() bytes, 16-byte
 *   aligned, no initial content; calls that overlap on the GPU need one each.
 * GDN_STATUS_BAD_SLOT, _BAD_LEN, _NO_ROOM as in gdn_attn_stage: the sequence's out and lse are
 * left unwritten; _BAD_PAGE: the sequence's out and lse are unspecified; _TIMEOUT, _DRAIN as in
 * gdnreplay.h: no output of the call may be trusted.
 */
int gdn_attn_verify(const gdn_page_cache *cache, int32_t layer, const gdn_attn_dims *dims,
                    const int32_t *state_idx, const int32_t *draft_len, const void *q,
                    const uint64_t *tree, void *out, float *lse, void *workspace,
                    int64_t workspace_bytes, int32_t *status, cudaStream_t stream);

/* Bytes of workspace that gdn_attn_verify needs for these dims on the current device, or a
 * negative GDN_ERR_* code. */
int64_t gdn_attn_workspace(const gdn_page_cache *cache, const gdn_attn_dims *dims);

/*
 * gdn_attn_accept -- for every sequence, p = accepted[b] and path int32 [B, T] (strictly
 * increasing over its first p entries; NULL: 0, 1, 2, ...): in every layer's k and v the row of
 * token seq_len + path[j] is moved to token seq_len + j, j < p, and new_len[slot] = seq_len + p.
 * new_len may be seq_len itself; only the batch's slots are written.  T <= 64.
 * GDN_STATUS_BAD_SLOT, _BAD_LEN, _BAD_ACCEPT (p outside [0, T]), _BAD_TREE, _NO_ROOM, _BAD_PAGE: the
 * sequence is skipped, new_len unwritten.
 */
int gdn_attn_accept(const gdn_page_cache *cache, int32_t B, int32_t T, const int32_t *state_idx,
                    const int32_t *path, const int32_t *accepted, int32_t *new_len, int32_t *status,
                    cudaStream_t stream);

/* Rows of slots that one gdn_pages_* call takes at most. */
#define GDN_PAGES_MAX_ROWS 4096

/*
 * gdn_pages_reserve -- room for `extra` tokens past seq_len in each of the n slots (int32 [n],
 * distinct): ceil((seq_len + extra) / page) - n_owned pages are taken from the free list, in the
 * order of the rows.  From the first row that the free list cannot serve on, rows that need pages
 * are skipped (GDN_STATUS_NO_PAGES).  _NO_ROOM: more than max_pages pages; _BAD_SLOT, _BAD_LEN (seq_len or
 * n_owned out of range): the row is skipped.
 */
int gdn_pages_reserve(const gdn_page_cache *cache, int32_t n, const int32_t *slots, int32_t extra,
                      int32_t *status, cudaStream_t stream);

/*
 * gdn_pages_fork -- sequence dst[i] (an empty slot: n_owned 0) becomes a copy of the committed
 * tokens of src[i]: it shares the full pages and, where seq_len is not a multiple of page, takes
 * one free page for the rest.  copies int32 [n, 2] gets that page's (source, copy), or (-1, -1):
 * gdn_pages_copy then copies its rows.  dst distinct and disjoint from src.  Rows are served
 * in order; _NO_PAGES as in gdn_pages_reserve; _BAD_SLOT (also: dst in use), _BAD_LEN: the row is skipped.
 */
int gdn_pages_fork(const gdn_page_cache *cache, int32_t n, const int32_t *src, const int32_t *dst,
                   int32_t *copies, int32_t *status, cudaStream_t stream);

/* gdn_pages_copy -- k and v of page copies[i][0] into page copies[i][1] in every layer; pairs of
 * (-1, -1) are passed over, others outside [0, n_page) set GDN_STATUS_BAD_PAGE.  No page may be both a
 * source and a copy. */
int gdn_pages_copy(const gdn_page_cache *cache, int32_t n, const int32_t *copies, int32_t *status,
                   cudaStream_t stream);

/*
 * gdn_pages_release -- the n slots (distinct) give up their pages: each page's count drops by one,
 * and pages that reach zero go to the end of the free list in the order of their last (row,
 * block-table entry).  seq_len and n_owned become 0.  A page released more often than it was
 * shared sets GDN_STATUS_BAD_PAGE and is not pushed.  _BAD_SLOT, _BAD_LEN (n_owned out of range): the
 * row is skipped.
 */
int gdn_pages_release(const gdn_page_cache *cache, int32_t n, const int32_t *slots, int32_t *status,
                      cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDNATTN_H */
