/*
 * gdndraft.h -- C ABI of the step that closes a round of speculative decoding in libgdnreplay
 * (sm_103a): which of the drafted tokens the target's probabilities accept, and the token
 * that follows them.  Its results are what gdn_replay_accept, gdn_conv_accept and
 * gdn_attn_accept take.  Conventions as in gdnreplay.h.
 */
#ifndef GDNDRAFT_H
#define GDNDRAFT_H

#include <stdint.h>

#include "gdnreplay.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_STATUS_BAD_TOKEN 1024  /* a drafted token outside [0, V); the sequence accepts nothing */
#define GDN_STATUS_BAD_PROB  2048  /* a row of probabilities that a token has to be drawn from has no
                                      positive finite sum; next is -1 */

/*
 * gdn_draft_accept -- speculative sampling over a block of T tokens per sequence (a chain or a tree), of which token
 * 0 is already decided (the token that the last step drew) and the others are drafts.  With p_t = probs[b,t],
 * the target's distribution after token t, and q_t = draft[b,t], the one that t's children were drawn
 * from (independently of one another), the walk starts at token 0 and takes the children x of the current
 * token, in the order of their numbers, by rejection sampling: with r = p at first and m = 1,
 *     x is accepted where u[b][x's number] q(x) m < r(x);
 *     rejected, r becomes max(r - m q, 0) and m its sum.
 * (In one step: r = max(p - c q, 0), c the sum of the masses m so far.)  An accepted child is the current token, with r
 * and m anew.  When no child is left, the next token is drawn from r: the smallest v with sum_{w <= v} r(w) > u[b][0]
 * sum_w r(w); from p where r has no mass.  draft NULL: a drafter that is certain of each child (q is 1 at it):
 * r loses the rejected tokens, and m is 1 less their p.  The accepted tokens and the next one are then distributed as
 * the target's (the random numbers u uniform in [0, 1)).  Terms and sums are held to 2^-46 of the probabilities or better.
 *   tokens   int32 [B, T]     the block's tokens (token 0 is not looked at)
 *   parent   int32 [B, T]     as in gdn_tree_build (gdnattn.h): parent[t] < t; -1 past token 0: never reached;
 *                             NULL: a chain
 *   probs    fp32  [B, T, V]  rows p_stride apart; entries >= 0 (negative ones and NaN count as 0) of sum 1
 *   draft    fp32  [B, T, V]  rows q_stride apart, finite, >= 0; NULL: see above
 *   u        fp32  [B, T]     in [0, 1)
 *   draft_len int32 [B]       tokens of the block in use, 0..T (NULL: T)
 *   accepted int32 [B]        accepted tokens, token 0 among them (0 when draft_len is 0)
 *   next     int32 [B]        the token that follows them (-1 when draft_len is 0)
 *   path     int32 [B, T]     their numbers, increasing, then -1 (may be NULL for a chain)
 * GDN_STATUS_BAD_LEN (draft_len), _BAD_TOKEN, _BAD_TREE (gdnattn.h; a parent outside [-1, t)): accepted 0, next -1, path
 * -1.
 */
typedef struct {
    int32_t B;          /* sequences, 0..65535 */
    int32_t T;          /* tokens of a block, 1..64 */
    int32_t V;          /* vocabulary, 1..2^24 */
    int32_t flags;      /* 0 */
    int64_t p_stride, q_stride;   /* elements from row to row, >= V (q_stride: 0 without draft) */
} gdn_draft_dims;

int gdn_draft_accept(const gdn_draft_dims *dims, const int32_t *tokens, const int32_t *parent,
                     const float *probs, const float *draft, const float *u, const int32_t *draft_len,
                     int32_t *accepted, int32_t *next, int32_t *path, int32_t *status, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDNDRAFT_H */
