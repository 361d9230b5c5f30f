// attn_common.h -- definitions shared by the translation units of the attention-layer
// operators (not part of the public ABI; see include/gdnattn.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdnattn.h"
#include "pair_math.cuh"
#include "replay_common.h"

namespace gdn {

// What a kernel needs to find a sequence's rows in the cache.
struct SeqArgs {
    const int32_t *state_idx, *draft_len, *seq_len, *table;
    const int32_t *owned;                       // NULL: the caller keeps the pages
    int32_t *status;
    int B, T, n_slot, max_pages, n_page, page_shift, Hkv;
};

struct Seq {
    int slot, len, n;           // slot, committed tokens, draft rows in use
    int own;                    // block-table entries of its own
    int bad;                    // GDN_STATUS_* bit, 0 when the sequence is sound
};

// Block-table entries of a slot that are its own.  Those behind them may hold pages that another
// sequence has by now (a release leaves them, a reserve without free pages does not replace them).
__device__ __forceinline__ int owned_pages(const SeqArgs &s, int slot) { return s.owned ? s.owned[slot] : s.max_pages; }

// PAGES: the sequence's committed and drafted tokens have to lie in pages of its own.
template <bool PAGES> __device__ __forceinline__ Seq load_seq(const SeqArgs &s, int b) {
    Seq q;
    q.slot = s.state_idx ? s.state_idx[b] : b;
    q.n = s.draft_len ? s.draft_len[b] : s.T;
    q.bad = 0;
    q.len = q.own = 0;
    if (q.slot < 0 || q.slot >= s.n_slot) {
        q.bad = GDN_STATUS_BAD_SLOT;
        return q;
    }
    q.len = s.seq_len[q.slot];
    q.own = owned_pages(s, q.slot);
    const int room = s.max_pages << s.page_shift;                 // <= 2^24
    if (q.len < 0 || q.len > room || q.n < 0 || q.n > s.T) q.bad = GDN_STATUS_BAD_LEN;
    else if (q.len + q.n > room) q.bad = GDN_STATUS_NO_ROOM;
    else if (PAGES && (q.len + q.n + (1 << s.page_shift) - 1) >> s.page_shift > q.own) q.bad = GDN_STATUS_BAD_PAGE;
    return q;
}

// One verify launch (device pointers, layouts of gdnattn.h); k and v are the layer's.
struct AttnArgs {
    SeqArgs s;
    const void *q, *k, *v;
    const uint64_t *tree;
    void *out;
    float *lse;
    float *ws;
    float scale_log2;           // score scale times log2(e): the kernels work in powers of two
    int Hq, G;                  // query heads, and per key head
    int splits;                 // parts of the key axis
    int flags;
};

// Draft rows of one key head's tile, tile after tile: row r = t G + g.
__device__ __forceinline__ uint64_t row_tree(const AttnArgs &a, int b, int t, int n) {
    const uint64_t live = n >= 64 ? ~0ull : (1ull << n) - 1;
    const uint64_t bits = a.tree ? a.tree[static_cast<size_t>(b) * a.s.T + t] : t >= 63 ? ~0ull : (2ull << t) - 1;
    return bits & live;
}

inline int page_shift(int page) {
    return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1;
}
inline bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
inline int elem_size(int dtype) { return dtype == GDN_DTYPE_BF16 ? 2 : 4; }

// Host checks of the cache's dims, and of a block's.
inline int check_cache(const gdn_page_cache *c) {
    if (!c) return GDN_ERR_NULL;
    if (c->dtype != GDN_DTYPE_BF16 && c->dtype != GDN_DTYPE_F32) return GDN_ERR_DTYPE;
    if (c->n_slot < 0 || c->max_pages < 1 || c->n_page < 1 || c->n_layer < 1 || c->n_layer > 32767 ||
        c->Hkv < 1 || c->Hkv > 128)
        return GDN_ERR_DIMS;
    if (page_shift(c->page) < 0 || (c->d != 64 && c->d != 128 && c->d != 256)) return GDN_ERR_DIMS;
    if (c->max_pages > 1 << 18 || static_cast<long long>(c->max_pages) * c->page > 1 << 24)
        return GDN_ERR_DIMS;                                      // sums over 4096 rows fit 32 bits
    if (static_cast<long long>(c->n_page) * c->Hkv * c->page > 0x7fffffffLL) return GDN_ERR_DIMS;
    return GDN_OK;
}
inline int check_attn(const gdn_page_cache *c, const gdn_attn_dims *a, int max_T) {
    if (const int rc = check_cache(c)) return rc;
    if (!a) return GDN_ERR_NULL;
    if (a->B < 0 || a->B > 65535 || a->T < 1 || a->T > max_T || (a->flags & ~(GDN_FLAG_TEST_EXPIRE | GDN_FLAG_TWO_TERMS))) return GDN_ERR_DIMS;
    if (static_cast<long long>(a->B) * a->T > (1ll << 30)) return GDN_ERR_DIMS;
    if (a->Hq < 1 || a->Hq % c->Hkv != 0 || a->Hq / c->Hkv > 64) return GDN_ERR_DIMS;
    if (!(a->scale > 0.f) || !(a->scale < 1e30f)) return GDN_ERR_DIMS;
    return GDN_OK;
}
inline SeqArgs seq_args(const gdn_page_cache *c, int B, int T, const int32_t *state_idx, const int32_t *draft_len,
                        int32_t *status) {
    return SeqArgs{state_idx, draft_len, c->seq_len, c->block_table, c->n_owned, status, B, T, c->n_slot, c->max_pages,
                   c->n_page, page_shift(c->page), c->Hkv};
}
// Elements of one layer's keys (or values).
inline size_t layer_elems(const gdn_page_cache *c) {
    return static_cast<size_t>(c->n_page) * c->Hkv * c->page * c->d;
}

// The bf16 verify (gdn_attn_tc.cu).
int64_t attn_tc_workspace(const gdn_page_cache *c, const gdn_attn_dims *d);
int attn_tc_verify(const gdn_page_cache *c, const gdn_attn_dims *d, const AttnArgs &a, cudaStream_t s);

}  // namespace gdn
