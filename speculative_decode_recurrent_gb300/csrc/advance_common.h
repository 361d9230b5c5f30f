// advance_common.h -- definitions shared by the translation units of gdn_replay_advance (not part of the
// public ABI; see include/gdnreplay.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdnreplay.h"
#include "replay_common.h"

namespace gdn {

struct AdvanceArgs {
    float *state;
    const int32_t *state_idx, *buf_len, *chunk_len, *fresh;
    const void *q, *k, *v;
    const float *g, *beta;
    float *out;
    char *ws;
    int32_t *status;
    int64_t q_stride, k_stride, v_stride;
    int B, T, H, Hk, n_slot, flags;
    float scale;
};

// What a kernel needs to know of sequence b.
struct AdvanceSeq {
    int slot, n;
    bool fresh;
    int bad;                    // GDN_STATUS_* bit, 0 when the sequence is sound
};
__device__ __forceinline__ AdvanceSeq advance_seq(const AdvanceArgs &a, int b) {
    AdvanceSeq s;
    s.slot = a.state_idx ? a.state_idx[b] : b;
    s.n = a.chunk_len ? a.chunk_len[b] : a.T;
    s.fresh = a.fresh && a.fresh[b] != 0;
    s.bad = 0;
    if (s.slot < 0 || s.slot >= a.n_slot) s.bad = GDN_STATUS_BAD_SLOT;
    else if (s.n < 0 || s.n > a.T || (a.buf_len && a.buf_len[s.slot] != 0)) s.bad = GDN_STATUS_BAD_LEN;
    return s;
}

// The chunked form on the tensor cores (gdn_advance_tc.cu): bf16 inputs.
bool advance_tc_shape(const gdn_advance_dims *d);
int64_t advance_tc_workspace(const gdn_advance_dims *d);
int advance_tc(const gdn_advance_dims *d, const AdvanceArgs &a, cudaStream_t s);

}  // namespace gdn
