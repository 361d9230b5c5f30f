// chunk_common.h -- definitions shared by the translation units of gdn_attn_chunk (not part of the public
// ABI; see include/gdnattn.h).
#pragma once

#include "attn_common.h"

namespace gdn {

// One launch (device pointers, layouts of gdnattn.h); k and v are the layer's.  A unit is (sequence, key head, row
// tile): the rows of `tpt` neighbouring tokens, row r = t G + g.  Its keys are cut into `splits` parts.
struct ChunkArgs {
    SeqArgs s;
    const void *q, *k, *v;
    void *out;
    float *lse, *ws;
    float scale_log2;
    int Hq, G, tpt, row_tiles, splits, flags;
};

// Tiles [first, end) of part i of `tiles`.
__device__ __forceinline__ void part_range(int tiles, int i, int parts, int &first, int &end) {
    first = static_cast<int>(static_cast<long long>(tiles) * i / parts);
    end = static_cast<int>(static_cast<long long>(tiles) * (i + 1) / parts);
}

// Partial results of a unit's part: o [rows][D] ([D][rows] of the bf16 kernel), m [rows], l [rows] in fp32; m in powers of two.
__host__ __device__ inline size_t part_floats(int rows, int d) { return static_cast<size_t>(rows) * (d + 2); }

// The bf16 kernel (gdn_attn_chunk_tc.cu).
int64_t chunk_tc_workspace(const gdn_page_cache *c, const gdn_attn_dims *d);
int chunk_tc(const gdn_page_cache *c, const gdn_attn_dims *d, ChunkArgs a, cudaStream_t s);

}  // namespace gdn
