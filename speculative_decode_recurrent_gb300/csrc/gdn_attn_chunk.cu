// gdn_attn_chunk.cu -- attention of a chunk of new tokens over the paged cache, for sm_103a: the C ABI entry
// points (include/gdnattn.h), the kernel on the CUDA cores (fp32 caches: the tensor cores have no fp32 product, and fp32 out
// of products of bf16 terms, six for each, is not built) and the join of its split keys.  bf16 caches take gdn_attn_chunk_tc.cu.
//
// Mathematics.  One pass over a row's keys with the running maximum m and sum l of its softmax in powers
// of two: for each tile of keys m' = max(m, max s), o <- 2^(m - m') o + sum_j 2^(s_j - m') v_j, l likewise; out = o / l,
// lse = (m + log2 l) ln 2.  Parts of the key axis join by the same rule.
#include <cuda_bf16.h>

#include "chunk_common.h"
#include "tc_common.cuh"

namespace gdn {
namespace {

constexpr int kRT = 64, kKT = 64, kThreads = 256;   // rows and keys of a tile
constexpr int kMaxSplits = 64;
using tc::sm_count;

template <int D> struct CorePlan {
    static constexpr int LD = D + 4;                // padded rows: 16 keys at the same column hit all banks
    static constexpr int LP = kKT + 4;
    static constexpr int FLOATS = kRT * LD + kKT * LD + kKT * D + kRT * LP;
    static constexpr int BYTES = FLOATS * 4;
};

__device__ __forceinline__ float4 load4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }

// 64 rows x 64 keys a tile, 16 x 16 threads with 4 x 4 scores and 4 x D / 16 sums each.  A tile's 16 reads of 16
// bytes serve 64 products in 32 two-wide instructions, so the products bound it, then the tile's
// loads, which nothing hides within a CTA (29 TFLOP/s over long contexts; 3 of 67 to 150 tokens after 5 to 700 38 us).
template <int D>
__global__ void __launch_bounds__(kThreads) chunk_core_kernel(const ChunkArgs a)
{
    using P = CorePlan<D>;
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm, *sK = sQ + kRT * P::LD, *sV = sK + kKT * P::LD, *sP = sV + kKT * D;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int rt = a.row_tiles - 1 - blockIdx.x / a.splits, part = blockIdx.x % a.splits;       // long ones first
    const int h = blockIdx.y, b = blockIdx.z, G = a.G, Hkv = a.s.Hkv;
    pdl_wait();
    pdl_release();
    const Seq sq = load_seq<true>(a.s, b);
    if (sq.bad) {
        if (tid == 0 && blockIdx.x == 0 && h == 0) atomicOr(a.s.status, sq.bad);
        return;
    }
    const int t0 = rt * a.tpt, live = min(a.tpt, sq.n - t0) * G;      // rows in use (may be <= 0)
    const int rows = min(a.tpt, a.s.T - t0) * G;                      // rows of the tensor
    const size_t row0 = (static_cast<size_t>(b) * a.s.T + t0) * a.Hq + h * G;
    // row r of the tile is token t0 + r / G, head h G + r % G
    auto at = [&](int r) { return row0 + static_cast<size_t>(r / G) * a.Hq + r % G; };
    float *out = static_cast<float *>(a.out);
    if (live <= 0) {
        if (part == 0)
            for (int r = ty; r < rows; r += 16) {
                for (int c = tx * 4; c < D; c += 64) *reinterpret_cast<float4 *>(out + at(r) * D + c) = make_float4(0.f, 0.f, 0.f, 0.f);
                if (a.lse && tx == 0) a.lse[at(r)] = -INFINITY;
            }
        return;
    }
    const int total = sq.len + sq.n, keys = sq.len + t0 + (live + G - 1) / G;      // those that the tile's last row sees
    int first, end;
    part_range((keys + kKT - 1) / kKT, part, a.splits, first, end);
    for (int e = tid; e < kRT * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        *reinterpret_cast<float4 *>(sQ + r * P::LD + c) =
            r < live ? load4(static_cast<const float *>(a.q) + at(r) * D + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float2 o[4][D / 32];
    float m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) o[i][c] = make_float2(0.f, 0.f);
    }
    int lim[4];                                                       // keys that each row sees
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        lim[i] = r < live ? sq.len + t0 + r / G + 1 : 0;
    }
    const int32_t *tab = a.s.table + static_cast<size_t>(sq.slot) * a.s.max_pages;
    const int unseen = sq.len + t0 + 1;                               // tokens from here on are not seen by every row
    for (int kt = first; kt < end; ++kt) {
        __syncthreads();                                              // the tile before has been read
        bool odd = false;                                             // an infinite or NaN value of such a token
        for (int e = tid; e < kKT * (D / 4); e += kThreads) {
            const int r = e / (D / 4), c = e % (D / 4) * 4, j = kt * kKT + r;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
            if (j < total) {
                const int id = __ldg(tab + (j >> a.s.page_shift));
                if (id < 0 || id >= a.s.n_page) {
                    if (c == 0) atomicOr(a.s.status, GDN_STATUS_BAD_PAGE);
                } else {
                    const size_t off = (((static_cast<size_t>(id) * Hkv + h) << a.s.page_shift) + (j & ((1 << a.s.page_shift) - 1))) * D + c;
                    x = load4(static_cast<const float *>(a.k) + off);
                    y = load4(static_cast<const float *>(a.v) + off);
                    odd |= j >= unseen && !(fabsf(y.x) < INFINITY && fabsf(y.y) < INFINITY && fabsf(y.z) < INFINITY && fabsf(y.w) < INFINITY);
                }
            }
            *reinterpret_cast<float4 *>(sK + r * P::LD + c) = x;
            *reinterpret_cast<float4 *>(sV + r * D + c) = y;
        }
        odd = __syncthreads_or(odd);
        float2 s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            float4 x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(sQ + (ty * 4 + i) * P::LD + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(sK + (tx + 16 * j) * P::LD + c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = fma2(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), s[i][j]);
                    s[i][j] = fma2(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), s[i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[4], top = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = kt * kKT + tx + 16 * j < lim[i] ? (s[i][j].x + s[i][j].y) * a.scale_log2 : -INFINITY;
                top = fmaxf(top, x[j]);
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float ref = top == -INFINITY ? 0.f : top, fix = exp2f(m[i] - ref);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = exp2f(x[j] - ref);
                sum += x[j];
                sP[(ty * 4 + i) * P::LP + tx + 16 * j] = x[j];
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l[i] = l[i] * fix + sum;
            m[i] = top;
            const float2 f2 = make_float2(fix, fix);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) o[i][c] = mul2(o[i][c], f2);
        }
        __syncwarp();                                                 // a row's weights are its half-warp's own
        if (!odd) {
            for (int j = 0; j < kKT; j += 4) {
                float4 p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4 *>(sP + (ty * 4 + i) * P::LP + j);
#pragma unroll
                for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const float4 y = *reinterpret_cast<const float4 *>(sV + (j + jj) * D + tx * 4 + 64 * c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float w = jj == 0 ? p[i].x : jj == 1 ? p[i].y : jj == 2 ? p[i].z : p[i].w;
                            const float2 w2 = make_float2(w, w);
                            o[i][2 * c] = fma2(w2, make_float2(y.x, y.y), o[i][2 * c]);
                            o[i][2 * c + 1] = fma2(w2, make_float2(y.z, y.w), o[i][2 * c + 1]);
                        }
                    }
            }
        } else {                                                      // a weight of 0 must not meet an infinity or NaN
#pragma unroll 1
            for (int j = 0; j < kKT; ++j)
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const float4 y = *reinterpret_cast<const float4 *>(sV + j * D + tx * 4 + 64 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float w = sP[(ty * 4 + i) * P::LP + j];
                        const float2 w2 = make_float2(w, w);
                        if (kt * kKT + j < lim[i]) {
                            o[i][2 * c] = fma2(w2, make_float2(y.x, y.y), o[i][2 * c]);
                            o[i][2 * c + 1] = fma2(w2, make_float2(y.z, y.w), o[i][2 * c + 1]);
                        }
                    }
                }
        }
        __syncwarp();
    }
    if (a.splits == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            if (r >= rows) continue;
            const bool use = r < live;
            const float inv = use ? 1.f / l[i] : 0.f;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                *reinterpret_cast<float4 *>(out + at(r) * D + tx * 4 + 64 * c) =
                    use ? make_float4(o[i][2 * c].x * inv, o[i][2 * c].y * inv, o[i][2 * c + 1].x * inv, o[i][2 * c + 1].y * inv)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
            if (a.lse && tx == 0) a.lse[at(r)] = use ? (m[i] + log2f(l[i])) * 0.6931471805599453f : -INFINITY;
        }
        return;
    }
    const size_t unit = (static_cast<size_t>(b) * Hkv + h) * a.row_tiles + rt;
    float *w = a.ws + (unit * a.splits + part) * (static_cast<size_t>(kRT) * (D + 2));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
            *reinterpret_cast<float4 *>(w + r * D + tx * 4 + 64 * c) =
                make_float4(o[i][2 * c].x, o[i][2 * c].y, o[i][2 * c + 1].x, o[i][2 * c + 1].y);
        if (tx == 0) {
            w[kRT * D + r] = m[i];
            w[kRT * (D + 1) + r] = l[i];
        }
    }
}

// A warp per row: the parts of its unit, in their order.  Rows not in use have been written already where their whole tile
// is not; the others get 0 here.
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(const ChunkArgs a)
{
    constexpr int tile_rows = kRT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.x % (tile_rows / 8) * 8 + warp, rt = blockIdx.x / (tile_rows / 8), h = blockIdx.y, b = blockIdx.z;
    pdl_wait();
    pdl_release();
    const Seq sq = load_seq<true>(a.s, b);
    const int t0 = rt * a.tpt, rows = min(a.tpt, a.s.T - t0) * a.G, live = min(a.tpt, sq.n - t0) * a.G;
    if (sq.bad || live <= 0 || r >= rows) return;
    const size_t row = (static_cast<size_t>(b) * a.s.T + t0 + r / a.G) * a.Hq + h * a.G + r % a.G;
    const size_t unit = (static_cast<size_t>(b) * a.s.Hkv + h) * a.row_tiles + rt;
    const size_t step = static_cast<size_t>(tile_rows) * (D + 2);
    const float *w = a.ws + unit * a.splits * step;
    float m = -INFINITY;
    if (r < live)
        for (int i = lane; i < a.splits; i += 32) m = fmaxf(m, w[i * step + static_cast<size_t>(tile_rows) * D + r]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float ref = m == -INFINITY ? 0.f : m;
    float o[D / 32], l = 0.f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[c] = 0.f;
    if (r < live)
        for (int i = 0; i < a.splits; ++i) {
            const float *p = w + i * step;
            const float li = p[static_cast<size_t>(tile_rows) * (D + 1) + r];
            if (li == 0.f) continue;                                  // a part without keys of this row
            const float f = exp2f(p[static_cast<size_t>(tile_rows) * D + r] - ref);
            l += f * li;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) o[c] += f * p[static_cast<size_t>(r) * D + lane + 32 * c];
        }
    const float inv = r < live ? 1.f / l : 0.f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        const float y = r < live ? o[c] * inv : 0.f;
        static_cast<float *>(a.out)[row * D + lane + 32 * c] = y;
    }
    if (a.lse && lane == 0) a.lse[row] = r < live ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

int core_tokens(const gdn_page_cache *c, const gdn_attn_dims *d) { return kRT / (d->Hq / c->Hkv); }
int core_tiles(const gdn_page_cache *c, const gdn_attn_dims *d) { return (d->T + core_tokens(c, d) - 1) / core_tokens(c, d); }
// Parts of the key axis: four CTAs for each SM, as far as one row tile has keys for them: 256 tokens after 20000
// (16 and 2 heads of 128) 1470 us, with two CTAs for each 1705, with one 1892; 3 of 150 after 400 (12 and 3 of 64) 35, 35, 49.
int core_splits(const gdn_page_cache *c, const gdn_attn_dims *d) {
    const long long units = static_cast<long long>(d->B) * c->Hkv * core_tiles(c, d), want = 4 * sm_count();
    const long long most = (static_cast<long long>(c->max_pages) * c->page + 4 * kKT - 1) / (4 * kKT);
    long long n = units >= want ? 1 : (want + units - 1) / units;
    if (n > most) n = most;
    return static_cast<int>(n > kMaxSplits ? kMaxSplits : n < 1 ? 1 : n);
}

template <int D>
int launch_core(const gdn_page_cache *c, const gdn_attn_dims *d, ChunkArgs a, cudaStream_t s) {
    using P = CorePlan<D>;
    a.tpt = core_tokens(c, d);
    a.row_tiles = core_tiles(c, d);
    a.splits = core_splits(c, d);
    if (cudaFuncSetAttribute(chunk_core_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::BYTES) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    const dim3 grid(static_cast<unsigned>(a.row_tiles) * a.splits, c->Hkv, d->B);
    if (launch_pdl(chunk_core_kernel<D>, grid, dim3(kThreads), P::BYTES, s, a) != cudaSuccess) return GDN_ERR_LAUNCH;
    if (a.splits > 1 &&
        launch_pdl(chunk_join_kernel<D>, dim3(static_cast<unsigned>(a.row_tiles) * (kRT / 8), c->Hkv, d->B), dim3(256), 0, s, a) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    return GDN_OK;
}

int check_chunk(const gdn_page_cache *c, const gdn_attn_dims *d) {
    if (const int rc = check_attn(c, d, 1 << 20)) return rc;
    if (static_cast<long long>(d->B) * d->T > 1 << 28) return GDN_ERR_DIMS;
    return GDN_OK;
}

}  // namespace

}  // namespace gdn

using namespace gdn;

extern "C" {

int64_t gdn_attn_chunk_workspace(const gdn_page_cache *c, const gdn_attn_dims *d)
{
    if (const int rc = check_chunk(c, d)) return rc;
    if (d->T <= 64) return gdn_attn_workspace(c, d);
    if (c->dtype == GDN_DTYPE_BF16) return chunk_tc_workspace(c, d);
    const int splits = core_splits(c, d);
    if (splits == 1) return 0;
    return static_cast<int64_t>(d->B) * c->Hkv * core_tiles(c, d) * splits * part_floats(kRT, c->d) * 4;
}

int gdn_attn_chunk(const gdn_page_cache *c, int32_t layer, const gdn_attn_dims *d, const int32_t *state_idx,
                   const int32_t *chunk_len, const void *q, void *out, float *lse, void *workspace,
                   int64_t workspace_bytes, int32_t *status, cudaStream_t stream)
{
    const int64_t need = gdn_attn_chunk_workspace(c, d);
    if (need < 0) return static_cast<int>(need);
    if (d->T <= 64)
        return gdn_attn_verify(c, layer, d, state_idx, chunk_len, q, nullptr, out, lse, workspace, workspace_bytes, status, stream);
    if (layer < 0 || layer >= c->n_layer || (!state_idx && c->n_slot < d->B)) return GDN_ERR_DIMS;
    if (d->B == 0) return GDN_OK;
    if (!c->k || !c->v || !c->block_table || !c->seq_len || !q || !out || !status || (need > 0 && !workspace))
        return GDN_ERR_NULL;
    if (workspace_bytes < need) return GDN_ERR_DIMS;
    if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16) || !aligned_to(q, 16) || !aligned_to(out, 16) ||
        !aligned_to(workspace, 16))
        return GDN_ERR_DIMS;
    const size_t off = layer_elems(c) * layer * elem_size(c->dtype);
    const ChunkArgs a{seq_args(c, d->B, d->T, state_idx, chunk_len, status), q, static_cast<const char *>(c->k) + off,
                      static_cast<const char *>(c->v) + off, out, lse, static_cast<float *>(workspace),
                      d->scale * 1.4426950408889634f, d->Hq, d->Hq / c->Hkv, 0, 0, 1, d->flags};
    if (c->dtype == GDN_DTYPE_BF16) return chunk_tc(c, d, a, stream);
    return c->d == 64 ? launch_core<64>(c, d, a, stream)
           : c->d == 128 ? launch_core<128>(c, d, a, stream) : launch_core<256>(c, d, a, stream);
}

}  // extern "C"
