// gdn_attn.cu -- the attention layers' steps beside the verify's tensor-core kernel, for
// sm_103a: norm + rotation + staging of a draft block, ancestors of a token tree, the
// verify on CUDA cores, the accept.  C ABI and layouts: include/gdnattn.h.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_common.h"

namespace gdn {
namespace {

// ------------------------------------------------------------ rows of 8 elements
// Eight consecutive elements of a row per lane: 16 bytes of bf16, 32 of fp32.
template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> {
    struct Raw { uint4 x; };
    __device__ static Raw load(const __nv_bfloat16 *p) { return Raw{*reinterpret_cast<const uint4 *>(p)}; }
    __device__ static void store(__nv_bfloat16 *p, const Raw &r) { *reinterpret_cast<uint4 *>(p) = r.x; }
    __device__ static void unpack(const Raw &r, float (&f)[8]) {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&r.x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __bfloat1622float2(h[i]);
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
    __device__ static Raw pack(const float (&f)[8]) {
        Raw r;
        __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&r.x);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        return r;
    }
};
template <> struct Vec8<float> {
    struct Raw { float4 a, b; };
    __device__ static Raw load(const float *p) {
        return Raw{reinterpret_cast<const float4 *>(p)[0], reinterpret_cast<const float4 *>(p)[1]};
    }
    __device__ static void store(float *p, const Raw &r) {
        reinterpret_cast<float4 *>(p)[0] = r.a;
        reinterpret_cast<float4 *>(p)[1] = r.b;
    }
    __device__ static void unpack(const Raw &r, float (&f)[8]) {
        f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
        f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
    }
    __device__ static Raw pack(const float (&f)[8]) {
        return Raw{make_float4(f[0], f[1], f[2], f[3]), make_float4(f[4], f[5], f[6], f[7])};
    }
};

// ------------------------------------------------ norm + rotation + staging
struct StageArgs {
    SeqArgs s;
    const void *q, *k, *v;
    const int32_t *pos;
    const float *qw, *kw, *cos_sin;
    void *q_out, *kc, *vc;
    long long q_stride, k_stride, v_stride;
    int Hq, rot, style, max_pos;
    float eps;
};

constexpr int kStageThreads = 256;

// One CTA per token; D / 8 lanes per row (head of q, k or v), eight elements a lane, so
// every load and store is a whole 16-byte vector and a row's sum of squares is a few
// shuffles.  Pairs (i, i + rot/2) lie rot/16 lanes apart: one shuffle per element.
template <typename T, int D>
__global__ void __launch_bounds__(kStageThreads) stage_kernel(const StageArgs a)
{
    constexpr int L = D / 8, GROUPS = kStageThreads / L;
    using V = Vec8<T>;
    const int tok = blockIdx.x, b = tok / a.s.T, t = tok - b * a.s.T;
    const int c = threadIdx.x % L, grp = threadIdx.x / L;
    pdl_wait();
    pdl_release();
    const Seq sq = load_seq(a.s, b);
    if (sq.bad) {
        if (t == 0 && threadIdx.x == 0) atomicOr(a.s.status, sq.bad);
        return;
    }
    bool live = t < sq.n;
    int p = 0;
    if (live) {
        p = a.pos ? a.pos[tok] : sq.len + t;
        if (p < 0 || p >= a.max_pos) {
            if (threadIdx.x == 0) atomicOr(a.s.status, GDN_STATUS_BAD_POS);
            live = false;
        }
    }
    long long row0 = -1;                                          // cache row of head 0
    if (live) {
        const int at = sq.len + t, page = 1 << a.s.page_shift;
        const int id = a.s.table[static_cast<size_t>(sq.slot) * a.s.max_pages + (at >> a.s.page_shift)];
        if (id >= 0 && id < a.s.n_page) row0 = static_cast<long long>(id) * a.s.Hkv * page + (at & (page - 1));
        else if (threadIdx.x == 0) atomicOr(a.s.status, GDN_STATUS_BAD_PAGE);
    }
    const int half = a.rot / 16;                                  // lanes of half the rotated dims
    const bool turned = c < 2 * half;
    float cs[8], sn[8];
    if (live && turned) {
        const float *tab = a.cos_sin + static_cast<size_t>(p) * a.rot;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = a.style == GDN_ROPE_HALF ? (c < half ? c : c - half) * 8 + i : c * 4 + i / 2;
            cs[i] = tab[j];
            sn[i] = tab[a.rot / 2 + j];
        }
    }
    const int rows = a.Hq + 2 * a.s.Hkv;
    const int rounds = (rows + GROUPS - 1) / GROUPS;              // uniform: the shuffles take whole warps
    for (int i = 0; i < rounds; ++i) {
        const int r = i * GROUPS + grp;
        const bool in = r < rows;
        const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.s.Hkv;
        T *dst = nullptr;
        const T *src = nullptr;
        if (in) {
            if (is_q) {
                src = static_cast<const T *>(a.q) + static_cast<size_t>(tok) * a.q_stride + r * D;
                dst = static_cast<T *>(a.q_out) + (static_cast<size_t>(tok) * a.Hq + r) * D;
            } else {
                const int h = is_v ? r - a.Hq - a.s.Hkv : r - a.Hq;
                src = is_v ? static_cast<const T *>(a.v) + static_cast<size_t>(tok) * a.v_stride + h * D
                           : static_cast<const T *>(a.k) + static_cast<size_t>(tok) * a.k_stride + h * D;
                if (row0 >= 0) {
                    const size_t row = static_cast<size_t>(row0) + (static_cast<size_t>(h) << a.s.page_shift);
                    dst = static_cast<T *>(is_v ? a.vc : a.kc) + row * D;
                }
            }
        }
        typename V::Raw raw = {};
        if (in && live) raw = V::load(src + c * 8);
        float x[8];
        V::unpack(raw, x);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const float inv = 1.f / sqrtf(ss / D + a.eps);
        const float *w = is_q ? a.qw : a.kw;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e] * inv * w[c * 8 + e];
        if (a.rot > 0) {
            if (a.style == GDN_ROPE_HALF) {
                const int lane = threadIdx.x & 31;
                const int other = lane - c + (c < half ? c + half : turned ? c - half : c);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float z = __shfl_sync(0xffffffffu, y[e], other);
                    if (turned) y[e] = c < half ? y[e] * cs[e] - z * sn[e] : y[e] * cs[e] + z * sn[e];
                }
            } else if (turned) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float u = y[e], z = y[e + 1];
                    y[e] = u * cs[e] - z * sn[e];
                    y[e + 1] = z * cs[e] + u * sn[e];
                }
            }
        }
        if (!dst) continue;
        if (is_v) V::store(dst + c * 8, raw);
        else if (live) V::store(dst + c * 8, V::pack(y));
        else V::store(dst + c * 8, typename V::Raw{});            // a query row not in use
    }
}

// -------------------------------------------------------------- token trees
// One warp per sequence, tokens lane and lane + 32.  The ancestors of a token are its
// parent's and itself: pointer doubling joins them in six rounds.
__global__ void __launch_bounds__(128) tree_kernel(const SeqArgs s, const int32_t *parent, uint64_t *tree, int32_t *pos)
{
    __shared__ uint64_t bits[4][64];
    __shared__ int up[4][64];
    pdl_wait();
    pdl_release();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.x * 4 + w;
    if (b >= s.B) return;
    const Seq q = load_seq(s, b);
    int bad = q.bad;
    if (!bad) {
        bool wrong = false;
        for (int t = lane; t < 64; t += 32) {
            int p = -1;
            if (t < q.n) {
                p = parent[static_cast<size_t>(b) * s.T + t];
                if (p < -1 || p >= t) wrong = true, p = -1;
            }
            up[w][t] = p;
            bits[w][t] = t < q.n ? 1ull << t : 0ull;
        }
        if (__any_sync(0xffffffffu, wrong)) bad = GDN_STATUS_BAD_TREE;
    }
    if (bad) {                                                    // warp-uniform
        if (lane == 0) atomicOr(s.status, bad);
        return;
    }
    __syncwarp();
    for (int round = 0; round < 6; ++round) {
        uint64_t m[2];
        int p[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = lane + 32 * i, u = up[w][t];
            m[i] = bits[w][t] | (u >= 0 ? bits[w][u] : 0ull);
            p[i] = u >= 0 ? up[w][u] : -1;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bits[w][lane + 32 * i] = m[i];
            up[w][lane + 32 * i] = p[i];
        }
        __syncwarp();
    }
    for (int t = lane; t < s.T; t += 32) {
        const size_t at = static_cast<size_t>(b) * s.T + t;
        tree[at] = bits[w][t];
        if (pos) pos[at] = q.len + max(0, __popcll(bits[w][t]) - 1);
    }
}

// ------------------------------------------- verify on CUDA cores (fp32 caches)
constexpr int kRT = 32, kKT = 32;               // rows and keys of a tile
constexpr int kCoreThreads = 128;

template <int D> struct CorePlan {
    static constexpr int STR = D + 4;           // padded row: lanes of a warp read 8 rows without conflicts
    static constexpr int BYTES = (kRT * STR + kKT * STR + kKT * D + kRT * (kKT + 4)) * 4;
};

// Partial results in the workspace: [unit][split][kRT] rows of D sums, the maximum (in
// powers of two) and the denominator; unit = (b Hkv + h) row tiles + row tile.
template <int D> __host__ __device__ constexpr int part_floats() { return D + 2; }

// One CTA per (row tile, split of the keys, key head, sequence).  A warp owns 8 rows: their
// scores (2 rows x 4 keys a lane), their running maximum and denominator, and their
// D output columns (D / 32 a lane), so the only barriers are those around the shared
// key and value tiles.
template <int D>
__global__ void __launch_bounds__(kCoreThreads) verify_core_kernel(const AttnArgs a, int row_tiles)
{
    using P = CorePlan<D>;
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm, *sK = sQ + kRT * P::STR, *sV = sK + kKT * P::STR, *sP = sV + kKT * D;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = blockIdx.x / row_tiles, rt = blockIdx.x % row_tiles, h = blockIdx.y, b = blockIdx.z;
    pdl_wait();
    pdl_release();
    const Seq sq = load_seq(a.s, b);
    if (sq.bad) {
        if (blockIdx.x == 0 && h == 0 && tid == 0) atomicOr(a.s.status, sq.bad);
        return;
    }
    const int rows = a.s.T * a.G, r0 = rt * kRT;
    const int total = sq.len + sq.n, tiles = (total + kKT - 1) / kKT;
    const int j_beg = static_cast<int>(static_cast<long long>(tiles) * split / a.splits) * kKT;
    const int j_end = static_cast<int>(static_cast<long long>(tiles) * (split + 1) / a.splits) * kKT;
    for (int i = tid; i < kRT * D; i += kCoreThreads) {           // queries, scaled
        const int r = r0 + i / D, col = i % D;
        float x = 0.f;
        if (r < rows && r / a.G < sq.n) {
            const size_t at = ((static_cast<size_t>(b) * a.s.T + r / a.G) * a.Hq + h * a.G + r % a.G) * D + col;
            x = static_cast<const float *>(a.q)[at] * a.scale_log2;
        }
        sQ[(i / D) * P::STR + col] = x;
    }
    constexpr int C = D / 32;                                     // output columns per lane
    float acc[8][C], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int i = 0; i < C; ++i) acc[r][i] = 0.f;
    const int lr = lane >> 3, lk = lane & 7;                      // rows 8 warp + 2 lr + {0, 1}, keys lk + 8 i
    uint64_t bits[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = (r0 + 8 * warp + 2 * lr + i) / a.G;
        bits[i] = t < sq.n ? row_tree(a, b, t, sq.n) : 0ull;
    }
    bool used[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) used[i] = (r0 + 8 * warp + 2 * lr + i) / a.G < sq.n;
    const int page = 1 << a.s.page_shift;
    for (int j0 = j_beg; j0 < j_end; j0 += kKT) {
        __syncthreads();
        for (int i = tid; i < kKT * D / 8; i += kCoreThreads) {
            const int j = i / (D / 8), c8 = i % (D / 8), at = j0 + j;
            float fk[8], fv[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) fk[e] = fv[e] = 0.f;
            if (at < total) {
                const int id = a.s.table[static_cast<size_t>(sq.slot) * a.s.max_pages + (at >> a.s.page_shift)];
                if (id >= 0 && id < a.s.n_page) {
                    const size_t row = ((static_cast<size_t>(id) * a.s.Hkv + h) << a.s.page_shift) + (at & (page - 1));
                    Vec8<float>::unpack(Vec8<float>::load(static_cast<const float *>(a.k) + row * D + c8 * 8), fk);
                    Vec8<float>::unpack(Vec8<float>::load(static_cast<const float *>(a.v) + row * D + c8 * 8), fv);
                } else if (c8 == 0) {
                    atomicOr(a.s.status, GDN_STATUS_BAD_PAGE);
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sK[j * P::STR + c8 * 8 + e] = fk[e];
                sV[j * D + c8 * 8 + e] = fv[e];
            }
        }
        __syncthreads();
        float s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[i][k] = 0.f;
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            float4 q4[2], k4[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) q4[i] = *reinterpret_cast<const float4 *>(sQ + (8 * warp + 2 * lr + i) * P::STR + c);
#pragma unroll
            for (int k = 0; k < 4; ++k) k4[k] = *reinterpret_cast<const float4 *>(sK + (lk + 8 * k) * P::STR + c);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s[i][k] = fmaf(q4[i].x, k4[k].x, s[i][k]);
                    s[i][k] = fmaf(q4[i].y, k4[k].y, s[i][k]);
                    s[i][k] = fmaf(q4[i].z, k4[k].z, s[i][k]);
                    s[i][k] = fmaf(q4[i].w, k4[k].w, s[i][k]);
                }
        }
        // unseen keys: -infinity before the maximum, and -1 in place of their weight, so that
        // their values are passed over below whatever they hold
        float fac[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bool seen[4];
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int u = j0 + lk + 8 * k - sq.len;           // < 0: committed
                seen[k] = used[i] && (u < 0 || (u < sq.n && ((bits[i] >> u) & 1)));
                if (seen[k]) top = fmaxf(top, s[i][k]);
            }
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float mn = fmaxf(m[i], top), ms = mn == -INFINITY ? 0.f : mn;
            fac[i] = exp2f(m[i] - ms);                            // 0 for the first keys
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float p = exp2f(s[i][k] - ms);
                if (seen[k]) sum += p;
                sP[(8 * warp + 2 * lr + i) * (kKT + 4) + lk + 8 * k] = seen[k] ? p : -1.f;
            }
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l[i] = l[i] * fac[i] + sum;
            m[i] = mn;
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const float f = __shfl_sync(0xffffffffu, fac[r & 1], (r >> 1) * 8);
#pragma unroll
            for (int i = 0; i < C; ++i) acc[r][i] *= f;
        }
        for (int j = 0; j < kKT; ++j) {
            float v[C];
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] = sV[j * D + lane + 32 * i];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const float p = sP[(8 * warp + r) * (kKT + 4) + j];
                if (p == -1.f) continue;                          // unseen (warp-uniform)
#pragma unroll
                for (int i = 0; i < C; ++i) acc[r][i] = fmaf(p, v[i], acc[r][i]);
            }
        }
        __syncwarp();
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const float mm = __shfl_sync(0xffffffffu, m[r & 1], (r >> 1) * 8);
        const float ll = __shfl_sync(0xffffffffu, l[r & 1], (r >> 1) * 8);
        const int row = r0 + 8 * warp + r;
        if (row >= rows) continue;
        if (a.splits > 1) {
            const size_t unit = (static_cast<size_t>(b) * a.s.Hkv + h) * row_tiles + rt;
            float *dst = a.ws + ((unit * a.splits + split) * kRT + 8 * warp + r) * part_floats<D>();
#pragma unroll
            for (int i = 0; i < C; ++i) dst[lane + 32 * i] = acc[r][i];
            if (lane == 0) {
                dst[D] = mm;
                dst[D + 1] = ll;
            }
        } else {
            const size_t orow = (static_cast<size_t>(b) * a.s.T + row / a.G) * a.Hq + h * a.G + row % a.G;
            const float inv = ll > 0.f || ll != ll ? 1.f / ll : 0.f;
#pragma unroll
            for (int i = 0; i < C; ++i) static_cast<float *>(a.out)[orow * D + lane + 32 * i] = acc[r][i] * inv;
            if (a.lse && lane == 0) a.lse[orow] = (mm + log2f(ll)) * 0.69314718055994531f;
        }
    }
}

// Joins the splits' partial results of a row (a warp): their common maximum, then the
// weighted sums in the order of the splits.
template <int D>
__global__ void __launch_bounds__(128) verify_join_kernel(const AttnArgs a, int row_tiles)
{
    const int rows = a.s.T * a.G, lane = threadIdx.x & 31;
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5), h = blockIdx.y, b = blockIdx.z;
    pdl_wait();
    pdl_release();
    if (row >= rows || load_seq(a.s, b).bad) return;
    const size_t unit = (static_cast<size_t>(b) * a.s.Hkv + h) * row_tiles + row / kRT;
    const float *src = a.ws + (unit * a.splits * kRT + row % kRT) * part_floats<D>();
    const size_t step = static_cast<size_t>(kRT) * part_floats<D>();
    float m = -INFINITY;
    for (int i = lane; i < a.splits; i += 32) m = fmaxf(m, src[i * step + D]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float ms = m == -INFINITY ? 0.f : m;
    constexpr int C = D / 32;
    float acc[C], l = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) acc[i] = 0.f;
    for (int k = 0; k < a.splits; ++k) {
        const float f = exp2f(src[k * step + D] - ms);
        l = fmaf(f, src[k * step + D + 1], l);
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i] = fmaf(f, src[k * step + lane + 32 * i], acc[i]);
    }
    const size_t orow = (static_cast<size_t>(b) * a.s.T + row / a.G) * a.Hq + h * a.G + row % a.G;
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) static_cast<float *>(a.out)[orow * D + lane + 32 * i] = acc[i] * inv;
    if (a.lse && lane == 0) a.lse[orow] = (m + log2f(l)) * 0.69314718055994531f;
}

int core_row_tiles(const gdn_page_cache *c, const gdn_attn_dims *d) {
    return (d->T * (d->Hq / c->Hkv) + kRT - 1) / kRT;
}
int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}
// Parts of the key axis: enough CTAs for four per SM, each part at least two tiles of the
// longest sequence the block table can hold.
int core_splits(const gdn_page_cache *c, const gdn_attn_dims *d) {
    const long long units = static_cast<long long>(d->B) * c->Hkv * core_row_tiles(c, d);
    const long long tiles = (static_cast<long long>(c->max_pages) * c->page + kKT - 1) / kKT;
    long long want = units > 0 ? (4ll * sm_count() + units - 1) / units : 1;
    if (want > tiles / 2) want = tiles / 2;
    return static_cast<int>(want < 1 ? 1 : want > 128 ? 128 : want);
}

template <int D>
int launch_core(const gdn_page_cache *c, const gdn_attn_dims *d, AttnArgs a, cudaStream_t s) {
    const int rts = core_row_tiles(c, d);
    a.splits = core_splits(c, d);
    if (cudaFuncSetAttribute(verify_core_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             CorePlan<D>::BYTES) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    if (launch_pdl(verify_core_kernel<D>, dim3(rts * a.splits, c->Hkv, d->B), dim3(kCoreThreads),
                   CorePlan<D>::BYTES, s, a, rts) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    if (a.splits > 1 && launch_pdl(verify_join_kernel<D>, dim3((d->T * a.G + 3) / 4, c->Hkv, d->B), dim3(128), 0, s,
                                   a, rts) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    return GDN_OK;
}

// ---------------------------------------------------------------------- accept
constexpr int kAcceptThreads = 256, kAcceptCluster = 8;

struct AcceptArgs {
    SeqArgs s;
    void *k, *v;
    const int32_t *path, *accepted;
    int32_t *new_len;
    int n_layer, row_vecs;                       // 16-byte vectors of a row of one head
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// One cluster per sequence; a thread owns a 16-byte column of a (layer, k or v, head) and
// moves it row by row.  path[j] >= j and path increases, so a row is read before any
// later row's move writes over it; eight rows are read before the first of them is
// written (the eight writes go to rows below every row read later).  The length
// is written once every CTA of the cluster has read it (new_len may be seq_len).
__global__ void __launch_bounds__(kAcceptThreads) __cluster_dims__(kAcceptCluster, 1, 1)
accept_rows_kernel(const AcceptArgs a)
{
    __shared__ long long from[64], to[64];       // vectors of head 0 before the row's head offset
    __shared__ int fault;
    const int b = blockIdx.y, rank = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) fault = 0;
    pdl_wait();
    pdl_release();
    const Seq sq = load_seq(a.s, b);             // n = T
    const int p = a.accepted[b];
    int bad = sq.bad & ~GDN_STATUS_NO_ROOM;      // the draft's rows past the path need no room
    if (!bad && (p < 0 || p > a.s.T)) bad = GDN_STATUS_BAD_ACCEPT;
    const int page = 1 << a.s.page_shift, room = a.s.max_pages << a.s.page_shift;
    __syncthreads();
    if (!bad && tid < p) {
        const int j = tid;
        int src = j;
        if (a.path) {
            src = a.path[static_cast<size_t>(b) * a.s.T + j];
            const int prev = j > 0 ? a.path[static_cast<size_t>(b) * a.s.T + j - 1] : -1;
            if (src <= prev || src >= a.s.T) atomicOr(&fault, GDN_STATUS_BAD_TREE), src = j;
        }
        if (sq.len + src >= room) {
            atomicOr(&fault, GDN_STATUS_NO_ROOM);
        } else if (a.path) {
            const int32_t *tab = a.s.table + static_cast<size_t>(sq.slot) * a.s.max_pages;
            const int pf = sq.len + src, pt = sq.len + j;
            const int idf = tab[pf >> a.s.page_shift], idt = tab[pt >> a.s.page_shift];
            if (idf < 0 || idf >= a.s.n_page || idt < 0 || idt >= a.s.n_page) {
                atomicOr(&fault, GDN_STATUS_BAD_PAGE);
            } else {
                from[j] = ((static_cast<long long>(idf) * a.s.Hkv << a.s.page_shift) + (pf & (page - 1))) * a.row_vecs;
                to[j] = ((static_cast<long long>(idt) * a.s.Hkv << a.s.page_shift) + (pt & (page - 1))) * a.row_vecs;
            }
        }
    }
    __syncthreads();
    if (!bad) bad = fault;
    cluster_arrive();                            // this CTA has read the length
    if (!bad && a.path) {
        const int per_layer = 2 * a.s.Hkv * a.row_vecs, items = a.n_layer * per_layer;
        const size_t layer_vecs = (static_cast<size_t>(a.s.n_page) * a.s.Hkv << a.s.page_shift) * a.row_vecs;
        for (int it = rank * kAcceptThreads + tid; it < items; it += kAcceptCluster * kAcceptThreads) {
            const int layer = it / per_layer, r = it % per_layer, col = r % a.row_vecs;
            const int hv = r / a.row_vecs, h = hv % a.s.Hkv;
            uint4 *base = static_cast<uint4 *>(hv < a.s.Hkv ? a.k : a.v) + layer * layer_vecs +
                          (static_cast<size_t>(h) << a.s.page_shift) * a.row_vecs + col;
            for (int j0 = 0; j0 < p; j0 += 8) {
                uint4 x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j0 + j < p && from[j0 + j] != to[j0 + j]) x[j] = base[from[j0 + j]];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j0 + j < p && from[j0 + j] != to[j0 + j]) base[to[j0 + j]] = x[j];
            }
        }
    }
    cluster_wait();
    if (rank == 0 && tid == 0) {
        if (bad) atomicOr(a.s.status, bad);
        else a.new_len[sq.slot] = sq.len + p;
    }
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_attn_stage(const gdn_page_cache *c, int32_t layer, const gdn_attn_dims *d, const gdn_rope_dims *r,
                   const int32_t *state_idx, const int32_t *draft_len, const void *q, const void *k, const void *v,
                   const int32_t *pos, const float *q_weight, const float *k_weight, const float *cos_sin, void *q_out,
                   int32_t *status, cudaStream_t stream)
{
    if (const int rc = check_attn(c, d, 1 << 20)) return rc;
    if (!r) return GDN_ERR_NULL;
    if (layer < 0 || layer >= c->n_layer || r->rot < 0 || r->rot > c->d || r->rot % 16 != 0 ||
        (r->style != GDN_ROPE_HALF && r->style != GDN_ROPE_PAIRS) || r->max_pos < 1 || !(r->eps >= 0.f))
        return GDN_ERR_DIMS;
    const int e = elem_size(c->dtype);
    if (r->q_stride < static_cast<int64_t>(d->Hq) * c->d || r->k_stride < static_cast<int64_t>(c->Hkv) * c->d ||
        r->v_stride < static_cast<int64_t>(c->Hkv) * c->d || r->q_stride * e % 16 || r->k_stride * e % 16 ||
        r->v_stride * e % 16)
        return GDN_ERR_DIMS;
    if (!state_idx && c->n_slot < d->B) return GDN_ERR_DIMS;
    if (d->B == 0) return GDN_OK;
    if (!c->k || !c->v || !c->block_table || !c->seq_len || !q || !k || !v || !q_weight || !k_weight || !q_out ||
        !status || (r->rot > 0 && !cos_sin))
        return GDN_ERR_NULL;
    if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16) || !aligned_to(q, 16) || !aligned_to(k, 16) ||
        !aligned_to(v, 16) || !aligned_to(q_out, 16))
        return GDN_ERR_DIMS;
    const size_t off = layer_elems(c) * layer * e;
    StageArgs a{seq_args(c, d->B, d->T, state_idx, draft_len, status), q, k, v, pos, q_weight, k_weight, cos_sin,
                q_out, static_cast<char *>(c->k) + off, static_cast<char *>(c->v) + off, r->q_stride, r->k_stride,
                r->v_stride, d->Hq, r->rot, r->style, r->max_pos, r->eps};
    const dim3 grid(d->B * d->T), block(kStageThreads);
    cudaError_t err;
    if (c->dtype == GDN_DTYPE_BF16)
        err = c->d == 64 ? launch_pdl(stage_kernel<__nv_bfloat16, 64>, grid, block, 0, stream, a)
              : c->d == 128 ? launch_pdl(stage_kernel<__nv_bfloat16, 128>, grid, block, 0, stream, a)
                            : launch_pdl(stage_kernel<__nv_bfloat16, 256>, grid, block, 0, stream, a);
    else
        err = c->d == 64 ? launch_pdl(stage_kernel<float, 64>, grid, block, 0, stream, a)
              : c->d == 128 ? launch_pdl(stage_kernel<float, 128>, grid, block, 0, stream, a)
                            : launch_pdl(stage_kernel<float, 256>, grid, block, 0, stream, a);
    return err == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

int gdn_tree_build(const gdn_page_cache *c, const gdn_attn_dims *d, const int32_t *state_idx, const int32_t *draft_len,
                   const int32_t *parent, uint64_t *tree, int32_t *pos, int32_t *status, cudaStream_t stream)
{
    if (const int rc = check_attn(c, d, 64)) return rc;
    if (!state_idx && c->n_slot < d->B) return GDN_ERR_DIMS;
    if (d->B == 0) return GDN_OK;
    if (!c->seq_len || !parent || !tree || !status) return GDN_ERR_NULL;
    return launch_pdl(tree_kernel, dim3((d->B + 3) / 4), dim3(128), 0, stream,
                      seq_args(c, d->B, d->T, state_idx, draft_len, status), parent, tree, pos) == cudaSuccess
               ? GDN_OK : GDN_ERR_LAUNCH;
}

int64_t gdn_attn_workspace(const gdn_page_cache *c, const gdn_attn_dims *d)
{
    if (const int rc = check_attn(c, d, 64)) return rc;
    if (c->dtype == GDN_DTYPE_BF16) return attn_tc_workspace(c, d);
    const int splits = core_splits(c, d);
    if (splits == 1) return 0;
    return static_cast<int64_t>(d->B) * c->Hkv * core_row_tiles(c, d) * splits * kRT * (c->d + 2) * 4;
}

int gdn_attn_verify(const gdn_page_cache *c, int32_t layer, const gdn_attn_dims *d, const int32_t *state_idx,
                    const int32_t *draft_len, const void *q, const uint64_t *tree, void *out, float *lse,
                    void *workspace, int32_t *status, cudaStream_t stream)
{
    const int64_t need = gdn_attn_workspace(c, d);
    if (need < 0) return static_cast<int>(need);
    if (layer < 0 || layer >= c->n_layer || (!state_idx && c->n_slot < d->B)) return GDN_ERR_DIMS;
    if (d->B == 0) return GDN_OK;
    if (!c->k || !c->v || !c->block_table || !c->seq_len || !q || !out || !status || (need > 0 && !workspace))
        return GDN_ERR_NULL;
    if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16) || !aligned_to(q, 16) || !aligned_to(out, 16) ||
        !aligned_to(workspace, 16))
        return GDN_ERR_DIMS;
    const size_t off = layer_elems(c) * layer * elem_size(c->dtype);
    AttnArgs a{seq_args(c, d->B, d->T, state_idx, draft_len, status), q, static_cast<const char *>(c->k) + off,
               static_cast<const char *>(c->v) + off, tree, out, lse, static_cast<float *>(workspace),
               d->scale * 1.4426950408889634f, d->Hq, d->Hq / c->Hkv, 1, d->flags};
    if (c->dtype == GDN_DTYPE_BF16) return attn_tc_verify(c, d, a, stream);
    return c->d == 64 ? launch_core<64>(c, d, a, stream)
           : c->d == 128 ? launch_core<128>(c, d, a, stream) : launch_core<256>(c, d, a, stream);
}

int gdn_attn_accept(const gdn_page_cache *c, int32_t B, int32_t T, const int32_t *state_idx, const int32_t *path,
                    const int32_t *accepted, int32_t *new_len, int32_t *status, cudaStream_t stream)
{
    if (const int rc = check_cache(c)) return rc;
    if (B < 0 || B > 65535 || T < 1 || T > 64 || (!state_idx && c->n_slot < B)) return GDN_ERR_DIMS;
    if (B == 0) return GDN_OK;
    if (!c->k || !c->v || !c->block_table || !c->seq_len || !accepted || !new_len || !status) return GDN_ERR_NULL;
    if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16)) return GDN_ERR_DIMS;
    AcceptArgs a{seq_args(c, B, T, state_idx, nullptr, status), c->k, c->v, path, accepted, new_len, c->n_layer,
                 c->d * elem_size(c->dtype) / 16};
    return launch_pdl(accept_rows_kernel, dim3(kAcceptCluster, B), dim3(kAcceptThreads), 0, stream, a) == cudaSuccess
               ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // extern "C"
