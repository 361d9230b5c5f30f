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

constexpr int kManyTokens = 4096;               // from which on a token gets one warp (some 27 tokens per SM)

// Four consecutive elements, twice per lane.
template <typename T> struct Vec4;
template <> struct Vec4<__nv_bfloat16> {
    using Raw = uint2;
    __device__ static void unpack(const uint2 &r, float (&f)[4]) {
        f[0] = __uint_as_float(r.x << 16);
        f[1] = __uint_as_float(r.x & 0xffff0000u);
        f[2] = __uint_as_float(r.y << 16);
        f[3] = __uint_as_float(r.y & 0xffff0000u);
    }
    __device__ static uint2 pack(const float (&f)[4]) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
        return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
};
template <> struct Vec4<float> {
    using Raw = uint4;
    __device__ static void unpack(const uint4 &r, float (&f)[4]) {
        f[0] = __uint_as_float(r.x);
        f[1] = __uint_as_float(r.y);
        f[2] = __uint_as_float(r.z);
        f[3] = __uint_as_float(r.w);
    }
    __device__ static uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

// y = x r w of one row (eight elements per lane, L lanes), the rotated pairs turned.
template <int D>
__device__ __forceinline__ void norm_turn(float (&x)[8], float4 wa, float4 wb, float eps, bool turned, bool half,
                                          const float (&cs)[4], const float (&sn)[4])
{
    float2 y[4], sq = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        y[e] = make_float2(x[2 * e], x[2 * e + 1]);
        sq = fma2(y[e], y[e], sq);
    }
    float ss = sq.x + sq.y;
#pragma unroll
    for (int off = D / 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float r = rsqrtf(ss * (1.f / D) + eps);                 // within 2 ulp
    const float2 wv[4] = {make_float2(wa.x, wa.y), make_float2(wa.z, wa.w), make_float2(wb.x, wb.y), make_float2(wb.z, wb.w)};
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = mul2(mul2(y[e], make_float2(r, r)), wv[e]);
    if (turned) {
        if (half) {                                               // pairs (y[e], y[e + 2])
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 c2 = make_float2(cs[2 * e], cs[2 * e + 1]), s2 = make_float2(sn[2 * e], sn[2 * e + 1]);
                const float2 u = y[e], z = y[2 + e];
                y[e] = fma2(u, c2, mul2(z, make_float2(-s2.x, -s2.y)));
                y[2 + e] = fma2(z, c2, mul2(u, s2));
            }
        } else {                                                  // pairs within a word of y
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[e] = make_float2(y[e].x * cs[e] - y[e].y * sn[e], y[e].y * cs[e] + y[e].x * sn[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x[2 * e] = y[e].x, x[2 * e + 1] = y[e].y;
}

// A CTA of W warps per token; D / 8 lanes per row (head of q, k or v).  A lane holds elements [a, a + 4) and
// [b, b + 4) of its row: with b = a + rot / 2 among the rotated dims of the half style, so that the
// pairs meet in one lane (turning them by shuffles cost eight more per row); elsewhere b = a + 4.
// NR rows per lane are requested before the chain slot -> length -> page, and the rotation's row, are
// waited for.  Few tokens are bound by that chain, and four warps share a token's rows (W 4: B 32,
// T 16, 20 heads of 128 in 3.4 us, with one warp 5.9); many are bound by instructions and then HBM,
// and one warp a token spends the least on the chain (W 1: 16,800 rows in use of 6 x 4096, 20 heads
// of 256: 75 us, 0.75 of the HBM peak; W 4: 89).
template <typename T, int D, bool HALF, int W, int NR>
__global__ void __launch_bounds__(32 * W) stage_kernel(const StageArgs a)
{
    constexpr int L = D / 8, GROUPS = 32 * W / L;
    using V = Vec4<T>;
    using Raw = typename V::Raw;
    const int tok = blockIdx.x, b = tok / a.s.T, t = tok - b * a.s.T;
    const int c = threadIdx.x % L, grp = threadIdx.x / L;
    const int rows = a.Hq + 2 * a.s.Hkv;
    const bool turned = 8 * c < a.rot;
    const int ea = HALF && turned ? 4 * c : 8 * c, eb = HALF && turned ? 4 * c + a.rot / 2 : 8 * c + 4;
    pdl_wait();
    pdl_release();
    const int n = a.s.draft_len ? a.s.draft_len[b] : a.s.T;
    const int slot = a.s.state_idx ? a.s.state_idx[b] : b;
    const bool in_use = t < n && n <= a.s.T;
    int p = in_use && a.pos ? a.pos[tok] : 0;
    auto source = [&](int r) {
        const T *base = r < a.Hq ? static_cast<const T *>(a.q) + static_cast<size_t>(tok) * a.q_stride + r * D
                        : r < a.Hq + a.s.Hkv
                            ? static_cast<const T *>(a.k) + static_cast<size_t>(tok) * a.k_stride + (r - a.Hq) * D
                            : static_cast<const T *>(a.v) + static_cast<size_t>(tok) * a.v_stride + (r - a.Hq - a.s.Hkv) * D;
        return base;
    };
    Raw ra[NR], rb[NR];
    auto request = [&](int r0) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int r = r0 + i * GROUPS + grp;
            ra[i] = Raw{};
            rb[i] = Raw{};
            if (in_use && r < rows) {
                const T *src = source(r);
                ra[i] = __ldcs(reinterpret_cast<const Raw *>(src + ea));
                rb[i] = __ldcs(reinterpret_cast<const Raw *>(src + eb));
            }
        }
    };
    request(0);
    // most rows are queries': their weights stay in registers
    const float4 wqa = *reinterpret_cast<const float4 *>(a.qw + ea), wqb = *reinterpret_cast<const float4 *>(a.qw + eb);
    int len = 0, own = 0, bad = 0;
    if (slot < 0 || slot >= a.s.n_slot) bad = GDN_STATUS_BAD_SLOT;
    else {
        const int room = a.s.max_pages << a.s.page_shift;
        len = a.s.seq_len[slot];
        own = owned_pages(a.s, slot);
        if (len < 0 || len > room || n < 0 || n > a.s.T) bad = GDN_STATUS_BAD_LEN;
        else if (len + n > room) bad = GDN_STATUS_NO_ROOM;
    }
    if (bad) {
        if (t == 0 && threadIdx.x == 0) atomicOr(a.s.status, bad);
        return;
    }
    bool live = in_use;
    if (live) {
        if (!a.pos) p = len + t;
        if (p < 0 || p >= a.max_pos) {
            if (threadIdx.x == 0) atomicOr(a.s.status, GDN_STATUS_BAD_POS);
            live = false;
        }
    }
    long long row0 = -1;                                          // cache row of head 0
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) {
        const int at = len + t, page = 1 << a.s.page_shift;
        const int id = a.s.table[static_cast<size_t>(slot) * a.s.max_pages + (at >> a.s.page_shift)];
        if (turned) {
            const float *tab = a.cos_sin + static_cast<size_t>(p) * a.rot + 4 * c;
            const float4 u = *reinterpret_cast<const float4 *>(tab);
            const float4 w = *reinterpret_cast<const float4 *>(tab + a.rot / 2);
            cs[0] = u.x; cs[1] = u.y; cs[2] = u.z; cs[3] = u.w;
            sn[0] = w.x; sn[1] = w.y; sn[2] = w.z; sn[3] = w.w;
        }
        if (id >= 0 && id < a.s.n_page && at >> a.s.page_shift < own) row0 = static_cast<long long>(id) * a.s.Hkv * page + (at & (page - 1));
        else if (threadIdx.x == 0) atomicOr(a.s.status, GDN_STATUS_BAD_PAGE);
    }
    for (int r0 = 0; r0 < rows; r0 += NR * GROUPS) {              // the same for the whole CTA
        if (r0 > 0) request(r0);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int r = r0 + i * GROUPS + grp;
            const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.s.Hkv;
            Raw ya = ra[i], yb = rb[i];
            if (__any_sync(0xffffffffu, !is_v && live)) {         // (whole warps: a row's lanes shuffle)
                float xa[4], xb[4], x[8];
                V::unpack(ya, xa);
                V::unpack(yb, xb);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = xa[e], x[4 + e] = xb[e];
                float4 wa = wqa, wb = wqb;
                if (!is_q) {
                    wa = *reinterpret_cast<const float4 *>(a.kw + ea);
                    wb = *reinterpret_cast<const float4 *>(a.kw + eb);
                }
                norm_turn<D>(x, wa, wb, a.eps, turned, HALF, cs, sn);
                if (!is_v) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) xa[e] = x[e], xb[e] = x[4 + e];
                    ya = V::pack(xa);
                    yb = V::pack(xb);
                }
            }
            if (r >= rows) continue;
            T *dst;
            if (is_q) {
                dst = static_cast<T *>(a.q_out) + (static_cast<size_t>(tok) * a.Hq + r) * D;
                if (!live) ya = Raw{}, yb = Raw{};                // a query row not in use
            } else {
                if (row0 < 0) continue;
                const int h = is_v ? r - a.Hq - a.s.Hkv : r - a.Hq;
                dst = static_cast<T *>(is_v ? a.vc : a.kc) + (row0 + (static_cast<long long>(h) << a.s.page_shift)) * D;
            }
            *reinterpret_cast<Raw *>(dst + ea) = ya;
            *reinterpret_cast<Raw *>(dst + eb) = yb;
        }
    }
}

template <typename T, int D>
cudaError_t launch_stage(const StageArgs &a, cudaStream_t s) {
    constexpr int NR4 = D == 256 ? 5 : D == 128 ? 3 : 2;          // 20 rows (16 + 2 + 2 heads) in one round
    const int tokens = a.s.B * a.s.T, W = tokens < kManyTokens ? 4 : 1;
    const dim3 grid(tokens), block(32 * W);
    const bool half = a.style == GDN_ROPE_HALF;
    if (W == 4)
        return half ? launch_pdl(stage_kernel<T, D, true, 4, NR4>, grid, block, 0, s, a)
                    : launch_pdl(stage_kernel<T, D, false, 4, NR4>, grid, block, 0, s, a);
    return half ? launch_pdl(stage_kernel<T, D, true, 1, 5>, grid, block, 0, s, a)
                : launch_pdl(stage_kernel<T, D, false, 1, 5>, grid, block, 0, s, a);
}

// -------------------------------------------------------------- token trees
// One warp per sequence, tokens lane and lane + 32.  The ancestors of a token are its
// parent's and itself: pointer doubling joins them in six rounds (a chain of 64 followed token by
// token would take 64).  Bound by latency.
__global__ void __launch_bounds__(128) tree_kernel(const SeqArgs s, const int32_t *parent, uint64_t *tree, int32_t *pos)
{
    __shared__ uint64_t bits[4][64];
    __shared__ int up[4][64];
    pdl_wait();
    pdl_release();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.x * 4 + w;
    if (b >= s.B) return;
    const Seq q = load_seq<false>(s, b);
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
// The mathematics of gdn_attn_tc.cu's verify in fp32 throughout (the tensor cores have no fp32
// product).  One CTA per (row tile, split of the keys, key head, sequence); key and value
// tiles of 32 tokens arrive by cp.async, the next pair while the present one is used.  A warp owns
// 8 rows: their scores (2 rows x 4 keys a lane), their running maximum and denominator, and their
// D output columns, so the only barriers are those around the tiles.  Products go two at a time
// (fma.rn.f32x2).  B 5, T 7, 12 query and 3 key heads of 64 over 333 to 2100 tokens: 17.5 us, 8 of them the
// products and shared-memory reads of a CTA's two tiles, 5 the join, the rest latency.
constexpr int kRT = 32, kKT = 32;               // rows and keys of a tile
constexpr int kCoreThreads = 128;

template <int D> struct CorePlan {
    static constexpr int STR = D + 4;           // padded row: lanes of a warp read 8 rows without conflicts
    static constexpr int PSTR = kKT + 4;
    static constexpr int TILE = kKT * STR + kKT * D;              // keys, then values
    static constexpr int BYTES = (kRT * STR + 2 * TILE + kRT * PSTR) * 4;
    static constexpr int CTAS = D == 64 ? 4 : D == 128 ? 2 : 1;   // per SM
    static_assert(CTAS * (BYTES + 1024) <= 228 * 1024, "shared memory");
};

__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool valid) {      // zeros when not valid
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Partial results in the workspace: [unit][split][kRT] rows of D sums, the maximum (in
// powers of two) and the denominator; unit = (b Hkv + h) row tiles + row tile.
template <int D> __host__ __device__ constexpr int part_floats() { return D + 2; }

template <int D>
__global__ void __launch_bounds__(kCoreThreads, CorePlan<D>::CTAS) verify_core_kernel(const AttnArgs a, int row_tiles)
{
    using P = CorePlan<D>;
    constexpr int VECS = D / 4;
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm, *tiles_s = sQ + kRT * P::STR, *sP = tiles_s + 2 * P::TILE;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = blockIdx.x / row_tiles, rt = blockIdx.x % row_tiles, h = blockIdx.y, b = blockIdx.z;
    pdl_wait();
    pdl_release();
    const Seq sq = load_seq<true>(a.s, b);
    if (sq.bad) {
        if (blockIdx.x == 0 && h == 0 && tid == 0) atomicOr(a.s.status, sq.bad);
        return;
    }
    const int rows = a.s.T * a.G, r0 = rt * kRT, live_rows = sq.n * a.G;
    const int total = r0 < live_rows ? sq.len + sq.n : 0, tiles = (total + kKT - 1) / kKT;   // no keys without rows in use
    const int t_beg = static_cast<int>(static_cast<long long>(tiles) * split / a.splits);
    const int t_end = static_cast<int>(static_cast<long long>(tiles) * (split + 1) / a.splits);
    const int page = 1 << a.s.page_shift;
    const int32_t *tab = a.s.table + static_cast<size_t>(sq.slot) * a.s.max_pages;
    auto request = [&](int tile) {                                // tile's keys and values on their way
        float *sK = tiles_s + (tile & 1) * P::TILE, *sV = sK + kKT * P::STR;
#pragma unroll 4
        for (int i = tid; i < kKT * VECS; i += kCoreThreads) {
            const int j = i / VECS, c = i % VECS, at = tile * kKT + j;
            size_t row = 0;
            if (at < total) {
                int id = __ldg(tab + (at >> a.s.page_shift));
                if (id < 0 || id >= a.s.n_page) {
                    if (c == 0) atomicOr(a.s.status, GDN_STATUS_BAD_PAGE);
                    id = 0;
                }
                row = ((static_cast<size_t>(id) * a.s.Hkv + h) << a.s.page_shift) + (at & (page - 1));
            }
            cp_async16(sK + j * P::STR + 4 * c, static_cast<const float *>(a.k) + row * D + 4 * c, at < total);
            cp_async16(sV + j * D + 4 * c, static_cast<const float *>(a.v) + row * D + 4 * c, at < total);
        }
    };
    if (t_beg < t_end) request(t_beg);
#pragma unroll 4
    for (int i = tid; i < kRT * VECS; i += kCoreThreads) {
        const int r = i / VECS, c = i % VECS, row = r0 + r, t = row / a.G;
        const bool valid = row < live_rows;
        const size_t at = valid ? ((static_cast<size_t>(b) * a.s.T + t) * a.Hq + h * a.G + row % a.G) * D + 4 * c : 0;
        cp_async16(sQ + r * P::STR + 4 * c, static_cast<const float *>(a.q) + at, valid);
    }
    cp_async_commit();
    constexpr int C = D / 64;                                     // pairs of output columns per lane: 2 lane + 64 i
    float2 acc[8][C];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int i = 0; i < C; ++i) acc[r][i] = make_float2(0.f, 0.f);
    const int lr = lane >> 3, lk = lane & 7;                      // rows 8 warp + 2 lr + {0, 1}, keys lk + 8 i
    const bool warp_live = r0 + 8 * warp < live_rows;
    uint64_t bits[2];
    bool used[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = r0 + 8 * warp + 2 * lr + i;
        used[i] = row < live_rows;
        bits[i] = used[i] ? row_tree(a, b, row / a.G, sq.n) : 0ull;
    }
    for (int tile = t_beg; tile < t_end; ++tile) {
        if (tile + 1 < t_end) request(tile + 1);
        cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
        const float *sK = tiles_s + (tile & 1) * P::TILE, *sV = sK + kKT * P::STR;
        const int j0 = tile * kKT;
        const bool edge = j0 + kKT > sq.len;                      // some tokens may be unseen
        if (warp_live) {
            float2 s2[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) s2[i][k] = make_float2(0.f, 0.f);
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
                        s2[i][k] = fma2(make_float2(q4[i].x, q4[i].y), make_float2(k4[k].x, k4[k].y), s2[i][k]);
                        s2[i][k] = fma2(make_float2(q4[i].z, q4[i].w), make_float2(k4[k].z, k4[k].w), s2[i][k]);
                    }
            }
            // unseen keys: -infinity before the maximum, and -1 in place of their weight, so that
            // their values are passed over below whatever they hold
            float fac[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                bool seen[4];
                float s[4], top = -INFINITY;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int u = j0 + lk + 8 * k - sq.len;       // < 0: committed
                    seen[k] = !edge || (used[i] && (u < 0 || (u < sq.n && ((bits[i] >> u) & 1))));
                    s[k] = (s2[i][k].x + s2[i][k].y) * a.scale_log2;
                    if (seen[k]) top = fmaxf(top, s[k]);
                }
#pragma unroll
                for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                const float mn = fmaxf(m[i], top), ms = mn == -INFINITY ? 0.f : mn;
                fac[i] = exp2f(m[i] - ms);                        // 0 for the first keys
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float p = exp2f(s[k] - ms);
                    if (seen[k]) sum += p;
                    sP[(8 * warp + 2 * lr + i) * P::PSTR + lk + 8 * k] = seen[k] ? p : -1.f;
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
                for (int i = 0; i < C; ++i) acc[r][i] = make_float2(acc[r][i].x * f, acc[r][i].y * f);
            }
            const float *pr = sP + 8 * warp * P::PSTR, *vr = sV + 2 * lane;
            if (!edge) {
#pragma unroll 2
                for (int j = 0; j < kKT; j += 4) {
                    float2 v[4][C];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int i = 0; i < C; ++i) v[k][i] = *reinterpret_cast<const float2 *>(vr + (j + k) * D + 64 * i);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float4 p = *reinterpret_cast<const float4 *>(pr + r * P::PSTR + j);
#pragma unroll
                        for (int i = 0; i < C; ++i) {
                            acc[r][i] = fma2(make_float2(p.x, p.x), v[0][i], acc[r][i]);
                            acc[r][i] = fma2(make_float2(p.y, p.y), v[1][i], acc[r][i]);
                            acc[r][i] = fma2(make_float2(p.z, p.z), v[2][i], acc[r][i]);
                            acc[r][i] = fma2(make_float2(p.w, p.w), v[3][i], acc[r][i]);
                        }
                    }
                }
            } else {
#pragma unroll 1
                for (int j = 0; j < kKT; j += 4) {
                    float2 v[4][C];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int i = 0; i < C; ++i) v[k][i] = *reinterpret_cast<const float2 *>(vr + (j + k) * D + 64 * i);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float4 p4 = *reinterpret_cast<const float4 *>(pr + r * P::PSTR + j);
                        const float p[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const bool seen = p[k] != -1.f;       // unseen: zero times zero, whatever the value is
                            const float2 pp = seen ? make_float2(p[k], p[k]) : make_float2(0.f, 0.f);
#pragma unroll
                            for (int i = 0; i < C; ++i)
                                acc[r][i] = fma2(pp, seen ? v[k][i] : make_float2(0.f, 0.f), acc[r][i]);
                        }
                    }
                }
            }
        }
        __syncthreads();                                          // the tile's place is free
    }
    cp_async_wait<0>();
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const float mm = __shfl_sync(0xffffffffu, m[r & 1], (r >> 1) * 8);
        const float ll = __shfl_sync(0xffffffffu, l[r & 1], (r >> 1) * 8);
        const int row = r0 + 8 * warp + r;
        if (row >= rows) continue;
        const bool in_use = row < live_rows;
        if (a.splits > 1) {
            const size_t unit = (static_cast<size_t>(b) * a.s.Hkv + h) * row_tiles + rt;
            float *dst = a.ws + ((unit * a.splits + split) * kRT + 8 * warp + r) * part_floats<D>();
#pragma unroll
            for (int i = 0; i < C; ++i) *reinterpret_cast<float2 *>(dst + 2 * lane + 64 * i) = acc[r][i];
            if (lane == 0) *reinterpret_cast<float2 *>(dst + D) = make_float2(in_use ? mm : -INFINITY, in_use ? ll : 0.f);
        } else {
            const size_t orow = (static_cast<size_t>(b) * a.s.T + row / a.G) * a.Hq + h * a.G + row % a.G;
            const bool any = in_use && (ll > 0.f || ll != ll);
            const float inv = any ? 1.f / ll : 0.f;
#pragma unroll
            for (int i = 0; i < C; ++i)
                *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + orow * D + 2 * lane + 64 * i) =
                    any ? make_float2(acc[r][i].x * inv, acc[r][i].y * inv) : make_float2(0.f, 0.f);
            if (a.lse && lane == 0) a.lse[orow] = any ? (mm + log2f(ll)) * 0.69314718055994531f : -INFINITY;
        }
    }
}

// Joins the splits' partial results of a row (a warp): lane k weighs splits k, k + 32, .., then
// the weighted sums in the order of the splits, eight of them requested at a time.
template <int D>
__global__ void __launch_bounds__(128) verify_join_kernel(const AttnArgs a, int row_tiles)
{
    const int rows = a.s.T * a.G, lane = threadIdx.x & 31;
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5), h = blockIdx.y, b = blockIdx.z;
    pdl_wait();
    pdl_release();
    if (row >= rows) return;
    const size_t unit = (static_cast<size_t>(b) * a.s.Hkv + h) * row_tiles + row / kRT;
    const float *src = a.ws + (unit * a.splits * kRT + row % kRT) * part_floats<D>();
    const size_t step = static_cast<size_t>(kRT) * part_floats<D>();
    if (load_seq<true>(a.s, b).bad) return;
    float w[4], m = -INFINITY, l = 0.f;                           // at most 128 splits
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = lane + 32 * i < a.splits ? src[(lane + 32 * i) * step + D] : -INFINITY;
        m = fmaxf(m, w[i]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = exp2f(w[i] - ms);                                  // 0 past the splits
        if (lane + 32 * i < a.splits) l = fmaf(w[i], src[(lane + 32 * i) * step + D + 1], l);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    constexpr int C = D / 64;
    float2 acc[C];
#pragma unroll
    for (int i = 0; i < C; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int k0 = 0; k0 < 128; k0 += 32) {
        if (k0 >= a.splits) break;
#pragma unroll 8
        for (int k = 0; k < min(32, a.splits - k0); ++k) {
            const float f = __shfl_sync(0xffffffffu, w[k0 / 32], k);
            const float *p = src + (k0 + k) * step + 2 * lane;
#pragma unroll
            for (int i = 0; i < C; ++i) acc[i] = fma2(make_float2(f, f), *reinterpret_cast<const float2 *>(p + 64 * i), acc[i]);
        }
    }
    const size_t orow = (static_cast<size_t>(b) * a.s.T + row / a.G) * a.Hq + h * a.G + row % a.G;
    const bool any = l > 0.f || l != l;                           // rows not in use: l = 0 in every split
    const float inv = any ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i)
        *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + orow * D + 2 * lane + 64 * i) =
            any ? make_float2(acc[i].x * inv, acc[i].y * inv) : make_float2(0.f, 0.f);
    if (a.lse && lane == 0) a.lse[orow] = any ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
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
// Parts of the key axis: the CTAs of as few whole waves as make kParts of them, of kWaves at most, each part
// at least two tiles of the longest sequence that the block table can hold.  A wave alone makes two parts
// or none where there are many units, and ragged batches end with the longest sequence's part: B 32, T 16,
// 8 and 2 heads of 128 over 500 to 4747 tokens 369 us with one wave, 234 so; B 64, T 4, 16 and 4 heads over
// 100 to 4000: 558 and 316; all sequences of one length cost the join instead (B 200, 128 tokens: 48 and
// 54 us; B 32, 4000 tokens: 340 and 311).  More parts (12): 230 and 310 us, but 28 instead of 26 for B 16.
constexpr int kParts = 8, kWaves = 6;
int core_splits(const gdn_page_cache *c, const gdn_attn_dims *d) {
    const int ctas = c->d == 64 ? CorePlan<64>::CTAS : c->d == 128 ? CorePlan<128>::CTAS : CorePlan<256>::CTAS;
    const long long units = static_cast<long long>(d->B) * c->Hkv * core_row_tiles(c, d);
    const long long tiles = (static_cast<long long>(c->max_pages) * c->page + kKT - 1) / kKT;
    const long long wave = static_cast<long long>(ctas) * sm_count();
    long long want = 1;
    for (int k = 1; k <= kWaves && units > 0 && want < kParts; ++k) want = k * wave / units;
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
// is written once every CTA of the cluster has read it (new_len may be seq_len).  Bound by HBM where
// there is much to move (96 sequences, T 64, 12 layers, 4 heads of 128: 149 MB in 28 us, 0.77 of
// the peak), by its chain of dependent reads elsewhere (32 sequences, 6 layers: 4.6 us).
__global__ void __launch_bounds__(kAcceptThreads) __cluster_dims__(kAcceptCluster, 1, 1)
accept_rows_kernel(const AcceptArgs a)
{
    __shared__ long long from[64], to[64];       // vectors of head 0 before the row's head offset
    __shared__ int fault;
    const int b = blockIdx.y, rank = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) fault = 0;
    pdl_wait();
    pdl_release();
    const Seq sq = load_seq<false>(a.s, b);      // n = T
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
        } else {
            const int pf = sq.len + src, pt = sq.len + j;
            bool lost = false;
            if (a.path) {
                const int32_t *tab = a.s.table + static_cast<size_t>(sq.slot) * a.s.max_pages;
                const int idf = tab[pf >> a.s.page_shift], idt = tab[pt >> a.s.page_shift];
                lost = idf < 0 || idf >= a.s.n_page || idt < 0 || idt >= a.s.n_page;
                from[j] = ((static_cast<long long>(idf) * a.s.Hkv << a.s.page_shift) + (pf & (page - 1))) * a.row_vecs;
                to[j] = ((static_cast<long long>(idt) * a.s.Hkv << a.s.page_shift) + (pt & (page - 1))) * a.row_vecs;
            }
            if (lost || pf >> a.s.page_shift >= sq.own) atomicOr(&fault, GDN_STATUS_BAD_PAGE);       // (pt <= pf)
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
        !aligned_to(v, 16) || !aligned_to(q_out, 16) || !aligned_to(q_weight, 16) || !aligned_to(k_weight, 16) ||
        !aligned_to(cos_sin, 16))
        return GDN_ERR_DIMS;
    const size_t off = layer_elems(c) * layer * e;
    StageArgs a{seq_args(c, d->B, d->T, state_idx, draft_len, status), q, k, v, pos, q_weight, k_weight, cos_sin,
                q_out, static_cast<char *>(c->k) + off, static_cast<char *>(c->v) + off, r->q_stride, r->k_stride,
                r->v_stride, d->Hq, r->rot, r->style, r->max_pos, r->eps};
    cudaError_t err;
    if (c->dtype == GDN_DTYPE_BF16)
        err = c->d == 64 ? launch_stage<__nv_bfloat16, 64>(a, stream)
              : c->d == 128 ? launch_stage<__nv_bfloat16, 128>(a, stream)
                            : launch_stage<__nv_bfloat16, 256>(a, stream);
    else
        err = c->d == 64 ? launch_stage<float, 64>(a, stream)
              : c->d == 128 ? launch_stage<float, 128>(a, stream) : launch_stage<float, 256>(a, stream);
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
                    void *workspace, int64_t workspace_bytes, int32_t *status, cudaStream_t stream)
{
    const int64_t need = gdn_attn_workspace(c, d);
    if (need < 0) return static_cast<int>(need);
    if (layer < 0 || layer >= c->n_layer || (!state_idx && c->n_slot < d->B)) return GDN_ERR_DIMS;
    if (d->B == 0) return GDN_OK;
    if (!c->k || !c->v || !c->block_table || !c->seq_len || !q || !out || !status || (need > 0 && !workspace))
        return GDN_ERR_NULL;
    if (workspace_bytes < need) return GDN_ERR_DIMS;
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
