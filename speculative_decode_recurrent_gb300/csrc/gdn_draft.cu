// gdn_draft.cu -- drafted tokens verified against the target's probabilities, and the next token,
// for sm_103a.  C ABI and layouts: include/gdndraft.h.
//
// Mathematics.  At a node with target p and drafter q, each rejected child takes r to max(r - m q, 0) with m
// the mass of r.  As q >= 0, the nested maxima are one: r = max(p - c q, 0), c the sum of the masses so far
// (c = 1 after the first rejection).  So a rejection needs one number, the mass of the new r, and a row of p and
// of q is read again rather than kept.  A chain has no second child: its one rejection's mass is that of the
// row from which the next token is drawn, and one pass over the rows serves both.
//
// Precision.  The next token is where a running sum of up to 2^24 terms passes a threshold: in 32 bits the
// sums of 10^5 terms are off by more than many a term.  A term is p - c q in two fp32 words (exact for c = 1), and sums,
// masses and thresholds are two words throughout (46 bits and more), so a token differs from the 64-bit one's
// only where the threshold lies within some 2^-44 of a border.  Two words, because fp64 is slow on this chip: with 64-bit
// sums above the lanes' the search alone took 12 us, a whole call over 32768 probabilities 23.
//
// What bounds it: a few rows of V numbers per sequence, and a chain of dependent steps (tokens, their probabilities,
// the walk, the pass, its sum across the cluster, the search).  A cluster of eight CTAs takes a sequence, each a
// stretch of the vocabulary, in segments of 1024 terms per warp (256 or 512 where those would leave warps without one); two
// CTAs share an SM.
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdnattn.h"
#include "gdndraft.h"
#include "replay_common.h"

namespace gdn {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kMaxT = 64;
constexpr int kSmallV = 4096;                       // vocabularies that one CTA takes alone

struct DraftArgs {
    const int32_t *tokens, *parent;
    const float *probs, *draft, *u;
    const int32_t *draft_len;
    int32_t *accepted, *next, *path, *status;
    int64_t p_stride, q_stride;
    int B, T, V;
    int segs;                                       // segments of a CTA's stretch
};

// A number in two fp32 words: h + l.
struct Two {
    float h, l;
};
__device__ __forceinline__ Two sum_of(float a, float b) {             // exact
    const float s = a + b, bp = s - a;
    return Two{s, (a - (s - bp)) + (b - bp)};
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
    Two s = sum_of(a.h, b.h);
    s.l += a.l + b.l;
    const float h = s.h + s.l;                      // (|l| is far below |h|)
    return Two{h, s.l - (h - s.h)};
}
__device__ __forceinline__ Two operator-(Two a, Two b) { return a + Two{-b.h, -b.l}; }
__device__ __forceinline__ Two operator*(Two a, float b) {
    const float h = a.h * b;
    return Two{h, fmaf(a.h, b, -h) + a.l * b};
}
__device__ __forceinline__ bool operator<(Two a, Two b) {
    const Two d = sum_of(a.h, -b.h);
    return d.h + (d.l + (a.l - b.l)) < 0.f;
}
// (adding only, without bringing l back below h's last place)
__device__ __forceinline__ void gather(Two &s, float h, float l) {
    const Two t = sum_of(s.h, h);
    s.h = t.h;
    s.l += t.l + l;
}
__device__ __forceinline__ Two shuffle_xor(Two x, int off) {
    return Two{__shfl_xor_sync(0xffffffffu, x.h, off), __shfl_xor_sync(0xffffffffu, x.l, off)};
}
__device__ __forceinline__ Two shuffle(Two x, int lane) {
    return Two{__shfl_sync(0xffffffffu, x.h, lane), __shfl_sync(0xffffffffu, x.l, lane)};
}
// Sum over the lanes up to this one.
__device__ __forceinline__ Two scan(Two x, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const Two y{__shfl_up_sync(0xffffffffu, x.h, off), __shfl_up_sync(0xffffffffu, x.l, off)};
        if (lane >= off) x = x + y;
    }
    return x;
}

// max(p - c q, 0) in two words.
__device__ __forceinline__ void rest(float p, float q, Two c, float &h, float &l) {
    p = fmaxf(p, 0.f);                              // (NaN: 0)
    const float t = c.h * q, e = fmaf(c.l, q, fmaf(c.h, q, -t));
    const float d = p - t, bb = d - p;
    const float err = (p - (d - bb)) - (t + bb) - e;
    const bool some = !(d + err <= 0.f);            // (an infinity leaves NaN: the row has no sound sum)
    h = some ? d : 0.f;
    l = some ? err : 0.f;
}

// What a row of r is made of.
struct Rest {
    const float *p, *q;                             // q NULL: r is p
    Two c;
    const int *gone;                                // tokens that r has lost (draft NULL)
    int n_gone;
    __device__ void term(int v, float pv, float qv, float &h, float &l) const {
        if (q) {
            rest(pv, qv, c, h, l);
        } else {
            h = fmaxf(pv, 0.f);
            l = 0.f;
            for (int i = 0; i < n_gone; ++i)
                if (v == gone[i]) h = 0.f;
        }
    }
};

// Terms v .. v + 3 (0 past the vocabulary).
template <bool VEC>
__device__ __forceinline__ void load4(const float *row, int v, int V, float (&x)[4]) {
    if (VEC && v + 4 <= V) {
        const float4 y = __ldg(reinterpret_cast<const float4 *>(row + v));
        x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = v + j < V ? __ldg(row + v + j) : 0.f;
    }
}

// The sum of the segment of 128 ROWS terms at v0, in every lane.  Four rows at a time: with 64 registers two CTAs share an SM.
template <int ROWS, bool VEC>
__device__ __forceinline__ Two segment_sum(const Rest &r, int v0, int V, int lane) {
    constexpr int SOME = ROWS < 4 ? ROWS : 4;
    Two s[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 1
    for (int at = v0 + lane * 4; at < v0 + ROWS * 128; at += SOME * 128) {
        float p[SOME][4], q[SOME][4];
#pragma unroll
        for (int i = 0; i < SOME; ++i) load4<VEC>(r.p, at + i * 128, V, p[i]);
        if (r.q)
#pragma unroll
            for (int i = 0; i < SOME; ++i) load4<VEC>(r.q, at + i * 128, V, q[i]);
#pragma unroll
        for (int i = 0; i < SOME; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float h, l;
                r.term(at + i * 128 + j, p[i][j], r.q ? q[i][j] : 0.f, h, l);
                gather(s[j & 1], h, l);
            }
    }
    Two x = s[0] + s[1];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x = x + shuffle_xor(x, off);
    return shuffle(x, 0);
}

// The first term of the segment at v0 at which the running sum passes `target`; the last term above 0 where none does (the
// segment's sum was taken in another order) or `past` says so, -1 where there is none.
template <int ROWS, bool VEC>
__device__ __forceinline__ int segment_find(const Rest &r, int v0, int V, int lane, Two target, bool past) {
    Two s[ROWS];                                    // of this lane's four terms in each row, then of whole rows
    unsigned some = 0u;                             // rows with a term above 0 (this lane's, then all)
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int v = v0 + i * 128 + lane * 4;
        float p[4], q[4] = {0.f, 0.f, 0.f, 0.f};
        load4<VEC>(r.p, v, V, p);
        if (r.q) load4<VEC>(r.q, v, V, q);
        s[i] = Two{0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float h, l;
            r.term(v + j, p[j], q[j], h, l);
            gather(s[i], h, l);
            if (h > 0.f) some |= 1u << i;
        }
    }
    some = __reduce_or_sync(0xffffffffu, some);
    if (!some) return -1;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < ROWS; ++i) s[i] = s[i] + shuffle_xor(s[i], off);
    // the row: every lane takes the same steps
    Two before{0.f, 0.f}, sum{0.f, 0.f};
    int row = -1;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const Two next = sum + s[i];
        if (!past && row < 0 && ((some >> i) & 1) && target < next) {
            row = i;
            before = sum;
        }
        sum = next;
    }
    past = row < 0;                                 // none: the last term of the last row with one
    if (past) row = 31 - __clz(some);
    row = __shfl_sync(0xffffffffu, row, 0);
    const int v = v0 + row * 128 + lane * 4;
    float p[4], q[4] = {0.f, 0.f, 0.f, 0.f};
    load4<VEC>(r.p, v, V, p);
    if (r.q) load4<VEC>(r.q, v, V, q);
    Two x[4], mine{0.f, 0.f};
    int last = -1;
    bool over0[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float h, l;
        r.term(v + j, p[j], q[j], h, l);
        gather(mine, h, l);
        x[j] = mine;
        over0[j] = h > 0.f;
        if (over0[j]) last = v + j;
    }
    const Two excl = before + (scan(mine, lane) - mine);
    int hit = -1;
#pragma unroll
    for (int j = 3; j >= 0; --j)
        if (!past && over0[j] && target < excl + x[j]) hit = v + j;
    const unsigned m = __ballot_sync(0xffffffffu, hit >= 0);
    if (m) return __shfl_sync(0xffffffffu, hit, __ffs(m) - 1);
    return __shfl_sync(0xffffffffu, last, 31 - __clz(__ballot_sync(0xffffffffu, last >= 0)));
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// `x` to the same place of the CTA of rank `to`.
__device__ __forceinline__ void put_remote(Two *at, int to, Two x) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(at)), r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(to));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(r), "f"(x.h), "f"(x.l) : "memory");
}

template <int C, int ROWS, bool VEC>
__device__ __forceinline__ void accept_body(const DraftArgs &a)
{
    constexpr int SEG = ROWS * 128;                 // terms of a segment
    extern __shared__ __align__(16) float seg_raw[];
    Two *seg = reinterpret_cast<Two *>(seg_raw);    // [segs] sums of this CTA's segments
    __shared__ __align__(8) Two totals[2][kCluster];          // of the cluster's CTAs; by turns
    __shared__ int tok[kMaxT], par[kMaxT], taken[kMaxT], gone[kMaxT];
    __shared__ float sp[kMaxT], sq[kMaxT], su[kMaxT];
    __shared__ unsigned okay[2];                    // tokens that would be accepted as first children
    __shared__ int bad;
    const int b = blockIdx.y, rank = C > 1 ? blockIdx.x : 0, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int T = a.T, V = a.V;
    if (tid == 0) bad = 0;
    pdl_wait();
    pdl_release();
    const size_t row0 = static_cast<size_t>(b) * T;
    const int n = a.draft_len ? a.draft_len[b] : T;
    int up = tid - 1, x = 0;                        // (requested with draft_len)
    float u = 0.f;
    if (tid < T) {
        if (a.parent) up = a.parent[row0 + tid];
        x = a.tokens[row0 + tid];
        u = a.u[row0 + tid];
    }
    __syncthreads();
    if (n < 0 || n > T) {                           // the same in the whole cluster
        if (tid == 0) bad = GDN_STATUS_BAD_LEN;
    } else if (tid < kMaxT) {                       // (two whole warps)
        float p = 0.f, q = 0.f;
        bool first = false;                         // whether it would be accepted as a first child
        if (tid > 0 && tid < n) {
            if (x < 0 || x >= V) {
                atomicOr(&bad, GDN_STATUS_BAD_TOKEN);
            } else if (up < -1 || up >= tid) {
                atomicOr(&bad, GDN_STATUS_BAD_TREE);
            } else if (up >= 0) {
                p = fmaxf(a.probs[(row0 + up) * a.p_stride + x], 0.f);
                q = a.draft ? a.draft[(row0 + up) * a.q_stride + x] : 1.f;
                const float y = u * q;                                // u q < p, exactly
                first = y < p || (y == p && fmaf(u, q, -y) < 0.f);
            }
        }
        par[tid] = tid > 0 && tid < n ? up : -1;
        tok[tid] = x;
        sp[tid] = p;
        sq[tid] = q;
        su[tid] = u;
        const unsigned m = __ballot_sync(0xffffffffu, first);
        if (lane == 0) okay[warp] = m;
    }
    __syncthreads();
    if (bad || n == 0) {
        if (rank == 0) {
            if (a.path)
                for (int t = tid; t < T; t += kThreads) a.path[static_cast<size_t>(b) * T + t] = -1;
            if (tid == 0) {
                a.accepted[b] = 0;
                a.next[b] = -1;
                if (bad) atomicOr(a.status, bad);
            }
        }
        return;
    }
    // ---- the walk: every thread of the cluster takes the same steps
    int turn = 0;
    // The mass of r over the whole vocabulary, and what lies before this CTA's stretch; fills seg.
    const int first = rank * a.segs;                // this CTA's first segment
    auto pass = [&](const Rest &r, Two &before) -> Two {
        for (int s = warp; s < a.segs; s += kWarps) {
            const int v0 = (first + s) * SEG;       // (below 2^24 + 2^13 SEG)
            const Two x = v0 < V ? segment_sum<ROWS, VEC>(r, v0, V, lane) : Two{0.f, 0.f};
            if (lane == 0) seg[s] = x;
        }
        __syncthreads();
        if (warp == 0) {                            // lane l adds segments l, l + 32, ..
            Two x{0.f, 0.f};
            for (int s = lane; s < a.segs; s += 32) x = x + seg[s];
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) x = x + shuffle_xor(x, off);
            x = shuffle(x, 0);
            if (C == 1) {
                if (lane == 0) totals[turn][0] = x;
            } else if (lane < C) {
                put_remote(&totals[turn][rank], lane, x);
            }
        }
        if (C == 1) __syncthreads();
        else cluster_sync();
        Two all{0.f, 0.f};
        before = Two{0.f, 0.f};
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (i == rank) before = all;
            all = all + totals[turn][i];
        }
        turn ^= 1;                                  // (the other words were read before the last barrier)
        return all;
    };
    auto rest_of = [&](int cur, Two c, int lost) {
        const size_t row = row0 + cur;
        return Rest{a.probs + row * a.p_stride, a.draft && c.h > 0.f ? a.draft + row * a.q_stride : nullptr, c, gone, a.draft ? 0 : lost};
    };
    int cur = 0, count = 1, lost = 0;               // lost: rejected children of the current token
    Two c{0.f, 0.f}, mass{1.f, 0.f}, before;
    bool known = true;                              // whether mass is that of the present r
    if (tid == 0) taken[0] = 0;
    const unsigned long long okays = static_cast<unsigned long long>(okay[1]) << 32 | okay[0];
    const int par0 = par[lane], par1 = par[lane + 32];
    auto children = [&](int node) {
        return static_cast<unsigned long long>(__ballot_sync(0xffffffffu, par1 == node)) << 32 | __ballot_sync(0xffffffffu, par0 == node);
    };
    for (unsigned long long left = children(0); left;) {
        const int t = __ffsll(left) - 1;
        left &= left - 1;
        bool accept;
        Two r{sp[t], 0.f};
        if (c.h == 0.f && lost == 0) {
            accept = (okays >> t) & 1;
        } else {
            if (!known) {                           // a second child (trees): the first one's rejection is carried out
                mass = pass(rest_of(cur, c, lost), before);
                known = true;
                __syncthreads();                    // seg has been read
            }
            if (!(mass.h > 0.f)) continue;
            if (a.draft) rest(sp[t], sq[t], c, r.h, r.l);
            else
                for (int i = 0; i < lost; ++i)
                    if (gone[i] == tok[t]) r.h = 0.f;
            // u q mass < r; u q in two words is exact
            const float y = su[t] * sq[t];
            accept = mass * y + mass * fmaf(su[t], sq[t], -y) < r;
        }
        if (accept) {
            cur = t;
            if (tid == 0) taken[count] = t;
            ++count;
            lost = 0;
            c = Two{0.f, 0.f};
            mass = Two{1.f, 0.f};
            known = true;
            left = children(t);
        } else if (a.draft) {
            c = c + mass;
            known = false;
        } else {
            mass = mass - r;
            __syncthreads();                        // gone has been read
            if (tid == 0) gone[lost] = tok[t];
            ++lost;
            __syncthreads();
        }
    }
    __syncthreads();
    // ---- the next token
    Rest r = rest_of(cur, c, lost);
    Two all = pass(r, before);
    if (!(all.h > 0.f)) {                           // the same in the whole cluster
        __syncthreads();
        r = rest_of(cur, Two{0.f, 0.f}, 0);
        all = pass(r, before);
    }
    const bool sound = all.h > 0.f && all.h < INFINITY;
    const Two target = all * su[0];
    // The owner: the first CTA whose stretch takes the sum past the target; the last one with mass
    // where rounding (or a u of 1 or more) leaves none.
    int owner = -1;
    if (sound) {
        Two x{0.f, 0.f};
#pragma unroll
        for (int i = C - 1; i >= 0; --i)
            if (owner < 0 && totals[turn ^ 1][i].h > 0.f) owner = i;
        bool found = false;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const Two y = totals[turn ^ 1][i];
            x = x + y;
            if (!found && y.h > 0.f && target < x) {
                owner = i;
                found = true;
            }
        }
    }
    if (warp == 0 && (sound ? rank == owner : rank == 0)) {
        int v = -1;
        if (sound) {
            // the segment: a warp's scan of 32 at a time
            Two x = before;
            int s_hit = -1, s_last = -1;
            for (int s0 = 0; s0 < a.segs && s_hit < 0; s0 += 32) {
                const int s = s0 + lane;
                const Two y = s < a.segs ? seg[s] : Two{0.f, 0.f}, incl = scan(y, lane);
                const unsigned m = __ballot_sync(0xffffffffu, y.h > 0.f && target < x + incl);
                const unsigned some = __ballot_sync(0xffffffffu, y.h > 0.f);
                if (m) {
                    const int l = __ffs(m) - 1;
                    s_hit = s0 + l;
                    x = x + shuffle(incl - y, l);
                } else {
                    if (some) s_last = s0 + 31 - __clz(some);
                    x = x + shuffle(incl, 31);
                }
            }
            v = segment_find<ROWS, VEC>(r, (first + (s_hit >= 0 ? s_hit : s_last)) * SEG, V, lane, target - x, s_hit < 0);
        }
        if (lane == 0) {
            a.next[b] = v;
            if (v < 0) atomicOr(a.status, GDN_STATUS_BAD_PROB);
        }
    }
    if (rank == 0) {
        if (a.path)
            for (int t = tid; t < T; t += kThreads) a.path[static_cast<size_t>(b) * T + t] = t < count ? taken[t] : -1;
        if (tid == 0) a.accepted[b] = count;
    }
}

template <int ROWS, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) __cluster_dims__(kCluster, 1, 1) draft_accept_kernel(const DraftArgs a)
{
    accept_body<kCluster, ROWS, VEC>(a);
}
template <bool VEC>
__global__ void __launch_bounds__(kThreads, 2) draft_accept_small_kernel(const DraftArgs a)
{
    accept_body<1, 2, VEC>(a);
}

template <int ROWS>
cudaError_t launch(const DraftArgs &a, bool vec, cudaStream_t s) {
    const dim3 grid(kCluster, a.B);
    const size_t smem = static_cast<size_t>(a.segs) * sizeof(Two);
    return vec ? launch_pdl(draft_accept_kernel<ROWS, true>, grid, dim3(kThreads), smem, s, a)
               : launch_pdl(draft_accept_kernel<ROWS, false>, grid, dim3(kThreads), smem, s, a);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" int gdn_draft_accept(const gdn_draft_dims *d, const int32_t *tokens, const int32_t *parent, const float *probs,
                                const float *draft, const float *u, const int32_t *draft_len, int32_t *accepted,
                                int32_t *next, int32_t *path, int32_t *status, cudaStream_t stream)
{
    if (!d) return GDN_ERR_NULL;
    if (d->B < 0 || d->B > 65535 || d->T < 1 || d->T > kMaxT || d->V < 1 || d->V > 1 << 24 || d->flags) return GDN_ERR_DIMS;
    if (d->p_stride < d->V || (draft && d->q_stride < d->V)) return GDN_ERR_DIMS;
    if (d->B == 0) return GDN_OK;
    if (!tokens || !probs || !u || !accepted || !next || !status || (parent && !path)) return GDN_ERR_NULL;
    // Terms of a segment: a CTA's 16 warps each get one as far as the vocabulary goes, 1024 at most (more in flight).
    const bool small = d->V <= kSmallV;
    const int share = small ? d->V : (d->V + kCluster - 1) / kCluster;
    const int rows = small || share <= 256 * kWarps ? 2 : share <= 512 * kWarps ? 4 : 8;
    DraftArgs a{tokens, parent, probs, draft, u, draft_len, accepted, next, path, status, d->p_stride, d->q_stride,
                d->B, d->T, d->V, (share + rows * 128 - 1) / (rows * 128)};
    // 16-byte loads where every row begins on such a boundary
    const bool vec = reinterpret_cast<uintptr_t>(probs) % 16 == 0 && d->p_stride % 4 == 0 &&
                     (!draft || (reinterpret_cast<uintptr_t>(draft) % 16 == 0 && d->q_stride % 4 == 0));
    cudaError_t e;
    if (small) {
        const size_t smem = static_cast<size_t>(a.segs) * sizeof(Two);
        e = vec ? launch_pdl(draft_accept_small_kernel<true>, dim3(1, d->B), dim3(kThreads), smem, stream, a)
                : launch_pdl(draft_accept_small_kernel<false>, dim3(1, d->B), dim3(kThreads), smem, stream, a);
    } else {
        e = rows == 2 ? launch<2>(a, vec, stream) : rows == 4 ? launch<4>(a, vec, stream) : launch<8>(a, vec, stream);
    }
    return e == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
