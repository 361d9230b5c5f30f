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
// sums of 10^5 terms are off by more than many a term.  A term is p - c q in two fp32 words (exact for c = 1), sums
// are kept in two words (48 bits) by lanes and in 64 bits above, so a token differs from the 64-bit one's only where the
// threshold lies within some 2^-44 of a border.  Two fp32 words, because fp64 runs at 2 results a clock
// and SM here.
//
// What bounds it: a few rows of V numbers per sequence, and a chain of dependent steps (tokens, their probabilities,
// the walk, the pass, its sum across the cluster, the search).  A cluster of eight CTAs takes a sequence, each a
// stretch of the vocabulary, in segments of 1024 terms per warp (four 16-byte loads of each row in flight per lane, two CTAs on an SM).
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdnattn.h"
#include "gdndraft.h"
#include "replay_common.h"

namespace gdn {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kSeg = 1024;                          // terms of a segment: a warp's unit
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

// A sum in two fp32 words.
struct Sum2 {
    float hi, lo;
    __device__ void add(float h, float l) {
        const float s = hi + h, bp = s - hi;
        lo += ((hi - (s - bp)) + (h - bp)) + l;
        hi = s;
    }
    __device__ double value() const { return static_cast<double>(hi) + static_cast<double>(lo); }
};

// max(p - c q, 0) in two words, c in two.
__device__ __forceinline__ void rest(float p, float q, float ch, float cl, float &h, float &l) {
    p = fmaxf(p, 0.f);                              // (NaN: 0)
    const float t = ch * q, e = fmaf(cl, q, fmaf(ch, q, -t));
    const float d = p - t, bb = d - p;
    const float err = (p - (d - bb)) - (t + bb) - e;
    const bool some = !(d + err <= 0.f);            // (an infinity leaves NaN: the row has no sound sum)
    h = some ? d : 0.f;
    l = some ? err : 0.f;
}

// What a row of r is made of.
struct Rest {
    const float *p, *q;                             // q NULL: r is p
    float ch, cl;
    const int *gone;                                // tokens that r has lost (draft NULL)
    int n_gone;
    __device__ void term(int v, float pv, float qv, float &h, float &l) const {
        if (q) {
            rest(pv, qv, ch, cl, h, l);
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

// The sum of the segment at v0, in every lane.  Half of it at a time: with 64 registers two CTAs share an SM.
template <bool VEC>
__device__ __forceinline__ double segment_sum(const Rest &r, int v0, int V, int lane) {
    constexpr int ROWS = kSeg / 256;                // rows of 128 terms in half a segment
    Sum2 s{0.f, 0.f};
#pragma unroll 1
    for (int at = v0; at < v0 + kSeg; at += kSeg / 2) {
        float p[ROWS][4], q[ROWS][4];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) load4<VEC>(r.p, at + i * 128 + lane * 4, V, p[i]);
        if (r.q)
#pragma unroll
            for (int i = 0; i < ROWS; ++i) load4<VEC>(r.q, at + i * 128 + lane * 4, V, q[i]);
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float h, l;
                r.term(at + i * 128 + lane * 4 + j, p[i][j], r.q ? q[i][j] : 0.f, h, l);
                s.add(h, l);
            }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float h = __shfl_xor_sync(0xffffffffu, s.hi, off), l = __shfl_xor_sync(0xffffffffu, s.lo, off);
        s.add(h, l);
    }
    return __shfl_sync(0xffffffffu, s.value(), 0);
}

// The first term of the segment at v0 at which the running sum passes `target`; the last term above 0 where none does (the
// segment's sum was taken in another order), -1 where there is none.  The sums of the segment's eight rows of 128 terms
// in two words first, so that the chain of 64-bit additions is one row's: 8 for the rows, 5 across the lanes, 4 in a lane.
template <bool VEC>
__device__ __forceinline__ int segment_find(const Rest &r, int v0, int V, int lane, double target) {
    constexpr int ROWS = kSeg / 128;
    float hi[ROWS], lo[ROWS];                       // of this lane's four terms in each row, then of whole rows
    unsigned some = 0u;                             // rows with a term above 0 (this lane's, then all)
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int v = v0 + i * 128 + lane * 4;
        float p[4], q[4] = {0.f, 0.f, 0.f, 0.f};
        load4<VEC>(r.p, v, V, p);
        if (r.q) load4<VEC>(r.q, v, V, q);
        Sum2 s{0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float h, l;
            r.term(v + j, p[j], q[j], h, l);
            s.add(h, l);
            if (h > 0.f) some |= 1u << i;
        }
        hi[i] = s.hi;
        lo[i] = s.lo;
    }
    some = __reduce_or_sync(0xffffffffu, some);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            Sum2 s{hi[i], lo[i]};
            const float h = __shfl_xor_sync(0xffffffffu, s.hi, off), l = __shfl_xor_sync(0xffffffffu, s.lo, off);
            s.add(h, l);
            hi[i] = s.hi;
            lo[i] = s.lo;
        }
    if (!some) return -1;
    // the row: every lane takes the same steps
    double before = 0.0, sum = 0.0;
    int row = -1;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const double next = sum + Sum2{hi[i], lo[i]}.value();
        if (row < 0 && ((some >> i) & 1) && next > target) {
            row = i;
            before = sum;
        }
        sum = next;
    }
    const bool past = row < 0;                      // none: the last term of the last row with one
    if (past) row = 31 - __clz(some);
    const int v = v0 + row * 128 + lane * 4;
    float p[4], q[4] = {0.f, 0.f, 0.f, 0.f};
    load4<VEC>(r.p, v, V, p);
    if (r.q) load4<VEC>(r.q, v, V, q);
    double x[4], mine = 0.0;
    int last = -1;
    bool over0[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float h, l;
        r.term(v + j, p[j], q[j], h, l);
        mine += static_cast<double>(h) + static_cast<double>(l);
        x[j] = mine;
        over0[j] = h > 0.f;
        if (over0[j]) last = v + j;
    }
    double incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    const double excl = before + (incl - mine);
    int hit = -1;
#pragma unroll
    for (int j = 3; j >= 0; --j)
        if (!past && over0[j] && excl + x[j] > target) hit = v + j;
    const unsigned m = __ballot_sync(0xffffffffu, hit >= 0);
    if (m) return __shfl_sync(0xffffffffu, hit, __ffs(m) - 1);
    return __shfl_sync(0xffffffffu, last, 31 - __clz(__ballot_sync(0xffffffffu, last >= 0)));
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// `x` to word `slot` of the same array in the CTA of rank `to`.
__device__ __forceinline__ void put_remote(double *word, int to, double x) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(word)), r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(to));
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(r), "d"(x) : "memory");
}

template <int C, bool VEC>
__device__ __forceinline__ void accept_body(const DraftArgs &a)
{
    extern __shared__ double seg[];                 // [segs] sums of this CTA's segments
    __shared__ double totals[2][kCluster];          // of the cluster's CTAs; by turns
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
                first = static_cast<double>(u) * q < p;               // (both sides exact)
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
    auto pass = [&](const Rest &r, double &before, double &own) -> double {
        for (int s = warp; s < a.segs; s += kWarps) {
            const int v0 = (first + s) * kSeg;      // (below 2^24 + 2^13 kSeg)
            const double x = v0 < V ? segment_sum<VEC>(r, v0, V, lane) : 0.0;
            if (lane == 0) seg[s] = x;
        }
        __syncthreads();
        if (warp == 0) {                            // lane l adds segments l, l + 32, ..
            double x = 0.0;
            for (int s = lane; s < a.segs; s += 32) x += seg[s];
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
            if (C == 1) {
                if (lane == 0) totals[turn][0] = x;
            } else if (lane < C) {
                put_remote(&totals[turn][rank], lane, x);
            }
        }
        if (C == 1) __syncthreads();
        else cluster_sync();
        double all = 0.0;
        before = 0.0;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (i == rank) before = all;
            all += totals[turn][i];
        }
        own = totals[turn][rank];
        turn ^= 1;                                  // (the other words were read before the last barrier)
        return all;
    };
    auto rest_of = [&](int cur, double c, int lost) {
        const size_t row = row0 + cur;
        const float ch = static_cast<float>(c);
        return Rest{a.probs + row * a.p_stride, a.draft && c > 0.0 ? a.draft + row * a.q_stride : nullptr, ch,
                    static_cast<float>(c - static_cast<double>(ch)), gone, a.draft ? 0 : lost};
    };
    int cur = 0, count = 1, lost = 0;               // lost: rejected children of the current token
    double c = 0.0, mass = 1.0;
    bool known = true;                              // whether mass is that of the present r
    double before, own;
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
        double r = 0.0;
        if (c == 0.0 && lost == 0) {
            accept = (okays >> t) & 1;
            r = sp[t];
        } else {
            if (!known) {                           // a second child (trees): the first one's rejection is carried out
                mass = pass(rest_of(cur, c, lost), before, own);
                known = true;
                __syncthreads();                    // seg has been read
            }
            if (!(mass > 0.0)) continue;
            const double p = sp[t], q = sq[t];
            r = a.draft ? fmax(p - c * q, 0.0) : p;
            if (!a.draft)
                for (int i = 0; i < lost; ++i)
                    if (gone[i] == tok[t]) r = 0.0;
            accept = static_cast<double>(su[t]) * q * mass < r;
        }
        if (accept) {
            cur = t;
            if (tid == 0) taken[count] = t;
            ++count;
            lost = 0;
            c = 0.0;
            mass = 1.0;
            known = true;
            left = children(t);
        } else if (a.draft) {
            c += mass;
            known = false;
        } else {
            mass -= r;
            __syncthreads();                        // gone has been read
            if (tid == 0) gone[lost] = tok[t];
            ++lost;
            __syncthreads();
        }
    }
    __syncthreads();
    // ---- the next token
    Rest r = rest_of(cur, c, lost);
    double all = pass(r, before, own);
    if (!(all > 0.0)) {                             // the same in the whole cluster
        __syncthreads();
        r = rest_of(cur, 0.0, 0);
        all = pass(r, before, own);
    }
    const bool sound = all > 0.0 && all < INFINITY;
    const double target = static_cast<double>(su[0]) * all;
    // The owner: the first CTA whose stretch takes the sum past the target; the last one with mass
    // where rounding (or a u of 1 or more) leaves none.
    int owner = -1;
    if (sound) {
        double x = 0.0;
        for (int i = 0; i < C; ++i) {
            const double y = totals[turn ^ 1][i];
            x += y;
            if (x > target && y > 0.0) {
                owner = i;
                break;
            }
        }
        if (owner < 0)
            for (int i = 0; i < C; ++i)
                if (totals[turn ^ 1][i] > 0.0) owner = i;
    }
    if (warp == 0 && (sound ? rank == owner : rank == 0)) {
        int v = -1;
        if (sound) {
            // the segment: a warp's scan of 32 at a time
            double x = before;
            int s_hit = -1, s_last = -1;
            for (int s0 = 0; s0 < a.segs && s_hit < 0; s0 += 32) {
                const int s = s0 + lane;
                const double y = s < a.segs ? seg[s] : 0.0;
                double incl = y;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const double z = __shfl_up_sync(0xffffffffu, incl, off);
                    if (lane >= off) incl += z;
                }
                const unsigned m = __ballot_sync(0xffffffffu, y > 0.0 && x + incl > target);
                const unsigned some = __ballot_sync(0xffffffffu, y > 0.0);
                if (m) {
                    const int l = __ffs(m) - 1;
                    s_hit = s0 + l;
                    x += __shfl_sync(0xffffffffu, incl, l) - __shfl_sync(0xffffffffu, y, l);
                } else {
                    if (some) s_last = s0 + 31 - __clz(some);
                    x += __shfl_sync(0xffffffffu, incl, 31);
                }
            }
            v = s_hit >= 0 ? segment_find<VEC>(r, (first + s_hit) * kSeg, V, lane, target - x)
                           : segment_find<VEC>(r, (first + s_last) * kSeg, V, lane, INFINITY);
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

template <bool VEC>
__global__ void __launch_bounds__(kThreads, 2) __cluster_dims__(kCluster, 1, 1) draft_accept_kernel(const DraftArgs a)
{
    accept_body<kCluster, VEC>(a);
}
template <bool VEC>
__global__ void __launch_bounds__(kThreads, 2) draft_accept_small_kernel(const DraftArgs a)
{
    accept_body<1, VEC>(a);
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
    const bool small = d->V <= kSmallV;
    const int all = (d->V + kSeg - 1) / kSeg, segs = small ? all : (all + kCluster - 1) / kCluster;
    const DraftArgs a{tokens, parent, probs, draft, u, draft_len, accepted, next, path, status, d->p_stride, d->q_stride,
                      d->B, d->T, d->V, segs};
    // 16-byte loads where every row begins on such a boundary
    const bool vec = reinterpret_cast<uintptr_t>(probs) % 16 == 0 && d->p_stride % 4 == 0 &&
                     (!draft || (reinterpret_cast<uintptr_t>(draft) % 16 == 0 && d->q_stride % 4 == 0));
    const size_t smem = static_cast<size_t>(segs) * sizeof(double);
    const dim3 grid(small ? 1 : kCluster, d->B), block(kThreads);
    const cudaError_t e = small ? (vec ? launch_pdl(draft_accept_small_kernel<true>, grid, block, smem, stream, a)
                                       : launch_pdl(draft_accept_small_kernel<false>, grid, block, smem, stream, a))
                                : (vec ? launch_pdl(draft_accept_kernel<true>, grid, block, smem, stream, a)
                                       : launch_pdl(draft_accept_kernel<false>, grid, block, smem, stream, a));
    return e == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
