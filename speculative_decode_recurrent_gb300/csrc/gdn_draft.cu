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
// masses and thresholds are two words throughout (46 bits and more of p), so a token differs from the 64-bit one's
// only where the threshold lies within some 2^-44 of a border (where rejections leave little of p, as much more of that rest).  Two words, because fp64 is slow on this chip: with 64-bit
// sums above the lanes' the search alone took 12 us, a whole call over 32768 probabilities 23.
//
// What bounds it: a few rows of V numbers per sequence, and a chain of dependent steps (tokens, their probabilities,
// the walk, the pass, its sum across the cluster, the search).  A cluster of eight CTAs takes a sequence, each a
// stretch of the vocabulary, in segments of 1024 terms per warp (256 or 512 where those would leave warps without one); two
// CTAs share an SM.  On the device: a chain of 8 over 32768 probabilities 5.8 us, 32 chains of 16 over 131072 12.3 (half of the copy
// bandwidth for the rows that have to be read).
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdnattn.h"
#include "gdndraft.h"
#include "pair_math.cuh"
#include "replay_common.h"
#include "tc_common.cuh"

namespace gdn {
namespace {

using tc::sm_count;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kMaxT = 64;

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
__device__ __forceinline__ Two shuffle_xor(Two x, int off) {
    return Two{__shfl_xor_sync(0xffffffffu, x.h, off), __shfl_xor_sync(0xffffffffu, x.l, off)};
}
__device__ __forceinline__ Two shuffle(Two x, int lane) {
    return Two{__shfl_sync(0xffffffffu, x.h, lane), __shfl_sync(0xffffffffu, x.l, lane)};
}
// Sum over the lanes up to this one.
__device__ __forceinline__ Two scan(Two x, int lane) {
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
        const Two y{__shfl_up_sync(0xffffffffu, x.h, off), __shfl_up_sync(0xffffffffu, x.l, off)};
        if (lane >= off) x = x + y;
    }
    return x;
}

// max(p - c q, 0) in two words, for two tokens (two operations an instruction).  The sign is that of both words: where p and c q agree in
// 24 bits, h is 0 or a last place or two and l decides (so l may be as large as h, and h 0 with l above it).  A negative p or
// NaN gives 0, an infinity leaves NaN (the row has no sound sum).
__device__ __forceinline__ void rest(float2 p, float2 q, Two c, float2 &h, float2 &l) {
    const float2 minus = make_float2(-1.f, -1.f), t = mul2(make_float2(-c.h, -c.h), q);      // - c.h q
    p = make_float2(fmaxf(p.x, 0.f), fmaxf(p.y, 0.f));
    float2 e = fma2(make_float2(c.h, c.h), q, t);
    e = fma2(make_float2(c.l, c.l), q, e);
    const float2 d = add2(p, t), bp = fma2(p, minus, d);
    const float2 err = fma2(e, minus, add2(fma2(fma2(bp, minus, d), minus, p), fma2(bp, minus, t)));
    const float2 s = add2(d, err);                  // (NaN of an infinity passes)
    h = make_float2(s.x <= 0.f ? 0.f : d.x, s.y <= 0.f ? 0.f : d.y);
    l = make_float2(s.x <= 0.f ? 0.f : err.x, s.y <= 0.f ? 0.f : err.y);
}
// Two sums side by side, without bringing l back below h's last place.
struct Two2 {
    float2 h, l;
};
__device__ __forceinline__ void gather(Two2 &s, float2 h, float2 l) {
    const float2 minus = make_float2(-1.f, -1.f), t = add2(s.h, h), bp = fma2(s.h, minus, t);
    s.l = add2(s.l, add2(l, add2(fma2(fma2(bp, minus, t), minus, s.h), fma2(bp, minus, h))));
    s.h = t;
}

// What a row of r is made of.
struct Rest {
    const float *p, *q;                             // q NULL: r is p
    Two c;
    const int *gone;                                // tokens that r has lost (draft NULL)
    int n_gone;
    // tokens v and v + 1
    __device__ __forceinline__ void terms(int v, float2 pv, float2 qv, float2 &h, float2 &l) const {
        if (q) {
            rest(pv, qv, c, h, l);
        } else {
            h = make_float2(fmaxf(pv.x, 0.f), fmaxf(pv.y, 0.f));
            l = make_float2(0.f, 0.f);
            for (int i = 0; i < n_gone; ++i) {
                if (v == gone[i]) h.x = 0.f;
                if (v + 1 == gone[i]) h.y = 0.f;
            }
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
    Two2 s{make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
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
            for (int j = 0; j < 4; j += 2) {
                float2 h, l;
                r.terms(at + i * 128 + j, make_float2(p[i][j], p[i][j + 1]), make_float2(q[i][j], q[i][j + 1]), h, l);
                gather(s, h, l);
            }
    }
    Two x = Two{s.h.x, s.l.x} + Two{s.h.y, s.l.y};
#pragma unroll 1
    for (int off = 16; off > 0; off >>= 1) x = x + shuffle_xor(x, off);
    return shuffle(x, 0);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
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
    __shared__ __align__(8) Two rows[ROWS];         // sums of the chosen segment's rows
    __shared__ int bad;
    const int b = blockIdx.y, rank = C > 1 ? blockIdx.x : 0, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int T = a.T, V = a.V;
    if (C > 1) cluster_arrive();                    // waited for below: no CTA writes to one that has not begun
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
    if (C > 1) cluster_wait();
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
#pragma unroll 1
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
#pragma unroll 1
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
    unsigned long long left = 0ull;
    if (a.parent) {
        left = children(0);
    } else {                                        // a chain: its accepted tokens lie in a row, one rejection ends them
        cur = min(__ffsll(~(okays >> 1)) - 1, n - 1);
        count = cur + 1;
        if (tid < count) taken[tid] = tid;
        if (count < n && a.draft) {
            c = mass;
            known = false;
        } else if (count < n) {
            if (tid == 0) gone[0] = tok[count];
            lost = 1;
        }
    }
    while (left) {
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
            if (a.draft) {
                float2 h, l;
                rest(make_float2(sp[t], 0.f), make_float2(sq[t], 0.f), c, h, l);
                r = Two{h.x, l.x};
            } else
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
    int owner = sound ? -1 : 0;
    bool found = false;
    if (sound) {
        Two x{0.f, 0.f};
#pragma unroll 1
        for (int i = 0; i < C && !found; ++i) {
            const Two y = totals[turn ^ 1][i];
            x = x + y;
            if (y.h > 0.f) owner = i;
            found = y.h > 0.f && target < x;
        }
    }
    if (rank == owner) {                            // (the same in a CTA)
        if (!sound) {
            if (tid == 0) {
                a.next[b] = -1;
                atomicOr(a.status, GDN_STATUS_BAD_PROB);
            }
        } else {
            // The segment, by a scan of 32 at a time (every warp for itself); then a warp per row of it, whose scan gives the
            // row's sum and, in the row of the target, the place.  (One warp for all rows took four times as
            // long: straight code that runs once waits for its instructions.)
            Two x = before;
            int s_hit = -1, s_last = 0;
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
            const Two goal = target - x;
            const int v = (first + (s_hit >= 0 ? s_hit : s_last)) * SEG + warp * 128 + lane * 4;
            Two2 h4[2];                             // this lane's four terms
            Two mine{0.f, 0.f}, incl{0.f, 0.f};
            if (warp < ROWS) {
                float p[4], q[4] = {0.f, 0.f, 0.f, 0.f};
                load4<VEC>(r.p, v, V, p);
                if (r.q) load4<VEC>(r.q, v, V, q);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    r.terms(v + 2 * j, make_float2(p[2 * j], p[2 * j + 1]), make_float2(q[2 * j], q[2 * j + 1]), h4[j].h, h4[j].l);
                mine = (Two{h4[0].h.x, h4[0].l.x} + Two{h4[0].h.y, h4[0].l.y}) + (Two{h4[1].h.x, h4[1].l.x} + Two{h4[1].h.y, h4[1].l.y});
                incl = scan(mine, lane);
                if (lane == 31) rows[warp] = incl;
            }
            __syncthreads();
            if (warp < ROWS) {
                Two sum{0.f, 0.f}, ahead{0.f, 0.f};
                int row = -1, last = 0;
#pragma unroll 1
                for (int i = 0; i < ROWS; ++i) {
                    const Two y = rows[i], next = sum + y;
                    if (y.h > 0.f) last = i;
                    if (row < 0 && s_hit >= 0 && y.h > 0.f && goal < next) {
                        row = i;
                        ahead = sum;
                    }
                    sum = next;
                }
                if (warp == (row >= 0 ? row : last)) {                // none past the goal: the last term with mass
                    const Two excl = ahead + (incl - mine);
                    const float h[4] = {h4[0].h.x, h4[0].h.y, h4[1].h.x, h4[1].h.y}, l[4] = {h4[0].l.x, h4[0].l.y, h4[1].l.x, h4[1].l.y};
                    int hit = -1, end = -1;
                    Two x4 = excl;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x4 = x4 + Two{h[j], l[j]};
                        if (h[j] + l[j] > 0.f) end = v + j;
                        if (hit < 0 && row >= 0 && h[j] + l[j] > 0.f && goal < x4) hit = v + j;
                    }
                    const unsigned m = __ballot_sync(0xffffffffu, hit >= 0), e = __ballot_sync(0xffffffffu, end >= 0);
                    const int at = m ? __shfl_sync(0xffffffffu, hit, __ffs(m) - 1) : __shfl_sync(0xffffffffu, end, e ? 31 - __clz(e) : 0);
                    if (lane == 0) a.next[b] = at;
                }
            }
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
template <int ROWS, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) draft_accept_one_kernel(const DraftArgs a)
{
    accept_body<1, ROWS, VEC>(a);
}

template <int ROWS>
cudaError_t launch(const DraftArgs &a, bool one, bool vec, cudaStream_t s) {
    const size_t smem = static_cast<size_t>(a.segs) * sizeof(Two);
    if (one)
        return vec ? launch_pdl(draft_accept_one_kernel<ROWS, true>, dim3(1, a.B), dim3(kThreads), smem, s, a)
                   : launch_pdl(draft_accept_one_kernel<ROWS, false>, dim3(1, a.B), dim3(kThreads), smem, s, a);
    const dim3 grid(kCluster, a.B);
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
    // One CTA for a sequence where the vocabulary is small (chains of 3, device time: 4096 probabilities 5.0 us, by clusters 5.3; 16384
    // 8.3 and 5.2), or where the clusters of so many sequences would come in several waves (two CTAs share an SM): 64 sequences of
    // 32768 10.1 us and 13.6, of 65536 15.3 and 15.5; 256 of 131072 46 and 72.
    const long long slots = 2ll * sm_count();
    const bool one = d->V <= 4096 || (kCluster * static_cast<long long>(d->B) > slots && d->V <= 131072 && d->V <= 512ll * d->B);
    // Terms of a segment: a CTA's 16 warps each get one as far as the vocabulary goes, 1024 at most (more in flight: 64 chains over
    // 262144 take 32.6 us, in segments of 256 terms 38.5; one over 32768 5.6, in segments of 512 6.0).
    const int share = one ? d->V : (d->V + kCluster - 1) / kCluster;
    const int rows = share <= 256 * kWarps ? 2 : share <= 512 * kWarps ? 4 : 8;
    DraftArgs a{tokens, parent, probs, draft, u, draft_len, accepted, next, path, status, d->p_stride, d->q_stride,
                d->B, d->T, d->V, (share + rows * 128 - 1) / (rows * 128)};
    // 16-byte loads where every row begins on such a boundary
    const bool vec = reinterpret_cast<uintptr_t>(probs) % 16 == 0 && d->p_stride % 4 == 0 &&
                     (!draft || (reinterpret_cast<uintptr_t>(draft) % 16 == 0 && d->q_stride % 4 == 0));
    const cudaError_t e = rows == 2 ? launch<2>(a, one, vec, stream) : rows == 4 ? launch<4>(a, one, vec, stream) : launch<8>(a, one, vec, stream);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
