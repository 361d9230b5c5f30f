// gdn_advance_tc.cu -- gdn_replay_advance on the tensor cores (tcgen05), for sm_103a: the gated delta rule over
// long bf16 chunks, 64 tokens at a time.  C ABI and layouts: include/gdnreplay.h.
//
// Mathematics.  For 64 tokens of one head, with G_t the running sum of the log-decays, gamma_t = e^{G_t}, and
// A[t][s] = beta_t e^{G_t - G_s} (k_t.k_s) (s < t), the recurrence unrolls into the chunkwise form of "Parallelizing
// Linear Transformers with the Delta Rule over Sequence Length" (NeurIPS 2024): with P = (I + A)^-1 diag(beta) and
//     x_t = v_t - gamma_t S k_t                  (rows of x; S the state before the chunk)
// the updates are u = P x, and so, with M[t][s] = scale e^{G_t - G_s} (q_t.k_s) (s <= t) and
// D = diag(e^{G_63 - G_t}),
//     o = scale gamma S q + (M P) x,    S' = gamma_63 S + E x,  E = K^T D P.
// E (dk x 64) and M P (64 x 64) do not involve the state: the first kernel makes them for many chunks at once.  The
// second walks the chunks of a head with the state at hand, two dependent products a chunk: [K;Q] S^T, then
// E x (and (M P) x beside what follows).  Value columns need nothing of one another: few heads are cut into
// slices of 32 columns, many are walked whole.
//
// Precision.  Keys and queries are exact in bf16; S, x, E, M P and what these are made of enter as three bf16 terms each (all 24 bits),
// products of a pair of them as the six of terms whose orders add up to two at most, the smallest first: additions in the tensor
// cores do not round to nearest, and few of them act on a full-size sum so (largest first, heads were off by two to three times as
// much).  Against 64 bits (root mean squares): outputs 3 to 4e-7 and states 1 to 2.5e-7, where a token at a time in fp32 gives 1.1e-7 and
// 0.6e-7; of decays of 0.999 a token, whose errors add up, 6 to 8e-7 and 4 to 8e-7 against 2 to 3e-6.  (Two terms and three products
// were 5e-6 off for some 30 % less time.)  The state itself stays in fp32 registers through the walk, the inverse is formed in fp32 by
// blocks.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "advance_common.h"
#include "advance_plan.h"
#include "pair_math.cuh"
#include "tc_async.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kC = kChunkTokens;
constexpr float kLog2e = 1.4426950408889634f;

// What the first kernel leaves of a chunk of a head, as the second one's operands lie in shared memory:
// E as [dk][64 tokens] bf16 rows of 128 bytes (swizzled), its three terms; M P as [64][64] likewise; gamma.
template <int DK> struct Unit {
    static constexpr int E_BYTES = DK * 128, MP_BYTES = kC * 128;      // of a term
    static constexpr int OFF_MP = 3 * E_BYTES, OFF_GAMMA = OFF_MP + 3 * MP_BYTES;
    static constexpr int BYTES = OFF_GAMMA + 512;   // gamma [64] fp32
};

struct TcAdvance {
    AdvanceArgs a;
    int b0;                                         // first sequence of the launch
    int c0, chunks;                                 // first chunk, chunks of the launch
    int dv;
    int behind;                                     // the first kernel runs beside the walk over the chunks before (see launch)
};

// Tokens of the launch's chunks that are in use.
__device__ __forceinline__ int tokens_here(const TcAdvance &ta, int n) { return max(0, min(n - ta.c0 * kC, ta.chunks * kC)); }

// Two numbers as three packed bf16 terms each, 8 bits of the mantissa after the other (so their sum is the number; NaN stays).
__device__ __forceinline__ void split_pair(float2 x, uint32_t (&t)[3]) {
    const float2 minus = make_float2(-1.f, -1.f);
    auto high = [](float2 y) {
        return make_float2(__uint_as_float(__float_as_uint(y.x) & 0xffff0000u), __uint_as_float(__float_as_uint(y.y) & 0xffff0000u));
    };
    const float2 m = fma2(high(x), minus, x);
    t[0] = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
    t[1] = __byte_perm(__float_as_uint(m.x), __float_as_uint(m.y), 0x7632);
    const float2 r = fma2(high(m), minus, m);
    const __nv_bfloat162 l = __floats2bfloat162_rn(r.x, r.y);
    t[2] = *reinterpret_cast<const uint32_t *>(&l);
}
// Bit 15 or 31 where a half of x is an infinite or NaN bf16 number.
__device__ __forceinline__ uint32_t odd_bits(uint32_t x) { return (x & 0x7f807f80u) + 0x00800080u; }
// Eight of them as one 16-byte chunk of each term.
__device__ __forceinline__ void split8(const float *y, uint4 (&t)[3]) {
    uint32_t p[4][3];
#pragma unroll
    for (int i = 0; i < 4; ++i) split_pair(make_float2(y[2 * i], y[2 * i + 1]), p[i]);
#pragma unroll
    for (int k = 0; k < 3; ++k) t[k] = make_uint4(p[0][k], p[1][k], p[2][k], p[3][k]);
}
// The products of two numbers of three terms: (term of A, term of B), the smallest first: an addition to a sum does not round to
// nearest, so the fewer come once it is large, the better.
__device__ constexpr int kTermA[6] = {2, 1, 0, 1, 0, 0}, kTermB[6] = {0, 1, 2, 0, 1, 0};
constexpr int kNever = 0x7fffffff;

// ------------------------------------------------------------- E and M P of every chunk
constexpr int kPrepThreads = 256;

// What bounds it: shared memory's bandwidth (six thousand cycles of loads and stores a chunk, two thousand of operands, of some
// ten thousand that an SM takes; 98 us for the 2800 chunks of 8 prompts of 16 heads, 200 MB of operators).
// Its size here, 50 KB, lets four CTAs share an SM: [K;Q] as
// atoms of 64 columns, 128 rows of 128 bytes each; A in fp32, T over it.  What is no longer needed makes room: the first two terms of M
// lie over the queries, the third (in registers until then) over the second half of the keys once E is there; F's terms over T (the third
// after the others' product), P's after them, its third over the first half of the keys; at the end E's and M P's over all of it.
template <int DK> struct PrepPlan {
    static constexpr int LD = 68;                   // floats of a row of A and T: 16-byte rows, 4 banks apart
    static constexpr int ATOM = 16384, TERM = kC * 128, OFF_M0 = 8192, OFF_M1 = 24576, OFF_M2 = 16384, OFF_P2 = 0;
    static constexpr int OFF_T = 32768, OFF_G = OFF_T + kC * LD * 4;   // then G (two words), gamma, beta, decay to the end
    static constexpr int OFF_BAR = OFF_G + 5 * kC * 4;
    static constexpr int BYTES = OFF_BAR + 64;
    static_assert(OFF_T % 1024 == 0 && 2 * TERM <= kC * LD * 4 && 3 * Unit<DK>::E_BYTES <= OFF_G, "room");
};

// One level of the inverse, in A's place: with the diagonal blocks of N rows of T = (I + A)^-1 there, those of 2 N:
// T21 = -T22 A21 T11.  X = A21 T11 lies in the block (1, 2) for the moment, so the loops stay clear of what
// is above the diagonal blocks of 8.  A thread has N / 8 neighbouring elements of a row, or of two.
template <int N, int LD>
__device__ __forceinline__ void inverse_level(float *sT, int tid) {
    constexpr int W = N / 8, R = N == 32 ? 2 : 1;   // columns and rows of a thread (two of 32: fewer loads, which shared memory bounds)
    const int c = (tid & 7) * W, r = (tid >> 3) * R % N, lo = tid * R / (8 * N) * 2 * N, hi = lo + N;
    const bool on = tid < kPrepThreads / R;
    float x[R][W];
    auto product = [&](const float *row, const float *cols, int k0, int k1, float sign) {      // sums over [k0, k1), multiples of 4
#pragma unroll
        for (int e = 0; e < R; ++e)
#pragma unroll
            for (int i = 0; i < W; ++i) x[e][i] = 0.f;
#pragma unroll 2
        for (int k = k0; k < k1; k += 4) {
            float yy[R][4];
#pragma unroll
            for (int e = 0; e < R; ++e) {
                const float4 y = *reinterpret_cast<const float4 *>(row + e * LD + k);
                yy[e][0] = sign * y.x; yy[e][1] = sign * y.y; yy[e][2] = sign * y.z; yy[e][3] = sign * y.w;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float *z = cols + (k + q) * LD;
                float zz[W];
                if constexpr (W == 4) {
                    const float4 z4 = *reinterpret_cast<const float4 *>(z);
                    zz[0] = z4.x; zz[1] = z4.y; zz[2] = z4.z; zz[3] = z4.w;
                } else {
#pragma unroll
                    for (int i = 0; i < W; ++i) zz[i] = z[i];
                }
#pragma unroll
                for (int e = 0; e < R; ++e)
#pragma unroll
                    for (int i = 0; i < W; ++i) x[e][i] = fmaf(yy[e][q], zz[i], x[e][i]);
            }
        }
    };
    auto put = [&](float *at) {
#pragma unroll
        for (int e = 0; e < R; ++e)
#pragma unroll
            for (int i = 0; i < W; ++i) at[e * LD + i] = x[e][i];
    };
    if (on) {
        product(sT + (hi + r) * LD + lo, sT + lo * LD + lo + c, c & ~7, N, 1.f);
        put(sT + (lo + r) * LD + hi + c);
    }
    __syncthreads();
    if (on) {
        product(sT + (hi + r) * LD + hi, sT + lo * LD + hi + c, 0, (r | 7) + 1, -1.f);
        put(sT + (hi + r) * LD + lo + c);
    }
    __syncthreads();
}

// 32 columns of this thread's lane from tcol on as three terms each, in columns 32 half .. of row `row` of the tiles, `step` bytes apart.
__device__ __forceinline__ void stage_row(uint32_t tcol, uint8_t *tile, int step, int row, int half) {
    uint32_t r[32];
    tmem_ld32(tcol, r);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint4 t[3];
        split8(reinterpret_cast<const float *>(r) + 8 * c, t);
        const uint32_t at = sw128(row, 4 * half + c);
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4 *>(tile + k * step + at) = t[k];
    }
}

// One CTA per (head, chunk, sequence).  Warps w and w + 4 share TMEM lanes 32 (w % 4) .. and halve the columns.
template <int DK>
__global__ void __launch_bounds__(kPrepThreads, 4) advance_prep_kernel(const TcAdvance ta)
{
    using P = PrepPlan<DK>;
    const AdvanceArgs &a = ta.a;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int h = blockIdx.x, c = blockIdx.y, b = ta.b0 + blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // Beside a walk, CTA 0 waits for it at its end instead (it also takes part in the launch when its own chunk is empty).
    const bool waiter = ta.behind && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0;
    if (!ta.behind) pdl_wait();
    const AdvanceSeq sq = advance_seq(a, b);
    const int n = sq.bad ? 0 : tokens_here(ta, sq.n) - c * kC;          // tokens of this chunk in use
    const bool expire = (saddr(smem) & 1023u) || (a.flags & GDN_FLAG_TEST_EXPIRE);
    if (n <= 0 || expire) {
        if (n > 0 && tid == 0) atomicOr(a.status, kStatusTimeout);
        if (waiter) pdl_wait();
        return;
    }
    float *sT = reinterpret_cast<float *>(smem + P::OFF_T);
    float *sGh = reinterpret_cast<float *>(smem + P::OFF_G), *sGl = sGh + kC, *sGam = sGl + kC, *sBeta = sGam + kC, *sEnd = sBeta + kC;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + P::OFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + 4);
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(&bar[i], 1);
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, 128);
    // ---- keys and queries into the swizzled tile, zeros past the last token
    const size_t tok0 = static_cast<size_t>(b) * a.T + (ta.c0 + c) * kC;
    const int hk = h / (a.H / a.Hk);
    const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16 *>(a.k) + tok0 * a.k_stride + hk * DK;
    const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(a.q) + tok0 * a.q_stride + hk * DK;
    constexpr int VR = DK / 8, ROWS = kPrepThreads / VR, IT = kC / ROWS;      // 16-byte vectors of a row, rows at a time
    {
        const int vc = tid % VR, vr = tid / VR;
        uint4 kr[IT], qr[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int t = vr + i * ROWS;
            kr[i] = qr[i] = make_uint4(0u, 0u, 0u, 0u);
            if (t < n) {
                kr[i] = __ldg(reinterpret_cast<const uint4 *>(kp + t * a.k_stride) + vc);
                qr[i] = __ldg(reinterpret_cast<const uint4 *>(qp + t * a.q_stride) + vc);
            }
        }
        if (warp == 0) {                            // compensated running sums of g
            float hi[2], lo[2], be[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = lane + 32 * i;
                const size_t at = (tok0 + t) * a.H + h;
                const float g = t < n ? a.g[at] : 0.f;
                hi[i] = g < -1000.f ? -1000.f : g;  // (e^-1000 is 0 as well; of -infinity there is no difference. NaN stays)
                be[i] = t < n ? a.beta[at] : 0.f;
                lo[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const float h2 = __shfl_up_sync(0xffffffffu, hi[i], off), l2 = __shfl_up_sync(0xffffffffu, lo[i], off);
                    if (lane >= off) {
                        const float s1 = hi[i] + h2, bp = s1 - hi[i];
                        lo[i] += l2 + ((hi[i] - (s1 - bp)) + (h2 - bp));
                        hi[i] = s1;
                    }
                }
            {
                const float ch = __shfl_sync(0xffffffffu, hi[0], 31), cl = __shfl_sync(0xffffffffu, lo[0], 31);
                const float s1 = hi[1] + ch, bp = s1 - hi[1];
                lo[1] += cl + ((hi[1] - (s1 - bp)) + (ch - bp));
                hi[1] = s1;
            }
            const float eh = __shfl_sync(0xffffffffu, hi[1], 31), el = __shfl_sync(0xffffffffu, lo[1], 31);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = lane + 32 * i;
                sGh[t] = hi[i];
                sGl[t] = lo[i];
                sGam[t] = __expf(hi[i] + lo[i]);
                sEnd[t] = __expf((eh - hi[i]) + (el - lo[i]));
                sBeta[t] = be[i];
            }
        }
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int t = vr + i * ROWS;
            uint8_t *at = smem + (vc >> 3) * P::ATOM;
            *reinterpret_cast<uint4 *>(at + sw128(t, vc & 7)) = kr[i];
            *reinterpret_cast<uint4 *>(at + sw128(kC + t, vc & 7)) = qr[i];
        }
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int half = warp >> 2;
    // ---- [K;Q] K^T
    if (warp == 0) {
        const uint64_t d = desc_sw128(saddr(smem));
        if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks) {
                const uint32_t off = (ks >> 2) * P::ATOM + (ks & 3) * 32;
                mma_bf16(tmem, desc_add(d, off), desc_add(d, off), idesc_mn(1, 128, kC), ks > 0);
            }
            mma_commit(&bar[0]);
        }
        __syncwarp();
    }
    bool ok = mbar_wait(&bar[0], 0);
    tc_fence_after();
    ok = __all_sync(0xffffffffu, ok);
    int issued = 0;                                 // the last barrier that MMAs may have been committed to
    const int t = ((warp & 1) << 5) + lane;
    const bool keys = (warp & 3) < 2;
    uint4 m2[4];                                    // M's third terms
    const int row = tid & (kC - 1), s0 = (tid >> 6) * 16;
    float y[16];
    // From the first token on whose key, decay or beta is not finite, all outputs and the state are NaN: the walk learns of it by a gamma of
    // NaN.  The rows before it must not meet it (they have zeros for it, which make NaN of it).  Such a token shows in P; then A, M
    // and P are made again as if it and those behind it had keys and betas of 0.
    int sound = kC;                                 // tokens before it
    for (bool again = false;; again = true) {
        // ---- A in fp32 (rows of K), M's terms (rows of Q)
        if (ok) {
            const float gh = sGh[t], gl = sGl[t], f = keys ? sBeta[t] : a.scale;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int j0 = 32 * half + 16 * v;
                uint32_t r[16];
                tmem_load16(tmem + lanes + j0, r);
                tmem_wait_ld();
                float y[16];
                const int seen = t < sound ? t - j0 + (keys ? 0 : 1) : 0;               // columns j < seen count
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 h4 = *reinterpret_cast<const float4 *>(sGh + j0 + j), l4 = *reinterpret_cast<const float4 *>(sGl + j0 + j);
                    y[j] = ex2(((gh - h4.x) + (gl - l4.x)) * kLog2e);
                    y[j + 1] = ex2(((gh - h4.y) + (gl - l4.y)) * kLog2e);
                    y[j + 2] = ex2(((gh - h4.z) + (gl - l4.z)) * kLog2e);
                    y[j + 3] = ex2(((gh - h4.w) + (gl - l4.w)) * kLog2e);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j)                          // (as bits: a select here became 32 branches)
                    y[j] = __uint_as_float(__float_as_uint(__uint_as_float(r[j]) * y[j] * f) & (j < seen ? 0xffffffffu : 0u));
                if (keys) {
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4 *>(sT + t * P::LD + j0 + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
                } else {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint4 m[3];
                        split8(y + 8 * c, m);
                        const uint32_t at = sw128(t, 4 * half + 2 * v + c);
                        *reinterpret_cast<uint4 *>(smem + P::OFF_M0 + at) = m[0];
                        *reinterpret_cast<uint4 *>(smem + P::OFF_M1 + at) = m[1];
                        m2[2 * v + c] = m[2];
                    }
                }
            }
        }
        tc_fence_before();
        __syncthreads();
        // ---- T = (I + A)^-1: diagonal blocks of 8 by substitution, a thread per column; then blocks of twice the size
        if (tid < kC) {
            const int bi = tid >> 3, j = tid & 7;
            float *Ab = sT + 8 * bi * P::LD + 8 * bi;
            float x[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const float4 y0 = *reinterpret_cast<const float4 *>(Ab + r * P::LD), y1 = *reinterpret_cast<const float4 *>(Ab + r * P::LD + 4);
                const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int k = 0; k < r; ++k) {
                    if (k & 1) s1 = fmaf(y[k], x[k], s1);
                    else s0 = fmaf(y[k], x[k], s0);
                }
                x[r] = r == j ? 1.f : r < j ? 0.f : -(s0 + s1);
            }
            __syncwarp();                               // a block's threads are in one warp
#pragma unroll
            for (int r = 0; r < 8; ++r) Ab[r * P::LD + j] = x[r];
        }
        __syncthreads();
        inverse_level<8, P::LD>(sT, tid);
        inverse_level<16, P::LD>(sT, tid);
        inverse_level<32, P::LD>(sT, tid);
        // ---- P = T diag(beta) and F = D P: a row's 16 columns; F's terms over T first, P's after the product with them
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const float4 x4 = *reinterpret_cast<const float4 *>(sT + row * P::LD + s0 + j), b4 = *reinterpret_cast<const float4 *>(sBeta + s0 + j);
            y[j] = x4.x * b4.x;
            y[j + 1] = x4.y * b4.y;
            y[j + 2] = x4.z * b4.z;
            y[j + 3] = x4.w * b4.w;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = __uint_as_float(__float_as_uint(y[j]) & (s0 + j <= row ? 0xffffffffu : 0u));
        float2 probe = make_float2(0.f, 0.f);           // (0 times a finite number adds nothing)
#pragma unroll
        for (int j = 0; j < 16; j += 2) probe = fma2(make_float2(y[j], y[j + 1]), make_float2(0.f, 0.f), probe);
        const bool odd = !(probe.x + probe.y == 0.f);
        if (!__syncthreads_or(odd) || again) break;     // (T has been read)
        int *first = reinterpret_cast<int *>(tmem_slot + 1);
        if (tid == 0) *first = kC;
        __syncthreads();
        if (tid < kC) {
            bool bad = !(fabsf(sGh[tid]) < INFINITY && fabsf(sBeta[tid]) < INFINITY);
            for (int v = 0; v < VR; ++v) {
                const uint4 x = *reinterpret_cast<const uint4 *>(smem + (v >> 3) * P::ATOM + sw128(tid, v & 7));
                bad |= ((odd_bits(x.x) | odd_bits(x.y) | odd_bits(x.z) | odd_bits(x.w)) & 0x80008000u) != 0;
            }
            if (bad) atomicMin(first, tid);
        }
        __syncthreads();
        sound = *first;
        if (tid < kC && tid >= sound) {
            sGam[tid] = __uint_as_float(0x7fffffffu);
            sBeta[tid] = 0.f;
        }
        __syncthreads();
    }
    const float end = sEnd[row];
    // Their terms: the first two in T's place; the third is returned.
    auto put = [&](float f, uint4 (&third)[2]) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            float z[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = f * y[8 * v + j];
            uint4 m[3];
            split8(z, m);
            const uint32_t at = P::OFF_T + sw128(row, (s0 >> 3) + v);
            *reinterpret_cast<uint4 *>(smem + at) = m[0];
            *reinterpret_cast<uint4 *>(smem + P::TERM + at) = m[1];
            third[v] = m[2];
        }
    };
    auto put_third = [&](int off, const uint4 (&third)[2]) {
#pragma unroll
        for (int v = 0; v < 2; ++v) *reinterpret_cast<uint4 *>(smem + off + sw128(row, (s0 >> 3) + v)) = third[v];
        fence_proxy_async();
    };
    auto wait = [&](int i) {                        // for barrier i, to which this warp takes MMAs to have been committed
        if (ok) {
            issued = i;
            ok = __all_sync(0xffffffffu, mbar_wait(&bar[i], 0));
        }
        tc_fence_after();
    };
    uint4 third[2];
    put(end, third);
    fence_proxy_async();
    __syncthreads();
    // ---- E = K^T F (rows dk: the keys read MN-major), then, over [K;Q] K^T, M P (lanes 64..127: each term of M begins 64 rows
    //      into its operand; lanes 0..63 are not read)
    const uint32_t one = elect_one();
    const uint64_t dt = desc_mn_sw128(saddr(smem) + P::OFF_T, 8192);
    const uint64_t dk = desc_mn_sw128(saddr(smem), P::ATOM);
    constexpr uint32_t idE = idesc_mn(1, 128, kC) | kIdescMnMajorA | kIdescMnMajorB;
    if (warp == 0 && ok) {
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k)
            mma_bf16_on(one, tmem + 64, desc_add(dk, (k & 3) * 2048), desc_add(dt, (k >> 2) * P::TERM + (k & 3) * 2048), idE, k > 0);
        mma_commit_on(one, &bar[1]);
    }
    wait(1);
    put_third(P::OFF_T, third);                     // F's
    __syncthreads();
    if (warp == 0 && ok) {
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_bf16_on(one, tmem + 64, desc_add(dk, k * 2048), desc_add(dt, k * 2048), idE, 1);
        mma_commit_on(one, &bar[2]);
    }
    wait(2);
    put(1.f, third);
    if (!keys && ok)
#pragma unroll
        for (int v = 0; v < 4; ++v) *reinterpret_cast<uint4 *>(smem + P::OFF_M2 + sw128(t, 4 * half + v)) = m2[v];
    put_third(P::OFF_P2, third);
    __syncthreads();
    if (warp == 0 && ok) {
        tc_fence_after();
        constexpr uint32_t idM = idesc_mn(1, 128, kC) | kIdescMnMajorB;
        constexpr int off_m[3] = {P::OFF_M0 - 8192, P::OFF_M1 - 8192, P::OFF_M2 - 8192}, off_p[3] = {P::OFF_T, P::OFF_T + P::TERM, P::OFF_P2};
        const uint64_t dm = desc_sw128(saddr(smem)), dp = desc_mn_sw128(saddr(smem), 8192);
#pragma unroll
        for (int k = 0; k < 24; ++k)
            mma_bf16_on(one, tmem, desc_add(dm, off_m[kTermA[k >> 2]] + (k & 3) * 32), desc_add(dp, off_p[kTermB[k >> 2]] + (k & 3) * 2048), idM, k > 0);
        mma_commit_on(one, &bar[3]);
    }
    wait(3);
    __syncthreads();                                // (a wait that ran out in another warp: its MMAs are drained below)
    // ---- the terms of both into shared memory as the walk wants them, and out
    char *unit = a.ws + ((static_cast<size_t>(blockIdx.z) * ta.chunks + c) * a.H + h) * Unit<DK>::BYTES;
    if (ok) {
        if ((warp & 3) * 32 < DK)
            stage_row(tmem + lanes + 64 + 32 * half, smem, Unit<DK>::E_BYTES, (warp & 3) * 32 + lane, half);
        if (tid < kC) reinterpret_cast<float *>(unit + Unit<DK>::OFF_GAMMA)[tid] = sGam[tid];
    } else if (lane == 0) {                         // one more bounded wait for what was issued
        atomicOr(a.status, kStatusTimeout);
        if (!mbar_wait(&bar[issued], 0)) atomicOr(a.status, GDN_STATUS_DRAIN);
    }
    fence_proxy_async();
    __syncthreads();
    if (tid == 0) {
        bulk_store(unit, smem, 3 * Unit<DK>::E_BYTES);
        bulk_store_wait();
    }
    __syncthreads();
    if (ok && !keys) stage_row(tmem + lanes + 32 * half, smem, Unit<DK>::MP_BYTES, t, half);
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
        bulk_store(unit + Unit<DK>::OFF_MP, smem, 3 * Unit<DK>::MP_BYTES);
        bulk_store_wait();
    }
    if (warp == 1) tmem_dealloc(tmem, 128);
    if (waiter) pdl_wait();
}

// ------------------------------------------------------------- the walk over the chunks, by slices
// One CTA per (slice of 32 or 16 value columns, head, sequence): the walk for few heads, whose chain of dependent steps bounds it
// (3100 cycles a chunk, with 16 columns 2580: 800 to [K;Q] S^T, 900 to x, 800 to E x, 600 to the new S).  S and x are the B operands:
// rows of a slice's first, second and third terms, so one product has all of them (55 cycles an MMA of 96 columns, against 39
// for 32).
template <int DK, int SL> struct SlicePlan {
    static constexpr int KQ = DK * 256, E = 3 * Unit<DK>::E_BYTES;
    static constexpr int M_BYTES = 3 * Unit<DK>::MP_BYTES + kC * 4, V_AT = 3 * Unit<DK>::MP_BYTES + 1024, MP = V_AT + (kC * SL * 2 + 1023) / 1024 * 1024;   // M P and gamma, values
    static constexpr int S_ATOM = DK * 128, X_ATOM = kC * 128, ATOMS = SL == 32 ? 2 : 1;      // rows of 64 columns: the third terms of 32 take a second one
    static constexpr int OFF_E = 2 * KQ, OFF_MP = OFF_E + E, OFF_S = OFF_MP + 2 * MP, OFF_X = OFF_S + ATOMS * S_ATOM;
    static constexpr int OFF_BAR = OFF_X + ATOMS * X_ATOM, OFF_BAD = OFF_BAR + 256, BYTES = OFF_BAD + SL * 4;      // barriers; the first bad token by column
    static constexpr int ROWS = 256, LOAD_WARP = 8, MMA_WARP = 9, THREADS = 320;
    static constexpr int N = 3 * SL, AT = SL == 32 ? 96 : 64, TMEM_COLS = SL == 32 ? 512 : 256;       // a product's columns, and from one to the next: [K;Q] S^T, E x, M P x
    static_assert(BYTES <= 227 * 1024 && OFF_E >= 8192 && MP % 1024 == 0, "plan");
};

// A thread's C numbers, the `half`-th of a slice's row, as three bf16 terms in row `row` of a tile: the first terms of 2 C, the
// second, the third (of 32 columns an atom on).
template <int C>
__device__ __forceinline__ void put_row(uint8_t *tile, int atom, int row, int half, const float (&y)[C]) {
#pragma unroll
    for (int c = 0; c < C / 8; ++c) {
        uint4 t[3];
        split8(y + 8 * c, t);
        const int at = C / 8 * half + c;
        *reinterpret_cast<uint4 *>(tile + sw128(row, at)) = t[0];
        *reinterpret_cast<uint4 *>(tile + sw128(row, at + C / 4)) = t[1];
        *reinterpret_cast<uint4 *>(C == 16 ? tile + atom + sw128(row, at) : tile + sw128(row, at + C / 2)) = t[2];
    }
}
// The product's C columns: those with the three terms added, the smallest first.
template <int C>
__device__ __forceinline__ void get_row(uint32_t tcol, float (&y)[C]) {
    uint32_t r[C], s[C], t[C];
    if constexpr (C == 16) {
        tmem_load16(tcol, r);
        tmem_load16(tcol + 32, s);
        tmem_load16(tcol + 64, t);
    } else {
        tmem_load8(tcol, r);
        tmem_load8(tcol + 16, s);
        tmem_load8(tcol + 32, t);
    }
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < C; ++j) y[j] = __uint_as_float(r[j]) + (__uint_as_float(s[j]) + __uint_as_float(t[j]));
}

// What both walks begin with: the sequence, rows of out past it, a state without tokens.  False: nothing is left to do.
__device__ __forceinline__ bool begin_walk(const TcAdvance &ta, const AdvanceSeq &sq, int n, int h, int b, int dv0, int cols, int dk, bool zero,
                                           bool first, int threads) {
    const AdvanceArgs &a = ta.a;
    if (sq.bad) {
        if (first && threadIdx.x == 0 && h == 0 && ta.c0 == 0) atomicOr(a.status, sq.bad);
        return false;
    }
    const int t1 = min(a.T, (ta.c0 + ta.chunks) * kC);
    float *out = a.out + (static_cast<size_t>(b) * a.T * a.H + h) * ta.dv + dv0;
    for (int e = threadIdx.x;; e += threads) {
        const int t = ta.c0 * kC + n + e / cols;
        if (t >= t1) break;
        out[static_cast<size_t>(t) * a.H * ta.dv + e % cols] = 0.f;
    }
    if (n == 0 && zero)
        for (int e = threadIdx.x; e < cols * dk; e += threads)
            a.state[((static_cast<size_t>(sq.slot) * a.H + h) * ta.dv + dv0) * dk + e] = 0.f;
    return n > 0;
}

// Row r has token r (K's products, r < 64), token r - 64 (Q's) and key dimension r of the state, 16 columns in each of
// two warps.  Everything that a buffer's next use overwrites has been read by then: see each arrival.
template <int DK, int SL>
__global__ void __launch_bounds__(SlicePlan<DK, SL>::THREADS, 1)
advance_slice_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TcAdvance ta)
{
    using P = SlicePlan<DK, SL>;
    constexpr int C = SL / 2;                       // columns of a thread
    const AdvanceArgs &a = ta.a;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int h = blockIdx.y, b = ta.b0 + blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t *full_k = reinterpret_cast<uint64_t *>(smem + P::OFF_BAR), *empty_k = full_k + 2, *full_m = empty_k + 2, *empty_m = full_m + 2,
             *full_e = empty_m + 2, *empty_e = full_e + 1, *d1 = empty_e + 1, *d2 = d1 + 1, *d3 = d2 + 1, *s_ready = d3 + 1,
             *x_ready = s_ready + 1, *drain = x_ready + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1), *any_bad = abort + 1;
    int *bad = reinterpret_cast<int *>(smem + P::OFF_BAD);
    pdl_wait();
    pdl_release();
    const AdvanceSeq sq = advance_seq(a, b);
    const int n = sq.bad ? 0 : tokens_here(ta, sq.n), chunks = (n + kC - 1) / kC, dv0 = blockIdx.x * SL;
    const bool zero = sq.fresh && ta.c0 == 0;       // starts from a zero state
    if (!begin_walk(ta, sq, n, h, b, dv0, SL, DK, zero, blockIdx.x == 0, P::THREADS)) return;
    if (saddr(smem) & 1023u) {
        if (tid == 0) atomicOr(a.status, kStatusTimeout);
        return;
    }
    if (tid == 0) {
        const bool expire = (a.flags & GDN_FLAG_TEST_EXPIRE) != 0;
        for (uint64_t *bar = full_k; bar <= drain; ++bar) mbar_init(bar, bar == s_ready || bar == x_ready ? P::ROWS / 32 : 1);
        *abort = expire;                            // (a warp arrives once: 256 arrivals at one word take 500 cycles)
        *any_bad = 0;
        if (expire) atomicOr(a.status, kStatusTimeout);
        fence_mbar_init();
    }
    if (tid < SL) bad[tid] = kNever;
    if (warp == P::LOAD_WARP) tmem_alloc(tmem_slot, P::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return warp_wait(bar, parity, abort, a.status); };
    const char *units = a.ws + (static_cast<size_t>(blockIdx.z) * ta.chunks * a.H + h) * Unit<DK>::BYTES;
    const size_t ustep = static_cast<size_t>(a.H) * Unit<DK>::BYTES;
    if (warp == P::LOAD_WARP) {
        // ------------------------------------------------------ loads
        // Keys and queries go when the first product of two chunks before is done, M P (with gamma and the values) after the last
        // product of two before, and E, the last to be free, after its one use in the chunk before.  (With one barrier for all, a chunk's operands came no sooner
        // than they were needed: 600 cycles a chunk more.)
        const int hk = h / (a.H / a.Hk);
        int c = 0, part = 0;
        for (; c < chunks; ++c) {
            const int st = c & 1, before = ((c >> 1) - 1) & 1;
            const char *unit = units + c * ustep;
            part = 0;
            if (*abort || (c >= 2 && !wait(&empty_k[st], before))) break;
            if (elect_one()) {
                uint8_t *dst = smem + st * P::KQ;
                const int tok = b * a.T + (ta.c0 + c) * kC;           // (B T <= 2^28)
                mbar_expect_tx(&full_k[st], P::KQ);
#pragma unroll
                for (int at = 0; at < DK / 64; ++at) {
                    tma_load_3d(dst + at * 16384, &tm_k, at * 64, hk, tok, &full_k[st]);
                    tma_load_3d(dst + at * 16384 + 8192, &tm_q, at * 64, hk, tok, &full_k[st]);
                }
            }
            __syncwarp();
            part = 1;
            if (c >= 2 && !wait(&empty_m[st], before)) break;
            if (elect_one()) {
                uint8_t *dst = smem + P::OFF_MP + st * P::MP;
                mbar_expect_tx(&full_m[st], P::M_BYTES + kC * SL * 2);
                bulk_load(dst, unit + Unit<DK>::OFF_MP, P::M_BYTES, &full_m[st]);
                tma_load_3d(dst + P::V_AT, &tm_v, dv0, h, b * a.T + (ta.c0 + c) * kC, &full_m[st]);
            }
            __syncwarp();
            part = 2;
            if (c >= 1 && !wait(empty_e, (c - 1) & 1)) break;
            if (elect_one()) {
                mbar_expect_tx(full_e, P::E);
                bulk_load(smem + P::OFF_E, unit, P::E, full_e);
            }
            __syncwarp();
        }
        {                                           // copies in flight end before the CTA does (their users may have given up)
            bool done = true;
            const int keys = c < chunks && part > 0 ? c + 1 : c, ms = c < chunks && part > 1 ? c + 1 : c;   // chunks whose keys, whose M P have been requested
            for (int i = max(0, keys - 2); i < keys; ++i) done = done && mbar_wait(&full_k[i & 1], (i >> 1) & 1);
            for (int i = max(0, ms - 2); i < ms; ++i) done = done && mbar_wait(&full_m[i & 1], (i >> 1) & 1);
            if (c > 0) done = done && mbar_wait(full_e, (c - 1) & 1);
            if (!done && lane == 0) atomicOr(a.status, GDN_STATUS_DRAIN);
        }
    } else if (warp == P::MMA_WARP) {
        // ------------------------------------------------------ MMAs
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dS = desc_mn_sw128(saddr(smem) + P::OFF_S, P::S_ATOM), dX = desc_mn_sw128(saddr(smem) + P::OFF_X, P::X_ATOM);
        const uint64_t dKQ = desc_sw128(saddr(smem)), dE = desc_sw128(saddr(smem) + P::OFF_E), dM = desc_sw128(saddr(smem) + P::OFF_MP - 8192);
        const uint32_t one = elect_one();
        // A term of E or M P with as many terms of x as count: 3, 2 and 1 of a slice's columns.
        auto terms = [&](uint32_t acc, uint64_t left, int step) {
#pragma unroll
            for (int k = 0; k < 12; ++k)
                mma_bf16_on(one, acc, desc_add(left, (k >> 2) * step + (k & 3) * 32), desc_add(dX, (k & 3) * 2048),
                            idesc_mn(1, 128, P::N - SL * (k >> 2)) | kIdescMnMajorB, k > 0);
        };
        bool ok = true;
        int c = 0;
        for (; c < chunks; ++c) {
            const int st = c & 1;
            ok = wait(&full_k[st], (c >> 1) & 1) && wait(s_ready, c & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks)
                mma_bf16_on(one, tm, desc_add(dKQ, st * P::KQ + (ks >> 2) * 16384 + (ks & 3) * 32), desc_add(dS, ks * 2048),
                            idesc_mn(1, 128, P::N) | kIdescMnMajorB, ks > 0);
            mma_commit_on(one, d1);
            mma_commit_on(one, &empty_k[st]);
            ok = wait(full_e, c & 1) && wait(x_ready, c & 1);
            if (!ok) break;
            tc_fence_after();
            terms(tm + P::AT, dE, Unit<DK>::E_BYTES);
            mma_commit_on(one, d2);
            mma_commit_on(one, empty_e);
            ok = wait(&full_m[st], (c >> 1) & 1);
            if (!ok) break;
            terms(tm + 2 * P::AT, desc_add(dM, st * P::MP), Unit<DK>::MP_BYTES);
            mma_commit_on(one, d3);
            mma_commit_on(one, &empty_m[st]);
        }
        if (!ok) {                                  // MMAs in flight end before their memory is given back
            mma_commit_on(one, drain);
            if (!mbar_wait(drain, 0) && lane == 0) atomicOr(a.status, GDN_STATUS_DRAIN);
        }
    } else {
        // ------------------------------------------------------ rows
        const int half = warp >> 2, row = tid & 127, t = row & (kC - 1);
        const bool keys = row < kC, has = row < DK;                   // (the same in a warp)
        const uint32_t tm = tmem + C * half + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        uint8_t *sS = smem + P::OFF_S, *sX = smem + P::OFF_X;
        const int col0 = dv0 + C * half;
        float *st = a.state + ((static_cast<size_t>(sq.slot) * a.H + h) * ta.dv + col0) * DK + row;
        float S[C];
#pragma unroll
        for (int j = 0; j < C; ++j) S[j] = has && !zero ? st[j * DK] : 0.f;
        const size_t tok0 = static_cast<size_t>(b) * a.T + ta.c0 * kC + t;
        float *op = a.out + (tok0 * a.H + h) * ta.dv + col0;
        auto arrive = [&](uint64_t *bar) {          // for the warp, behind each lane's fences
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        if (has) put_row(sS, P::S_ATOM, row, half, S);
        fence_proxy_async();
        arrive(s_ready);
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
            float y[C], o[C];
            const uint8_t *slot = smem + P::OFF_MP + (c & 1) * P::MP;
            const float *gam = reinterpret_cast<const float *>(slot + 3 * Unit<DK>::MP_BYTES);
            ok = wait(&full_m[c & 1], (c >> 1) & 1) && wait(d1, c & 1);
            if (!ok) break;
            tc_fence_after();
            get_row(tm, y);
            if (keys) {                             // x = v - gamma S k; nothing of rows past the last token
                const bool live = c * kC + t < n;
                const float f = -gam[t];
#pragma unroll
                for (int i = 0; i < C / 8; ++i) {
                    float v[8];
                    bf16x8_to_f32(*reinterpret_cast<const uint4 *>(slot + P::V_AT + t * (SL * 2) + C * 2 * half + 16 * i), v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[8 * i + e] = live ? fmaf(f, y[8 * i + e], v[e]) : 0.f;
                }
                put_row(sX, P::X_ATOM, t, half, y);
                // An infinity or NaN enters the products as 0 (a row before it has a 0 for it there); its column is NaN from this token on.
                float2 probe[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int j = 0; j < C; j += 2) probe[j / 2 & 1] = fma2(make_float2(y[j], y[j + 1]), make_float2(0.f, 0.f), probe[j / 2 & 1]);
                probe[0] = add2(probe[0], probe[1]);
                if (!(probe[0].x + probe[0].y == 0.f)) {
                    *any_bad = 1;
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        if (!(fabsf(y[j]) < INFINITY)) {
                            y[j] = 0.f;
                            atomicMin(bad + C * half + j, c * kC + t);
                        }
                    put_row(sX, P::X_ATOM, t, half, y);
                }
                fence_proxy_async();
            } else {
                const float f = gam[t] * a.scale;
#pragma unroll
                for (int j = 0; j < C; ++j) o[j] = f * y[j];
            }
            const float ge = gam[kC - 1];
            tc_fence_before();
            arrive(x_ready);                        // this row has read [K;Q] S^T (and, before it, the last M P x)
            ok = wait(d2, c & 1);
            if (!ok) break;
            tc_fence_after();
            const bool spoilt = *any_bad != 0;
            if (has) {
                get_row(tm + P::AT, y);
#pragma unroll
                for (int j = 0; j < C; ++j) S[j] = fmaf(ge, S[j], y[j]);
                if (spoilt)
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        if (bad[C * half + j] != kNever) S[j] = __uint_as_float(0x7fffffffu);
                put_row(sS, P::S_ATOM, row, half, S);
                fence_proxy_async();
            }
            tc_fence_before();
            arrive(s_ready);                        // this row has read E x; S is in place
            if (!keys) {
                ok = wait(d3, c & 1);
                if (!ok) break;
                tc_fence_after();
                get_row(tm + 2 * P::AT, y);
                if (spoilt)
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        if (bad[C * half + j] <= c * kC + t) y[j] = __uint_as_float(0x7fffffffu);
                if (c * kC + t < n) {
                    float4 *dst = reinterpret_cast<float4 *>(op + static_cast<size_t>(c) * kC * a.H * ta.dv);
#pragma unroll
                    for (int j = 0; j < C / 4; ++j)
                        dst[j] = make_float4(o[4 * j] + y[4 * j], o[4 * j + 1] + y[4 * j + 1], o[4 * j + 2] + y[4 * j + 2],
                                             o[4 * j + 3] + y[4 * j + 3]);
                }
            }
        }
        if (ok && has)
#pragma unroll
            for (int j = 0; j < C; ++j) st[j * DK] = S[j];
        tc_fence_before();
    }
    __syncthreads();
    if (warp == P::LOAD_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, P::TMEM_COLS);
    }
}

// ------------------------------------------------------------- the walk over the chunks, by heads
// One CTA per (head of 128 value columns, sequence): the walk for many heads, where the work on an SM counts and not the chain.
// Here the state's columns are the rows (TMEM lanes): S and x are the A operands, straight from TMEM, and keys, queries, E and M P
// the B operands as they lie.  A head costs an SM 240 KB of shared memory traffic a chunk instead of the 800 KB of
// four slices, and nothing of S or x goes through it: 6500 cycles a chunk, of which the MMAs are 3900 (8 prompts of 16 heads, up to
// 32 chunks: 118 us).
//
// TMEM columns: S (three terms, dk / 2 each), [K;Q] S^T and over it x (three terms of 32), E x, M P x.
template <int DK> struct HeadPlan {
    static constexpr int KQ = DK * 256, E = 3 * Unit<DK>::E_BYTES;
    static constexpr int M_BYTES = 3 * Unit<DK>::MP_BYTES + kC * 4, V_AT = 3 * Unit<DK>::MP_BYTES + 1024, MP = V_AT + kC * 256;   // M P and gamma, values
    static constexpr int OFF_E = 2 * KQ, OFF_MP = OFF_E + E, OFF_BAR = OFF_MP + 2 * MP, OFF_BAD = OFF_BAR + 256, BYTES = OFF_BAD + 128 * 4;
    static constexpr int ROWS = 512, LOAD_WARP = 16, MMA_WARP = 17, THREADS = 576;
    static constexpr int COL_D1 = 3 * DK / 2, COL_X = COL_D1, COL_D2 = COL_D1 + 128, COL_D3 = COL_D2 + DK, TMEM_COLS = 512;
    static_assert(COL_D3 + kC <= TMEM_COLS && BYTES <= 227 * 1024 && MP % 1024 == 0, "plan");
};

// Row r is value column r, in four threads: each has 16 of the chunk's tokens and a quarter of the key dimensions.  An
// expired wait only stops the waiting (a thread that left would leave others at a barrier).
template <int DK>
__global__ void __launch_bounds__(HeadPlan<DK>::THREADS, 1)
advance_head_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TcAdvance ta)
{
    using P = HeadPlan<DK>;
    constexpr int DV = 128, DQ = DK / 4;            // key dimensions of a thread
    const AdvanceArgs &a = ta.a;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int h = blockIdx.y, b = ta.b0 + blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t *full_k = reinterpret_cast<uint64_t *>(smem + P::OFF_BAR), *empty_k = full_k + 2, *full_m = empty_k + 2, *empty_m = full_m + 2,
             *full_e = empty_m + 2, *empty_e = full_e + 1, *d1 = empty_e + 1, *d2 = d1 + 1, *d3 = d2 + 1, *s_ready = d3 + 1,
             *x_ready = s_ready + 1, *drain = x_ready + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1), *any_bad = abort + 1;
    int *bad = reinterpret_cast<int *>(smem + P::OFF_BAD);
    pdl_wait();
    pdl_release();
    const AdvanceSeq sq = advance_seq(a, b);
    const int n = sq.bad ? 0 : tokens_here(ta, sq.n), chunks = (n + kC - 1) / kC;
    const bool zero = sq.fresh && ta.c0 == 0;       // starts from a zero state
    if (!begin_walk(ta, sq, n, h, b, 0, DV, DK, zero, true, P::THREADS)) return;
    if (saddr(smem) & 1023u) {
        if (tid == 0) atomicOr(a.status, kStatusTimeout);
        return;
    }
    if (tid == 0) {
        const bool expire = (a.flags & GDN_FLAG_TEST_EXPIRE) != 0;
        for (uint64_t *bar = full_k; bar <= drain; ++bar) mbar_init(bar, bar == s_ready || bar == x_ready ? P::ROWS / 32 : 1);
        *abort = expire;
        *any_bad = 0;
        if (expire) atomicOr(a.status, kStatusTimeout);
        fence_mbar_init();
    }
    if (tid < DV) bad[tid] = kNever;
    if (warp == P::LOAD_WARP) tmem_alloc(tmem_slot, P::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return warp_wait(bar, parity, abort, a.status); };
    if (warp == P::LOAD_WARP) {
        // ------------------------------------------------------ loads
        const char *units = a.ws + (static_cast<size_t>(blockIdx.z) * ta.chunks * a.H + h) * Unit<DK>::BYTES;
        const size_t ustep = static_cast<size_t>(a.H) * Unit<DK>::BYTES;
        const int hk = h / (a.H / a.Hk);
        int c = 0, part = 0;
        for (; c < chunks; ++c) {
            const int st = c & 1, before = ((c >> 1) - 1) & 1;
            const char *unit = units + c * ustep;
            part = 0;
            if (*abort || (c >= 2 && !wait(&empty_k[st], before))) break;
            if (elect_one()) {
                uint8_t *dst = smem + st * P::KQ;
                const int tok = b * a.T + (ta.c0 + c) * kC;           // (B T <= 2^28)
                mbar_expect_tx(&full_k[st], P::KQ);
#pragma unroll
                for (int at = 0; at < DK / 64; ++at) {
                    tma_load_3d(dst + at * 16384, &tm_k, at * 64, hk, tok, &full_k[st]);
                    tma_load_3d(dst + at * 16384 + 8192, &tm_q, at * 64, hk, tok, &full_k[st]);
                }
            }
            __syncwarp();
            part = 1;
            if (c >= 2 && !wait(&empty_m[st], before)) break;
            if (elect_one()) {
                uint8_t *dst = smem + P::OFF_MP + st * P::MP;
                mbar_expect_tx(&full_m[st], P::M_BYTES + kC * 256);
                bulk_load(dst, unit + Unit<DK>::OFF_MP, P::M_BYTES, &full_m[st]);
                tma_load_3d(dst + P::V_AT, &tm_v, 0, h, b * a.T + (ta.c0 + c) * kC, &full_m[st]);
            }
            __syncwarp();
            part = 2;
            if (c >= 1 && !wait(empty_e, (c - 1) & 1)) break;
            if (elect_one()) {
                mbar_expect_tx(full_e, P::E);
                bulk_load(smem + P::OFF_E, unit, P::E, full_e);
            }
            __syncwarp();
        }
        {                                           // copies in flight end before the CTA does (their users may have given up)
            bool done = true;
            const int keys = c < chunks && part > 0 ? c + 1 : c, ms = c < chunks && part > 1 ? c + 1 : c;   // chunks whose keys, whose M P have been requested
            for (int i = max(0, keys - 2); i < keys; ++i) done = done && mbar_wait(&full_k[i & 1], (i >> 1) & 1);
            for (int i = max(0, ms - 2); i < ms; ++i) done = done && mbar_wait(&full_m[i & 1], (i >> 1) & 1);
            if (c > 0) done = done && mbar_wait(full_e, (c - 1) & 1);
            if (!done && lane == 0) atomicOr(a.status, GDN_STATUS_DRAIN);
        }
    } else if (warp == P::MMA_WARP) {
        // ------------------------------------------------------ MMAs
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dKQ = desc_sw128(saddr(smem)), dE = desc_sw128(saddr(smem) + P::OFF_E), dM = desc_sw128(saddr(smem) + P::OFF_MP);
        const uint32_t one = elect_one();
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1;
            ok = wait(&full_k[st], (c >> 1) & 1) && wait(s_ready, c & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 3 * DK / 16; ++k) { // the terms of S, the smallest first
                const int ks = k % (DK / 16);
                mma_bf16_ts_on(one, tm + P::COL_D1, tm + (2 - k / (DK / 16)) * (DK / 2) + ks * 8, desc_add(dKQ, st * P::KQ + (ks >> 2) * 16384 + (ks & 3) * 32), idesc_mn(1, 128, 128), k > 0);
            }
            mma_commit_on(one, d1);
            mma_commit_on(one, &empty_k[st]);
            ok = wait(full_e, c & 1) && wait(x_ready, c & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 24; ++k)
                mma_bf16_ts_on(one, tm + P::COL_D2, tm + P::COL_X + kTermA[k >> 2] * 32 + (k & 3) * 8,
                               desc_add(dE, kTermB[k >> 2] * Unit<DK>::E_BYTES + (k & 3) * 32), idesc_mn(1, 128, DK), k > 0);
            mma_commit_on(one, d2);
            mma_commit_on(one, empty_e);
            ok = wait(&full_m[st], (c >> 1) & 1);
            if (!ok) break;
#pragma unroll
            for (int k = 0; k < 24; ++k)            // (onto scale gamma S q, which the rows have put there)
                mma_bf16_ts_on(one, tm + P::COL_D3, tm + P::COL_X + kTermA[k >> 2] * 32 + (k & 3) * 8,
                               desc_add(dM, st * P::MP + kTermB[k >> 2] * Unit<DK>::MP_BYTES + (k & 3) * 32), idesc_mn(1, 128, kC), 1);
            mma_commit_on(one, d3);
            mma_commit_on(one, &empty_m[st]);
        }
        if (!ok) {                                  // MMAs in flight end before their memory is given back
            mma_commit_on(one, drain);
            if (!mbar_wait(drain, 0) && lane == 0) atomicOr(a.status, GDN_STATUS_DRAIN);
        }
    } else {
        // ------------------------------------------------------ rows
        const int q4 = warp >> 2, row = tid & 127, tq = 16 * q4;      // this thread's first token of a chunk
        const uint32_t tm = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        float *st = a.state + ((static_cast<size_t>(sq.slot) * a.H + h) * DV + row) * DK + DQ * q4;
        float2 S[DQ / 2];
#pragma unroll
        for (int j = 0; j < DQ; j += 4) {
            const float4 x = zero ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4 *>(st + j);
            S[j / 2] = make_float2(x.x, x.y);
            S[j / 2 + 1] = make_float2(x.z, x.w);
        }
        const size_t tok0 = static_cast<size_t>(b) * a.T + ta.c0 * kC + tq;
        float *op = a.out + (tok0 * a.H + h) * DV + row;
        const size_t ostep = static_cast<size_t>(a.H) * DV;
        auto put_state = [&]() {                    // S's terms: A operand, dk / 2 columns each
#pragma unroll
            for (int j = 0; j < DQ; j += 16) {
                uint32_t w[3][8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t t[3];
                    split_pair(S[j / 2 + i], t);
                    w[0][i] = t[0]; w[1][i] = t[1]; w[2][i] = t[2];
                }
#pragma unroll
                for (int k = 0; k < 3; ++k) tmem_store8(tm + k * (DK / 2) + (DQ * q4 + j) / 2, w[k]);
            }
            tmem_wait_st();
            tc_fence_before();
        };
        auto arrive = [&](uint64_t *bar) {          // for the warp, behind each lane's fences
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        put_state();
        arrive(s_ready);
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
            const int sm = c & 1;
            const float *gam = reinterpret_cast<const float *>(smem + P::OFF_MP + sm * P::MP + 3 * Unit<DK>::MP_BYTES);
            const unsigned short *val = reinterpret_cast<const unsigned short *>(smem + P::OFF_MP + sm * P::MP + P::V_AT) + tq * DV + row;
            ok = wait(&full_m[sm], (c >> 1) & 1) && ok;               // gamma and the values
            ok = wait(d1, c & 1) && ok;
            tc_fence_after();
            uint32_t y[16], z[16], w[3][8];
            tmem_load16(tm + P::COL_D1 + tq, y);
            tmem_load16(tm + P::COL_D1 + kC + tq, z);
            tmem_wait_ld();
            const bool whole = (c + 1) * kC <= n;
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                const float4 g4 = *reinterpret_cast<const float4 *>(gam + tq + j);
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float2 g = e ? make_float2(g4.z, g4.w) : make_float2(g4.x, g4.y);
                    // x = v - gamma S k; nothing of tokens past the last
                    float2 x = fma2(make_float2(-g.x, -g.y), make_float2(__uint_as_float(y[j + e]), __uint_as_float(y[j + e + 1])),
                                    make_float2(__uint_as_float(val[(j + e) * DV] << 16), __uint_as_float(val[(j + e + 1) * DV] << 16)));
                    if (!whole) {
                        x.x = c * kC + tq + j + e < n ? x.x : 0.f;
                        x.y = c * kC + tq + j + e + 1 < n ? x.y : 0.f;
                    }
                    uint32_t t[3];
                    split_pair(x, t);
                    w[0][(j + e) / 2] = t[0]; w[1][(j + e) / 2] = t[1]; w[2][(j + e) / 2] = t[2];
                    const float2 o = mul2(mul2(g, make_float2(a.scale, a.scale)), make_float2(__uint_as_float(z[j + e]), __uint_as_float(z[j + e + 1])));
                    z[j + e] = __float_as_uint(o.x);
                    z[j + e + 1] = __float_as_uint(o.y);
                }
            }
            const float ge = gam[kC - 1];
            tmem_st16(tm + P::COL_D3 + tq, z);      // (the last M P x has been read)
            tc_fence_before();
            bar_sync(1 + (warp & 3), 128);          // these lanes' [K;Q] S^T has been read: x goes over it
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 3; ++k) tmem_store8(tm + P::COL_X + 32 * k + 8 * q4, w[k]);
            // An infinity or NaN, whose second and third terms are NaN, enters the products as 0 (a token before it has a 0 for it there); its row is
            // NaN from this token on.
            uint32_t odd = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) odd |= odd_bits(w[2][j]);
            if (__any_sync(0xffffffffu, (odd & 0x80008000u) != 0)) {
                *any_bad = 1;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if ((w[2][j / 2] >> (j % 2 * 16) & 0x7f80u) == 0x7f80u) {
#pragma unroll
                        for (int k = 0; k < 3; ++k) w[k][j / 2] &= j % 2 ? 0xffffu : 0xffff0000u;
                        atomicMin(bad + row, c * kC + tq + j);
                    }
#pragma unroll
                for (int k = 0; k < 3; ++k) tmem_store8(tm + P::COL_X + 32 * k + 8 * q4, w[k]);
            }
            tmem_wait_st();
            tc_fence_before();
            arrive(x_ready);
            ok = wait(d2, c & 1) && ok;
            tc_fence_after();
            const int from = *any_bad ? bad[row] : kNever;            // the first bad token of this row
#pragma unroll
            for (int j = 0; j < DQ; j += 16) {
                tmem_load16(tm + P::COL_D2 + DQ * q4 + j, y);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i += 2)
                    S[(j + i) / 2] = fma2(make_float2(ge, ge), S[(j + i) / 2], make_float2(__uint_as_float(y[i]), __uint_as_float(y[i + 1])));
            }
            if (from != kNever)
#pragma unroll
                for (int j = 0; j < DQ / 2; ++j) S[j] = make_float2(__uint_as_float(0x7fffffffu), __uint_as_float(0x7fffffffu));
            put_state();
            arrive(s_ready);
            ok = wait(d3, c & 1) && ok;
            tc_fence_after();
            tmem_load16(tm + P::COL_D3 + tq, z);
            tmem_wait_ld();
            if (from != kNever)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c * kC + tq + j >= from) z[j] = 0x7fffffffu;
            if (ok)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c * kC + tq + j < n) op[(static_cast<size_t>(c) * kC + j) * ostep] = __uint_as_float(z[j]);
        }
        if (ok)
#pragma unroll
            for (int j = 0; j < DQ; j += 4) *reinterpret_cast<float4 *>(st + j) = make_float4(S[j / 2].x, S[j / 2].y, S[j / 2 + 1].x, S[j / 2 + 1].y);
        tc_fence_before();
    }
    __syncthreads();
    if (warp == P::LOAD_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, P::TMEM_COLS);
    }
}

// ------------------------------------------------------------------ host side
int64_t unit_bytes(const gdn_advance_dims *d) { return d->dk == 64 ? Unit<64>::BYTES : Unit<128>::BYTES; }
AdvancePlan plan_of(const gdn_advance_dims *d) { return advance_plan(d->B, d->T, d->H, d->dv, unit_bytes(d), sm_count()); }

// Keys, queries or values as [B T][heads][dim]; boxes of `cols` columns of one head, 64 tokens.
bool token_map(CUtensorMap *m, const void *base, const gdn_advance_dims *d, int heads, int dim, int64_t stride, int cols, bool swizzle) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(d->B) * d->T};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(dim) * 2, static_cast<cuuint64_t>(stride) * 2};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(cols), 1, kC}, estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The launches alternate: prep 0, walk 0, prep 1, walk 1, ..  Prep k + 1 needs nothing of walk k and runs beside it: it does not wait
// for the launch before it at its start (that launch's blocks have by then waited for prep k, so all that came before
// is over), but one of its CTAs does at its end, so that walk k + 1, which waits for prep k + 1, also comes
// after walk k.  Two workspaces: prep k + 1 begins when walk k has, and so after walk k - 1, the last reader of its own.
template <int DK>
int launch(const gdn_advance_dims *d, const AdvanceArgs &a, cudaStream_t s) {
    CUtensorMap mk, mq, mv[2];
    const AdvancePlan p = plan_of(d);
    const int columns[2] = {p.walk_columns(false), p.walk_columns(true)};
    if (!token_map(&mk, a.k, d, d->Hk, d->dk, d->k_stride, 64, true) || !token_map(&mq, a.q, d, d->Hk, d->dk, d->q_stride, 64, true) ||
        !token_map(&mv[0], a.v, d, d->H, d->dv, d->v_stride, columns[0], false) ||
        !token_map(&mv[1], a.v, d, d->H, d->dv, d->v_stride, columns[1], false))
        return GDN_ERR_LAUNCH;
    if (cudaFuncSetAttribute(advance_prep_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, PrepPlan<DK>::BYTES) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    auto walk = [&](int cols, int nb, const CUtensorMap &m, const TcAdvance &ta) {
        const int bytes = cols == 128 ? HeadPlan<DK>::BYTES : cols == 32 ? SlicePlan<DK, 32>::BYTES : SlicePlan<DK, 16>::BYTES;
        const int threads = cols == 128 ? HeadPlan<DK>::THREADS : SlicePlan<DK, 32>::THREADS;
        auto *kern = cols == 128 ? advance_head_kernel<DK> : cols == 32 ? advance_slice_kernel<DK, 32> : advance_slice_kernel<DK, 16>;
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        return e != cudaSuccess ? e : launch_pdl(kern, dim3(d->dv / cols, d->H, nb), dim3(threads), bytes, s, mk, mq, m, ta);
    };
    const int64_t second = p.unit * d->H * p.seqs * p.first_room();
    TcAdvance ta{a, 0, 0, 0, d->dv, 0};
    for (ta.b0 = 0; ta.b0 < d->B; ta.b0 += p.seqs) {
        const int nb = d->B - ta.b0 < p.seqs ? d->B - ta.b0 : p.seqs;
        ta.chunks = 0;
        for (int i = 0, c0 = 0; c0 < p.all; ++i, c0 += ta.chunks) {
            ta.c0 = c0;
            ta.chunks = p.next(i, ta.chunks, p.all - c0);
            const bool last = c0 + ta.chunks == p.all && ta.b0 + nb == d->B;
            cudaError_t e = launch_pdl(advance_prep_kernel<DK>, dim3(d->H, ta.chunks, nb), dim3(kPrepThreads), PrepPlan<DK>::BYTES, s, ta);
            if (e == cudaSuccess) e = walk(columns[last], nb, mv[last], ta);
            if (e != cudaSuccess) return GDN_ERR_LAUNCH;
            ta.behind = 1;
            ta.a.ws = ta.a.ws == a.ws ? a.ws + second : a.ws;
        }
    }
    return GDN_OK;
}

}  // namespace

// Short chunks go token by token, whose time grows with them, where the chunked form's is that of a whole chunk (heads of 128 and
// 128): 16 heads, whose rows spread over the SMs, 9.0 us for 32 tokens and 11.3 for 40, chunked 13.6; with 32 rows a CTA 13.9 for 40;
// where the CTAs share the SMs, 128 heads 14.2 for 16 and 20.7 for 24, chunked 20.9; 512 heads 46 and 68, chunked 63.
bool advance_tc_shape(const gdn_advance_dims *d) {
    if (d->in_dtype != GDN_DTYPE_BF16 || d->T <= 23) return false;
    const long long rows = static_cast<long long>(d->B) * d->H * d->dv, sms = sm_count();
    return d->T > (rows <= 16 * sms ? 50 : rows <= 32 * sms ? 38 : 23);
}

int64_t advance_tc_workspace(const gdn_advance_dims *d) {
    return plan_of(d).workspace();
}

int advance_tc(const gdn_advance_dims *d, const AdvanceArgs &a, cudaStream_t s) {
    return d->dk == 64 ? launch<64>(d, a, s) : launch<128>(d, a, s);
}

}  // namespace gdn
