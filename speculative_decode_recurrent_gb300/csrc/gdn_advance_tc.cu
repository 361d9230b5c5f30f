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
// E (dk x 64) and M P (64 x 64) do not involve the state: the first kernel makes them for all chunks at once.  The
// second walks the chunks of a head with the state at hand, two dependent products a chunk: [K;Q] S^T, then
// E x (and (M P) x beside the next).  A slice of 32 value columns needs nothing of the others, so few heads still fill
// many SMs.
//
// Precision.  Keys and queries are exact in bf16.  S, x, E and M P enter as two bf16 terms each (relative 2^-17), with
// one product less where both operands have two; the state itself stays in fp32 registers through the walk.  (One tf32
// term would leave 2^-11 of S per chunk in the state.)  The inverse is formed in fp32 by 16 x 16 blocks.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "advance_common.h"
#include "tc_async.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kC = 64;                              // tokens of a chunk
constexpr int kSlice = 32;                          // value columns of a slice
constexpr float kLog2e = 1.4426950408889634f;

// What the first kernel leaves of a chunk of a head, as the second one's operands lie in shared memory:
// E as [dk][64 tokens] bf16 rows of 128 bytes (swizzled), first and second terms; M P as [64][64] likewise; gamma.
template <int DK> struct Unit {
    static constexpr int E_BYTES = DK * 128, MP_BYTES = kC * 128;
    static constexpr int TILES = 2 * E_BYTES + 2 * MP_BYTES;
    static constexpr int BYTES = TILES + 512;       // gamma [64] fp32 at TILES
};

struct TcAdvance {
    AdvanceArgs a;
    int b0;                                         // first sequence of the launch
    int c0, chunks;                                 // first chunk, chunks of the launch
    int dv;
};

// Tokens of the launch's chunks that are in use.
__device__ __forceinline__ int tokens_here(const TcAdvance &ta, int n) { return max(0, min(n - ta.c0 * kC, ta.chunks * kC)); }

// Two numbers as two packed bf16 terms each (the sum is the number to a relative 2^-17); NaN stays in both.
__device__ __forceinline__ void split_pair(float x, float y, uint32_t &h, uint32_t &l) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x, y);
    h = *reinterpret_cast<const uint32_t *>(&a);
    const __nv_bfloat162 b = __floats2bfloat162_rn(x - __uint_as_float(h << 16), y - __uint_as_float(h & 0xffff0000u));
    l = *reinterpret_cast<const uint32_t *>(&b);
}
// Eight of them as one 16-byte chunk of each term.
__device__ __forceinline__ void split8(const float *y, uint4 &h, uint4 &l) {
    split_pair(y[0], y[1], h.x, l.x);
    split_pair(y[2], y[3], h.y, l.y);
    split_pair(y[4], y[5], h.z, l.z);
    split_pair(y[6], y[7], h.w, l.w);
}

// ------------------------------------------------------------- E and M P of every chunk
constexpr int kPrepThreads = 256;

// Shared memory, 70 KB, so that three CTAs share an SM: [K;Q] as atoms of 64 columns, 128 rows of 128 bytes each (M's
// terms go over the queries' rows of the two, E's over the whole at the end); A in fp32 (then F, then M P's terms); T in
// fp32 (then P).
template <int DK> struct PrepPlan {
    static constexpr int LD = 68;                   // floats of a row of A and T: 16-byte rows, 4 banks apart
    static constexpr int OFF_M = 8192, ATOM = 16384;
    static constexpr int OFF_A = 32768, OFF_T = OFF_A + 18432;
    static constexpr int OFF_G = OFF_T + kC * LD * 4;      // G (two words), gamma, beta, decay to the end
    static constexpr int OFF_BAR = OFF_G + 5 * kC * 4;
    static constexpr int BYTES = OFF_BAR + 64;
    static_assert(kC * LD * 4 <= 18432 && OFF_T % 1024 == 0, "A's room");
};

// One level of the inverse: with the diagonal blocks of N rows of T = (I + A)^-1 in place, those of 2 N:
// T21 = -T22 A21 T11.  X = A21 T11 lies in the block (1, 2) for the moment, so the loops stay clear of what
// is above the diagonal blocks of 8.  A thread has N / 8 neighbouring elements.
template <int N, int LD>
__device__ __forceinline__ void inverse_level(const float *sA, float *sT, int tid) {
    constexpr int W = N / 8;
    const int c = (tid & 7) * W, r = (tid >> 3) % N, lo = tid / (8 * N) * 2 * N, hi = lo + N;
    float x[W];
    auto product = [&](const float *row, const float *cols, int k0, int k1, float sign) {      // sums over [k0, k1), multiples of 4
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = 0.f;
#pragma unroll 2
        for (int k = k0; k < k1; k += 4) {
            const float4 y = *reinterpret_cast<const float4 *>(row + k);
            const float yy[4] = {sign * y.x, sign * y.y, sign * y.z, sign * y.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float *z = cols + (k + q) * LD;
                if constexpr (W == 4) {
                    const float4 zz = *reinterpret_cast<const float4 *>(z);
                    x[0] = fmaf(yy[q], zz.x, x[0]); x[1] = fmaf(yy[q], zz.y, x[1]);
                    x[2] = fmaf(yy[q], zz.z, x[2]); x[3] = fmaf(yy[q], zz.w, x[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < W; ++i) x[i] = fmaf(yy[q], z[i], x[i]);
                }
            }
        }
    };
    product(sA + (hi + r) * LD + lo, sT + lo * LD + lo + c, c & ~7, N, 1.f);
#pragma unroll
    for (int i = 0; i < W; ++i) sT[(lo + r) * LD + hi + c + i] = x[i];
    __syncthreads();
    product(sT + (hi + r) * LD + hi, sT + lo * LD + hi + c, 0, (r | 7) + 1, -1.f);
#pragma unroll
    for (int i = 0; i < W; ++i) sT[(hi + r) * LD + lo + c + i] = x[i];
    __syncthreads();
}

// 32 columns of this thread's lane from tcol on as two terms each, in columns 32 half .. of row `row` of the tiles hi and lo.
__device__ __forceinline__ void stage_row(uint32_t tcol, uint8_t *hi, uint8_t *lo, int row, int half) {
    uint32_t r[32];
    tmem_ld32(tcol, r);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint4 h, l;
        split8(reinterpret_cast<const float *>(r) + 8 * c, h, l);
        const uint32_t at = sw128(row, 4 * half + c);
        *reinterpret_cast<uint4 *>(hi + at) = h;
        *reinterpret_cast<uint4 *>(lo + at) = l;
    }
}

// One CTA per (head, chunk, sequence).  Warps w and w + 4 share TMEM lanes 32 (w % 4) .. and halve the columns.
template <int DK>
__global__ void __launch_bounds__(kPrepThreads, 3) advance_prep_kernel(const TcAdvance ta)
{
    using P = PrepPlan<DK>;
    const AdvanceArgs &a = ta.a;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int h = blockIdx.x, c = blockIdx.y, b = ta.b0 + blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_release();
    const AdvanceSeq sq = advance_seq(a, b);
    const int n = sq.bad ? 0 : tokens_here(ta, sq.n) - c * kC;          // tokens of this chunk in use
    if (n <= 0) return;
    if ((saddr(smem) & 1023u) || (a.flags & GDN_FLAG_TEST_EXPIRE)) {
        if (tid == 0) atomicOr(a.status, kStatusTimeout);
        return;
    }
    float *sA = reinterpret_cast<float *>(smem + P::OFF_A), *sT = reinterpret_cast<float *>(smem + P::OFF_T);
    float *sGh = reinterpret_cast<float *>(smem + P::OFF_G), *sGl = sGh + kC, *sGam = sGl + kC, *sBeta = sGam + kC, *sEnd = sBeta + kC;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + P::OFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + 4);
    if (tid == 0) {
        mbar_init(&bar[0], 1);
        mbar_init(&bar[1], 1);
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
                hi[i] = t < n ? a.g[at] : 0.f;
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
    // ---- A in fp32 (rows of K), M as two bf16 terms (rows of Q)
    const int t = ((warp & 1) << 5) + lane;
    const bool keys = (warp & 3) < 2;
    if (__all_sync(0xffffffffu, ok)) {
        const float gh = sGh[t], gl = sGl[t], f = keys ? sBeta[t] : a.scale;
        uint32_t r[32];
        tmem_ld32(tmem + lanes + 32 * half, r);
        tmem_wait_ld();
        float y[32];
        const int seen = t - 32 * half + (keys ? 0 : 1);          // columns j < seen count
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            const float4 h4 = *reinterpret_cast<const float4 *>(sGh + 32 * half + j), l4 = *reinterpret_cast<const float4 *>(sGl + 32 * half + j);
            y[j] = ex2(((gh - h4.x) + (gl - l4.x)) * kLog2e);
            y[j + 1] = ex2(((gh - h4.y) + (gl - l4.y)) * kLog2e);
            y[j + 2] = ex2(((gh - h4.z) + (gl - l4.z)) * kLog2e);
            y[j + 3] = ex2(((gh - h4.w) + (gl - l4.w)) * kLog2e);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j)                              // (as bits: a select here became 32 branches)
            y[j] = __uint_as_float(__float_as_uint(__uint_as_float(r[j]) * y[j] * f) & (j < seen ? 0xffffffffu : 0u));
        if (keys) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
                *reinterpret_cast<float4 *>(sA + t * P::LD + 32 * half + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                uint4 hh, ll;
                split8(y + 8 * v, hh, ll);
                const uint32_t at = P::OFF_M + sw128(t, 4 * half + v);
                *reinterpret_cast<uint4 *>(smem + at) = hh;
                *reinterpret_cast<uint4 *>(smem + P::ATOM + at) = ll;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // ---- T = (I + A)^-1: diagonal blocks of 8 by substitution, a thread per column; then blocks of twice the size
    if (tid < kC) {
        const int bi = tid >> 3, j = tid & 7;
        const float *Ab = sA + 8 * bi * P::LD + 8 * bi;
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
            sT[(8 * bi + r) * P::LD + 8 * bi + j] = x[r];
        }
    }
    __syncthreads();
    inverse_level<8, P::LD>(sA, sT, tid);
    inverse_level<16, P::LD>(sA, sT, tid);
    inverse_level<32, P::LD>(sA, sT, tid);
    // ---- P = T diag(beta) and F = D P as two bf16 terms each: a row's 16 columns, P over T and F over A
    {
        const int row = tid & (kC - 1), s0 = (tid >> 6) * 16;
        const float end = sEnd[row];
        float y[16], z[16];
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const float4 x4 = *reinterpret_cast<const float4 *>(sT + row * P::LD + s0 + j), b4 = *reinterpret_cast<const float4 *>(sBeta + s0 + j);
            y[j] = x4.x * b4.x;
            y[j + 1] = x4.y * b4.y;
            y[j + 2] = x4.z * b4.z;
            y[j + 3] = x4.w * b4.w;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            y[j] = __uint_as_float(__float_as_uint(y[j]) & (s0 + j <= row ? 0xffffffffu : 0u));
            z[j] = y[j] * end;
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            uint4 hh, ll;
            const uint32_t at = sw128(row, (s0 >> 3) + v);
            split8(y + 8 * v, hh, ll);
            *reinterpret_cast<uint4 *>(smem + P::OFF_T + at) = hh;
            *reinterpret_cast<uint4 *>(smem + P::OFF_T + 8192 + at) = ll;
            split8(z + 8 * v, hh, ll);
            *reinterpret_cast<uint4 *>(smem + P::OFF_A + at) = hh;
            *reinterpret_cast<uint4 *>(smem + P::OFF_A + 8192 + at) = ll;
        }
    }
    fence_proxy_async();
    __syncthreads();
    // ---- E = K^T F (rows dk: the keys read MN-major) and, over [K;Q] K^T, M P (lanes 64..127: M's rows follow the keys' in each
    //      atom; where dk is 64 the rows before M's second term are no data, and lanes 0..63 are not read)
    if (warp == 0) {
        tc_fence_after();
        const uint64_t dk = desc_mn_sw128(saddr(smem), P::ATOM), df = desc_mn_sw128(saddr(smem) + P::OFF_A, 8192);
        const uint64_t dp = desc_mn_sw128(saddr(smem) + P::OFF_T, 8192), dm = desc_sw128(saddr(smem));
        constexpr uint32_t idE = idesc_mn(1, 128, kC) | kIdescMnMajorA | kIdescMnMajorB, idM = idesc_mn(1, 128, kC) | kIdescMnMajorB;
        if (elect_one() && ok) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                mma_bf16(tmem + 64, desc_add(dk, ks * 2048), desc_add(df, ks * 2048), idE, ks > 0);
                mma_bf16(tmem + 64, desc_add(dk, ks * 2048), desc_add(df, 8192 + ks * 2048), idE, 1);
            }
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                mma_bf16(tmem, desc_add(dm, ks * 32), desc_add(dp, ks * 2048), idM, ks > 0);
                mma_bf16(tmem, desc_add(dm, ks * 32), desc_add(dp, 8192 + ks * 2048), idM, 1);
                mma_bf16(tmem, desc_add(dm, P::ATOM + ks * 32), desc_add(dp, ks * 2048), idM, 1);
            }
            mma_commit(&bar[1]);
        }
        __syncwarp();
    }
    ok = ok && mbar_wait(&bar[1], 0);
    tc_fence_after();
    // ---- the terms of both into shared memory as the walk wants them, and out in two copies
    char *unit = a.ws + ((static_cast<size_t>(blockIdx.z) * ta.chunks + c) * a.H + h) * Unit<DK>::BYTES;
    if (__all_sync(0xffffffffu, ok)) {
        if ((warp & 3) * 32 < DK)
            stage_row(tmem + lanes + 64 + 32 * half, smem, smem + Unit<DK>::E_BYTES, (warp & 3) * 32 + lane, half);
        if (!keys)
            stage_row(tmem + lanes + 32 * half, smem + P::OFF_A, smem + P::OFF_A + Unit<DK>::MP_BYTES, t, half);
        if (tid < kC) reinterpret_cast<float *>(unit + Unit<DK>::TILES)[tid] = sGam[tid];
    } else if (lane == 0) {                         // (nothing more was issued unless the second wait ran out: one more bounded wait)
        atomicOr(a.status, kStatusTimeout);
        if (!mbar_wait(&bar[1], 0)) atomicOr(a.status, GDN_STATUS_DRAIN);
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
        bulk_store(unit, smem, 2 * Unit<DK>::E_BYTES);
        bulk_store(unit + 2 * Unit<DK>::E_BYTES, smem + P::OFF_A, 2 * Unit<DK>::MP_BYTES);
        bulk_store_wait();
    }
    if (warp == 1) tmem_dealloc(tmem, 128);
}

// ------------------------------------------------------------- the walk over the chunks
template <int DK, int NS> struct ScanPlan {
    static constexpr int KQ = DK * 256, STAGE = KQ + Unit<DK>::TILES, STAGES = 2;
    static constexpr int S_BYTES = DK * 128, X_BYTES = kC * 128;      // rows of 32 first terms, 32 second ones
    static constexpr int OFF_S = STAGES * STAGE, OFF_X = OFF_S + NS * S_BYTES, OFF_BAR = OFF_X + NS * X_BYTES;
    static constexpr int BYTES = OFF_BAR + 256;
    static constexpr int ROWS = NS * 256, LOAD_WARP = ROWS / 32, MMA_WARP = LOAD_WARP + 1, THREADS = ROWS + 64;
    static constexpr int N = NS * 64, TMEM_COLS = NS == 1 ? 256 : 512;         // columns of a product; [K;Q] S^T, E x, M P x
    static_assert(3 * N <= TMEM_COLS && BYTES <= 227 * 1024 && STAGE % 1024 == 0, "plan");
};

// A thread's 16 numbers as two bf16 terms in row `row` of a tile of 128-byte rows: 32 first terms, then 32 second ones.
__device__ __forceinline__ void put_row(uint8_t *tile, int row, int half, const float (&y)[16]) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint4 h, l;
        split8(y + 8 * c, h, l);
        *reinterpret_cast<uint4 *>(tile + sw128(row, 2 * half + c)) = h;
        *reinterpret_cast<uint4 *>(tile + sw128(row, 2 * half + c + 4)) = l;
    }
}
// The product's 16 columns: those with the first terms and those with the second ones added.
__device__ __forceinline__ void get_row(uint32_t tcol, float (&y)[16]) {
    uint32_t r[16], s[16];
    tmem_load16(tcol, r);
    tmem_load16(tcol + 32, s);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; ++j) y[j] = __uint_as_float(r[j]) + __uint_as_float(s[j]);
}

// One CTA per (NS slices of value columns, head, sequence).  A slice has eight row warps; one warp loads and one issues
// the products of all slices together (a product's rows are read once for them: an MMA of 64 columns takes 50 cycles
// for its 128 rows of 32 bytes, one of 128 columns 67).  Row r of a slice has token r (K's products, r < 64), token r - 64 (Q's) and key dimension r of the state, 16
// columns in each of two warps (one per row: 800 cycles for x and as many for S instead of half).  Everything that a buffer's next use overwrites has been read by then: see each arrival.
template <int DK, int NS>
__global__ void __launch_bounds__(ScanPlan<DK, NS>::THREADS, 1)
advance_scan_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ TcAdvance ta)
{
    using P = ScanPlan<DK, NS>;
    const AdvanceArgs &a = ta.a;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int h = blockIdx.y, b = ta.b0 + blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t *full_k = reinterpret_cast<uint64_t *>(smem + P::OFF_BAR), *empty_k = full_k + 2, *full_e = empty_k + 2,
             *empty_e = full_e + 2, *d1 = empty_e + 2, *d2 = d1 + 1, *d3 = d2 + 1, *s_ready = d3 + 1, *x_ready = s_ready + 1, *drain = x_ready + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    pdl_wait();
    pdl_release();
    const AdvanceSeq sq = advance_seq(a, b);
    if (sq.bad) {
        if (tid == 0 && blockIdx.x == 0 && h == 0 && ta.c0 == 0) atomicOr(a.status, sq.bad);
        return;
    }
    const int n = tokens_here(ta, sq.n), chunks = (n + kC - 1) / kC;
    const int dv0 = blockIdx.x * (NS * kSlice);
    // rows of this launch past the sequence's last token
    {
        const int t1 = min(a.T, (ta.c0 + ta.chunks) * kC);
        float *out = a.out + (static_cast<size_t>(b) * a.T * a.H + h) * ta.dv + dv0;
        for (int e = tid; ; e += P::THREADS) {
            const int t = ta.c0 * kC + n + e / (NS * kSlice);
            if (t >= t1) break;
            out[static_cast<size_t>(t) * a.H * ta.dv + e % (NS * kSlice)] = 0.f;
        }
    }
    const bool zero = sq.fresh && ta.c0 == 0;       // starts from a zero state
    if (n == 0) {
        if (zero)
            for (int e = tid; e < NS * kSlice * DK; e += P::THREADS)
                a.state[((static_cast<size_t>(sq.slot) * a.H + h) * ta.dv + dv0) * DK + e] = 0.f;
        return;
    }
    if (saddr(smem) & 1023u) {
        if (tid == 0) atomicOr(a.status, kStatusTimeout);
        return;
    }
    if (tid == 0) {
        const bool expire = (a.flags & GDN_FLAG_TEST_EXPIRE) != 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full_k[i], 1);
            mbar_init(&empty_k[i], 1);
            mbar_init(&full_e[i], 1);
            mbar_init(&empty_e[i], 1);
        }
        mbar_init(d1, 1);
        mbar_init(d2, 1);
        mbar_init(d3, 1);
        mbar_init(s_ready, P::ROWS / 32);           // a warp arrives once: 256 arrivals at one word take 500 cycles
        mbar_init(x_ready, P::ROWS / 32);
        mbar_init(drain, 1);
        *abort = expire;
        if (expire) atomicOr(a.status, kStatusTimeout);
        fence_mbar_init();
    }
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
        // Keys and queries go when the first product of two chunks before is done, E and M P after its last: with one
        // barrier for both, a chunk's 80 KB came no sooner than it was needed (3000 cycles a chunk instead of 2400).
        const int hk = h / (a.H / a.Hk);
        int c = 0, half = 0;
        for (; c < chunks; ++c) {
            const int st = c & 1, before = ((c >> 1) - 1) & 1;
            uint8_t *dst = smem + st * P::STAGE;
            half = 0;
            if (*abort || (c >= 2 && !wait(&empty_k[st], before))) break;
            if (elect_one()) {
                const int tok = b * a.T + (ta.c0 + c) * kC;           // (B T <= 2^28)
                mbar_expect_tx(&full_k[st], P::KQ);
#pragma unroll
                for (int at = 0; at < DK / 64; ++at) {
                    tma_load_3d(dst + at * 16384, &tm_k, at * 64, hk, tok, &full_k[st]);
                    tma_load_3d(dst + at * 16384 + 8192, &tm_q, at * 64, hk, tok, &full_k[st]);
                }
            }
            __syncwarp();
            half = 1;
            if (c >= 2 && !wait(&empty_e[st], before)) break;
            if (elect_one()) {
                mbar_expect_tx(&full_e[st], Unit<DK>::TILES);
                bulk_load(dst + P::KQ, units + c * ustep, Unit<DK>::TILES, &full_e[st]);
            }
            __syncwarp();
        }
        if (*abort) {                               // copies in flight end before the CTA does
            bool done = true;
            const int keys = c < chunks ? c + half : c;               // chunks whose keys, and whose E, have been requested
            for (int i = max(0, keys - 2); i < keys; ++i) done = done && mbar_wait(&full_k[i & 1], (i >> 1) & 1);
            for (int i = max(0, c - 2); i < c; ++i) done = done && mbar_wait(&full_e[i & 1], (i >> 1) & 1);
            if (!done && lane == 0) atomicOr(a.status, GDN_STATUS_DRAIN);
        }
    } else if (warp == P::MMA_WARP) {
        // ------------------------------------------------------ MMAs
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dS = desc_mn_sw128(saddr(smem) + P::OFF_S, P::S_BYTES), dX = desc_mn_sw128(saddr(smem) + P::OFF_X, P::X_BYTES);
        const uint64_t dA = desc_sw128(saddr(smem));
        constexpr uint32_t id = idesc_mn(1, 128, P::N) | kIdescMnMajorB;
        const uint32_t one = elect_one();
        bool ok = true;
        int c = 0;
        for (; c < chunks; ++c) {
            const int st = c & 1;
            ok = wait(&full_k[st], (c >> 1) & 1) && wait(s_ready, c & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kq = desc_add(dA, st * P::STAGE), e = desc_add(kq, P::KQ), mp = desc_add(e, 2 * Unit<DK>::E_BYTES - 8192);
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks)
                mma_bf16_on(one, tm, desc_add(kq, (ks >> 2) * 16384 + (ks & 3) * 32), desc_add(dS, ks * 2048), id, ks > 0);
            mma_commit_on(one, d1);
            mma_commit_on(one, &empty_k[st]);
            ok = wait(&full_e[st], (c >> 1) & 1) && wait(x_ready, c & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)          // the first terms of E, then the second ones
                mma_bf16_on(one, tm + P::N, desc_add(e, (ks >> 2) * Unit<DK>::E_BYTES + (ks & 3) * 32), desc_add(dX, (ks & 3) * 2048), id, ks > 0);
            mma_commit_on(one, d2);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
                mma_bf16_on(one, tm + 2 * P::N, desc_add(mp, (ks >> 2) * Unit<DK>::MP_BYTES + (ks & 3) * 32), desc_add(dX, (ks & 3) * 2048), id, ks > 0);
            mma_commit_on(one, d3);
            mma_commit_on(one, &empty_e[st]);
        }
        if (!ok && c > 0) {                         // MMAs in flight end before their memory is given back
            if (elect_one()) mma_commit(drain);
            __syncwarp();
            if (!mbar_wait(drain, 0) && lane == 0) atomicOr(a.status, GDN_STATUS_DRAIN);
        }
    } else {
        // ------------------------------------------------------ rows
        const int sl = warp >> 3, half = (warp >> 2) & 1, row = tid & 127, t = row & (kC - 1);
        const bool keys = row < kC;                 // (the same in a warp, as the next)
        const bool has = row < DK;
        const uint32_t tm = tmem + sl * 64 + 16 * half + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        uint8_t *sS = smem + P::OFF_S + sl * P::S_BYTES, *sX = smem + P::OFF_X + sl * P::X_BYTES;
        const int col0 = dv0 + sl * kSlice + 16 * half;
        float *st = a.state + ((static_cast<size_t>(sq.slot) * a.H + h) * ta.dv + col0) * DK + row;
        float S[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) S[j] = has && !zero ? st[j * DK] : 0.f;
        const size_t tok0 = static_cast<size_t>(b) * a.T + ta.c0 * kC + t;
        const __nv_bfloat16 *vp = static_cast<const __nv_bfloat16 *>(a.v) + tok0 * a.v_stride + h * ta.dv + col0;
        float *op = a.out + (tok0 * a.H + h) * ta.dv + col0;
        uint4 v[2];
        float gam = 0.f, gend = 0.f;
        auto arrive = [&](uint64_t *bar) {          // for the warp, behind each lane's fences
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        auto fetch = [&](int c) {
            const float *gp = reinterpret_cast<const float *>(units + c * ustep + Unit<DK>::TILES);
            gam = __ldcg(gp + t);
            gend = __ldcg(gp + kC - 1);
            if (keys) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    v[i] = c * kC + t < n ? __ldg(reinterpret_cast<const uint4 *>(vp + static_cast<size_t>(c) * kC * a.v_stride) + i)
                                          : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        fetch(0);
        if (has) put_row(sS, row, half, S);
        fence_proxy_async();
        arrive(s_ready);
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
            float y[16], o[16];
            ok = wait(d1, c & 1);
            if (!ok) break;
            tc_fence_after();
            get_row(tm, y);
            if (keys) {                             // x = v - gamma S k; nothing of rows past the last token
                const bool live = c * kC + t < n;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float f[8];
                    bf16x8_to_f32(v[i], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[8 * i + e] = live ? fmaf(-gam, y[8 * i + e], f[e]) : 0.f;
                }
                put_row(sX, t, half, y);
                fence_proxy_async();
            } else {
                const float f = gam * a.scale;
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = f * y[j];
            }
            const float ge = gend;
            tc_fence_before();
            arrive(x_ready);                        // this row has read [K;Q] S^T (and, before it, the last M P x)
            if (c + 1 < chunks) fetch(c + 1);
            ok = wait(d2, c & 1);
            if (!ok) break;
            tc_fence_after();
            if (has) {
                get_row(tm + P::N, y);
#pragma unroll
                for (int j = 0; j < 16; ++j) S[j] = fmaf(ge, S[j], y[j]);
                put_row(sS, row, half, S);
                fence_proxy_async();
            }
            tc_fence_before();
            arrive(s_ready);                        // this row has read E x; S is in place
            if (!keys) {
                ok = wait(d3, c & 1);
                if (!ok) break;
                tc_fence_after();
                get_row(tm + 2 * P::N, y);
                if (c * kC + t < n) {
                    float4 *dst = reinterpret_cast<float4 *>(op + static_cast<size_t>(c) * kC * a.H * ta.dv);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        dst[j] = make_float4(o[4 * j] + y[4 * j], o[4 * j + 1] + y[4 * j + 1], o[4 * j + 2] + y[4 * j + 2],
                                             o[4 * j + 3] + y[4 * j + 3]);
                }
            }
        }
        if (ok && has)
#pragma unroll
            for (int j = 0; j < 16; ++j) st[j * DK] = S[j];
        tc_fence_before();
    }
    __syncthreads();
    if (warp == P::LOAD_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, P::TMEM_COLS);
    }
}

// ------------------------------------------------------------------ host side
constexpr int64_t kBudget = 256ll << 20;            // of workspace: chunks beyond it follow in further launches

int64_t unit_bytes(const gdn_advance_dims *d) { return d->dk == 64 ? Unit<64>::BYTES : Unit<128>::BYTES; }
int seqs_per_launch(const gdn_advance_dims *d) {
    const int64_t n = kBudget / (unit_bytes(d) * d->H);
    return static_cast<int>(n < 1 ? 1 : n < d->B ? n : d->B);
}
int chunks_per_launch(const gdn_advance_dims *d) {
    const int64_t all = (d->T + kC - 1) / kC, n = kBudget / (unit_bytes(d) * d->H * seqs_per_launch(d));
    return static_cast<int>(n < 1 ? 1 : n < all ? n : all);
}

// Keys or queries as [B T][Hk][dk]; boxes of 64 columns of one head, 64 tokens.
bool token_map(CUtensorMap *m, const void *base, const gdn_advance_dims *d, int64_t stride) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(d->dk), static_cast<cuuint64_t>(d->Hk), static_cast<cuuint64_t>(d->B) * d->T};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(d->dk) * 2, static_cast<cuuint64_t>(stride) * 2};
    cuuint32_t box[3] = {64, 1, kC}, estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int NS>
int launch(const gdn_advance_dims *d, const AdvanceArgs &a, cudaStream_t s) {
    using P = ScanPlan<DK, NS>;
    CUtensorMap mk, mq;
    if (!token_map(&mk, a.k, d, d->k_stride) || !token_map(&mq, a.q, d, d->q_stride)) return GDN_ERR_LAUNCH;
    if (cudaFuncSetAttribute(advance_prep_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, PrepPlan<DK>::BYTES) != cudaSuccess ||
        cudaFuncSetAttribute(advance_scan_kernel<DK, NS>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::BYTES) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    const int all = (d->T + kC - 1) / kC, step = chunks_per_launch(d), seqs = seqs_per_launch(d);
    TcAdvance ta{a, 0, 0, 0, d->dv};
    for (ta.b0 = 0; ta.b0 < d->B; ta.b0 += seqs)
        for (ta.c0 = 0; ta.c0 < all; ta.c0 += step) {
            const int nb = d->B - ta.b0 < seqs ? d->B - ta.b0 : seqs;
            ta.chunks = all - ta.c0 < step ? all - ta.c0 : step;
            if (launch_pdl(advance_prep_kernel<DK>, dim3(d->H, ta.chunks, nb), dim3(kPrepThreads), PrepPlan<DK>::BYTES, s, ta) != cudaSuccess ||
                launch_pdl(advance_scan_kernel<DK, NS>, dim3(d->dv / (NS * kSlice), d->H, nb), dim3(P::THREADS), P::BYTES, s, mk, mq, ta) !=
                    cudaSuccess)
                return GDN_ERR_LAUNCH;
        }
    return GDN_OK;
}

}  // namespace

// Up to 32 tokens the token-by-token kernel is faster.
bool advance_tc_shape(const gdn_advance_dims *d) { return d->in_dtype == GDN_DTYPE_BF16 && d->T > 32; }

int64_t advance_tc_workspace(const gdn_advance_dims *d) {
    return unit_bytes(d) * d->H * seqs_per_launch(d) * chunks_per_launch(d);
}

int advance_tc(const gdn_advance_dims *d, const AdvanceArgs &a, cudaStream_t s) {
    // Slices of a CTA: one where that leaves SMs without work, else two.
    const bool one = static_cast<long long>(d->B) * d->H * (d->dv / kSlice) <= sm_count();
    return d->dk == 64 ? (one ? launch<64, 1>(d, a, s) : launch<64, 2>(d, a, s)) : one ? launch<128, 1>(d, a, s) : launch<128, 2>(d, a, s);
}

}  // namespace gdn
