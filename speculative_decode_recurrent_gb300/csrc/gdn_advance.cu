// gdn_advance.cu -- committed tokens over the checkpoint of a GDN layer, for sm_103a: the C ABI entry points
// (include/gdnreplay.h) and the token-by-token kernel.  Long bf16 chunks take gdn_advance_tc.cu.
//
// Token by token, a row i of the state (one value column) is independent of the others:
//     w = beta (v_i - alpha S_i.k),   S_i <- alpha S_i + w k,   o_i = S_i.(scale q).
// Eight lanes hold a row in registers, so a token costs a row two dot products over them.  A short call
// (single tokens without a draft: 16 heads 4 us) is bound by its chain of loads and launch; a long one by that of
// dependent instructions from token to token, some 360 cycles (fp32 keys and values, whose products would be six of bf16
// terms in the chunked form, which is not built for them; 333 tokens of 30 heads 64 us, 8192 of 16 heads of 128 x 128 1.75 ms.  Four tokens at a time, with their products among themselves made ahead, took 75 where one at a time took 70; the last
// output's sum beside the next token's 63, but a sixth longer where heads share the SMs.)
#include <cuda_bf16.h>

#include "advance_common.h"
#include "tc_common.cuh"

namespace gdn {
namespace {

constexpr int kLanes = 8;                                             // of a state row
constexpr int kTile = 16;                                             // tokens staged at a time

__device__ __forceinline__ void widen(const uint4 &r, float (&f)[8]) {
    const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = __bfloat1622float2(p[i]);
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
    }
}

// Rows of DK numbers of the tile's tokens, kept as they are in memory until they go to shared memory: a thread has
// 8 numbers of each of PER rows.
template <int DK, typename TIn, int kThreads> struct RowTile {
    static constexpr int VECS = DK / 8, PER = (kTile * VECS + kThreads - 1) / kThreads;
    static constexpr int W = sizeof(TIn) == 2 ? 1 : 2;                // 16-byte words of 8 numbers
    uint4 raw[PER][W];
    __device__ __forceinline__ void load(const TIn *src, int64_t stride, int n, int tid) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = tid + i * kThreads, t = e / VECS, c = e % VECS;
#pragma unroll
            for (int w = 0; w < W; ++w)
                raw[i][w] = t < n && e < kTile * VECS ? __ldg(reinterpret_cast<const uint4 *>(src + t * stride) + c * W + w)
                                                      : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    __device__ __forceinline__ void store(float *dst, float scale, int tid) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = tid + i * kThreads;
            if (e >= kTile * VECS) break;
            float f[8];
            if constexpr (W == 1) {
                widen(raw[i][0], f);
            } else {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    f[4 * w] = __uint_as_float(raw[i][w].x); f[4 * w + 1] = __uint_as_float(raw[i][w].y);
                    f[4 * w + 2] = __uint_as_float(raw[i][w].z); f[4 * w + 3] = __uint_as_float(raw[i][w].w);
                }
            }
            float4 *p = reinterpret_cast<float4 *>(dst + e * 8);
            p[0] = make_float4(scale * f[0], scale * f[1], scale * f[2], scale * f[3]);
            p[1] = make_float4(scale * f[4], scale * f[5], scale * f[6], scale * f[7]);
        }
    }
};

__device__ __forceinline__ float wide(float x) { return x; }
__device__ __forceinline__ float wide(__nv_bfloat16 x) { return __bfloat162float(x); }

// One CTA per (ROWS state rows, head, sequence).  Lane l of a row owns the columns 32 i + 4 l .. + 3, so that a row's
// lanes move 128 contiguous bytes of the state at a time.  The next tile of tokens is on its way to
// registers while the present one is in use.
template <int DK, typename TIn, int ROWS>
__global__ void __launch_bounds__(ROWS * kLanes) advance_tokens_kernel(const AdvanceArgs a, int dv)
{
    constexpr int NC = DK / kLanes, kThreads = ROWS * kLanes;
    __shared__ float sK[2][kTile * DK], sQ[2][kTile * DK], sV[2][kTile * ROWS], sA[2][kTile], sB[2][kTile];
    const int row0 = blockIdx.x * ROWS, h = blockIdx.y, b = blockIdx.z, H = a.H;
    const int tid = threadIdx.x, r = tid / kLanes, l = tid % kLanes, c0 = l * 4;
    pdl_wait();
    pdl_release();
    const AdvanceSeq sq = advance_seq(a, b);
    if (sq.bad) {
        if (tid == 0 && blockIdx.x == 0 && h == 0) atomicOr(a.status, sq.bad);
        return;
    }
    const int n = sq.n, hk = h / (H / a.Hk);
    const size_t tok0 = static_cast<size_t>(b) * a.T;
    const TIn *qi = static_cast<const TIn *>(a.q) + tok0 * a.q_stride + hk * DK;
    const TIn *ki = static_cast<const TIn *>(a.k) + tok0 * a.k_stride + hk * DK;
    const TIn *vi = static_cast<const TIn *>(a.v) + tok0 * a.v_stride + h * dv + row0;
    const float *gi = a.g + tok0 * H + h, *bi = a.beta + tok0 * H + h;
    RowTile<DK, TIn, kThreads> tk, tq;
    float tv[2], tg = 0.f, tb = 0.f;
    auto load = [&](int t0) {
        const int m = min(kTile, n - t0);
        tk.load(ki + t0 * a.k_stride, a.k_stride, m, tid);
        tq.load(qi + t0 * a.q_stride, a.q_stride, m, tid);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = tid / ROWS + 8 * i;
            tv[i] = t < m ? wide(vi[(t0 + t) * a.v_stride + tid % ROWS]) : 0.f;
        }
        if (tid < m) {
            tg = gi[static_cast<size_t>(t0 + tid) * H];
            tb = bi[static_cast<size_t>(t0 + tid) * H];
        }
    };
    if (n > 0) load(0);
    float S[NC];
    float *st = a.state + ((static_cast<size_t>(sq.slot) * H + h) * dv + row0 + r) * DK + c0;
#pragma unroll
    for (int i = 0; i < NC / 4; ++i) {
        const float4 x = sq.fresh ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4 *>(st + 32 * i);
        S[4 * i] = x.x; S[4 * i + 1] = x.y; S[4 * i + 2] = x.z; S[4 * i + 3] = x.w;
    }
    float *out = a.out + (tok0 * H + h) * dv + row0 + r;
    const size_t ostep = static_cast<size_t>(H) * dv;
    int buf = 0;
    for (int t0 = 0; t0 < n; t0 += kTile, buf ^= 1) {
        tk.store(sK[buf], 1.f, tid);
        tq.store(sQ[buf], a.scale, tid);
#pragma unroll
        for (int i = 0; i < 2; ++i) sV[buf][tid + i * kThreads] = tv[i];
        if (tid < kTile) {
            sA[buf][tid] = expf(tg);
            sB[buf][tid] = tb;
        }
        __syncthreads();                            // (one barrier a tile: the other buffer's readers are behind it)
        if (t0 + kTile < n) load(t0 + kTile);
        const int m = min(kTile, n - t0);
        for (int t = 0; t < m; ++t) {
            float kv[NC], qv[NC];
#pragma unroll
            for (int i = 0; i < NC / 4; ++i) {
                const float4 x = *reinterpret_cast<const float4 *>(&sK[buf][t * DK + c0 + 32 * i]);
                const float4 y = *reinterpret_cast<const float4 *>(&sQ[buf][t * DK + c0 + 32 * i]);
                kv[4 * i] = x.x; kv[4 * i + 1] = x.y; kv[4 * i + 2] = x.z; kv[4 * i + 3] = x.w;
                qv[4 * i] = y.x; qv[4 * i + 1] = y.y; qv[4 * i + 2] = y.z; qv[4 * i + 3] = y.w;
            }
            float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < NC; ++c) p[c & 3] = fmaf(S[c], kv[c], p[c & 3]);
            float sk = (p[0] + p[1]) + (p[2] + p[3]);
#pragma unroll
            for (int m2 = 1; m2 < kLanes; m2 <<= 1) sk += __shfl_xor_sync(0xffffffffu, sk, m2);
            const float alpha = sA[buf][t];
            const float w = sB[buf][t] * (sV[buf][t * ROWS + r] - alpha * sk);
            float o = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                S[c] = fmaf(w, kv[c], alpha * S[c]);
                o = fmaf(S[c], qv[c], o);
            }
#pragma unroll
            for (int m2 = 1; m2 < kLanes; m2 <<= 1) o += __shfl_xor_sync(0xffffffffu, o, m2);
            if (l == 0) out[(t0 + t) * ostep] = o;
        }
    }
#pragma unroll
    for (int i = 0; i < NC / 4; ++i)
        *reinterpret_cast<float4 *>(st + 32 * i) = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
    for (int t = n + tid / ROWS; t < a.T; t += kLanes)               // rows past the chunk
        a.out[((tok0 + t) * H + h) * dv + row0 + tid % ROWS] = 0.f;
}

int check_advance(const gdn_advance_dims *d) {
    if (!d) return GDN_ERR_NULL;
    if (d->in_dtype != GDN_DTYPE_BF16 && d->in_dtype != GDN_DTYPE_F32) return GDN_ERR_DTYPE;
    if (d->B < 0 || d->B > 65535 || d->T < 1 || d->T > 1 << 20 || static_cast<long long>(d->B) * d->T > 1 << 28) return GDN_ERR_DIMS;
    if (d->H < 1 || d->H > 1024 || d->Hk < 1 || d->H % d->Hk != 0 || d->n_slot < d->B) return GDN_ERR_DIMS;
    if ((d->dk != 64 && d->dk != 128) || (d->dv != 64 && d->dv != 128) || (d->flags & ~GDN_FLAG_TEST_EXPIRE)) return GDN_ERR_DIMS;
    if (static_cast<long long>(d->n_slot) * d->H * d->dv > 0x7fffffffLL) return GDN_ERR_DIMS;
    const int e = d->in_dtype == GDN_DTYPE_BF16 ? 2 : 4;
    const int64_t lim = 1ll << 38;                                    // (a tensor map's stride is below 2^40 bytes)
    if (d->q_stride < static_cast<int64_t>(d->Hk) * d->dk || d->k_stride < static_cast<int64_t>(d->Hk) * d->dk ||
        d->v_stride < static_cast<int64_t>(d->H) * d->dv || d->q_stride * e % 16 || d->k_stride * e % 16 ||
        d->v_stride * e % 16 || d->q_stride > lim || d->k_stride > lim || d->v_stride > lim)
        return GDN_ERR_DIMS;
    return GDN_OK;
}
bool on16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename TIn, int ROWS>
cudaError_t launch_rows(const gdn_advance_dims *d, const AdvanceArgs &a, cudaStream_t s) {
    const dim3 grid(d->dv / ROWS, d->H, d->B), block(ROWS * kLanes);
    return d->dk == 64 ? launch_pdl(advance_tokens_kernel<64, TIn, ROWS>, grid, block, 0, s, a, d->dv)
                       : launch_pdl(advance_tokens_kernel<128, TIn, ROWS>, grid, block, 0, s, a, d->dv);
}
template <typename TIn>
cudaError_t launch_tokens(const gdn_advance_dims *d, const AdvanceArgs &a, cudaStream_t s) {
    // Fewer rows a CTA while each then has an SM of its own: its warps share the SM's way to shared memory (16 heads of 128 x 128, 32
    // tokens: 16 rows 9.0 us, 32 rows 11.3; a token alone 3.6 and 4.3).
    const long long rows = static_cast<long long>(d->B) * d->H * d->dv, sms = tc::sm_count();
    return rows <= 8 * sms ? launch_rows<TIn, 8>(d, a, s) : rows <= 16 * sms ? launch_rows<TIn, 16>(d, a, s) : launch_rows<TIn, 32>(d, a, s);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int64_t gdn_replay_advance_workspace(const gdn_advance_dims *d) {
    if (const int rc = check_advance(d)) return rc;
    return advance_tc_shape(d) && d->B > 0 ? advance_tc_workspace(d) : 0;
}

int gdn_replay_advance(const gdn_advance_dims *d, float *state, const int32_t *state_idx, const int32_t *buf_len,
                       const int32_t *chunk_len, const int32_t *fresh, const void *q, const void *k, const void *v,
                       const float *g, const float *beta, float *out, void *workspace, int64_t workspace_bytes,
                       int32_t *status, cudaStream_t stream)
{
    const int64_t need = gdn_replay_advance_workspace(d);
    if (need < 0) return static_cast<int>(need);
    if (d->B == 0) return GDN_OK;
    if (!state || !q || !k || !v || !g || !beta || !out || !status || (need > 0 && !workspace)) return GDN_ERR_NULL;
    if (workspace_bytes < need || !on16(state) || !on16(q) || !on16(k) || !on16(v) || !on16(out) || !on16(workspace))
        return GDN_ERR_DIMS;
    const AdvanceArgs a{state, state_idx, buf_len, chunk_len, fresh, q, k, v, g, beta, out, static_cast<char *>(workspace),
                        status, d->q_stride, d->k_stride, d->v_stride, d->B, d->T, d->H, d->Hk, d->n_slot, d->flags, d->scale};
    if (advance_tc_shape(d)) return advance_tc(d, a, stream);
    const cudaError_t e = d->in_dtype == GDN_DTYPE_BF16 ? launch_tokens<__nv_bfloat16>(d, a, stream)
                                                        : launch_tokens<float>(d, a, stream);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // extern "C"
