// gdn_attn_chunk_tc.cu -- attention of a chunk of new tokens over the paged cache on the tensor cores (bf16, tcgen05), for
// sm_103a.  C ABI and layouts: include/gdnattn.h.
//
// Mathematics.  As in gdn_attn_chunk.cu, with a reference m in the maximum's place: it is raised (o and l rescaled)
// only when a tile's maximum exceeds it by more than 8 in powers of two, so weights stay below 2^8 and most tiles
// rescale nothing.  Weights enter the second product as one bf16 term: each is off by 2^-8 of itself at most, unbiased,
// which over a row's keys adds about as much as rounding the output does (two terms, as the verify of drafts takes
// them, would make the second product, half of all the work here, twice as long).  l is the sum of the weights in fp32.
//
// What bounds it: the MMAs, and shared memory with them (an MMA of 128 rows by 128 keys takes 63 cycles with 64 of reads, one of
// 64 keys 47 instead of 32).  A CTA has two tiles of 128 rows (row r = t G + g: tokens times the query heads of a key
// head) whose softmaxes and products overlap.  Tiles of 128 keys leave TMEM for one score buffer of each row tile, so a
// tile's softmax, its weights' product and the next scores follow one another: the weights go to their product in
// halves, so that the first half's runs while the second is computed.  (Whole: 3500 cycles for the 2000 of a pair's
// MMAs; tiles of 64 keys in two buffers: 2 x 1770.)
//
// Roles.  Two groups of 128 threads, one per row (no exchange between lanes; the scores of a row are in registers), and
// for each group a warp that issues: O += P_i V_i, then the scores of the next tile into the buffer that held P_i (the weights
// go over the scores in TMEM and are the A operand from there; the order of issue keeps the two apart).  A warp each loads
// keys and values (TMA through the block table).  d 256: the sums of 256 columns of two row tiles leave no room for
// scores, so a CTA takes 128 columns of the values and both halves form the scores; its tiles of 64 keys (shared
// memory holds no larger ones) have two buffers.
//
// Work.  A CTA is (pair of row tiles, key head, sequence, part of the keys); the longest come first.  Keys are cut
// into parts where the pairs alone would leave SMs without work (best_splits), joined by gdn_attn_chunk.cu.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "chunk_common.h"
#include "tc_async.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kRows = 128;                          // rows of a tile
constexpr int kMaxSplits = 64;

template <int D> struct Plan {
    static constexpr int DV = D == 256 ? 128 : D;   // value columns of a CTA
    static constexpr int KT = D == 256 ? 64 : 128, NB = D == 256 ? 2 : 1;      // keys of a tile, score buffers
    static constexpr int NK = D == 64 ? 5 : D == 128 ? 3 : 2, NV = D == 64 ? 4 : 2;      // stages
    static constexpr int QA = D / 64, VA = DV / 64; // 64-column atoms of 128-byte rows
    static constexpr int Q_BYTES = kRows * D * 2, K_BYTES = KT * D * 2, V_BYTES = KT * DV * 2;
    static constexpr int OFF_K = 2 * Q_BYTES, OFF_V = OFF_K + NK * K_BYTES, OFF_XCH = OFF_V + NV * V_BYTES;
    static constexpr int OFF_BAR = OFF_XCH + 512 * 4, BYTES = OFF_BAR + 512;
    static constexpr int MMA_WARP = 0, LOAD_WARP = 2, ROW_WARP = 4, THREADS = 20 * 32;
    static constexpr int COL_S = 0, COL_O = 2 * NB * KT;       // TMEM: the score buffers of each row tile, then their sums
    static_assert(COL_O + 2 * DV <= 512 && BYTES <= 227 * 1024, "plan");
};

template <int D>
__global__ void __launch_bounds__(Plan<D>::THREADS, 1)
chunk_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ ChunkArgs a)
{
    using P = Plan<D>;
    constexpr int DV = P::DV, KT = P::KT, HALVES = D / DV;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.G, Hkv = a.s.Hkv;
    int id = blockIdx.x;                            // ((pair, part, half), sequence, key head)
    const int h = id % Hkv;
    id /= Hkv;
    const int b = id % a.s.B;
    id /= a.s.B;
    const int half = id % HALVES;
    id /= HALVES;
    const int part = id % a.splits, pairs = (a.row_tiles + 1) / 2, rt0 = (pairs - 1 - id / a.splits) * 2;      // long ones first
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + P::OFF_BAR), *k_empty = k_full + P::NK, *v_full = k_empty + P::NK,
             *v_empty = v_full + P::NV, *q_full = v_empty + P::NV, *s_full = q_full + 1, *p_full = s_full + 4, *o_done = p_full + 4,
             *turn = o_done + 2, *drain = turn + 2;                 // s_full [group][buffer], p_full [group][buffer]; o_done, turn, drain [group]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 2);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    static_assert((2 * P::NK + 2 * P::NV + 15) * 8 + 8 <= 512, "barriers");
    if (saddr(smem) & 1023u) {
        if (tid == 0) atomicOr(a.s.status, kStatusTimeout);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < P::NK; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 2);              // the warps of both groups
        }
        for (int i = 0; i < P::NV; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 2);
        }
        mbar_init(q_full, 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&o_done[i], 1);
            mbar_init(&turn[i], 1);
            mbar_init(&drain[i], 1);
        }
        *abort = (a.flags & GDN_FLAG_TEST_EXPIRE) != 0;
        fence_mbar_init();
    }
    pdl_wait();
    pdl_release();
    const Seq sq = load_seq<true>(a.s, b);
    const int t0 = rt0 * a.tpt;                     // first token of the pair
    if (sq.bad) {
        if (tid == 0 && blockIdx.x == static_cast<unsigned>(b * Hkv)) atomicOr(a.s.status, sq.bad);
        return;
    }
    // A tile's rows in use and the keys that its last one sees; nothing of a tile without rows in use
    int live[2], tiles[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int tg = t0 + g * a.tpt, n = min(a.tpt, sq.n - tg);
        live[g] = max(n, 0) * G;
        tiles[g] = n > 0 ? (sq.len + tg + n + KT - 1) / KT : 0;
    }
    // row r of tile g is token t0 + g tpt + r / G, head h G + r % G
    auto row_at = [&](int g, int r) {
        return (static_cast<size_t>(b) * a.s.T + t0 + g * a.tpt + r / G) * a.Hq + h * G + r % G;
    };
    if (live[0] == 0) {                             // no rows in use: zeros
        if (part == 0)
            for (int g = 0; g < 2; ++g) {
                const int rows = min(a.tpt, a.s.T - t0 - g * a.tpt) * G;
                for (int r = warp; r < rows; r += P::THREADS / 32) {
                    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.out) + row_at(g, r) * D + half * DV;
                    for (int c = lane * 8; c < DV; c += 256) *reinterpret_cast<uint4 *>(o + c) = make_uint4(0u, 0u, 0u, 0u);
                    if (a.lse && half == 0 && lane == 0) a.lse[row_at(g, r)] = -INFINITY;
                }
            }
        return;
    }
    if (warp == P::MMA_WARP) {
        if (*abort && lane == 0) atomicOr(a.s.status, kStatusTimeout);
        tmem_alloc(tmem_slot, 512);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return warp_wait(bar, parity, abort, a.s.status); };
    int first, end;                                 // this part's tiles of keys, and those that each row tile sees of them
    part_range(max(tiles[0], tiles[1]), part, a.splits, first, end);
    const int count = end - first, n0 = max(0, min(end, tiles[0]) - first), n1 = max(0, min(end, tiles[1]) - first);
    const int total = sq.len + sq.n;                // tokens whose keys and values are there
    if (warp == P::LOAD_WARP || warp == P::LOAD_WARP + 1) {
        // ------------------------------------------------------ loads: keys, values
        const bool vals = warp != P::LOAD_WARP;
        const CUtensorMap *map = vals ? &tm_v : &tm_k;
        uint64_t *full = vals ? v_full : k_full, *empty = vals ? v_empty : k_empty;
        const int ns = vals ? P::NV : P::NK, bytes = vals ? P::V_BYTES : P::K_BYTES, atoms = vals ? P::VA : P::QA;
        const int x0 = vals ? half * DV : 0, shift = a.s.page_shift;
        const int rows = min(1 << shift, KT), per = KT / rows;        // rows of a copy, copies of a tile (and atom)
        uint8_t *base = smem + (vals ? P::OFF_V : P::OFF_K);
        const int32_t *tab = a.s.table + static_cast<size_t>(sq.slot) * a.s.max_pages;
        const bool asked = !vals && count > 0 && __all_sync(0xffffffffu, !*abort);
        if (asked && elect_one()) {                 // the queries of both row tiles
            const int two = live[1] > 0 ? 2 : 1;
            mbar_expect_tx(q_full, two * P::QA * a.tpt * G * 128);
            for (int g = 0; g < two; ++g)
                for (int x = 0; x < P::QA; ++x)
                    tma_load_3d(smem + g * P::Q_BYTES + x * (kRows * 128), &tm_q, x * 64, h * G, b * a.s.T + t0 + g * a.tpt, q_full);
        }
        __syncwarp();
        int st = 0, round = 0, i = 0;
        int ids = 0, base_p = -1;                   // block-table entries base_p + lane
        for (; i < count; ++i) {
            if (*abort || (round > 0 && !wait(&empty[st], (round - 1) & 1))) break;
            const int j0 = (first + i) * KT, p0 = j0 >> shift;
            if (base_p < 0 || p0 + per > base_p + 32) {               // (a tile's entries, 8 at most, lie in one batch)
                base_p = p0;
                const int p = p0 + lane;
                ids = 0;
                if (static_cast<long long>(p) << shift < total) {
                    ids = __ldg(tab + p);
                    if (ids < 0 || ids >= a.s.n_page) {
                        atomicOr(a.s.status, GDN_STATUS_BAD_PAGE);
                        ids = 0;
                    }
                }
            }
            const int here = min(per, (total - j0 + rows - 1) / rows);         // copies that hold tokens
            const bool one = elect_one();
            if (one) mbar_expect_tx(&full[st], here * rows * 128 * atoms);
            for (int c = 0; c < here; ++c) {
                const int row = ((__shfl_sync(0xffffffffu, ids, p0 + c - base_p) * Hkv + h) << shift) + ((j0 + c * rows) & ((1 << shift) - 1));
                if (one)
                    for (int x = 0; x < atoms; ++x)
                        tma_load_2d(base + st * bytes + x * (KT * 128) + c * rows * 128, map, x0 + x * 64, row, &full[st]);
                __syncwarp();
            }
            if (++st == ns) st = 0, ++round;
        }
        {                                           // copies in flight end before the CTA does (their users may have given up)
            bool done = vals || !asked || mbar_wait(q_full, 0);
            for (int y = max(0, i - ns); y < i; ++y) done = done && mbar_wait(&full[y % ns], (y / ns) & 1);
            if (!done && lane == 0) atomicOr(a.s.status, GDN_STATUS_DRAIN);
        }
    } else if (warp < P::LOAD_WARP) {
        // ------------------------------------------------------ MMAs of a group
        // Issuing holds a warp up until its MMAs have nearly run, and each wait on a barrier costs it some 300 cycles, which
        // one warp for both groups left the tensor cores idle.  Each group's warp waits while the other's MMAs
        // run; a group's last product and its next scores go in one piece, in turns (`turn`), so that the groups' softmaxes
        // stay half a period apart (without turns they fall into step, and both wait for the tensor cores at once).
        const int g = __shfl_sync(0xffffffffu, warp - P::MMA_WARP, 0), n = g ? n1 : n0;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), t_s = tm + P::COL_S + g * (P::NB * KT), t_o = tm + P::COL_O + g * DV;
        const uint64_t dq = desc_sw128(saddr(smem) + g * P::Q_BYTES), dk0 = desc_sw128(saddr(smem) + P::OFF_K),
                       dv0 = desc_mn_sw128(saddr(smem) + P::OFF_V, KT * 128);
        constexpr uint32_t idS = idesc_mn(1, kRows, KT), idO = idesc_mn(1, kRows, DV) | kIdescMnMajorB;
        const uint32_t one = elect_one();
        int ks = 0, kr = 0, vs = 0, vr = 0;         // stages of the next keys and values, and their rounds
        bool issued = false;
        auto scores = [&](int i) {                  // Q K^T of tile i, whose keys are there, into buffer i % NB
            const uint64_t kd = desc_add(dk0, ks * P::K_BYTES);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                mma_bf16_on(one, t_s + i % P::NB * KT, desc_add(dq, (k >> 2) * (kRows * 128) + (k & 3) * 32),
                            desc_add(kd, (k >> 2) * (KT * 128) + (k & 3) * 32), idS, k > 0);
            mma_commit_on(one, &s_full[2 * g + i % P::NB]);
            issued = true;
        };
        // A tile that only the other group sees is passed on once it is there (an arrival before that would count for
        // the round before).
        auto free_keys = [&](int i) {
            if (i < n) mma_commit_on(one, &k_empty[ks]);
            else if (lane == 0) mbar_arrive(&k_empty[ks]);
            if (++ks == P::NK) ks = 0, ++kr;
        };
        bool ok = count == 0 || wait(q_full, 0);
        for (int i = 0; ok && i < min(count, P::NB); ++i) {
            ok = wait(&k_full[ks], kr & 1);
            if (!ok) break;
            tc_fence_after();
            if (i < n) scores(i);
            free_keys(i);
        }
        for (int i = 0; ok && i < count; ++i) {
            const int j = i + P::NB;                // the tile whose scores follow
            ok = wait(&v_full[vs], vr & 1) && (j >= count || wait(&k_full[ks], kr & 1));
            const uint64_t vd = desc_add(dv0, vs * P::V_BYTES);
            if (i < n) ok = ok && wait(&p_full[2 * g + i % P::NB], (i / P::NB) & 1);
            ok = ok && ((g == 0 && i == 0) || wait(&turn[g], (g ? i : i - 1) & 1));
            if (!ok) break;
            tc_fence_after();
            if (i < n) {
#pragma unroll
                for (int k = 0; k < KT / 16; ++k)   // O += P_i V_i
                    mma_bf16_ts_on(one, t_o, t_s + i % P::NB * KT + k * 8, desc_add(vd, k * 2048), idO, i > 0 || k > 0);
            }
            if (i < n) {
                mma_commit_on(one, &o_done[g]);
                mma_commit_on(one, &v_empty[vs]);
            } else if (lane == 0) {
                mbar_arrive(&v_empty[vs]);
            }
            if (++vs == P::NV) vs = 0, ++vr;
            if (j < n) scores(j);
            if (lane == 0) mbar_arrive(&turn[g ^ 1]);
            if (j < count) free_keys(j);
            __syncwarp();
        }
        if (!ok && issued) {                        // MMAs in flight end before their memory is given back
            mma_commit_on(one, &drain[g]);
            if (!mbar_wait(&drain[g], 0) && lane == 0) atomicOr(a.s.status, GDN_STATUS_DRAIN);
        }
    } else {
        // ------------------------------------------------------ rows
        // Thread (group, half of a tile's keys and of the output's columns, row).  An expired wait only stops the waiting
        // (a thread that left would leave its pair at a barrier).
        const int rw = warp - P::ROW_WARP, rt = tid - P::ROW_WARP * 32;
        const int g = rw >> 3, kh = (rw >> 2) & 1, r = (warp & 3) * 32 + lane, n = g ? n1 : n0, pair_id = 1 + g * 4 + (warp & 3);
        constexpr int KH = KT / 2, DH = DV / 2;
        const int tg = t0 + g * a.tpt;
        float *xch = reinterpret_cast<float *>(smem + P::OFF_XCH);
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s0 = tmem + lanes + P::COL_S + g * (P::NB * KT), t_o = tmem + lanes + P::COL_O + g * DV + kh * DH;
        const bool used = r < (g ? live[1] : live[0]);
        const int lim = used ? sq.len + tg + r / G + 1 : 0;           // keys that this row sees
        const int free_to = sq.len + tg + 1;                          // keys that every row in use sees
        const bool whole = (g ? live[1] : live[0]) == kRows;
        float m = -INFINITY, l = 0.f;               // m: the same in both threads of a row; l: of this one's keys
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int j0 = (first + i) * KT;
            if (j0 + KT > total) {
                // values past the last token hold anything: zeros in their place (by both groups, each before its weights
                // go to their product)
                const int vst = i % P::NV;
                ok = wait(&v_full[vst], (i / P::NV) & 1) && ok;
                const int from = max(0, total - j0);
                for (int e = (rt & 255) + from * (DV / 8); e < KT * (DV / 8); e += 256) {
                    const int row = e / (DV / 8), c = e % (DV / 8);
                    *reinterpret_cast<uint4 *>(smem + P::OFF_V + vst * P::V_BYTES + (c >> 3) * (KT * 128) + sw128(row, c & 7)) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async();
            }
            const uint32_t t_s = t_s0 + i % P::NB * KT;
            ok = wait(&s_full[2 * g + i % P::NB], (i / P::NB) & 1) && ok;
            tc_fence_after();
            uint32_t x[KH / 32][32];
#pragma unroll
            for (int c = 0; c < KH / 32; ++c) tmem_ld32(t_s + kh * KH + 32 * c, x[c]);
            tmem_wait_ld();
            if (!whole || j0 + KT > free_to) {
                const int seen = lim - j0 - kh * KH;
#pragma unroll
                for (int k = 0; k < KH; ++k) x[k >> 5][k & 31] = k < seen ? x[k >> 5][k & 31] : 0xff800000u;
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < KH; k += 8)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    top[q] = fmaxf(top[q], fmaxf(__uint_as_float(x[k >> 5][(k & 31) + 2 * q]), __uint_as_float(x[k >> 5][(k & 31) + 2 * q + 1])));
            const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2;
            // (also: both threads of each row have read their scores, which the weights go over)
            if (pair_any(pair_id, mt > m + 8.f)) {
                xch[rt] = mt;
                bar_sync(pair_id, 64);
                const float mp = fmaxf(mt, xch[rt ^ 128]);
                bar_sync(pair_id, 64);              // read before it is written again
                float fac = 1.f;
                if (mp > m + 8.f) {
                    fac = ex2(m - mp);              // 0 when nothing was summed
                    m = mp;
                    l *= fac;
                }
                if (i > 0) {                        // the sums so far: their last product must be done (the one before it
                                                    // is, as its weights' buffer holds these scores)
                    ok = wait(&o_done[g], (i - 1) & 1) && ok;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < DH; c += 8) {                 // (few at a time: the scores stay in registers)
                        uint32_t o[8];
                        tmem_load8(t_o + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fac);
                        tmem_store8(t_o + c, o);
                    }
                }
            }
            const float ms = m == -INFINITY ? 0.f : m;
            const float2 sc = make_float2(a.scale_log2, a.scale_log2), mm = make_float2(-ms, -ms);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < KH / 32; ++c) {
                uint32_t p[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float2 e = fma2(make_float2(__uint_as_float(x[c][2 * k]), __uint_as_float(x[c][2 * k + 1])), sc, mm);
                    e = make_float2(ex2(e.x), ex2(e.y));
                    sum[k & 1] = add2(sum[k & 1], e);
                    const __nv_bfloat162 w = __floats2bfloat162_rn(e.x, e.y);
                    p[k] = *reinterpret_cast<const uint32_t *>(&w);
                }
                tmem_st16(t_s + kh * (KH / 2) + 16 * c, p);
            }
            l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * g + i % P::NB]);
        }
        if (n > 0) {                                // the last scores came after the product of NB + 1 tiles before: one phase after the other
            ok = (P::NB == 1 || n == 1 || wait(&o_done[g], n & 1)) && wait(&o_done[g], (n - 1) & 1) && ok;
            tc_fence_after();
        }
        xch[rt] = l;
        bar_sync(pair_id, 64);
        l += xch[rt ^ 128];
        const int rows = min(a.tpt, a.s.T - tg) * G, c0 = half * DV + kh * DH;          // this thread's first output column
        if (ok && a.splits > 1 && (g ? live[1] : live[0]) > 0) {
            const size_t unit = (static_cast<size_t>(b) * Hkv + h) * a.row_tiles + rt0 + g;
            float *w = a.ws + (unit * a.splits + part) * (static_cast<size_t>(kRows) * (D + 2));
            if (n > 0)
#pragma unroll 1
                for (int c = 0; c < DH; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(t_o + c, o);
                    tmem_wait_ld();
                    float4 *dst = reinterpret_cast<float4 *>(w + static_cast<size_t>(r) * D + c0 + c);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        dst[k] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]), __uint_as_float(o[4 * k + 2]),
                                             __uint_as_float(o[4 * k + 3]));
                }
            if (half == 0 && kh == 0) {
                w[static_cast<size_t>(kRows) * D + r] = m;
                w[static_cast<size_t>(kRows) * (D + 1) + r] = l;
            }
        } else if (ok && (a.splits == 1 || part == 0)) {              // (the join passes over a tile without rows in use)
            const float inv = used ? 1.f / l : 0.f;
            const size_t at = r < rows ? row_at(g, r) : 0;
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + at * D + c0);
#pragma unroll 1
            for (int c = 0; c < DH; c += 32) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld32(t_o + c, o);
                    tmem_wait_ld();
                }
                if (r < rows) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __nv_bfloat162 z = __floats2bfloat162_rn(__uint_as_float(o[8 * k + 2 * e]) * inv, __uint_as_float(o[8 * k + 2 * e + 1]) * inv);
                            y[e] = used ? *reinterpret_cast<const uint32_t *>(&z) : 0u;
                        }
                        dst[c / 8 + k] = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
            }
            if (a.lse && half == 0 && kh == 0 && r < rows) a.lse[at] = used ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == P::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ host side
// The layer's keys or values as rows of d; boxes of 64 columns of a page's rows (at most a tile's).
bool rows_map(CUtensorMap *m, const void *base, const gdn_page_cache *c, int keys) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(c->d), static_cast<cuuint64_t>(c->n_page) * c->Hkv * c->page};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(c->d) * 2};
    cuuint32_t box[2] = {64, static_cast<cuuint32_t>(c->page < keys ? c->page : keys)}, estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The queries as [B T][Hq][d]; boxes of a row tile's tokens and a key head's queries.
bool query_map(CUtensorMap *m, const void *base, const gdn_page_cache *c, const gdn_attn_dims *d, int tpt) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(c->d), static_cast<cuuint64_t>(d->Hq), static_cast<cuuint64_t>(d->B) * d->T};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(c->d) * 2, static_cast<cuuint64_t>(c->d) * 2 * d->Hq};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(d->Hq / c->Hkv), static_cast<cuuint32_t>(tpt)}, estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int tile_tokens(const gdn_page_cache *c, const gdn_attn_dims *d) { return kRows / (d->Hq / c->Hkv); }
int row_tiles(const gdn_page_cache *c, const gdn_attn_dims *d) { return (d->T + tile_tokens(c, d) - 1) / tile_tokens(c, d); }
long long units(const gdn_page_cache *c, const gdn_attn_dims *d) {
    return static_cast<long long>(d->B) * c->Hkv * ((row_tiles(c, d) + 1) / 2) * (c->d == 256 ? 2 : 1);
}
// Parts of the key axis: the waves of CTAs times a part's share, plus a tenth of a unit for each part's beginning, end and
// join; at least 512 keys each, as far as a sequence can be long.
int best_splits(const gdn_page_cache *c, const gdn_attn_dims *d) {
    const long long u = units(c, d), sms = sm_count();
    if (u >= 4 * sms || sms < 1) return 1;
    const int keys = 512;
    long long most = (static_cast<long long>(c->max_pages) * c->page + keys - 1) / keys;
    if (most > kMaxSplits) most = kMaxSplits;
    int best = 1;
    double cost = 1e30;
    for (int s = 1; s <= most; ++s) {
        const double x = static_cast<double>((u * s + sms - 1) / sms) / s + (s > 1 ? 0.01 * s : 0.0);
        if (x < cost * 0.98) {
            cost = x;
            best = s;
        }
    }
    return best;
}

template <int D>
int launch(const gdn_page_cache *c, const gdn_attn_dims *d, ChunkArgs a, cudaStream_t s) {
    using P = Plan<D>;
    a.tpt = tile_tokens(c, d);
    a.row_tiles = row_tiles(c, d);
    a.splits = best_splits(c, d);
    CUtensorMap mq, mk, mv;
    if (!query_map(&mq, a.q, c, d, a.tpt) || !rows_map(&mk, a.k, c, P::KT) || !rows_map(&mv, a.v, c, P::KT)) return GDN_ERR_LAUNCH;
    if (cudaFuncSetAttribute(chunk_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::BYTES) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    const long long grid = units(c, d) * a.splits;
    if (grid > 0x7fffffffLL) return GDN_ERR_DIMS;
    if (launch_pdl(chunk_tc_kernel<D>, dim3(static_cast<unsigned>(grid)), dim3(P::THREADS), P::BYTES, s, mq, mk, mv, a) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    return a.splits == 1 ? GDN_OK : chunk_join(a, kRows, D, true, s);
}

}  // namespace

int64_t chunk_tc_workspace(const gdn_page_cache *c, const gdn_attn_dims *d) {
    const int splits = best_splits(c, d);
    return splits == 1 ? 0 : static_cast<int64_t>(d->B) * c->Hkv * row_tiles(c, d) * splits * part_floats(kRows, c->d) * 4;
}

int chunk_tc(const gdn_page_cache *c, const gdn_attn_dims *d, ChunkArgs a, cudaStream_t s) {
    return c->d == 64 ? launch<64>(c, d, a, s) : c->d == 128 ? launch<128>(c, d, a, s) : launch<256>(c, d, a, s);
}

}  // namespace gdn
