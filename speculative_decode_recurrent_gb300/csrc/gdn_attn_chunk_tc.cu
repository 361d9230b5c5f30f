// gdn_attn_chunk_tc.cu -- attention of a chunk of new tokens over the paged cache on the tensor cores (bf16, tcgen05), for
// sm_103a.  C ABI and layouts: include/gdnattn.h.
//
// Mathematics.  As in gdn_attn_chunk.cu, with a reference m in the maximum's place: it is raised (o and l rescaled)
// only when a tile's maximum exceeds it by more than 8 in powers of two, so weights stay below 2^8 and most tiles
// rescale nothing.  Weights enter the second product as one bf16 term: each is off by 2^-8 of itself at most, unbiased,
// which over a row's keys adds about as much as rounding the output does: 2.1e-3 to 2.3e-3 of the outputs, of which their own rounding is 1.7e-3.
// With GDN_FLAG_TWO_TERMS it is two terms (2^-17), as in the verify of drafts, and what is left is the outputs' rounding; the second
// product, half of all the work here, is then twice as long (prompts 215 us on the device instead of 161, 256 tokens after 60001 122
// instead of 93, 64 prompts of 256 tokens 60 instead of 49).  l is the sum of the weights in fp32.
//
// What bounds it: the MMAs, and shared memory with them (an MMA of 128 rows by 128 keys takes 63 cycles with 64 of reads, one of
// 64 keys 47 instead of 32).  A CTA has two tiles of 128 rows (row r = t G + g: tokens times the query heads of a key
// head) whose softmaxes and products overlap.  Tiles of 128 keys leave TMEM for one score buffer of each row tile, so a
// tile's softmax, its weights' product and the next scores follow one another: a pair's tiles take some 2500 cycles, their MMAs
// 2000.  (Tiles of 64 keys in two buffers: 2 x 1770.)  4 sequences of 4096 tokens after 16384: 1.46 ms, 1690 TFLOP/s; 4 prompts of up
// to 4096 tokens 171 us; 256 tokens after 60001 (16 query heads, 2 key heads of 128) 97 us.  Head dims of 64: 133 and 77 us (0.43 of the
// peak: half the products a score, for the same softmax), of 256: 459 and 268 us (0.5: scores formed twice, once for each half of the values).
//
// Roles.  Two groups of 256 threads, two per row (each half of a tile's keys; the scores of a row are in registers), and
// for each group a warp that issues: O += P_i V_i, then the scores of the next tile into the buffer that held P_i (the weights
// go over the scores in TMEM and are the A operand from there; the order of issue keeps the two apart).  A warp each loads
// keys and values (TMA through the block table).  d 256: the sums of 256 columns of two row tiles leave no room for
// scores, so a CTA takes 128 columns of the values and both halves form the scores; its tiles of 64 keys (shared
// memory holds no larger ones) have two buffers.
//
// Work.  A unit is (pair of row tiles, key head, sequence, part of the keys); the longest come first.  A CTA takes over the
// units of CTAs of the grid that have not begun (cluster launch control), so that a unit's keys, values and queries are loaded and
// its first scores formed while the rows of the one before are scaled and written: with a CTA for each unit its beginning and
// end cost 8 us each time (64 prompts of 256 tokens 73 us, without 46, which is 49 with the look at the values; 4 of 4096 211 and 187).  Keys are cut
// into parts where the pairs alone would leave SMs without work (best_splits), joined by chunk_tc_join_kernel.
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
    static constexpr int OFF_BAR = OFF_XCH + 512 * 4, BYTES = OFF_BAR + 384 + 176;
    static constexpr int MMA_WARP = 0, LOAD_WARP = 2, ROW_WARP = 4, WARPS = 20, THREADS = WARPS * 32;
    static constexpr int OFF_SLOT = OFF_BAR + 352, OFF_NEXT = OFF_SLOT + 16, OFF_UNIT = OFF_BAR + 384;      // TMEM address and abort; the next CTA's index; units
    static constexpr int COL_S = 0, COL_O = 2 * NB * KT;       // TMEM: the score buffers of each row tile, then their sums
    static_assert(COL_O + 2 * DV <= 512 && BYTES <= 227 * 1024, "plan");
};

// 32 bytes, in one store where the address allows it.
__device__ __forceinline__ void store_32(void *dst, const uint32_t (&x)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
                     "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]) : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(x[4], x[5], x[6], x[7]);
    }
}

// Bit 15 or 31 where a half of x is an infinite or NaN bf16 number (all bits of its exponent); those halves as a mask.
__device__ __forceinline__ uint32_t odd_bits(uint32_t x) { return (x & 0x7f807f80u) + 0x00800080u; }
__device__ __forceinline__ uint32_t odd_halves(uint32_t x) {
    const uint32_t e = x & 0x7f807f80u;
    return ((e & 0xffffu) == 0x7f80u ? 0xffffu : 0u) | (e >= 0x7f800000u ? 0xffff0000u : 0u);
}

template <bool X> struct Flag {
    static constexpr bool value = X;
};
// What the warps need to know of a unit of work.
struct Unit {
    int h, b, half, part, rt0, slot, len, n;
    int live[2], tiles[2];                          // of each row tile: rows in use; tiles of keys that this part has of it
    int keys[2];                                    // and its last row's keys from this part's first on
    int first, count;                               // this part's tiles of keys
    int before[2], all;                             // tiles of the CTA's units before: each group's, both groups' (so, of values)
    int sums[2];                                    // of those units, how many had tiles of each group
    int stop;
};
static_assert(sizeof(Unit) == 88, "unit");

// NaN in the sums (N columns from t_o and column c0 on) of a row where it sees an infinite or NaN value of the tokens [j0, j1), which its
// products have met as 0.  A rare path: the values are read from memory again.
template <int N>
__device__ __noinline__ void spoil_sums(const ChunkArgs &a, int slot, int h, int c0, int d, int j0, int j1, uint32_t t_o) {
    unsigned long long odd = 0ull;
    const int32_t *tab = a.s.table + static_cast<size_t>(slot) * a.s.max_pages;
    for (int j = j0; j < j1; ++j) {
        const int id = __ldg(tab + (j >> a.s.page_shift));
        if (id < 0 || id >= a.s.n_page) continue;
        const size_t row = ((static_cast<size_t>(id) * a.s.Hkv + h) << a.s.page_shift) + (j & ((1 << a.s.page_shift) - 1));
        const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.v) + row * d + c0);
#pragma unroll 4
        for (int c = 0; c < N / 8; ++c) {
            const uint4 x = __ldg(v + c);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t y = odd_halves(w[k]);
                m |= ((y & 1u) | (y >> 30 & 2u)) << 2 * k;
            }
            odd |= static_cast<unsigned long long>(m) << 8 * c;
        }
    }
    for (int c = 0; c < N; c += 8) {
        const uint32_t m = static_cast<uint32_t>(odd >> c) & 0xffu;
        if (!__any_sync(0xffffffffu, m != 0)) continue;
        uint32_t o[8];
        tmem_load8(t_o + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (m >> k & 1u) o[k] = 0x7fffffffu;
        tmem_store8(t_o + c, o);
    }
    tmem_wait_st();
}

// The index of a CTA of the grid that has not begun, which this one takes over: asked for, and read.
__device__ __forceinline__ void ask_next(uint32_t at, uint64_t *bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(at), "r"(saddr(bar)) : "memory");
}
__device__ __forceinline__ int read_next(uint32_t at) {
    int x;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\tld.shared.b128 r, [%1];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tmov.b32 %0, -1;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, r;\n\t}"
        : "=r"(x) : "r"(at) : "memory");
    return x;
}

template <int D, bool TWO>                          // TWO: weights in two bf16 terms
__global__ void __launch_bounds__(Plan<D>::THREADS, 1)
chunk_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ ChunkArgs a)
{
    using P = Plan<D>;
    constexpr int DV = P::DV, KT = P::KT, HALVES = D / DV;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.G, Hkv = a.s.Hkv;
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + P::OFF_BAR), *k_empty = k_full + P::NK, *v_full = k_empty + P::NK,
             *v_empty = v_full + P::NV, *q_full = v_empty + P::NV, *q_empty = q_full + 1, *s_full = q_empty + 1, *p_full = s_full + 4,
             *o_done = p_full + 4, *o_last = o_done + 2, *o_free = o_last + 2, *turn = o_free + 2, *drain = turn + 2,     // s_full, p_full [group][buffer]; then [group]
             *u_full = drain + 2, *u_empty = u_full + 2, *asked_next = u_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + P::OFF_SLOT);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *odd_values = abort + 1;           // [2]: the last unit in the slot (its number plus 1) of whose values infinities or NaN have been zeroed
    Unit *units = reinterpret_cast<Unit *>(smem + P::OFF_UNIT);
    static_assert((2 * P::NK + 2 * P::NV + 25) * 8 <= 352, "barriers");
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
        mbar_init(q_empty, 2);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&o_done[i], 1);
            mbar_init(&o_last[i], 1);
            mbar_init(&o_free[i], 8);
            mbar_init(&turn[i], 1);
            mbar_init(&drain[i], 1);
            mbar_init(&u_full[i], 1);
            mbar_init(&u_empty[i], P::WARPS - 1);   // every warp but the one that fills it
        }
        mbar_init(asked_next, 1);
        *abort = (a.flags & GDN_FLAG_TEST_EXPIRE) != 0;
        odd_values[0] = odd_values[1] = 0;
        fence_mbar_init();
    }
    if (warp == P::MMA_WARP) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && *abort) atomicOr(a.s.status, kStatusTimeout);
    pdl_wait();
    pdl_release();
    const uint32_t tmem = *tmem_slot;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return warp_wait(bar, parity, abort, a.s.status); };
    // Unit u of this CTA, in slot u % 2, which its warps give back when they are through with it
    auto next_unit = [&](int u) { return wait(&u_full[u & 1], (u >> 1) & 1); };
    auto end_unit = [&](int u) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&u_empty[u & 1]);
    };
    if (warp == P::LOAD_WARP || warp == P::LOAD_WARP + 1) {
        // ------------------------------------------------------ loads: keys, values
        const bool vals = warp != P::LOAD_WARP;
        const CUtensorMap *map = vals ? &tm_v : &tm_k;
        uint64_t *full = vals ? v_full : k_full, *empty = vals ? v_empty : k_empty;
        const int ns = vals ? P::NV : P::NK, bytes = vals ? P::V_BYTES : P::K_BYTES, atoms = vals ? P::VA : P::QA;
        const int shift = a.s.page_shift;
        const int rows = min(1 << shift, KT), per = KT / rows;        // rows of a copy, copies of a tile (and atom)
        uint8_t *base = smem + (vals ? P::OFF_V : P::OFF_K);
        int st = 0, round = 0, loaded = 0, queries = 0;               // stages and rounds, tiles loaded; units with keys (so with queries)
        // The values' warp also decides on the units: the CTA's own, then those of CTAs that have not begun, asked for while
        // a unit's values are on their way and passed on once they have been requested.
        int asked = 0, before[2] = {0, 0}, sums[2] = {0, 0};
        auto unit_of = [&](int id, Unit &x) {       // ((pair, part, half), sequence, key head), long ones first; false: a bad sequence
            int i = id;
            x.h = i % Hkv;
            i /= Hkv;
            x.b = i % a.s.B;
            i /= a.s.B;
            x.half = i % HALVES;
            i /= HALVES;
            x.part = i % a.splits;
            x.rt0 = ((a.row_tiles + 1) / 2 - 1 - i / a.splits) * 2;
            const Seq sq = load_seq<true>(a.s, x.b);
            if (sq.bad) {
                if (lane == 0 && id == x.b * Hkv) atomicOr(a.s.status, sq.bad);
                return false;
            }
            x.slot = sq.slot;
            x.len = sq.len;
            x.n = sq.n;
            // a tile's rows in use and the keys that its last one sees; nothing of a tile without rows in use
            int tiles[2], end;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int tg = (x.rt0 + g) * a.tpt, n = min(a.tpt, sq.n - tg);
                x.live[g] = max(n, 0) * G;
                x.keys[g] = sq.len + tg + n;
                tiles[g] = n > 0 ? (x.keys[g] + KT - 1) / KT : 0;
            }
            part_range(max(tiles[0], tiles[1]), x.part, a.splits, x.first, end);
            x.count = end - x.first;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                x.tiles[g] = max(0, min(end, tiles[g]) - x.first);
                x.keys[g] -= x.first * KT;
            }
            x.stop = 0;
            return true;
        };
        auto ask = [&]() {
            if (lane == 0) {
                mbar_expect_tx(asked_next, 16);
                ask_next(saddr(smem) + P::OFF_NEXT, asked_next);
            }
            __syncwarp();
        };
        // Passes on unit u: of this CTA's index (u 0) or of the one that was asked for; stop where there is none.
        auto pass_on = [&](int u, Unit &x) {
            int id = blockIdx.x;
            for (bool first = u == 0;; first = false) {
                if (!first) {
                    if (!wait(asked_next, asked & 1)) {
                        if (!mbar_wait(asked_next, asked & 1) && lane == 0) atomicOr(a.s.status, GDN_STATUS_DRAIN);
                        return false;
                    }
                    ++asked;
                    id = read_next(saddr(smem) + P::OFF_NEXT);
                    __syncwarp();
                    fence_proxy_async();
                }
                x.stop = id < 0;
                if (id < 0 || unit_of(id, x)) break;
                ask();
            }
            if (u >= 2 && !wait(&u_empty[u & 1], ((u >> 1) - 1) & 1)) return false;
            if (lane == 0) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    x.before[g] = before[g];
                    x.sums[g] = sums[g];
                }
                x.all = loaded;
                units[u & 1] = x;
                mbar_arrive(&u_full[u & 1]);
            }
            __syncwarp();
            return true;
        };
        bool ok = !*abort;
        for (int u = 0; ok; ++u) {
            Unit x;
            if (vals ? !pass_on(u, x) : !next_unit(u)) break;
            if (!vals) x = units[u & 1];
            if (x.stop) break;
            if (vals) {
                ask();
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    before[g] += x.tiles[g];
                    sums[g] += x.tiles[g] > 0;
                }
            }
            const int t0 = x.rt0 * a.tpt, total = x.len + x.n;        // tokens whose keys and values are there
            if (!vals && x.count > 0) {             // the queries of both row tiles, when the last scores of those before are done
                ok = queries == 0 || wait(q_empty, (queries - 1) & 1);
                if (!ok) break;
                if (elect_one()) {
                    const int two = x.live[1] > 0 ? 2 : 1;
                    mbar_expect_tx(q_full, two * P::QA * a.tpt * G * 128);
                    for (int g = 0; g < two; ++g)
                        for (int c = 0; c < P::QA; ++c)
                            tma_load_3d(smem + g * P::Q_BYTES + c * (kRows * 128), &tm_q, c * 64, x.h * G, x.b * a.s.T + t0 + g * a.tpt, q_full);
                }
                __syncwarp();
                ++queries;
            }
            const int x0 = vals ? x.half * DV : 0;
            const int32_t *tab = a.s.table + static_cast<size_t>(x.slot) * a.s.max_pages;
            int ids = 0, base_p = -1;               // block-table entries base_p + lane
            for (int i = 0; i < x.count; ++i, ++loaded) {
                ok = !*abort && (round == 0 || wait(&empty[st], (round - 1) & 1));
                if (!ok) break;
                const int j0 = (x.first + i) * KT, p0 = j0 >> shift;
                if (base_p < 0 || p0 + per > base_p + 32) {           // (a tile's entries, 8 at most, lie in one batch)
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
                const int here = min(per, (total - j0 + rows - 1) / rows);     // copies that hold tokens
                const bool one = elect_one();
                if (one) mbar_expect_tx(&full[st], here * rows * 128 * atoms);
                for (int c = 0; c < here; ++c) {
                    const int row = ((__shfl_sync(0xffffffffu, ids, p0 + c - base_p) * Hkv + x.h) << shift) + ((j0 + c * rows) & ((1 << shift) - 1));
                    if (one)
                        for (int y = 0; y < atoms; ++y)
                            tma_load_2d(base + st * bytes + y * (KT * 128) + c * rows * 128, map, x0 + y * 64, row, &full[st]);
                    __syncwarp();
                }
                if (++st == ns) st = 0, ++round;
            }
            if (!vals) end_unit(u);
            else if (!ok && !mbar_wait(asked_next, asked & 1) && lane == 0) atomicOr(a.s.status, GDN_STATUS_DRAIN);
        }
        {                                           // copies in flight end before the CTA does (their users may have given up)
            bool done = queries == 0 || mbar_wait(q_full, (queries - 1) & 1);
            for (int y = max(0, loaded - ns); y < loaded; ++y) done = done && mbar_wait(&full[y % ns], (y / ns) & 1);
            if (!done && lane == 0) atomicOr(a.s.status, GDN_STATUS_DRAIN);
        }
    } else if (warp < P::LOAD_WARP) {
        // ------------------------------------------------------ MMAs of a group
        // Issuing holds a warp up until its MMAs have nearly run, and each wait on a barrier costs it some 300 cycles, which
        // one warp for both groups left the tensor cores idle.  Each group's warp waits while the other's MMAs
        // run; a group's last product and its next scores go in one piece, in turns (`turn`), so that the groups' softmaxes
        // stay half a period apart (without turns they fall into step, and both wait for the tensor cores at once).
        const int g = __shfl_sync(0xffffffffu, warp - P::MMA_WARP, 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), t_s = tm + P::COL_S + g * (P::NB * KT), t_o = tm + P::COL_O + g * DV;
        const uint64_t dq = desc_sw128(saddr(smem) + g * P::Q_BYTES), dk0 = desc_sw128(saddr(smem) + P::OFF_K),
                       dv0 = desc_mn_sw128(saddr(smem) + P::OFF_V, KT * 128);
        constexpr uint32_t idS = idesc_mn(1, kRows, KT), idO = idesc_mn(1, kRows, DV) | kIdescMnMajorB;
        const uint32_t one = elect_one();
        int ks = 0, kr = 0, vs = 0, vr = 0;         // stages of the next keys and values, and their rounds
        bool issued = false;
        int before = 0, all = 0, queries = 0, sums = 0;       // tiles of the units before (this group's; both groups'), units with keys, with sums of this group
        auto scores = [&](int i) {                  // Q K^T of tile i (since the beginning), whose keys are there, into buffer i % NB
            const uint64_t kd = desc_add(dk0, ks * P::K_BYTES);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                mma_bf16_on(one, t_s + i % P::NB * KT, desc_add(dq, (k >> 2) * (kRows * 128) + (k & 3) * 32),
                            desc_add(kd, (k >> 2) * (KT * 128) + (k & 3) * 32), idS, k > 0);
            mma_commit_on(one, &s_full[2 * g + i % P::NB]);
            issued = true;
        };
        bool ok = true, ended = false;
        for (int u = 0; ok && next_unit(u); ++u) {
            const int stop = __shfl_sync(0xffffffffu, units[u & 1].stop, 0), count = __shfl_sync(0xffffffffu, units[u & 1].count, 0),
                      n = __shfl_sync(0xffffffffu, units[u & 1].tiles[g], 0), keys = __shfl_sync(0xffffffffu, units[u & 1].keys[g], 0);
            if (stop) {
                ended = true;
                break;
            }
            // A tile that only the other group sees is passed on once it is there (an arrival before that would count for
            // the round before).
            auto free_keys = [&](int i) {
                if (i < n) mma_commit_on(one, &k_empty[ks]);
                else if (lane == 0) mbar_arrive(&k_empty[ks]);
                if (i == n - 1) mma_commit_on(one, q_empty);          // the last scores
                if (++ks == P::NK) ks = 0, ++kr;
            };
            ok = count == 0 || wait(q_full, queries & 1);
            if (ok && count > 0 && n == 0 && lane == 0) mbar_arrive(q_empty);
            __syncwarp();
            for (int i = 0; ok && i < min(count, P::NB); ++i) {
                ok = wait(&k_full[ks], kr & 1);
                if (!ok) break;
                tc_fence_after();
                if (i < n) scores(before + i);
                free_keys(i);
                __syncwarp();
            }
            if (n > 0 && sums > 0) ok = ok && wait(&o_free[g], (sums - 1) & 1);       // the last unit's sums have been read
            for (int i = 0; ok && i < count; ++i) {
                const int j = i + P::NB;            // the tile whose scores follow
                ok = wait(&v_full[vs], vr & 1) && (j >= count || wait(&k_full[ks], kr & 1));
                const uint64_t vd = desc_add(dv0, vs * P::V_BYTES);
                const int at = before + i;
                if (i < n) ok = ok && wait(&p_full[2 * g + at % P::NB], (at / P::NB) & 1);
                ok = ok && ((g == 0 && all + i == 0) || wait(&turn[g], (g ? all + i : all + i - 1) & 1));
                if (!ok) break;
                tc_fence_after();
                if (i < n) {
                    const uint32_t t_p = t_s + at % P::NB * KT;       // O += P_i V_i, the second terms (KT / 2 columns on) first
                    if (P::NB > 1 || keys >= (i + 1) * KT) {
#pragma unroll
                        for (int k = TWO ? -KT / 16 : 0; k < KT / 16; ++k) {
                            const int at_k = k & (KT / 16 - 1);
                            mma_bf16_ts_on(one, t_o, t_p + (k < 0 ? KT / 2 : 0) + at_k * 8, desc_add(vd, at_k * 2048), idO, i > 0 || k != (TWO ? -KT / 16 : 0));
                        }
                    } else {                        // no further than the group's last row sees
                        const int some = __shfl_sync(0xffffffffu, (keys - i * KT + 15) / 16, 0);
#pragma unroll 1
                        for (int k = 0; k < some; ++k) {
                            if (TWO) mma_bf16_ts_on(one, t_o, t_p + KT / 2 + k * 8, desc_add(vd, k * 2048), idO, i > 0 || k > 0);
                            mma_bf16_ts_on(one, t_o, t_p + k * 8, desc_add(vd, k * 2048), idO, TWO || i > 0 || k > 0);
                        }
                    }
                }
                if (i < n) {
                    mma_commit_on(one, &o_done[g]);
                    if (i == n - 1) mma_commit_on(one, &o_last[g]);
                    mma_commit_on(one, &v_empty[vs]);
                } else if (lane == 0) {
                    mbar_arrive(&v_empty[vs]);
                }
                if (++vs == P::NV) vs = 0, ++vr;
                if (j < n) scores(before + j);
                if (lane == 0) mbar_arrive(&turn[g ^ 1]);
                if (j < count) free_keys(j);
                __syncwarp();
            }
            before += n;
            all += count;
            queries += count > 0;
            sums += n > 0;
            end_unit(u);
        }
        if (!ended && issued) {                     // MMAs in flight end before their memory is given back
            mma_commit_on(one, &drain[g]);
            if (!mbar_wait(&drain[g], 0) && lane == 0) atomicOr(a.s.status, GDN_STATUS_DRAIN);
        }
    } else {
        // ------------------------------------------------------ rows
        // Thread (group, half of a tile's keys and of the output's columns, row).  An expired wait only stops the waiting
        // (a thread that left would leave its pair at a barrier).
        const int rw = warp - P::ROW_WARP, rt = tid - P::ROW_WARP * 32;
        const int g = rw >> 3, kh = (rw >> 2) & 1, r = (warp & 3) * 32 + lane, pair_id = 1 + g * 4 + (warp & 3);
        constexpr int KH = KT / 2, DH = DV / 2;
        float *xch = reinterpret_cast<float *>(smem + P::OFF_XCH);
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s0 = tmem + lanes + P::COL_S + g * (P::NB * KT);
        auto sums = [&]() { return *const_cast<volatile uint32_t *>(tmem_slot) + lanes + P::COL_O + g * DV + kh * DH; };      // (as w)
        for (int u = 0;; ++u) {
        if (pair_any(pair_id, !next_unit(u))) break;                  // (both warps of a pair go on or neither)
        const Unit &w = units[u & 1];               // (read again where it is needed: registers are short)
        if (w.stop) break;
        // Tiles of this group since the beginning, of which those below `plain` are seen by every row, all of them in use.
        const int end = w.before[g] + w.tiles[g];
        const int whole = (w.len + (w.rt0 + g) * a.tpt + 1) / KT - w.first + w.before[g];       // (tiles of tokens that they all see)
        const int plain = w.live[g] == kRows ? whole : 0;
        float m = -INFINITY, l = 0.f;               // m: the same in both threads of a row; l: of this one's keys
        bool ok = true;
        // (before the scores, while the warps would wait for them; for tiles in two buffers, whose scores are there, behind them)
        constexpr bool LATE = P::NB > 1;
        auto clean = [&](auto edge, int at) {
            if (!edge.value || at < whole) return;
            // A weight of 0 must not meet an infinity or NaN.  The product of this group takes the tile's keys up to its last row's, in
            // sixteens; of those, values past the last token, which hold anything, become 0, and so do infinite and NaN ones of tokens that
            // some of its rows do not see.  The rows that do, of either group, get NaN at the unit's end: the second group's product of a tile
            // comes after the first one's, so it meets the same zeros each time.  (Both: 1 % of the prompts' time, 4 % of 256 tokens'.)
            const int i = at - w.before[g], j0 = (w.first + i) * KT, tile = w.all + i, vst = tile % P::NV;
            const int lo = max(0, w.len + (w.rt0 + g) * a.tpt + 1 - j0), vecs = ((LATE ? KT : min(KT, (w.keys[g] - i * KT + 15) & ~15)) - lo) * (DV / 8);
            if (vecs > 0) {
                const int used = w.len + w.n - j0;
                ok = wait(&v_full[vst], (tile / P::NV) & 1) && ok;
                for (int e0 = rt & 255; e0 < vecs; e0 += 512) {
                    uint4 y[2], *at_v[2];
                    bool past = false;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int e = min(e0 + 256 * k, vecs - 1), row = lo + e / (DV / 8), c = e % (DV / 8);
                        at_v[k] = reinterpret_cast<uint4 *>(smem + P::OFF_V + vst * P::V_BYTES + (c >> 3) * (KT * 128) + sw128(row, c & 7));
                        y[k] = *at_v[k];
                        if (row >= used) {
                            past = true;
                            y[k] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    const uint32_t odd = (odd_bits(y[0].x) | odd_bits(y[0].y) | odd_bits(y[0].z) | odd_bits(y[0].w) | odd_bits(y[1].x) |
                                          odd_bits(y[1].y) | odd_bits(y[1].z) | odd_bits(y[1].w)) & 0x80008000u;
                    if (past || odd) {
                        if (odd) odd_values[u & 1] = u + 1;
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            *at_v[k] = make_uint4(y[k].x & ~odd_halves(y[k].x), y[k].y & ~odd_halves(y[k].y), y[k].z & ~odd_halves(y[k].z),
                                                  y[k].w & ~odd_halves(y[k].w));
                        fence_proxy_async();
                    }
                }
            }
        };
        // (in two copies: the tiles that every row sees have nothing of the others' masks)
        auto tile_of = [&](auto edge, int at) {
            if constexpr (!LATE) clean(edge, at);
            const uint32_t t_s = t_s0 + at % P::NB * KT;
            ok = wait(&s_full[2 * g + at % P::NB], (at / P::NB) & 1) && ok;
            tc_fence_after();
            uint32_t x[KH / 32][32];
#pragma unroll
            for (int c = 0; c < KH / 32; ++c) tmem_ld32(t_s + kh * KH + 32 * c, x[c]);
            tmem_wait_ld();
            if constexpr (edge.value) {
                const int j0 = (w.first + at - w.before[g]) * KT;
                const int seen = (r < w.live[g] ? w.len + (w.rt0 + g) * a.tpt + r / G + 1 : 0) - j0 - kh * KH;       // keys that this row sees
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
                if (at > w.before[g]) {                   // the sums so far: their last product must be done (the one before it
                                                    // is, as its weights' buffer holds these scores)
                    ok = wait(&o_done[g], (at - 1) & 1) && ok;
                    tc_fence_after();
                    const uint32_t t_o = sums();
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
                [[maybe_unused]] uint32_t rest[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float2 e = fma2(make_float2(__uint_as_float(x[c][2 * k]), __uint_as_float(x[c][2 * k + 1])), sc, mm);
                    e = make_float2(ex2(e.x), ex2(e.y));
                    sum[k & 1] = add2(sum[k & 1], e);
                    const __nv_bfloat162 w = __floats2bfloat162_rn(e.x, e.y);
                    p[k] = *reinterpret_cast<const uint32_t *>(&w);
                    if constexpr (TWO) {
                        const float2 r = fma2(make_float2(__uint_as_float(p[k] << 16), __uint_as_float(p[k] & 0xffff0000u)), make_float2(-1.f, -1.f), e);
                        const __nv_bfloat162 second = __floats2bfloat162_rn(r.x, r.y);
                        rest[k] = *reinterpret_cast<const uint32_t *>(&second);
                    }
                }
                tmem_st16(t_s + kh * (KH / 2) + 16 * c, p);
                if constexpr (TWO) tmem_st16(t_s + KT / 2 + kh * (KH / 2) + 16 * c, rest);
            }
            l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
            if constexpr (LATE) clean(edge, at);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * g + at % P::NB]);
        };
        int at = w.before[g];
        for (; at < min(plain, end); ++at) tile_of(Flag<false>{}, at);
        for (; at < end; ++at) tile_of(Flag<true>{}, at);
        const int n = w.tiles[g];
        const uint32_t t_o = sums();
        if (n > 0) {                                // (by a barrier of its own: o_done may be a phase or two behind)
            ok = wait(&o_last[g], w.sums[g] & 1) && ok;
            tc_fence_after();
            if (__any_sync(0xffffffffu, odd_values[u & 1] == u + 1) && ok)
                spoil_sums<DH>(a, w.slot, w.h, w.half * DV + kh * DH, D, max(w.first * KT, w.len + w.rt0 * a.tpt + 1),
                               r < w.live[g] ? min((w.first + n) * KT, w.len + (w.rt0 + g) * a.tpt + r / G + 1) : 0, t_o);
        }
        xch[rt] = l;
        bar_sync(pair_id, 64);
        l += xch[rt ^ 128];
        const int h = w.h, b = w.b, half = w.half, part = w.part, rt0 = w.rt0, tg = (rt0 + g) * a.tpt, in_use = w.live[g];
        const bool used = r < in_use;
        // row r of tile g is token tg + r / G, head h G + r % G
        auto row_at = [&](int r) { return (static_cast<size_t>(b) * a.s.T + tg + r / G) * a.Hq + h * G + r % G; };
        const int rows = min(a.tpt, a.s.T - tg) * G, c0 = half * DV + kh * DH;          // this thread's first output column
        if (ok && a.splits > 1 && in_use > 0) {
            const size_t unit = (static_cast<size_t>(b) * Hkv + h) * a.row_tiles + rt0 + g;
            float *dst = a.ws + (unit * a.splits + part) * part_floats(kRows, D) + r;
            if (n > 0)
#pragma unroll 1
                for (int c = 0; c < DH; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(t_o + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; ++k) dst[(c0 + c + k) * kRows] = __uint_as_float(o[k]);
                }
            if (half == 0 && kh == 0) {
                dst[D * kRows] = m;
                dst[(D + 1) * kRows] = l;
            }
        } else if (ok && (a.splits == 1 || part == 0)) {              // (the join passes over a tile without rows in use)
            const float inv = used ? 1.f / l : 0.f;
            constexpr int UNITS = DH / 16;          // of 16 columns, 32 bytes
            uint32_t y[UNITS][8];
#pragma unroll
            for (int c = 0; c < DH; c += 32) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld32(t_o + c, o);
                    tmem_wait_ld();
                } else {                            // (not the last unit's: those would stay in registers all along)
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0u;
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const __nv_bfloat162 z = __floats2bfloat162_rn(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
                    y[c / 16 + (k >> 3)][k & 7] = used ? *reinterpret_cast<const uint32_t *>(&z) : 0u;
                }
            }
            // Neighbouring lanes exchange, so that a store has whole lines of fewer rows: a row a lane costs a cycle for each of them
            // (4100 for a pair's tiles by 16 bytes, and the next unit's first wait stood behind them).
#pragma unroll
            for (int e = 1; e < UNITS; e <<= 1)
#pragma unroll
                for (int c = 0; c < UNITS; ++c)
                    if ((c & e) == 0)
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const bool up = (lane & e) != 0;
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? y[c][k] : y[c | e][k], e);
                            y[c][k] = up ? got : y[c][k];
                            y[c | e][k] = up ? y[c | e][k] : got;
                        }
            const int first_row = r & ~(UNITS - 1);
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + c0 + 16 * (lane & (UNITS - 1));
#pragma unroll
            for (int c = 0; c < UNITS; ++c)
                if (first_row + c < rows) store_32(out + row_at(first_row + c) * D, y[c], (reinterpret_cast<uintptr_t>(a.out) & 31) == 0);
            const size_t at = r < rows ? row_at(r) : 0;
            if (a.lse && half == 0 && kh == 0 && r < rows) a.lse[at] = used ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
        }
        tc_fence_before();
        __syncwarp();
        if (n > 0 && lane == 0) mbar_arrive(&o_free[g]);              // the sums have been read
        end_unit(u);
        if (pair_any(pair_id, !ok)) break;
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == P::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The parts of a unit of 128 rows, joined: o [d][128 rows], m [128], l [128] each.  A thread has a row's 8 columns, of four parts at
// a time: what bounds it is the way to L2 (19 MB of 9 parts for 256 tokens of 16 heads of 128).
template <int D>
__global__ void __launch_bounds__(D * 4) chunk_tc_join_kernel(const ChunkArgs a)
{
    constexpr int Q = kRows / 32, C = 8, SOME = 4;
    const int lane = threadIdx.x & 31, c0 = threadIdx.x / 32 * C, r = blockIdx.x % Q * 32 + lane, rt = blockIdx.x / Q, h = blockIdx.y, b = blockIdx.z;
    pdl_wait();
    pdl_release();
    const Seq sq = load_seq<true>(a.s, b);
    const int t0 = rt * a.tpt, rows = min(a.tpt, a.s.T - t0) * a.G, live = min(a.tpt, sq.n - t0) * a.G;
    if (sq.bad || live <= 0) return;                // (a tile without rows in use has been written already)
    const size_t unit = (static_cast<size_t>(b) * a.s.Hkv + h) * a.row_tiles + rt, step = part_floats(kRows, D);
    const float *w = a.ws + unit * a.splits * step + r;
    float m = -INFINITY, l = 0.f, o[C];
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = 0.f;
    for (int i0 = 0; i0 < a.splits; i0 += SOME) {
        float x[SOME][C], mi[SOME], li[SOME];
#pragma unroll
        for (int i = 0; i < SOME; ++i) {            // (past the last part: the last one again, without weight)
            const float *p = w + min(i0 + i, a.splits - 1) * step;
            mi[i] = p[D * kRows];
            li[i] = p[(D + 1) * kRows];
#pragma unroll
            for (int c = 0; c < C; ++c) x[i][c] = p[(c0 + c) * kRows];         // (not written by a part without keys of this row's tile)
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < SOME; ++i) {
            if (i0 + i >= a.splits) li[i] = 0.f;
            if (li[i] != 0.f) top = fmaxf(top, mi[i]);
        }
        const float ref = top == -INFINITY ? 0.f : top, fix = ex2(m - ref);
        m = top;
        l *= fix;
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] *= fix;
#pragma unroll
        for (int i = 0; i < SOME; ++i) {
            const float f = ex2(mi[i] - ref);
            if (li[i] != 0.f) {
                l = fmaf(f, li[i], l);
#pragma unroll
                for (int c = 0; c < C; ++c) o[c] = fmaf(f, x[i][c], o[c]);
            }
        }
    }
    if (r >= rows) return;
    const size_t row = (static_cast<size_t>(b) * a.s.T + t0 + r / a.G) * a.Hq + h * a.G + r % a.G;
    const float inv = 1.f / l;
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 z = __floats2bfloat162_rn(o[2 * k] * inv, o[2 * k + 1] * inv);
        y[k] = r < live ? *reinterpret_cast<const uint32_t *>(&z) : 0u;
    }
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + row * D + c0) = make_uint4(y[0], y[1], y[2], y[3]);
    if (a.lse && c0 == 0) a.lse[row] = r < live ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
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
// Parts of the key axis, at least 512 keys each, as far as a sequence can be long: the fewest tiles' times (of 128 keys, about
// 2400 cycles) until the last CTA is through.  A unit costs 2.5 of them beside its own tiles, a part's way through memory and the
// join 0.064 (divided among the SMs already) and the join's launch 3.  Units of nearly one length come in waves; those of a prompt,
// whose length falls from the longest to nothing, fill the SMs, with half a unit at the end.  The lengths are on the device: the cache's
// capacity stands for them here, so where sequences are far shorter there are parts without keys, which cost their CTA a unit's
// 2.5 tiles and the join its loads.  The figures are of head dims of 128.
int best_splits(const gdn_page_cache *c, const gdn_attn_dims *d) {
    const long long sms = sm_count(), u = units(c, d);
    if (sms < 1 || u >= 4 * sms) return 1;
    const long long keys = static_cast<long long>(c->max_pages) * c->page;
    const double longest = keys / 128.0, shortest = keys > d->T ? (keys - d->T) / 128.0 : 0.0, mean = (longest + shortest) / 2;
    int best = 1;
    double least = 1e30;
    for (int s = 1; s <= kMaxSplits && (s == 1 || keys >= 512ll * s); ++s) {
        const double n = static_cast<double>(u) * s, own = mean / s + 2.5, top = longest / s + 2.5;
        double cost = 2 * shortest >= longest ? static_cast<double>((u * s + sms - 1) / sms) * own : n * own / sms + (n > sms ? own / 2 : 0.0);
        if (cost < top) cost = top;
        if (s > 1) cost += 3 + 0.064 * n;
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

template <int D, bool TWO>
int launch(const gdn_page_cache *c, const gdn_attn_dims *d, ChunkArgs a, cudaStream_t s) {
    using P = Plan<D>;
    constexpr auto kern = chunk_tc_kernel<D, TWO>;
    a.tpt = tile_tokens(c, d);
    a.row_tiles = row_tiles(c, d);
    a.splits = best_splits(c, d);
    CUtensorMap mq, mk, mv;
    if (!query_map(&mq, a.q, c, d, a.tpt) || !rows_map(&mk, a.k, c, P::KT) || !rows_map(&mv, a.v, c, P::KT)) return GDN_ERR_LAUNCH;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, P::BYTES) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    const long long grid = units(c, d) * a.splits;
    if (grid > 0x7fffffffLL) return GDN_ERR_DIMS;
    if (launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(P::THREADS), P::BYTES, s, mq, mk, mv, a) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    if (a.splits > 1 && launch_pdl(chunk_tc_join_kernel<D>, dim3(static_cast<unsigned>(a.row_tiles) * (kRows / 32), c->Hkv, d->B), dim3(D * 4), 0, s,
                                   a) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    return GDN_OK;
}

}  // namespace

int64_t chunk_tc_workspace(const gdn_page_cache *c, const gdn_attn_dims *d) {
    const int splits = best_splits(c, d);
    return splits == 1 ? 0 : static_cast<int64_t>(d->B) * c->Hkv * row_tiles(c, d) * splits * part_floats(kRows, c->d) * 4;
}

int chunk_tc(const gdn_page_cache *c, const gdn_attn_dims *d, ChunkArgs a, cudaStream_t s) {
    if (d->flags & GDN_FLAG_TWO_TERMS)
        return c->d == 64 ? launch<64, true>(c, d, a, s) : c->d == 128 ? launch<128, true>(c, d, a, s) : launch<256, true>(c, d, a, s);
    return c->d == 64 ? launch<64, false>(c, d, a, s) : c->d == 128 ? launch<128, false>(c, d, a, s) : launch<256, false>(c, d, a, s);
}

}  // namespace gdn
