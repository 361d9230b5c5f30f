// gdn_attn_tc.cu -- the bf16 verify of the attention layers on the tensor cores (tcgen05),
// for sm_103a.  C ABI and layouts: include/gdnattn.h.
//
// Mathematics.  For a row (draft token t, query head of the group of a key head) with scores
// s_j = scale q.k_j over the visible tokens, in powers of two (s'_j = s_j log2 e): one pass over
// the keys keeps a reference m, the sum l = sum_j 2^(s'_j - m) and o = sum_j 2^(s'_j - m) v_j;
// out = o / l, lse = (m + log2 l) ln 2.  m need not be the maximum: it is raised (o and l
// rescaled) only when a tile's maximum exceeds it by more than 8, so the weights stay below 2^8
// and most tiles rescale nothing.  The second product takes each weight as two bf16
// terms (relative 2^-17): rounded to one, 2^-8, a row of few keys would be twice as far off as
// its output's rounding alone.  Everything else is fp32.
//
// What bounds it: the keys and values are read once for all T x (Hq / Hkv) rows of a key head,
// so up to about 128 rows the kernel is bound by HBM; above, by the softmax and the MMAs.
//
// Work.  A unit is (sequence, key head, tile of 128 rows); its keys come in tiles of 64.  All
// units' tiles in a row are cut into equal shares, one per resident CTA, so ragged lengths
// balance and one long sequence fills the GPU.  A unit that one CTA covers is finished there; the
// others leave partial results (o, m, l) that a second kernel joins in a fixed order.
//
// A CTA: warp 4 loads (TMA, one copy per page and 64-column atom, through the block table), warp
// 5 issues the MMAs, warps 0-3 own a row per thread: S = Q K^T (M 128, N 64) in two TMEM buffers;
// the weights' two terms go back over S and are the A operands of O += P V straight from TMEM, with
// the value rows read MN-major as they lie.  S of the next tile is formed while the softmax of the
// present one runs.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "attn_common.h"
#include "tc_common.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kKeys = 64, kRows = 128;              // tile of keys, tile of rows
constexpr int kTcThreads = 192;
constexpr int kMaxSeqs = 512;                       // sequences of one launch (their table in shared memory)
constexpr uint32_t kIdescMnMajorB = 1u << 16;

template <int D> struct TcPlan {
    static constexpr int ATOMS = D / 64;                        // 128-byte column atoms of a row
    static constexpr int STAGE = kKeys * D * 2;                 // a tile of keys or of values
    static constexpr int NST = D == 64 ? 8 : 4;
    static constexpr int OFF_RING = kRows * D * 2;              // after the queries
    static constexpr int OFF_SEQ = OFF_RING + NST * STAGE;      // prefix (int64), slot, len, n
    static constexpr int OFF_BAR = OFF_SEQ + (kMaxSeqs + 1) * 8 + kMaxSeqs * 12 + 8;
    static constexpr int BYTES = OFF_BAR + 320;
    static constexpr int CTAS = D == 256 ? 1 : 2;               // per SM
    static constexpr int COL_O = 2 * kKeys;                     // TMEM: S in [0, 64) and [64, 128), then O
    static constexpr int TMEM_COLS = D == 256 ? 512 : 256;
    static_assert(OFF_BAR % 8 == 0, "mbarriers");
    static_assert(CTAS * (BYTES + 1024) <= 228 * 1024 && BYTES <= 227 * 1024, "shared memory");
};

struct TcArgs {
    AttnArgs a;
    int b0, nb;                 // sequences [b0, b0 + nb) of the call
    int row_tiles, rp;          // row tiles of a unit; rows of a partial result (a multiple of 32)
    int2 *desc;                 // per unit: first CTA and number of CTAs
    float *part;                // [2 grid][D + 2][rp]
};

__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// 32 consecutive columns of this thread's TMEM lane; the caller waits.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
        ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
          "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(bar)) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// ------------------------------------------------------------- the work's layout
// Tiles of one (sequence, key head): the row tiles that hold rows in use take every tile of
// keys, the others one tile without keys (their rows get zeros).
struct Shape {
    int live, dead, tiles, total;                   // total: keys
    __device__ Shape(int len, int n, int G, int row_tiles) {
        live = (n * G + kRows - 1) / kRows;
        dead = row_tiles - live;
        total = len + n;
        tiles = (total + kKeys - 1) / kKeys;        // >= 1 when live > 0
    }
    __device__ long long per_head() const { return static_cast<long long>(live) * tiles + dead; }
};

struct SeqTable {
    long long *prefix;                              // [nb + 1] tiles before each sequence
    int *slot, *len, *n;                            // [nb]
};

struct Segment {
    int b, h, rt;                                   // sequence (within the launch), key head, row tile
    int slot, len, n, total;                        // total 0: a row tile without rows in use
    int first, count, tiles;                        // tiles [first, first + count) of the unit's `tiles`
    long long unit_w;                               // the unit's first tile in the launch's order
};

// Walks a CTA's share [w, w1) unit by unit.
struct Cursor {
    long long w, w1;
    int b;
    __device__ bool next(const SeqTable &st, int G, int row_tiles, Segment &s) {
        if (w >= w1) return false;
        while (st.prefix[b + 1] <= w) ++b;
        const Shape sh(st.len[b], st.n[b], G, row_tiles);
        const long long in_b = w - st.prefix[b], per = sh.per_head();
        s.b = b;
        s.slot = st.slot[b];
        s.len = st.len[b];
        s.n = st.n[b];
        s.h = static_cast<int>(in_b / per);
        const long long r = in_b - s.h * per, live_tiles = static_cast<long long>(sh.live) * sh.tiles;
        if (r < live_tiles) {
            s.rt = static_cast<int>(r / sh.tiles);
            s.first = static_cast<int>(r - static_cast<long long>(s.rt) * sh.tiles);
            s.tiles = sh.tiles;
            s.total = sh.total;
        } else {
            s.rt = sh.live + static_cast<int>(r - live_tiles);
            s.first = 0;
            s.tiles = 1;
            s.total = 0;
        }
        s.unit_w = w - s.first;
        const long long left = w1 - w;
        s.count = left < s.tiles - s.first ? static_cast<int>(left) : s.tiles - s.first;
        w += s.count;
        return true;
    }
};

// Share c of W tiles cut into N: [c W / N, (c + 1) W / N).
__device__ __forceinline__ long long share(long long W, int N, int c) { return W / N * c + W % N * c / N; }
__device__ __forceinline__ int owner(long long W, int N, long long w) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (share(W, N, mid) <= w) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// ------------------------------------------------------------------ the kernel
template <int D>
__global__ void __launch_bounds__(kTcThreads, TcPlan<D>::CTAS)
verify_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const TcArgs ta)
{
    using P = TcPlan<D>;
    const AttnArgs &a = ta.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    if (saddr(smem_raw) & 1023u) {                  // the swizzled tiles need a 1024-byte aligned base
        if (tid == 0) atomicOr(a.s.status, kStatusTimeout);
        return;
    }
    uint8_t *sQ = smem_raw, *ring = smem_raw + P::OFF_RING;
    SeqTable st;
    st.prefix = reinterpret_cast<long long *>(smem_raw + P::OFF_SEQ);
    st.slot = reinterpret_cast<int *>(st.prefix + kMaxSeqs + 1);
    st.len = st.slot + kMaxSeqs;
    st.n = st.len + kMaxSeqs;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem_raw + P::OFF_BAR);
    uint64_t *full = bar, *empty = bar + P::NST, *s_full = bar + 2 * P::NST, *p_full = s_full + 2;
    uint64_t *o_done = p_full + 2, *q_full = o_done + 1, *rows_bar = q_full + 1, *drain = rows_bar + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    unsigned long long *odd = reinterpret_cast<unsigned long long *>(tmem_slot + 2);      // [2]
    long long *warp_sum = reinterpret_cast<long long *>(odd + 2);                         // [6]
    static_assert((2 * P::NST + 8) * 8 + 8 + 16 + 48 <= 320, "barrier area");

    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < P::NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        mbar_init(&p_full[0], 128);
        mbar_init(&p_full[1], 128);
        mbar_init(o_done, 1);
        mbar_init(q_full, 128);
        mbar_init(rows_bar, 128);
        mbar_init(drain, 1);
        *abort = 0;
        odd[0] = odd[1] = 0ull;
        fence_mbar_init();
    }
    if (warp == 5) tmem_alloc(tmem_slot, P::TMEM_COLS);
    pdl_wait();
    pdl_release();
    // ---- the sequences' table: the tiles before each
    long long before = 0;
    for (int i0 = 0; i0 < ta.nb; i0 += kTcThreads) {
        const int i = i0 + tid;
        long long mine = 0;
        if (i < ta.nb) {
            const Seq q = load_seq(a.s, ta.b0 + i);
            if (!q.bad) mine = Shape(q.len, q.n, a.G, ta.row_tiles).per_head() * a.s.Hkv;
            else if (blockIdx.x == 0) atomicOr(a.s.status, q.bad);
            st.slot[i] = q.slot;
            st.len[i] = q.len;
            st.n[i] = q.n;
        }
        long long incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        if (i0 > 0) __syncthreads();                // the sums of the round before have been read
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kTcThreads / 32; ++w) {
            if (w == warp && i < ta.nb) st.prefix[i] = before + incl - mine;
            before += warp_sum[w];
        }
    }
    if (tid == 0) st.prefix[ta.nb] = before;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const long long W = st.prefix[ta.nb];
    const int N = W < gridDim.x ? static_cast<int>(W) : gridDim.x;        // every share has a tile
    Cursor cur{0, 0, 0};
    if (static_cast<int>(blockIdx.x) < N) {
        cur.w = share(W, N, blockIdx.x);
        cur.w1 = share(W, N, blockIdx.x + 1);
        int lo = 0, hi = ta.nb - 1;                 // the last sequence that starts at or before w
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (st.prefix[mid] <= cur.w) lo = mid;
            else hi = mid - 1;
        }
        cur.b = lo;
    }
    // GDN_FLAG_TEST_EXPIRE: the wait-expiry exit, with nothing issued before it
    if (a.flags & GDN_FLAG_TEST_EXPIRE) {
        if (tid == 0) {
            *abort = 1;
            atomicOr(a.s.status, kStatusTimeout);
        }
        __syncthreads();
    }
    // A bounded wait: false when it, or another role's, expired.
    auto wait = [&](uint64_t *b, uint32_t parity) {
        for (uint32_t i = 0; i < kWaitLimit; ++i) {
            if (mbar_try_wait(b, parity)) return true;
            if (*abort) return false;
        }
        *abort = 1;
        atomicOr(a.s.status, kStatusTimeout);
        return false;
    };
    Segment s;
    uint32_t pos = 0;                               // warp 4: tiles loaded
    bool issued = false;                            // warp 5: some MMA
    if (warp == 4) {
        // ------------------------------------------------------ loads
        // Tile by tile, keys then values; a lane per (page of the tile, 64-column atom).
        const int ps = a.s.page_shift < 6 ? a.s.page_shift : 6;            // rows of a copy: 16, 32 or 64
        const int copies = (kKeys >> ps) * P::ATOMS;
        const int chunk = lane / P::ATOMS, atom = lane % P::ATOMS;
        bool ok = !*abort;
        while (ok && cur.next(st, a.G, ta.row_tiles, s)) {
            const int32_t *tab = a.s.table + static_cast<size_t>(s.slot) * a.s.max_pages;
            for (int i = 0; ok && i < s.count; ++i) {
                const int j0 = (s.first + i) * kKeys, j = j0 + (chunk << ps);
                const bool mine = lane < copies && j < s.total;
                int row = 0;
                if (mine) {
                    int id = __ldg(tab + (j >> a.s.page_shift));
                    if (id < 0 || id >= a.s.n_page) {
                        atomicOr(a.s.status, GDN_STATUS_BAD_PAGE);
                        id = 0;
                    }
                    row = ((id * a.s.Hkv + s.h) << a.s.page_shift) + (j & ((1 << a.s.page_shift) - 1));
                }
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine)) << (ps + 7);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++pos) {
                    const uint32_t stage = pos % P::NST, round = pos / P::NST;
                    if (ok && round > 0) ok = wait(&empty[stage], (round - 1) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_expect_tx(&full[stage], bytes);
                    __syncwarp();
                    if (mine)
                        tma_load_2d(ring + stage * P::STAGE + atom * (kKeys * 128) + (chunk << ps) * 128, kv ? &tm_v : &tm_k,
                                    atom * 64, row, &full[stage]);
                }
            }
        }
    } else if (warp == 5) {
        // ------------------------------------------------------ MMAs
        if (lane == 0) {
            const uint64_t dq = desc_sw128(saddr(sQ));
            const uint32_t idS = idesc_mn(1, kRows, kKeys), idO = idesc_mn(1, kRows, D) | kIdescMnMajorB;
            uint32_t g = 0, segs = 0;               // tiles and segments so far
            bool ok = !*abort;
            auto scores = [&](uint32_t t) {         // S of tile t into its buffer
                const uint32_t pos = 2 * t, stage = pos % P::NST;
                if (!wait(&full[stage], (pos / P::NST) & 1)) return false;
                tc_fence_after();
                const uint64_t dk = desc_sw128(saddr(ring + stage * P::STAGE));
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t at = (k & 3) * 32;
                    mma_bf16(tmem + (t & 1) * kKeys, desc_add(dq, (k >> 2) * (kRows * 128) + at),
                             desc_add(dk, (k >> 2) * (kKeys * 128) + at), idS, k > 0);
                }
                mma_commit(&s_full[t & 1]);
                mma_commit(&empty[stage]);
                issued = true;
                return true;
            };
            while (ok && cur.next(st, a.G, ta.row_tiles, s)) {
                ok = wait(q_full, segs++ & 1) && scores(g);
                for (int i = 0; ok && i < s.count; ++i, ++g) {
                    if (i + 1 < s.count) {
                        // the other buffer held the weights of tile g - 1: their product is done
                        if (i > 0) ok = wait(o_done, (g - 1) & 1);
                        if (ok) ok = scores(g + 1);
                        if (!ok) break;
                    }
                    const uint32_t pos = 2 * g + 1, stage = pos % P::NST;
                    ok = wait(&p_full[g & 1], (g >> 1) & 1) && wait(&full[stage], (pos / P::NST) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t dv = desc_mn_sw128(saddr(ring + stage * P::STAGE), kKeys * 128);
#pragma unroll
                    for (int k = 0; k < kKeys / 8; ++k)           // the weights' first terms, then their second
                        mma_bf16_ts(tmem + P::COL_O, tmem + (g & 1) * kKeys + k * 8, desc_add(dv, (k & 3) * 2048), idO,
                                    i > 0 || k > 0);
                    mma_commit(&empty[stage]);
                    mma_commit(o_done);
                }
            }
        }
    } else {
        // ------------------------------------------------------ rows
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        uint32_t g = 0, syncs = 0;
        bool ok = !*abort;
        // a bounded wait of a whole warp (the TMEM loads and stores take all lanes), and one for
        // all 128 rows
        auto wait_warp = [&](uint64_t *b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };
        auto rows_sync = [&]() {
            mbar_arrive(rows_bar);
            return wait_warp(rows_bar, syncs++ & 1);
        };
        while (ok && cur.next(st, a.G, ta.row_tiles, s)) {
            const int r0 = s.rt * kRows, rows = a.s.T * a.G;
            const int b = ta.b0 + s.b;
            {                                       // the unit's queries, rows not in use zero
                constexpr int VECS = D / 8;
#pragma unroll 8
                for (int i = 0; i < VECS; ++i) {
                    const int x = i * 128 + tid, r = x / VECS, c = x % VECS;
                    const int t = (r0 + r) / a.G, qh = (r0 + r) - t * a.G;
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (r0 + r < rows && t < s.n)
                        v = __ldg(reinterpret_cast<const uint4 *>(
                                      static_cast<const __nv_bfloat16 *>(a.q) +
                                      ((static_cast<size_t>(b) * a.s.T + t) * a.Hq + s.h * a.G + qh) * D) + c);
                    *reinterpret_cast<uint4 *>(sQ + (c >> 3) * (kRows * 128) + sw128(r, c & 7)) = v;
                }
                fence_proxy_async();
                mbar_arrive(q_full);
            }
            const int row = r0 + tid, t = row / a.G;
            const bool used = row < rows && t < s.n;
            const bool warp_live = __any_sync(0xffffffffu, used);
            const uint64_t bits = used ? row_tree(a, b, t, s.n) : 0ull;
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < s.count; ++i, ++g) {
                const int j0 = (s.first + i) * kKeys;
                const bool edge = j0 + kKeys > (s.total ? s.len : 0);      // some tokens may be unseen
                const uint32_t t_s = t_lane + (g & 1) * kKeys;
                uint64_t seen = ~0ull;
                if (!(ok = wait_warp(&s_full[g & 1], (g >> 1) & 1))) break;
                tc_fence_after();
                if (warp_live) {
                    uint32_t x0[32], x1[32];
                    tmem_ld32(t_s, x0);
                    tmem_ld32(t_s + 32, x1);
                    tmem_wait_ld();
                    if (edge) {
                        const int sh = s.len - j0;                          // draft token 0's place in the tile
                        seen = sh >= 64 ? ~0ull : sh > 0 ? (1ull << sh) - 1 : 0ull;
                        seen |= sh >= 64 ? 0ull : sh >= 0 ? bits << sh : sh > -64 ? bits >> -sh : 0ull;
                        if (!used) seen = 0ull;
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            if (!((seen >> k) & 1)) x0[k] = 0xff800000u;
                            if (!((seen >> (k + 32)) & 1)) x1[k] = 0xff800000u;
                        }
                    }
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        top[k & 3] = fmaxf(top[k & 3], fmaxf(__uint_as_float(x0[k]), __uint_as_float(x1[k])));
                    }
                    const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2;
                    float fac = 1.f;
                    bool raise = false;
                    if (mt > m + 8.f || m == -INFINITY) {       // m -inf: nothing summed yet
                        fac = ex2(m - (mt == -INFINITY ? 0.f : mt));
                        raise = i > 0 && m != mt;
                        m = mt;
                        l *= fac;
                    }
                    if (__any_sync(0xffffffffu, raise)) {
                        if (!(ok = wait_warp(o_done, (g - 1) & 1))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(t_lane + P::COL_O + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fac);
                            tmem_st32(t_lane + P::COL_O + c, o);
                        }
                        tmem_wait_st();
                    }
                    const float ms = m == -INFINITY ? 0.f : m;
                    const float2 sc = make_float2(a.scale_log2, a.scale_log2), mm = make_float2(-ms, -ms);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    uint32_t hi[32], lo[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const uint32_t *x = k < 16 ? x0 + 2 * k : x1 + 2 * k - 32;
                        float2 e = fma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), sc, mm);
                        e = make_float2(ex2(e.x), ex2(e.y));
                        sum[k & 1] = add2(sum[k & 1], e);
                        __nv_bfloat162 h = __floats2bfloat162_rn(e.x, e.y);
                        hi[k] = *reinterpret_cast<const uint32_t *>(&h);
                        e = fma2(make_float2(__uint_as_float(hi[k] << 16), __uint_as_float(hi[k] & 0xffff0000u)),
                                 make_float2(-1.f, -1.f), e);
                        h = __floats2bfloat162_rn(e.x, e.y);
                        lo[k] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                    l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
                    tmem_st32(t_s, hi);
                    tmem_st32(t_s + 32, lo);
                    tmem_wait_st();
                }
                unsigned long long special = 0ull;
                if (edge) {
                    // Value rows past the last token hold anything: zeros in their place.  The
                    // draft's values may be unseen by some rows, whose zero weights must not meet
                    // an infinity or NaN: those elements are zeroed too, and added below to
                    // the rows that do see them.
                    const uint32_t pos = 2 * g + 1, stage = pos % P::NST;
                    if (!(ok = wait_warp(&full[stage], (pos / P::NST) & 1))) break;
                    uint8_t *sv = ring + stage * P::STAGE;
                    const int from = max(0, s.len - j0) * (s.total ? 1 : 0), live = s.total - j0;
                    for (int x = tid + from * (D / 8); x < kKeys * (D / 8); x += 128) {
                        const int r = x / (D / 8), c = x % (D / 8);
                        uint4 *at = reinterpret_cast<uint4 *>(sv + (c >> 3) * (kKeys * 128) + sw128(r, c & 7));
                        if (r >= live) {
                            *at = make_uint4(0u, 0u, 0u, 0u);
                            continue;
                        }
                        uint32_t w[4] = {at->x, at->y, at->z, at->w};
                        bool bad = false;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if ((w[k] & 0x7f80u) == 0x7f80u) w[k] &= 0xffff0000u, bad = true;
                            if ((w[k] & 0x7f800000u) == 0x7f800000u) w[k] &= 0x0000ffffu, bad = true;
                        }
                        if (bad) {
                            *at = make_uint4(w[0], w[1], w[2], w[3]);
                            atomicOr(&odd[g & 1], 1ull << r);
                        }
                    }
                    fence_proxy_async();
                    if (!(ok = rows_sync())) break;
                    special = odd[g & 1];
                }
                // The product before is done (it nearly always is: the softmax takes longer), so that a
                // wait for this tile's cannot mistake that one's phase for its own.
                if (i > 0 && !(ok = wait_warp(o_done, (g - 1) & 1))) break;
                tc_fence_before();
                mbar_arrive(&p_full[g & 1]);
                if (special) {                      // the same for all 128 rows
                    if (!(ok = wait_warp(o_done, g & 1))) break;
                    tc_fence_after();
                    if (warp_live) {
                        const uint64_t mine = used ? seen & special : 0ull;
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(t_lane + P::COL_O + c, o);
                            tmem_wait_ld();
                            for (int r = 0; r < kKeys; ++r) {
                                if (!((special >> r) & 1)) continue;
                                const int j = j0 + r;
                                int id = __ldg(a.s.table + static_cast<size_t>(s.slot) * a.s.max_pages + (j >> a.s.page_shift));
                                if (id < 0 || id >= a.s.n_page) id = 0;
                                const size_t vrow = ((static_cast<size_t>(id) * a.s.Hkv + s.h) << a.s.page_shift) +
                                                    (j & ((1 << a.s.page_shift) - 1));
                                const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) + vrow * D + c;
#pragma unroll
                                for (int k = 0; k < 32; ++k) {
                                    const float y = __bfloat162float(v[k]);
                                    if (((mine >> r) & 1) && !(fabsf(y) < INFINITY)) o[k] = __float_as_uint(__uint_as_float(o[k]) + y);
                                }
                            }
                            tmem_st32(t_lane + P::COL_O + c, o);
                        }
                        tmem_wait_st();
                    }
                    if (!(ok = rows_sync())) break;
                    if (tid == 0) odd[g & 1] = 0ull;
                    if (!(ok = rows_sync())) break;
                }
            }
            if (!ok) break;
            // ---- the unit's result, or this CTA's part of it
            if (!(ok = wait_warp(o_done, (g - 1) & 1))) break;
            tc_fence_after();
            const bool whole = s.count == s.tiles;
            const size_t unit = (static_cast<size_t>(b) * a.s.Hkv + s.h) * ta.row_tiles + s.rt;
            if (tid == 0 && s.first == 0)
                ta.desc[unit] = make_int2(blockIdx.x, whole ? 1 : owner(W, N, s.unit_w + s.tiles - 1) - static_cast<int>(blockIdx.x) + 1);
            if (__any_sync(0xffffffffu, row < rows)) {
                if (whole) {
                    const float inv = used && (l > 0.f || l != l) ? 1.f / l : 0.f;
                    const size_t orow = (static_cast<size_t>(b) * a.s.T + t) * a.Hq + s.h * a.G + (row - t * a.G);
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + orow * D);
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(t_lane + P::COL_O + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t h[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(o[8 * k + 2 * e]) * inv,
                                                                               __uint_as_float(o[8 * k + 2 * e + 1]) * inv);
                                h[e] = inv != 0.f ? *reinterpret_cast<const uint32_t *>(&y) : 0u;
                            }
                            if (row < rows) dst[c / 8 + k] = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                        __syncwarp();
                    }
                    if (a.lse && row < rows) a.lse[orow] = used ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
                } else {
                    // column by column, so that a warp's rows are one run of memory
                    float *dst = ta.part + static_cast<size_t>(2 * blockIdx.x + (s.first == 0 ? 1 : 0)) * (D + 2) * ta.rp + tid;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(t_lane + P::COL_O + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (row < rows) dst[static_cast<size_t>(c + k) * ta.rp] = __uint_as_float(o[k]);
                        __syncwarp();
                    }
                    if (row < rows) {
                        dst[static_cast<size_t>(D) * ta.rp] = m;
                        dst[static_cast<size_t>(D + 1) * ta.rp] = l;
                    }
                }
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort) {                                   // nothing of this CTA runs on when it ends
        if (warp == 4) {
            for (uint32_t k = pos > P::NST ? pos - P::NST : 0; k < pos; ++k)
                if (!mbar_wait(&full[k % P::NST], (k / P::NST) & 1) && lane == 0) atomicOr(a.s.status, GDN_STATUS_DRAIN);
        } else if (warp == 5 && issued) {
            mma_commit(drain);
            if (!mbar_wait(drain, 0)) atomicOr(a.s.status, GDN_STATUS_DRAIN);
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
    }
    if (warp == 5) tmem_dealloc(tmem, P::TMEM_COLS);
}

// ------------------------------------------------------------------- the join
// One CTA per (unit, 8 output columns): a thread per row in each of kGroups groups, which take
// every kGroups-th part; the groups' sums are joined in shared memory in their order.
constexpr int kGroups = 4;

template <int D>
__global__ void __launch_bounds__(kGroups * kRows) verify_tc_join_kernel(const TcArgs ta, int grid)
{
    const AttnArgs &a = ta.a;
    const int rt = blockIdx.x % ta.row_tiles, bh = blockIdx.x / ta.row_tiles;
    const int h = bh % a.s.Hkv, b = ta.b0 + bh / a.s.Hkv;
    const int r = threadIdx.x % kRows, grp = threadIdx.x / kRows;
    __shared__ float acc_s[kGroups][8][kRows], m_s[kGroups][kRows], l_s[kGroups][kRows];
    pdl_wait();
    pdl_release();
    const int2 d = ta.desc[(static_cast<size_t>(b) * a.s.Hkv + h) * ta.row_tiles + rt];
    if (d.y < 2 || d.x < 0 || d.x + d.y > grid) return;           // finished by one CTA
    const Seq sq = load_seq(a.s, b);
    if (sq.bad) return;
    const int row = rt * kRows + r, t = row / a.G, rows = a.s.T * a.G;
    const bool used = row < rows && t < sq.n;
    auto part = [&](int k) {                                      // part k: the first CTA's second slot, then first slots
        return ta.part + static_cast<size_t>(2 * (d.x + k) + (k == 0 ? 1 : 0)) * (D + 2) * ta.rp + r;
    };
    float m = -INFINITY, l = 0.f, acc[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = 0.f;
    if (used) {
        const int c0 = blockIdx.y * 8;
#pragma unroll 2
        for (int k = grp; k < d.y; k += kGroups) {
            const float *p = part(k);
            const float mk = p[static_cast<size_t>(D) * ta.rp], lk = p[static_cast<size_t>(D + 1) * ta.rp];
            float x[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) x[c] = p[static_cast<size_t>(c0 + c) * ta.rp];
            const float mn = fmaxf(m, mk), ms = mn == -INFINITY ? 0.f : mn;
            const float f0 = ex2(m - ms), f1 = ex2(mk - ms);
            m = mn;
            l = l * f0 + lk * f1;
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[c] = acc[c] * f0 + x[c] * f1;
        }
    }
    m_s[grp][r] = m;
    l_s[grp][r] = l;
#pragma unroll
    for (int c = 0; c < 8; ++c) acc_s[grp][c][r] = acc[c];
    __syncthreads();
    if (grp != 0 || row >= rows) return;
    float mn = -INFINITY;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) mn = fmaxf(mn, m_s[k][r]);
    const float ms = mn == -INFINITY ? 0.f : mn;
    float lt = 0.f, o[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] = 0.f;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        const float f = ex2(m_s[k][r] - ms);
        lt = fmaf(l_s[k][r], f, lt);
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c] = fmaf(acc_s[k][c][r], f, o[c]);
    }
    const size_t orow = (static_cast<size_t>(b) * a.s.T + t) * a.Hq + h * a.G + (row - t * a.G);
    const bool any = used && (lt > 0.f || lt != lt);
    const float inv = any ? 1.f / lt : 0.f;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(o[2 * e] * inv, o[2 * e + 1] * inv);
        w[e] = any ? *reinterpret_cast<const uint32_t *>(&y) : 0u;
    }
    reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + orow * D)[blockIdx.y] = make_uint4(w[0], w[1], w[2], w[3]);
    if (a.lse && blockIdx.y == 0) a.lse[orow] = used ? (mn + log2f(lt)) * 0.69314718055994531f : -INFINITY;
}

// ------------------------------------------------------------------- host side
bool page_map(CUtensorMap *m, const void *base, const gdn_page_cache *c) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(c->d), static_cast<cuuint64_t>(c->n_page) * c->Hkv * c->page};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(c->d) * 2};
    cuuint32_t box[2] = {64, static_cast<cuuint32_t>(c->page < kKeys ? c->page : kKeys)};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
int tc_row_tiles(const gdn_page_cache *c, const gdn_attn_dims *d) {
    return (d->T * (d->Hq / c->Hkv) + kRows - 1) / kRows;
}
int tc_rp(const gdn_page_cache *c, const gdn_attn_dims *d) {
    const int rows = d->T * (d->Hq / c->Hkv);
    return rows >= kRows ? kRows : (rows + 31) / 32 * 32;
}
// CTAs of a launch over nb sequences: as many as can be resident, but no more than there may be tiles.
int tc_grid(const gdn_page_cache *c, const gdn_attn_dims *d, int nb) {
    const long long tiles = (static_cast<long long>(c->max_pages) * c->page + kKeys - 1) / kKeys;
    const long long all = tiles * nb * c->Hkv * tc_row_tiles(c, d);
    const int resident = sm_count() * (c->d == 256 ? TcPlan<256>::CTAS : TcPlan<128>::CTAS);
    return static_cast<int>(all < resident ? all : resident);
}
size_t desc_bytes(const gdn_page_cache *c, const gdn_attn_dims *d) {
    return (static_cast<size_t>(d->B) * c->Hkv * tc_row_tiles(c, d) * sizeof(int2) + 15) & ~static_cast<size_t>(15);
}

template <int D>
int launch_tc(const gdn_page_cache *c, const gdn_attn_dims *d, const AttnArgs &a, cudaStream_t s) {
    using P = TcPlan<D>;
    CUtensorMap mk, mv;
    if (!page_map(&mk, a.k, c) || !page_map(&mv, a.v, c)) return GDN_ERR_LAUNCH;
    if (cudaFuncSetAttribute(verify_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::BYTES) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    TcArgs ta{a, 0, 0, tc_row_tiles(c, d), tc_rp(c, d), reinterpret_cast<int2 *>(a.ws),
              reinterpret_cast<float *>(reinterpret_cast<char *>(a.ws) + desc_bytes(c, d))};
    for (ta.b0 = 0; ta.b0 < d->B; ta.b0 += kMaxSeqs) {
        ta.nb = d->B - ta.b0 < kMaxSeqs ? d->B - ta.b0 : kMaxSeqs;
        const int grid = tc_grid(c, d, ta.nb);
        if (launch_pdl(verify_tc_kernel<D>, dim3(grid), dim3(kTcThreads), P::BYTES, s, mk, mv, ta) != cudaSuccess ||
            launch_pdl(verify_tc_join_kernel<D>, dim3(ta.nb * c->Hkv * ta.row_tiles, D / 8), dim3(kGroups * kRows), 0, s,
                       ta, grid) != cudaSuccess)
            return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}

}  // namespace

int64_t attn_tc_workspace(const gdn_page_cache *c, const gdn_attn_dims *d) {
    const int nb = d->B < kMaxSeqs ? d->B : kMaxSeqs;
    return static_cast<int64_t>(desc_bytes(c, d)) +
           static_cast<int64_t>(2) * tc_grid(c, d, nb) * (c->d + 2) * tc_rp(c, d) * 4;
}

int attn_tc_verify(const gdn_page_cache *c, const gdn_attn_dims *d, const AttnArgs &a, cudaStream_t s) {
    return c->d == 64 ? launch_tc<64>(c, d, a, s) : c->d == 128 ? launch_tc<128>(c, d, a, s) : launch_tc<256>(c, d, a, s);
}

}  // namespace gdn
