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
// so up to about 128 rows the tiles go by at the HBM rate (d 128: 1400 cycles each); above, by the softmax
// and the MMAs (a pair of row tiles: 2400 cycles a tile of keys).  B 32, T 16, Hq 16, Hkv 2, d 128 over 900 to
// 8000 tokens: 43.1 us with the join, 3.6 TB/s; B 128, T 8, d 256: 104 us, 5.2 TB/s; one token over 700: 10 us.  Some 4 us
// pass before the first tile (length, share, unit, page, first load), 3 at the end.
//
// Work.  A unit is (sequence, key head, tile of 128 rows or pair of such tiles); its keys come in
// tiles of 64.  All units' tiles in a row are cut into equal shares, one per SM, so ragged lengths
// balance and one long sequence fills the GPU.  A unit that one CTA covers is finished there; the
// others leave partial results (o, m, l) that a second kernel joins in a fixed order.
//
// A CTA.  Two warps load (TMA through the block table, one copy a tile or, of pages below 64, per page and
// atom) into a ring of NST / 2 tiles of keys and as many of values (8, 4 or 2 for d 64, 128, 256).  Two
// groups of 256 threads with an MMA warp each work side by side: on a pair of row tiles, both on every
// tile of keys; on a single one, on every second tile, their results joined at the end (d = 256 has TMEM for
// one group).  A group forms S = Q K^T (M 128, N 64) in two TMEM buffers; its threads, two per row, each take
// half of the tile's keys; the weights' two terms go back over S and are the A operands of
// O += P V straight from TMEM, with the value rows read MN-major as they lie.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "attn_common.h"
#include "tc_common.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kKeys = 64, kRows = 128;              // tile of keys, tile of rows
constexpr uint32_t kIdleLimit = 1u << 24;           // polls of an MMA warp without work before giving up
constexpr int kGroupThreads = 256;                  // two per row
constexpr int kMaxSeqs = 512;                       // most sequences of one launch (their table in shared memory)
constexpr uint32_t kIdescMnMajorB = 1u << 16;

// D: head dim; NQ: most row tiles of a unit.
template <int D, int NQ> struct TcPlan {
    static constexpr int NG = D == 256 ? 1 : 2;                 // groups
    static constexpr int ATOMS = D / 64;                        // 128-byte column atoms of a row
    static constexpr int STAGE = kKeys * D * 2;                 // a tile of keys or of values
    static constexpr int NST = D == 64 ? 16 : D == 256 ? 4 : 8;
    static constexpr int ROWS = NG * kGroupThreads;             // row threads
    static constexpr int LOAD_WARP = ROWS / 32, MMA_WARP = LOAD_WARP + 2;      // two and NG warps
    static constexpr int THREADS = ROWS + 32 * (2 + NG);
    static constexpr int QTILE = kRows * D * 2;
    static constexpr int OFF_RING = NQ * QTILE;                 // after the queries
    static constexpr int OFF_SEQ = OFF_RING + NST * STAGE;      // prefix, slot, len, n, live, units
    static constexpr int OFF_XCH = OFF_SEQ + (6 * kMaxSeqs + 4) * 4;                      // two words per row thread
    static constexpr int OFF_BAR = OFF_XCH + ROWS * 8;
    static constexpr int BYTES = OFF_BAR + 640;
    static constexpr int TCOLS = 2 * kKeys + D;                 // TMEM of a group: S in [0, 64) and [64, 128), then O
    static constexpr int TMEM_COLS = 512;
    static_assert(NG * TCOLS <= TMEM_COLS && NQ <= NG, "tensor memory");
    // Where the groups take every second tile, a stage always serves the same group (the one of
    // its tile's parity): a group that had not seen a stage's last round could take its phase for the
    // next.  From such a unit to a pair the queries' barriers (all scores of the unit before are
    // done) and the row threads' (all its products are) keep a group from running ahead.
    // Row threads wait for values in the draft's tiles alone and skip a stage's other rounds; the stage's
    // round before must then be over, or its phase would pass for this one's.  It is: scores of a group's
    // tile t wait for its product of t - 2, and a stage comes round after NST / 2 tiles, two of the one
    // group at d 256, two or four of each where the groups take turns, four or eight on pairs.
    static_assert(NST % 4 == 0, "stages of a tile alternate between the groups");
    static_assert(OFF_BAR % 16 == 0 && BYTES <= 227 * 1024, "shared memory");
};

struct TcArgs {
    AttnArgs a;
    int b0, nb;                 // sequences [b0, b0 + nb) of the call
    int tpt, row_tiles;         // tokens of a row tile (128 / G), row tiles of a key head
    int rp;                     // rows of a partial result (a multiple of 32)
    int4 *rec;                  // records of the units that are split: row tile, row tiles of it, first CTA, parts
    int by_cta;                 // a record's place: the first CTA's number, or (fewer units than CTAs) the row tile's
    float *part;                // [2 CTAs][NQ][D + 2][rp]
};

__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15};"
        ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(taddr)
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
// True in one lane of a converged warp (the same one each time: commits track the issuing thread's MMAs).
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(saddr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(saddr(bar))
        : "memory");
}
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(saddr(bar)), "r"(parity) : "memory");
    return ok != 0;
}
// As mbar_try_wait, suspended for about `ns` at most.
__device__ __forceinline__ bool mbar_doze(uint64_t *bar, uint32_t parity, uint32_t ns) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(saddr(bar)), "r"(parity), "r"(ns) : "memory");
    return ok != 0;
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(bar)) : "memory");
}
// Named barriers of the row threads: of all of them (id 1), of a group (2, 3), and of the 64 threads
// of a group's TMEM lane quarter (4 ..).  They complete because all threads of a barrier take it equally
// often: no row warp leaves its loops early (an expired wait only stops the waiting), loop counts
// and branches around a barrier follow from the share alone or, for a tile's non-finite values, from
// one word in shared memory that all threads of the barrier read between the same two barriers.
__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool pair_any(int id, bool x) {
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\tbar.red.or.pred q, %1, 64, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(any) : "r"(id), "r"(static_cast<uint32_t>(x)) : "memory");
    return any != 0;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ------------------------------------------------------------- the work's layout
// Units of one (sequence, key head): the row tiles that hold rows in use, in pairs where NQ is 2
// (`pairs`, then `single`), take every tile of keys; each of the others is one tile without keys (its
// rows get zeros).  Work is counted in row tiles times tiles of keys (a pair's tile counts 2), and a
// unit counts `fixed` more: beginning and ending one costs a CTA as much as some tiles.
struct Shape {
    int live, dead, pairs, single, tiles, total;    // total: keys
    __device__ Shape(int len, int n, int live_, int row_tiles, int nq) {
        live = live_;
        dead = row_tiles - live;
        pairs = nq == 2 ? live / 2 : 0;
        single = live - 2 * pairs;
        total = len + n;
        tiles = (total + kKeys - 1) / kKeys;        // >= 1 when live > 0
    }
    __device__ int units() const { return pairs + single + dead; }
    __device__ int per_head(int fixed) const { return live * tiles + dead + fixed * units(); }
};
// Measured: 4 of 4, 6, 8 and 10 is best where all units are single (B 128, T 8, Hq 16, Hkv 2, d 256: 0 and
// 8 cost 1 to 2 % more), 8 where there are pairs (B 12, T 48, Hq 32, Hkv 4, d 128: 71 us with 0, 64 with
// 4, 62 with 8 and 10).
template <int NQ> constexpr int kFixed = NQ == 2 ? 8 : 4;
constexpr int kFixedFrom = 16;                      // tiles a CTA from which on it is counted: below, every tile
                                                    // on a CTA of its own is faster

// a / b for quotients below 2^20 (a >= 0, b > 0): one step corrects the float quotient.  The compiler's
// integer division takes three times as long, and several follow one another before the first load.
__device__ __forceinline__ int quotient(int a, int b) {
    int q = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
    const int r = a - q * b;
    return r < 0 ? q - 1 : r >= b ? q + 1 : q;
}

struct SeqTable {
    int *prefix;                                    // [nb + 1] work before each sequence
    int *slot, *len, *n;                            // [nb]
    int *live;                                      // [nb] row tiles with rows in use
    int *units;                                     // [nb] units before each sequence
    int nb;
    // The last sequence that starts at or before w, among those with work.
    __device__ int find(int w) const {
        int lo = 0, hi = nb - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= w) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
};

struct Segment {
    int b, h, rt, nq;                               // sequence (within the launch), key head, first row tile, row tiles
    int slot, len, n, total;                        // total 0: a row tile without rows in use
    int first, count, tiles;                        // tiles [first, first + count) of the unit's `tiles`
    int begin, end;                                 // the unit's place in the launch's work
};

// The unit that holds work item w, and the tile of it.
__device__ __forceinline__ void locate(const SeqTable &st, int b, int w, int row_tiles, int nq, int fixed, Segment &s) {
    const Shape sh(st.len[b], st.n[b], st.live[b], row_tiles, nq);
    const int in_b = w - st.prefix[b], per = sh.per_head(fixed);
    s.b = b;
    s.slot = st.slot[b];
    s.len = st.len[b];
    s.n = st.n[b];
    s.h = quotient(in_b, per);
    int r = in_b - s.h * per, size = 2 * sh.tiles + fixed, u;
    const int head = w - r, paired = sh.pairs * size, live = paired + sh.single * (sh.tiles + fixed);
    s.nq = 1;                                       // (nq is a constant: with 1 it stays one)
    s.tiles = sh.tiles;
    s.total = sh.total;
    int start = 0;
    if (nq == 2 && r < paired) {
        u = sh.pairs == 1 ? 0 : quotient(r, size);
        s.nq = 2;
        s.rt = 2 * u;
    } else if (r < live) {
        start = nq == 2 ? paired : 0;
        size = sh.tiles + fixed;
        u = sh.single == 1 ? 0 : quotient(r - start, size);
        s.rt = 2 * sh.pairs + u;
    } else {
        start = live;
        size = 1 + fixed;
        u = quotient(r - start, size);
        s.rt = sh.live + u;
        s.tiles = 1;
        s.total = 0;
    }
    s.begin = head + start + u * size;
    s.end = s.begin + size;
    s.first = max(0, w - s.begin - fixed) >> (nq == 2 ? s.nq - 1 : 0);
}

// W work items cut into N shares: share c starts at c W / N, rounded down to where a tile (or,
// in a unit's fixed part and its first tile, the unit) begins.
struct Cut {
    int W, N, q, r, fixed;                          // W = q N + r
    __device__ int raw(int c) const { return q * c + quotient(r * c, N); }         // r c < N^2
};
template <int NQ> __device__ __forceinline__ int rounded(const Segment &s, int fixed) {
    return s.first == 0 ? s.begin : s.begin + fixed + (s.first << (NQ == 2 ? s.nq - 1 : 0));
}

// The CTAs that hold tiles of the unit, counted from the one that holds its first.
__device__ __forceinline__ int parts_of(const Cut &cut, const Segment &s) {
    int lo = blockIdx.x, hi = cut.N - 1;
    while (lo < hi) {                               // the last share that starts before the unit's end
        const int mid = (lo + hi + 1) >> 1;
        if (cut.raw(mid) < s.end) lo = mid;
        else hi = mid - 1;
    }
    return lo - static_cast<int>(blockIdx.x) + 1;
}

// Walks a CTA's share [w, w1) unit by unit.
struct Cursor {
    int w, w1, b, fixed;
    __device__ void take(int nq, Segment &s) {      // as much of the unit at w as is in the share
        if (w1 >= s.end) s.count = s.tiles - s.first;
        else s.count = ((w1 - s.begin - fixed) >> (nq == 2 ? s.nq - 1 : 0)) - s.first;
        w = min(w1, s.end);
    }
    __device__ bool next(const SeqTable &st, int row_tiles, int nq, Segment &s) {
        if (w >= w1) return false;
        while (st.prefix[b + 1] <= w) ++b;
        locate(st, b, w, row_tiles, nq, fixed, s);
        take(nq, s);
        return true;
    }
};

// The infinities and NaN among the values of the tile at j0 (rows `special`) added to the sums of the
// rows that see them (`view`, per thread); a whole warp calls it.
template <int D>
__device__ __noinline__ void add_odd_values(const AttnArgs &a, uint32_t t_o, int slot, int h, int j0, int half,
                                            unsigned long long special, uint64_t view)
{
#pragma unroll 1
    for (int c = 0; c < D / 2; c += 32) {
        uint32_t o[32];
        tmem_ld32(t_o + c, o);
        tmem_wait_ld();
#pragma unroll 1
        for (int r = 0; r < kKeys; ++r) {
            if (!((special >> r) & 1)) continue;
            const int j = j0 + r;
            int id = __ldg(a.s.table + static_cast<size_t>(slot) * a.s.max_pages + (j >> a.s.page_shift));
            if (id < 0 || id >= a.s.n_page) id = 0;
            const size_t vrow = ((static_cast<size_t>(id) * a.s.Hkv + h) << a.s.page_shift) + (j & ((1 << a.s.page_shift) - 1));
            const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) + vrow * D + half * (D / 2) + c;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                const float y = __bfloat162float(v[k]);
                if (((view >> r) & 1) && !(fabsf(y) < INFINITY)) o[k] = __float_as_uint(__uint_as_float(o[k]) + y);
            }
        }
        tmem_st32(t_o + c, o);
    }
    tmem_wait_st();
}

// ------------------------------------------------------------------ the kernel
template <int D, int NQ>
__global__ void __launch_bounds__(TcPlan<D, NQ>::THREADS, 1)
verify_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TcArgs ta)
{
    using P = TcPlan<D, NQ>;
    constexpr int NG = P::NG;
    const AttnArgs &a = ta.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    if (saddr(smem_raw) & 1023u) {                  // the swizzled tiles need a 1024-byte aligned base
        if (tid == 0) atomicOr(a.s.status, kStatusTimeout);
        return;
    }
    uint8_t *sQ = smem_raw, *ring = smem_raw + P::OFF_RING;
    SeqTable st;
    st.prefix = reinterpret_cast<int *>(smem_raw + P::OFF_SEQ);
    st.slot = st.prefix + kMaxSeqs + 4;
    st.len = st.slot + kMaxSeqs;
    st.n = st.len + kMaxSeqs;
    st.live = st.n + kMaxSeqs;
    st.units = st.live + kMaxSeqs;
    st.nb = ta.nb;
    float *xch = reinterpret_cast<float *>(smem_raw + P::OFF_XCH);
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem_raw + P::OFF_BAR);
    uint64_t *full = bar, *empty = bar + P::NST, *q_full = bar + 2 * P::NST, *q_empty = q_full + 1;
    uint64_t *s_full = q_empty + 1, *p_full = s_full + 2 * NG, *o_done = p_full + 2 * NG, *drain = o_done + 2 * NG;   // [group][2]; drain [group]
    unsigned long long *odd = reinterpret_cast<unsigned long long *>(drain + NG);         // [group][2]
    int2 *warp_sum = reinterpret_cast<int2 *>(odd + 2 * NG);                              // [warps]
    Cut *cut = reinterpret_cast<Cut *>(warp_sum + P::THREADS / 32);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(cut + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    static_assert((2 * P::NST + 2 + 9 * NG + P::THREADS / 32) * 8 + sizeof(Cut) + 8 <= 640, "barrier area");

    if (tid == 0) {
        for (int i = 0; i < P::NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], NG);               // a commit of each group, or two of the only one that reads it
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, NG);
        for (int i = 0; i < 2 * NG; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], kGroupThreads);
            mbar_init(&o_done[i], 1);
            odd[i] = 0ull;
        }
        for (int i = 0; i < NG; ++i) mbar_init(&drain[i], 1);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == P::LOAD_WARP) {
        tmem_alloc(tmem_slot, P::TMEM_COLS);
        if (lane < 3)
            asm volatile("prefetch.tensormap [%0];"
                         ::"l"(reinterpret_cast<uint64_t>(lane == 0 ? &tm_k : lane == 1 ? &tm_v : &tm_q)) : "memory");
    }
    pdl_wait();
    pdl_release();
    // ---- the sequences' table: the work before each
    int before = 0, units = 0;
    for (int i0 = 0; i0 < ta.nb; i0 += P::THREADS) {
        const int i = i0 + tid;
        int mine = 0, own_units = 0;
        if (i < ta.nb) {
            const Seq q = load_seq<true>(a.s, ta.b0 + i);
            const int live = q.bad ? 0 : quotient(q.n + ta.tpt - 1, ta.tpt);
            st.live[i] = live;
            if (!q.bad) {
                const Shape sh(q.len, q.n, live, ta.row_tiles, NQ);
                mine = sh.per_head(0) * a.s.Hkv;
                own_units = sh.units() * a.s.Hkv;
            }
            st.slot[i] = q.slot;
            st.len[i] = q.len;
            st.n[i] = q.n;
            if (q.bad && blockIdx.x == 0) {         // none of its row tiles is for the join
                atomicOr(a.s.status, q.bad);
                const int per = a.s.Hkv * ta.row_tiles;
                if (!ta.by_cta)
                    for (int u = 0; u < per; ++u) ta.rec[i * per + u] = make_int4(0, 0, 0, 0);
            }
        }
        int incl = mine, incl_u = own_units;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off), z = __shfl_up_sync(0xffffffffu, incl_u, off);
            if (lane >= off) incl += y, incl_u += z;
        }
        if (i0 > 0) __syncthreads();                // the sums of the round before have been read
        if (lane == 31) warp_sum[warp] = make_int2(incl, incl_u);
        __syncthreads();
        const int warps = min(P::THREADS / 32, (ta.nb - i0 + 31) / 32);
        for (int w = 0; w < warps; ++w) {
            if (w == warp && i < ta.nb) {
                st.prefix[i] = before + incl - mine;
                st.units[i] = units + incl_u - own_units;
            }
            before += warp_sum[w].x;
            units += warp_sum[w].y;
        }
    }
    // (every thread has the totals)
    const int fixed = before >= kFixedFrom * static_cast<int>(gridDim.x) ? kFixed<NQ> : 0;
    if (fixed)
        for (int i = tid; i < ta.nb; i += P::THREADS) st.prefix[i] += fixed * st.units[i];
    if (tid == 0) {
        const int W = before + fixed * units, most = NQ == 2 && W > 1 ? W / 2 : W;         // every share has a tile
        const int N = min(most, static_cast<int>(gridDim.x));
        st.prefix[ta.nb] = W;
        const int q = N ? W / N : 0;
        *cut = Cut{W, N, q, W - q * N, fixed};
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // This CTA's share and its first unit: every warp for itself, the share's two ends in its even and
    // odd lanes.
    const Cut c = *cut;
    Cursor cur{0, 0, 0, fixed};
    Segment s;
    const bool any_work = static_cast<int>(blockIdx.x) < c.N;
    if (any_work) {
        const int raw0 = c.raw(blockIdx.x), raw1 = c.raw(blockIdx.x + 1);       // (the last share ends at W)
        const bool odd_lane = lane & 1;
        const int raw = odd_lane ? raw1 : raw0;
        int seq;
        if (ta.nb <= 32) {
            const int pre = lane < ta.nb ? st.prefix[lane] : 0x7fffffff;
            const uint32_t m0 = __ballot_sync(0xffffffffu, pre <= raw0), m1 = __ballot_sync(0xffffffffu, pre <= raw1);
            seq = 31 - __clz(odd_lane ? m1 : m0);
        } else {
            seq = st.find(raw);
        }
        int w = raw;
        if (raw < c.W) {
            locate(st, seq, raw, ta.row_tiles, NQ, fixed, s);
            w = rounded<NQ>(s, fixed);
        }
        __syncwarp();
        int *word = reinterpret_cast<int *>(&s);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(Segment) / 4); ++i) word[i] = __shfl_sync(0xffffffffu, word[i], 0);
        cur.w = __shfl_sync(0xffffffffu, w, 0);
        cur.w1 = __shfl_sync(0xffffffffu, w, 1);
        cur.b = s.b;
        cur.take(NQ, s);
    }
    // GDN_FLAG_TEST_EXPIRE: the wait-expiry exit, with nothing issued before it
    if (a.flags & GDN_FLAG_TEST_EXPIRE) {
        if (tid == 0) {
            *abort = 1;
            atomicOr(a.s.status, kStatusTimeout);
        }
        __syncthreads();
    }
    auto expire = [&]() {
        *abort = 1;
        atomicOr(a.s.status, kStatusTimeout);
    };
    // A bounded wait: false when it, or another role's, expired.
    auto wait = [&](uint64_t *b, uint32_t parity) {
        for (uint32_t i = 0; i < kWaitLimit; ++i) {
            if (mbar_try_wait(b, parity)) return true;
            if (*abort) return false;
        }
        expire();
        return false;
    };
    if (ta.by_cta && tid == P::ROWS - 1) ta.rec[blockIdx.x] = make_int4(0, 0, 0, 0);
    uint32_t pos = 0;                               // load warps: tiles loaded (of keys, or of values)
    bool issued = false;                            // MMA warps: some MMA
    uint32_t queries = 0;                           // first MMA warp: loads of queries
    if (warp >= P::LOAD_WARP && warp < P::MMA_WARP) {
        // ------------------------------------------------------ loads
        // The first warp loads the tiles of keys, the second those of values: one copy a tile, or one for
        // each page and 64-column atom of it where pages are shorter.  (Where one key head has few rows, all
        // warps with rows in use share a scheduler with the keys' warp, and its instructions count: B 64, T 4,
        // 8 heads of 64 over 100 to 8000 tokens in pages of 64: 121 us, with the short pages' loop 134.)  Lane c holds the page of place c in the block table's next 32
        // entries, read 32 entries ahead; the copies are issued by one lane from values that are
        // the same in every lane (issued lane by lane, each cost 100 cycles).
        const int kv = warp - P::LOAD_WARP, shift = a.s.page_shift;
        const int ps = shift < 6 ? shift : 6;                              // rows of a copy: 16, 32 or 64
        const CUtensorMap *map = kv ? &tm_v : &tm_k;
        bool ok = !*abort;
        for (bool have = ok && any_work; have; have = ok && cur.next(st, ta.row_tiles, NQ, s)) {
            const int32_t *tab = a.s.table + static_cast<size_t>(s.slot) * a.s.max_pages;
            const int count = __shfl_sync(0xffffffffu, s.count, 0), first = __shfl_sync(0xffffffffu, s.first, 0);
            const int total = __shfl_sync(0xffffffffu, s.total, 0), head = __shfl_sync(0xffffffffu, s.h, 0);
            const int p0 = first * kKeys >> shift;                         // the segment's first block-table entry
            const int p_end = min((first + count) * kKeys, total);         // tokens
            auto read_ids = [&](int at) {                                  // entries p0 + at + lane
                const int p = p0 + at + lane;
                if (static_cast<long long>(p) << shift >= p_end) return -1;
                const int id = __ldg(tab + p);
                if (id >= 0 && id < a.s.n_page) return id;
                if (kv == 0) atomicOr(a.s.status, GDN_STATUS_BAD_PAGE);
                return 0;
            };
            int ids = read_ids(0), ids_next = read_ids(32), base = 0;
            auto tiles = [&](auto load) {
                for (int i = 0; i < count; ++i, ++pos) {
                    const int j0 = (first + i) * kKeys, at = (j0 >> shift) - p0;
                    if (at - base >= 32) {
                        base += 32;
                        ids = ids_next;
                        ids_next = read_ids(base + 32);
                    }
                    const uint32_t spos = 2 * pos + kv, stage = spos % P::NST, round = spos / P::NST;
                    if (round > 0) ok = __all_sync(0xffffffffu, wait(&empty[stage], (round - 1) & 1)) != 0;
                    if (!ok) break;
                    load(j0, at - base, ring + stage * P::STAGE, &full[stage]);
                    __syncwarp();
                }
            };
            if (ps == 6) {                          // one copy for all of a tile
                tiles([&](int j0, int place, uint8_t *dst, uint64_t *done) {
                    const int id = __shfl_sync(0xffffffffu, ids, place & 31);
                    const int row = ((id * a.s.Hkv + head) << shift) + (j0 & ((1 << shift) - 1));
                    if (elect_one()) {
                        mbar_expect_tx(done, total ? P::STAGE : 0);
                        if (total) tma_load_3d(dst, map, 0, row, 0, done);
                    }
                });
            } else {
                tiles([&](int j0, int place, uint8_t *dst, uint64_t *done) {
                    int row[kKeys / 16];
                    uint32_t bytes = 0;
#pragma unroll
                    for (int c = 0; c < kKeys / 16; ++c) {
                        const int id = __shfl_sync(0xffffffffu, ids, (place + c) & 31);
                        row[c] = c < (kKeys >> ps) && j0 + (c << ps) < total ? (id * a.s.Hkv + head) << shift : -1;
                        bytes += row[c] >= 0 ? (P::ATOMS * 128u) << ps : 0u;
                    }
                    if (elect_one()) {
                        mbar_expect_tx(done, bytes);
#pragma unroll
                        for (int c = 0; c < kKeys / 16; ++c)
                            if (row[c] >= 0) {
#pragma unroll
                                for (int x = 0; x < P::ATOMS; ++x)
                                    tma_load_2d(dst + x * (kKeys * 128) + (c << (ps + 7)), map, x * 64, row[c], done);
                            }
                    }
                });
            }
        }
    } else if (warp >= P::MMA_WARP) {
        // ------------------------------------------------------ MMAs
        // The whole warp walks the tiles and one elected lane issues: values that the compiler
        // can see to be the same in every lane stay in uniform registers, where the MMA takes its
        // operands from (issued inside a one-lane branch, each MMA cost about 125 cycles).
        const int group = warp - P::MMA_WARP;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0) + group * P::TCOLS;
        const uint64_t dk0 = desc_sw128(saddr(ring)), dv0 = desc_mn_sw128(saddr(ring), kKeys * 128);
        constexpr uint32_t idS = idesc_mn(1, kRows, kKeys), idO = idesc_mn(1, kRows, D) | kIdescMnMajorB;
        uint64_t *sf = s_full + 2 * group, *pf = p_full + 2 * group, *od = o_done + 2 * group;
        uint32_t g = 0, tile0 = 0, segs = 0;        // this group's tiles, the CTA's tiles and segments so far
        bool ok = !*abort;
        Segment next;
        auto load_queries = [&](const Segment &u) {
            const int nq = NQ == 1 ? 1 : __shfl_sync(0xffffffffu, u.nq, 0), y = __shfl_sync(0xffffffffu, u.h, 0) * a.G;
            const int z = (ta.b0 + __shfl_sync(0xffffffffu, u.b, 0)) * a.s.T + __shfl_sync(0xffffffffu, u.rt, 0) * ta.tpt;
            if (elect_one()) {
                mbar_expect_tx(q_full, nq * P::ATOMS * ta.tpt * a.G * 128);
#pragma unroll 1
                for (int q = 0; q < nq; ++q)
#pragma unroll
                    for (int x = 0; x < P::ATOMS; ++x)
                        tma_load_3d(sQ + q * P::QTILE + x * (kRows * 128), &tm_q, x * 64, y, z + q * ta.tpt, q_full);
            }
            __syncwarp();
            ++queries;
        };
        bool have = ok && any_work;
        while (have) {
            const bool alternate = NG == 2 && (NQ == 1 || s.nq == 1);
            const int step = alternate ? 2 : 1, off = alternate ? (group ^ tile0) & 1 : 0;
            const int count = __shfl_sync(0xffffffffu, (s.count - off + step - 1) / step, 0);
            const bool twice = __shfl_sync(0xffffffffu, alternate ? 1 : 0, 0) != 0;
            const uint64_t dq = desc_sw128(saddr(sQ) + (alternate ? 0 : group * P::QTILE));
            if (group == 0 && segs == 0) load_queries(s);
            const bool more = group == 0 && cur.next(st, ta.row_tiles, NQ, next);
            bool wanted = more;                     // the next unit's queries, once all scores of this one are done
            ok = ok && __all_sync(0xffffffffu, wait(q_full, segs & 1)) != 0;
            ++segs;
            if (ok && count == 0 && elect_one()) mbar_arrive(q_empty);
            int sn = 0, pn = 0;                     // next tile to score, next to multiply with the values
            uint32_t idle = 0;
            while (ok && pn < count) {
                bool did = false;
                if (wanted && sn == count && __all_sync(0xffffffffu, mbar_test(q_empty, (segs - 1) & 1))) {
                    load_queries(next);
                    wanted = false;
                }
                if (sn < count && sn < pn + 2) {
                    // the buffer held the weights of the group's tile t - 2: their product must be done
                    const uint32_t t = g + sn, kpos = 2 * (tile0 + sn * step + off), stage = kpos % P::NST;
                    const bool ready = mbar_test(&full[stage], (kpos / P::NST) & 1) &&
                                       (t < 2 || mbar_test(&od[t & 1], ((t - 2) >> 1) & 1));
                    if (__all_sync(0xffffffffu, ready)) {
                        tc_fence_after();
                        const uint64_t dk = desc_add(dk0, stage * P::STAGE);
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                const uint32_t at = (k & 3) * 32;
                                mma_bf16(tm + (t & 1) * kKeys, desc_add(dq, (k >> 2) * (kRows * 128) + at),
                                         desc_add(dk, (k >> 2) * (kKeys * 128) + at), idS, k > 0);
                            }
                            mma_commit(&sf[t & 1]);
                            mma_commit(&empty[stage]);
                            if (twice) mma_commit(&empty[stage]);
                            if (sn + 1 == count) mma_commit(q_empty);
                        }
                        issued = did = true;
                        ++sn;
                    }
                }
                if (pn < sn) {
                    const uint32_t t = g + pn, vpos = 2 * (tile0 + pn * step + off) + 1, stage = vpos % P::NST;
                    const bool ready = mbar_test(&pf[t & 1], (t >> 1) & 1) && mbar_test(&full[stage], (vpos / P::NST) & 1);
                    if (__all_sync(0xffffffffu, ready)) {
                        tc_fence_after();
                        const uint64_t dv = desc_add(dv0, stage * P::STAGE);
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < kKeys / 8; ++k)   // the weights' first terms, then their second
                                mma_bf16_ts(tm + 2 * kKeys, tm + (t & 1) * kKeys + k * 8, desc_add(dv, (k & 3) * 2048), idO,
                                            pn > 0 || k > 0);
                            mma_commit(&empty[stage]);
                            if (twice) mma_commit(&empty[stage]);
                            mma_commit(&od[t & 1]);
                        }
                        did = true;
                        ++pn;
                    }
                }
                if (did) {
                    idle = 0;
                    continue;
                }
                // asleep until the next weights are there (or, before any, the next keys), but not
                // for long: the other may come first
                const uint32_t t = g + pn, kpos = 2 * (tile0 + sn * step + off), stage = kpos % P::NST;
                if (pn < sn) mbar_doze(&pf[t & 1], (t >> 1) & 1, 200);
                else mbar_doze(&full[stage], (kpos / P::NST) & 1, 200);
                ++idle;
                if (*abort || idle > kIdleLimit) {
                    if (idle > kIdleLimit) expire();
                    ok = false;
                }
                ok = __all_sync(0xffffffffu, ok);
            }
            if (ok && wanted) {
                ok = __all_sync(0xffffffffu, wait(q_empty, (segs - 1) & 1)) != 0;
                if (ok) load_queries(next);
            }
            g += count;
            tile0 += s.count;
            if (group == 0) {
                have = ok && more;
                s = next;
            } else {
                have = ok && cur.next(st, ta.row_tiles, NQ, s);
            }
        }
    } else {
        // ------------------------------------------------------ rows
        // Thread (group, half, row): keys [32 half, 32 half + 32) of the group's tiles, output columns
        // [D/2 half, + D/2).
        const int group = NG == 2 ? warp >> 3 : 0, quarter = warp & 3, half = (warp >> 2) & 1;
        const int r_in = quarter * 32 + lane, gtid = tid & (kGroupThreads - 1), pair_id = 4 + group * 4 + quarter;
        const uint32_t t_lane = tmem + group * P::TCOLS + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t t_o = t_lane + 2 * kKeys + half * (D / 2);
        uint64_t *sf = s_full + 2 * group, *pf = p_full + 2 * group, *od = o_done + 2 * group;
        float *xm = xch, *xl = xch + P::ROWS;       // maxima and sums of the row threads
        uint32_t g = 0, tile0 = 0;
        auto wait_rows = [&](uint64_t *b, uint32_t parity) {   // reconverged: TMEM accesses take whole warps
            wait(b, parity);
            __syncwarp();
            tc_fence_after();
        };
        Segment next;
        bool more = any_work;
        auto token_of = [&](const Segment &u) {      // this thread's draft token in unit u
            return (u.rt + (NQ == 2 && u.nq == 2 ? group : 0)) * ta.tpt + r_in / a.G;
        };
        auto word_of = [&](const Segment &u) {
            const int t = token_of(u);
            return r_in < ta.tpt * a.G && t < a.s.T && t < u.n ? row_tree(a, ta.b0 + u.b, t, u.n) : 0ull;
        };
        uint64_t bits = more ? word_of(s) : 0ull, next_bits = 0ull;
        while (more) {
            const bool alternate = NG == 2 && (NQ == 1 || s.nq == 1);
            const int step = alternate ? 2 : 1, off = alternate ? (group ^ tile0) & 1 : 0;
            const int per_tile = ta.tpt * a.G;
            const int b = ta.b0 + s.b;
            if (NG == 2) bar_sync(1, P::ROWS);      // both groups have left each other's O and exchange words
            const int t = token_of(s), qh = r_in % a.G;                    // draft token, head of the group
            const bool exists = r_in < per_tile && t < a.s.T, used = exists && t < s.n;
            const bool warp_live = __any_sync(0xffffffffu, used);
            float m = -INFINITY, l = 0.f;           // m: the same in both threads of a row; l: of this thread's keys
            int mine = 0;                           // tiles of this group
            for (int i = off; i < s.count; i += step, ++g, ++mine) {
                const int j0 = (s.first + i) * kKeys;
                const bool edge = j0 + kKeys > (s.total ? s.len : 0);      // some tokens may be unseen
                const uint32_t t_s = t_lane + (g & 1) * kKeys;
                wait_rows(&sf[g & 1], (g >> 1) & 1);
                if (warp_live) {
                    uint32_t x[32];
                    tmem_ld32(t_s + 32 * half, x);
                    tmem_wait_ld();
                    if (edge) {
                        const int sh = s.len - j0;                          // draft token 0's place in the tile
                        uint64_t all = sh >= 64 ? ~0ull : sh > 0 ? (1ull << sh) - 1 : 0ull;
                        all |= sh >= 64 ? 0ull : sh >= 0 ? bits << sh : sh > -64 ? bits >> -sh : 0ull;
                        const uint32_t seen = used ? static_cast<uint32_t>(all >> (32 * half)) : 0u;
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!((seen >> k) & 1)) x[k] = 0xff800000u;
                    }
                    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 32; k += 2)
                        top[(k >> 1) & 1] = fmaxf(top[(k >> 1) & 1], fmaxf(__uint_as_float(x[k]), __uint_as_float(x[k + 1])));
                    const float mt = fmaxf(top[0], top[1]) * a.scale_log2;
                    // (also: both threads have read their scores, which the weights go over)
                    if (pair_any(pair_id, mt > m + 8.f)) {
                        xm[tid] = mt;
                        bar_sync(pair_id, 64);
                        const float mp = fmaxf(mt, xm[tid ^ 128]);
                        bar_sync(pair_id, 64);                              // read before it is written again
                        float fac = 1.f;
                        if (mp > m + 8.f) {
                            fac = ex2(m - mp);                              // 0 when nothing was summed
                            m = mp;
                            l *= fac;
                        }
                        if (mine > 0) {
                            wait_rows(&od[(g - 1) & 1], ((g - 1) >> 1) & 1);
#pragma unroll 1
                            for (int c = 0; c < D / 2; c += 32) {
                                uint32_t o[32];
                                tmem_ld32(t_o + c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fac);
                                tmem_st32(t_o + c, o);
                            }
                        }
                    }
                    const float ms = m == -INFINITY ? 0.f : m;
                    const float2 sc = make_float2(a.scale_log2, a.scale_log2), mm = make_float2(-ms, -ms);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float2 e = fma2(make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), sc, mm);
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
                    tmem_st16(t_s + 16 * half, hi);
                    tmem_st16(t_s + 32 + 16 * half, lo);
                    tmem_wait_st();
                }
                // The word of the tile's non-finite values: a group's own where it is alone on the tile; on
                // a pair, one for both groups, chosen by what they both count, the CTA's tiles (their own
                // counts g differ by one after a single row tile of an odd number of tiles).
                unsigned long long special = 0ull, *flags = &odd[alternate ? 2 * group + (g & 1) : (tile0 + i) & 1];
                const int who = alternate || NG == 1 ? gtid : tid, whole_id = alternate ? 2 + group : 1;
                const int whole_n = alternate || NG == 1 ? kGroupThreads : P::ROWS;
                if (edge) {
                    // Value rows past the last token hold anything: zeros in their place.  The
                    // draft's values may be unseen by some rows, whose zero weights must not meet
                    // an infinity or NaN: those elements are zeroed too, and added below to
                    // the rows that do see them.  (All threads that use the tile do this together.)
                    const uint32_t vpos = 2 * (tile0 + i) + 1, stage = vpos % P::NST;
                    wait_rows(&full[stage], (vpos / P::NST) & 1);
                    uint8_t *sv = ring + stage * P::STAGE;
                    const int from = s.total ? max(0, s.len - j0) : 0, live = s.total - j0;
                    for (int y = who + from * (D / 8); y < kKeys * (D / 8); y += whole_n) {
                        const int r = y / (D / 8), c = y % (D / 8);
                        uint4 *at = reinterpret_cast<uint4 *>(sv + (c >> 3) * (kKeys * 128) + sw128(r, c & 7));
                        if (r >= live) {
                            *at = make_uint4(0u, 0u, 0u, 0u);
                            continue;
                        }
                        // an exponent of ones carries into its half's sign bit
                        const uint4 w = *at;
                        const uint4 c4 = make_uint4((w.x & 0x7f807f80u) + 0x00800080u, (w.y & 0x7f807f80u) + 0x00800080u,
                                                    (w.z & 0x7f807f80u) + 0x00800080u, (w.w & 0x7f807f80u) + 0x00800080u);
                        if ((c4.x | c4.y | c4.z | c4.w) & 0x80008000u) {
                            auto keep = [](uint32_t v, uint32_t c) {
                                return v & ~((c & 0x80000000u ? 0xffff0000u : 0u) | (c & 0x8000u ? 0xffffu : 0u));
                            };
                            *at = make_uint4(keep(w.x, c4.x), keep(w.y, c4.y), keep(w.z, c4.z), keep(w.w, c4.w));
                            atomicOr(flags, 1ull << r);
                        }
                    }
                    fence_proxy_async();
                    bar_sync(whole_id, whole_n);
                    special = *flags;
                }
                tc_fence_before();
                mbar_arrive(&pf[g & 1]);
                if (special) {                      // read from one word by all threads that use the tile
                    wait_rows(&od[g & 1], (g >> 1) & 1);
                    if (warp_live) {
                        const int sh = s.len - j0;
                        const uint64_t view = sh >= 64 ? 0ull : sh >= 0 ? bits << sh : sh > -64 ? bits >> -sh : 0ull;
                        add_odd_values<D>(a, t_o, s.slot, s.h, j0, half, special, used ? view & special : 0ull);
                    }
                    bar_sync(whole_id, whole_n);
                    if (who == 0) *flags = 0ull;
                    bar_sync(whole_id, whole_n);
                }
            }
            tile0 += s.count;
            more = cur.next(st, ta.row_tiles, NQ, next);
            next_bits = more ? word_of(next) : 0ull;
            // ---- the unit's result, or this CTA's part of it
            if (mine > 0) wait_rows(&od[(g - 1) & 1], ((g - 1) >> 1) & 1);
            const bool whole = s.count == s.tiles;
            if (tid == P::ROWS - 1 && s.first == 0) {             // the unit's record
                const int tile = (s.b * a.s.Hkv + s.h) * ta.row_tiles + s.rt;
                if (ta.by_cta) {
                    if (!whole) ta.rec[blockIdx.x] = make_int4(tile, s.nq, blockIdx.x, parts_of(*cut, s));
                } else {
                    ta.rec[tile] = make_int4(tile, s.nq, blockIdx.x, whole ? 0 : parts_of(*cut, s));
                    if (s.nq == 2) ta.rec[tile + 1] = make_int4(0, 0, 0, 0);
                }
            }
            // the row's threads: two, or four when both groups worked on it (each group's O scaled to
            // the common maximum)
            xm[tid] = m;
            xl[tid] = l;
            tc_fence_before();
            bar_sync(alternate ? 1 : 2 + group, alternate ? P::ROWS : kGroupThreads);
            tc_fence_after();
            l += xl[tid ^ 128];                     // (commutative: the same in all the row's threads)
            float f0 = 1.f, f1 = 0.f;               // of this group's O, of the other's
            const bool both = alternate && s.count > 1;
            if (both) {
                const float m1 = xm[tid ^ 256], mn = fmaxf(m, m1), ms = mn == -INFINITY ? 0.f : mn;
                f0 = ex2(m - ms);
                f1 = ex2(m1 - ms);
                const float l0 = l * f0, l1 = (xl[tid ^ 256] + xl[tid ^ 384]) * f1;
                l = group == 0 ? l0 + l1 : l1 + l0;
                m = mn;
            }
            const bool writer = !alternate || mine > 0;                    // a single tile leaves one group without
            if (writer && __any_sync(0xffffffffu, exists)) {
                const int cols = both ? D / 4 : D / 2, c0 = both ? (2 * group + half) * (D / 4) : half * (D / 2);
                const uint32_t o_mine = t_lane + 2 * kKeys + c0;
                const uint32_t o_other = both ? o_mine + (group == 0 ? P::TCOLS : -P::TCOLS) : o_mine;
                const float inv = !whole ? 1.f : used && (l > 0.f || l != l) ? 1.f / l : 0.f;
                f0 *= inv;
                f1 *= inv;
                const size_t orow = (static_cast<size_t>(b) * a.s.T + t) * a.Hq + s.h * a.G + qh;
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + orow * D + c0);
                float *slot = ta.part + static_cast<size_t>((2 * blockIdx.x + (s.first == 0 ? 1 : 0)) * NQ + (NQ == 2 && s.nq == 2 ? group : 0)) *
                                            (D + 2) * ta.rp + r_in;
#pragma unroll 1
                for (int c = 0; c < cols; c += 16) {
                    float o[16];
                    tmem_ld16(o_mine + c, o);
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] *= f0;
                    if (both) {
                        float o1[16];
                        tmem_ld16(o_other + c, o1);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = fmaf(o1[k], f1, o[k]);
                    }
                    if (exists) {
                        if (whole) {
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                uint32_t h[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const __nv_bfloat162 y = __floats2bfloat162_rn(o[8 * k + 2 * e], o[8 * k + 2 * e + 1]);
                                    h[e] = inv != 0.f ? *reinterpret_cast<const uint32_t *>(&y) : 0u;
                                }
                                dst[c / 8 + k] = make_uint4(h[0], h[1], h[2], h[3]);
                            }
                        } else {                    // column by column: a warp's rows are one run of memory
#pragma unroll
                            for (int k = 0; k < 16; ++k) slot[static_cast<size_t>(c0 + c + k) * ta.rp] = o[k];
                        }
                    }
                    __syncwarp();
                }
                if (exists && c0 == 0) {
                    if (whole) {
                        if (a.lse) a.lse[orow] = used ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
                    } else {
                        slot[static_cast<size_t>(D) * ta.rp] = used ? m : -INFINITY;
                        slot[static_cast<size_t>(D + 1) * ta.rp] = used ? l : 0.f;
                    }
                }
            }
            tc_fence_before();
            if (NG == 1) bar_sync(1, P::ROWS);      // the exchange words have been read
            s = next;
            bits = next_bits;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort) {                                   // nothing of this CTA runs on when it ends
        if (warp >= P::LOAD_WARP && warp < P::MMA_WARP) {
            for (uint32_t t = pos > P::NST / 2 ? pos - P::NST / 2 : 0; t < pos; ++t) {
                const uint32_t k = 2 * t + warp - P::LOAD_WARP;
                if (!mbar_wait(&full[k % P::NST], (k / P::NST) & 1) && lane == 0) atomicOr(a.s.status, GDN_STATUS_DRAIN);
            }
        } else if (warp >= P::MMA_WARP) {
            if (issued) {
                if (elect_one()) mma_commit(&drain[warp - P::MMA_WARP]);
                if (!mbar_wait(&drain[warp - P::MMA_WARP], 0)) atomicOr(a.s.status, GDN_STATUS_DRAIN);
            }
            if (queries > 0 && !mbar_wait(q_full, (queries - 1) & 1)) atomicOr(a.s.status, GDN_STATUS_DRAIN);
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
    }
    if (warp == P::LOAD_WARP) tmem_dealloc(tmem, P::TMEM_COLS);
}

// ------------------------------------------------------------------- the join
// A task is 32 rows (a lane each) and 8 output columns of a split unit; `wide` warps (a power of
// two, about one for every four parts) take its parts in turn, and the first of them joins
// their sums in a fixed order.  gridDim.y CTAs share a record's tasks.
template <int D, int NQ, int kJoinWarps>
__global__ void __launch_bounds__(kJoinWarps * 32, kJoinWarps == 8 ? 3 : 1) verify_tc_join_kernel(const TcArgs ta, int grid)
{
    const AttnArgs &a = ta.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __shared__ float sums[kJoinWarps][10][32];
    pdl_wait();
    pdl_release();
    const int4 rec = ta.rec[blockIdx.x];
    const int cta = rec.z, parts = rec.w;
    if (parts < 2 || cta < 0 || cta + parts > grid || rec.x < 0 || rec.y < 1 || rec.y > NQ) return;
    const int rt0 = rec.x % ta.row_tiles, bh = rec.x / ta.row_tiles, h = bh % a.s.Hkv, b = ta.b0 + bh / a.s.Hkv;
    if (b >= ta.b0 + ta.nb || rt0 + rec.y > ta.row_tiles) return;
    int wide = 1;
    while (wide < kJoinWarps && wide * 4 < parts) wide *= 2;
    const int at_once = kJoinWarps / wide, mine = warp / wide, sub = warp % wide;
    const int per_tile = ta.tpt * a.G, tasks = rec.y * (ta.rp / 32) * (D / 8), slot = (D + 2) * ta.rp;
    for (int t0 = blockIdx.y * at_once; t0 < tasks; t0 += gridDim.y * at_once) {
        const int task = t0 + mine, c0 = task % (D / 8) * 8, rg = task / (D / 8);
        const int place = rg / (ta.rp / 32), r = rg % (ta.rp / 32) * 32 + lane, rt = rt0 + place;
        const int rows = min(per_tile, (a.s.T - rt * ta.tpt) * a.G);
        const bool exists = task < tasks && r < rows;
        float m = -INFINITY, l = 0.f, acc[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = 0.f;
        if (exists) {
            // part k: the first slot of CTA cta + k, but the second one of the first CTA
            const float *first = ta.part + static_cast<size_t>(2 * cta * NQ + place) * slot + r;
            const float *col = first + c0 * ta.rp;
#pragma unroll 1
            for (int k0 = sub; k0 < parts; k0 += 4 * wide) {             // four parts requested at a time
                float mk[4], lk[4], x[4][8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = k0 + i * wide;
                    const bool in = k < parts;
                    const int at = (2 * k + (k == 0 ? 1 : 0)) * NQ * slot;        // < 2^31: 2 N NQ (D + 2) rp floats
                    mk[i] = in ? first[at + D * ta.rp] : -INFINITY;
                    lk[i] = in ? first[at + (D + 1) * ta.rp] : 0.f;
#pragma unroll
                    for (int c = 0; c < 8; ++c) x[i][c] = in ? col[at + c * ta.rp] : 0.f;
                }
                const float mn = fmaxf(m, fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3])));
                const float ms = mn == -INFINITY ? 0.f : mn, f0 = ex2(m - ms);
                m = mn;
                l *= f0;
#pragma unroll
                for (int c = 0; c < 8; ++c) acc[c] *= f0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = ex2(mk[i] - ms);
                    l = fmaf(lk[i], f, l);
#pragma unroll
                    for (int c = 0; c < 8; ++c) acc[c] = fmaf(x[i][c], f, acc[c]);
                }
            }
        }
        if (wide > 1) {                                                  // the same in the whole CTA
            sums[warp][8][lane] = m;
            sums[warp][9][lane] = l;
#pragma unroll
            for (int c = 0; c < 8; ++c) sums[warp][c][lane] = acc[c];
            __syncthreads();
            if (sub == 0) {
                for (int w = 1; w < wide; ++w) {
                    const float mk = sums[warp + w][8][lane], mn = fmaxf(m, mk), ms = mn == -INFINITY ? 0.f : mn;
                    const float f0 = ex2(m - ms), f1 = ex2(mk - ms);
                    m = mn;
                    l = l * f0 + sums[warp + w][9][lane] * f1;
#pragma unroll
                    for (int c = 0; c < 8; ++c) acc[c] = acc[c] * f0 + sums[warp + w][c][lane] * f1;
                }
            }
            __syncthreads();
        }
        if (sub != 0 || !exists) continue;
        const int t = rt * ta.tpt + r / a.G;
        const size_t orow = (static_cast<size_t>(b) * a.s.T + t) * a.Hq + h * a.G + r % a.G;
        const bool any = l > 0.f || l != l;                              // rows not in use: l = 0 in every part
        const float inv = any ? 1.f / l : 0.f;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 y = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
            w[e] = any ? *reinterpret_cast<const uint32_t *>(&y) : 0u;
        }
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + orow * D + c0) = make_uint4(w[0], w[1], w[2], w[3]);
        if (a.lse && c0 == 0) a.lse[orow] = any ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
}

// ------------------------------------------------------------------- host side
// A layer's keys or values: as [d / 64][rows of all pages][64] in boxes of a tile, in the column atoms that
// the MMAs read; where the pages are shorter, as [rows][d] in boxes of a page's rows of one atom.
bool page_map(CUtensorMap *m, const void *base, const gdn_page_cache *c) {
    auto fn = encode_fn();
    if (!fn) return false;
    const bool tile = c->page >= kKeys;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(tile ? 64 : c->d), static_cast<cuuint64_t>(c->n_page) * c->Hkv * c->page,
                          static_cast<cuuint64_t>(c->d) / 64};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(c->d) * 2, 128};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(tile ? kKeys : c->page), static_cast<cuuint32_t>(c->d) / 64};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, tile ? 3 : 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The queries as [B T][Hq][d]; boxes of a row tile's tokens and a key head's queries.
bool query_map(CUtensorMap *m, const void *base, const gdn_page_cache *c, const gdn_attn_dims *d) {
    auto fn = encode_fn();
    if (!fn) return false;
    const int G = d->Hq / c->Hkv;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(c->d), static_cast<cuuint64_t>(d->Hq),
                          static_cast<cuuint64_t>(d->B) * d->T};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(c->d) * 2, static_cast<cuuint64_t>(c->d) * 2 * d->Hq};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(kRows / G)};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
int tc_tokens(const gdn_page_cache *c, const gdn_attn_dims *d) { return kRows / (d->Hq / c->Hkv); }
int tc_row_tiles(const gdn_page_cache *c, const gdn_attn_dims *d) {
    return (d->T + tc_tokens(c, d) - 1) / tc_tokens(c, d);
}
int tc_rp(const gdn_page_cache *c, const gdn_attn_dims *d) {
    const int t = d->T < tc_tokens(c, d) ? d->T : tc_tokens(c, d);
    return (t * (d->Hq / c->Hkv) + 31) / 32 * 32;
}
// Row tiles of a unit: pairs where there are any and TMEM has room for two groups.
int tc_nq(const gdn_page_cache *c, const gdn_attn_dims *d) { return c->d != 256 && tc_row_tiles(c, d) > 1 ? 2 : 1; }
// Sequences of one launch: its table has kMaxSeqs entries, its work is counted in 32 bits.
int tc_seqs(const gdn_page_cache *c, const gdn_attn_dims *d) {
    const long long tiles = (static_cast<long long>(c->max_pages) * c->page + kKeys - 1) / kKeys;   // <= 2^18
    const long long most = (1ll << 30) / (tiles * c->Hkv * tc_row_tiles(c, d));                     // >= 1
    const int n = most < kMaxSeqs ? static_cast<int>(most) : kMaxSeqs;
    return d->B < n ? d->B : n;
}
// CTAs of a launch over nb sequences: one per SM, but no more than there may be tiles.
int tc_grid(const gdn_page_cache *c, const gdn_attn_dims *d, int nb) {
    const long long tiles = (static_cast<long long>(c->max_pages) * c->page + kKeys - 1) / kKeys;
    const long long all = tiles * nb * c->Hkv * tc_row_tiles(c, d);
    const int sms = sm_count();
    return static_cast<int>(all < sms ? all : sms);
}
// Records of a launch: one per CTA, or per row tile where those are fewer.
int tc_records(const gdn_page_cache *c, const gdn_attn_dims *d, int nb, bool *by_cta) {
    const long long units = static_cast<long long>(nb) * c->Hkv * tc_row_tiles(c, d);
    const int grid = tc_grid(c, d, nb);
    *by_cta = grid < units;
    return *by_cta ? grid : static_cast<int>(units);
}
size_t rec_bytes(const gdn_page_cache *c, const gdn_attn_dims *d) {
    bool by_cta;
    return static_cast<size_t>(tc_records(c, d, tc_seqs(c, d), &by_cta)) * sizeof(int4);
}

template <int D, int NQ>
int launch_tc(const gdn_page_cache *c, const gdn_attn_dims *d, const AttnArgs &a, cudaStream_t s) {
    using P = TcPlan<D, NQ>;
    CUtensorMap mq, mk, mv;
    if (!query_map(&mq, a.q, c, d) || !page_map(&mk, a.k, c) || !page_map(&mv, a.v, c)) return GDN_ERR_LAUNCH;
    if (cudaFuncSetAttribute(verify_tc_kernel<D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::BYTES) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    TcArgs ta{a, 0, 0, tc_tokens(c, d), tc_row_tiles(c, d), tc_rp(c, d), reinterpret_cast<int4 *>(a.ws), 0,
              reinterpret_cast<float *>(reinterpret_cast<char *>(a.ws) + rec_bytes(c, d))};
    const int step = tc_seqs(c, d);
    for (ta.b0 = 0; ta.b0 < d->B; ta.b0 += step) {
        ta.nb = d->B - ta.b0 < step ? d->B - ta.b0 : step;
        const int grid = tc_grid(c, d, ta.nb);
        bool by_cta;
        const int recs = tc_records(c, d, ta.nb, &by_cta), tasks = NQ * (ta.rp / 32) * (D / 8);
        ta.by_cta = by_cta;
        // Where records may be of many parts, 16 warps take a task's parts (one sequence of 131,001
        // tokens, 2 key heads, 76 parts: 36.1 us against 38.9 with 8); elsewhere 8 do (700 tokens, 11 parts:
        // 9.9 us against 10.7 with 16; 32 sequences: 42.8 against 44.3).  Two or three waves of CTAs.
        const bool few = grid >= 32 * recs;
        const int share = (few ? 4 : 8) * sm_count() / recs;
        const dim3 jgrid(recs, share < 1 ? 1 : share > tasks ? tasks : share);
        if (launch_pdl(verify_tc_kernel<D, NQ>, dim3(grid), dim3(P::THREADS), P::BYTES, s, mq, mk, mv, ta) != cudaSuccess ||
            (few ? launch_pdl(verify_tc_join_kernel<D, NQ, 16>, jgrid, dim3(16 * 32), 0, s, ta, grid)
                 : launch_pdl(verify_tc_join_kernel<D, NQ, 8>, jgrid, dim3(8 * 32), 0, s, ta, grid)) != cudaSuccess)
            return GDN_ERR_LAUNCH;
    }
    return GDN_OK;
}

}  // namespace

int64_t attn_tc_workspace(const gdn_page_cache *c, const gdn_attn_dims *d) {
    return static_cast<int64_t>(rec_bytes(c, d)) +
           static_cast<int64_t>(2) * tc_grid(c, d, tc_seqs(c, d)) * tc_nq(c, d) * (c->d + 2) * tc_rp(c, d) * 4;
}

int attn_tc_verify(const gdn_page_cache *c, const gdn_attn_dims *d, const AttnArgs &a, cudaStream_t s) {
    const bool pairs = tc_nq(c, d) == 2;
    if (c->d == 256) return launch_tc<256, 1>(c, d, a, s);
    if (c->d == 128) return pairs ? launch_tc<128, 2>(c, d, a, s) : launch_tc<128, 1>(c, d, a, s);
    return pairs ? launch_tc<64, 2>(c, d, a, s) : launch_tc<64, 1>(c, d, a, s);
}

}  // namespace gdn
