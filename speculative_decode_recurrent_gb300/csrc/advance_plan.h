// advance_plan.h -- how gdn_replay_advance cuts long bf16 chunks into launches (host arithmetic alone, so that it can be
// compiled and checked without a GPU; not part of the public ABI).
#pragma once

#include <stdint.h>

namespace gdn {

// Tokens of a chunk, and the workspace: what is beyond it follows in further launches.
constexpr int kChunkTokens = 64;
constexpr int64_t kAdvanceBudget = 768ll << 20;

// B sequences of T tokens, H heads of dk x dv, on a GPU of `sms`; `unit`: bytes of a chunk of a head.
struct AdvancePlan {
    int64_t unit;
    int B, H, dv, sms;
    int all;                    // chunks of T tokens
    int seqs;                   // sequences of a launch
    int most;                   // chunks of a launch, by the workspace
    int first, n;               // the first launch's chunks, launches that were counted on
    double r;                   // beside c chunks of the walk the first kernel has time for r c

    // Value columns of a walk's CTA: slices of 32 while each has an SM of its own, heads beyond (which need 128 value columns);
    // slices of 16 where even those have (8192 tokens of 16 heads: 172 us of walking, against 205 with 32) and no first kernel is to run beside
    // them, for which they leave no SMs.
    int walk_columns(bool last) const {
        const long long heads = static_cast<long long>(seqs) * H;
        return last && heads * (dv / 16) <= sms ? 16 : dv == 128 && heads * (dv / 32) > sms ? 128 : 32;
    }
    // Chunks of launch i, after one of `size`, with `rest` left.
    int next(int i, int size, int rest) const {
        const double c = i >= n - 1 ? rest : i == 0 ? first : size * r;
        const int room = most < rest ? most : rest;
        return c < 1 ? 1 : c > room ? room : static_cast<int>(c);
    }
    // Two workspaces take turns, the first of as many chunks as its largest launch has; both together have no more than all chunks, nor
    // than twice the most of a launch.  (Where sequences come in several groups the turns go on, so each has room for any launch.)
    int first_room() const {
        const bool groups = seqs < B;
        int room = 0, size = 0;
        for (int i = 0, rest = all; rest > 0; ++i, rest -= size) {
            size = next(i, size, rest);
            if ((groups || i % 2 == 0) && size > room) room = size;
        }
        return room;
    }
    int64_t room() const {                          // of both; does not fall where T grows
        const bool groups = seqs < B;
        const int64_t both = 2ll * (groups && all < most ? all : most);
        return groups || both < all ? both : all;
    }
    int64_t workspace() const { return unit * H * seqs * room(); }
};

// The chunks come in launches of the two kernels, so that the first one's work for the next chunks runs beside the walk,
// on SMs that the walk leaves free: beside c chunks of it there is time for r c.  The first launch's own work runs alone (5.3 us a
// chunk and SM), as does what of a later one's the walk before it leaves no time for, and each launch costs some 12 us (by heads
// 20: more state comes in and goes out); their number and the first one's size follow from that.  8192 tokens of 16 heads:
// 224 us in three launches, 252 in one, 250 in six; 8 prompts of 16 heads, whose walk leaves few SMs: 218 in one, 225 in two.
// These times are of 16 heads of 128 x 128 and stand for the other sizes too.  (With 64 key dims a walk's CTA leaves shared memory for one of the
// first kernel on its SM, but no TMEM: one of the two then waits for the other's columns, and less runs beside.)
// Where the workspace holds fewer chunks than a plan wants, its launches are as large as that lets them be (16 prompts of 4096
// tokens, 16 heads: 966 us in four; in 44, all but the first of one chunk, 1811).
inline AdvancePlan advance_plan(int B, int T, int H, int dv, int64_t unit, int sms) {
    AdvancePlan p{unit, B, H, dv, sms < 1 ? 1 : sms, (T + kChunkTokens - 1) / kChunkTokens, 1, 1, 1, 1, 0.0};
    const int64_t seqs = kAdvanceBudget / 2 / (unit * H);
    p.seqs = static_cast<int>(seqs < 1 ? 1 : seqs < B ? seqs : B < 1 ? 1 : B);
    const int64_t most = kAdvanceBudget / 2 / (unit * H * p.seqs);
    p.most = static_cast<int>(most < 1 ? 1 : most < p.all ? most : p.all);
    const int cols = p.walk_columns(false);
    const double units = static_cast<double>(p.seqs) * H, ctas = units * (dv / cols), free = ctas < p.sms ? 1 - ctas / p.sms : 0;
    const double prep = 16.0 / 3 * units / p.sms, walk = cols == 128 ? 3.4 : 1.6, launch = cols == 128 ? 20.0 : 12.0;        // us a chunk, a launch
    p.r = walk * free / prep;
    double best = 1e30, sum = 0, pow = 1;
    int first = p.all, n = 1;
    for (int k = 1; k <= 6; ++k, pow *= p.r) {
        sum += pow;
        p.n = k;
        p.first = static_cast<int>(p.all / sum + 0.999);
        double cost = p.most < p.all ? 0 : prep * p.all / sum + launch * k;
        if (p.most < p.all)                         // launches that the workspace cuts short: one by one
            for (int i = 0, rest = p.all, size = 0; rest > 0; ++i, rest -= size) {
                const double beside = size * p.r;
                size = p.next(i, size, rest);
                cost += launch + (size > beside ? prep * (size - beside) : 0);
            }
        if (cost < best) {
            best = cost;
            first = p.first;
            n = k;
        }
    }
    p.first = first;
    p.n = n;
    return p;
}

}  // namespace gdn
