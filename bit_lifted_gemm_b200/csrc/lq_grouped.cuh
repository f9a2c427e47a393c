// What the two kernels of the grouped products share: the walk over their units of
// work on ragged groups that only the device knows.
#pragma once

#include "lq_internal.h"

namespace lq {

// A unit: one expert, up to `per` of its slots, one of nblk blocks of weight rows.
struct Unit {
    int e, slot0, slots, blk;
};

// Walks the units in order of expert; every warp that needs units walks on its own,
// with ascending unit numbers. Experts' ranges are cut to 0..n and taken as
// empty when they descend. A window of 32 experts, one to a lane, is kept between calls, and
// divisions are of 32 bits wherever the numbers are: a block of few rows starts with a walk in
// every warp, and with 64-bit divisions it took 0.5 us.
struct UnitWalk {
    long long before = 0;  // units of the experts before e0
    int e0 = -32;          // first expert of the current window
    int lo, hi;            // this lane's expert: its slots
    long long upto = 0;    // units of the window up to it

    // Unit number `unit`, if there is one (warp-collective). Within an expert the
    // slots run fastest if slots_fastest (the blocks' weights are then read again
    // while they are in L2), else the blocks (the slots' rows of u are).
    template <bool slots_fastest>
    __device__ __forceinline__ bool find(const GroupedCall& c, int per, int nblk, long long unit, int lane, Unit& u) {
        for (;;) {
            const unsigned past = e0 < 0 ? 0 : __ballot_sync(0xffffffffu, before + upto > unit);
            if (past) {
                const int src = __ffs(past) - 1;
                const int first = __shfl_sync(0xffffffffu, lo, src), end = __shfl_sync(0xffffffffu, hi, src);
                const int passes = (end - first + per - 1) / per, by = slots_fastest ? passes : nblk;
                const long long rest = unit - before - __shfl_sync(0xffffffffu, upto, src) + (long long)passes * nblk;
                const int slow = rest >> 32 ? (int)(rest / by) : (int)((unsigned)rest / (unsigned)by);
                const int fast = (int)(rest - (long long)slow * by);
                u.e = e0 + src;
                u.slot0 = first + (slots_fastest ? fast : slow) * per;
                u.slots = min(per, end - u.slot0);
                u.blk = slots_fastest ? slow : fast;
                return true;
            }
            if (e0 >= 0) before += __shfl_sync(0xffffffffu, upto, 31);
            e0 += 32;
            if (e0 >= c.experts) return e0 = c.experts, upto = 0, false;
            const int mine = e0 + lane;
            lo = hi = 0;
            if (mine < c.experts) {
                lo = c.offsets ? min(max(__ldg(c.offsets + mine), 0), c.n) : 0;
                hi = c.offsets ? max(min(__ldg(c.offsets + mine + 1), c.n), lo) : c.n;
            }
            upto = (long long)((hi - lo + per - 1) / per) * nblk;
            for (int d = 1; d < 32; d <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += x;
            }
        }
    }
};

}  // namespace lq
