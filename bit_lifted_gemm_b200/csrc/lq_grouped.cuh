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
// empty when they descend.
struct UnitWalk {
    long long before = 0;  // units of the experts before e0
    int e0 = 0;            // first expert of the current window of 32

    // Unit number `unit`, if there is one (warp-collective). Within an expert the
    // slots run fastest if slots_fastest (the blocks' weights are then read again
    // while they are in L2), else the blocks (the slots' rows of u are).
    template <bool slots_fastest>
    __device__ __forceinline__ bool find(const GroupedCall& c, int per, int nblk, long long unit, int lane, Unit& u) {
        while (e0 < c.experts) {
            const int mine = e0 + lane;
            int lo = 0, hi = 0;
            if (mine < c.experts) {
                lo = c.offsets ? min(max(__ldg(c.offsets + mine), 0), c.n) : 0;
                hi = c.offsets ? max(min(__ldg(c.offsets + mine + 1), c.n), lo) : c.n;
            }
            const long long units = (long long)((hi - lo + per - 1) / per) * nblk;
            long long upto = units;
            for (int d = 1; d < 32; d <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += x;
            }
            const unsigned past = __ballot_sync(0xffffffffu, before + upto > unit);
            if (past) {
                const int src = __ffs(past) - 1;
                const long long rest = unit - before - __shfl_sync(0xffffffffu, upto - units, src);
                lo = __shfl_sync(0xffffffffu, lo, src);
                hi = __shfl_sync(0xffffffffu, hi, src);
                const int by = slots_fastest ? (hi - lo + per - 1) / per : nblk;
                const int slow = (int)(rest / by), fast = (int)(rest - (long long)slow * by);
                u.e = e0 + src;
                u.slot0 = lo + (slots_fastest ? fast : slow) * per;
                u.slots = min(per, hi - u.slot0);
                u.blk = slots_fastest ? slow : fast;
                return true;
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
            e0 += 32;
        }
        return false;
    }
};

}  // namespace lq
