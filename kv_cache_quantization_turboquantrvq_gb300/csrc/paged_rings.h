// paged_rings.h - rings of shared-memory slots between the roles of a kernel, and the
// walk of the weighing kernel's product warps over theirs.  No device code: the walk
// also runs against modelled barriers on the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define VQ_HD __host__ __device__ __forceinline__
#else
#define VQ_HD inline
#endif

namespace vq {
namespace {

// Position in a ring of N barriers: slot and the parity of its current pass.
template <int N> struct PgRing {
    int s = 0;
    uint32_t par = 0;
    VQ_HD void step()
    {
        if (++s == N) {
            s = 0;
            par ^= 1u;
        }
    }
};

// Rings of the weighing kernel, over a 16-bit cache and over codes.
template <bool Q8> struct WgRings {
    static constexpr int KST = Q8 ? 3 : 4;   // key tiles
    static constexpr int QST = 3;            // query tiles
    static constexpr int RAW = Q8 ? 2 : 0;   // tiles of codes
    static constexpr int LST = 2;            // rows' -lse
    static constexpr int IST = 4;            // units known ahead
    static constexpr int SST = 2;            // score tiles of a group
    static constexpr int CONV = Q8 ? 4 : 0;  // warps that convert codes
    static constexpr int READERS = 2;        // arrivals that free a key or a query tile: one of each product warp
};

// One unit of product warp g (0, 1): its key tile g (where the unit has it; `two`: it
// has both) against `count` query tiles.
//
// Each warp passes every tile of both rings, the other warp's key tile too: it waits
// until that is there and gives it back at once.  A barrier's parity tells two passes
// of a slot apart, not three.  A warp that stepped over the other's tiles would take
// the pass before its own for its own where a slot changes hands (units of one and of
// two tiles in turn) and multiply what is not there yet; and one that waited but did
// not have to be waited for could miss a pass.
//
// ops: keys(ring), queries(ring), scores(ring): wait for a key tile, a query tile, a free
// score tile (both: queries and scores, asked together), false: give up;
// product(keys, queries, scores); keys_used, queries_used(ring): free the tile when the
// products so far are done; keys_passed, queries_passed(ring): now.
template <class Keys, class Queries, class Scores, class Ops>
VQ_HD bool wg_products(Ops &&ops, Keys &ks, Queries &qs, Scores &ss, int g, bool two, int count)
{
    const bool mine = g == 0 || two;
    auto pass = [&]() -> bool {
        if (!ops.keys(ks)) return false;
        ops.keys_passed(ks);
        ks.step();
        return true;
    };
    if (g == 1 && !pass()) return false;
    if (mine && !ops.keys(ks)) return false;
    for (int j = 0; j < count; ++j) {
        if (mine) {
            if (!ops.both(qs, ss)) return false;
            ops.product(ks, qs, ss);
            ss.step();
            ops.queries_used(qs);
        } else {
            if (!ops.queries(qs)) return false;
            ops.queries_passed(qs);
        }
        qs.step();
    }
    if (mine) {
        ops.keys_used(ks);
        ks.step();
    }
    return g == 1 || !two || pass();
}

}  // namespace
}  // namespace vq
