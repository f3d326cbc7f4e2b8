// pa_cluster.cuh -- how many CTAs share a tile's key blocks in the windowed and
// 8-bit multi-query calls (plain C++: the host tests compile it too).
#pragma once

#include <cstdint>

namespace pa {

constexpr int kSplitMinBlocks = 4;  // key blocks worth a CTA of their own
constexpr int kMaxRanks = 16;       // CTAs of a cluster, at most

struct ClusterChoice {
    unsigned ranks;  // CTAs a tile, 1: no cluster
    bool alone;      // a CTA has its SM to itself
};

// CTAs that share a tile's key blocks: two while they fit two per SM, more (to
// kMaxRanks) while they fit one per SM, as long as the longest row that the tables
// and the window allow gives each its blocks.  The lengths are on the device, so
// wide tables cost short contexts the larger launch.  Measured without and with
// it, bf16 and 8-bit cache, 32/8 heads of 128: one token over 16,000 tokens 237
// and 347 -> 29 and 42 us; 16 sequences of 4 rows over 2,000 37 and 54 -> 32 and
// 41 us; heads of 64 over 60 tokens of 65,536 possible 6.4 and 6.9 -> 8.6 and 9.8
// us; 8 sequences of 16 rows over 500, heads of 64, 10.9 and 12.2 -> 12.5 and 13.0,
// over 1,000 16.4 and 19.1 -> 15.1 and 16.4.
inline unsigned wanted_ranks(unsigned tiles, int64_t blocks, int64_t sms) {
    unsigned n = 1;
    while (n < unsigned(kMaxRanks) && int64_t(tiles) * n * 2 <= (n == 1 ? 2 * sms : sms) &&
           blocks >= int64_t(n) * 2 * kSplitMinBlocks)
        n *= 2;
    return n;
}

// The wanted cluster, or the largest half of it that the device holds: clusters
// need their CTAs' room on one group of SMs, and a part of a GPU (a partition, a
// device that others share) may have less.  held(n, alone): the clusters of n CTAs
// that the device holds at once, with `alone` each CTA taking an SM's shared memory
// for itself; that is asked for only where all of a call's clusters find room so.
// (Two CTAs to an SM share its issue slots while other SMs idle: 8-bit cache, one
// sequence of 4 rows over 16,000 tokens, 4 heads of 128, 35.5 us, alone 30.2 us; 4 of
// 4 rows over 8,000, 8 heads, 67.7 and 53.3 us.  Eight clusters of 16 do not fit alone
// on 148 SMs: 61.9 us in two turns, 45.1 us two to an SM.)
template <class Held>
ClusterChoice choose_cluster(unsigned tiles, int64_t blocks, int64_t sms, Held held) {
    unsigned n = wanted_ranks(tiles, blocks, sms);
    while (n > 1 && held(n, false) < 1) n /= 2;
    return {n, n > 1 && int64_t(tiles) <= held(n, true)};
}

}  // namespace pa
