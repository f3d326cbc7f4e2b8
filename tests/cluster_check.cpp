// Host check of csrc/pa_cluster.cuh over many calls and devices: never a cluster
// that the device does not hold, never alone where not all of a call's find room,
// the wanted size wherever the device holds it, at least kSplitMinBlocks blocks a CTA.
#include <cstdio>
#include <initializer_list>

#include "../paged_kv_attention_36_b200/csrc/pa_cluster.cuh"

int main() {
    long checked = 0;
    for (unsigned tiles = 1; tiles < 400; tiles += tiles < 20 ? 1 : 7)
        for (int64_t blocks : {0LL, 1LL, 7LL, 8LL, 15LL, 16LL, 40LL, 127LL, 128LL, 250LL, 100000LL})
            for (int sms : {1, 8, 20, 132, 148})
                for (unsigned largest = 1; largest <= 16; largest *= 2)     // cluster the device holds
                    for (int alone_room : {0, 1, 7, 1000}) {                // and how many of them alone
                        auto held = [&](unsigned n, bool alone) -> int64_t {
                            return n > largest ? 0 : alone ? alone_room : 2 * alone_room + 1;
                        };
                        const unsigned want = pa::wanted_ranks(tiles, blocks, sms);
                        const pa::ClusterChoice c = pa::choose_cluster(tiles, blocks, sms, held);
                        const bool ok = c.ranks >= 1 && c.ranks <= want && want <= unsigned(pa::kMaxRanks) &&
                                        (c.ranks == 1 || c.ranks <= largest) &&
                                        c.ranks == (want < largest ? want : largest) &&
                                        (want == 1 || blocks >= int64_t(want) * pa::kSplitMinBlocks) &&
                                        (!c.alone || (c.ranks > 1 && tiles <= unsigned(alone_room)));
                        if (!ok) {
                            std::printf("tiles %u blocks %lld sms %d largest %u room %d: ranks %u alone %d\n", tiles,
                                        (long long)blocks, sms, largest, alone_room, c.ranks, c.alone);
                            return 1;
                        }
                        ++checked;
                    }
    std::printf("ok %ld\n", checked);
    return 0;
}
