// Brute-force check of pa_window.cuh on the host: the listed pages are exactly
// those that hold a seen token, visible_tokens is the definition, list order
// keeps the prefill kernels' interval form (a query sees list tokens [0, a) and
// [lo, hi)), and cut segments are covered once by the CTAs segment_owners names.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../paged_kv_attention_36_b200/csrc/pa_split.cuh"
#include "../paged_kv_attention_36_b200/csrc/pa_window.cuh"

using namespace pa;

static bool sees(int t, int p, int window, int sinks) { return t <= p && (t > p - window || t < sinks); }

#define CHECK(x)                                                  \
    do {                                                          \
        if (!(x)) {                                               \
            std::printf("failed: %s (line %d)\n", #x, __LINE__); \
            return 1;                                             \
        }                                                         \
    } while (0)

int main() {
    std::srand(7);
    const int all = 0x7fffffff;
    for (int trial = 0; trial < 60000; ++trial) {
        const int L = 1 + std::rand() % 200;
        const int window = std::rand() % 8 == 0 ? all : 1 + std::rand() % 120;
        const int sinks = std::rand() % 8 == 0 ? all : std::rand() % 4 == 0 ? 0 : std::rand() % 90;
        const int n = 1 + std::rand() % (L < 40 ? L : 40);  // queries at the end of the context
        const int p0 = L - n, p1 = p0 + std::rand() % n;    // a tile's first and last position
        // the tile's list
        const WindowPages w(window_first(p0, window), p1 + 1, sinks);
        std::vector<int> listed;
        for (int i = 0; i < w.np; ++i) listed.push_back(w.page(i));
        std::vector<int> need;
        for (int pg = 0; pg * 16 <= p1; ++pg) {
            bool any = false;
            for (int t = pg * 16; t < pg * 16 + 16 && !any; ++t)
                for (int p = p0; p <= p1 && !any; ++p) any = sees(t, p, window, sinks);
            if (any) need.push_back(pg);
        }
        CHECK(listed == need);
        for (int p = p0; p <= p1; ++p) {  // the interval form, in list tokens
            const int hi = p + 1 - w.skip * 16, lo = window_first(p, window) - w.skip * 16;
            const int a = sinks < hi ? sinks : hi;
            for (int i = 0; i < w.np * 16; ++i) {
                const int t = w.page(i / 16) * 16 + i % 16;
                CHECK(sees(t, p, window, sinks) == (i < a || (i >= lo && i < hi)));
            }
        }
        // the decode's masks
        const WindowPages d(window_first(L - 1, window), L, sinks);
        for (int i = 0; i < d.np; ++i) {
            const uint32_t vis = visible_tokens(d.page(i), L, d.first, sinks);
            CHECK(vis != 0 && vis <= 0xffffu);
            for (int t = 0; t < 16; ++t)
                CHECK(((vis >> t) & 1u) == (sees(d.page(i) * 16 + t, L - 1, window, sinks) ? 1u : 0u));
        }
    }
    // shares of a line of segments, cut at pages
    for (int trial = 0; trial < 20000; ++trial) {
        const int min_pages = 2 + std::rand() % 20, snap = min_pages / 2, weight = std::rand() % 20;
        const int segs = 1 + std::rand() % 12, sms = 1 + std::rand() % 40;
        std::vector<int> np(segs);
        std::vector<int64_t> u0(segs);
        int64_t W = 0;
        for (int i = 0; i < segs; ++i) {
            np[i] = 1 + std::rand() % (std::rand() % 3 == 0 ? 300 : 12);
            u0[i] = W;
            W += np[i] + weight;
        }
        const int64_t want = (W + min_pages - 1) / min_pages, grid = want < sms ? want : sms;
        const Split s{W / grid, W % grid};
        for (int i = 0; i < segs; ++i) {
            int32_t k0, k1, at = 0;
            segment_owners(s, u0[i], np[i], snap, k0, k1);
            CHECK(0 <= k0 && k0 <= k1 && k1 < grid);
            for (int64_t k = 0; k < grid; ++k) {
                const int lo = cut_page(s.start(k), u0[i], np[i], snap), hi = cut_page(s.start(k + 1), u0[i], np[i], snap);
                CHECK(lo <= hi && (hi == lo || lo == at));
                CHECK((hi > lo) == (k >= k0 && k <= k1));
                if (hi > lo) at = hi;
                // a CTA finds its pages by the raw share: it overlaps the segment
                CHECK(hi == lo || (s.start(k) < u0[i] + np[i] + weight && s.start(k + 1) > u0[i]));
            }
            CHECK(at == np[i]);
        }
    }
    std::printf("ok\n");
    return 0;
}
