// pa_window.cuh -- which pages and tokens a sliding window with sinks reaches
// (host and device).
//
// A query at position p sees the tokens t <= p with t > p - window or
// t < sinks.  Compiled by the host tests too.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define PA_WINDOW_FN __host__ __device__ __forceinline__
#else
#define PA_WINDOW_FN inline
#endif

namespace pa {

// First token of the window of a query at position p.
PA_WINDOW_FN int32_t window_first(int32_t p, int32_t window) { return p >= window ? p - window + 1 : 0; }

// The pages that queries whose windows start at token `first` or later and
// whose positions are below `end` see, as a list: `ns` pages of sinks before
// the window's first page, then the pages of tokens first .. end-1.  Entry i is
// page i for i < ns and page i + skip after that, and token t of the list is
// token t or t + 16 skip.  Where pages are skipped, sinks <= 16 ns <= first.
struct WindowPages {
    int32_t first, ns, skip, np;
    PA_WINDOW_FN WindowPages(int32_t first_, int32_t end, int32_t sinks) : first(first_) {
        const int32_t wpage = first / 16, seen = sinks < first ? sinks : first, spages = seen / 16 + (seen % 16 != 0);
        ns = spages < wpage ? spages : wpage;
        skip = wpage - ns;
        np = end / 16 + (end % 16 != 0) - skip;
    }
    PA_WINDOW_FN int32_t page(int32_t i) const { return i < ns ? i : i + skip; }
};

// Which of the 16 tokens of page pg a query at the end of L tokens sees, whose
// window starts at token `first`.
PA_WINDOW_FN uint32_t visible_tokens(int32_t pg, int32_t L, int32_t first, int32_t sinks) {
    const int32_t t0 = pg * 16;
    auto below = [](int32_t n) -> uint32_t {  // bits 0 .. n-1
        return n <= 0 ? 0u : n >= 16 ? 0xffffu : (1u << n) - 1u;
    };
    return below(L - t0) & (~below(first - t0) | below(sinks < L ? sinks - t0 : 16));
}

// Page at which a share boundary at line position t cuts a segment of np
// pages that starts at u0: 0 or np where fewer than `snap` pages (or half
// the segment) would lie before or behind it.
PA_WINDOW_FN int32_t cut_page(int64_t t, int64_t u0, int32_t np, int32_t snap) {
    if (t <= u0) return 0;
    if (t >= u0 + np) return np;
    const int32_t c = int32_t(t - u0), lo = snap < (np + 1) / 2 ? snap : (np + 1) / 2;
    return c < lo ? 0 : np - c < lo ? np : c;
}

// The CTAs k0 <= k1 that hold the first and the last page of a segment, for
// the shares [start(k), start(k+1)) of `split` (a Split) after cut_page.
// Needs shares of at least `snap` units.
template <class S>
PA_WINDOW_FN void segment_owners(const S& split, int64_t u0, int32_t np, int32_t snap, int32_t& k0, int32_t& k1) {
    k0 = split.owner(u0);
    k1 = split.owner(u0 + np - 1);
    if (cut_page(split.start(k0 + 1), u0, np, snap) == 0) ++k0;
    if (cut_page(split.start(k1), u0, np, snap) == np) --k1;
}

}  // namespace pa
