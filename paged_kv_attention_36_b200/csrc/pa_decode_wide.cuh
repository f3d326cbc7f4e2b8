// pa_decode_wide.cuh -- paged decode with a sliding window, and over 8-bit
// caches with a scale for each (block, kv head).
//
// The work line, the ring of TMA-staged pages and the split-KV pieces are those
// of pa_decode.cuh.  What differs:
//
//   * A CTA has 8 consumer warps, WPH = the largest power of two <= 8 / HG of
//     them per head of the head group; part w of a head takes the pages whose
//     running number is w modulo WPH and keeps a softmax state of its own.  At
//     a segment's end the parts meet in shared memory and part 0 finishes the
//     segment while the others go on.  (Sixteen warps hold twice the stages, of
//     which fewer are then in flight: 72 against 62 us on the 8-bit batch, 92
//     against 73 us on one long context.)
//   * A head group's page (at most 8 KB of K) is one ring stage; wider groups
//     are cut into groups, which also halves the bytes of a piece where long
//     contexts are merged.
//   * Only the pages that a window or a sink reaches are on the line
//     (WindowPages), and each page comes with a 16-bit mask of the tokens
//     that count.
//   * Share boundaries that would cut fewer than `snap` pages off a segment
//     move to the segment's end (cut_page): short contexts stay whole, so a
//     small batch needs no merge between CTAs.
//   * Pieces are stored as the accumulator fragments lie (RawPiece), 16 bytes
//     at a time; two pieces are folded in registers by whichever CTA is last,
//     more are merged in one level or, past kWideFanIn, in two of about
//     sqrt(pieces).
//   * A page of an 8-bit cache brings its heads' scales along: two bulk
//     copies where they are 16-byte pieces (kv heads in fours), else 4-byte
//     cp.async copies that arrive on the stage's barrier.
//   * Launched as a programmatic dependent: the set-up overlaps the end of
//     the kernel before it.
//
// Bound by HBM.  Measured on B200 (floor: bytes at 6548 GB/s): 8-bit, batch 128
// of 512-4096 tokens, 32/8 heads of 64: 57.1 us (floor 48.8); 8-bit, one
// context of 131072 among 63 of 1024, 32/8 heads of 128: 68.8 us (61.5);
// window 1024 and 4 sinks over the first batch in bf16: 47.2 us (40.6).  What is
// left is the launch and the share scan (2 us), CTAs that stream slower than
// the median (3 us) and the last merge (1-4 us); four short sequences take
// 5.4-6.3 us, a chain of dependent loads.
#pragma once

#include <type_traits>

#include "pa_decode.cuh"
#include "pa_tcgen05.cuh"
#include "pa_window.cuh"

namespace pa {

// ldmatrix and mma forms of this file: shared-memory addresses as they are,
// and a product without an accumulator to start from.
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// Integer products on the tensor cores: c[16x8 s32] = a[16x32 s8, row-major] *
// b[32x8, col-major] + c0, b signed or unsigned.
template <bool B_UNSIGNED>
__device__ __forceinline__ void imma_16832(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                           const int (&c0)[4]) {
    if constexpr (B_UNSIGNED)
        asm(
            "mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(c0[0]), "r"(c0[1]), "r"(c0[2]),
              "r"(c0[3]));
    else
        asm(
            "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(c0[0]), "r"(c0[1]), "r"(c0[2]),
              "r"(c0[3]));
}
// An integer accumulator that starts at these bits reads as the float
// 12582912 + n while |n| < 2^22, so a subtraction converts it.
constexpr int kIntBase = 0x4B400000;
constexpr float kIntBaseF = 12582912.f;

// ---- page math over 8-bit codes ------------------------------------------------
// Both products run on the integer tensor cores, so no code is ever
// converted: the tiles (K [16][D], V transposed in its token order) are A
// operands of mma.sync m16n8k32 as ldmatrix delivers them.  (Converted to f16
// by byte permutes, the same batch took 65-67 us and was bound by the ALU
// chain; an s8 m16n8k32 takes 2.0 cycles of an SM, as an f16 m16n8k16 does.)
// The other operand is fixed point in 16 bits, as two 8-bit halves:
//
//   q = qmax / 32512 * (256 hi + lo), hi and lo signed: off by at most 2^-16
//     of the row's largest value.  S = 256 (K hi) + K lo, exact in integers.
//   P: for the tokens of a step (4 pages, 2 at head_dim 128), y = logit +
//     log2(v_scale) and its maximum over the step; w = 2^(y - max) =
//     (256 hi + lo) / 65535, hi and lo unsigned.  A token's weight is off by
//     at most 2^-17 of the heaviest contribution of its own step, whatever
//     the other steps' weights or the other blocks' scales are.
//
// With up to four heads the halves of P share an mma: columns 0-3 take the
// high halves, columns 4-7 the low ones of the same heads (S has each head
// in both), and the two sums meet at the end.  With eight heads each half
// has an mma of its own.  Sums of a step stay below 2^22 and become fp32 by
// one subtraction (kIntBase); the state (m, l, O) is fp32.  l comes
// from the same w, unrounded: 2^(logit - m) = w * 2^(max - m - log2(v_scale)).
// m follows the maxima of the steps lazily (raised when one passes it by 15).
template <int D, int G>
struct I8Math : MmaMath<D, G, 16> {
    using Base = MmaMath<D, G, 16>;
    using Base::KS;
    using Base::acc;
    using Base::m;
    using Base::l;
    static constexpr int kElemBytes = 1;
    static constexpr bool kShared = G <= 4;  // high and low halves share an mma
    static constexpr int NQ = kShared ? 1 : 2;
    static constexpr int kPages = D == 64 ? 4 : 2;  // of a softmax step
    uint32_t qi[2][D / 32][2];   // q's halves as B fragments
    float qs[2];                 // scale * log2(e) * qmax / 32512 of this lane's two heads
    uint32_t koff[D / 32];       // this lane's K row, for each 32 columns

    // Byte offset of 16-byte chunk ch (d 16ch .. 16ch+15) of token t in a K tile.
    static __device__ __forceinline__ int k_off(int t, int ch) {
        const int line = D == 128 ? t : (t >> 1);
        const int lch = D == 128 ? ch : (((t & 1) << 2) + ch);
        return (line << 7) + ((lch ^ (line & 7)) << 4);
    }

    __device__ __forceinline__ void load_q_global(const uint8_t* gq, int lane, float qscale) {
        const int n = lane >> 2, c = lane & 3;  // this lane's column of the mma
        const int h = kShared ? n & 3 : n;
        uint2 w[D / 32][2];
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                w[j][i] = h < G ? __ldca(reinterpret_cast<const uint2*>(gq + (h * D + 32 * j + 16 * i + 4 * c) * 2))
                                : make_uint2(0u, 0u);
                const float2 x = bf16x2_to_float2(w[j][i].x), y = bf16x2_to_float2(w[j][i].y);
                top = fmaxf(fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(y.x), fabsf(y.y)));
            }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // v * down is exact and at most 4, so the product with r neither
        // overflows nor vanishes, however large or small q is
        int e = int(__float_as_uint(top) >> 23) - 127;
        e = e < -126 ? -126 : e > 126 ? 126 : e;
        const float down = __uint_as_float(uint32_t(127 - e) << 23);
        const float r = top > 0.f ? 32512.f / (top * down) : 0.f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 x = bf16x2_to_float2(w[j][i].x), y = bf16x2_to_float2(w[j][i].y);
                const float v[4] = {x.x, x.y, y.x, y.y};
                uint32_t hi = 0, lo = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int q16 = __float2int_rn(v[e] * down * r);
                    const int up = (q16 + 128) >> 8;
                    hi |= uint32_t(up & 0xff) << (8 * e);
                    lo |= uint32_t((q16 - (up << 8)) & 0xff) << (8 * e);
                }
                qi[0][j][i] = hi;
                qi[1][j][i] = lo;
            }
        // columns 2c and 2c + 1 of S are this lane's; their rows lie in lanes 4 n ..
        const float unit = qscale * (top / 32512.f);
#pragma unroll
        for (int i = 0; i < 2; ++i) qs[i] = __shfl_sync(0xffffffffu, unit, 4 * (2 * c + i));
        const int mi = lane >> 3, t = (lane & 7) + ((mi & 1) << 3);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) koff[j] = uint32_t(k_off(t, 2 * j + (mi >> 1)));
    }

    // NP pages (shared-memory addresses of their K and V tiles), the tokens
    // of `vis` counting (0: the page is not there; its addresses are valid).
    template <int NP>
    __device__ __forceinline__ void pages(const uint32_t (&kt)[NP], const uint32_t (&vt)[NP],
                                          const uint32_t (&vis)[NP], const float (&ks)[NP], const float (&vs)[NP],
                                          int lane) {
        static_assert(NP % 2 == 0 && NP * 16 * 255 * 127 < 1 << 22, "whole k32 steps, sums below 2^22");
        constexpr int base[4] = {kIntBase, kIntBase, kIntBase, kIntBase};
        // ---- every fragment of K first, then the products of the pages in turn ----
        int s[NP][2][4];
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            uint32_t ka[NP][4];
#pragma unroll
            for (int i = 0; i < NP; ++i) ldsm_x4(ka[i], kt[i] + koff[j]);
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (j == 0) imma_16832<false>(s[i][x], ka[i], qi[x][j][0], qi[x][j][1], base);
                    else imma_16832<false>(s[i][x], ka[i], qi[x][j][0], qi[x][j][1], s[i][x]);
                }
        }
        // ---- y = scale * K . q + log2(v_scale) ----
        float y[NP][4], lv[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            lv[i] = vs[i] <= 0x1p-100f ? -100.f : __log2f(vs[i]);  // a scale of 0: codes of 0, weight still in l
            const float c[2] = {qs[0] * ks[i], qs[1] * ks[i]};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float hi = __int_as_float(s[i][0][e]) - kIntBaseF, lo = __int_as_float(s[i][1][e]) - kIntBaseF;
                y[i][e] = fmaf(fmaf(hi, 256.f, lo), c[e & 1], lv[i]);
            }
            if (vis[i] != 0xffffu) {
                const int t0 = lane >> 2;
                if (!((vis[i] >> t0) & 1)) y[i][0] = y[i][1] = -INFINITY;
                if (!((vis[i] >> (t0 + 8)) & 1)) y[i][2] = y[i][3] = -INFINITY;
            }
        }
        // ---- the step's maximum of each head column, and the running one ----
        float b0 = fmaxf(y[0][0], y[0][2]), b1 = fmaxf(y[0][1], y[0][3]);
#pragma unroll
        for (int i = 1; i < NP; ++i) {
            b0 = fmax3(b0, y[i][0], y[i][2]);
            b1 = fmax3(b1, y[i][1], y[i][3]);
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, off));
            b1 = fmaxf(b1, __shfl_xor_sync(0xffffffffu, b1, off));
        }
        if (__any_sync(0xffffffffu, b0 > m[0] + 15.f || b1 > m[1] + 15.f)) {
            const float n0 = fmaxf(m[0], b0), n1 = fmaxf(m[1], b1);
            rescale(ex2_approx(m[0] - n0), ex2_approx(m[1] - n1));
            m[0] = n0;
            m[1] = n1;
        }
        // ---- weights; l; the 16-bit weights as B fragments ----
        uint32_t pb[NQ][NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const float w0 = ex2_approx(y[i][0] - b0), w1 = ex2_approx(y[i][1] - b1);
            const float w2 = ex2_approx(y[i][2] - b0), w3 = ex2_approx(y[i][3] - b1);
            l[0] = fmaf(w0 + w2, ex2_approx(b0 - m[0] - lv[i]), l[0]);
            l[1] = fmaf(w1 + w3, ex2_approx(b1 - m[1] - lv[i]), l[1]);
            // 2^23 + rint(65535 w): the integer is in the low 16 bits
            auto fix = [](float w) { return __float_as_uint(fmaf(w, 65535.f, 8388608.f)); };
            const uint32_t t0 = movmatrix_trans(__byte_perm(fix(w0), fix(w1), 0x5410));  // tokens 2c, 2c+1
            const uint32_t t8 = movmatrix_trans(__byte_perm(fix(w2), fix(w3), 0x5410));  // tokens 2c+8, 2c+9
            // one byte of each, in the V rows' token order
            if constexpr (kShared) {
                pb[0][i] = __byte_perm(t0, t8, lane < 16 ? 0x7531 : 0x6420);
            } else {
                pb[0][i] = __byte_perm(t0, t8, 0x7531);
                pb[NQ - 1][i] = __byte_perm(t0, t8, 0x6420);
            }
        }
        // ---- O^T += V^T . P^T, two m-tiles (32 rows of V^T) per ldmatrix ----
        const float wt = kShared && (lane & 3) >= 2 ? 1.f / 65535.f : 256.f / 65535.f;
        const float f0 = ex2_approx(b0 - m[0]) * wt, f1 = ex2_approx(b1 - m[1]) * wt;
        const uint64_t f2 = f2_pack(f0, f1), down = f2_pack(-kIntBaseF, -kIntBaseF);
#pragma unroll
        for (int j = 0; j < KS / 2; ++j) {
            uint32_t va[NP][4];
#pragma unroll
            for (int i = 0; i < NP; ++i) ldsm_x4(va[i], vt[i] + uint32_t((32 * j + lane) * 16));
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                int o[NQ][4];
#pragma unroll
                for (int i = 0; i < NP; i += 2) {
                    const uint32_t a[4] = {va[i][2 * t], va[i][2 * t + 1], va[i + 1][2 * t], va[i + 1][2 * t + 1]};
#pragma unroll
                    for (int x = 0; x < NQ; ++x) {
                        if (i == 0) imma_16832<true>(o[x], a, pb[x][i], pb[x][i + 1], base);
                        else imma_16832<true>(o[x], a, pb[x][i], pb[x][i + 1], o[x]);
                    }
                }
                float* dst = acc[2 * j + t];
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    uint64_t v = f2_add(f2_pack(__int_as_float(o[0][e]), __int_as_float(o[0][e + 1])), down);
                    if constexpr (!kShared) {  // 256 high + low, in units of the high half's factor
                        const uint64_t w =
                            f2_add(f2_pack(__int_as_float(o[NQ - 1][e]), __int_as_float(o[NQ - 1][e + 1])), down);
                        v = f2_fma(w, f2_pack(1.f / 256.f, 1.f / 256.f), v);
                    }
                    f2_unpack(f2_fma(v, f2, f2_pack(dst[e], dst[e + 1])), dst[e], dst[e + 1]);
                }
            }
        }
    }

    __device__ __forceinline__ void rescale(float a0, float a1) {
        l[0] *= a0;
        l[1] *= a1;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            acc[i][0] *= a0;
            acc[i][1] *= a1;
            acc[i][2] *= a0;
            acc[i][3] *= a1;
        }
    }

    // The high and the low halves' sums of each head meet (before finish()).
    __device__ __forceinline__ void join_halves() {
        if constexpr (kShared) {
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] += __shfl_xor_sync(0xffffffffu, acc[i][e], 2);
        }
    }
};

// ---- shared memory ---------------------------------------------------------------
#ifndef PA_WIDE_WARPS
#define PA_WIDE_WARPS 8
#endif
constexpr int kWideWarps = PA_WIDE_WARPS;  // consumer warps
constexpr int kWideThreads = (kWideWarps + 1) * 32;
constexpr int kWideSegs = 4;    // segment descriptors in flight
constexpr int kWideMaxRing = 32;

// How a call's head layout uses the CTA (computed on the host).
struct WideShape {
    int32_t HG, HS, SPL_LOG, WPH_LOG;  // heads per group and per stage, log2 of stages per page and of warps per head
    int32_t R;                         // ring stages, a multiple of (stages per page) * (warps per head)
    int32_t stage_k;                   // K bytes of a stage (as many V bytes follow)
    int32_t snap;                      // fewest pages worth cutting off a segment
    int32_t smem;                      // bytes
};

struct WideLayout {  // byte offsets from the 1024-byte aligned base
    int32_t ring, parts, scales, descs, bars, misc, total;
};

// A part's state in shared memory: the accumulator fragments as they lie in
// the lanes, then (m, l) of the lane's two heads.
__host__ __device__ constexpr int part_bytes(int D) { return (D / 16 + 1) * 32 * 16; }

struct WideMisc {
    int abort;
    int b0, L0;         // sequence where the share starts, its length
    long long pre0;     // line position of its first unit
    long long red[kWideWarps + 1];
};

__host__ __device__ inline WideLayout wide_layout(const WideShape& s, int D) {
    WideLayout w;
    const int wph = 1 << s.WPH_LOG;
    w.ring = 0;
    w.parts = s.R * 2 * s.stage_k;
    w.scales = w.parts + (wph - 1) * s.HG * part_bytes(D);
    w.descs = w.scales + s.R * 64;
    w.bars = w.descs + kWideSegs * 32;
    w.misc = w.bars + (2 * s.R + 2 * kWideSegs + 2 * s.HG) * 8;
    w.total = w.misc + ((int(sizeof(WideMisc)) + 15) & ~15);
    return w;
}

constexpr int kWideFanIn = 8;  // pieces merged at once; more go in two levels

// ---- pieces of a (b, kv head) that share boundaries cut --------------------------
// A piece's state goes to its partial slot as it lies in the fragments,
// unnormalised: float4 (16-row tile mt, row d0, head pair c) at
// (8 mt + d0) * G/2 + c holds (h, d), (h+1, d), (h, d+8), (h+1, d+8) with
// h = 2c, d = 16 mt + d0, and ml[c] = (m_h, m_h+1, l_h, l_h+1); with one head
// the pairs (d, d+8) are float2 and ml is (m, l).  The same bytes as [G][D]
// floats, written and read 16 at a time.
template <int G>
struct RawPiece {
    static constexpr int GP = G > 1 ? G / 2 : 1;
    // After finish(): this warp's state to o, ml.
    template <class M>
    static __device__ __forceinline__ void store(const M& st, float* o, float2* ml, int lane) {
        const int c = lane & 3, d0 = lane >> 2;
        if (c >= GP) return;
#pragma unroll
        for (int mt = 0; mt < M::KS; ++mt) {
            if constexpr (G > 1)
                reinterpret_cast<float4*>(o)[(8 * mt + d0) * GP + c] =
                    make_float4(st.acc[mt][0], st.acc[mt][1], st.acc[mt][2], st.acc[mt][3]);
            else
                reinterpret_cast<float2*>(o)[8 * mt + d0] = make_float2(st.acc[mt][0], st.acc[mt][2]);
        }
        if (d0 == 0) {
            if constexpr (G > 1)
                reinterpret_cast<float4*>(ml)[c] = make_float4(st.m[0], st.m[1], st.l[0], st.l[1]);
            else
                ml[0] = make_float2(st.m[0], st.l[0]);
        }
    }
    // After finish(): folds the stored piece (the one before this state in
    // page order iff before) into the state; the same bits whichever of the
    // two was stored.
    template <class M>
    static __device__ __forceinline__ void fold(M& st, const float* o, const float2* ml, bool before, int lane) {
        const int c = lane & 3, d0 = lane >> 2;
        if (c >= GP) return;
        float4 v[M::KS], w;
#pragma unroll
        for (int mt = 0; mt < M::KS; ++mt) {
            if constexpr (G > 1) {
                v[mt] = __ldcg(reinterpret_cast<const float4*>(o) + (8 * mt + d0) * GP + c);
            } else {
                const float2 x = __ldcg(reinterpret_cast<const float2*>(o) + 8 * mt + d0);
                v[mt] = make_float4(x.x, 0.f, x.y, 0.f);
            }
        }
        if constexpr (G > 1) {
            w = __ldcg(reinterpret_cast<const float4*>(ml) + c);
        } else {
            const float2 x = __ldcg(ml);
            w = make_float4(x.x, st.m[1], x.y, 0.f);
        }
        const float n0 = fmaxf(st.m[0], w.x), n1 = fmaxf(st.m[1], w.y);
        const float a0 = exp2f(st.m[0] - n0), a1 = exp2f(st.m[1] - n1);
        const float b0 = exp2f(w.x - n0), b1 = exp2f(w.y - n1);
        // first * its weight, then second * its weight on top
        auto mix = [&](float mine, float a, float theirs, float b) {
            return before ? fmaf(mine, a, __fmul_rn(theirs, b)) : fmaf(theirs, b, __fmul_rn(mine, a));
        };
        st.m[0] = n0;
        st.m[1] = n1;
        st.l[0] = mix(st.l[0], a0, w.z, b0);
        st.l[1] = mix(st.l[1], a1, w.w, b1);
#pragma unroll
        for (int mt = 0; mt < M::KS; ++mt) {
            st.acc[mt][0] = mix(st.acc[mt][0], a0, v[mt].x, b0);
            st.acc[mt][1] = mix(st.acc[mt][1], a1, v[mt].y, b1);
            st.acc[mt][2] = mix(st.acc[mt][2], a0, v[mt].z, b0);
            st.acc[mt][3] = mix(st.acc[mt][3], a1, v[mt].w, b1);
        }
    }
};

// Merges the n stored pieces of one warp's (b, kv head) in the slots of the
// leaves off, off + stride, ... in that order: into out (bf16 [G][D]) if
// given, else over the first of them.  Lane l takes the float4s l, l+32, ...
// of each piece, all of one head pair; maxima and sums run along (no pass
// over the pieces before their values).
template <int D, int G>
__device__ __noinline__ void merge_raw(const DecodeParams& p, int k0, int off, int stride, int n, int HG, int head,
                                       int lane, __nv_bfloat16* out) {
    constexpr int GP = RawPiece<G>::GP;
    constexpr int N4 = D * G / 4;            // float4s of a piece
    constexpr int T = (N4 + 31) / 32;        // of a lane
    constexpr int U = T >= 4 ? 16 / T : 8;   // pieces in flight
    const int c = lane % GP;
    auto slot = [&](int i) -> int64_t { return (leaf_slot(k0, off + i * stride) * HG + head) * G; };
    float M0 = -INFINITY, M1 = -INFINITY, L0 = 0.f, L1 = 0.f;
    float4 a[T];
#pragma unroll
    for (int t = 0; t < T; ++t) a[t] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n; i0 += U) {
        float4 v[U][T], w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool there = i0 + u < n;
            const int64_t s = slot(there ? i0 + u : 0);
#pragma unroll
            for (int t = 0; t < T; ++t)
                v[u][t] = N4 % 32 == 0 || lane + 32 * t < N4
                              ? __ldcg(reinterpret_cast<const float4*>(p.part_o + s * D) + lane + 32 * t)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
            if constexpr (G > 1) {
                w[u] = __ldcg(reinterpret_cast<const float4*>(p.part_ml + s) + c);
            } else {
                const float2 x = __ldcg(p.part_ml + s);
                w[u] = make_float4(x.x, x.x, x.y, x.y);
            }
            if (!there) w[u] = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float n0 = fmaxf(M0, w[u].x), n1 = fmaxf(M1, w[u].y);  // finite from the first piece on
            const float s0 = exp2f(M0 - n0), s1 = exp2f(M1 - n1);
            const float w0 = exp2f(w[u].x - n0), w1 = exp2f(w[u].y - n1);
            M0 = n0;
            M1 = n1;
            L0 = L0 * s0 + w[u].z * w0;
            L1 = L1 * s1 + w[u].w * w1;
#pragma unroll
            for (int t = 0; t < T; ++t) {
                a[t].x = a[t].x * s0 + v[u][t].x * w0;
                a[t].y = a[t].y * s1 + v[u][t].y * w1;
                a[t].z = a[t].z * s0 + v[u][t].z * w0;
                a[t].w = a[t].w * s1 + v[u][t].w * w1;
            }
        }
    }
    __syncwarp();  // every lane has read the first slot
    const float r0 = 1.f / L0, r1 = 1.f / L1;
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int i = lane + 32 * t;
        if (N4 % 32 != 0 && i >= N4) continue;
        if (!out) {
            reinterpret_cast<float4*>(p.part_o + slot(0) * D)[i] = a[t];
        } else if constexpr (G > 1) {
            const int r = i / GP, d = 16 * (r / 8) + r % 8;
            __nv_bfloat16* o = out + 2 * c * D + d;
            o[0] = __float2bfloat16_rn(a[t].x * r0);
            o[D] = __float2bfloat16_rn(a[t].y * r1);
            o[8] = __float2bfloat16_rn(a[t].z * r0);
            o[D + 8] = __float2bfloat16_rn(a[t].w * r1);
        } else {
            const int r = 2 * i, d = 16 * (r / 8) + r % 8;  // rows r and r + 1 (r even: one tile)
            out[d] = __float2bfloat16_rn(a[t].x * r0);
            out[d + 8] = __float2bfloat16_rn(a[t].y * r0);
            out[d + 1] = __float2bfloat16_rn(a[t].z * r0);
            out[d + 9] = __float2bfloat16_rn(a[t].w * r0);
        }
    }
    if (!out && lane < GP) {
        if constexpr (G > 1) reinterpret_cast<float4*>(p.part_ml + slot(0))[lane] = make_float4(M0, M1, L0, L1);
        else p.part_ml[slot(0)] = make_float2(M0, L0);
    }
}

// One more arrival at a counter, after the calling warp's writes and before
// its later reads; true in every lane if it completes `count`.
__device__ __forceinline__ bool arrive_last(int32_t* counter, int count, int lane) {
    __syncwarp();
    int old = 0;
    if (lane == 0)
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
    old = __shfl_sync(0xffffffffu, old, 0);
    return old == count - 1;
}

struct WideDesc {  // one segment, from the producer to the consumers
    int32_t b, hg;   // sequence, head group
    int32_t j0, npg; // first listed page and pages; npg = 0 marks the end of the share
    int32_t L;
    int32_t k0, k1;  // CTAs that hold pages of (b, hg)
    int32_t pad;
};

struct WideParams {
    DecodeParams d;  // k_scale and v_scale: [NB][Hkv] for 8-bit caches
    WideShape shape;
    int32_t window, sinks;
};

// The pages a decode over L > 0 tokens streams.
__device__ __forceinline__ WindowPages window_pages(const WideParams& wp, int32_t L) {
    return WindowPages(window_first(L - 1, wp.window), L, wp.sinks);
}

__device__ __forceinline__ void cp_async4(void* smem_dst, const void* gmem_src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(smem_dst)), "l"(gmem_src) : "memory");
}
// Arrives on `bar` once when all of this thread's earlier cp.async copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <class MathT, int D, int G, bool I8>
__global__ void __launch_bounds__(kWideThreads, 1) decode_wide_kernel(const __grid_constant__ WideParams wp) {
    constexpr int NT = kWideThreads, S = kWideSegs;
    constexpr int kTile = 16 * D * (I8 ? 1 : 2);
    const DecodeParams& p = wp.d;
    const WideShape& sh = wp.shape;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const WideLayout lay = wide_layout(sh, D);
    uint8_t* ring = smem + lay.ring;
    float* scales = reinterpret_cast<float*>(smem + lay.scales);  // per stage: 8 K scales, 8 V scales
    WideDesc* descs = reinterpret_cast<WideDesc*>(smem + lay.descs);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + lay.bars);
    uint64_t* empty = full + sh.R;
    uint64_t* segfull = empty + sh.R;
    uint64_t* segempty = segfull + S;
    uint64_t* partfull = segempty + S;   // per head: the other parts' states are written
    uint64_t* partempty = partfull + sh.HG;  // and read
    WideMisc* misc = reinterpret_cast<WideMisc*>(smem + lay.misc);
    volatile int* abort = &misc->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int HG = sh.HG, HS = sh.HS, SPL = 1 << sh.SPL_LOG, WPH = 1 << sh.WPH_LOG, R = sh.R;

    // a stage's scales are 16-byte pieces: one bulk copy each for K and V
    const bool bulk_scales = I8 && HS % 4 == 0 && p.Hkv % 4 == 0 &&
                             ((reinterpret_cast<uintptr_t>(p.k_scale) | reinterpret_cast<uintptr_t>(p.v_scale)) & 15) == 0;

    if (warp == kWideWarps && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_v)) : "memory");
    }
    if (warp == 0) {
        for (int r = lane; r < R; r += 32) {
            mbar_init(&full[r], I8 && !bulk_scales ? 2 : 1);  // the copies' expectation, and the scales' arrival
            mbar_init(&empty[r], uint32_t(HS));
        }
        if (lane < S) {
            mbar_init(&segfull[lane], 1);
            mbar_init(&segempty[lane], uint32_t(HG * WPH));
        }
        if (lane < HG) {
            mbar_init(&partfull[lane], uint32_t(WPH > 1 ? WPH - 1 : 1));
            mbar_init(&partempty[lane], 1);
        }
        if (lane == 0) misc->abort = 0;
        fence_mbar_init();
    }
    // everything below reads what kernels before this one may have written
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- the CTA's share: a scan of NG * (pages + seg_weight) over the sequences ----
    const bool one_chunk = p.B <= NT;
    long long v_mine = 0, incl_mine = 0, Wt = 0;
    int32_t L_mine = 0;
    auto units = [&](int32_t L) -> long long {
        return L > 0 ? (long long)(window_pages(wp, L).np + p.seg_weight) * p.NG : 0;
    };
    for (int base = 0; base < p.B; base += NT) {
        const int b = base + threadIdx.x;
        long long v = 0;
        if (b < p.B) {
            L_mine = clamp_len<16>(p, b, blockIdx.x == 0);
            v = units(L_mine);
            if (L_mine == 0 && (b % int(gridDim.x)) == int(blockIdx.x)) {
                uint4* o = reinterpret_cast<uint4*>(p.out + int64_t(b) * p.Hq * D);
                for (int i = 0; i < p.Hq * D / 8; ++i) o[i] = make_uint4(0, 0, 0, 0);
            }
        }
        long long chunk_total;
        const long long incl = Wt + block_incl_scan<NT>(v, misc->red, chunk_total);
        Wt += chunk_total;
        v_mine = v;
        incl_mine = incl;
    }
    const int64_t want = (Wt + p.min_pages - 1) / p.min_pages;
    const int64_t grid_eff = want < int64_t(gridDim.x) ? want : int64_t(gridDim.x);
    if (Wt == 0 || int64_t(blockIdx.x) >= grid_eff) return;
    const Split split = Wt >> 31 ? Split{Wt / grid_eff, Wt % grid_eff}
                                 : Split{int32_t(Wt) / int32_t(grid_eff), int32_t(Wt) % int32_t(grid_eff)};
    const int64_t p_start = split.start(blockIdx.x), p_end = split.start(int64_t(blockIdx.x) + 1);
    auto locate = [&](int b, long long v, long long incl, int32_t L) {
        if (v > 0 && incl - v <= p_start && p_start < incl) {
            misc->b0 = b;
            misc->L0 = L;
            misc->pre0 = incl - v;
        }
    };
    if (one_chunk) {
        locate(threadIdx.x, v_mine, incl_mine, L_mine);
    } else {
        long long carry = 0;
        for (int base = 0; base < p.B; base += NT) {
            const int b = base + threadIdx.x;
            const int32_t L = b < p.B ? clamp_len<16>(p, b, false) : 0;
            const long long v = units(L);
            long long chunk_total;
            const long long incl = carry + block_incl_scan<NT>(v, misc->red, chunk_total);
            locate(b, v, incl, L);
            carry += chunk_total;
        }
    }
    __syncthreads();

    if (warp == kWideWarps) {
        // ======================= producer warp =======================
        uint32_t stage_i = 0, seg_i = 0;
        int slot0 = 0;       // slot of the batch's first stage
        uint32_t use0 = 0;   // parity of that slot's use
        const int C = R < 32 ? R : 32;
        bool ok = true;
        const uint64_t pol = policy_evict_first();
        const uint32_t stage_tx = uint32_t(2 * HS * kTile);

        // The segments of the share in order; within a segment block ids are
        // read one batch of stages ahead.
        struct Seg {
            int32_t b, hg, L, j, npg;
            int64_t u0;  // line position of its first page
        };
        auto pages_of = [&](const Seg& g) { return window_pages(wp, g.L); };
        auto cut = [&](Seg& g, int32_t np) {
            g.j = cut_page(p_start, g.u0, np, sh.snap);
            g.npg = cut_page(p_end, g.u0, np, sh.snap) - g.j;
        };
        // The segment after g (u0 >= p_end: none); L_next: the length of
        // sequence g.b + 1, read ahead and not checked.
        auto checked = [&](int32_t L) {
            const int64_t cap = int64_t(p.M) * 16;
            return L < 0 ? 0 : L > cap ? int32_t(cap) : L;
        };
        auto after = [&](const Seg& g, int32_t L_next) {
            Seg n = g;
            do {
                n.u0 += pages_of(n).np + p.seg_weight;
                if (n.u0 >= p_end) return n;
                if (++n.hg == p.NG) {
                    n.hg = 0;
                    ++n.b;
                    n.L = checked(L_next);
                    while (n.L == 0) n.L = clamp_len<16>(p, ++n.b, false);
                    if (n.b + 1 < p.B) L_next = __ldca(p.context_lens + n.b + 1);
                }
                cut(n, pages_of(n).np);
            } while (n.npg == 0);
            return n;
        };
        // Block id of this lane's stage c0 + lane of segment g (0 past its end).
        auto block_of = [&](const Seg& g, int c0) -> int32_t {
            const int x = c0 + lane;
            if (lane >= C || x >= g.npg << sh.SPL_LOG) return 0;
            return __ldca(p.block_tables + int64_t(g.b) * p.M + pages_of(g).page(g.j + (x >> sh.SPL_LOG)));
        };

        Seg seg;
        seg.b = misc->b0;
        seg.L = misc->L0;
        const int64_t unit0 = pages_of(seg).np + p.seg_weight;
        seg.hg = p_start - misc->pre0 < unit0 ? 0 : int((p_start - misc->pre0) / unit0);
        seg.u0 = misc->pre0 + int64_t(seg.hg) * unit0;
        cut(seg, pages_of(seg).np);
        if (seg.npg == 0) seg = after(seg, seg.b + 1 < p.B ? __ldca(p.context_lens + seg.b + 1) : 0);
        int32_t blk = seg.u0 < p_end ? block_of(seg, 0) : 0;
        while (ok && seg.u0 < p_end) {
            // (as it is: checked where it is used, so that nothing waits for it here)
            const int32_t L_next = seg.b + 1 < p.B ? __ldca(p.context_lens + seg.b + 1) : 0;
            if (lane == 0) {
                const int s = seg_i % S;
                if (seg_i >= S) ok = mbar_wait(&segempty[s], ((seg_i / S) - 1) & 1, abort);
                if (ok) {
                    // the CTAs of the segment's first and last page
                    const int np = pages_of(seg).np;
                    int32_t k0 = int(blockIdx.x), k1 = k0;
                    if (seg.npg < np) segment_owners(split, seg.u0, np, sh.snap, k0, k1);
                    descs[s] = WideDesc{seg.b, seg.hg, seg.j, seg.npg, seg.L, k0, k1, 0};
                    mbar_arrive(&segfull[s]);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            // one lane per stage: HS heads' K tiles, then their V tiles
            const int tile0 = seg.hg * HG;
            const int nst = seg.npg << sh.SPL_LOG;
            Seg next = seg;
            for (int c0 = 0; ok && c0 < nst; c0 += C) {
                int32_t blk_next = c0 + C < nst ? block_of(seg, c0 + C) : 0;
                const int n = (nst - c0) < C ? (nst - c0) : C;
                bool lane_ok = true;
                if (lane < n) {
                    if (blk < 0 || blk >= p.NB) {
                        raise_error(PA_DEVERR_BLOCK_ID);
                        blk = 0;
                    }
                    const int x = c0 + lane;
                    int slot = slot0 + lane;  // of stage stage_i + x, in its use of parity `use`
                    uint32_t use = use0;
                    if (slot >= R) {
                        slot -= R;
                        use ^= 1;
                    }
                    if (stage_i + x >= uint32_t(R)) lane_ok = mbar_wait(&empty[slot], use ^ 1, abort);
                    if (lane_ok) {
                        uint8_t* st = ring + slot * 2 * sh.stage_k;
                        mbar_arrive_expect_tx(&full[slot], stage_tx + (bulk_scales ? uint32_t(8 * HS) : 0u));
                        const int tile = blk * p.Hkv + tile0 + (x & (SPL - 1)) * HS;
                        tma_load_4d(st, &p.tmap_k, 0, 0, 0, tile, &full[slot], pol);
                        tma_load_4d(st + sh.stage_k, &p.tmap_v, 0, 0, 0, tile, &full[slot], pol);
                        if constexpr (I8) {
                            float* sc = scales + slot * 16;
                            if (bulk_scales) {
                                bulk_g2s(sc, p.k_scale + tile, uint32_t(4 * HS), &full[slot]);
                                bulk_g2s(sc + 8, p.v_scale + tile, uint32_t(4 * HS), &full[slot]);
                            } else {
                                for (int h = 0; h < HS; ++h) {
                                    cp_async4(sc + h, p.k_scale + tile + h);
                                    cp_async4(sc + 8 + h, p.v_scale + tile + h);
                                }
                                cp_async_arrive(&full[slot]);
                            }
                        }
                    }
                }
                ok = __all_sync(0xffffffffu, lane_ok);
                if (c0 + C >= nst) {
                    // the next segment's first ids, once this one's last copies
                    // are under way (a call of few pages starts them that much sooner)
                    next = after(seg, L_next);
                    if (next.u0 < p_end) blk_next = block_of(next, 0);
                }
                blk = blk_next;
                slot0 += n;
                if (slot0 >= R) {
                    slot0 -= R;
                    use0 ^= 1;
                }
            }
            stage_i += nst;
            ++seg_i;
            seg = next;
        }
        if (ok && lane == 0) {  // end-of-share marker
            const int s = seg_i % S;
            if (seg_i >= S) ok = mbar_wait(&segempty[s], ((seg_i / S) - 1) & 1, abort);
            if (ok) {
                descs[s].npg = 0;
                mbar_arrive(&segfull[s]);
            }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok && lane == 0) {
            // error path: let every copy that may have started land before
            // the CTA's shared memory is freed
            const uint32_t last = stage_i + C;
            for (uint32_t i = (last > uint32_t(R) ? last - R : 0); i < last; ++i)
                mbar_wait(&full[i % R], (i / R) & 1, nullptr, 20000000ull);
        }
        return;
    }
    if (warp >= HG << sh.WPH_LOG) return;

    // ========================= consumer warps =========================
    const int head = warp % HG, part = warp / HG;
    const int sub = head / HS, pos = head - sub * HS;  // stage of a page, tile of the stage
    uint32_t page_base = 0, seg_i = 0;
    // this warp's next stage: R is a multiple of the step, so its pages recur
    // in the same slots and every parity wait is exact
    const int step = SPL << sh.WPH_LOG;
    int slot = (part << sh.SPL_LOG) + sub;
    uint32_t phase = 0;
    float4* mine = reinterpret_cast<float4*>(smem + lay.parts + ((part - 1) * HG + head) * part_bytes(D));  // part > 0
    const uint32_t tiles = smem_u32(ring) + uint32_t(pos * kTile);  // this head's K tile in stage 0
    MathT st;

    while (true) {
        const int s = seg_i % S;
        if (!mbar_wait(&segfull[s], (seg_i / S) & 1, abort)) return;
        const WideDesc d = descs[s];
        __syncwarp();
        if (lane == 0) mbar_arrive(&segempty[s]);
        if (d.npg == 0) break;
        const int g = d.hg * HG + head;
        const int64_t row = int64_t(d.b) * p.Hq + int64_t(g) * G;  // its first query head
        st.load_q_global(p.q + row * (D * 2), lane, p.qscale);
        st.reset();
        const WindowPages pages = window_pages(wp, d.L);
        // this part's pages: those whose running number is `part` modulo WPH
        auto advance = [&]() {
            slot += step;
            if (slot >= R) {
                slot -= R;
                phase ^= 1;
            }
        };
        // the tokens of listed page k that count (whole inside the window)
        auto seen = [&](int k) -> uint32_t {
            const int pg = pages.page(d.j0 + k);
            return pg * 16 >= pages.first && pg * 16 + 16 <= d.L ? 0xffffu
                                                                 : visible_tokens(pg, d.L, pages.first, wp.sinks);
        };
        int k = int((part - page_base) & uint32_t(WPH - 1));
        if constexpr (I8) {
            // this part's next pages, NP at a time; of the last step only `have` are there
            auto run = [&](auto count, int have) -> bool {
                constexpr int NP = decltype(count)::value;
                uint32_t kt[NP], vt[NP], vis[NP];
                float ks[NP], vs[NP];
                int slots[NP];
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    if (i >= have) {
                        kt[i] = kt[0], vt[i] = vt[0], ks[i] = ks[0], vs[i] = vs[0], vis[i] = 0u;
                        continue;
                    }
                    slots[i] = slot;
                    vis[i] = seen(k);
                    if (!mbar_wait(&full[slot], phase, abort)) return false;
                    kt[i] = tiles + uint32_t(slot * 2 * sh.stage_k);
                    vt[i] = kt[i] + uint32_t(sh.stage_k);
                    ks[i] = scales[slot * 16 + pos];
                    vs[i] = scales[slot * 16 + 8 + pos];
                    k += WPH;
                    advance();
                }
                st.template pages<NP>(kt, vt, vis, ks, vs, lane);
                __syncwarp();
                if (lane == 0) {
#pragma unroll
                    for (int i = 0; i < NP; ++i)
                        if (i < have) mbar_arrive(&empty[slots[i]]);
                }
                return true;
            };
            constexpr int NP = MathT::kPages;
            while (k + (NP - 1) * WPH < d.npg)
                if (!run(std::integral_constant<int, NP>{}, NP)) return;
            while (k < d.npg)
                if (!run(std::integral_constant<int, 2>{}, k + WPH < d.npg ? 2 : 1)) return;
        } else {
            for (; k < d.npg; k += WPH) {
                const uint32_t vis = seen(k);
                if (!mbar_wait(&full[slot], phase, abort)) return;
                uint8_t* kt = ring + slot * 2 * sh.stage_k + pos * kTile;
                uint8_t* vt = kt + sh.stage_k;
                if (vis != 0xffffu) {
                    // rows that do not count may hold anything (NaN included): clear them
                    // in the V tile so that 0 * row stays 0 in the tensor core
                    for (int x = lane; x < D / 64 * 128; x += 32) {
                        const int t = (x >> 3) & 15;
                        if (!((vis >> t) & 1))
                            *reinterpret_cast<uint4*>(vt + (x >> 7) * 2048 + t * 128 + (x & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                    fence_proxy_async_smem();  // before the stage is refilled by TMA
                }
                st.template page<true>(kt, vt, int(vis), lane);
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[slot]);
                advance();
            }
        }

        // ---- the parts meet: part 0 takes the others' states over in order ----
        const int first_part = int(page_base & uint32_t(WPH - 1));  // of the segment's page 0
        page_base += uint32_t(d.npg);
        auto has_pages = [&](int w) { return int((w - first_part) & (WPH - 1)) < d.npg; };
        if (part > 0) {
            if (seg_i > 0 && !mbar_wait(&partempty[head], (seg_i - 1) & 1, abort)) return;
            if (has_pages(part)) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    mine[i * 32 + lane] = make_float4(st.acc[i][0], st.acc[i][1], st.acc[i][2], st.acc[i][3]);
                mine[D / 16 * 32 + lane] = make_float4(st.m[0], st.m[1], st.l[0], st.l[1]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&partfull[head]);
            ++seg_i;
            continue;
        }
        // A cut segment's first piece ends its CTA's share, its last piece
        // starts another's, so with two pieces the last one is usually there
        // already: its arrival is looked up while the parts meet.
        const int nk = d.k1 - d.k0 + 1;
        const int leaf = int(blockIdx.x) - d.k0;
        int32_t* top = p.counters + int64_t(d.b) * p.Hkv + g;
        const bool there = nk == 2 && leaf == 0 && ld_acquire_gpu(top) == 1;
        if (WPH > 1 && !mbar_wait(&partfull[head], seg_i & 1, abort)) return;
        for (int w = 1; w < WPH; ++w) {
            if (!has_pages(w)) continue;
            const float4* o =
                reinterpret_cast<const float4*>(smem + lay.parts + ((w - 1) * HG + head) * part_bytes(D));
            const float4 ml = o[D / 16 * 32 + lane];
            const float n0 = fmaxf(st.m[0], ml.x), n1 = fmaxf(st.m[1], ml.y);
            // a state that has seen no token has m = -inf and sums of 0
            const float a0 = exp2f(st.m[0] - n0), a1 = exp2f(st.m[1] - n1);
            const float w0 = exp2f(ml.x - n0), w1 = exp2f(ml.y - n1);
            st.m[0] = n0;
            st.m[1] = n1;
            st.l[0] = st.l[0] * a0 + ml.z * w0;
            st.l[1] = st.l[1] * a1 + ml.w * w1;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const float4 v = o[i * 32 + lane];
                st.acc[i][0] = st.acc[i][0] * a0 + v.x * w0;
                st.acc[i][1] = st.acc[i][1] * a1 + v.y * w1;
                st.acc[i][2] = st.acc[i][2] * a0 + v.z * w0;
                st.acc[i][3] = st.acc[i][3] * a1 + v.w * w1;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&partempty[head]);

        // ---- segment end: this (b, g)'s result, or its piece and the merge of the pieces ----
        auto slot_of = [&](int lf) -> int64_t { return (leaf_slot(d.k0, lf) * HG + head) * G; };
        const int64_t ps = slot_of(leaf);
        if constexpr (I8) st.join_halves();
        st.finish();
        bool last = nk == 1 || __all_sync(0xffffffffu, there);
        if (!last) {
            RawPiece<G>::store(st, p.part_o + ps * D, p.part_ml + ps, lane);
            if (nk <= kWideFanIn) {
                last = arrive_last(top, nk, lane);
                if (last && nk > 2) {
                    merge_raw<D, G>(p, d.k0, 0, 1, nk, HG, head, lane, p.out + row * D);
                    if (lane == 0) *top = 0;
                    last = false;
                }
            } else {
                // runs of about sqrt(nk) pieces, each merged by the last of its
                // pieces to arrive, then the runs by the last of them
                int fan = 2;
                while (fan * fan < nk) ++fan;
                const int first = leaf - leaf % fan;
                const int runs = (nk + fan - 1) / fan;
                const int in_run = nk - first < fan ? nk - first : fan;
                int32_t* gc = p.slot_sync + leaf_slot(d.k0, first) * HG + head;
                if (arrive_last(gc, in_run, lane)) {
                    merge_raw<D, G>(p, d.k0, first, 1, in_run, HG, head, lane, nullptr);
                    if (lane == 0) *gc = 0;
                    if (arrive_last(top, runs, lane)) {
                        merge_raw<D, G>(p, d.k0, 0, fan, runs, HG, head, lane, p.out + row * D);
                        if (lane == 0) *top = 0;
                    }
                }
            }
        }
        if (last) {
            if (nk == 2) {
                const int64_t os = slot_of(1 - leaf);
                RawPiece<G>::fold(st, p.part_o + os * D, p.part_ml + os, leaf == 1, lane);
                if (lane == 0) *top = 0;
            }
            st.store_out(p.out + row * D, lane);
        }
        ++seg_i;
    }
}

}  // namespace pa
