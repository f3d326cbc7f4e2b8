// pa_prefill_i8.cuh -- multi-query (chunked prefill) attention over the 8-bit
// cache with a scale for each (block, kv head), with a sliding window and
// sinks, on the tcgen05 tensor cores.
//
// The tile, its walk over the listed pages in blocks of 64 tokens, the lazy
// softmax and the MMA order are those of pa_prefill_tc.cuh.  What differs:
//
//   * Four converter warps take the place of the TMA producer.  They read the
//     tiles' codes into registers one block ahead (a tile is contiguous: each
//     thread has the same 16 bytes of every page), and write f16 operands
//     into the swizzled ring.  A code b becomes an f16 by its bytes,
//     0x6400 | (b ^ 0x80) is 1152 + b, and an exact subtraction.  (Keys that
//     kept the 1152 would save the subtraction, but their logits would be
//     differences of sums as large as 1152 sum(q).)
//   * V stays transposed: its tile rows are head_dim, so a block is the
//     K-major B operand [D][64 tokens] of P V.
//   * Queries are scaled by a power of two to below 4 in f16, which loses
//     nothing bf16 holds down to 2^-14 of the row's largest value.
//   * Scales cost no work per value: with c = scale * log2(e) * k_scale of
//     the page and v = log2(v_scale), P = 2^(s c + (v - m)) is the
//     weight times v_scale, so P V needs no scale, and l adds the page's sum
//     of P times 1 / v_scale.  m is the largest exponent less kLift, raised
//     when one passes it by 15: P lies in [0, 2^15], and f16's smallest step
//     is 2^-31 of the heaviest contribution.
//   * setmaxnreg moves registers from the converters to the softmax.
//   * SPLIT: a cluster of CTAs shares each tile's keys (KeySplit).
//
// Bound by the hand-offs: of the 3500 cycles of a block with clock stamps in
// the loops the softmax works 1980 and waits 1520 for S, the converters work
// 2010 and wait 1390 for a free slot (two ring blocks, two S buffers); 51 % of
// the issue slots are taken, the tensor pipe is busy 28 % of the time.
// Measured on B200: 16 chunks of 512 tokens behind 0-3500, 32/8 heads of 128:
// 457 us, 589 TFLOP/s of visible pairs (floor at 1624 TFLOP/s: 166 us).
#pragma once

#include "pa_prefill_tc.cuh"

namespace pa {

// f16 x f16 -> f32, A and B K-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
    return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

template <int D>
struct I8PrefillCfg {
    static constexpr int kBM = 128, kBN = 64;
    static constexpr int kPages = kBN / 16;
    static constexpr int kPanels = D / 64;
    static constexpr int kPanelQ = kBM * 128;   // bytes of a 64-wide panel of Q
    static constexpr int kPanelK = kBN * 128;   // and of a K block
    static constexpr int kQBytes = kPanels * kPanelQ;
    static constexpr int kKBytes = kBN * D * 2;  // a K block; a V block ([D][64 tokens]) has as many
    static constexpr int kStage = 2 * kKBytes;
    static constexpr int KS = D == 64 ? 4 : 2;   // ring blocks
    static constexpr int NS = D == 64 ? 3 : 2;   // S buffers in TMEM
    static constexpr int kBarOff = kQBytes + KS * kStage;
    static constexpr int kNumBars = 1 + 4 * KS + 2 * NS + 1;
    static constexpr int kSmemBytes = kBarOff + kNumBars * 8 + 16 + 1024;
    static constexpr int kThreads = 384;  // warps 0-3 softmax, 4-7 converters, 8 MMA issue, 9-11 idle
    static constexpr int kTmemCols = 256;
    // registers: two CTAs of 12 warps leave 80 a thread; the converters and
    // the MMA warps hand theirs to the softmax
    static constexpr int kRegs = 80, kSoftmaxRegs = 152, kConvertRegs = 64, kIssueRegs = 24;
    static_assert(kSoftmaxRegs + kConvertRegs + kIssueRegs <= 3 * kRegs, "register pool");
    static_assert(NS * kBN + D <= kTmemCols, "TMEM columns");
    static_assert(2 * (kSmemBytes + 1024) <= 233472, "two CTAs per SM");
};

// tmem_ld64 as two loads of 32 columns under one wait (a single x64 load does
// not fit the registers the kernel is launched with).
__device__ __forceinline__ void tmem_ld2x32(uint32_t taddr, float* v) {
    uint32_t r[64];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr), "r"(taddr + 32)
        : "memory");
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

struct PrefillI8Params {
    PrefillParams a;         // tensor maps unused
    const int8_t* k_cache;   // [NB][Hkv][16][D]
    const int8_t* v_cache;   // [NB][Hkv][D][16]
    const float* k_scale;    // [NB][Hkv]
    const float* v_scale;
};

// 16 codes as f16 pairs in order: words 0-3 the first 8 values, 4-7 the next.
__device__ __forceinline__ void codes_to_f16(const uint4& r, uint32_t (&o)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = w[i] ^ 0x80808080u;
        o[2 * i] = __byte_perm(x, 0x64646464u, 0x4140);
        o[2 * i + 1] = __byte_perm(x, 0x64646464u, 0x4342);
        const __half2 b = __floats2half2_rn(1152.f, 1152.f);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&o[2 * i + k]), b);
            o[2 * i + k] = *reinterpret_cast<const uint32_t*>(&v);
        }
    }
}

template <int D, int G, bool SPLIT>
__global__ void __launch_bounds__(I8PrefillCfg<D>::kThreads, 2) prefill_i8_kernel(const __grid_constant__
                                                                                  PrefillI8Params pp) {
    using Cfg = I8PrefillCfg<D>;
    constexpr int BN = Cfg::kBN, KS = Cfg::KS, NS = Cfg::NS;
    constexpr float kLift = 7.f;
    const PrefillParams& p = pp.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* qs = smem;
    uint8_t* stages = smem + Cfg::kQBytes;
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff);
    uint64_t* k_full = q_full + 1;
    uint64_t* v_full = k_full + KS;
    uint64_t* k_empty = v_full + KS;
    uint64_t* v_empty = k_empty + KS;
    uint64_t* s_full = v_empty + KS;
    uint64_t* p_full = s_full + NS;
    uint64_t* drain = p_full + NS;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    int* s_abort = reinterpret_cast<int*>(tmem_slot + 1);
    volatile int* abort = s_abort;
    int& s_ranks = s_abort[1];  // CTAs that share the tile
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- this tile's rows and the pages it attends ----
    const TileOfCta cta(p, int(SPLIT ? blockIdx.x / cluster_size() : blockIdx.x));
    const int b = cta.b, tile = cta.tile, g = cta.g;
    const bool report = tile == 0 && g == 0 && threadIdx.x == 0;
    int L = __ldca(p.context_lens + b);
    const int64_t cap = int64_t(p.M) * 16;
    if (L < 0 || L > cap) {
        if (report) raise_error(PA_DEVERR_CONTEXT);
        L = L < 0 ? 0 : int32_t(cap);
    }
    const int q0 = __ldca(p.cu_q_lens + b);
    int32_t q_len = __ldca(p.cu_q_lens + b + 1) - q0;
    if (q_len < 0 || q_len > L) {
        if (report) raise_error(PA_DEVERR_CONTEXT);
        q_len = q_len < 0 ? 0 : L;
    }
    const int nrows = q_len * G, row0 = tile * Cfg::kBM;
    if (row0 >= nrows) return;  // whole CTA, before any barrier or TMEM use
    const int first_pos = L - q_len;
    const int last_row = (row0 + Cfg::kBM < nrows ? row0 + Cfg::kBM : nrows) - 1;
    int nkeys = first_pos + last_row / G + 1;
    // the list: the pages of the sinks, then those from the first row's window on
    const WindowPages listed(window_first(first_pos + row0 / G, p.window), nkeys, p.sinks);
    const int skip = listed.skip;
    nkeys -= skip * 16;
    int pages = (nkeys + 15) / 16, nblk = (nkeys + BN - 1) / BN;
    const int32_t* bt = p.block_tables + int64_t(b) * p.M;
    int ns = listed.ns, shift = skip * 16, sinks = p.sinks;
    if constexpr (SPLIT) {
        const KeySplit split(nblk);
        if (int(cluster_rank()) >= split.ranks) return;  // before any barrier or TMEM use
        if (threadIdx.x == 0) s_ranks = split.ranks;
        // the list from this rank's first block on: pages, keys and sinks count from there
        const int first_pg = int(cluster_rank()) * split.per * Cfg::kPages;
        bt += first_pg;
        ns -= first_pg;
        shift += first_pg * 16;
        sinks -= first_pg * 16;
        nkeys -= first_pg * 16;
        pages -= first_pg;
        if (pages > split.per * Cfg::kPages) pages = split.per * Cfg::kPages;
        nblk = (pages + Cfg::kPages - 1) / Cfg::kPages;
    }
    // (block, kv head) tile of listed page pg; past the list its last page again
    // (masked, and not multiplied)
    auto tile_of = [&](int pg) -> int {
        if (pg >= pages) pg = pages - 1;
        int32_t blk = __ldca(bt + (pg < ns ? pg : pg + skip));
        if (blk < 0 || blk >= p.NB) {
            raise_error(PA_DEVERR_BLOCK_ID);
            blk = 0;
        }
        return blk * p.Hkv + g;
    };

    if (threadIdx.x == 0) {
        mbar_init(q_full, 128);
        for (int s = 0; s < KS; ++s) {
            mbar_init(&k_full[s], 128);
            mbar_init(&v_full[s], 128);
            mbar_init(&k_empty[s], 1);
            mbar_init(&v_empty[s], 1);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
        }
        mbar_init(drain, 1);
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(tmem_slot, Cfg::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t t_o = tmem + NS * BN;  // O columns; S buffer i at tmem + i*BN

    if (warp >= 8) {
        // ===================== MMA issue (one thread) =====================
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kIssueRegs));
        if (warp == 8 && lane == 0) {
            constexpr uint32_t id_qk = idesc_f16_f32(128, BN);
            constexpr uint32_t id_pv = idesc_f16_f32(128, D);
            const uint64_t qd = sw128_desc(smem_u32(qs), 16, 1024);
            const uint32_t st0 = smem_u32(stages);
            bool ok = mbar_wait_sleep(q_full, 0, abort);
            // S_i = Q K_i^T into buffer i % NS, once the P V that last read it has completed
            auto issue_qk = [&](int i) -> bool {
                const int s = i % KS, bb = i % NS;
                if (!mbar_wait_sleep(&k_full[s], uint32_t(i / KS) & 1, abort)) return false;
                if (i >= NS && !mbar_wait_sleep(&v_empty[(i - NS) % KS], uint32_t((i - NS) / KS) & 1, abort))
                    return false;
                tc_fence_after();
                const uint64_t kd = sw128_desc(st0 + s * Cfg::kStage, 16, 1024);
#pragma unroll
                for (int c = 0; c < Cfg::kPanels; ++c)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_ss(tmem + bb * BN, qd + uint64_t((c * Cfg::kPanelQ + kk * 32) >> 4),
                                kd + uint64_t((c * Cfg::kPanelK + kk * 32) >> 4), id_qk, uint32_t(c | kk));
                umma_commit(&s_full[bb]);
                umma_commit(&k_empty[s]);
                return true;
            };
            for (int i = 0; ok && i < NS - 1 && i < nblk; ++i) ok = issue_qk(i);
            for (int j = 0; ok && j < nblk; ++j) {
                if (j + NS - 1 < nblk && !(ok = issue_qk(j + NS - 1))) break;
                const int s = j % KS, bb = j % NS;
                ok = mbar_wait_sleep(&p_full[bb], uint32_t(j / NS) & 1, abort) &&
                     mbar_wait_sleep(&v_full[s], uint32_t(j / KS) & 1, abort);
                if (!ok) break;
                tc_fence_after();
                const int npg = pages - j * Cfg::kPages < Cfg::kPages ? pages - j * Cfg::kPages : Cfg::kPages;
                const uint64_t vd = sw128_desc(st0 + s * Cfg::kStage + Cfg::kKBytes, 16, 1024);
#pragma unroll
                for (int pg = 0; pg < Cfg::kPages; ++pg)
                    if (pg < npg) umma_ts(t_o, tmem + bb * BN + pg * 8, vd + uint64_t(pg * 2), id_pv, uint32_t(j | pg));
                umma_commit(&v_empty[s]);
            }
            // no MMA may still run when TMEM and shared memory are released
            umma_commit(drain);
            mbar_wait_sleep(drain, 0, nullptr, 20000000ull);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ========================= converter warps =========================
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kConvertRegs));
        constexpr int NP = D / 32;  // pages of a block that a thread has 16 bytes of
        const int ct = threadIdx.x - 128;
        // byte offset within a tile, and the pages of a block (D = 128: all, a
        // tile is 128 pieces; D = 64: every second, half the threads each)
        const int off = (D == 128 ? ct : ct & 63) * 16;
        auto page_in_block = [&](int i) { return D == 128 ? i : 2 * i + (ct >> 6); };
        // where the 16 values go: K row t, columns 16 cc ..; V row d, tokens of the page
        const int t_in = off / D, cc = off % D / 16, d_in = off / 16;
        int tl[NP], tl_next[NP];  // tiles of block t, and of block t + 1
        uint4 kr[NP], vr[NP];
        auto tiles_of = [&](int j, int (&t)[NP]) {
#pragma unroll
            for (int i = 0; i < NP; ++i) t[i] = tile_of(j * Cfg::kPages + page_in_block(i));
        };
        auto fetch = [&](const int8_t* cache, const int (&t)[NP], uint4 (&r)[NP]) {
#pragma unroll
            for (int i = 0; i < NP; ++i)
                r[i] = __ldca(reinterpret_cast<const uint4*>(cache + int64_t(t[i]) * (16 * D) + off));
        };
        tiles_of(0, tl);
        fetch(pp.k_cache, tl, kr);
        fetch(pp.v_cache, tl, vr);
        tiles_of(1, tl_next);
        bool ok = true;
        // K runs one block ahead of V; each half's registers are refilled as
        // soon as they are written out
        int tv[NP];  // tiles of the V block to fetch next
#pragma unroll
        for (int i = 0; i < NP; ++i) tv[i] = tl_next[i];
        for (int t = 0; t <= nblk; ++t) {
            if (t < nblk) {
                const int s = t % KS;
                if (t >= KS && !(ok = __all_sync(0xffffffffu, mbar_wait_sleep(&k_empty[s], uint32_t(t / KS - 1) & 1,
                                                                              abort))))
                    break;
                uint8_t* kb = stages + s * Cfg::kStage;
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    // two 16-byte chunks of the row; the second panel's threads write
                    // theirs in the other order, into the banks the first's leave
                    const bool f = D == 128 && cc >= 4;
                    uint32_t o[8];
                    codes_to_f16(f ? make_uint4(kr[i].z, kr[i].w, kr[i].x, kr[i].y) : kr[i], o);
                    const int row = page_in_block(i) * 16 + t_in;  // row % 8 = t_in % 8
                    uint8_t* dst = kb + (cc >> 2) * Cfg::kPanelK + row * 128;
                    const int ch = ((cc & 3) * 2) ^ (t_in & 7) ^ (f ? 1 : 0);
                    *reinterpret_cast<uint4*>(dst + (ch << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4*>(dst + ((ch ^ 1) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
                }
                fence_proxy_async_smem();
                mbar_arrive(&k_full[s]);
                if (t + 1 < nblk) {
                    fetch(pp.k_cache, tl_next, kr);
#pragma unroll
                    for (int i = 0; i < NP; ++i) tl[i] = tl_next[i];
                    tiles_of(t + 2, tl_next);
                }
            }
            if (t >= 1) {
                const int j = t - 1, s = j % KS;
                if (j >= KS && !(ok = __all_sync(0xffffffffu, mbar_wait_sleep(&v_empty[s], uint32_t(j / KS - 1) & 1,
                                                                              abort))))
                    break;
                uint8_t* vb = stages + s * Cfg::kStage + Cfg::kKBytes;
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    // stored byte order: words hold tokens 2c, 2c+1, 2c+8, 2c+9
                    uint32_t o[8];
                    codes_to_f16(vr[i], o);
                    uint8_t* dst = vb + d_in * 128;
                    const int ch = page_in_block(i) * 2;
                    *reinterpret_cast<uint4*>(dst + ((ch ^ (d_in & 7)) << 4)) = make_uint4(o[0], o[2], o[4], o[6]);
                    *reinterpret_cast<uint4*>(dst + (((ch + 1) ^ (d_in & 7)) << 4)) = make_uint4(o[1], o[3], o[5], o[7]);
                }
                fence_proxy_async_smem();
                mbar_arrive(&v_full[s]);
                if (t < nblk) {  // block t's V: its tiles are tv
                    fetch(pp.v_cache, tv, vr);
#pragma unroll
                    for (int i = 0; i < NP; ++i) tv[i] = tl[i];
                }
            }
        }
    } else {
        // ========================= softmax warpgroup =========================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kSoftmaxRegs));
        const int row = threadIdx.x;  // of the tile; TMEM lane
        const uint32_t lanes = uint32_t(warp * 32) << 16;
        const int r = row0 + row;
        const bool valid = r < nrows;
        // list keys [0, sink) and [lo, lim) are visible (rows past the task as its last one)
        const int lim = valid ? first_pos + r / G + 1 - shift : nkeys;
        const int lo = window_first(lim - 1 + shift, p.window) - shift;
        const int sink = sinks < lim ? sinks : lim;

        // ---- Q row: a power of two times it, as f16, in shared memory ----
        float ce;  // logits = s * ce * k_scale
        {
            uint4 qv[D / 8];
            const uint4* src =
                reinterpret_cast<const uint4*>(p.q + ((int64_t(q0) + r / G) * p.Hq + g * G + r % G) * (D * 2));
            float top = 0.f;
#pragma unroll
            for (int ch = 0; ch < D / 8; ++ch) {
                qv[ch] = valid ? __ldca(src + ch) : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t w[4] = {qv[ch].x, qv[ch].y, qv[ch].z, qv[ch].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = bf16x2_to_float2(w[i]);
                    top = fmax3(top, fabsf(f.x), fabsf(f.y));
                }
            }
            // v * down is exact and below 4, whatever finite values the row has
            int e = int(__float_as_uint(top) >> 23) - 127;
            e = e < -126 ? -126 : e > 126 ? 126 : e;
            const float down = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
            for (int ch = 0; ch < D / 8; ++ch) {
                uint32_t w[4] = {qv[ch].x, qv[ch].y, qv[ch].z, qv[ch].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = bf16x2_to_float2(w[i]);
                    w[i] = float2_to_f16x2(f.x * down, f.y * down);
                }
                *reinterpret_cast<uint4*>(qs + (ch >> 3) * Cfg::kPanelQ + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
            fence_proxy_async_smem();
            mbar_arrive(q_full);
            ce = p.qscale * __uint_as_float(uint32_t(127 + e) << 23);
        }
        const bool positive = ce > 0.f;

        // lane i of each warp holds page i % 4's scales, read one block ahead
        auto page_tile = [&](int j) { return tile_of(j * Cfg::kPages + (lane & (Cfg::kPages - 1))); };
        const int tl = page_tile(0);
        float ks_next = __ldca(pp.k_scale + tl), vs_next = __ldca(pp.v_scale + tl);
        int tl_next = page_tile(1);

        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < nblk; ++j) {
            const int bb = j % NS, n0 = j * BN;
            const float ks = ks_next, vs = vs_next;
            ks_next = __ldca(pp.k_scale + tl_next);
            vs_next = __ldca(pp.v_scale + tl_next);
            tl_next = page_tile(j + 2);
            // a scale of 0: codes of 0, weight still in l; NaN stays
            const float lvl = vs <= 0x1p-100f ? -100.f : __log2f(vs);
            const float inv = ex2_approx(-lvl);

            ok = __all_sync(0xffffffffu, mbar_wait_sleep(&s_full[bb], uint32_t(j / NS) & 1, abort));
            if (!ok) break;
            tc_fence_after();
            float s[BN];
            tmem_ld2x32(tmem + lanes + bb * BN, s);
            if (!positive) {
#pragma unroll
                for (int i = 0; i < BN; ++i) s[i] *= ce;
            }
            // exponent of value s in page pg: s * c[pg] + a[pg].  c stays above 0, so that
            // a masked value (s = -inf) keeps its exponent where the keys or the row are 0
            // or tiny: |s| < 2^16, so the other exponents do not notice
            float c[Cfg::kPages], a[Cfg::kPages];
#pragma unroll
            for (int pg = 0; pg < Cfg::kPages; ++pg) {
                const float k1 = __shfl_sync(0xffffffffu, ks, pg), v1 = __shfl_sync(0xffffffffu, lvl, pg);
                const float c1 = positive ? ce * k1 : k1;
                c[pg] = c1 < 0x1p-126f ? 0x1p-126f : c1;  // NaN stays
                a[pg] = v1;
            }
            if (!(n0 >= lo && n0 + BN <= lim) && n0 + BN > sink) {
#pragma unroll
                for (int i = 0; i < BN; ++i)
                    if (n0 + i >= sink && (n0 + i < lo || n0 + i >= lim)) s[i] = -INFINITY;
#pragma unroll
                for (int pg = 0; pg < Cfg::kPages; ++pg) {
                    // a page of which the row sees nothing: its scales stay out
                    const int n = n0 + 16 * pg;
                    if (n >= sink && (n + 16 <= lo || n >= lim)) {
                        c[pg] = 1.f;
                        a[pg] = 0.f;
                    }
                }
            }
            float m_blk = -INFINITY;
#pragma unroll
            for (int pg = 0; pg < Cfg::kPages; ++pg) {
                const float* x = &s[16 * pg];
                float u = fmax3(x[0], x[1], x[2]), v = fmax3(x[3], x[4], x[5]);
                u = fmax3(u, x[6], x[7]);
                v = fmax3(v, x[8], x[9]);
                u = fmax3(u, x[10], x[11]);
                v = fmax3(v, x[12], x[13]);
                u = fmax3(u, x[14], x[15]);
                m_blk = fmaxf(m_blk, fmaf(fmaxf(u, v), c[pg], a[pg]));
            }
            if (__any_sync(0xffffffffu, m_blk > m + 15.f)) {
                const float m_new = fmaxf(m, m_blk - kLift);
                // 0 while m = -inf; a row that has not seen a key yet keeps O = 0 and l = 0
                const float alpha = m_new == -INFINITY ? 1.f : ex2_approx(m - m_new);
                if (j > 0) {
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait_sleep(&v_empty[(j - 1) % KS], uint32_t((j - 1) / KS) & 1, abort));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        float o[32];
                        tmem_ld32(t_o + lanes + 32 * k, o);
                        uint32_t w[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(o[i] * alpha);
                        tmem_st32(t_o + lanes + 32 * k, w);
                    }
                }
                l *= alpha;
                m = m_new;
            }
            const float mu = m == -INFINITY ? 0.f : m;
            // P as f16 pairs over the first BN/2 columns of the buffer
            uint32_t w[BN / 2];
#pragma unroll
            for (int pg = 0; pg < Cfg::kPages; ++pg) {
                const uint64_t c2 = f2_pack(c[pg], c[pg]), a2 = f2_pack(a[pg] - mu, a[pg] - mu);
                uint64_t acc0 = 0ull, acc1 = 0ull;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float t0, t1;
                    f2_unpack(f2_fma(f2_pack(s[16 * pg + 2 * i], s[16 * pg + 2 * i + 1]), c2, a2), t0, t1);
                    const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
                    if (i & 1) acc1 = f2_add(acc1, f2_pack(p0, p1));
                    else acc0 = f2_add(acc0, f2_pack(p0, p1));
                    w[8 * pg + i] = float2_to_f16x2(p0, p1);
                }
                float x, y;
                f2_unpack(f2_add(acc0, acc1), x, y);
                const float by = __shfl_sync(0xffffffffu, inv, pg);
                l = x + y != 0.f ? fmaf(x + y, by, l) : l;  // a page the row does not see: whatever its scale
            }
            tmem_st32(tmem + lanes + bb * BN, w);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&p_full[bb]);
        }

        // ---- output: O / l as bf16 rows, staged in the Q and ring space (idle
        // once the last P V has completed), then copied out row by row ----
        if (ok)
            ok = __all_sync(0xffffffffu,
                            mbar_wait_sleep(&v_empty[(nblk - 1) % KS], uint32_t((nblk - 1) / KS) & 1, abort));
        constexpr int kRowStride = D * 2 + 16;
        static_assert(Cfg::kBM * kRowStride <= Cfg::kBarOff, "output staging");
        if (SPLIT && s_ranks > 1) {
            if (ok) {  // this rank's sums, for the cluster
                static_assert(SplitRows<D>::kBytes <= Cfg::kBarOff, "split staging");
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    float o[32];
                    tmem_ld32(t_o + lanes + 32 * k, o);
                    SplitRows<D>::store(smem, row, o, 32 * k);
                }
                *reinterpret_cast<float2*>(smem + SplitRows<D>::kMl + row * 8) = make_float2(m, l);
            }
        } else if (ok) {
            tc_fence_after();
            const float inv = 1.f / l;
            uint8_t* mine = smem + row * kRowStride;
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                float o[64];
                tmem_ld2x32(t_o + lanes + 64 * k, o);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    *reinterpret_cast<uint4*>(mine + (64 * k + 8 * q) * 2) =
                        make_uint4(float2_to_bf16x2(o[8 * q] * inv, o[8 * q + 1] * inv),
                                   float2_to_bf16x2(o[8 * q + 2] * inv, o[8 * q + 3] * inv),
                                   float2_to_bf16x2(o[8 * q + 4] * inv, o[8 * q + 5] * inv),
                                   float2_to_bf16x2(o[8 * q + 6] * inv, o[8 * q + 7] * inv));
            }
        }
        if (SPLIT && s_ranks > 1) {
            __syncwarp();
            cluster_sync();  // every rank's rows are staged
            SplitRows<D>::join(smem, s_ranks, nrows - row0 < Cfg::kBM ? nrows - row0 : Cfg::kBM, threadIdx.x,
                               [&](int rr) {
                                   const int rg = row0 + rr;
                                   return p.out + ((int64_t(q0) + rg / G) * p.Hq + g * G + rg % G) * D;
                               });
        } else {
            asm volatile("bar.sync 1, 128;" ::: "memory");  // the softmax warps: rows staged
        }
        if (!*abort && !(SPLIT && s_ranks > 1)) {
            constexpr int kChunks = D / 8, kRowsPerPass = 32 / kChunks;
            for (int rr = warp * kRowsPerPass + lane / kChunks; rr < Cfg::kBM; rr += 4 * kRowsPerPass) {
                const int rg = row0 + rr;
                if (rg >= nrows) break;
                const int ch = lane % kChunks;
                const uint4 v = *reinterpret_cast<const uint4*>(smem + rr * kRowStride + ch * 16);
                const int64_t grow = (int64_t(q0) + rg / G) * p.Hq + g * G + rg % G;
                reinterpret_cast<uint4*>(p.out + grow * D)[ch] = v;
            }
        }
    }

    if (SPLIT && s_ranks > 1) {
        __syncwarp();
        if (warp >= 4) cluster_sync();
        cluster_sync();  // every rank's rows are read
    }

    // ---- release TMEM once every warp's tcgen05 work has finished ----
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::kTmemCols);
    }
}

}  // namespace pa
