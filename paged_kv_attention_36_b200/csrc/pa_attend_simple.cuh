// pa_attend_simple.cuh -- attention over the paged cache, one warp per
// (query token, query head), fp32 CUDA cores: the plainest kernel of the
// windowed and the 8-bit calls, right for every shape they take.
#pragma once

#include "pa_decode.cuh"

namespace pa {

struct AttendParams {
    const __nv_bfloat16* q;       // [total][Hq][D]
    const void* k_cache;          // bf16 [NB][Hkv][16][D], or int8 codes
    const void* v_cache;          // bf16 [NB][Hkv][16][D], or int8 codes [NB][Hkv][D][16]
    const float* k_scale;         // [NB][Hkv], null for bf16 caches
    const float* v_scale;
    const int32_t* cu_q_lens;     // [B + 1], null for a decode (one token per sequence)
    const int32_t* block_tables;  // [B][M]
    const int32_t* context_lens;  // [B]
    __nv_bfloat16* out;
    int32_t B, Hq, Hkv, NB, M;
    int32_t window, sinks;
    float qscale;                 // scale * log2(e)
};

template <int D, bool I8>
__global__ void __launch_bounds__(128) attend_simple_kernel(AttendParams p) {
    constexpr int E = D / 32;  // values of a row a lane holds: d = lane + 32 e
    const int b = blockIdx.x, lane = threadIdx.x & 31;
    const int h = blockIdx.y * 4 + (threadIdx.x >> 5);
    if (h >= p.Hq) return;
    const int g = h / (p.Hq / p.Hkv);
    int32_t L = p.context_lens[b];
    const bool report = blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0;
    if (L < 0 || L > p.M * 16) {
        if (report) raise_error(PA_DEVERR_CONTEXT);
        L = L < 0 ? 0 : p.M * 16;
    }
    int32_t row0 = b, n = 1;
    if (p.cu_q_lens) {
        row0 = p.cu_q_lens[b];
        n = p.cu_q_lens[b + 1] - row0;
        if (n < 0 || n > L) {
            if (report) raise_error(PA_DEVERR_CONTEXT);
            n = n < 0 ? 0 : L;
        }
    }
    for (int i = blockIdx.z; i < n; i += gridDim.z) {
        const int64_t at = (int64_t(row0 + i) * p.Hq + h) * D;
        float q[E], o[E], m = -INFINITY, l = 0.f;
        for (int e = 0; e < E; ++e) {
            q[e] = __bfloat162float(p.q[at + lane + 32 * e]) * p.qscale;
            o[e] = 0.f;
        }
        const int32_t seen = L - n + i + 1;  // tokens up to the query's own
        const int32_t first = seen > p.window ? seen - p.window : 0;
        for (int32_t t = 0; t < seen; ++t) {
            if (t == p.sinks && t < first) t = first;  // between the sinks and the window
            int32_t blk = p.block_tables[int64_t(b) * p.M + t / 16];
            if (blk < 0 || blk >= p.NB) {
                if (lane == 0) raise_error(PA_DEVERR_BLOCK_ID);
                blk = 0;
            }
            const int64_t tile = int64_t(blk) * p.Hkv + g;
            float s = 0.f, v[E];
            for (int e = 0; e < E; ++e) {
                const int d = lane + 32 * e;
                float k;
                if constexpr (I8) {
                    k = float(static_cast<const int8_t*>(p.k_cache)[(tile * 16 + t % 16) * D + d]) * p.k_scale[tile];
                    v[e] = float(static_cast<const int8_t*>(p.v_cache)[(tile * D + d) * 16 + vt_position(t % 16)]) *
                           p.v_scale[tile];
                } else {
                    k = __bfloat162float(static_cast<const __nv_bfloat16*>(p.k_cache)[(tile * 16 + t % 16) * D + d]);
                    v[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v_cache)[(tile * 16 + t % 16) * D + d]);
                }
                s += q[e] * k;
            }
            for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            const float mn = fmaxf(m, s), a = exp2f(m - mn), w = exp2f(s - mn);
            m = mn;
            l = l * a + w;
            for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * v[e];
        }
        for (int e = 0; e < E; ++e) p.out[at + lane + 32 * e] = __float2bfloat16_rn(seen > 0 ? o[e] / l : 0.f);
    }
}

}  // namespace pa
