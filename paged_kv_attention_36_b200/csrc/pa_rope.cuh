// pa_rope.cuh -- the step's append with the position rotation on the way:
// q and k rows are turned by the angles of their tokens' positions, k and v
// land in their slots of the paged cache (bf16, or 8-bit codes with a scale
// for each (block, kv head)).
//
// A row's first rd values are rd/2 pairs; pair i is (x_i, x_{i+rd/2}), or
// (x_2i, x_2i+1) when interleaved, and becomes
//     (a cos_i - b sin_i,  b cos_i + a sin_i)
// with the angles' cosines and sines read from the caller's fp32 table
// [max_position][rd] (rd/2 cosines, then rd/2 sines).  Products and sums are
// single fp32 operations (no contraction), rounded once at the end.
#pragma once

#include "pa_append.cuh"
#include "pa_device.cuh"

namespace pa {

struct RopeParams {
    const __nv_bfloat16* q;       // [T][Hq][D], token stride q_stride (null: no queries)
    const __nv_bfloat16* k_new;   // [T][Hkv][D], token stride k_stride
    const __nv_bfloat16* v_new;   // [T][Hkv][D], token stride v_stride
    int64_t q_stride, k_stride, v_stride;  // in values
    const int32_t* positions;     // [T]
    const float* cos_sin;         // [max_position][rd]
    const int32_t* slot_mapping;  // [T]
    __nv_bfloat16* q_out;         // [T][Hq][D]
    void* k_cache;                // bf16 [NB][Hkv][bs][D], or int8 [NB][Hkv][16][D]
    void* v_cache;                // bf16 [NB][Hkv][bs][D], or int8 [NB][Hkv][D][16]
    float* k_scale;               // [NB][Hkv] (8-bit)
    float* v_scale;
    int32_t T, Hq, Hkv, D, bs, NB;
    int32_t max_position, rd, interleaved;
    int32_t kv_ctas;              // 8-bit: the first kv_ctas CTAs take the blocks, the others the queries
    int32_t tokens_per_cta;       // 8-bit: tokens whose blocks a CTA looks at, at most 32
};

constexpr int kRopeThreads = 256;

// (a, b) turned by the angle whose cosine and sine are c and s.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// The table row of token t's position (its own row 0, with an error, if the
// position has none).
__device__ __forceinline__ const float* angles(const RopeParams& p, int64_t t, bool report) {
    int32_t pos = __ldg(p.positions + t);
    if (pos < 0 || pos >= p.max_position) {
        if (report) raise_error(PA_DEVERR_POSITION);
        pos = 0;
    }
    return p.cos_sin + int64_t(pos) * p.rd;
}

// 16 values of a row as two 16-byte chunks: the columns of chunk pair c of a
// row of D values (c < D/16).  Rotated pairs lie within one chunk pair.
struct ChunkPair {
    int32_t lo, hi;  // first columns of the two chunks
    int32_t angle;   // index of the first angle, -1 past the rotated part
};
__device__ __forceinline__ ChunkPair chunk_pair(int c, int rd, bool interleaved) {
    const int n = rd / 16;  // chunk pairs that are rotated
    if (c >= n) return {16 * c, 16 * c + 8, -1};
    if (interleaved) return {16 * c, 16 * c + 8, 8 * c};
    return {8 * c, 8 * c + rd / 2, 8 * c};
}

// Turns the 16 values of a chunk pair in place (8 angles, cosines cs[0..7], sines cs[rd/2 ..]).
__device__ __forceinline__ void turn_chunks(uint4& lo, uint4& hi, const float (&c)[8], const float (&s)[8],
                                            bool interleaved) {
    uint32_t* w[2] = {&lo.x, &hi.x};
    float x[16];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = bf16x2_to_float2(w[h][j]);
            x[8 * h + 2 * j] = f.x;
            x[8 * h + 2 * j + 1] = f.y;
        }
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn(x[2 * i], x[2 * i + 1], c[i], s[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn(x[i], x[8 + i], c[i], s[i]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) w[h][j] = float2_to_bf16x2(x[8 * h + 2 * j], x[8 * h + 2 * j + 1]);
}

// HP rows of token t from head h0 on (heads 0 .. Hq-1 are the queries, then
// the keys, then the values), chunk pair c.  The angles are read once for
// the HP rows, and the rows' loads are in flight together.
template <int HP>
__device__ __forceinline__ void rope_rows(const RopeParams& p, int t, int h0, int heads, int c) {
    const int32_t slot = __ldg(p.slot_mapping + t);
    const ChunkPair cp = chunk_pair(c, p.rd, p.interleaved);
    if (slot < 0) return;  // padding
    const int32_t block = slot / p.bs, offset = slot - block * p.bs;
    const bool stored = block < p.NB;
    if (!stored && c == 0 && h0 == 0) raise_error(PA_DEVERR_SLOT);
    uint4 lo[HP], hi[HP];
    __nv_bfloat16* dst[HP];
#pragma unroll
    for (int i = 0; i < HP; ++i) {
        const int h = h0 + i;
        const __nv_bfloat16* src;
        if (h < p.Hq) {
            src = p.q + t * p.q_stride + h * p.D;
            dst[i] = p.q_out + (int64_t(t) * p.Hq + h) * p.D;
        } else {
            const bool v = h >= p.Hq + p.Hkv;
            const int g = h - p.Hq - (v ? p.Hkv : 0);
            src = v ? p.v_new + t * p.v_stride + g * p.D : p.k_new + t * p.k_stride + g * p.D;
            dst[i] = static_cast<__nv_bfloat16*>(v ? p.v_cache : p.k_cache) +
                     ((int64_t(block) * p.Hkv + g) * p.bs + offset) * p.D;
            if (!stored) dst[i] = nullptr;
        }
        if (h >= heads) dst[i] = nullptr;
        if (dst[i]) {
            lo[i] = *reinterpret_cast<const uint4*>(src + cp.lo);
            hi[i] = *reinterpret_cast<const uint4*>(src + cp.hi);
        }
    }
    if (cp.angle >= 0 && h0 < p.Hq + p.Hkv) {
        const float* a = angles(p, t, c == 0 && h0 == 0) + cp.angle;
        float cs[8], sn[8];
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(a + i));
            const float4 y = __ldg(reinterpret_cast<const float4*>(a + p.rd / 2 + i));
            cs[i] = x.x, cs[i + 1] = x.y, cs[i + 2] = x.z, cs[i + 3] = x.w;
            sn[i] = y.x, sn[i + 1] = y.y, sn[i + 2] = y.z, sn[i + 3] = y.w;
        }
#pragma unroll
        for (int i = 0; i < HP; ++i)
            if (dst[i] && h0 + i < p.Hq + p.Hkv) turn_chunks(lo[i], hi[i], cs, sn, p.interleaved);
    }
#pragma unroll
    for (int i = 0; i < HP; ++i)
        if (dst[i]) {
            *reinterpret_cast<uint4*>(dst[i] + cp.lo) = lo[i];
            *reinterpret_cast<uint4*>(dst[i] + cp.hi) = hi[i];
        }
}

// One thread per chunk pair of HP consecutive rows of a token.
template <int HP>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_append_kernel(const __grid_constant__ RopeParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t heads = p.Hq + 2 * p.Hkv, cpr = p.D / 16, per_token = (heads + HP - 1) / HP * cpr;
    const uint32_t i = blockIdx.x * uint32_t(kRopeThreads) + threadIdx.x;
    const uint32_t t = i / per_token, r = i - t * per_token;
    if (t >= uint32_t(p.T)) return;
    rope_rows<HP>(p, int(t), int(r / cpr) * HP, int(heads), int(r % cpr));
}

// ---- 8-bit caches ------------------------------------------------------------
// A block's codes share one scale per kv head, so its new rows are taken
// together: the CTA of the first token (in call order) whose slot lies in
// the block writes all of the call's rows of that block, the CTAs of its
// other tokens leave.  A warp owns one (kv head, K or V) tile at a time.
// Lane l holds four values of a row (16 lanes cover a row at head_dim 64, so
// a warp takes two rows at once there), chosen so that a rotated pair never
// crosses lanes; all 16 rows of its columns stay in registers, so a V row of
// the transposed tile is one 16-byte (head_dim 64: 8-byte) store.
//
//   top = max |x| over the block's new rows,  old = the block's scale (0 if
//   the call writes the block's row 0: the block starts anew),
//   scale = max(old, top / 127),  code = round(x / scale);
//   a larger scale rounds the block's old codes again: round(code old / scale).
//
// Division, product and rounding are IEEE fp32 (ties to even).  NaN and
// infinity go into the scale and poison the block until it starts anew.

// Largest magnitude as bits: non-finite values compare above finite ones, NaN highest.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// round(x / scale) of four values as bytes, the division and the rounding IEEE
// fp32 (ties to even).  t = x * (1/scale) is within 2^-15 of the quotient
// (|t| <= 127 and three roundings), so away from ties it rounds to the same
// code.  Near one, at mid = n +- 1/2: r = x - mid * scale is exact in one fma
// (both sides agree in all but their last bits), and the divided quotient
// rounds to mid itself iff |r| <= scale * half an ulp of mid; then the even
// neighbour is taken, else the side of mid that r says.  Scales whose
// reciprocal leaves the normal range divide.
struct Quantizer {
    float scale, inv;
    bool divide;
    __device__ __forceinline__ explicit Quantizer(float s) : scale(s) {
        divide = !(s > 1e-30f && s < 1e30f);
        inv = divide ? 0.f : 1.f / s;
    }
    __device__ __noinline__ uint32_t divided(float a, float b, float c, float d) const {
        const float x[4] = {a, b, c, d};
        uint32_t w = 0;
        for (int i = 0; i < 4; ++i) {
            int q = scale > 0.f ? __float2int_rn(__fdiv_rn(x[i], scale)) : 0;
            q = q > 127 ? 127 : q < -127 ? -127 : q;
            w |= uint32_t(q & 0xff) << (8 * i);
        }
        return w;
    }
    __device__ __forceinline__ uint32_t operator()(float a, float b, float c, float d) const {
        const float x[4] = {a, b, c, d};
        float n[4], off[4], worst = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float t = x[i] * inv;
            n[i] = t + 12582912.f - 12582912.f;  // rint(t)
            off[i] = t - n[i];
            worst = fmaxf(worst, fabsf(off[i]));
        }
        if (worst > 0.5f - 0x1p-15f) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (fabsf(off[i]) <= 0.5f - 0x1p-15f) continue;
                const float way = off[i] < 0.f ? -1.f : 1.f, mid = n[i] + 0.5f * way;
                const float r = fmaf(-mid, scale, x[i]);
                // half an ulp of mid: 2^(exponent - 24)
                const float half = __uint_as_float((__float_as_uint(mid) & 0x7f800000u) - (24u << 23));
                const bool tie = fabsf(r) <= scale * half;
                const bool odd = (__float_as_uint(n[i] + 12582912.f) & 1u) != 0;
                if (tie ? odd : r * way > 0.f) n[i] += way;
            }
        }
        // the integers in the low bits of n + 12582912, two's complement
        const uint32_t lo = __byte_perm(__float_as_uint(n[0] + 12582912.f), __float_as_uint(n[1] + 12582912.f), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(n[2] + 12582912.f), __float_as_uint(n[3] + 12582912.f), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    }
};

template <int D>
__device__ __forceinline__ void quantize_tile(const RopeParams& p, const int* src, int64_t block, int g, bool v,
                                              uint8_t* stage, int lane) {
    constexpr int LPR = D / 4;        // lanes per row
    constexpr int NR = 16 * LPR / 32;  // rows a lane has: 16, or 8 at head_dim 64
    const int half = lane / LPR, l = lane % LPR;
    // this lane's four columns: lo, lo+1, hi, hi+1
    const int rd = v ? 0 : p.rd;
    int lo = 4 * l, hi = 4 * l + 2;
    const bool rotate = 4 * l < rd;
    if (rotate && !p.interleaved) {
        lo = 2 * l;
        hi = 2 * l + rd / 2;
    }
    // rows in the order of the V tile's bytes: at head_dim 64 the first half
    // warp has tokens 0-3 and 8-11, the second 4-7 and 12-15
    auto row_of = [&](int j) -> int { return NR == 16 ? j : (j & 3) + ((j >> 2) << 3) + 4 * half; };
    const __nv_bfloat16* rows = (v ? p.v_new : p.k_new) + int64_t(g) * D;
    const int64_t stride = v ? p.v_stride : p.k_stride;
    // All of the call's rows of this tile at once into the warp's staging
    // area (row by row from global memory, each group of rows waited a memory
    // latency, twice).
    __syncwarp();
#pragma unroll
    for (int x = lane; x < 16 * (D / 8); x += 32) {
        const int t = src[x / (D / 8)];
        if (t >= 0) cp_async16(stage + x * 16, rows + t * stride + x % (D / 8) * 8);
    }
    cp_async_commit();
    const int64_t tile = block * p.Hkv + g;
    float* scale_at = (v ? p.v_scale : p.k_scale) + tile;
    const bool anew = src[0] >= 0;
    const float old = anew ? 0.f : *scale_at;
    cp_async_wait_all();
    __syncwarp();
    // the lane's four values of row r (token t), turned
    auto load = [&](int r, int t, float (&x)[4]) {
        const uint8_t* row = stage + r * D * 2;
        const float2 a = bf16x2_to_float2(*reinterpret_cast<const uint32_t*>(row + lo * 2));
        const float2 b = bf16x2_to_float2(*reinterpret_cast<const uint32_t*>(row + hi * 2));
        x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
        if (rotate) {
            const float* cs = angles(p, t, false) + 2 * l;
            const float2 c = __ldg(reinterpret_cast<const float2*>(cs));
            const float2 s = __ldg(reinterpret_cast<const float2*>(cs + rd / 2));
            if (p.interleaved) {
                turn(x[0], x[1], c.x, s.x);
                turn(x[2], x[3], c.y, s.y);
            } else {
                turn(x[0], x[2], c.x, s.x);
                turn(x[1], x[3], c.y, s.y);
            }
        }
    };

    uint32_t top = 0;
    bool any_old = false;  // rows of the block that the call does not write
#pragma unroll 4
    for (int j = 0; j < NR; ++j) {
        const int t = src[row_of(j)];
        if (t < 0) {
            any_old = true;
            continue;
        }
        float x[4];
        load(row_of(j), t, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, abs_bits(x[e]));
    }
    top = __reduce_max_sync(0xffffffffu, top);

    const float need = __fdiv_rn(__uint_as_float(top), 127.f);
    const float scale = need <= old || old != old ? old : need;  // NaN stays
    const bool grown = !(scale <= old);
    __syncwarp();
    if (lane == 0 && (grown || anew)) *scale_at = scale;

    const Quantizer quantize(scale);
    auto codes = [&](float a, float b, float c, float d) {
        return quantize.divide ? quantize.divided(a, b, c, d) : quantize(a, b, c, d);
    };
    // four old codes (bytes) under the new scale
    auto again = [&](uint32_t w) -> uint32_t {
        return codes(__fmul_rn(float(int8_t(w)), old), __fmul_rn(float(int8_t(w >> 8)), old),
                     __fmul_rn(float(int8_t(w >> 16)), old), __fmul_rn(float(int8_t(w >> 24)), old));
    };
    if (!v) {
        uint8_t* base = static_cast<uint8_t*>(p.k_cache) + tile * 16 * D;
#pragma unroll 4
        for (int j = 0; j < NR; ++j) {
            const int r = row_of(j), t = src[r];
            uint16_t* at_lo = reinterpret_cast<uint16_t*>(base + r * D + lo);
            uint16_t* at_hi = reinterpret_cast<uint16_t*>(base + r * D + hi);
            if (t < 0 && !anew && !grown) continue;
            uint32_t w = 0;
            if (t >= 0) {
                float x[4];
                load(r, t, x);
                w = codes(x[0], x[1], x[2], x[3]);
            } else if (!anew) {
                w = again(uint32_t(*at_lo) | uint32_t(*at_hi) << 16);
            }
            *at_lo = uint16_t(w);
            *at_hi = uint16_t(w >> 16);
        }
    } else {
        // column lo + e: this lane's NR of its 16 bytes
        uint8_t* base = static_cast<uint8_t*>(p.v_cache) + tile * 16 * D + 4 * l * 16 + 8 * half;
        uint32_t w[4][NR / 4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (NR == 16) {
                const uint4 o = any_old && !anew ? *reinterpret_cast<const uint4*>(base + e * 16) : make_uint4(0, 0, 0, 0);
                w[e][0] = o.x, w[e][1] = o.y, w[e][2] = o.z, w[e][3] = o.w;
            } else {
                const uint2 o = any_old && !anew ? *reinterpret_cast<const uint2*>(base + e * 16) : make_uint2(0, 0);
                w[e][0] = o.x, w[e][1] = o.y;
            }
            if (any_old && grown && !anew) {
#pragma unroll
                for (int k = 0; k < NR / 4; ++k) w[e][k] = again(w[e][k]);
            }
        }
        // a word of a column holds rows 2k, 2k+1, 2k+8, 2k+9 (of the lane's rows)
#pragma unroll
        for (int k = 0; k < NR / 4; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = row_of(2 * k + (i & 1) + (i >> 1) * (NR / 2)), t = src[r];
                if (t < 0) continue;
                float x[4];
                load(r, t, x);
                const uint32_t c = codes(x[0], x[1], x[2], x[3]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t sel = (0x3210u & ~(0xfu << (4 * i))) | uint32_t(4 + e) << (4 * i);
                    w[e][k] = __byte_perm(w[e][k], c, sel);
                }
            }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (NR == 16) *reinterpret_cast<uint4*>(base + e * 16) = make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
            else *reinterpret_cast<uint2*>(base + e * 16) = make_uint2(w[e][0], w[e][1]);
        }
    }
}

template <int D, int HP>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_append_i8_kernel(const __grid_constant__ RopeParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (int(blockIdx.x) >= p.kv_ctas) {  // the queries
        constexpr uint32_t cpr = D / 16;
        const uint32_t per_token = (p.Hq + HP - 1) / HP * cpr;
        const uint32_t i = (blockIdx.x - p.kv_ctas) * uint32_t(kRopeThreads) + threadIdx.x;
        const uint32_t t = i / per_token, r = i - t * per_token;
        if (t < uint32_t(p.T)) rope_rows<HP>(p, int(t), int(r / cpr) * HP, p.Hq, int(r % cpr));
        return;
    }
    __shared__ __align__(16) uint8_t stages[kRopeThreads / 32][16 * D * 2];
    __shared__ int src[16];    // the call's token of each row of the block, -1: none
    __shared__ int not_first;  // another token of the block comes before
    // This CTA's tokens (at most 32); those right behind a token of their own
    // block cannot be its first.  Every warp sees the same mask.
    const int lane = threadIdx.x & 31, t0 = blockIdx.x * p.tokens_per_cta;
    const bool here = lane < p.tokens_per_cta && t0 + lane < p.T;
    const int32_t my_slot = here ? __ldg(p.slot_mapping + t0 + lane) : -1;
    const int32_t before = here && t0 + lane > 0 ? __ldg(p.slot_mapping + t0 + lane - 1) : -1;
    bool candidate = my_slot >= 0;
    if (candidate && my_slot / 16 >= p.NB) {
        if (threadIdx.x < 32) raise_error(PA_DEVERR_SLOT);
        candidate = false;
    }
    if (candidate && p.rd > 0) angles(p, t0 + lane, threadIdx.x < 32);  // reports a position without a table row
    if (before >= 0 && before / 16 == my_slot / 16) candidate = false;
    for (unsigned todo = __ballot_sync(0xffffffffu, candidate); todo; todo &= todo - 1) {
        const int i = __ffs(todo) - 1, t = t0 + i;
        const int32_t block = __shfl_sync(0xffffffffu, my_slot, i) / 16;
        __syncthreads();  // the last block's src has been read
        if (threadIdx.x < 16) src[threadIdx.x] = -1;
        if (threadIdx.x == 0) not_first = 0;
        __syncthreads();
#pragma unroll 8
        for (int u = threadIdx.x; u < p.T; u += kRopeThreads) {
            const int32_t s = __ldg(p.slot_mapping + u);
            if (s < 0 || s / 16 != block) continue;
            if (u < t) not_first = 1;
            atomicMax(&src[s & 15], u);  // of two tokens in one slot the later lands
        }
        __syncthreads();
        if (not_first) continue;
        for (int x = threadIdx.x >> 5; x < 2 * p.Hkv; x += kRopeThreads / 32)
            quantize_tile<D>(p, src, block, x >> 1, x & 1, stages[threadIdx.x >> 5], lane);
    }
}

}  // namespace pa
