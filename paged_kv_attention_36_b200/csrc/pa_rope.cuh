// pa_rope.cuh -- the step's append with the position rotation on the way:
// q and k rows are turned by the angles of their tokens' positions, k and v
// land in their slots of the paged cache (bf16, or 8-bit codes with a scale
// for each (block, kv head)).
//
// A row's first rd values are rd/2 pairs; pair i is (x_i, x_{i+rd/2}), or
// (x_2i, x_2i+1) when interleaved, and becomes
//     (a cos_i - b sin_i,  b cos_i + a sin_i)
// with the angles' cosines and sines read from the caller's fp32 table
// [max_position][rd] (rd/2 cosines, then rd/2 sines), in fp32 and rounded once
// at the end.  On the way to 8-bit codes each product and sum is rounded by
// itself, so that the codes are those of the documented operations.
#pragma once

#include "pa_append.cuh"
#include "pa_device.cuh"
#include "pa_tcgen05.cuh"  // packed fp32 pairs

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
    int32_t parts;                // 8-bit: CTAs that share the tiles of the same tokens
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
    int32_t pos = __ldca(p.positions + t);
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
template <bool interleaved>
__device__ __forceinline__ void turn_chunks(uint4& lo, uint4& hi, const float (&c)[8], const float (&s)[8]) {
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
    // two pairs at once; the rounding to bf16 leaves no room for the last bit of
    // fp32, so products and sums are fused here
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const int a0 = interleaved ? 2 * i : i, a1 = interleaved ? 2 * i + 2 : i + 1;
        const int b0 = interleaved ? 2 * i + 1 : 8 + i, b1 = interleaved ? 2 * i + 3 : 9 + i;
        const uint64_t a = f2_pack(x[a0], x[a1]), b = f2_pack(x[b0], x[b1]);
        const uint64_t cc = f2_pack(c[i], c[i + 1]), ss = f2_pack(s[i], s[i + 1]), ns = f2_pack(-s[i], -s[i + 1]);
        f2_unpack(f2_fma(a, cc, f2_mul(b, ns)), x[a0], x[a1]);
        f2_unpack(f2_fma(b, cc, f2_mul(a, ss)), x[b0], x[b1]);
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
    const int32_t slot = __ldca(p.slot_mapping + t);
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
            const float4 x = __ldca(reinterpret_cast<const float4*>(a + i));
            const float4 y = __ldca(reinterpret_cast<const float4*>(a + p.rd / 2 + i));
            cs[i] = x.x, cs[i + 1] = x.y, cs[i + 2] = x.z, cs[i + 3] = x.w;
            sn[i] = y.x, sn[i + 1] = y.y, sn[i + 2] = y.z, sn[i + 3] = y.w;
        }
#pragma unroll
        for (int i = 0; i < HP; ++i)
            if (dst[i] && h0 + i < p.Hq + p.Hkv) {
                if (p.interleaved) turn_chunks<true>(lo[i], hi[i], cs, sn);
                else turn_chunks<false>(lo[i], hi[i], cs, sn);
            }
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
    static __device__ __noinline__ uint32_t divided(float scale, float a, float b, float c, float d) {
        const float x[4] = {a, b, c, d};
        uint32_t w = 0;
        for (int i = 0; i < 4; ++i) {
            int q = scale > 0.f ? __float2int_rn(__fdiv_rn(x[i], scale)) : 0;
            q = q > 127 ? 127 : q < -127 ? -127 : q;
            w |= uint32_t(q & 0xff) << (8 * i);
        }
        return w;
    }
    // values (x01, x23) as packed pairs
    __device__ __forceinline__ uint32_t operator()(uint64_t x01, uint64_t x23) const {
        const uint64_t up = f2_pack(12582912.f, 12582912.f), down = f2_pack(-12582912.f, -12582912.f);
        const uint64_t by = f2_pack(inv, inv), minus = f2_pack(-1.f, -1.f);
        const uint64_t t01 = f2_mul(x01, by), t23 = f2_mul(x23, by);
        const uint64_t r01 = f2_add(t01, up), r23 = f2_add(t23, up);  // the integers in the low bits
        const uint64_t o01 = f2_fma(f2_add(r01, down), minus, t01), o23 = f2_fma(f2_add(r23, down), minus, t23);
        float r[4], off[4];
        f2_unpack(r01, r[0], r[1]);
        f2_unpack(r23, r[2], r[3]);
        f2_unpack(o01, off[0], off[1]);
        f2_unpack(o23, off[2], off[3]);
        const float worst = fmaxf(fmax3(fabsf(off[0]), fabsf(off[1]), fabsf(off[2])), fabsf(off[3]));
        if (worst > 0.5f - 0x1p-15f) {
            float x[4];
            f2_unpack(x01, x[0], x[1]);
            f2_unpack(x23, x[2], x[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (fabsf(off[i]) <= 0.5f - 0x1p-15f) continue;
                const float way = off[i] < 0.f ? -1.f : 1.f, mid = r[i] - 12582912.f + 0.5f * way;
                const float rest = fmaf(-mid, scale, x[i]);
                // half an ulp of mid: 2^(exponent - 24)
                const float half = __uint_as_float((__float_as_uint(mid) & 0x7f800000u) - (24u << 23));
                const bool tie = fabsf(rest) <= scale * half, odd = (__float_as_uint(r[i]) & 1u) != 0;
                if (tie ? odd : rest * way > 0.f) r[i] += way;
            }
        }
        const uint32_t lo = __byte_perm(__float_as_uint(r[0]), __float_as_uint(r[1]), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(r[2]), __float_as_uint(r[3]), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    }
};

// Starts the copy of all of the call's rows of a tile (kv head g, K or V) into
// `stage` ([16][D] bf16); rows the call does not have are left alone.
template <int D>
__device__ __forceinline__ void stage_rows(const RopeParams& p, const int* src, int g, bool v, uint8_t* stage, int lane) {
    const __nv_bfloat16* rows = (v ? p.v_new : p.k_new) + int64_t(g) * D;
    const int64_t stride = v ? p.v_stride : p.k_stride;
#pragma unroll
    for (int x = lane; x < 16 * (D / 8); x += 32) {
        const int t = src[x / (D / 8)];
        if (t >= 0) cp_async16(stage + x * 16, rows + t * stride + x % (D / 8) * 8);
    }
}

// `stage`: the tile's rows (stage_rows), `table`: the angles of the block's
// rows, [16][rd] as in cos_sin.
template <int D>
__device__ __forceinline__ void quantize_tile(const RopeParams& p, const int* src, int64_t block, int g, bool v,
                                              const uint8_t* stage, const float* table, int lane) {
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
    const int64_t tile = block * p.Hkv + g;
    float* scale_at = (v ? p.v_scale : p.k_scale) + tile;
    const bool anew = src[0] >= 0;
    const float old = anew ? 0.f : *scale_at;
    // the lane's four values of row r, turned, as (lo, lo+1) and (hi, hi+1)
    auto load = [&](int r, uint64_t& x01, uint64_t& x23) {
        const uint8_t* row = stage + r * D * 2;
        float2 a = bf16x2_to_float2(*reinterpret_cast<const uint32_t*>(row + lo * 2));
        float2 b = bf16x2_to_float2(*reinterpret_cast<const uint32_t*>(row + hi * 2));
        if (rotate) {
            const float2 c = *reinterpret_cast<const float2*>(table + r * rd + 2 * l);
            const float2 s = *reinterpret_cast<const float2*>(table + r * rd + rd / 2 + 2 * l);
            if (p.interleaved) {
                turn(a.x, a.y, c.x, s.x);
                turn(b.x, b.y, c.y, s.y);
            } else {
                turn(a.x, b.x, c.x, s.x);
                turn(a.y, b.y, c.y, s.y);
            }
        }
        x01 = f2_pack(a.x, a.y);
        x23 = f2_pack(b.x, b.y);
    };

    // the lane's rows that the call has, as bits
    const uint32_t have = [&] {
        const uint32_t all = __ballot_sync(0xffffffffu, l < NR && src[row_of(l < NR ? l : 0)] >= 0);
        return NR == 16 ? all & 0xffffu : all >> (16 * half) & 0xffu;
    }();
    uint32_t top = 0;
    if (v) {  // bf16 magnitudes as 16-bit integers, two at a time
        uint32_t pair = 0;
#pragma unroll 2
        for (uint32_t left = have; left; left &= left - 1) {
            const uint2 w = *reinterpret_cast<const uint2*>(stage + row_of(__ffs(left) - 1) * D * 2 + lo * 2);
            pair = __vmaxu2(__vmaxu2(pair, w.x & 0x7fff7fffu), w.y & 0x7fff7fffu);
        }
        top = max(pair << 16, pair & 0xffff0000u);
    } else {
#pragma unroll 1
        for (uint32_t left = have; left; left &= left - 1) {
            uint64_t x01, x23;
            load(row_of(__ffs(left) - 1), x01, x23);
            float x[4];
            f2_unpack(x01, x[0], x[1]);
            f2_unpack(x23, x[2], x[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, abs_bits(x[e]));
        }
    }
    __syncwarp();
    top = __reduce_max_sync(0xffffffffu, top);

    const float need = __fdiv_rn(__uint_as_float(top), 127.f);
    const float scale = need <= old || old != old ? old : need;  // NaN stays
    const bool grown = !(scale <= old);
    __syncwarp();
    if (lane == 0 && (grown || anew)) *scale_at = scale;

    // The codes of the lane's four columns of row r.  The loops below are
    // rolled around one copy of this.
    const Quantizer quantize(scale);
    auto codes = [&](uint64_t x01, uint64_t x23) -> uint32_t {
        if (!quantize.divide) return quantize(x01, x23);
        float x[4];
        f2_unpack(x01, x[0], x[1]);
        f2_unpack(x23, x[2], x[3]);
        return Quantizer::divided(scale, x[0], x[1], x[2], x[3]);
    };
    auto row_codes = [&](int r) -> uint32_t {
        uint64_t x01, x23;
        load(r, x01, x23);
        return codes(x01, x23);
    };
    // four old codes under the new scale
    auto again = [&](uint32_t kept) -> uint32_t {
        return codes(f2_pack(__fmul_rn(float(int8_t(kept)), old), __fmul_rn(float(int8_t(kept >> 8)), old)),
                     f2_pack(__fmul_rn(float(int8_t(kept >> 16)), old), __fmul_rn(float(int8_t(kept >> 24)), old)));
    };
    uint8_t* base = static_cast<uint8_t*>(v ? p.v_cache : p.k_cache) + tile * 16 * D;
    if (!anew && !grown) {
        // only the new rows change
#pragma unroll 1
        for (uint32_t left = have; left; left &= left - 1) {
            const int r = row_of(__ffs(left) - 1);
            const uint32_t w = row_codes(r);
            if (!v) {
                *reinterpret_cast<uint16_t*>(base + r * D + lo) = uint16_t(w);
                *reinterpret_cast<uint16_t*>(base + r * D + hi) = uint16_t(w >> 16);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) base[(4 * l + e) * 16 + vt_position(r)] = uint8_t(w >> (8 * e));
            }
        }
        return;
    }
    if (!v) {
#pragma unroll 1
        for (int j = 0; j < NR; ++j) {
            const int r = row_of(j);
            uint16_t* at_lo = reinterpret_cast<uint16_t*>(base + r * D + lo);
            uint16_t* at_hi = reinterpret_cast<uint16_t*>(base + r * D + hi);
            const uint32_t w = have >> j & 1 ? row_codes(r)
                               : anew        ? 0u
                                             : again(uint32_t(*at_lo) | uint32_t(*at_hi) << 16);
            *at_lo = uint16_t(w);
            *at_hi = uint16_t(w >> 16);
        }
    } else {
        // column lo + e: this lane's NR of its 16 bytes.  Word k of a column
        // holds the lane's rows 2k, 2k+1, 2k + NR/2, 2k+1 + NR/2; the words
        // move through the registers so that the loop's body names only w[.][0].
        constexpr int NW = NR / 4;
        uint8_t* at = base + 4 * l * 16 + 8 * half;
        uint32_t w[4][NW];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (NR == 16) {
                const uint4 o = anew ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(at + e * 16);
                w[e][0] = o.x, w[e][1] = o.y, w[e][2] = o.z, w[e][3] = o.w;
            } else {
                const uint2 o = anew ? make_uint2(0, 0) : *reinterpret_cast<const uint2*>(at + e * 16);
                w[e][0] = o.x, w[e][1] = o.y;
            }
        }
#pragma unroll 1
        for (int k = 0; k < NW; ++k) {
            uint32_t c[4] = {0u, 0u, 0u, 0u};  // the codes of four rows, a row each
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const int j = 2 * k + (i & 1) + (i >> 1) * (NR / 2);
                const uint32_t pick = 0x40u + 0x11u * uint32_t(i);  // byte i of each word
                c[0] = c[1], c[1] = c[2], c[2] = c[3];
                c[3] = have >> j & 1 ? row_codes(row_of(j))
                       : anew        ? 0u
                                     : again(__byte_perm(__byte_perm(w[0][0], w[1][0], pick),
                                                         __byte_perm(w[2][0], w[3][0], pick), 0x5410));
            }
            // rows to columns: four 4-byte rows become four 4-byte columns
            const uint32_t a = __byte_perm(c[0], c[1], 0x5140), b = __byte_perm(c[2], c[3], 0x5140);
            const uint32_t d = __byte_perm(c[0], c[1], 0x7362), f = __byte_perm(c[2], c[3], 0x7362);
            const uint32_t n[4] = {__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632), __byte_perm(d, f, 0x5410),
                                   __byte_perm(d, f, 0x7632)};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int i = 0; i + 1 < NW; ++i) w[e][i] = w[e][i + 1];
                w[e][NW - 1] = n[e];
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (NR == 16) *reinterpret_cast<uint4*>(at + e * 16) = make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
            else *reinterpret_cast<uint2*>(at + e * 16) = make_uint2(w[e][0], w[e][1]);
        }
    }
}

template <int D, int HP>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_append_i8_kernel(const __grid_constant__ RopeParams p) {
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
    extern __shared__ __align__(16) uint8_t rope_smem[];
    constexpr int kStage = 16 * D * 2, kWarps = kRopeThreads / 32;
    float* table = reinterpret_cast<float*>(rope_smem);           // [16][rd]
    uint8_t* stages = rope_smem + 16 * D * 4;                      // a tile a warp
    __shared__ int src[16];    // the call's token of each row of the block, -1: none
    __shared__ int not_first;  // another token of the block comes before
    // This CTA's tokens (at most 32); those right behind a token of their own
    // block cannot be its first.  Every warp sees the same mask.
    const int lane = threadIdx.x & 31, t0 = int(blockIdx.x) / p.parts * p.tokens_per_cta;
    const bool here = lane < p.tokens_per_cta && t0 + lane < p.T;
    const int32_t my_slot = here ? __ldca(p.slot_mapping + t0 + lane) : -1;
    const int32_t before = here && t0 + lane > 0 ? __ldca(p.slot_mapping + t0 + lane - 1) : -1;
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
        auto look = [&](int u, int32_t s) {
            if (uint32_t(s) >> 4 != uint32_t(block)) return;  // padding is negative: in no block
            if (u < t) not_first = 1;
            atomicMax(&src[s & 15], u);  // of two tokens in one slot the later lands
        };
        const bool vec = (reinterpret_cast<uintptr_t>(p.slot_mapping) & 15) == 0;
        const int whole = vec ? p.T / 4 : 0;
#pragma unroll 8
        for (int u = threadIdx.x; u < whole; u += kRopeThreads) {
            const int4 s = __ldca(reinterpret_cast<const int4*>(p.slot_mapping) + u);
            if (uint32_t(s.x) >> 4 != uint32_t(block) && uint32_t(s.y) >> 4 != uint32_t(block) &&
                uint32_t(s.z) >> 4 != uint32_t(block) && uint32_t(s.w) >> 4 != uint32_t(block))
                continue;
            look(4 * u, s.x);
            look(4 * u + 1, s.y);
            look(4 * u + 2, s.z);
            look(4 * u + 3, s.w);
        }
        for (int u = 4 * whole + threadIdx.x; u < p.T; u += kRopeThreads) look(u, __ldca(p.slot_mapping + u));
        __syncthreads();
        if (not_first) continue;
        // the angles of the block's rows, for every head; they land with the first tile
        const int per_row = p.rd / 4;
        for (int x = threadIdx.x; x < 16 * per_row; x += kRopeThreads) {
            const int u = src[x / per_row];
            if (u >= 0) cp_async16(table + x * 4, angles(p, u, false) + x % per_row * 4);
        }
        uint8_t* mine = stages + (threadIdx.x >> 5) * kStage;
        const int step = p.parts * kWarps, tiles = 2 * p.Hkv;
        for (int x = int(blockIdx.x) % p.parts * kWarps + (threadIdx.x >> 5), n = 0; n < tiles; x += step, n += step) {
            __syncwarp();  // the tile before has been read
            if (x < tiles) stage_rows<D>(p, src, x >> 1, x & 1, mine, lane);
            cp_async_commit();
            cp_async_wait_all();
            if (n == 0) __syncthreads();  // the table
            else __syncwarp();
            if (x < tiles) quantize_tile<D>(p, src, block, x >> 1, x & 1, mine, table, lane);
        }
    }
}

}  // namespace pa
