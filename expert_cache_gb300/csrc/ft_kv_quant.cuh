// Quantising a block of 16 dims of a token's key or value into its tile: the device side that every kernel
// which stores keys and values shares.
//
// Quotients are the definition's x / (scale * s), rounded to nearest, in three operations: with
// r = RN(1/d) and q0 = RN(x r), q0 + RN(x - q0 d) r rounds to RN(x/d) (Markstein's correction, 1990;
// compared with the division for every bf16 significand over every fp32 one: no difference), as long
// as nothing over- or underflows; a block where something could, with a NaN, an infinity or
// a saturated scale, takes the division itself.  The conversion instructions round to nearest even
// and saturate like the definition; only a zero's sign is dropped afterwards.
#pragma once
#include "ft_kv.cuh"
#include "ft_quant.cuh"

namespace ft {

namespace {

// Signed E4M3 of v, round to nearest even, saturating; NaN becomes 0.
__device__ __forceinline__ uint32_t e4m3_encode_signed(float v) {
    const uint32_t c = e4m3_encode_rne(fabsf(v));
    return c | ((v < 0.f && c) ? 0x80u : 0u);
}

template <int N>
__device__ __forceinline__ void store_run(uint8_t* dst, const uint32_t* w) {
    if constexpr (N == 4) *reinterpret_cast<uint32_t*>(dst) = w[0];
    if constexpr (N == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    if constexpr (N == 16) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The codes of a block of 16 dims lie in one run, except V's at D = 64, whose lanes hold 8
// dims each: two runs.
template <int D, int kFormat, bool kV>
__device__ __forceinline__ void store_codes(uint8_t* tile, int r, int d, const uint32_t* w) {
    constexpr int kBytes = kFormat == FT_KV_NVFP4 ? 8 : 16;
    if constexpr (kV && D == 64) {
        store_run<kBytes / 2>(tile + kv_v_byte<D, kFormat>(r, d), w);
        store_run<kBytes / 2>(tile + kv_v_byte<D, kFormat>(r, d + 8), w + kBytes / 8);
    } else {
        store_run<kBytes>(tile + (kV ? kv_v_byte<D, kFormat>(r, d) : kv_k_byte<D, kFormat>(r, d)), w);
    }
}

__device__ __forceinline__ uint8_t* kv_tile_ptr(const KvView& kv, int slot, int head, int tile_bytes) {
    const int page = slot >> kv.page_shift, in = slot & ((1 << kv.page_shift) - 1);
    const int per = 1 << (kv.page_shift - 4);
    return kv.pool + (((size_t)page * kv.hkv + head) * per + (in >> 4)) * tile_bytes;
}

// max |x| of a block of 16 bf16 (8 words); NaN if there is one.
__device__ __forceinline__ float block_amax(const uint32_t (&xw)[8]) {
    __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&xw[0]));
#pragma unroll
    for (int j = 1; j < 8; ++j) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&xw[j])));
    const __nv_bfloat16 h = __hmax_nan(__low2bfloat16(m), __high2bfloat16(m));
    return __bfloat162float(h);
}
__device__ __forceinline__ float bf16_at(const uint32_t (&xw)[8], int j) {
    return __uint_as_float(j & 1 ? xw[j >> 1] & 0xFFFF0000u : xw[j >> 1] << 16);
}

// RN(x / d) with r = RN(1/d), in the range where the remainder is exact.
__device__ __forceinline__ float quotient(float x, float d, float r) {
    const float q = __fmul_rn(x, r);
    return __fmaf_rn(__fmaf_rn(-q, d, x), r, q);
}
// Magnitudes for which quotients of the block are in that range.
__device__ __forceinline__ bool tame(float amax, float d) {
    return amax < 1e30f && d > 1e-25f && d < 1e25f && amax < 1e4f * d;
}

// The codes of a block by the division itself (out of line: rare, and ten copies of it would not fit
// the instruction cache).
template <int kFormat>
__device__ __noinline__ uint4 codes_by_division(uint4 x0, uint4 x1, float d) {
    const uint32_t xw[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float q = __fdiv_rn(bf16_at(xw, j), d);
        if constexpr (kFormat == FT_KV_FP8) w[j >> 2] |= e4m3_encode_signed(q) << (8 * (j & 3));
        else w[j >> 3] |= (uint32_t)e2m1_encode_rne(q) << (4 * (j & 7));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 codes of a block (xw: 8 words of bf16) with divisor d, and for NVFP4 its scale byte.
// FP8: 16 bytes; NVFP4: 8 bytes.
template <int kFormat>
__device__ __forceinline__ uint32_t quantise(const uint32_t (&xw)[8], float st, float inv_st, uint32_t* w) {
    const float amax = block_amax(xw);
    if constexpr (kFormat == FT_KV_FP8) {
        if (tame(amax, st)) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float q[4] = {quotient(bf16_at(xw, 4 * j), st, inv_st), quotient(bf16_at(xw, 4 * j + 1), st, inv_st),
                                    quotient(bf16_at(xw, 4 * j + 2), st, inv_st), quotient(bf16_at(xw, 4 * j + 3), st, inv_st)};
                uint32_t c;
                asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
                    "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
                    : "=r"(c) : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]));
                const uint32_t mag = c & 0x7F7F7F7Fu;                 // a sign only where the magnitude is not zero
                w[j] = mag | (c & (mag + 0x7F7F7F7Fu) & 0x80808080u);
            }
        } else {
            const uint4 c = codes_by_division<kFormat>(make_uint4(xw[0], xw[1], xw[2], xw[3]), make_uint4(xw[4], xw[5], xw[6], xw[7]), st);
            w[0] = c.x; w[1] = c.y; w[2] = c.z; w[3] = c.w;
        }
        return 0;
    } else {
        const bool number = amax == amax;
        float m = amax;
        if (!number) {                                                // the largest of the others
            m = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(bf16_at(xw, j)));
        }
        const float sixth = m > 1e-30f && m < 1e30f ? quotient(m, 6.0f, 1.0f / 6.0f) : __fdiv_rn(m, 6.0f);
        uint32_t sc, sc2;
        asm("{\n\t.reg .b16 x;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %3;\n\tcvt.rn.f16x2.e4m3x2 %1, x;\n\t"
            "cvt.u32.u16 %0, x;\n\t}" : "=r"(sc), "=r"(sc2) : "f"(0.f), "f"(__fdiv_rn(sixth, st)));
        const float d = __fmul_rn(__low2float(*reinterpret_cast<const __half2*>(&sc2)), st);
        w[0] = w[1] = 0;
        if (d == 0.f) return 0;
        if (number && sc < 0x7E && tame(amax, d)) {
            const float r = __frcp_rn(d);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float q[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) q[e] = quotient(bf16_at(xw, 8 * j + e), d, r);
                uint32_t c;
                asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tcvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
                    "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
                    "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\tmov.b32 %0, {b0, b1, b2, b3};\n\t}"
                    : "=r"(c) : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
                const uint32_t mag = c & 0x77777777u;
                w[j] = mag | (c & (mag + 0x77777777u) & 0x88888888u);
            }
        } else {
            const uint4 c = codes_by_division<kFormat>(make_uint4(xw[0], xw[1], xw[2], xw[3]), make_uint4(xw[4], xw[5], xw[6], xw[7]), d);
            w[0] = c.x; w[1] = c.y;
        }
        return sc;
    }
}

__device__ __forceinline__ void load_block(uint32_t (&xw)[8], const __nv_bfloat16* src) {
    const uint4 x0 = *reinterpret_cast<const uint4*>(src), x1 = *reinterpret_cast<const uint4*>(src + 8);
    xw[0] = x0.x; xw[1] = x0.y; xw[2] = x0.z; xw[3] = x0.w;
    xw[4] = x1.x; xw[5] = x1.y; xw[6] = x1.z; xw[7] = x1.w;
}

// Quantise block b (16 dims) of one token's K or V row into its tile.
template <int D, int kFormat, bool kV>
__device__ __forceinline__ void append_block(uint8_t* tile, int r, int b, const uint32_t (&xw)[8], float st, float inv_st) {
    uint32_t w[4];
    const uint32_t sc = quantise<kFormat>(xw, st, inv_st, w);
    if constexpr (kFormat == FT_KV_NVFP4) tile[kV ? kv_v_scale_byte<D>(r, b) : kv_k_scale_byte<D>(r, b)] = (uint8_t)sc;
    store_codes<D, kFormat, kV>(tile, r, 16 * b, w);
}

}  // namespace

}  // namespace ft
