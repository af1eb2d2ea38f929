// The quantised key/value cache: host side of the C ABI, the writing kernels (bf16 -> codes
// and scales in their tiles) and the reading ones (codes -> bf16).
//
// Both directions are bound by the bytes of the bf16 side (4 of 5.1 bytes per element of NVFP4).
// A call of few tokens takes one thread per 16 dims of a row: latency is all there is.  A call of
// many takes a warp per 16 tokens and head: where the tokens are a whole tile in order, a lane has
// exactly the tokens and dims whose codes it stores as 16-byte vectors, so that both the rows and
// the tile move in full sectors (one 8-byte store per block cost 20 us for 8192 tokens of 8 heads
// of 128 where the bytes take 6.3); the other tokens go row by row.
//
// Quotients are the definition's x / (scale * s), rounded to nearest, in three operations: with
// r = RN(1/d) and q0 = RN(x r), q0 + RN(x - q0 d) r rounds to RN(x/d) (Markstein's correction, 1990;
// compared with the division for every bf16 significand over every fp32 one: no difference), as long
// as nothing over- or underflows; a block where something could, with a NaN, an infinity or
// a saturated scale, takes the division itself.  The conversion instructions round to nearest even
// and saturate like the definition; only a zero's sign is dropped afterwards.
#include <atomic>
#include <cmath>
#include <cstdio>
#include <new>

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

template <int N>
__device__ __forceinline__ void load_run(uint32_t* w, const uint8_t* src) {
    if constexpr (N == 4) w[0] = *reinterpret_cast<const uint32_t*>(src);
    if constexpr (N == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(src);
        w[0] = v.x; w[1] = v.y;
    }
    if constexpr (N == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(src);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    }
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

template <int D, int kFormat, bool kV>
__device__ __forceinline__ void load_codes(uint32_t* w, const uint8_t* tile, int r, int d) {
    constexpr int kBytes = kFormat == FT_KV_NVFP4 ? 8 : 16;
    if constexpr (kV && D == 64) {
        load_run<kBytes / 2>(w, tile + kv_v_byte<D, kFormat>(r, d));
        load_run<kBytes / 2>(w + kBytes / 8, tile + kv_v_byte<D, kFormat>(r, d + 8));
    } else {
        load_run<kBytes>(w, tile + (kV ? kv_v_byte<D, kFormat>(r, d) : kv_k_byte<D, kFormat>(r, d)));
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
__device__ __forceinline__ void append_block(uint8_t* tile, int r, int b, const __nv_bfloat16* src, float st, float inv_st) {
    uint32_t xw[8], w[4];
    load_block(xw, src);
    const uint32_t sc = quantise<kFormat>(xw, st, inv_st, w);
    if constexpr (kFormat == FT_KV_NVFP4) tile[kV ? kv_v_scale_byte<D>(r, b) : kv_k_scale_byte<D>(r, b)] = (uint8_t)sc;
    store_codes<D, kFormat, kV>(tile, r, 16 * b, w);
}

// bf16 pairs of 8 (NVFP4: one word) or 4 (FP8: one word) codes; sc: the block's scale as two f16.
__device__ __forceinline__ uint32_t to_bf16(uint32_t f16x2, float st) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&f16x2));
    const __nv_bfloat162 p = __floats2bfloat162_rn(__fmul_rn(f.x, st), __fmul_rn(f.y, st));
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void dequant_e2m1(uint32_t w, uint32_t sc2, float st, uint32_t* out) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b32 x0, x1, x2, x3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 x0, b0;\n\tcvt.rn.f16x2.e2m1x2 x1, b1;\n\tcvt.rn.f16x2.e2m1x2 x2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 x3, b3;\n\tmul.rn.f16x2 %0, x0, %5;\n\tmul.rn.f16x2 %1, x1, %5;\n\t"
        "mul.rn.f16x2 %2, x2, %5;\n\tmul.rn.f16x2 %3, x3, %5;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w), "r"(sc2));
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = to_bf16(h[j], st);          // code * scale is exact in f16
}
__device__ __forceinline__ void dequant_e4m3(uint32_t w, float st, uint32_t* out) {
    uint32_t h[2];
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(h[0]), "=r"(h[1]) : "r"(w));
    out[0] = to_bf16(h[0], st);
    out[1] = to_bf16(h[1], st);
}
__device__ __forceinline__ uint32_t scale_pair(uint32_t byte) {
    uint32_t o;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(o) : "r"(byte * 0x101u));
    return o;
}

template <int D, int kFormat, bool kV>
__device__ __forceinline__ void read_block(const uint8_t* tile, int r, int b, __nv_bfloat16* dst, float st) {
    uint32_t w[4], out[8];
    load_codes<D, kFormat, kV>(w, tile, r, 16 * b);
    if constexpr (kFormat == FT_KV_NVFP4) {
        const uint32_t sc2 = scale_pair(tile[kV ? kv_v_scale_byte<D>(r, b) : kv_k_scale_byte<D>(r, b)]);
#pragma unroll
        for (int j = 0; j < 2; ++j) dequant_e2m1(w[j], sc2, st, out + 4 * j);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) dequant_e4m3(w[j], st, out + 2 * j);
    }
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(out[0], out[1], out[2], out[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

// ---------------------------------------------------------------------------- whole tiles

// A warp's window of 16 tokens of a call and what they are.
struct Window {
    int head;            // token (from the window's first) that starts a whole tile, or -1: it runs past the window
    unsigned rest;       // tokens of the window that belong to no whole tile: bits
    int slot;            // of token `lane` (0..31 from the window's first), -1 past the end
};
// Tokens first.. of the call; the lanes hold the slots of 32 tokens from the window's first on and of the 16
// before it.
__device__ __forceinline__ Window window_of(const KvView& kv, const int32_t* slots, int n, int first, int lane) {
    const int most = kv.n_pages << kv.page_shift;
    auto slot_of = [&](int i) {
        const int s = i >= 0 && i < n ? slots[i] : -1;
        return s >= 0 && s < most ? s : -1;
    };
    Window w;
    w.slot = slot_of(first + lane);
    const int before = slot_of(first - 16 + lane);           // lanes 0..15: the 16 tokens before the window
    // bit i: tokens i and i + 1 of the 32 (of the 16 before and the 16 of the window) stand in order
    const int next = __shfl_down_sync(0xffffffffu, w.slot, 1), next_before = __shfl_down_sync(0xffffffffu, before, 1);
    const unsigned run = __ballot_sync(0xffffffffu, w.slot >= 0 && next == w.slot + 1);
    const unsigned run_before = __ballot_sync(0xffffffffu, before >= 0 && next_before == before + 1);
    const unsigned lead = __ballot_sync(0xffffffffu, w.slot >= 0 && (w.slot & 15) == 0);
    const unsigned lead_before = __ballot_sync(0xffffffffu, before >= 0 && (before & 15) == 0);
    auto head = [](unsigned runs, unsigned leads) {          // the token i < 16 that starts 16 in order at a tile's start
        int h = -1;
        for (unsigned x = leads & 0xFFFFu; x; x &= x - 1) {
            const int i = __ffs(x) - 1;
            if ((runs >> i & 0x7FFFu) == 0x7FFFu) h = i;
        }
        return h;
    };
    w.head = head(run, lead);
    const int prev = head(run_before, lead_before);          // a tile that began before reaches tokens 0 .. prev - 1
    w.rest = 0xFFFFu;
    if (prev >= 0) w.rest &= ~((1u << prev) - 1);
    if (w.head >= 0) w.rest &= (1u << w.head) - 1;
    const int left = n - first;
    if (left < 16) w.rest &= (1u << left) - 1;
    return w;
}

// The next 512 / D tokens of a set, one per group of D / 16 lanes (-1: none), taken out of it.
template <int D>
__device__ __forceinline__ int pick(unsigned& x, int lane) {
    int tok = -1;
#pragma unroll
    for (int y = 0; y < 512 / D; ++y) {
        if (lane / (D / 16) == y && x) tok = __ffs(x) - 1;
        x &= x - 1;
    }
    return tok;
}

// A whole tile of one head: the lane (g, t) quantises the blocks whose codes it stores.
template <int D, int kFormat, bool kV>
__device__ __forceinline__ void append_tile(uint8_t* tile, const __nv_bfloat16* src, size_t stride, float st, float inv_st, int lane) {
    const int g = lane >> 2, t = lane & 3;
    constexpr bool kFour = kFormat == FT_KV_NVFP4;
    // the lane's blocks: K [token v][b < D/64]; V [token q][b < D/128], at D = 64 (a block of two lanes) two
    // of the four tokens each.  Four at a time, every load of them first.
    constexpr int kBlocks = !kV ? 2 * (D / 64) : D == 64 ? 2 : 4 * (D / 128), kAt = kBlocks < 4 ? kBlocks : 4;
#pragma unroll
    for (int x0 = 0; x0 < kBlocks; x0 += kAt) {
        uint32_t xw[kAt][8];
        auto place = [&](int x, int& r, int& blk) {
            if (!kV) {
                r = 8 * (x / (D / 64)) + g;
                blk = t * (D / 64) + x % (D / 64);
            } else {
                const int q = D == 64 ? 2 * x + (g & 1) : x / (D / 128 > 0 ? D / 128 : 1);
                r = 2 * t + (q & 1) + 8 * (q >> 1);
                blk = D == 64 ? g >> 1 : g * (D / 128) + x % (D / 128 > 0 ? D / 128 : 1);
            }
        };
#pragma unroll
        for (int x = 0; x < kAt; ++x) {
            int r, blk;
            place(x0 + x, r, blk);
            load_block(xw[x], src + (size_t)r * stride + 16 * blk);
        }
#pragma unroll
        for (int x = 0; x < kAt; ++x) {
            int r, blk;
            place(x0 + x, r, blk);
            uint32_t w[4];
            const uint32_t sc = quantise<kFormat>(xw[x], st, inv_st, w);
            store_codes<D, kFormat, kV>(tile, r, 16 * blk, w);
            if constexpr (kFour) tile[kV ? kv_v_scale_byte<D>(r, blk) : kv_k_scale_byte<D>(r, blk)] = (uint8_t)sc;
        }
    }
}

}  // namespace

// A warp per 16 tokens of the call and head, K then V.
template <int D, int kFormat>
__global__ void __launch_bounds__(256, 4) kv_append_tiles_kernel(const KvView kv, const __nv_bfloat16* k, const __nv_bfloat16* v,
                                                              size_t k_stride, size_t v_stride, const int32_t* slots, int n) {
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31;
    const float inv_k = __frcp_rn(kv.k_scale), inv_v = __frcp_rn(kv.v_scale);
    const long long items = (long long)((n + 15) / 16) * kv.hkv * 2;
    for (long long it = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += (long long)gridDim.x * 8) {
        const int first = (int)(it / (2 * kv.hkv)) * 16, rest = (int)(it % (2 * kv.hkv));
        const bool is_v = rest >= kv.hkv;
        const int head = is_v ? rest - kv.hkv : rest;
        const Window w = window_of(kv, slots, n, first, lane);
        const __nv_bfloat16* src = (is_v ? v : k) + (size_t)head * D;
        const size_t stride = is_v ? v_stride : k_stride;
        if (w.head >= 0) {
            const int slot = __shfl_sync(0xffffffffu, w.slot, w.head);
            uint8_t* tile = kv_tile_ptr(kv, slot, head, kv_tile(D, kFormat).bytes);
            const __nv_bfloat16* from = src + (size_t)(first + w.head) * stride;
            if (is_v) append_tile<D, kFormat, true>(tile, from, stride, kv.v_scale, inv_v, lane);
            else append_tile<D, kFormat, false>(tile, from, stride, kv.k_scale, inv_k, lane);
        }
        for (unsigned x = w.rest; x;) {                      // kAt tokens at a time, kBatch times under way
            constexpr int kAt = 512 / D, kBatch = 2;
            int tok[kBatch], slot[kBatch];
            uint32_t xw[kBatch][8];
            const int b = lane % (D / 16);
#pragma unroll
            for (int z = 0; z < kBatch; ++z) {
                tok[z] = pick<D>(x, lane);
                slot[z] = __shfl_sync(0xffffffffu, w.slot, max(tok[z], 0));
                if (tok[z] >= 0 && slot[z] >= 0) load_block(xw[z], src + (size_t)(first + tok[z]) * stride + 16 * b);
            }
#pragma unroll
            for (int z = 0; z < kBatch; ++z) {
                if (tok[z] < 0) continue;
                if (slot[z] < 0) {
                    if (rest == 0 && b == 0 && slots[first + tok[z]] != -1) atomicOr(kv.status, FT_DEV_BAD_ID);
                    continue;
                }
                uint8_t* tile = kv_tile_ptr(kv, slot[z], head, kv_tile(D, kFormat).bytes);
                const int r = slot[z] & 15;
                uint32_t c[4];
                const uint32_t sc = quantise<kFormat>(xw[z], is_v ? kv.v_scale : kv.k_scale, is_v ? inv_v : inv_k, c);
                if constexpr (kFormat == FT_KV_NVFP4) tile[is_v ? kv_v_scale_byte<D>(r, b) : kv_k_scale_byte<D>(r, b)] = (uint8_t)sc;
                if (is_v) store_codes<D, kFormat, true>(tile, r, 16 * b, c);
                else store_codes<D, kFormat, false>(tile, r, 16 * b, c);
            }
        }
    }
}

namespace {

// A whole tile of one head back: the lane's 16-byte vectors to rows.
template <int D, int kFormat, bool kV>
__device__ __forceinline__ void read_tile(const uint8_t* tile, __nv_bfloat16* dst, size_t stride, float st, int lane) {
    const int g = lane >> 2, t = lane & 3;
    constexpr bool kFour = kFormat == FT_KV_NVFP4;
    constexpr int kVecs = kFour ? D / 64 : D / 32, kDims = kFour ? 32 : 16;      // vectors of a lane, codes of one
    constexpr int kRow = kV ? D / 8 : D / 4;                                     // dims of a token that the lane has
    uint4 c[kVecs];
    uint32_t sc[kVecs][kFour ? 4 : 1];
    auto place = [&](int x, int y, int& r, int& d) {                             // of code y of vector x
        const int at = x * kDims + y, q = at / kRow;
        d = (kV ? g : t) * kRow + at % kRow;
        r = kV ? 2 * t + (q & 1) + 8 * (q >> 1) : 8 * q + g;
    };
#pragma unroll
    for (int x = 0; x < kVecs; ++x) {                                            // every load first
        c[x] = *reinterpret_cast<const uint4*>(tile + (kV ? kv_tile(D, kFormat).code_bytes : 0) + x * 512 + lane * 16);
        if constexpr (kFour) {
#pragma unroll
            for (int y = 0; y < 32; y += 8) {
                int r, d;
                place(x, y, r, d);
                sc[x][y / 8] = tile[kV ? kv_v_scale_byte<D>(r, d / 16) : kv_k_scale_byte<D>(r, d / 16)];
            }
        }
    }
#pragma unroll
    for (int x = 0; x < kVecs; ++x) {
        const uint32_t w[4] = {c[x].x, c[x].y, c[x].z, c[x].w};
#pragma unroll
        for (int y = 0; y < kDims; y += 8) {                                     // 8 codes: 16 bytes of a row
            int r, d;
            place(x, y, r, d);
            uint32_t out[4];
            if constexpr (kFour) {
                dequant_e2m1(w[y / 8], scale_pair(sc[x][y / 8]), st, out);
            } else {
                dequant_e4m3(w[y / 4], st, out);
                dequant_e4m3(w[y / 4 + 1], st, out + 2);
            }
            *reinterpret_cast<uint4*>(dst + (size_t)r * stride + d) = make_uint4(out[0], out[1], out[2], out[3]);
        }
    }
}

}  // namespace

template <int D, int kFormat>
__global__ void __launch_bounds__(256, 4) kv_read_tiles_kernel(const KvView kv, const int32_t* slots, int n, __nv_bfloat16* k,
                                                            __nv_bfloat16* v) {
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31;
    const size_t stride = (size_t)kv.hkv * D;
    const long long items = (long long)((n + 15) / 16) * kv.hkv * 2;
    for (long long it = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += (long long)gridDim.x * 8) {
        const int first = (int)(it / (2 * kv.hkv)) * 16, rest = (int)(it % (2 * kv.hkv));
        const bool is_v = rest >= kv.hkv;
        const int head = is_v ? rest - kv.hkv : rest;
        const Window w = window_of(kv, slots, n, first, lane);
        __nv_bfloat16* dst = (is_v ? v : k) + (size_t)head * D;
        if (w.head >= 0) {
            const int slot = __shfl_sync(0xffffffffu, w.slot, w.head);
            const uint8_t* tile = kv_tile_ptr(kv, slot, head, kv_tile(D, kFormat).bytes);
            __nv_bfloat16* to = dst + (size_t)(first + w.head) * stride;
            if (is_v) read_tile<D, kFormat, true>(tile, to, stride, kv.v_scale, lane);
            else read_tile<D, kFormat, false>(tile, to, stride, kv.k_scale, lane);
        }
        for (unsigned x = w.rest; x;) {
            const int tok = pick<D>(x, lane);
            const int slot = __shfl_sync(0xffffffffu, w.slot, max(tok, 0)), b = lane % (D / 16);
            if (tok < 0) continue;
            __nv_bfloat16* to = dst + (size_t)(first + tok) * stride + 16 * b;
            if (slot < 0) {
                if (rest == 0 && b == 0 && slots[first + tok] != -1) atomicOr(kv.status, FT_DEV_BAD_ID);
                reinterpret_cast<uint4*>(to)[0] = make_uint4(0, 0, 0, 0);
                reinterpret_cast<uint4*>(to)[1] = make_uint4(0, 0, 0, 0);
                continue;
            }
            const uint8_t* tile = kv_tile_ptr(kv, slot, head, kv_tile(D, kFormat).bytes);
            if (is_v) read_block<D, kFormat, true>(tile, slot & 15, b, to, kv.v_scale);
            else read_block<D, kFormat, false>(tile, slot & 15, b, to, kv.k_scale);
        }
    }
}

// One thread per 16 dims of a token's key or value row; the threads of a token run over K's
// heads and blocks, then V's, so a warp reads whole rows.
template <int D, int kFormat>
__global__ void __launch_bounds__(256) kv_append_kernel(const KvView kv, const __nv_bfloat16* k, const __nv_bfloat16* v,
                                                        size_t k_stride, size_t v_stride, const int32_t* slots, int n) {
    pdl_wait_and_release();
    const int per = kv.hkv * (D / 16);
    const float inv_k = __frcp_rn(kv.k_scale), inv_v = __frcp_rn(kv.v_scale);
    const long long total = 2LL * n * per;
    for (long long g = (long long)blockIdx.x * blockDim.x + threadIdx.x; g < total; g += (long long)gridDim.x * blockDim.x) {
        const int tok = (int)(g / (2 * per)), rest = (int)(g % (2 * per));
        const int slot = slots[tok];
        if (slot < 0 || (slot >> kv.page_shift) >= kv.n_pages) {
            if (slot != -1 && rest == 0) atomicOr(kv.status, FT_DEV_BAD_ID);
            continue;
        }
        const bool is_v = rest >= per;
        const int hb = is_v ? rest - per : rest;
        const int head = hb / (D / 16), b = hb % (D / 16);
        uint8_t* tile = kv_tile_ptr(kv, slot, head, kv_tile(D, kFormat).bytes);
        const int r = slot & 15;
        if (is_v) append_block<D, kFormat, true>(tile, r, b, v + (size_t)tok * v_stride + hb * 16, kv.v_scale, inv_v);
        else append_block<D, kFormat, false>(tile, r, b, k + (size_t)tok * k_stride + hb * 16, kv.k_scale, inv_k);
    }
}

template <int D, int kFormat>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvView kv, const int32_t* slots, int n, __nv_bfloat16* k,
                                                      __nv_bfloat16* v) {
    pdl_wait_and_release();
    const int per = kv.hkv * (D / 16);
    const long long total = 2LL * n * per;
    for (long long g = (long long)blockIdx.x * blockDim.x + threadIdx.x; g < total; g += (long long)gridDim.x * blockDim.x) {
        const int tok = (int)(g / (2 * per)), rest = (int)(g % (2 * per));
        const int slot = slots[tok];
        const bool is_v = rest >= per;
        const int hb = is_v ? rest - per : rest;
        __nv_bfloat16* dst = (is_v ? v : k) + ((size_t)tok * per + hb) * 16;
        if (slot < 0 || (slot >> kv.page_shift) >= kv.n_pages) {
            if (slot != -1 && rest == 0) atomicOr(kv.status, FT_DEV_BAD_ID);
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(0, 0, 0, 0);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(0, 0, 0, 0);
            continue;
        }
        const int head = hb / (D / 16), b = hb % (D / 16);
        const uint8_t* tile = kv_tile_ptr(kv, slot, head, kv_tile(D, kFormat).bytes);
        const int r = slot & 15;
        if (is_v) read_block<D, kFormat, true>(tile, r, b, dst, kv.v_scale);
        else read_block<D, kFormat, false>(tile, r, b, dst, kv.k_scale);
    }
}

namespace {

// fn<D, format>
template <template <int, int> class F, typename... A>
cudaError_t by_shape(int D, int format, A&&... a) {
    if (format == FT_KV_NVFP4) {
        if (D == 64) return F<64, FT_KV_NVFP4>::run(a...);
        if (D == 128) return F<128, FT_KV_NVFP4>::run(a...);
        return F<256, FT_KV_NVFP4>::run(a...);
    }
    if (D == 64) return F<64, FT_KV_FP8>::run(a...);
    if (D == 128) return F<128, FT_KV_FP8>::run(a...);
    return F<256, FT_KV_FP8>::run(a...);
}

unsigned grid_of(long long threads) {
    const long long need = (threads + 255) / 256, most = (long long)sm_count() * 16;
    return (unsigned)(need < most ? need : most);
}

// Rows (tokens times kv heads) from which a call goes by tiles.
constexpr long long kManyRows = 4096;

// Once per kernel and device.
template <auto kKernel>
cudaError_t prepare() {
    static std::atomic<bool> done[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices || done[dev].load(std::memory_order_relaxed)) return e;
    e = all_shared(kKernel);
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_relaxed);
    return e;
}

template <int D, int kFormat>
struct Append {
    static cudaError_t run(const KvView& kv, const void* k, const void* v, size_t ks, size_t vs, const int32_t* slots,
                           int n, cudaStream_t s) {
        if ((long long)n * kv.hkv >= kManyRows) {
            const cudaError_t e = prepare<kv_append_tiles_kernel<D, kFormat>>();
            if (e != cudaSuccess) return e;
            return launch_pdl(kv_append_tiles_kernel<D, kFormat>, dim3(grid_of(((n + 15LL) / 16) * kv.hkv * 64)), dim3(256), 0, s, kv,
                              static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), ks, vs, slots, n);
        }
        const cudaError_t e = prepare<kv_append_kernel<D, kFormat>>();
        if (e != cudaSuccess) return e;
        return launch_pdl(kv_append_kernel<D, kFormat>, dim3(grid_of(2LL * n * kv.hkv * (D / 16))), dim3(256), 0, s, kv,
                          static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), ks, vs, slots, n);
    }
};

template <int D, int kFormat>
struct Read {
    static cudaError_t run(const KvView& kv, const int32_t* slots, int n, void* k, void* v, cudaStream_t s) {
        if ((long long)n * kv.hkv >= kManyRows) {
            const cudaError_t e = prepare<kv_read_tiles_kernel<D, kFormat>>();
            if (e != cudaSuccess) return e;
            return launch_pdl(kv_read_tiles_kernel<D, kFormat>, dim3(grid_of(((n + 15LL) / 16) * kv.hkv * 64)), dim3(256), 0, s, kv,
                              slots, n, static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v));
        }
        const cudaError_t e = prepare<kv_read_kernel<D, kFormat>>();
        if (e != cudaSuccess) return e;
        return launch_pdl(kv_read_kernel<D, kFormat>, dim3(grid_of(2LL * n * kv.hkv * (D / 16))), dim3(256), 0, s, kv,
                          slots, n, static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v));
    }
};

}  // namespace

cudaError_t launch_kv_append(const KvView& kv, int D, int format, const void* k, const void* v, size_t k_stride,
                             size_t v_stride, const int32_t* slots, int n, cudaStream_t s) {
    return by_shape<Append>(D, format, kv, k, v, k_stride, v_stride, slots, n, s);
}

cudaError_t launch_kv_read(const KvView& kv, int D, int format, const int32_t* slots, int n, void* k_out, void* v_out,
                           cudaStream_t s) {
    return by_shape<Read>(D, format, kv, slots, n, k_out, v_out, s);
}

}  // namespace ft

using namespace ft;

namespace {

ft_status fail(ft_kv* kv, ft_status s, const char* what) {
    if (kv) snprintf(kv->err, sizeof kv->err, "%s", what);
    return s;
}

ft_status cuda_fail(ft_kv* kv, cudaError_t e, const char* what) {
    if (kv) snprintf(kv->err, sizeof kv->err, "%s: %s", what, cudaGetErrorString(e));
    return FT_ERR_CUDA;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool positive(float x) { return std::isfinite(x) && x > 0.f; }

int shift_of(int page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

ft_status check_desc(const ft_kv_desc* d) {
    if (!d) return FT_ERR_ARG;
    if (d->L < 1 || d->n_pages < 1 || shift_of(d->page_size) < 0) return FT_ERR_ARG;
    if ((long long)d->n_pages * d->page_size > 0x7FFFFFFFLL) return FT_ERR_ARG;
    if (d->n_kv_heads < 1 || d->n_kv_heads > 1024) return FT_ERR_ARG;
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return FT_ERR_ARG;
    if (d->n_q_heads < 1 || d->n_q_heads > 1024 || d->n_q_heads % d->n_kv_heads) return FT_ERR_ARG;
    if (d->max_seqs < 1 || d->max_seqs > kMaxSeqs) return FT_ERR_ARG;
    if (d->format != FT_KV_NVFP4 && d->format != FT_KV_FP8) return FT_ERR_ARG;
    if (!positive(d->k_scale) || !positive(d->v_scale)) return FT_ERR_ARG;
    return FT_OK;
}

size_t layer_bytes(const ft_kv_desc& d) {
    return (size_t)d.n_pages * d.n_kv_heads * (d.page_size / kKvTile) * kv_tile(d.head_dim, d.format).bytes;
}

bool on_device(const void* p) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged;
}

KvView view(const ft_kv* kv, int layer) {
    const ft_kv_desc& d = kv->d;
    return KvView{static_cast<uint8_t*>(d.pool) + (size_t)layer * kv->layer_bytes, d.n_pages, kv->page_shift,
                  d.n_kv_heads, d.k_scale, d.v_scale, static_cast<int*>(d.workspace)};
}

}  // namespace

extern "C" {

ft_status ft_kv_required_sizes(const ft_kv_desc* d, size_t* pool_bytes, size_t* workspace_bytes) {
    const ft_status s = check_desc(d);
    if (s != FT_OK) return s;
    if (pool_bytes) *pool_bytes = (size_t)d->L * layer_bytes(*d);
    if (workspace_bytes) *workspace_bytes = kKvHeadBytes + kv_task_bytes() + kv_parts_bytes(d->head_dim);
    return FT_OK;
}

ft_status ft_kv_create(const ft_kv_desc* d, ft_kv** out) {
    if (!out) return FT_ERR_ARG;
    *out = nullptr;
    const ft_status s = check_desc(d);
    if (s != FT_OK) return s;
    if (!d->pool || !d->workspace || !aligned(d->pool, 256) || !aligned(d->workspace, 256)) return FT_ERR_ARG;
    if (!on_device(d->pool) || !on_device(d->workspace)) return FT_ERR_ARG;
    ft_kv* kv = new (std::nothrow) ft_kv();
    if (!kv) return FT_ERR_ARG;
    kv->d = *d;
    kv->tile = kv_tile(d->head_dim, d->format);
    kv->layer_bytes = layer_bytes(*d);
    kv->page_shift = shift_of(d->page_size);
    kv->err[0] = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemset(d->workspace, 0, kKvHeadBytes);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        delete kv;
        return FT_ERR_CUDA;
    }
    *out = kv;
    return FT_OK;
}

void ft_kv_destroy(ft_kv* kv) { delete kv; }

ft_status ft_kv_append(ft_kv* kv, int32_t layer, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                       const int32_t* slots, int32_t n, void* stream) {
    if (!kv) return FT_ERR_ARG;
    if (layer < 0 || layer >= kv->d.L || n < 0) return fail(kv, FT_ERR_ARG, "append: layer or n out of range");
    if (n == 0) return FT_OK;
    if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16))
        return fail(kv, FT_ERR_ARG, "append: NULL or misaligned k, v or slots");
    const int64_t row = (int64_t)kv->d.n_kv_heads * kv->d.head_dim;
    if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8)
        return fail(kv, FT_ERR_ARG, "append: token strides");
    NvtxRange r("ft_kv_append");
    const cudaError_t e = launch_kv_append(view(kv, layer), kv->d.head_dim, kv->d.format, k, v, (size_t)k_stride,
                                           (size_t)v_stride, slots, n, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FT_OK : cuda_fail(kv, e, "append launch");
}

ft_status ft_kv_read(ft_kv* kv, int32_t layer, const int32_t* slots, int32_t n, void* k_out, void* v_out, void* stream) {
    if (!kv) return FT_ERR_ARG;
    if (layer < 0 || layer >= kv->d.L || n < 0) return fail(kv, FT_ERR_ARG, "read: layer or n out of range");
    if (n == 0) return FT_OK;
    if (!slots || !k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16))
        return fail(kv, FT_ERR_ARG, "read: NULL or misaligned slots, k_out or v_out");
    NvtxRange r("ft_kv_read");
    const cudaError_t e = launch_kv_read(view(kv, layer), kv->d.head_dim, kv->d.format, slots, n, k_out, v_out,
                                         static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FT_OK : cuda_fail(kv, e, "read launch");
}

ft_status ft_kv_attention(ft_kv* kv, int32_t layer, const void* q, int64_t q_stride, const int32_t* q_start,
                          const int32_t* kv_len, const int32_t* block_table, int32_t table_stride, int32_t n_seqs,
                          int32_t n_tokens, int32_t max_q, const uint64_t* tree_mask, int32_t window, int32_t n_sink,
                          float sm_scale, void* o, int64_t o_stride, float* lse, void* stream) {
    if (!kv) return FT_ERR_ARG;
    const ft_kv_desc& d = kv->d;
    if (layer < 0 || layer >= d.L) return fail(kv, FT_ERR_ARG, "attention: layer out of range");
    if (n_seqs < 0 || n_seqs > d.max_seqs || n_tokens < 0)
        return fail(kv, FT_ERR_ARG, "attention: n_seqs or n_tokens out of range");
    if (table_stride < 1 || max_q < 1 || (tree_mask && max_q > kTreeMax))
        return fail(kv, FT_ERR_ARG, "attention: table_stride or max_q out of range");
    if (window < 0 || n_sink < 0 || !std::isfinite(sm_scale))
        return fail(kv, FT_ERR_ARG, "attention: window, n_sink or sm_scale");
    if (n_seqs == 0 || n_tokens == 0) return FT_OK;
    if (!q || !q_start || !kv_len || !block_table || !o || !aligned(q, 16) || !aligned(o, 16) || !aligned(tree_mask, 8))
        return fail(kv, FT_ERR_ARG, "attention: NULL or misaligned pointer");
    const int64_t row = (int64_t)d.n_q_heads * d.head_dim;
    if (q_stride < row || o_stride < row || q_stride % 8 || o_stride % 8)
        return fail(kv, FT_ERR_ARG, "attention: token strides");
    NvtxRange r("ft_kv_attention");
    AttnArgs a;
    a.kv = view(kv, layer);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_stride = (size_t)q_stride;
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.table = block_table;
    a.table_stride = table_stride;
    a.n_seqs = n_seqs;
    a.n_tokens = n_tokens;
    a.max_q = max_q;
    a.hq = d.n_q_heads;
    a.G = d.n_q_heads / d.n_kv_heads;
    a.g_shift = 0;
    while ((1 << a.g_shift) < a.G) ++a.g_shift;
    a.g_mul = (unsigned)((((uint64_t)1 << 32) * (uint64_t)((1 << a.g_shift) - a.G)) / (uint64_t)a.G + 1);
    a.tree = reinterpret_cast<const unsigned long long*>(tree_mask);
    a.window = window;
    a.n_sink = n_sink;
    a.scale = sm_scale;
    a.o = static_cast<__nv_bfloat16*>(o);
    a.o_stride = (size_t)o_stride;
    a.lse = lse;
    uint8_t* ws = static_cast<uint8_t*>(d.workspace);
    a.tasks = reinterpret_cast<JoinTask*>(ws + kKvHeadBytes);
    a.parts = reinterpret_cast<float*>(ws + kKvHeadBytes + kv_task_bytes());
    const cudaError_t e = launch_kv_attention(a, d.head_dim, d.format, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FT_OK : cuda_fail(kv, e, "attention launch");
}

ft_status ft_kv_status(ft_kv* kv, int32_t* device_status) {
    if (!kv || !device_status) return FT_ERR_ARG;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(device_status, kv->d.workspace, 4, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess) e = cudaMemset(kv->d.workspace, 0, 4);
    return e == cudaSuccess ? FT_OK : cuda_fail(kv, e, "status");
}

const char* ft_kv_last_error(const ft_kv* kv) { return kv ? kv->err : ""; }

}  // extern "C"
