// The quantised key/value cache: host side of the C ABI, the writing kernels (bf16 -> codes
// and scales in their tiles) and the reading ones (codes -> bf16).
//
// A thread has 16 dims of a token, K's and V's.  A call of few tokens is bound by its launch.  To write 8192 tokens of 8
// heads of 128 in NVFP4 and read them back (86 MB) takes 21.8 us where every pass has other tensors, 3.9 TB/s: 12.6
// us to write and 10.1 to read, of which the bytes need 6.3 each.  Writing takes 263 instructions per 16 values (quotients, packing, place)
// and issues 65 % of the time; reading 165, 53 %, and waits for the codes behind the slots.
//
// Quotients are the definition's x / (scale * s), rounded to nearest, in three operations: with
// r = RN(1/d) and q0 = RN(x r), q0 + RN(x - q0 d) r rounds to RN(x/d) (Markstein's correction, 1990;
// compared with the division for every bf16 significand over every fp32 one: no difference), as long
// as nothing over- or underflows; a block where something could, with a NaN, an infinity or
// a saturated scale, takes the division itself.  The conversion instructions round to nearest even
// and saturate like the definition; only a zero's sign is dropped afterwards.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <new>

#include "ft_kv.cuh"
#include "ft_quant.cuh"

namespace ft {

namespace {

constexpr int kPlaceThreads = 128;

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
__device__ __forceinline__ void append_block(uint8_t* tile, int r, int b, const uint32_t (&xw)[8], float st, float inv_st) {
    uint32_t w[4];
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

// What a warp takes, a block of 16 dims of a token per lane: 8 tokens, in the call's order, by 4 blocks (64 dims)
// of a head.  Of tokens that are neighbours in a tile the codes are then stored in full sectors, and rows read
// 128 bytes at a time (8192 tokens of 8 heads of 128 written and read, the same tensors again and again, which L2 holds in
// part: 18.2 us; 4 tokens by 8 blocks 19 us; tokens by whole rows, which store V in pieces of 8 bytes, 20.6 us).
constexpr int kPatchBlocks = 4, kPatchTokens = 32 / kPatchBlocks;

struct Place {
    int tok, hb, slot;       // token, block among a token's, where it stands (-1: nowhere)
};
template <int D, typename F>
__device__ __forceinline__ void each_place(const KvView& kv, const int32_t* slots, int n, F f) {
    const int lane = threadIdx.x & 31, patches = kv.hkv * (D / 16 / kPatchBlocks);
    const int warps = gridDim.x * (kPlaceThreads / 32), at = blockIdx.x * (kPlaceThreads / 32) + (threadIdx.x >> 5);
    int group = at / patches, patch = at % patches;
    const int groups = (int)(((long long)n + kPatchTokens - 1) / kPatchTokens), dg = warps / patches, dp = warps % patches;
    while (group < groups) {
        Place p;
        p.tok = group * kPatchTokens + lane / kPatchBlocks;
        p.hb = patch * kPatchBlocks + lane % kPatchBlocks;
        if (p.tok < n) {
            p.slot = slots[p.tok];
            if (p.slot < 0 || (p.slot >> kv.page_shift) >= kv.n_pages) {
                if (p.slot != -1 && p.hb == 0) atomicOr(kv.status, FT_DEV_BAD_ID);
                p.slot = -1;
            }
            f(p);
        }
        group += dg;
        patch += dp;
        if (patch >= patches) {
            patch -= patches;
            ++group;
        }
    }
}

}  // namespace

// kBoth: a thread has K's block and V's; otherwise those with blockIdx.y = 0 K's, with 1 V's.
template <int D, int kFormat, bool kBoth>
__global__ void __launch_bounds__(kPlaceThreads) kv_append_kernel(const KvView kv, const __nv_bfloat16* k, const __nv_bfloat16* v,
                                                                  size_t k_stride, size_t v_stride, const int32_t* slots, int n) {
    pdl_wait_and_release();
    const float inv_k = __frcp_rn(kv.k_scale), inv_v = __frcp_rn(kv.v_scale);
    each_place<D>(kv, slots, n, [&](const Place& p) {
        if (p.slot < 0) return;
        const int r = p.slot & 15, b = p.hb % (D / 16);
        uint8_t* tile = kv_tile_ptr(kv, p.slot, p.hb / (D / 16), kv_tile(D, kFormat).bytes);
        uint32_t xk[8], xv[8];
        if (kBoth || blockIdx.y == 0) load_block(xk, k + (size_t)p.tok * k_stride + p.hb * 16);
        if (kBoth || blockIdx.y == 1) load_block(xv, v + (size_t)p.tok * v_stride + p.hb * 16);
        if (kBoth || blockIdx.y == 0) append_block<D, kFormat, false>(tile, r, b, xk, kv.k_scale, inv_k);
        if (kBoth || blockIdx.y == 1) append_block<D, kFormat, true>(tile, r, b, xv, kv.v_scale, inv_v);
    });
}

template <int D, int kFormat, bool kBoth>
__global__ void __launch_bounds__(kPlaceThreads) kv_read_kernel(const KvView kv, const int32_t* slots, int n, __nv_bfloat16* k,
                                                                __nv_bfloat16* v) {
    pdl_wait_and_release();
    const int per = kv.hkv * (D / 16);
    each_place<D>(kv, slots, n, [&](const Place& p) {
        const size_t at = ((size_t)p.tok * per + p.hb) * 16;
        if (p.slot < 0) {
            for (int is_v = 0; is_v < 2; ++is_v) {
                if (!kBoth && (int)blockIdx.y != is_v) continue;
                uint4* dst = reinterpret_cast<uint4*>((is_v ? v : k) + at);
                dst[0] = dst[1] = make_uint4(0, 0, 0, 0);
            }
            return;
        }
        const int r = p.slot & 15, b = p.hb % (D / 16);
        const uint8_t* tile = kv_tile_ptr(kv, p.slot, p.hb / (D / 16), kv_tile(D, kFormat).bytes);
        if (kBoth || blockIdx.y == 0) read_block<D, kFormat, false>(tile, r, b, k + at, kv.k_scale);
        if (kBoth || blockIdx.y == 1) read_block<D, kFormat, true>(tile, r, b, v + at, kv.v_scale);
    });
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

// A warp per patch, at most 2^20 CTAs (32-bit indexes).  A thread has both K's block and V's, so that it finds its
// place once (two threads: 21.8 us instead of 18.2 for 8192 tokens of 8 heads of 128, the same tensors again), but one of them where
// that leaves fewer than four warps per SM (16 tokens: 3.7 us instead of 4.3).
struct PlaceGrid {
    unsigned ctas;
    bool both;
};
PlaceGrid place_grid(int n, int blocks) {
    const long long warps = ((long long)n + kPatchTokens - 1) / kPatchTokens * (blocks / kPatchBlocks);
    const long long ctas = (warps + kPlaceThreads / 32 - 1) / (kPlaceThreads / 32);
    return {(unsigned)(ctas < (1 << 20) ? ctas : 1 << 20), warps >= 4LL * sm_count()};
}

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
    static cudaError_t run(const KvView& kv, const void* k, const void* v, size_t ks, size_t vs, const int32_t* slots, int n,
                           cudaStream_t s) {
        const PlaceGrid g = place_grid(n, kv.hkv * (D / 16));
        const cudaError_t e = g.both ? prepare<kv_append_kernel<D, kFormat, true>>() : prepare<kv_append_kernel<D, kFormat, false>>();
        if (e != cudaSuccess) return e;
        return launch_pdl(g.both ? kv_append_kernel<D, kFormat, true> : kv_append_kernel<D, kFormat, false>, dim3(g.ctas, g.both ? 1 : 2),
                          dim3(kPlaceThreads), 0, s, kv, static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), ks, vs, slots, n);
    }
};

template <int D, int kFormat>
struct Read {
    static cudaError_t run(const KvView& kv, const int32_t* slots, int n, void* k, void* v, cudaStream_t s) {
        const PlaceGrid g = place_grid(n, kv.hkv * (D / 16));
        const cudaError_t e = g.both ? prepare<kv_read_kernel<D, kFormat, true>>() : prepare<kv_read_kernel<D, kFormat, false>>();
        if (e != cudaSuccess) return e;
        return launch_pdl(g.both ? kv_read_kernel<D, kFormat, true> : kv_read_kernel<D, kFormat, false>, dim3(g.ctas, g.both ? 1 : 2),
                          dim3(kPlaceThreads), 0, s, kv, slots, n, static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v));
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

size_t layer_bytes(const ft_kv_desc& d) {
    return (size_t)d.n_pages * d.n_kv_heads * (d.page_size / kKvTile) * kv_tile(d.head_dim, d.format).bytes;
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
    if ((size_t)d->L > (SIZE_MAX >> 1) / layer_bytes(*d)) return FT_ERR_ARG;     // the pool's bytes
    return FT_OK;
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

ft_status ft_kv_attention(ft_kv* kv, const ft_kv_attn* call, void* stream) {
    if (!kv) return FT_ERR_ARG;
    if (!call) return fail(kv, FT_ERR_ARG, "attention: NULL call");
    const ft_kv_desc& d = kv->d;
    const ft_kv_attn& c = *call;
    if (c.layer < 0 || c.layer >= d.L) return fail(kv, FT_ERR_ARG, "attention: layer out of range");
    if (c.n_seqs < 0 || c.n_seqs > d.max_seqs || c.n_tokens < 0)
        return fail(kv, FT_ERR_ARG, "attention: n_seqs or n_tokens out of range");
    if (c.table_stride < 1 || c.max_q < 1 || (c.tree_mask && c.max_q > kTreeMax) ||
        (int64_t)c.max_q * (d.n_q_heads / d.n_kv_heads) > (1 << 30))
        return fail(kv, FT_ERR_ARG, "attention: table_stride or max_q out of range");
    if (c.window < 0 || c.n_sink < 0 || !std::isfinite(c.sm_scale))
        return fail(kv, FT_ERR_ARG, "attention: window, n_sink or sm_scale");
    if (c.n_seqs == 0 || c.n_tokens == 0) return FT_OK;
    if (!c.q || !c.q_start || !c.kv_len || !c.block_table || !c.o || !aligned(c.q, 16) || !aligned(c.o, 16) ||
        !aligned(c.tree_mask, 8))
        return fail(kv, FT_ERR_ARG, "attention: NULL or misaligned pointer");
    const int64_t row = (int64_t)d.n_q_heads * d.head_dim;
    if (c.q_stride < row || c.o_stride < row || c.q_stride % 8 || c.o_stride % 8)
        return fail(kv, FT_ERR_ARG, "attention: token strides");
    NvtxRange r("ft_kv_attention");
    AttnArgs a;
    a.kv = view(kv, c.layer);
    a.q = static_cast<const __nv_bfloat16*>(c.q);
    a.q_stride = (size_t)c.q_stride;
    a.q_start = c.q_start;
    a.kv_len = c.kv_len;
    a.table = c.block_table;
    a.table_stride = c.table_stride;
    a.n_seqs = c.n_seqs;
    a.n_tokens = c.n_tokens;
    a.max_q = c.max_q;
    a.hq = d.n_q_heads;
    a.G = d.n_q_heads / d.n_kv_heads;
    a.g_shift = 0;
    while ((1 << a.g_shift) < a.G) ++a.g_shift;
    a.g_mul = (unsigned)((((uint64_t)1 << 32) * (uint64_t)((1 << a.g_shift) - a.G)) / (uint64_t)a.G + 1);
    a.tree = reinterpret_cast<const unsigned long long*>(c.tree_mask);
    a.window = c.window;
    a.n_sink = c.n_sink;
    a.scale = c.sm_scale;
    a.o = static_cast<__nv_bfloat16*>(c.o);
    a.o_stride = (size_t)c.o_stride;
    a.lse = c.lse;
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

ft_status ft_kv_check_bounded_waits(uint32_t* expired) {
    if (!expired) return FT_ERR_ARG;
    unsigned* bits = nullptr;
    cudaError_t e = cudaMalloc(&bits, sizeof(unsigned));
    if (e != cudaSuccess) return FT_ERR_CUDA;
    e = cudaMemset(bits, 0, sizeof(unsigned));
    if (e == cudaSuccess) e = check_rows_waits(bits);
    if (e == cudaSuccess) e = check_tiles_waits(bits);
    if (e == cudaSuccess) e = cudaMemcpy(expired, bits, sizeof(unsigned), cudaMemcpyDeviceToHost);
    cudaFree(bits);
    return e == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}

const char* ft_kv_last_error(const ft_kv* kv) { return kv ? kv->err : ""; }

}  // extern "C"
