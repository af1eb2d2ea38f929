// The quantised key/value cache: host side of the C ABI, the writing kernels (bf16 -> codes
// and scales in their tiles) and the reading ones (codes -> bf16).
//
// A thread has 16 dims of a token, K's and V's.  A call of few tokens is bound by its launch.  To write 8192 tokens of 8
// heads of 128 in NVFP4 and read them back (86 MB) takes 21.8 us where every pass has other tensors, 3.9 TB/s: 12.6
// us to write and 10.1 to read, of which the bytes need 6.3 each.  Writing takes 263 instructions per 16 values (quotients, packing, place)
// and issues 65 % of the time; reading 165, 53 %, and waits for the codes behind the slots.
#include <cmath>
#include <cstdint>
#include <new>

#include "ft_kv_host.cuh"
#include "ft_kv_quant.cuh"

namespace ft {

namespace {

constexpr int kPlaceThreads = 128;

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
    if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16) || !words(slots))
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
    if (!slots || !k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16) || !words(slots))
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
        !aligned(c.tree_mask, 8) || !words(c.q_start, c.kv_len, c.block_table, c.lse))
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
