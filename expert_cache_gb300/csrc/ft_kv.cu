// The quantised key/value cache: host side of the C ABI, the writing kernel (bf16 -> codes
// and scales in their tiles) and the reading one (codes -> bf16).
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

// Quantise block b (16 dims) of one token's K or V row into its tile.
template <int D, int kFormat, bool kV>
__device__ __forceinline__ void append_block(uint8_t* tile, int r, int b, const __nv_bfloat16* src, float st) {
    const uint4 x0 = *reinterpret_cast<const uint4*>(src), x1 = *reinterpret_cast<const uint4*>(src + 8);
    const uint32_t xw[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    float x[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        x[2 * j] = __uint_as_float(xw[j] << 16);
        x[2 * j + 1] = __uint_as_float(xw[j] & 0xFFFF0000u);
    }
    uint32_t w[4] = {0, 0, 0, 0};
    if constexpr (kFormat == FT_KV_FP8) {
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j >> 2] |= e4m3_encode_signed(__fdiv_rn(x[j], st)) << (8 * (j & 3));
    } else {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(x[j]));       // fmaxf drops a NaN
        const uint8_t sc = e4m3_encode_rne(__fdiv_rn(__fdiv_rn(amax, 6.0f), st));
        const float denom = __fmul_rn(e4m3_value(sc), st);
        if (denom != 0.f) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                w[j >> 3] |= (uint32_t)e2m1_encode_rne(__fdiv_rn(x[j], denom)) << (4 * (j & 7));
        }
        tile[kV ? kv_v_scale_byte<D>(r, b) : kv_k_scale_byte<D>(r, b)] = denom != 0.f ? sc : 0;
    }
    store_codes<D, kFormat, kV>(tile, r, 16 * b, w);
}

template <int D, int kFormat, bool kV>
__device__ __forceinline__ void read_block(const uint8_t* tile, int r, int b, __nv_bfloat16* dst, float st) {
    uint32_t w[4];
    load_codes<D, kFormat, kV>(w, tile, r, 16 * b);
    float sc = 1.f;
    if constexpr (kFormat == FT_KV_NVFP4)
        sc = e4m3_value(tile[kV ? kv_v_scale_byte<D>(r, b) : kv_k_scale_byte<D>(r, b)]);
    uint32_t out[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * j + e;
            if constexpr (kFormat == FT_KV_NVFP4) {
                const uint32_t c = w[i >> 3] >> (4 * (i & 7)) & 15u;
                const uint32_t m = c & 7u;
                const float mag = m < 2 ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
                f[e] = __fmul_rn(__fmul_rn(c & 8u ? -mag : mag, sc), st);
            } else {
                const uint32_t c = w[i >> 2] >> (8 * (i & 3)) & 255u;
                const float mag = e4m3_value((uint8_t)(c & 127u));
                f[e] = __fmul_rn(c & 128u ? -mag : mag, st);
            }
        }
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[0], f[1]);
        out[j] = *reinterpret_cast<const uint32_t*>(&p);
    }
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(out[0], out[1], out[2], out[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

}  // namespace

// One thread per 16 dims of a token's key or value row; the threads of a token run over K's
// heads and blocks, then V's, so a warp reads whole rows.
template <int D, int kFormat>
__global__ void __launch_bounds__(256) kv_append_kernel(const KvView kv, const __nv_bfloat16* k, const __nv_bfloat16* v,
                                                        size_t k_stride, size_t v_stride, const int32_t* slots, int n) {
    pdl_wait_and_release();
    const int per = kv.hkv * (D / 16);
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
        if (is_v) append_block<D, kFormat, true>(tile, r, b, v + (size_t)tok * v_stride + hb * 16, kv.v_scale);
        else append_block<D, kFormat, false>(tile, r, b, k + (size_t)tok * k_stride + hb * 16, kv.k_scale);
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
        const cudaError_t e = prepare<kv_append_kernel<D, kFormat>>();
        if (e != cudaSuccess) return e;
        return launch_pdl(kv_append_kernel<D, kFormat>, dim3(grid_of(2LL * n * kv.hkv * (D / 16))), dim3(256), 0, s, kv,
                          static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), ks, vs, slots, n);
    }
};

template <int D, int kFormat>
struct Read {
    static cudaError_t run(const KvView& kv, const int32_t* slots, int n, void* k, void* v, cudaStream_t s) {
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
