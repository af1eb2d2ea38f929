// What the host sides of the key/value calls share.
#pragma once
#include <atomic>
#include <cstdint>
#include <cstdio>

#include "ft_kv.cuh"

namespace ft {

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

inline ft_status fail(ft_kv* kv, ft_status s, const char* what) {
    if (kv) snprintf(kv->err, sizeof kv->err, "%s", what);
    return s;
}

inline ft_status cuda_fail(ft_kv* kv, cudaError_t e, const char* what) {
    if (kv) snprintf(kv->err, sizeof kv->err, "%s: %s", what, cudaGetErrorString(e));
    return FT_ERR_CUDA;
}

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
// Arrays of 32-bit elements (or NULL).
template <typename... P>
bool words(const P*... p) { return (((uintptr_t)p | ...) & 3) == 0; }

inline KvView view(const ft_kv* kv, int layer) {
    const ft_kv_desc& d = kv->d;
    return KvView{static_cast<uint8_t*>(d.pool) + (size_t)layer * kv->layer_bytes, d.n_pages, kv->page_shift,
                  d.n_kv_heads, d.k_scale, d.v_scale, static_cast<int*>(d.workspace)};
}

}  // namespace

}  // namespace ft
