// Attention over the quantised key/value cache.
//
// o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i.k_j - m_i), one pass over the keys with
// the running maximum m_i and sum: a larger maximum m' rescales both by exp(m - m').
#include "ft_kv.cuh"
#include "ft_quant.cuh"

namespace ft {

namespace {

// Stored value (without the tensor scale) of token r's dim d.
template <int D, int kFormat, bool kV>
__device__ __forceinline__ float kv_value(const uint8_t* tile, int r, int d) {
    const int at = (kV ? kv_v_byte<D, kFormat>(r, d & ~7) : kv_k_byte<D, kFormat>(r, d & ~7)) +
                   (kFormat == FT_KV_NVFP4 ? (d & 7) >> 1 : d & 7);
    const uint32_t byte = tile[at];
    if constexpr (kFormat == FT_KV_FP8) {
        const float m = e4m3_value((uint8_t)(byte & 127u));
        return byte & 128u ? -m : m;
    } else {
        const uint32_t c = byte >> (4 * (d & 1)) & 15u, m = c & 7u;
        const float mag = m < 2 ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
        const float sc = e4m3_value(tile[kV ? kv_v_scale_byte<D>(r, d / 16) : kv_k_scale_byte<D>(r, d / 16)]);
        return (c & 8u ? -mag : mag) * sc;
    }
}

}  // namespace

// One warp per row and query head; lane l holds the dims l, l + 32, ...
template <int D, int kFormat>
__global__ void __launch_bounds__(128) kv_attention_simple_kernel(const AttnArgs a) {
    const int lane = threadIdx.x & 31;
    const int s = blockIdx.y;
    const SeqInfo si = seq_info(a, s);
    if (si.bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.kv.status, FT_DEV_BAD_ID);
    const int base = si.len - si.n;
    for (long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5); w < (long long)si.n * a.hq; w += (long long)gridDim.x * 4) {
        const int i = (int)(w / a.hq), h = (int)(w % a.hq), kvh = h / a.G;
        const size_t row = (size_t)si.q0 + i;
        float q[D / 32], acc[D / 32];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
            q[e] = __bfloat162float(a.q[row * a.q_stride + (size_t)h * D + lane + 32 * e]);
            acc[e] = 0.f;
        }
        const unsigned long long mine = a.tree ? a.tree[row] : 0;
        const int pos = base + (a.tree ? __popcll(mine & ~(1ull << (i & 63))) : i);
        float m = -INFINITY, l = 0.f;
        for (int j = 0; j < si.len; ++j) {
            const int jj = j - base;
            if (a.tree ? (jj >= 0 && (jj > 63 || !(mine >> jj & 1))) : jj > i) continue;
            if (a.window > 0 && j >= a.n_sink) {
                const int pj = a.tree && jj >= 0 ? base + __popcll(a.tree[si.q0 + jj] & ~(1ull << jj)) : j;
                if (pos - pj >= a.window) continue;
            }
            const int page = a.table[(size_t)s * a.table_stride + (j >> a.kv.page_shift)];
            if (page < 0 || page >= a.kv.n_pages) {
                if (lane == 0) atomicOr(a.kv.status, FT_DEV_BAD_ID);
                continue;
            }
            const int in = j & ((1 << a.kv.page_shift) - 1);
            const uint8_t* tile = a.kv.pool + ((((size_t)page * a.kv.hkv + kvh) << (a.kv.page_shift - 4)) + (in >> 4)) *
                                                  kv_tile(D, kFormat).bytes;
            float z = 0.f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) z += q[e] * kv_value<D, kFormat, false>(tile, in & 15, lane + 32 * e);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
            z *= a.kv.k_scale * a.scale;
            const float mn = fmaxf(m, z), ms = mn == -INFINITY ? 0.f : mn;      // a NaN logit stays a NaN weight
            const float f = expf(m - ms), p = expf(z - ms);
            m = mn;
            l = l * f + p;
#pragma unroll
            for (int e = 0; e < D / 32; ++e)
                acc[e] = acc[e] * f + p * kv_value<D, kFormat, true>(tile, in & 15, lane + 32 * e);
        }
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            a.o[row * a.o_stride + (size_t)h * D + lane + 32 * e] =
                __float2bfloat16(l > 0.f ? acc[e] / l * a.kv.v_scale : (l == 0.f ? 0.f : l));
        if (a.lse && lane == 0) a.lse[row * a.hq + h] = l == 0.f ? -INFINITY : m + logf(l);
    }
}

cudaError_t launch_kv_attention(const AttnArgs& a, int D, int format, cudaStream_t s) {
    const dim3 grid(256, a.n_seqs);
#define FT_RUN(d, f) if (D == d && format == f) kv_attention_simple_kernel<d, f><<<grid, 128, 0, s>>>(a);
    FT_RUN(64, FT_KV_NVFP4) FT_RUN(128, FT_KV_NVFP4) FT_RUN(256, FT_KV_NVFP4)
    FT_RUN(64, FT_KV_FP8) FT_RUN(128, FT_KV_FP8) FT_RUN(256, FT_KV_FP8)
#undef FT_RUN
    return cudaGetLastError();
}

}  // namespace ft
