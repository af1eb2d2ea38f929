// Log probabilities of given tokens, entropy and the most likely tokens of rows of logits.
#include <cfloat>
#include <cmath>

#include "ft_internal.cuh"

namespace ft {

namespace {

constexpr int kLogThreads = 256;

// A logit as the formula takes it: NaN is -inf, +inf the largest number.
__device__ __forceinline__ float logit(float x) { return x == x ? fminf(x, FLT_MAX) : -INFINITY; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return logit(__bfloat162float(*p)); }
__device__ __forceinline__ float load_logit(const float* p) { return logit(*p); }

struct Best {
    float x;
    int i;
};
__device__ __forceinline__ bool better(Best a, Best b) { return a.x > b.x || (a.x == b.x && a.i < b.i); }

template <typename L>
__global__ void __launch_bounds__(kLogThreads) logprobs_kernel(const ft_logprob c) {
    __shared__ float red[2][kLogThreads / 32];
    __shared__ Best top[kLogThreads / 32];
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long r = blockIdx.x;
    const L* row = static_cast<const L*>(c.logits) + r * c.stride;
    float m = -INFINITY;
    for (int i = threadIdx.x; i < c.V; i += kLogThreads) m = fmaxf(m, load_logit(row + i));
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
    for (int w = 0; w < kLogThreads / 32; ++w) m = fmaxf(m, red[0][w]);
    const bool none = m == -INFINITY;
    __syncthreads();
    float sum = 0.f, dot = 0.f;
    if (!none) {
        for (int i = threadIdx.x; i < c.V; i += kLogThreads) {
            const float y = fmaxf((load_logit(row + i) - m) * c.scale, -200.f), e = expf(y);
            sum += e;
            dot = fmaf(e, y, dot);
        }
    }
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    if (lane == 0) red[0][warp] = sum, red[1][warp] = dot;
    __syncthreads();
    sum = dot = 0.f;
    for (int w = 0; w < kLogThreads / 32; ++w) sum += red[0][w], dot += red[1][w];
    const float log_sum = none ? 0.f : logf(sum);
    if (threadIdx.x == 0) {
        if (c.logp) {
            const int t = c.tokens[r];
            float p = -INFINITY;
            if (!none && t >= 0 && t < c.V) p = (load_logit(row + t) - m) * c.scale - log_sum;
            c.logp[r] = p;
        }
        if (c.entropy) c.entropy[r] = none ? 0.f : fmaxf(log_sum - dot / sum, 0.f);
    }
    Best last{INFINITY, -1};
    for (int j = 0; j < c.k; ++j) {
        Best b{-INFINITY, 0x7FFFFFFF};
        for (int i = threadIdx.x; i < c.V; i += kLogThreads) {
            const Best x{load_logit(row + i), i};
            if (x.x > -INFINITY && better(last, x) && better(x, b)) b = x;
        }
        for (int o = 16; o > 0; o >>= 1) {
            const Best x{__shfl_xor_sync(0xffffffffu, b.x, o), __shfl_xor_sync(0xffffffffu, b.i, o)};
            if (better(x, b)) b = x;
        }
        __syncthreads();
        if (lane == 0) top[warp] = b;
        __syncthreads();
        for (int w = 0; w < kLogThreads / 32; ++w)
            if (better(top[w], b)) b = top[w];
        const bool got = b.x > -INFINITY;
        if (threadIdx.x == 0) {
            c.top_ids[r * c.k + j] = got ? b.i : -1;
            c.top_logp[r * c.k + j] = got ? (b.x - m) * c.scale - log_sum : -INFINITY;
        }
        last = got ? b : Best{-INFINITY, 0x7FFFFFFF};
    }
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace

}  // namespace ft

using namespace ft;

extern "C" ft_status ft_logprobs(const ft_logprob* call, void* stream) {
    if (!call) return FT_ERR_ARG;
    const ft_logprob& c = *call;
    if (c.n < 0 || c.V < 1 || c.V > 1 << 30 || c.k < 0 || c.k > kMaxK || c.k > c.V || c.stride < c.V) return FT_ERR_ARG;
    if ((c.dtype != FT_DTYPE_BF16 && c.dtype != FT_DTYPE_F32) || !std::isfinite(c.scale) || c.scale <= 0.f) return FT_ERR_ARG;
    if (c.n == 0) return FT_OK;
    if (!c.logits || !aligned(c.logits, c.dtype == FT_DTYPE_BF16 ? 2 : 4) || (c.logp && !c.tokens) || (c.k && (!c.top_ids || !c.top_logp)))
        return FT_ERR_ARG;
    if (!aligned(c.tokens, 4) || !aligned(c.logp, 4) || !aligned(c.entropy, 4) || !aligned(c.top_ids, 4) || !aligned(c.top_logp, 4)) return FT_ERR_ARG;
    NvtxRange r("ft_logprobs");
    const cudaError_t e = launch_pdl(c.dtype == FT_DTYPE_BF16 ? logprobs_kernel<__nv_bfloat16> : logprobs_kernel<float>, dim3((unsigned)c.n),
                                     dim3(kLogThreads), 0, static_cast<cudaStream_t>(stream), c);
    return e == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}
