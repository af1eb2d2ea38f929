// Router: logits to the k experts of each token and their weights.  A warp per token; its choices stand in shared memory.
//
// Choices are computed in fp32 with a bound on their error.  Where two neighbours of the sorted first k + 1 (or the last
// group that stays and the first that does not) lie within their bounds, and do not come from the same logit and bias, the row is
// decided again in 64 bits; so the ids are the formula's.  Without a bias, and without sums of a group's choices, the scores' order
// is the logits' own and needs no rounding at all.
#include <cfloat>
#include <cmath>

#include "ft_internal.cuh"

namespace ft {

namespace {

constexpr int kRouteWarps = 4;
constexpr float kNone = -INFINITY;

struct RouteArgs {
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* w;
    long long stride;
    int T, E, k, n_group, topk_group, group_best, size;     // size: experts of a group
    bool sigmoid, renormalise, by_logit;
    float scale;
};

// A logit as the formula takes it: NaN is -inf, +inf the largest number.
__device__ __forceinline__ float route_logit(float x) { return x == x ? fminf(x, FLT_MAX) : kNone; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return route_logit(__bfloat162float(*p)); }
__device__ __forceinline__ float load_logit(const float* p) { return route_logit(*p); }

template <typename V>
__device__ __forceinline__ V warp_max(V v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The scores of a row in type V: softmax's as exp(x - top) / sum.
template <typename V>
struct Scores {
    V top, sum;
    bool sigmoid;
    __device__ __forceinline__ V of(float x) const {
        if (sigmoid) return V(1) / (V(1) + exp(-V(x)));
        return exp(V(x) - top) / sum;
    }
};
template <typename V>
__device__ __forceinline__ Scores<V> scores_of(const RouteArgs& a, const float* x) {
    const int lane = threadIdx.x & 31;
    Scores<V> s{V(0), V(1), a.sigmoid};
    if (a.sigmoid) return s;
    V top = kNone, sum = 0;
    for (int e = lane; e < a.E; e += 32) top = fmax(top, V(x[e]));
    top = warp_max(top);
    if (top == V(kNone)) top = 0;
    for (int e = lane; e < a.E; e += 32) sum += exp(V(x[e]) - top);
    s.top = top;
    s.sum = warp_sum(sum);
    return s;
}

// A bound on the error of an fp32 choice: the roundings of the exponentials, of their arguments (at most -log of the score in
// magnitude) and of the sum (E / 32 + 5 additions), what underflows, and the bias' addition.
__device__ __forceinline__ float choice_error(const RouteArgs& a, float choice, float bias) {
    const float score = fabsf(choice - bias);
    return 0x1p-23f * (((float)(a.E / 32 + 16) - __log2f(fmaxf(score, 0x1p-120f))) * score + 2.f * fabsf(choice) + 0x1p-100f);
}
__device__ __forceinline__ double choice_error(const RouteArgs&, double, float) { return -1.0; }

// The choices of a row in type V, the groups that stay, and the k first experts: lane j < k gets the j-th (-1: none).
// Returns false if fp32 does not tell.
template <typename V>
__device__ bool decide(const RouteArgs& a, const float* x, V* key, int& id) {
    const int lane = threadIdx.x & 31;
    bool sure = true;
    if (a.by_logit) {
        for (int e = lane; e < a.E; e += 32) key[e] = x[e];
    } else {
        const Scores<V> s = scores_of<V>(a, x);
        for (int e = lane; e < a.E; e += 32) {
            V c = s.of(x[e]) + (a.bias ? V(a.bias[e]) : V(0));
            if (x[e] == kNone || !(c == c)) c = kNone;
            key[e] = c;
        }
    }
    __syncwarp();
    if (a.n_group > 1) {
        // lane g has the two largest of group g
        V one = kNone, two = kNone;
        if (lane < a.n_group) {
            for (int i = 0; i < a.size; ++i) {
                const V c = key[lane * a.size + i];
                two = fmax(two, fmin(one, c));
                one = fmax(one, c);
            }
        }
        const V worth = a.group_best == 2 && two > V(kNone) ? one + two : one;
        float err = 0.f;
        if (!a.by_logit && sizeof(V) == 4 && one > V(kNone)) {
            // the scores of a sum's terms are at most 1, and their magnitudes bound its own rounding
            err = 0x1p-23f * (float)((a.E / 32 + 16) * a.group_best) + 0x1p-22f * (fabsf((float)one) + (two > V(kNone) ? fabsf((float)two) : 0.f));
        }
        int before = 0;
        V least = INFINITY, most = kNone;
        for (int g = 0; g < a.n_group; ++g) {
            const V other = __shfl_sync(0xffffffffu, worth, g);
            before += other > worth || (other == worth && g < lane);
        }
        const bool stays = lane < a.n_group && before < a.topk_group;
        if (sizeof(V) == 4 && !a.by_logit) {
            // worth - err of those that stay against worth + err of those that do not
            if (lane < a.n_group) {
                if (stays) least = worth - V(err);
                else most = worth + V(err);
            }
            least = -warp_max(-least);
            most = warp_max(most);
            if (!(least > most) && most > V(kNone)) sure = false;
        }
        if (lane < a.n_group && !stays)
            for (int i = 0; i < a.size; ++i) key[lane * a.size + i] = kNone;
        __syncwarp();
    }
    id = -1;
    V last = 0;
    int last_id = -1;
    for (int j = 0; j <= a.k; ++j) {
        V best = kNone;
        int at = 0x7FFFFFFF;
        for (int e = lane; e < a.E; e += 32)
            if (key[e] > best) best = key[e], at = e;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const V b = __shfl_xor_sync(0xffffffffu, best, o);
            const int i = __shfl_xor_sync(0xffffffffu, at, o);
            if (b > best || (b == best && i < at)) best = b, at = i;
        }
        if (best == V(kNone)) break;
        if (sizeof(V) == 4 && !a.by_logit && j) {
            const float b0 = a.bias ? a.bias[last_id] : 0.f, b1 = a.bias ? a.bias[at] : 0.f;
            if (!(x[last_id] == x[at] && b0 == b1) && last - best <= choice_error(a, last, b0) + choice_error(a, best, b1)) sure = false;
        }
        if (lane == j && j < a.k) id = at;
        last = best;
        last_id = at;
        if (lane == (at & 31)) key[at] = kNone;
        __syncwarp();
    }
    return sure;
}

template <typename L>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteArgs a) {
    extern __shared__ double route_smem[];
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long t = (long long)blockIdx.x * (blockDim.x >> 5) + warp;
    if (t >= a.T) return;
    double* key = route_smem + (size_t)warp * a.E;
    float* x = reinterpret_cast<float*>(route_smem + (size_t)(blockDim.x >> 5) * a.E) + (size_t)warp * a.E;
    const L* row = static_cast<const L*>(a.logits) + t * a.stride;
    for (int e = lane; e < a.E; e += 32) x[e] = load_logit(row + e);
    __syncwarp();
    int id;
    if (!decide(a, x, reinterpret_cast<float*>(key), id)) {
        __syncwarp();
        decide(a, x, key, id);
    }
    // weights: against the largest of the selected, so that they do not underflow together
    const float mine = id >= 0 ? x[id] : kNone;
    float w = 0.f;
    if (a.renormalise) {
        float top = warp_max(mine);
        if (a.sigmoid) {
            // sigmoid(x) = e^min(x,0) / (1 + e^-|x|)
            top = fminf(top, 0.f);
            if (id >= 0) w = expf(fminf(mine, 0.f) - top) / (1.f + expf(-fabsf(mine)));
        } else if (id >= 0) {
            w = expf(mine - top);
        }
        const float sum = warp_sum(w);
        if (id >= 0) w = w / sum;
    } else {
        const Scores<float> s = scores_of<float>(a, x);
        if (id >= 0) w = s.of(mine);
    }
    if (lane < a.k) {
        a.ids[t * a.k + lane] = id;
        a.w[t * a.k + lane] = w * a.scale;
    }
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace

}  // namespace ft

using namespace ft;

extern "C" ft_status ft_moe_route(const ft_route* call, void* stream) {
    if (!call) return FT_ERR_ARG;
    const ft_route& c = *call;
    if (c.T < 0 || c.E < 1 || c.E > kMaxE || c.k < 1 || c.k > kMaxK || c.k > c.E || c.stride < c.E) return FT_ERR_ARG;
    if ((c.dtype != FT_DTYPE_BF16 && c.dtype != FT_DTYPE_F32) || (c.score != FT_ROUTE_SOFTMAX && c.score != FT_ROUTE_SIGMOID)) return FT_ERR_ARG;
    if (c.n_group < 1 || c.n_group > 32 || c.E % c.n_group || c.topk_group < 1 || c.topk_group > c.n_group) return FT_ERR_ARG;
    if (c.group_best < 1 || c.group_best > 2 || c.renormalise < 0 || c.renormalise > 1 || !std::isfinite(c.scale)) return FT_ERR_ARG;
    if (c.T == 0) return FT_OK;
    const size_t element = c.dtype == FT_DTYPE_BF16 ? 2 : 4;
    if (!c.logits || !c.topk_ids || !c.topk_w || !aligned(c.logits, element) || !aligned(c.bias, 4) || !aligned(c.topk_ids, 4) ||
        !aligned(c.topk_w, 4))
        return FT_ERR_ARG;
    NvtxRange r("ft_moe_route");
    RouteArgs a;
    a.logits = c.logits;
    a.bias = c.bias;
    a.ids = c.topk_ids;
    a.w = c.topk_w;
    a.stride = c.stride;
    a.T = c.T;
    a.E = c.E;
    a.k = c.k;
    a.n_group = c.n_group;
    a.topk_group = c.topk_group;
    a.group_best = c.group_best;
    a.size = c.E / c.n_group;
    a.sigmoid = c.score == FT_ROUTE_SIGMOID;
    a.renormalise = c.renormalise != 0;
    a.by_logit = !c.bias && (c.n_group == 1 || c.group_best == 1);
    a.scale = c.scale;
    const int warps = c.E > 1024 ? 1 : kRouteWarps;
    const size_t smem = (size_t)warps * c.E * 12;                // at most 48 KB
    const unsigned ctas = (unsigned)((c.T + (long long)warps - 1) / warps);
    const cudaError_t e = launch_pdl(c.dtype == FT_DTYPE_BF16 ? route_kernel<__nv_bfloat16> : route_kernel<float>, dim3(ctas),
                                     dim3(warps * 32), smem, static_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}
