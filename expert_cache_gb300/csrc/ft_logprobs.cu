// Log probabilities of given tokens, entropy and the most likely tokens of rows of logits.
//
// One pass over a row, by a cluster of 1 to 8 CTAs: with y = scale (x - ref) per thread the sums S = sum e^y and D = sum e^y y
// give log sum = log S and entropy = log S - D / S.  A thread's ref is a maximum of a sample of the row, so that no
// sum has to be rescaled unless a logit lies e^69 above it; the row's own maximum is taken at the end.
//
// The k largest come out of the same pass.  From the sample (4 vectors of every thread, spread over the CTA's part
// of the row and kept in registers) the k-th largest of some 64 logits is a lower bound of the row's k-th; only what reaches it is
// put on a list in shared memory (some dozens of 100,000), and the list is ranked at the end.  Where more reach it than
// the list holds, its own k-th largest is the next bound and the part is read again; where that does not help (equal
// logits by the thousand), k searches find them.  Which ones these are does not depend on any order: value, then index.
#include <cfloat>
#include <cmath>

#include "ft_internal.cuh"

namespace ft {

namespace {

constexpr int kLogThreads = 512, kLogWarps = kLogThreads / 32;
constexpr int kSample = 4;             // vectors of a thread's sample
constexpr int kListed = 1024;          // entries of a CTA's list
constexpr int kMaxCtas = 8;            // of a row
constexpr float kNone = -INFINITY;

struct Best {
    float x;
    int i;
};
__device__ __forceinline__ bool better(Best a, Best b) { return a.x > b.x || (a.x == b.x && a.i < b.i); }

// 16 bytes of logits.
template <typename L>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    uint4 w;
    __device__ __forceinline__ void none() { w = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void first(const __nv_bfloat16* p) { w.x = (w.x & 0xFFFF0000u) | *reinterpret_cast<const uint16_t*>(p); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) x[2 * j] = __uint_as_float(u[j] << 16), x[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
    }
    // the largest, NaN aside
    __device__ __forceinline__ float max() const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(u);
        const float2 f = __bfloat1622float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
        return fmaxf(f.x, f.y);
    }
};
template <>
struct Vec<float> {
    static constexpr int kN = 4;
    float4 w;
    __device__ __forceinline__ void none() { w = make_float4(kNone, kNone, kNone, kNone); }
    __device__ __forceinline__ void load(const float* p) { w = __ldg(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void first(const float* p) { w.x = *p; }
    __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w; }
    __device__ __forceinline__ float max() const { return fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w)); }
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Unsigned words in the order of the floats.
__device__ __forceinline__ unsigned ordered(float x) {
    const unsigned u = __float_as_uint(x);
    return u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(unsigned u) { return __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xFFFFFFFFu)); }

struct LogShared {
    Best list[kListed];
    Best top[kMaxCtas * kMaxK];        // the row's CTAs' k best, this one's at its rank in the first
    float few[kLogWarps * 4];          // the sample's largest
    float red[3][kLogWarps];
    float sum[3];                      // this CTA's largest, S and D
    Best one;
    int count;
    float bound, ref;
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word of the same place in another CTA's shared memory.
__device__ __forceinline__ uint32_t remote_word(const void* p, int rank) {
    uint32_t a = (uint32_t)__cvta_generic_to_shared(p), v;
    asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %1, %2;\n\tld.shared::cluster.b32 %0, [r];\n\t}"
                 : "=r"(v) : "r"(a), "r"(rank) : "memory");
    return v;
}

// A thread's sums against its ref (in units of log 2).
struct Sums {
    float ref, far, top, s, d;         // far: where a logit needs another ref; top: the largest seen
    __device__ __forceinline__ void start(float at, float c) {
        ref = at;
        far = at == kNone ? kNone : at + 100.f / c;
        s = d = 0.f;
    }
    template <int N>
    __device__ __forceinline__ void add(const float (&x)[N], float c) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float y = fmaxf((x[j] - ref) * c, -200.f), e = exp2_fast(y);       // -200: what adds nothing; NaN too
            s += e;
            d = fmaf(e, y, d);
        }
    }
    // The sums against another ref.
    __device__ __forceinline__ void move(float to, float c) {
        if (s > 0.f) {
            const float y = fmaxf((ref - to) * c, -1e30f), f = exp2_fast(y);
            d = f > 0.f ? f * fmaf(y, s, d) : 0.f;
            s *= f;
        }
        ref = to;
    }
};

// A vector with a logit far above a thread's ref (out of line, by value: rare, and the sums stay in registers).
template <typename L>
__device__ __noinline__ Sums add_far(Sums a, Vec<L> v, float most, float c) {
    const float to = fminf(most, FLT_MAX);
    if (to > a.ref) {
        a.move(to, c);
        a.far = to + 100.f / c;
    }
    float x[Vec<L>::kN];
    v.get(x);
#pragma unroll
    for (int j = 0; j < Vec<L>::kN; ++j) x[j] = x[j] == x[j] ? fminf(x[j], FLT_MAX) : kNone;
    a.add(x, c);
    return a;
}

template <typename L>
__device__ __forceinline__ void put_on_list(LogShared& sm, const Vec<L>& v, int index, float bound) {
    float x[Vec<L>::kN];
    v.get(x);
#pragma unroll
    for (int j = 0; j < Vec<L>::kN; ++j) {
        if (x[j] >= bound && x[j] > kNone) {
            const int at = atomicAdd(&sm.count, 1);
            if (at < kListed) sm.list[at] = Best{fminf(x[j], FLT_MAX), index + j};
        }
    }
}

template <typename L, bool kTop>
__device__ __forceinline__ void take(LogShared& sm, Sums& a, const Vec<L>& v, int index, float bound, float c) {
    const float most = v.max();
    a.top = fmaxf(a.top, most);
    if (most > a.far) {
        a = add_far(a, v, most, c);
    } else {
        float x[Vec<L>::kN];
        v.get(x);
        a.add(x, c);
    }
    if (kTop && most >= bound) put_on_list(sm, v, index, bound);
}

// A CTA's part of a row: vectors lo .. hi, and for the first one the elements before and behind the row's vectors.
template <typename L>
struct Part {
    const L* row;
    int head, lo, hi, steps, V, rest;  // rest: elements outside the vectors (rank 0)
    __device__ __forceinline__ Part(const L* r, int V_, int rank, int ctas) : row(r), V(V_) {
        constexpr int kN = Vec<L>::kN;
        head = min((int)((16 - ((uintptr_t)row & 15)) & 15) / (int)sizeof(L), V);
        const int n = (V - head) / kN;
        lo = (int)((long long)n * rank / ctas);
        hi = (int)((long long)n * (rank + 1) / ctas);
        steps = (hi - lo + kLogThreads - 1) / kLogThreads;
        rest = rank == 0 ? V - n * kN : 0;
    }
    __device__ __forceinline__ int index(int vec) const { return head + vec * Vec<L>::kN; }
    // The it-th vector of this thread; false (and no logits) past the end.
    __device__ __forceinline__ bool load(Vec<L>& v, int it, int& at) const {
        const int vec = lo + it * kLogThreads + (int)threadIdx.x;
        at = index(vec);
        if (vec < hi) {
            v.load(row + at);
            return true;
        }
        v.none();
        return false;
    }
    __device__ __forceinline__ bool load_rest(Vec<L>& v, int& at) const {
        v.none();
        if ((int)threadIdx.x >= rest) return false;
        at = (int)threadIdx.x < head ? threadIdx.x : V - rest + threadIdx.x;
        v.first(row + at);
        return true;
    }
};

// Puts everything that reaches the bound on the list.
template <typename L>
__device__ void collect(LogShared& sm, const Part<L>& p) {
    const float bound = sm.bound;
    Vec<L> v;
    int at;
    for (int it = -1; it < p.steps; ++it) {
        if (!(it < 0 ? p.load_rest(v, at) : p.load(v, it, at))) continue;
        put_on_list(sm, v, at, bound);
    }
}

// The k best of the list's n entries, in order, to out (entries without one: -inf).
__device__ __forceinline__ void rank_list(const Best* list, int n, int k, Best* out) {
    for (int j = threadIdx.x; j < k; j += kLogThreads)
        if (j >= n) out[j] = Best{kNone, -1};
    for (int e = threadIdx.x; e < n; e += kLogThreads) {
        const Best mine = list[e];
        int before = 0;
        for (int i = 0; i < n; ++i) before += better(list[i], mine) || (list[i].x == mine.x && list[i].i == mine.i && i < e);   // several may be none
        if (before < k) out[before] = mine;
    }
}

// The k best by k searches.
template <typename L>
__device__ void search(LogShared& sm, const Part<L>& p, int k, Best* out) {
    Best last{INFINITY, -1};
    for (int j = 0; j < k; ++j) {
        Best b{kNone, 0x7FFFFFFF};
        Vec<L> v;
        int at;
        for (int it = -1; it < p.steps; ++it) {
            if (!(it < 0 ? p.load_rest(v, at) : p.load(v, it, at))) continue;
            float x[Vec<L>::kN];
            v.get(x);
#pragma unroll
            for (int i = 0; i < Vec<L>::kN; ++i) {
                const Best e{fminf(x[i], FLT_MAX), at + i};
                if (x[i] > kNone && better(last, e) && better(e, b)) b = e;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const Best e{__shfl_xor_sync(0xffffffffu, b.x, o), __shfl_xor_sync(0xffffffffu, b.i, o)};
            if (better(e, b)) b = e;
        }
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sm.list[threadIdx.x >> 5] = b;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kLogWarps; ++w)
                if (better(sm.list[w], b)) b = sm.list[w];
            sm.one = b.x > kNone ? b : Best{kNone, 0x7FFFFFFF};
            out[j] = b.x > kNone ? b : Best{kNone, -1};
        }
        __syncthreads();
        last = sm.one;
    }
}

template <typename L, bool kTop>
__global__ void __launch_bounds__(kLogThreads, 2) logprobs_kernel(const ft_logprob c, int ctas) {
    __shared__ LogShared sm;
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long r = blockIdx.x / ctas;
    const int rank = blockIdx.x % ctas;
    const L* row = static_cast<const L*>(c.logits) + r * c.stride;
    const Part<L> p(row, c.V, rank, ctas);
    const float c2 = fminf(c.scale * 1.4426950408889634f, FLT_MAX);

    // the sample
    Vec<L> v[kSample], extra;
    int at[kSample], extra_at = 0;
    const int stride = max(p.steps / kSample, 1);
#pragma unroll
    for (int i = 0; i < kSample; ++i) p.load(v[i], i * stride, at[i]);
    const bool has_extra = p.load_rest(extra, extra_at);
    float asked = kNone;                                         // the given token's logit
    if (rank == 0 && threadIdx.x == 0 && c.logp) {
        const int t = c.tokens[r];
        if (t >= 0 && t < c.V) {
            asked = (float)row[t];
            asked = asked == asked ? fminf(asked, FLT_MAX) : kNone;
        }
    }
    float most = v[0].max();
#pragma unroll
    for (int i = 1; i < kSample; ++i) most = fmaxf(most, v[i].max());
    most = most == most ? fminf(most, FLT_MAX) : kNone;
    // the warp's four largest
    unsigned key = ordered(most);
#pragma unroll
    for (int i = 0; i < (kTop ? 4 : 1); ++i) {
        const unsigned u = __reduce_max_sync(0xffffffffu, key);
        if (lane == 0) sm.few[warp * 4 + i] = unordered(u);
        if (kTop && lane == __ffs(__ballot_sync(0xffffffffu, key == u)) - 1) key = ordered(kNone);
    }
    if (threadIdx.x == 0) sm.count = 0;
    __syncthreads();
    if (kTop) {
        if (threadIdx.x < kLogWarps * 4) {
            const float mine = sm.few[threadIdx.x];
            int before = 0;
#pragma unroll 16
            for (int i = 0; i < kLogWarps * 4; ++i) {
                const float x = sm.few[i];
                before += x > mine || (x == mine && i < (int)threadIdx.x);
            }
            if (before == c.k - 1) sm.bound = mine;
            if (before == 0) sm.ref = mine;
        }
    } else if (threadIdx.x == 0) {
        float m = sm.few[0];
        for (int w = 1; w < kLogWarps; ++w) m = fmaxf(m, sm.few[4 * w]);
        sm.ref = m;
    }
    __syncthreads();

    const float bound = kTop ? sm.bound : 0.f;
    Sums a;
    a.start(sm.ref, c2);
    a.top = kNone;
#pragma unroll
    for (int i = 0; i < kSample; ++i)
        if (i < p.steps) take<L, kTop>(sm, a, v[i], at[i], bound, c2);
    if (has_extra) take<L, kTop>(sm, a, extra, extra_at, bound, c2);
    // the rest of the part
    for (int i = 0; i < kSample; ++i) {
        const int end = i == kSample - 1 ? p.steps : min((i + 1) * stride, p.steps);
        for (int it = i * stride + 1; it < end; it += kSample) {
#pragma unroll
            for (int j = 0; j < kSample; ++j) {
                if (it + j < end) p.load(v[j], it + j, at[j]);
                else v[j].none();
            }
#pragma unroll
            for (int j = 0; j < kSample; ++j)
                if (it + j < end) take<L, kTop>(sm, a, v[j], at[j], bound, c2);
        }
    }
    a.top = a.top == a.top ? fminf(a.top, FLT_MAX) : kNone;

    // the CTA's sums against its largest
    float m = unordered(__reduce_max_sync(0xffffffffu, ordered(a.top)));
    if (lane == 0) sm.red[0][warp] = m;
    __syncthreads();
    m = sm.red[0][0];
#pragma unroll
    for (int w = 1; w < kLogWarps; ++w) m = fmaxf(m, sm.red[0][w]);
    a.move(m, c2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
        a.d += __shfl_xor_sync(0xffffffffu, a.d, o);
    }
    if (lane == 0) sm.red[1][warp] = a.s, sm.red[2][warp] = a.d;
    __syncthreads();
    if (threadIdx.x < 3) {
        float x = sm.red[threadIdx.x][0];
        for (int w = 1; w < kLogWarps; ++w) x = threadIdx.x ? x + sm.red[threadIdx.x][w] : fmaxf(x, sm.red[0][w]);
        sm.sum[threadIdx.x] = x;
    }

    if (kTop) {
        int n = sm.count;
        while (n > kListed) {
            // the list's k-th largest bounds the row's; if it is no better than the last one, the searches
            rank_list(sm.list, kListed, c.k, sm.top);
            __syncthreads();
            const float next = sm.top[c.k - 1].x;
            if (!(next > sm.bound)) break;
            __syncthreads();
            if (threadIdx.x == 0) sm.bound = next, sm.count = 0;
            __syncthreads();
            collect(sm, p);
            __syncthreads();
            n = sm.count;
        }
        if (n > kListed) search(sm, p, c.k, sm.top);
        else rank_list(sm.list, n, c.k, sm.top);
    }

    if (ctas > 1) {
        cluster_sync();
        if (rank == 0) {
            // the other CTAs' best behind this one's, and all of them on the list
            for (int e = threadIdx.x; kTop && e < ctas * c.k; e += kLogThreads) {
                const int from = e / c.k;
                const Best* b = &sm.top[e % c.k];
                sm.list[e] = Best{__uint_as_float(remote_word(&b->x, from)), (int)remote_word(&b->i, from)};
            }
            if (threadIdx.x == 0) {
                Sums all;
                all.s = all.d = 0.f;
                float to = sm.sum[0];
                for (int q = 1; q < ctas; ++q) to = fmaxf(to, __uint_as_float(remote_word(&sm.sum[0], q)));
                for (int q = 0; q < ctas; ++q) {
                    Sums one;
                    one.ref = __uint_as_float(remote_word(&sm.sum[0], q));
                    one.s = __uint_as_float(remote_word(&sm.sum[1], q));
                    one.d = __uint_as_float(remote_word(&sm.sum[2], q));
                    one.move(to, c2);
                    all.s += one.s;
                    all.d += one.d;
                }
                sm.red[0][0] = to;
                sm.red[1][0] = all.s;
                sm.red[2][0] = all.d;
            }
        }
        cluster_sync();
        if (rank) return;
        if (kTop) {
            rank_list(sm.list, ctas * c.k, c.k, sm.top);
        }
    } else if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) sm.red[i][0] = sm.sum[i];
    }
    __syncthreads();
    m = sm.red[0][0];
    const bool none = m == kNone;
    const float log_sum = none ? 0.f : logf(sm.red[1][0]);
    if (threadIdx.x == 0) {
        if (c.logp) c.logp[r] = asked == kNone ? kNone : (asked - m) * c.scale - log_sum;
        if (c.entropy) c.entropy[r] = none ? 0.f : fmaxf(log_sum - sm.red[2][0] / sm.red[1][0] * 0.6931471805599453f, 0.f);
    }
    if (kTop && (int)threadIdx.x < c.k) {
        const Best b = sm.top[threadIdx.x];
        c.top_ids[r * c.k + threadIdx.x] = b.x > kNone ? b.i : -1;
        c.top_logp[r * c.k + threadIdx.x] = b.x > kNone ? (b.x - m) * c.scale - log_sum : kNone;
    }
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

template <typename L, bool kTop>
cudaError_t launch(const ft_logprob& c, int ctas, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c.n * ctas);
    cfg.blockDim = dim3(kLogThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<L, kTop>, c, ctas);
}

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
    // CTAs of a row: as many as there is room for at two per SM, each with a vector or more per thread
    int ctas = 1;
    const long long vectors = (long long)c.V / (c.dtype == FT_DTYPE_BF16 ? 8 : 4);
    while (ctas < kMaxCtas && 2LL * ctas * c.n <= 2LL * sm_count() && vectors > (long long)ctas * kLogThreads) ctas *= 2;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = c.dtype == FT_DTYPE_BF16 ? (c.k ? launch<__nv_bfloat16, true>(c, ctas, s) : launch<__nv_bfloat16, false>(c, ctas, s))
                                                   : (c.k ? launch<float, true>(c, ctas, s) : launch<float, false>(c, ctas, s));
    return e == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}
