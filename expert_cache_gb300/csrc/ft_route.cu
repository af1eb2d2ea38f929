// Router: logits to the k experts of each token and their weights.  A warp per token.
//
// Up to 512 experts the choices stay in registers.  The (k + 1)-th largest of the lanes' maxima bounds the (k + 1)-th largest choice
// from below; what reaches it, for small k k to some 1.3 k of 256, goes through shared memory and is ranked, each lane one.  With more
// choices the lanes' maxima bound less and less: from some 14 (of scores with a bias) or 16 (of logits) on more than 32 experts reach the bound
// in some rows, at k = 32 in all of them (of scores always: 33 maxima are asked for), and the row goes to the searches below.
// 8192 tokens of 256 experts, by logits: k = 1 6.2 us, 8 6.8, 12 7.4, 16 13.8, 20 23, 24 40, 32 50; sigmoid with a bias: 4 10.5, 8 12.2, 12 13.8, 16 20, 18 48,
// 24 93, 32 115.
//
// Choices are computed in fp32 with a bound on their error.  Where two neighbours of the sorted first k, the k-th and one behind it
// or the last group that stays and the first that does not lie within their bounds, and do not come from the same logit and bias, the
// row is decided again in 64 bits; so the ids are the formula's.  Without a bias, and without sums of a group's choices, the scores' order
// is the logits' own and needs no rounding at all.
//
// Bound by latency and, for many tokens, by instructions (570 a row of 256), not by the 4.7 MB of 8192 tokens of 256 experts
// (0.7 us): those take 6.8 us, one token 2.0 us, 16 with groups and a bias 3.7 us, 5003 of 160 experts with groups and a bias 8.3 us, 12 to 15 us
// where a row among them goes to 64 bits for its choices, and 20 us where one does for its groups: their latency stands alone at the end.
// With that bias (0.05 beside scores of 160) the one is 2 rows in 10,000 and the other 1 in 20,000: of 60 such calls 17, 29 and 14.  k searches of
// a warp through shared memory take 14.2, 4.3, 7.3 and 31 us for those; above 512 experts it is the only form (k = 8: 513 experts 6.1 us for a token and
// 8.0 for 1024, 1024 experts 6.8 and 8.4, 4096 experts 16 and 34; k = 32 of 4096 82 us for 1024).
#include <cfloat>
#include <cmath>
#include <type_traits>

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
    int group_shift;       // 1 << group_shift lanes look at a group
    unsigned group_mul;    // expert e < 512 is of group e * group_mul >> 20
    bool sigmoid, renormalise, by_logit;
    float scale;
};

// A logit as the formula takes it: NaN is -inf, +inf the largest number.
__device__ __forceinline__ float route_logit(float x) { return fminf(fmaxf(x, kNone), FLT_MAX); }
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

// e^y for y <= 0 to some 2^-51, or half of 2^-1074: y = n ln 2 + r with ln 2 in two parts (Cody and Waite 1980), the first of 41 bits, so
// that n times it is exact; Taylor's series to r^13 / 13!, whose rest is below 2^-57 for |r| <= ln 2 / 2.
__device__ __forceinline__ double exp_negative(double y) {
    y = fmax(y, -750.0);                                         // 0, as all below -745.2
    const double n = rint(y * 1.4426950408889634);
    const double r = fma(n, -0x1.3de6af278ece6p-42, fma(n, -0x1.62e42fefa3000p-1, y));
    double p = 1.0 / 6227020800.0;
    constexpr double c[] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320, 1.0 / 362880, 1.0 / 3628800,
                            1.0 / 39916800, 1.0 / 479001600};
#pragma unroll
    for (int i = 12; i >= 0; --i) p = fma(p, r, c[i]);
    const int m = (int)n, h = m / 2;                             // 2^m in two factors: below 2^-1022 there is only the second rounding
    return p * __longlong_as_double((long long)(1023 + h) << 52) * __longlong_as_double((long long)(1023 + m - h) << 52);
}

// 1 / x to some 2^-52 for a normal fp32 range of x: two steps of Newton's from the fp32 reciprocal.
__device__ __forceinline__ double inverse_double(double x) {
    double r = 1.0f / (float)x;
    r = fma(r, fma(-x, r, 1.0), r);
    return fma(r, fma(-x, r, 1.0), r);
}

__device__ __forceinline__ float exp_of(float y) { return expf(y); }
__device__ __forceinline__ double exp_of(double y) { return exp_negative(y); }
__device__ __forceinline__ float inverse(float x) { return __frcp_rn(x); }
__device__ __forceinline__ double inverse(double x) { return inverse_double(x); }

// sigmoid(x), by an exponential that does not grow.
template <typename V>
__device__ __forceinline__ V sigmoid(float x) {
    const V p = exp_of(-V(fabsf(x)));
    return (x >= 0.f ? V(1) : p) * inverse(V(1) + p);
}

// What softmax's scores e^(x - top) / sum are made of.
struct Scores {
    float top, sum;
};

// A bound on the error of an fp32 score: the roundings of the exponential (2^-22) and of its argument (at most -log2 of the
// score in magnitude), those of the sum's terms and its E / 32 + 5 additions, two more operations, what underflows.  It rises with the score.
__device__ __forceinline__ float score_error(const RouteArgs& a, float score) {
    return 0x1p-24f * ((float)(a.E / 32 + 16) - 2.f * __log2f(fmaxf(score, 0x1p-120f))) * score + 0x1p-123f;
}
// Whether two neighbours among the sorted choices may stand the other way round, or one that is sorted further down belong between them:
// any choice may be off by what the row's largest score may (most), and by the bias' addition.
__device__ __forceinline__ bool too_near(const RouteArgs& a, float first, float second, float most) {
    return first - second <= 2.f * score_error(a, most) + 0x1p-22f * (fabsf(first) + fabsf(second));
}

// The choices of a row in type V, the groups that stay, and the k first experts: lane j < k gets the j-th (-1: none).
// Returns false if fp32 does not tell.
template <typename V>
__device__ __forceinline__ bool decide(const RouteArgs& a, const float* x, V* key, Scores& s, int& id) {
    const int lane = threadIdx.x & 31;
    bool sure = true;
    float largest = 1.f;                                         // no score is above it
    if (!a.sigmoid && !(a.by_logit && a.renormalise)) {
        float top = kNone;
        V sum = 0;
        for (int e = lane; e < a.E; e += 32) top = fmaxf(top, x[e]);
        top = warp_max(top);
        if (top == kNone) top = 0.f;
#pragma unroll 1
        for (int e = lane; e < a.E; e += 32) {
            const V p = exp_of(V(x[e]) - V(top));
            sum += p;
            key[e] = p;
        }
        sum = warp_sum(sum);
        s.top = top;
        s.sum = (float)sum;
        const V inv = inverse(sum);
        largest = (float)inv;
        for (int e = lane; e < a.E; e += 32) key[e] *= inv;
    } else if (!a.by_logit) {
#pragma unroll 1
        for (int e = lane; e < a.E; e += 32) key[e] = sigmoid<V>(x[e]);
    }
    for (int e = lane; e < a.E; e += 32) {
        V c = a.by_logit ? V(x[e]) : a.bias ? key[e] + V(a.bias[e]) : key[e];
        if (x[e] == kNone || !(c == c)) c = kNone;
        key[e] = c;
    }
    __syncwarp();
    if (a.n_group > 1) {
        // some lanes for each group: their two largest
        const int g = lane >> a.group_shift, parts = 1 << a.group_shift;
        V one = kNone, two = kNone;
        if (g < a.n_group) {
            for (int i = lane & (parts - 1); i < a.size; i += parts) {
                const V c = key[g * a.size + i];
                two = fmax(two, fmin(one, c));
                one = fmax(one, c);
            }
        }
        for (int o = 1; o < parts; o <<= 1) {
            const V c = __shfl_xor_sync(0xffffffffu, one, o), d = __shfl_xor_sync(0xffffffffu, two, o);
            two = fmax(fmax(two, d), fmin(one, c));
            one = fmax(one, c);
        }
        const V worth = a.group_best == 2 && two > V(kNone) ? one + two : one;
        float err = 0.f;
        if (!a.by_logit && sizeof(V) == 4 && one > V(kNone)) {
            // the magnitudes of a sum's terms bound its own rounding
            err = score_error(a, largest) * a.group_best + 0x1p-22f * (fabsf((float)one) + (two > V(kNone) ? fabsf((float)two) : 0.f));
        }
        int before = 0;
        for (int i = 0; i < a.n_group; ++i) {
            const V other = __shfl_sync(0xffffffffu, worth, i << a.group_shift);
            before += other > worth || (other == worth && i < g);
        }
        const bool stays = g < a.n_group && before < a.topk_group;
        if (sizeof(V) == 4 && !a.by_logit) {
            // worth - err of those that stay against worth + err of those that do not; sums past fp32's range have no order
            const float least = -warp_max(stays && worth > V(kNone) ? err - (float)worth : kNone);
            const float most = warp_max(!stays && g < a.n_group && worth > V(kNone) ? (float)worth + err : kNone);
            if ((!(least > most) && most > kNone) || __any_sync(0xffffffffu, one > V(kNone) && isinf((float)worth))) sure = false;
        }
        if (g < a.n_group && !stays)
            for (int i = lane & (parts - 1); i < a.size; i += parts) key[g * a.size + i] = kNone;
        __syncwarp();
    }
    id = -1;
    V last = 0;
    int last_id = -1;
    for (int j = 0; j < a.k; ++j) {
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
            if (!(x[last_id] == x[at] && b0 == b1) && too_near(a, last, best, largest)) sure = false;
        }
        if (lane == j) id = at;
        last = best;
        last_id = at;
        if (lane == (at & 31)) key[at] = kNone;
        __syncwarp();
    }
    if (sizeof(V) == 4 && !a.by_logit && last_id >= 0) {
        // none of the others may belong before the last: not the next one alone, which may be equal to it
        const float x0 = x[last_id], b0 = a.bias ? a.bias[last_id] : 0.f;
        bool near = false;
        for (int e = lane; e < a.E; e += 32)
            near |= key[e] > V(kNone) && !(x[e] == x0 && (a.bias ? a.bias[e] : 0.f) == b0) && too_near(a, last, key[e], largest);
        if (__any_sync(0xffffffffu, near)) sure = false;
    }
    return sure;
}

// The weights of a row's experts: lane j has the j-th, its logit `mine` (-inf: none).  Renormalised ones against the largest
// selected, so that they do not underflow together.
__device__ __forceinline__ float weight(const RouteArgs& a, float mine, const Scores& s) {
    const bool some = mine > kNone;
    float w = 0.f;
    if (a.renormalise) {
        float top = warp_max(mine);
        if (a.sigmoid) {
            // sigmoid(x) = e^min(x,0) / (1 + e^-|x|)
            top = fminf(top, 0.f);
            if (some) w = expf(fminf(mine, 0.f) - top) * __frcp_rn(1.f + expf(-fabsf(mine)));
        } else if (some) {
            w = expf(mine - top);
        }
        const float sum = warp_sum(w);
        if (some) w *= __frcp_rn(sum);
    } else if (some) {
        w = a.sigmoid ? sigmoid<float>(mine) : expf(mine - s.top) * __frcp_rn(s.sum);
    }
    return w * a.scale;
}

// A row whose logits stand in shared memory (x, E values; key, E values of 64 bits).  sure: whether fp32 may still tell.
__device__ __noinline__ void route_row(const RouteArgs& a, float* x, double* key, bool sure, long long t) {
    const int lane = threadIdx.x & 31;
    Scores s{0.f, 1.f};
    int id;
    if (!sure || !decide(a, x, reinterpret_cast<float*>(key), s, id)) {
        __syncwarp();
        decide(a, x, key, s, id);
    }
    const float w = weight(a, id >= 0 ? x[id] : kNone, s);
    if (lane < a.k) {
        a.ids[t * a.k + lane] = id;
        a.w[t * a.k + lane] = w;
    }
}

// More than 512 experts.
template <typename L>
__global__ void __launch_bounds__(kRouteWarps * 32) route_wide_kernel(const RouteArgs a) {
    extern __shared__ double route_smem[];
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long t = (long long)blockIdx.x * (blockDim.x >> 5) + warp;
    if (t >= a.T) return;
    float* x = reinterpret_cast<float*>(route_smem + (size_t)(blockDim.x >> 5) * a.E) + (size_t)warp * a.E;
    const L* row = static_cast<const L*>(a.logits) + t * a.stride;
    for (int e = lane; e < a.E; e += 32) x[e] = load_logit(row + e);
    __syncwarp();
    route_row(a, x, route_smem + (size_t)warp * a.E, true, t);
}

__device__ __forceinline__ unsigned ordered(float x) {
    const unsigned u = __float_as_uint(x);
    return u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(unsigned u) { return __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xFFFFFFFFu)); }
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// kEach logits of a lane, in runs of kRun neighbours; element i of a lane is expert index(i).  Runs of two: of the experts of a group,
// or of neighbours that come out on top together, hardly two are a lane's, and its maximum bounds little else (runs of eight, one
// load each: 3 of 8 groups left 8 lanes and often more than 32 experts to rank, 16 us instead of 9 us for 5003 tokens of 160).
template <int kEach>
struct Held {
    static constexpr int kRun = kEach < 2 ? kEach : 2;
    static __device__ __forceinline__ int index(int i) { return (i / kRun * 32 + (int)(threadIdx.x & 31)) * kRun + i % kRun; }
};

// A warp's logits (-inf past the last expert).  Runs are loaded at once where they are aligned.
template <typename L, int kEach>
__device__ __forceinline__ void load_row(float (&x)[kEach], const L* row, int E) {
    constexpr int kRun = Held<kEach>::kRun, kBytes = kRun * (int)sizeof(L);
    typedef typename std::conditional<kBytes == 8, uint2, typename std::conditional<kBytes == 4, uint32_t, uint16_t>::type>::type Word;
    const bool whole = ((uintptr_t)row & (sizeof(Word) - 1)) == 0 && E % kRun == 0;
    if (whole) {
        Word v[kEach / kRun];                                      // all of them under way at once
#pragma unroll
        for (int r = 0; r < kEach / kRun; ++r) v[r] = *reinterpret_cast<const Word*>(row + min(Held<kEach>::index(r * kRun), E - kRun));
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            x[i] = Held<kEach>::index(i) < E ? load_logit(reinterpret_cast<const L*>(&v[i / kRun]) + i % kRun) : kNone;
    } else {
        L v[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) v[i] = row[min(Held<kEach>::index(i), E - 1)];
#pragma unroll
        for (int i = 0; i < kEach; ++i) x[i] = Held<kEach>::index(i) < E ? load_logit(&v[i]) : kNone;
    }
}

// A choice and its expert as a number whose order is theirs: the larger choice first, then the lower index.  0 stands for none.
typedef unsigned long long Key;
__device__ __forceinline__ Key key_of(float choice, int e) { return (Key)ordered(choice + 0.f) << 32 | ~(unsigned)e; }
__device__ __forceinline__ float key_choice(Key k) { return k ? unordered((unsigned)(k >> 32)) : kNone; }
__device__ __forceinline__ int key_expert(Key k) { return k ? (int)~(unsigned)k : -1; }

// What a warp keeps in shared memory for a row: the choices of one with groups, or the logits and 64-bit choices of one that
// is decided again; what is ranked, unsorted and sorted.
struct Ranked {
    Key key[64];
    float x[64];
};
__host__ __device__ inline size_t route_bytes(int E) { return (((size_t)E * 12 + 15) & ~(size_t)15) + sizeof(Ranked); }

// Ranks the n choices of the lanes (logit mine, expert e) in 64 bits; returns the lane's logit and expert (as its bits).  Little
// code, rolled: it is fetched while the row's warp waits (a few KB of it took 6 us).
__device__ __noinline__ float2 rank_again(const RouteArgs& a, const float* x, float top, float mine, int e, int n) {
    const int lane = threadIdx.x & 31;
    double sum = 0;
    if (!a.sigmoid) {
#pragma unroll 1
        for (int i = lane; i < a.E; i += 32) sum += exp_negative((double)x[i] - top);
        sum = warp_sum(sum);
    }
    double choice = kNone;
    if (lane < n) {
        const double p = exp_negative(a.sigmoid ? -fabs((double)mine) : (double)mine - top);
        choice = (a.sigmoid && mine >= 0.f ? 1.0 : p) * inverse_double(a.sigmoid ? 1.0 + p : sum);
        if (a.bias) choice += (double)a.bias[e];
    }
    int rank = lane < n ? 0 : lane;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const double c = __shfl_sync(0xffffffffu, choice, i);
        const int of = __shfl_sync(0xffffffffu, e, i);
        if (lane < n) rank += c > choice || (c == choice && of < e);
    }
    // to the lane of its rank
    float2 out = make_float2(kNone, __int_as_float(-1));
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const int to = __shfl_sync(0xffffffffu, rank, i);
        const float y = __shfl_sync(0xffffffffu, mine, i);
        const int of = __shfl_sync(0xffffffffu, e, i);
        if (lane == to) out = make_float2(y, __int_as_float(of));
    }
    return out;
}

// A row's k experts and their logits; lane j gets the j-th (expert -1: none).
enum Picked { kDone, kUnsure, kMany };       // kUnsure: fp32 does not tell the groups; kMany: a lane each is not enough for the ranking
template <int kEach, bool kByLogit>
__device__ __forceinline__ Picked pick(const RouteArgs& a, const float (&x)[kEach], uint8_t* mem, Scores& s, float& logit, int& expert) {
    const int lane = threadIdx.x & 31;
    Ranked& ranked = *reinterpret_cast<Ranked*>(mem + route_bytes(a.E) - sizeof(Ranked));
    float key[kEach];

    // the choices
    float inv = 1.f;
    if (kByLogit ? !a.renormalise && !a.sigmoid : !a.sigmoid) {
        float top = x[0], sum = 0.f;
#pragma unroll
        for (int i = 1; i < kEach; ++i) top = fmaxf(top, x[i]);
        top = warp_max(top);
        if (top == kNone) top = 0.f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            key[i] = exp2_fast((x[i] - top) * 1.4426950408889634f);
            sum += key[i];
        }
        s.top = top;
        s.sum = warp_sum(sum);
        inv = __frcp_rn(s.sum);
    }
    if (kByLogit) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) key[i] = x[i];
    } else {
#pragma unroll
        for (int i = 0; i < kEach; ++i) key[i] = a.sigmoid ? __frcp_rn(1.f + exp2_fast(x[i] * -1.4426950408889634f)) : key[i] * inv;
        if (a.bias) {
            float bias[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i) bias[i] = a.bias[min(Held<kEach>::index(i), a.E - 1)];
#pragma unroll
            for (int i = 0; i < kEach; ++i) key[i] += bias[i];
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) key[i] = x[i] > kNone && key[i] == key[i] ? key[i] : kNone;
    }

    const float largest = a.sigmoid ? 1.f : inv;                   // no score is above it
    // the groups that stay: some lanes for each group, their two largest choices
    if (a.n_group > 1) {
        float* flat = reinterpret_cast<float*>(mem);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (Held<kEach>::index(i) < a.E) flat[Held<kEach>::index(i)] = key[i];
        __syncwarp();
        const int g = lane >> a.group_shift, parts = 1 << a.group_shift;
        float one = kNone, two = kNone;
        if (g < a.n_group) {
            for (int i = lane & (parts - 1); i < a.size; i += parts) {
                const float c = flat[g * a.size + i];
                two = fmaxf(two, fminf(one, c));
                one = fmaxf(one, c);
            }
        }
        for (int o = 1; o < parts; o <<= 1) {
            const float c = __shfl_xor_sync(0xffffffffu, one, o), d = __shfl_xor_sync(0xffffffffu, two, o);
            two = fmaxf(fmaxf(two, d), fminf(one, c));
            one = fmaxf(one, c);
        }
        const float worth = a.group_best == 2 && two > kNone ? one + two : one;
        int before = 0;
        for (int i = 0; i < a.n_group; ++i) {
            const float other = __shfl_sync(0xffffffffu, worth, i << a.group_shift);
            before += other > worth || (other == worth && i < g);
        }
        const bool stays = g < a.n_group && before < a.topk_group;
        const unsigned kept = __ballot_sync(0xffffffffu, stays);
        if (!kByLogit) {
            // the magnitudes of a sum's terms bound its own rounding; past fp32's range they have no order
            const float err = score_error(a, largest) * a.group_best + 0x1p-22f * ((one > kNone ? fabsf(one) : 0.f) + (two > kNone ? fabsf(two) : 0.f));
            const float least = -warp_max(stays && worth > kNone ? err - worth : kNone);
            const float most = warp_max(!stays && g < a.n_group && worth > kNone ? worth + err : kNone);
            if ((!(least > most) && most > kNone) || __any_sync(0xffffffffu, one > kNone && isinf(worth))) return kUnsure;
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int of = (int)(((unsigned)Held<kEach>::index(i) * a.group_mul) >> 20);
            if (of >= a.n_group || !(kept >> (of << a.group_shift) & 1)) key[i] = kNone;
        }
        __syncwarp();
    }

    // the bound: of the lanes' maxima, largest first, the (k + 1)-th; by logits the k-th is enough
    float most = key[0];
#pragma unroll
    for (int i = 1; i < kEach; ++i) most = fmaxf(most, key[i]);
    unsigned left = ordered(most), bound = ordered(kNone);
    for (int n = 0; n < a.k + (kByLogit ? 0 : 1);) {
        bound = __reduce_max_sync(0xffffffffu, left);
        if (bound <= ordered(kNone)) break;
        const bool is = left == bound;
        n += __popc(__ballot_sync(0xffffffffu, is));
        if (is) left = 0;
    }
    float least = bound <= ordered(kNone) ? -FLT_MAX : unordered(bound);
    if (!kByLogit) least = fmaxf(least - 2.f * (2.f * score_error(a, largest) + 0x1p-21f * fabsf(least)), -FLT_MAX);      // nothing that may be a (k + 1)-th is left out
    int n = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const bool in = key[i] >= least;
        const unsigned who = __ballot_sync(0xffffffffu, in);
        const int at = n + __popc(who & ((1u << lane) - 1));
        if (in && at < 32) {
            ranked.key[at] = key_of(key[i], Held<kEach>::index(i));
            if (!kByLogit) ranked.x[at] = x[i];
        }
        n += __popc(who);
    }
    if (n > 32) return kMany;           // too few maxima to bound the (k + 1)-th choice, or many equal ones
    __syncwarp();
    Key mine = 0;
    int rank = lane;
    if (lane < n) {
        mine = ranked.key[lane];
        rank = 0;
        for (int i = 0; i < n; ++i) rank += ranked.key[i] > mine;
    }
    ranked.key[32 + rank] = mine;                                  // those without one behind
    if (!kByLogit) ranked.x[32 + rank] = lane < n ? ranked.x[lane] : kNone;
    __syncwarp();
    mine = ranked.key[32 + lane];
    expert = key_expert(mine);
    logit = kByLogit ? key_choice(mine) : ranked.x[32 + lane];
    if (!kByLogit) {
        // each of the first k against the one before it, the others against the k-th (the next one may be equal to it)
        const int before = lane < a.k ? max(lane - 1, 0) : a.k - 1;
        const float key1 = key_choice(mine), key0 = __shfl_sync(0xffffffffu, key1, before), x0 = __shfl_sync(0xffffffffu, logit, before);
        const int e0 = __shfl_sync(0xffffffffu, expert, before);
        bool near = false;
        if (lane > 0 && expert >= 0) {
            const float b0 = a.bias ? a.bias[e0] : 0.f, b1 = a.bias ? a.bias[expert] : 0.f;
            near = !(x0 == logit && b0 == b1) && too_near(a, key0, key1, largest);
        }
        if (__any_sync(0xffffffffu, near)) {
            // the row's logits, for the sum in 64 bits
            float* again = reinterpret_cast<float*>(mem + (size_t)a.E * 8);
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (Held<kEach>::index(i) < a.E) again[Held<kEach>::index(i)] = x[i];
            __syncwarp();
            const float2 m = rank_again(a, again, s.top, logit, expert, n);
            logit = m.x;
            expert = __float_as_int(m.y);
        }
    }
    return kDone;
}

template <typename L, int kEach, bool kByLogit>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteArgs a) {
    extern __shared__ __align__(16) uint8_t route_mem[];
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long t = (long long)blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    uint8_t* mem = route_mem + warp * route_bytes(a.E);
    float x[kEach];
    load_row<L, kEach>(x, static_cast<const L*>(a.logits) + t * a.stride, a.E);
    Scores s{0.f, 1.f};
    float logit;
    int expert;
    const Picked p = pick<kEach, kByLogit>(a, x, mem, s, logit, expert);
    if (p == kDone) {
        const bool some = lane < a.k && expert >= 0;
        const float w = weight(a, some ? logit : kNone, s);
        if (lane < a.k) {
            a.ids[t * a.k + lane] = some ? expert : -1;
            a.w[t * a.k + lane] = w;
        }
        return;
    }
    float* again = reinterpret_cast<float*>(mem + (size_t)a.E * 8);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (Held<kEach>::index(i) < a.E) again[Held<kEach>::index(i)] = x[i];
    __syncwarp();
    route_row(a, again, reinterpret_cast<double*>(mem), p == kMany, t);
}

template <typename L, int kEach, bool kByLogit>
cudaError_t launch(const RouteArgs& a, cudaStream_t s) {
    return launch_pdl(route_kernel<L, kEach, kByLogit>, dim3((unsigned)((a.T + (long long)kRouteWarps - 1) / kRouteWarps)), dim3(kRouteWarps * 32),
                      kRouteWarps * route_bytes(a.E), s, a);
}

// Lanes hold as few logits as E takes.
template <typename L, bool kByLogit>
cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
    if (a.E <= 32) return launch<L, 1, kByLogit>(a, s);
    if (a.E <= 64) return launch<L, 2, kByLogit>(a, s);
    if (a.E <= 128) return launch<L, 4, kByLogit>(a, s);
    if (a.E <= 256) return launch<L, 8, kByLogit>(a, s);
    if (a.E <= 512) return launch<L, 16, kByLogit>(a, s);
    const int warps = a.E > 1024 ? 1 : kRouteWarps;
    return launch_pdl(route_wide_kernel<L>, dim3((unsigned)((a.T + (long long)warps - 1) / warps)), dim3(warps * 32), (size_t)warps * a.E * 12, s, a);
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
    a.group_shift = 0;
    while (c.n_group << (a.group_shift + 1) <= 32) ++a.group_shift;
    a.group_mul = ((1u << 20) + a.size - 1) / a.size;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = c.dtype == FT_DTYPE_BF16 ? (a.by_logit ? launch_route<__nv_bfloat16, true>(a, s) : launch_route<__nv_bfloat16, false>(a, s))
                                                   : (a.by_logit ? launch_route<float, true>(a, s) : launch_route<float, false>(a, s));
    return e == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}
