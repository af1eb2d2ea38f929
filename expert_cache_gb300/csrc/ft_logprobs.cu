// Log probabilities of given tokens, entropy and the most likely tokens of rows of logits.
//
// One pass over a row, by a cluster of 1 to 8 CTAs: with y = scale (x - ref) per thread the sums S = sum e^y and D = sum e^y y
// give log sum = log S and entropy = log S - D / S.  A thread's ref is a maximum of a sample of the row, so that no
// sum has to be rescaled unless a logit lies e^44 above it; the row's own maximum is taken at the end.
//
// The k largest come out of the same pass.  From the sample (the first 8 vectors of every thread) the k-th largest of some 2 k
// logits is a lower bound of the row's k-th; only what reaches it is kept and put on a list in shared memory (4 to 8 k of
// 100,000), which is ranked at the end.  Where more reach it than the list holds, its own k-th largest is the next bound and
// the part is read again; where that does not help (equal logits by the thousand, rising ones), k searches find them.  Which ones
// these are does not depend on any order: value, then index.
//
// 2048 rows of 131,072 bf16: 89.1 us, 6.03 TB/s, 0.90 of the copy rate; without the k largest 80.5 us, the copy rate.  The k
// largest cost the barriers of the sample and of the list, during which an SM has only its other CTAs' loads under way.  (fp32: 156 us,
// of 65,536 82 us.)  Two kinds of rows are slow: where the scale times the logits passes 2^26 every vector goes out of line (see Sums), 575 us; and
// where a CTA's part has fewer than k logits above thousands of equal ones it is read again and again: rows of the type's lowest value but
// for their first 3 take 2.2 ms for k = 5 and 7.2 ms for k = 32, a row whose second half is masked so 88 and 165 us instead of 5.3.  One
// row: 5.3 us in 8 CTAs, launch and barriers.  On the way: vectors through registers, 4 or 8 under way, 151 to 193 us; through
// thread-owned shared memory 114 us; neighbouring vectors instead of four stretches of the row 103 us; the list by warps instead of at
// once 101 us; ranks by several threads per entry (one row 7.3 -> 5.5 us), of few warps 95 us; three CTAs of 384 threads an SM
// instead of two of 512 (see launch) 89 us.  Rows in a loop with the next one's first vectors loaded ahead (127 us instead of 101),
// and the bound worked out by every warp for itself (107 us) were slower.
#include <atomic>
#include <cfloat>
#include <cmath>

#include "ft_internal.cuh"
#include "ft_pair.cuh"

namespace ft {

namespace {

constexpr int kVectors = 4;            // vectors of a thread in a round
constexpr int kRounds = 2;             // rounds under way
constexpr int kListed = 1024;          // entries of a CTA's list
constexpr int kMaxCtas = 8;            // of a row
constexpr float kNone = -INFINITY;
// How far, in powers of 2, a logit may lie above a thread's reference.  2^y loses 22 roundings of 2^-24 to y's own just below 64 (45 at
// 100, where the sums would still be numbers, and 1 at 2; but every step up costs a call: 2048 rows of 131,072 at a scale of 20 take
// 90.0, 91.6 and 94.2 us with 100, 64 and 40, rising ones 132, 167 and 230).
constexpr float kFar = 64.f;

// What follows from the number of a CTA's threads.
template <int T>
struct Cta {
    static constexpr int kWarps = T / 32, kPerSm = 1152 / T;
    static constexpr int kSlot = T * 16, kRing = kRounds * kVectors * kSlot;
    static constexpr int kHits = T == 384 ? 48 : 64;           // vectors that a warp keeps for the list
};

// 16 bytes of logits.  Max: the largest so far, NaN aside, in the form that costs least; Floor: where logits are cut off.
template <typename L>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    typedef __nv_bfloat162 Max;
    uint32_t w[4];
    __device__ __forceinline__ void none() {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = 0xFF80FF80u;
    }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
    }
    __device__ __forceinline__ void from_shared(uint32_t a) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
    }
    __device__ __forceinline__ void to_shared(uint32_t a) const {
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(a), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]));
    }
    __device__ __forceinline__ void first(const __nv_bfloat16* p) { w[0] = (w[0] & 0xFFFF0000u) | *reinterpret_cast<const uint16_t*>(p); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[2 * j] = __uint_as_float(w[j] << 16), x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
    __device__ __forceinline__ __nv_bfloat162 at(int j) const { return *reinterpret_cast<const __nv_bfloat162*>(&w[j]); }
    __device__ __forceinline__ Max max() const { return __hmax2(__hmax2(at(0), at(1)), __hmax2(at(2), at(3))); }
    static __device__ __forceinline__ Max larger(Max a, Max b) { return __hmax2(a, b); }
    static __device__ __forceinline__ float value(Max m) {
        const float2 f = __bfloat1622float2(m);
        return fmaxf(f.x, f.y);
    }
    // x rounded down, twice
    static __device__ __forceinline__ Max limit(float x) { return __bfloat162bfloat162(__float2bfloat16_rd(x)); }
    static __device__ __forceinline__ bool reaches(Max m, Max limit) { return !__hblt2(m, limit); }
    __device__ __forceinline__ Pair get(int j, Max floor) const {
        const __nv_bfloat162 h = __hmax2(at(j), floor);
        const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
        return pair(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    }
};
template <>
struct Vec<float> {
    static constexpr int kN = 4;
    typedef float Max;
    float w[4];
    __device__ __forceinline__ void none() {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = kNone;
    }
    __device__ __forceinline__ void load(const float* p) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3]) : "l"(p));
    }
    __device__ __forceinline__ void from_shared(uint32_t a) {
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3]) : "r"(a));
    }
    __device__ __forceinline__ void to_shared(uint32_t a) const {
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" :: "r"(a), "f"(w[0]), "f"(w[1]), "f"(w[2]), "f"(w[3]));
    }
    __device__ __forceinline__ void first(const float* p) { w[0] = *p; }
    __device__ __forceinline__ void get(float (&x)[4]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = w[j];
    }
    __device__ __forceinline__ Max max() const { return fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])); }
    static __device__ __forceinline__ Max larger(Max a, Max b) { return fmaxf(a, b); }
    static __device__ __forceinline__ float value(Max m) { return m; }
    static __device__ __forceinline__ Max limit(float x) { return x; }
    static __device__ __forceinline__ bool reaches(Max m, Max limit) { return !(m < limit); }
    __device__ __forceinline__ Pair get(int j, Max floor) const { return pair(fmaxf(w[2 * j], floor), fmaxf(w[2 * j + 1], floor)); }
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float inverse_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Unsigned words in the order of the floats.
__device__ __forceinline__ unsigned ordered(float x) {
    const unsigned u = __float_as_uint(x);
    return u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(unsigned u) { return __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xFFFFFFFFu)); }

// A logit and its index as a number whose order is theirs: the larger logit first (NaN aside, +inf as the largest number, both
// zeros equal), then the lower index.  Numbers below 2^32 stand for none.
typedef unsigned long long Key;
__device__ __forceinline__ Key key_of(float x, int i) { return (Key)ordered(fminf(x, FLT_MAX) + 0.f) << 32 | ~(unsigned)i; }
__device__ __forceinline__ float key_logit(Key k) { return k >> 32 ? unordered((unsigned)(k >> 32)) : kNone; }
__device__ __forceinline__ int key_index(Key k) { return k >> 32 ? (int)~(unsigned)k : -1; }

template <int T>
struct LogShared {
    static constexpr int kWarps = Cta<T>::kWarps, kHits = Cta<T>::kHits;
    alignas(16) Key list[kListed];
    alignas(16) Key top[kMaxK];                   // this CTA's k best
    alignas(16) Key tops[kMaxCtas * kMaxK];       // the row's CTAs' (in its first one)
    alignas(16) uint4 hit[kWarps][kHits];      // the warps' vectors that reach the bound, and where they stand
    int hit_at[kWarps][kHits];
    float few[2 * kMaxK + kWarps];                // the sample's largest
    float red[3][kWarps];                         // the warps' largest, S and D
    float sums[kMaxCtas][4];                      // the row's CTAs' largest, S and D (in its first one)
    Key one;
    int count;
    float bound, ref;
};

// (a - b) c + d, for c > 0.  Below `halved` the difference is taken in halves: it may pass fp32's range where its product does not
// (or, at the default, where that is not so far out that its power of 2 is 0).
__device__ __forceinline__ float apart(float a, float b, float c, float d, float halved = 1e-36f) {
    float x = a - b;
    if (c < halved) x = 0.5f * a - 0.5f * b, c *= 2.f;
    return fmaf(x, c, d);
}

// A word to the same place in the shared memory of the cluster's first CTA.
__device__ __forceinline__ void store_first(const void* p, uint32_t v) {
    const uint32_t a = (uint32_t)__cvta_generic_to_shared(p);
    asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\tst.shared::cluster.b32 [r], %1;\n\t}" :: "r"(a), "r"(v) : "memory");
}

// A thread's sums against its ref, in units of log 2: with y = c x - rc, rc = RN(c ref), S = sum 2^y and D = sum 2^y y.  What
// rc's rounding moves them by is taken back at the end: below 2^26 it is at most 2, so that S keeps its bits and D two fewer (from 2^31 on
// 2^y could be infinite, or 0 for every logit).  Logits below floor, whose 2^y is 0, are raised to it, so that y is a
// number; those from limit on go out of line, as do all where c ref, the floor or far would be too large (plain: x is cut to the
// largest number and x - ref comes first).  Since far is a smaller number than the largest elsewhere, an infinity always lies above it.
template <typename L>
struct Sums {
    typedef typename Vec<L>::Max Max;
    float ref, far, rc;                // far: a logit above it needs another ref
    bool plain;
    Max floor, limit;
    float top;                         // the largest seen: the sample's, or one that reached the limit
    Pair s, d;

    // span: some 100 / c, 0 or infinite where that is no normal number.
    __device__ __forceinline__ void against(float to, float bound, float c, float span) {
        ref = to;
        // rounded down: next to a large ref one step may be worth more than the span
        far = to == kNone ? kNone : __fadd_rd(to, kFar / 100.f * span);
        plain = !(fabsf(to) * c < 0x1p26f && span > 0.f && to - 2.f * span > -1e38f && far < FLT_MAX);
        rc = plain ? 0.f : to * c;
        floor = Vec<L>::limit(to - 2.f * span);
        limit = Vec<L>::limit(plain ? kNone : fminf(bound, far));
    }
    __device__ __forceinline__ void add(const Vec<L>& v, float c) {
        const Pair c2 = pair(c, c), r2 = pair(-rc, -rc);
#pragma unroll
        for (int j = 0; j < Vec<L>::kN / 2; ++j) {
            const Pair y = fma2(v.get(j, floor), c2, r2);
            const float2 f = halves(y);
            const Pair e = pair(exp2_fast(f.x), exp2_fast(f.y));
            s = add2(s, e);
            d = fma2(e, y, d);
        }
    }
    // Both sums against `to` exactly.
    __device__ __forceinline__ float2 moved(float to, float c) const {
        const float2 a = halves(s), b = halves(d);
        const float sum = a.x + a.y, dot = b.x + b.y;
        if (!(sum > 0.f)) return make_float2(0.f, 0.f);
        // (otherwise the very number that y was for such a logit, so that its rounding cancels)
        const float y = fmaxf(plain ? apart(ref, to, c, 0.f) : fmaf(-to, c, rc), -1e30f), f = exp2_fast(y);
        return make_float2(f * sum, f > 0.f ? f * fmaf(y, sum, dot) : 0.f);
    }
};

// A vector with a logit far above a thread's ref, or of a thread whose ref is too large (out of line, by value: rare, and
// the sums stay in registers).
template <typename L>
__device__ __noinline__ Sums<L> add_far(Sums<L> a, Vec<L> v, float bound, float c) {
    float most = Vec<L>::value(v.max());
    most = most == most ? fminf(most, FLT_MAX) : kNone;
    if (most > a.far || apart(most, a.ref, c, 0.f) > kFar) {          // far is no bound where it is infinite
        const float2 m = a.moved(most, c);
        a.against(most, bound, c, 100.f * inverse_fast(c));
        const float off = a.plain ? 0.f : fmaf(a.ref, c, -a.rc), f = exp2_fast(off);
        a.s = pair(f * m.x, 0.f);
        a.d = pair(f * fmaf(off, m.x, m.y), 0.f);
    }
    if (!a.plain) {
        a.add(v, c);
        return a;
    }
    float x[Vec<L>::kN];
    v.get(x);
    float2 s = halves(a.s), d = halves(a.d);
#pragma unroll
    for (int j = 0; j < Vec<L>::kN; ++j) {
        const float y = x[j] == x[j] ? fmaxf(apart(fminf(x[j], FLT_MAX), a.ref, c, 0.f), -200.f) : -200.f, e = exp2_fast(y);
        s.x += e;
        d.x = fmaf(e, y, d.x);
    }
    a.s = pair(s.x, s.y);
    a.d = pair(d.x, d.y);
    return a;
}

// Puts what reaches the bound on the list.
template <typename L, int T>
__device__ __forceinline__ void put_on_list(LogShared<T>& sm, const Vec<L>& v, int index, float bound) {
    float x[Vec<L>::kN];
    v.get(x);
#pragma unroll
    for (int j = 0; j < Vec<L>::kN; ++j) {
        if (x[j] >= bound && x[j] > kNone) {
            const int at = atomicAdd(&sm.count, 1);
            if (at < kListed) sm.list[at] = key_of(x[j], index + j);
        }
    }
}

// Adds N vectors to a thread's sums; a whole warp calls it.  Vectors for the list are kept (hits of them so far) and looked
// at when the warp is through: the atomic operations of the list at once cost a row of 131,072 logits a microsecond more.
// index(j): where vector j stands.
template <typename L, bool kTop, int T, int N, typename I>
__device__ __forceinline__ void take(LogShared<T>& sm, Sums<L>& a, int& hits, const Vec<L> (&v)[N], I index, float bound, float c) {
    typename Vec<L>::Max reach = v[0].max();
#pragma unroll
    for (int j = 1; j < N; ++j) reach = Vec<L>::larger(reach, v[j].max());
    if (__any_sync(0xffffffffu, Vec<L>::reaches(reach, a.limit))) {
        float top = Vec<L>::value(reach);
        top = top == top ? fminf(top, FLT_MAX) : kNone;
        a.top = fmaxf(a.top, top);
        if (kTop) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float most = Vec<L>::value(v[j].max());
                const bool keep = most >= bound && most > kNone;
                const unsigned kept = __ballot_sync(0xffffffffu, keep);
                if (!kept) continue;
                const int at = hits + __popc(kept & ((1u << (threadIdx.x & 31)) - 1));
                if (keep && at < Cta<T>::kHits) {
                    v[j].to_shared((uint32_t)__cvta_generic_to_shared(&sm.hit[threadIdx.x >> 5][at]));
                    sm.hit_at[threadIdx.x >> 5][at] = index(j);
                }
                hits += __popc(kept);
            }
        }
        if (a.plain || top > a.far) {
#pragma unroll
            for (int j = 0; j < N; ++j) a = add_far(a, v[j], bound, c);
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) a.add(v[j], c);
}

// A CTA's part of a row: the row's vectors from lo on, `steps` for every thread and one more for the first `more`; for the
// row's first CTA also the elements before and behind its vectors.
template <typename L, int T>
struct Part {
    const L* row;
    int head, lo, steps, more, V, rest;
    __device__ __forceinline__ Part(const L* r, int V_, int rank, int shift) : row(r), V(V_) {       // of 1 << shift CTAs
        constexpr int kN = Vec<L>::kN;
        head = min((int)((16 - ((uintptr_t)row & 15)) & 15) / (int)sizeof(L), V);
        const int n = (V - head) / kN;
        lo = (int)((unsigned)n * rank >> shift);                    // n is at most 2^28
        const int own = (int)((unsigned)n * (rank + 1) >> shift) - lo;
        steps = own / T;
        more = own % T;
        rest = rank == 0 ? V - n * kN : 0;
    }
    __device__ __forceinline__ int index(int it) const { return head + (lo + it * T + (int)threadIdx.x) * Vec<L>::kN; }
    __device__ __forceinline__ void load(Vec<L>& v, int it) const { v.load(row + index(it)); }
    // Those that not every thread has (no logits for the others).
    __device__ __forceinline__ void load_more(Vec<L>& v) const {
        v.none();
        if ((int)threadIdx.x < more) load(v, steps);
    }
    __device__ __forceinline__ int rest_index() const { return (int)threadIdx.x < head ? threadIdx.x : V - rest + threadIdx.x; }
    __device__ __forceinline__ void load_rest(Vec<L>& v) const {
        v.none();
        if ((int)threadIdx.x < rest) v.first(row + rest_index());
    }
    // f(vector, index of its first logit) for everything.
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        Vec<L> v;
        for (int it = 0; it < steps; ++it) {
            load(v, it);
            f(v, index(it));
        }
        load_more(v);
        f(v, index(steps));
        load_rest(v);
        f(v, rest_index());
    }
};

// A thread's vectors on their way through its own slots of shared memory, kRounds rounds of kVectors; the last round may
// have fewer.  Nobody else reads a thread's slots, so its own wait for its copies is all there is to wait for.
template <typename L, int T>
struct Ring {
    static constexpr int kSlot = Cta<T>::kSlot;
    const Part<L, T>& p;
    uint32_t slots;
    int full, rounds;
    __device__ __forceinline__ Ring(const Part<L, T>& part, const void* smem) : p(part) {
        slots = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
        full = p.steps / kVectors;
        rounds = full + (p.steps % kVectors || p.more ? 1 : 0);
    }
    __device__ __forceinline__ void issue(int round, uint32_t at) const {
        if (round < full) {
            const L* from = p.row + p.index(round * kVectors);
#pragma unroll
            for (int j = 0; j < kVectors; ++j)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(slots + at + j * kSlot), "l"(from + j * T * Vec<L>::kN) : "memory");
        } else if (round < rounds) {
#pragma unroll
            for (int j = 0; j < kVectors; ++j) {
                const int it = round * kVectors + j;
                if (it < p.steps || (it == p.steps && (int)threadIdx.x < p.more)) {
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(slots + at + j * kSlot), "l"(p.row + p.index(it)) : "memory");
                } else {
                    Vec<L> v;
                    v.none();
                    v.to_shared(slots + at + j * kSlot);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void start() const {
#pragma unroll
        for (int i = 0; i < kRounds; ++i) issue(i, i * kVectors * kSlot);
    }
    // Round i's copies are there once only those of the kRounds - 1 issued behind it are not.
    __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" :: "n"(kRounds - 1) : "memory"); }
    __device__ __forceinline__ Vec<L> get(uint32_t at, int j) const {
        Vec<L> v;
        v.from_shared(slots + at + j * kSlot);
        return v;
    }
};

// Puts everything that reaches the bound on the list.
template <typename L, int T>
__device__ void collect(LogShared<T>& sm, const Part<L, T>& p, float bound) {
    p.each([&](const Vec<L>& v, int index) { put_on_list(sm, v, index, bound); });
}

// How many of n things come before the one that is this thread's: `parts` neighbouring threads share one.
template <typename F>
__device__ __forceinline__ int count_before(int n, int parts, F before) {
    int count = 0;
#pragma unroll 4
    for (int i = threadIdx.x & (parts - 1); i < n; i += parts) count += before(i);
    for (int o = parts >> 1; o > 0; o >>= 1) count += __shfl_xor_sync(0xffffffffu, count, o);
    return count;
}

// The k largest of n different keys, in order, to out; where there are fewer, numbers for none that no other CTA of the row has.
// Few keys by few warps: the others have nothing to wait for but a barrier.
template <int T>
__device__ __forceinline__ void rank_list(const Key* list, int n, int k, int rank, Key* out) {
    for (int j = n + threadIdx.x; j < k; j += T) out[j] = 1 + rank * kMaxK + j;
    const int shift = n <= 64 ? 3 : n <= 128 ? 2 : n <= 256 ? 1 : 0;              // 1 << shift threads for an entry
    for (int first = threadIdx.x & ~31; first < n << shift; first += T) {
        const int e = (first + (int)(threadIdx.x & 31)) >> shift;
        const Key mine = e < n ? list[e] : 0;
        const int before = count_before(n, 1 << shift, [&](int i) { return list[i] > mine; });
        if (e < n && before < k && (threadIdx.x & ((1 << shift) - 1)) == 0) out[before] = mine;
    }
}

// The k largest by k searches.
template <typename L, int T>
__device__ void search(LogShared<T>& sm, const Part<L, T>& p, int k, int rank, Key* out) {
    Key last = ~0ULL;
    for (int j = 0; j < k; ++j) {
        Key b = 0;
        p.each([&](const Vec<L>& v, int index) {
            float x[Vec<L>::kN];
            v.get(x);
#pragma unroll
            for (int i = 0; i < Vec<L>::kN; ++i) {
                const Key e = x[i] > kNone ? key_of(x[i], index + i) : 0;
                if (e < last && e > b) b = e;
            }
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) b = max(b, __shfl_xor_sync(0xffffffffu, b, o));
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sm.list[threadIdx.x >> 5] = b;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < Cta<T>::kWarps; ++w) b = max(b, sm.list[w]);
            sm.one = b;
            out[j] = b ? b : 1 + rank * kMaxK + j;
        }
        __syncthreads();
        last = sm.one;
    }
}

// The sums of a warp's lanes, each against its own largest, against the largest of all; returns that.
__device__ __forceinline__ float join(float own, float2 part, float c, float2& all) {
    const float m = unordered(__reduce_max_sync(0xffffffffu, ordered(own)));
    if (part.x > 0.f) {
        const float y = fmaxf(apart(own, m, c, 0.f), -1e30f), f = exp2_fast(y);
        part = make_float2(f * part.x, f > 0.f ? f * fmaf(y, part.x, part.y) : 0.f);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        part.x += __shfl_xor_sync(0xffffffffu, part.x, o);
        part.y += __shfl_xor_sync(0xffffffffu, part.y, o);
    }
    all = part;
    return m;
}

template <typename L, bool kTop, int T>
__global__ void __launch_bounds__(T, Cta<T>::kPerSm) logprobs_kernel(const ft_logprob c, int shift) {
    constexpr int kWarps = Cta<T>::kWarps, kSlot = Cta<T>::kSlot, kHits = Cta<T>::kHits;
    __shared__ LogShared<T> sm;
    extern __shared__ __align__(16) uint8_t log_ring[];
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ctas = 1 << shift, rank = blockIdx.x & (ctas - 1);
    if (ctas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");      // waited for before the first remote store
    const float c2 = fminf(c.scale * 1.4426950408889634f, FLT_MAX);
    const long long r = blockIdx.x >> shift;
    const Part<L, T> p(static_cast<const L*>(c.logits) + r * c.stride, c.V, rank, shift);
    const Ring<L, T> ring(p, log_ring);
    ring.start();
    Vec<L> rest[1];
    p.load_rest(rest[0]);
    float asked = kNone;                                     // the given token's logit
    if (rank == 0 && threadIdx.x == 0 && c.logp) {
        const int token = c.tokens[r];
        if (token >= 0 && token < c.V) asked = (float)p.row[token];
    }

    // the sample, all that is under way: its largest, and the warps' few largest
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    typename Vec<L>::Max largest = Vec<L>::limit(kNone);
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        if (i < ring.rounds) {
#pragma unroll
            for (int j = 0; j < kVectors; ++j) largest = Vec<L>::larger(largest, ring.get(i * kVectors * kSlot, j).max());
        }
    }
    float most = Vec<L>::value(largest);
    most = most == most ? fminf(most, FLT_MAX) : kNone;
    unsigned key = ordered(most);
    const int each = kTop ? (2 * c.k + kWarps - 1) / kWarps : 1;  // of a warp: together at least 2 k, which hold about the sample's k largest
    for (int i = 0;;) {
        const unsigned u = __reduce_max_sync(0xffffffffu, key);
        if (lane == 0) sm.few[warp * each + i] = unordered(u);
        if (++i == each) break;
        if (lane == __ffs(__ballot_sync(0xffffffffu, key == u)) - 1) key = ordered(kNone);
    }
    if (threadIdx.x == 0) sm.count = 0;
    __syncthreads();
    if ((int)(threadIdx.x & ~31) < 4 * kWarps * each) {           // four threads for each of them
        const int n = kWarps * each, mine_at = threadIdx.x >> 2;
        const float mine = mine_at < n ? sm.few[mine_at] : kNone;
        const int before = count_before(n, 4, [&](int i) { return sm.few[i] > mine || (sm.few[i] == mine && i < mine_at); });
        if (mine_at < n && before == 0) sm.ref = mine;
        if (mine_at < n && before == (kTop ? c.k - 1 : 0)) sm.bound = mine;
    }
    __syncthreads();
    const float bound = sm.bound;
    Sums<L> a;
    a.s = a.d = 0;
    a.top = sm.ref;
    a.against(sm.ref, bound, c2, 100.f * inverse_fast(c2));
    int hits = 0;
    if (p.rest) take<L, kTop, T, 1>(sm, a, hits, rest, [&](int) { return p.rest_index(); }, bound, c2);
    uint32_t slot = 0;
    for (int i = 0; i < ring.rounds; ++i) {
        ring.wait();
        Vec<L> v[kVectors];
#pragma unroll
        for (int j = 0; j < kVectors; ++j) v[j] = ring.get(slot, j);
        take<L, kTop, T, kVectors>(sm, a, hits, v, [&](int j) { return p.index(i * kVectors + j); }, bound, c2);
        ring.issue(i + kRounds, slot);
        slot = slot == Cta<T>::kRing - kVectors * kSlot ? 0 : slot + kVectors * kSlot;
    }
    if (kTop) {
        __syncwarp();
        for (int e = lane; e < min(hits, kHits); e += 32) {
            Vec<L> v;
            v.from_shared((uint32_t)__cvta_generic_to_shared(&sm.hit[warp][e]));
            put_on_list(sm, v, sm.hit_at[warp][e], bound);
        }
        if (lane == 0 && hits > kHits) atomicAdd(&sm.count, kListed + 1);        // not all of them: the part is read again
    }

    // the warp's sums against its largest
    float m = unordered(__reduce_max_sync(0xffffffffu, ordered(a.top)));
    float2 sums = a.moved(m, c2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sums.x += __shfl_xor_sync(0xffffffffu, sums.x, o);
        sums.y += __shfl_xor_sync(0xffffffffu, sums.y, o);
    }
    if (lane == 0) sm.red[0][warp] = m, sm.red[1][warp] = sums.x, sm.red[2][warp] = sums.y;
    __syncthreads();
    if (kTop) {
        int n = sm.count;
        if (n > kListed) {
            // at most twice (rising logits let a list's worth through each time)
            float next = bound;
            for (int i = 0; i < 2; ++i) {
                __syncthreads();
                if (threadIdx.x == 0) sm.count = 0;
                __syncthreads();
                collect(sm, p, next);
                __syncthreads();
                n = sm.count;
                if (n <= kListed) break;
                // the list's k-th largest bounds the row's
                rank_list<T>(sm.list, kListed, c.k, rank, sm.top);
                __syncthreads();
                next = key_logit(sm.top[c.k - 1]);
            }
            __syncthreads();
        }
        if (n > kListed) search(sm, p, c.k, rank, sm.top);
        else rank_list<T>(sm.list, n, c.k, rank, sm.top);
        __syncthreads();
    }
    if (warp == 0) {
        m = join(lane < kWarps ? sm.red[0][lane] : kNone, lane < kWarps ? make_float2(sm.red[1][lane], sm.red[2][lane]) : make_float2(0.f, 0.f),
                 c2, sums);
        if (ctas > 1) {
            // what each CTA found, to the first one
            asm volatile("barrier.cluster.wait;" ::: "memory");
            if (kTop && lane < c.k) {
                const Key b = sm.top[lane];
                const uint32_t* to = reinterpret_cast<const uint32_t*>(&sm.tops[rank * c.k + lane]);
                store_first(to, (uint32_t)b);
                store_first(to + 1, (uint32_t)(b >> 32));
            }
            if (lane == 0) {
                store_first(&sm.sums[rank][0], __float_as_uint(m));
                store_first(&sm.sums[rank][1], __float_as_uint(sums.x));
                store_first(&sm.sums[rank][2], __float_as_uint(sums.y));
            }
        }
    } else if (ctas > 1) {
        asm volatile("barrier.cluster.wait;" ::: "memory");
    }
    if (ctas > 1) {
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        if (rank) return;
        if (kTop) {
            rank_list<T>(sm.tops, ctas * c.k, c.k, 0, sm.top);
            __syncthreads();
        }
        if (warp == 0)
            m = join(lane < ctas ? sm.sums[lane][0] : kNone, lane < ctas ? make_float2(sm.sums[lane][1], sm.sums[lane][2]) : make_float2(0.f, 0.f),
                     c2, sums);
    }
    if (warp) return;                                            // k is at most a warp's threads
    const bool none = m == kNone;
    const float log_sum = none ? 0.f : logf(sums.x);
    if (lane == 0) {
        const float x = asked == asked ? fminf(asked, FLT_MAX) : kNone;
        if (c.logp) c.logp[r] = x == kNone ? kNone : apart(x, m, c.scale, -log_sum, 2.f);
        if (c.entropy) c.entropy[r] = none ? 0.f : fmaxf(log_sum - sums.y / sums.x * 0.6931471805599453f, 0.f);
    }
    if (kTop && lane < c.k) {
        const float x = key_logit(sm.top[lane]);
        c.top_ids[r * c.k + lane] = key_index(sm.top[lane]);
        c.top_logp[r * c.k + lane] = x > kNone ? apart(x, m, c.scale, -log_sum, 2.f) : kNone;
    }
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

template <typename L, bool kTop, int T>
cudaError_t launch(const ft_logprob& c, int shift, cudaStream_t s) {
    static std::atomic<bool> done[kMaxDevices];                  // the kernel's attribute is set on this device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices || !done[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(logprobs_kernel<L, kTop, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cta<T>::kRing);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) done[dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c.n << shift);
    cfg.blockDim = dim3(T);
    cfg.dynamicSmemBytes = Cta<T>::kRing;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1 << shift;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<L, kTop, T>, c, shift);
}

// Threads of a CTA: 512 (2 CTAs per SM), 384 (3) or 256 (4).  More CTAs overlap more of the rows' barriers, but their samples are
// smaller and let more logits, k V / sample, through to be ranked; and few rows leave few CTAs.  us with 512, 384, 256 threads, bf16:
// (fp32 rows go by the same rule, unmeasured with other widths)
//   2048 rows of 131,072: k = 1 91 83.5 85, k = 5 95.5 89 89, k = 20 110 106 114, k = 32 121 125 168
//   2048 rows of 50,304: k = 5 60.5 50 45, k = 32 75 67 65;  of 8192: k = 5 35 25.5 20
//   304 rows of 131,072: 17.1 22.8 19.4;  456: 25.5 24.4 28.8
template <typename L, bool kTop>
cudaError_t launch(const ft_logprob& c, int shift, cudaStream_t s) {
    const long long vectors = c.V / Vec<L>::kN, listed = vectors * c.k;
    if (c.n <= 2 * sm_count() || listed > 450000) return launch<L, kTop, 512>(c, shift, s);
    if (vectors > 14000 || listed > 200000) return launch<L, kTop, 384>(c, shift, s);
    return launch<L, kTop, 256>(c, shift, s);
}
template <typename L>
cudaError_t launch(const ft_logprob& c, int shift, cudaStream_t s) {
    return c.k ? launch<L, true>(c, shift, s) : launch<L, false>(c, shift, s);
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
    // CTAs of a row, a power of two: as many as leave no SM with two, each with a vector or more per thread (48 rows of 100,003 fp32, k =
    // 20: 2 CTAs 11.0 us, 3 12.2 us, 4, of which some share an SM, 12.3 us; 24 rows: 4 8.5 us, 6 10.5 us)
    int shift = 0;
    const long long vectors = (long long)c.V / (c.dtype == FT_DTYPE_BF16 ? 8 : 4);
    while (1 << shift < kMaxCtas && (2LL << shift) * c.n <= sm_count() && vectors > 512LL << shift) ++shift;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = c.dtype == FT_DTYPE_BF16 ? launch<__nv_bfloat16>(c, shift, s) : launch<float>(c, shift, s);
    return e == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}
