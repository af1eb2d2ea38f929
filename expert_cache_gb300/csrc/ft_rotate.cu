// New queries, keys and values on their way to attention: the norm of each head, the rotation by position, queries rounded
// to bf16, keys and values quantised into the cache.
//
// A warp has whole heads of neighbouring tokens, a lane 16 dims of a head as 8 pairs: 8 dims of the first half of what turns and
// their 8 partners, or 16 neighbours.  So a rotation needs nothing from another lane, and the mean of the squares takes two
// to four shuffles.  For a query the norm's weights and the angles fold into two factors per dim, which serve all heads of a run:
//   out[d] = r (x[d] A[d] + x[partner of d] B[d]),  A = w[d] c, B = -+ w[partner] s,  r = (mean x^2 + eps)^-1/2.
// A key is rounded to a few bits, and a last bit that differs can move its code by a whole step, so its values are carried as
// unevaluated sums of two fp32 (products split by a fused multiply-add, sums by Knuth's two-sum) down to the rounding.
//
// 8192 tokens of 32 query and 8 + 8 key and value heads of 128, NVFP4, all normalised and turned: 41 us for 194 MB, 0.7 of the copy
// rate (reading them back takes another 10 us).  Bound by no one thing: instructions are issued 60 % of the time by up to 20 warps per SM, which
// wait for results, for loads and for their turn about equally; some 190 for
// a query's 16 dims of 32 lanes, 1000 for a key's and a value's together (of which the two parts take 400, quantising 260).  A token
// alone: 4.1 us with reading back, two launches.  On the way: a lane per scale block with its partners in another lane, 16 shuffles
// a head, 94 us with reading back; partners in the same lane and packed arithmetic 82 us; heads asked for four ahead through
// shared memory instead of one through registers 56 us; words taken one by one, so that 96 registers are enough for 20 warps per SM 52 us; CTAs of one warp, whose
// place is free as soon as it is through, 50.4 us (of four 50.7; 3001 tokens of 20 + 4 + 4 heads of 64 11.8 us, of four 13.1).
#include <cmath>

#include "ft_kv_host.cuh"
#include "ft_kv_quant.cuh"
#include "ft_pair.cuh"

namespace ft {

namespace {

constexpr int kRotThreads = 32, kRotPerSm = 20;
constexpr int kAhead = 4;              // heads that a lane has under way

struct RotateArgs {
    KvView kv;
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *q_out, *k_out;
    size_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
    const float *q_norm, *k_norm, *rope;
    const int32_t *positions, *slots;
    int n, hq, rope_dim, n_positions;
    int run, units;      // heads of a warp, and how many such runs the k, v and q heads (in this order) make
    float eps;
};

// The bf16 words of a lane: word j holds the dims lo + 2 j and on (j < 4) or hi + 2 (j - 4).  Partners: of word j word j ^ 4, or
// (kInter) the two dims of a word.
template <int D, bool kInter>
struct Lane {
    static constexpr int kLanes = D / 16;
    int b;               // of the head's lanes
    int lo, hi;
    bool turns;
    __device__ __forceinline__ Lane(int rope_dim) {
        b = (threadIdx.x & 31) % kLanes;
        turns = 16 * b < rope_dim;
        lo = !kInter && turns ? 8 * b : 16 * b;
        hi = !kInter && turns ? rope_dim / 2 + lo : lo + 8;
    }
    __device__ __forceinline__ void store(__nv_bfloat16* head, const uint32_t (&x)[8]) const {
        *reinterpret_cast<uint4*>(head + lo) = make_uint4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<uint4*>(head + hi) = make_uint4(x[4], x[5], x[6], x[7]);
    }
    // The norm's weights of the lane's dims (none: 1).
    __device__ __forceinline__ void norms(Pair (&w)[8], const float* norm) const {
        if (!norm) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = pair(1.f, 1.f);
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 v = reinterpret_cast<const float4*>(norm + (j < 2 ? lo : hi - 8))[j];
            w[2 * j] = pair(v.x, v.y);
            w[2 * j + 1] = pair(v.z, v.w);
        }
    }
    // Those of word j.
    __device__ __forceinline__ Pair norm(const float* norm, int j) const {
        const float2 v = *reinterpret_cast<const float2*>(norm + (j < 4 ? lo + 2 * j : hi + 2 * (j - 4)));
        return pair(v.x, v.y);
    }
    // Cosines and signed sines of the lane's dims at a position (none: 1 and 0).
    __device__ __forceinline__ void angles(Pair (&c)[8], Pair (&s)[8], const float* table, int rope_dim, int pos) const {
        if (!turns) {
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = pair(1.f, 1.f), s[j] = pair(0.f, 0.f);
            return;
        }
        const float4* row = reinterpret_cast<const float4*>(table + (size_t)pos * rope_dim + 8 * b);
        const float4* sines = row + rope_dim / 8;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 cv = row[j], sv = sines[j];
            if constexpr (kInter) {
                c[4 * j] = pair(cv.x, cv.x); c[4 * j + 1] = pair(cv.y, cv.y); c[4 * j + 2] = pair(cv.z, cv.z); c[4 * j + 3] = pair(cv.w, cv.w);
                s[4 * j] = pair(-sv.x, sv.x); s[4 * j + 1] = pair(-sv.y, sv.y); s[4 * j + 2] = pair(-sv.z, sv.z); s[4 * j + 3] = pair(-sv.w, sv.w);
            } else {
                c[2 * j] = c[2 * j + 4] = pair(cv.x, cv.y);
                c[2 * j + 1] = c[2 * j + 5] = pair(cv.z, cv.w);
                s[2 * j] = pair(-sv.x, -sv.y); s[2 * j + 4] = pair(sv.x, sv.y);
                s[2 * j + 1] = pair(-sv.z, -sv.w); s[2 * j + 5] = pair(sv.z, sv.w);
            }
        }
    }
    // What stands at the partners of word j.
    static __device__ __forceinline__ Pair partner(const Pair (&x)[8], int j) { return kInter ? swap2(x[j]) : x[j ^ 4]; }
};

__device__ __forceinline__ Pair unpack(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
__device__ __forceinline__ uint32_t pack_bf16(Pair p) {
    const float2 f = halves(p);
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void zero(uint32_t (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0;
}
// An inverse norm r that is no positive number.  0, of an infinite norm: numbers become 0 before a weight can make them infinite,
// infinities and NaN become NaN.  NaN, of a head with a NaN: all dims do.
__device__ __forceinline__ void times(uint32_t (&x)[8], float r) {
    const __nv_bfloat162 none = __floats2bfloat162_rn(r, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const __nv_bfloat162 a = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&x[j]), none);
        x[j] = *reinterpret_cast<const uint32_t*>(&a);
    }
}

// One head in fp32 by the folded factors.
template <int D, bool kInter>
__device__ __forceinline__ void turn_plainly(const Lane<D, kInter>& p, uint32_t (&w)[8], const Pair (&A)[8], const Pair (&B)[8], float r, bool part) {
    Pair x[8];
    const Pair rr = pair(r, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = mul2(unpack(w[j]), rr);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        Pair y = Lane<D, kInter>::partner(x, j);
        if (part && !p.turns) y = 0;                               // 0 times an infinity is none
        w[j] = pack_bf16(fma2(x[j], A[j], mul2(y, B[j])));
    }
}

// A lane's bytes of a run of heads on their way through its own slots of shared memory, kAhead heads of them.  Nobody else
// reads them, so its own wait for its copies is all there is to wait for.
struct Heads {
    const __nv_bfloat16 *k, *v, *q;    // the token's
    const __nv_bfloat16 *lo, *hi;      // the lane's dims of the next head to ask for
    int hkv, at, end, D;               // that head, in the order k, v, q; end of the run
    int turn;                          // where lo and hi pass on to the next of the three
    uint32_t slots, ask, take;         // this thread's shared memory, where the next head goes, where the first one is

    template <typename L>
    __device__ __forceinline__ void point(const L& p) {
        const bool is_v = at >= hkv && at < 2 * hkv;
        const __nv_bfloat16* head = at < hkv ? k + at * D : is_v ? v + (at - hkv) * D : q + (at - 2 * hkv) * D;
        lo = head + (is_v ? 16 * p.b : p.lo);
        hi = head + (is_v ? 16 * p.b + 8 : p.hi);
        turn = at < hkv ? hkv : is_v ? 2 * hkv : end;
    }
    template <typename L>
    __device__ __forceinline__ void issue(const L& p) {
        if (at < end) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(slots + ask), "l"(lo) : "memory");
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(slots + ask + kRotThreads * 16), "l"(hi) : "memory");
            lo += D;
            hi += D;
            if (++at == turn) point(p);
        }
        ask = (ask + 2 * kRotThreads * 16) & (2 * kAhead * kRotThreads * 16 - 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    template <typename L>
    __device__ __forceinline__ void next(const L& p, uint32_t (&x)[8]) {
        asm volatile("cp.async.wait_group %0;" :: "n"(kAhead - 1) : "memory");
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(slots + take));
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]) : "r"(slots + take + kRotThreads * 16));
        issue(p);                      // into the slots just read
        take = (take + 2 * kRotThreads * 16) & (2 * kAhead * kRotThreads * 16 - 1);
    }
};

// Query heads head .. end - 1 of a token.
template <int D, bool kInter>
__device__ __forceinline__ void turn_queries(const RotateArgs& a, const Lane<D, kInter>& p, Heads& heads, const Pair (&c)[8], const Pair (&s)[8],
                                             int tok, bool live, int head, int end) {
    Pair A[8], B[8], w[8];
    p.norms(w, a.q_norm);
#pragma unroll
    for (int j = 0; j < 8; ++j) A[j] = mul2(c[j], w[j]), B[j] = mul2(s[j], Lane<D, kInter>::partner(w, j));
    for (; head < end; ++head) {
        uint32_t x[8];
        heads.next(p, x);
        float r = 1.f;
        if (a.q_norm) {
            Pair two = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const Pair u = unpack(x[j]);
                two = fma2(u, u, two);
            }
            float sum = halves(two).x + halves(two).y;
#pragma unroll
            for (int o = 1; o < D / 16; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            r = rsqrtf(sum * (1.f / D) + a.eps);
            if (r == 0.f) times(x, r);
        }
        turn_plainly(p, x, A, B, r, a.rope_dim < D);
        if (live) p.store(a.q_out + (size_t)tok * a.q_out_stride + head * D, x);
    }
}

struct Two {
    float h, l;          // the value is h + l
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), z = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z))};
}
__device__ __forceinline__ void two_sum2(Pair a, Pair b, Pair& h, Pair& l) {
    h = add2(a, b);
    const Pair z = from2(a, h);
    l = add2(from2(from2(z, h), a), from2(z, b));
}

// (mean x^2 + eps)^-1/2 of a head; squares of bf16 are exact in fp32.
template <int D>
__device__ __forceinline__ Two inverse_norm(const uint32_t (&x)[8], float eps) {
    Pair h = unpack(x[0]), l = 0;
    h = mul2(h, h);
#pragma unroll
    for (int j = 1; j < 8; ++j) {
        const Pair u = unpack(x[j]);
        Pair e;
        two_sum2(h, mul2(u, u), h, e);
        l = add2(l, e);
    }
    const float2 hh = halves(h), ll = halves(l);
    Two sum = two_sum(hh.x, hh.y);
    sum.l = __fadd_rn(sum.l, __fadd_rn(ll.x, ll.y));
#pragma unroll
    for (int o = 1; o < D / 16; o <<= 1) {
        const float oh = __shfl_xor_sync(0xffffffffu, sum.h, o), ol = __shfl_xor_sync(0xffffffffu, sum.l, o);
        const Two t = two_sum(sum.h, oh);
        sum = {t.h, __fadd_rn(__fadd_rn(sum.l, ol), t.l)};
    }
    Two m = two_sum(__fmul_rn(sum.h, 1.f / D), eps);
    m.l = __fmaf_rn(sum.l, 1.f / D, m.l);
    // one step of Newton's on the fp32 root, its residual 1 - m r^2 by way of m r in two parts (r^2 would leave the range at both ends)
    const float r = rsqrtf(m.h), t = __fmul_rn(m.h, r), tl = __fmaf_rn(m.h, r, -t);
    float e = __fmaf_rn(-t, r, 1.f);
    e = __fmaf_rn(-tl, r, e);
    e = __fmaf_rn(-__fmul_rn(m.l, r), r, e);
    return {r, isinf(m.h) ? 0.f : __fmul_rn(__fmul_rn(0.5f, r), e)};
}

// (x - n) c + (y - m) s times rh + rl, rounded to fp32 and to bf16: x - n and y - m stand for a pair's dims times their weights.
__device__ __forceinline__ uint32_t turned(Pair x, Pair n, Pair y, Pair m, Pair c, Pair s, Pair nc, Pair ns, Pair rh, Pair rl) {
    const Pair u = mul2(x, c), ul = fma2(x, nc, u), v = mul2(y, s), vl = fma2(y, ns, v);
    Pair h, l;
    two_sum2(u, v, h, l);
    l = from2(add2(fma2(n, c, ul), fma2(m, s, vl)), l);
    const Pair o = mul2(h, rh), ol = fma2(neg2(h), rh, o);
    return pack_bf16(add2(o, from2(ol, fma2(h, rl, mul2(l, rh)))));
}

// x c + y s in 64 bits, for a head of which a norm leaves nothing but 0, infinities and NaN (turns: 0 times an infinity is none).
__device__ __forceinline__ uint32_t turned_plainly(Pair x, Pair y, Pair c, Pair s, bool turns) {
    const float2 xx = halves(x), yy = turns ? halves(y) : make_float2(0.f, 0.f), cc = halves(c), ss = halves(s);
    return pack_bf16(pair((float)((double)xx.x * cc.x + (double)yy.x * ss.x), (float)((double)xx.y * cc.y + (double)yy.y * ss.y)));
}

// Key heads head .. end - 1 of a token.
template <int D, int kFormat, bool kInter>
__device__ __forceinline__ void turn_keys(const RotateArgs& a, const Lane<D, kInter>& p, Heads& heads, const Pair (&c)[8], const Pair (&s)[8],
                                          int tok, int slot, int head, int end, float inv_k) {
    Pair nc[8], ns[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) nc[j] = neg2(c[j]), ns[j] = neg2(s[j]);
    for (; head < end; ++head) {
        uint32_t k[8];
        heads.next(p, k);
        // an infinity or a NaN has no second part, nor has what a turn takes past fp32's range
        __nv_bfloat162 most = __habs2(*reinterpret_cast<__nv_bfloat162*>(&k[0]));
#pragma unroll
        for (int j = 1; j < 8; ++j) most = __hmax2_nan(most, __habs2(*reinterpret_cast<__nv_bfloat162*>(&k[j])));
        const float2 mm = __bfloat1622float2(most);
        Two r = {1.f, 0.f};
        if (a.k_norm) {
            r = inverse_norm<D>(k, a.eps);
            if (!(r.h > 0.f)) times(k, r.h);
        }
        const Pair rh = pair(r.h, r.h), rl = pair(r.l, r.l);
        const bool numbers = mm.x < 0x1p120f && mm.y < 0x1p120f;
        // word j and, unless its two dims are partners, word j + 4
#pragma unroll
        for (int j = 0; j < (kInter ? 8 : 4); ++j) {
            Pair x = unpack(k[j]), n = 0, y = kInter ? 0 : unpack(k[j ^ 4]), m = 0;
            if (a.k_norm) {
                const Pair w = p.norm(a.k_norm, j), u = x;
                x = mul2(u, w);
                n = fma2(neg2(u), w, x);
                if (!kInter) {
                    const Pair z = p.norm(a.k_norm, j ^ 4), v = y;
                    y = mul2(v, z);
                    m = fma2(neg2(v), z, y);
                }
            }
            if (kInter) y = swap2(x), m = swap2(n);
            if (numbers) {
                k[j] = turned(x, n, y, m, c[j], s[j], nc[j], ns[j], rh, rl);
                if (!kInter) k[j ^ 4] = turned(y, m, x, n, c[j], ns[j], nc[j], s[j], rh, rl);
            } else {
                k[j] = turned_plainly(x, y, c[j], s[j], p.turns);
                if (!kInter) k[j ^ 4] = turned_plainly(y, x, c[j], neg2(s[j]), p.turns);
            }
        }
        if (slot >= 0 && a.k_out) p.store(a.k_out + (size_t)tok * a.k_out_stride + head * D, k);
        int block = p.b;
        if constexpr (!kInter) {
            // of two neighbouring lanes' first and second halves, one lane gets the first block of 16 dims and one the second
            const bool odd = p.b & 1;
            uint32_t other[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) other[j] = __shfl_xor_sync(0xffffffffu, odd ? k[j] : k[j + 4], 1);
            if (p.turns) {
                block = p.b / 2 + (odd ? a.rope_dim / 32 : 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) (odd ? k[j] : k[j + 4]) = other[j];
            }
        }
        if (slot >= 0)
            append_block<D, kFormat, false>(kv_tile_ptr(a.kv, slot, head, kv_tile(D, kFormat).bytes), slot & 15, block, k, a.kv.k_scale, inv_k);
    }
}

template <int D, int kFormat, bool kInter>
__global__ void __launch_bounds__(kRotThreads, kRotPerSm) kv_rotate_kernel(const RotateArgs a) {
    __shared__ __align__(16) uint8_t ring[2 * kAhead * kRotThreads * 16];
    pdl_wait_and_release();
    constexpr int kTokens = 32 / (D / 16);
    const Lane<D, kInter> p(a.rope_dim);
    const long long warps = (long long)gridDim.x * (kRotThreads / 32), groups = ((long long)a.n + kTokens - 1) / kTokens;
    const long long all = groups * a.units;
    const int hkv = a.kv.hkv;
    // runs of k's heads, which take longest, first
    for (long long u = (long long)blockIdx.x * (kRotThreads / 32) + (threadIdx.x >> 5); u < all; u += warps) {
        const int first = (int)(u / groups) * a.run, end = min(first + a.run, a.hq + 2 * hkv);
        const long long token = u % groups * kTokens + (threadIdx.x & 31) / Lane<D, kInter>::kLanes;
        const int tok = (int)min(token, (long long)a.n - 1);
        Heads heads{a.k + (size_t)tok * a.k_stride, a.v + (size_t)tok * a.v_stride, a.q + (size_t)tok * a.q_stride, nullptr, nullptr, hkv, first, end, D,
                    0, (uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * 16, 0, 0};
        heads.point(p);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) heads.issue(p);
        int slot = token < a.n ? a.slots[tok] : -1, pos = a.rope_dim ? a.positions[tok] : 0;
        if (slot < 0 || (slot >> a.kv.page_shift) >= a.kv.n_pages || (a.rope_dim && (pos < 0 || pos >= a.n_positions))) {
            if (slot != -1 && first == 0 && p.b == 0) atomicOr(a.kv.status, FT_DEV_BAD_ID);
            slot = -1;
            pos = 0;                                               // there is a row
        }
        Pair c[8], s[8];
        p.angles(c, s, a.rope, a.rope_dim, pos);
        if (first < hkv) turn_keys<D, kFormat, kInter>(a, p, heads, c, s, tok, slot, first, min(end, hkv), __frcp_rn(a.kv.k_scale));
        for (int head = max(first, hkv); head < min(end, 2 * hkv); ++head) {
            uint32_t x[8];
            heads.next(p, x);
            if (slot >= 0)
                append_block<D, kFormat, true>(kv_tile_ptr(a.kv, slot, head - hkv, kv_tile(D, kFormat).bytes), slot & 15, p.b, x, a.kv.v_scale,
                                               __frcp_rn(a.kv.v_scale));
        }
        if (end > 2 * hkv) turn_queries(a, p, heads, c, s, tok, slot >= 0, max(first - 2 * hkv, 0), end - 2 * hkv);
    }
}

template <int D, int kFormat>
struct Rotate {
    static cudaError_t run(RotateArgs& a, bool inter, cudaStream_t s) {
        const cudaError_t e = inter ? prepare<kv_rotate_kernel<D, kFormat, true>>() : prepare<kv_rotate_kernel<D, kFormat, false>>();
        if (e != cudaSuccess) return e;
        const long long groups = ((long long)a.n + 32 / (D / 16) - 1) / (32 / (D / 16));
        const int heads = a.hq + 2 * a.kv.hkv;
        // heads of a warp: its start (slot, position, angles, weights) is shared by them (8192 tokens of 32 + 8 + 8 heads of 128, with
        // reading back: 1 head 113 us, 2 70, 4 58, 8 53, 16 50), but there are to be 32 runs per SM (3001 tokens of 20 + 4 + 4 heads
        // of 64: 1 head 15.1 us, 2 11.8, 4 13.6, 8 12.8, 16 13.4)
        const long long want = groups * heads / (32LL * sm_count());
        a.run = want < 1 ? 1 : want > 16 ? 16 : (int)want;
        a.units = (heads + a.run - 1) / a.run;
        const long long ctas = (groups * a.units + kRotThreads / 32 - 1) / (kRotThreads / 32);
        return launch_pdl(inter ? kv_rotate_kernel<D, kFormat, true> : kv_rotate_kernel<D, kFormat, false>,
                          dim3((unsigned)(ctas < (1 << 20) ? ctas : 1 << 20)), dim3(kRotThreads), 0, s, a);
    }
};

__global__ void rope_table_kernel(const double* inv_freq, int half, long long all, double mscale, float* table) {
    for (long long at = (long long)blockIdx.x * blockDim.x + threadIdx.x; at < all; at += (long long)gridDim.x * blockDim.x) {
        const long long p = at / half;
        const int i = (int)(at % half);
        double s, c;
        sincos((double)p * inv_freq[i], &s, &c);
        table[p * 2 * half + i] = (float)(mscale * c);
        table[p * 2 * half + half + i] = (float)(mscale * s);
    }
}

}  // namespace

}  // namespace ft

using namespace ft;

extern "C" {

ft_status ft_rope_table(const double* inv_freq, int32_t rope_dim, int32_t n_positions, double mscale, float* table, void* stream) {
    if (!inv_freq || !table || !aligned(inv_freq, 8) || !aligned(table, 4)) return FT_ERR_ARG;
    if (rope_dim < 2 || rope_dim > 256 || rope_dim % 2 || n_positions < 1 || !std::isfinite(mscale)) return FT_ERR_ARG;
    const long long all = (long long)n_positions * (rope_dim / 2), ctas = (all + 255) / 256, most = 16LL * sm_count();
    rope_table_kernel<<<(unsigned)(ctas < most ? ctas : most), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        inv_freq, rope_dim / 2, all, mscale, table);
    return cudaGetLastError() == cudaSuccess ? FT_OK : FT_ERR_CUDA;
}

ft_status ft_kv_append_rotated(ft_kv* kv, const ft_kv_qkv* call, void* stream) {
    if (!kv) return FT_ERR_ARG;
    if (!call) return fail(kv, FT_ERR_ARG, "append_rotated: NULL call");
    const ft_kv_desc& d = kv->d;
    const ft_kv_qkv& c = *call;
    if (c.layer < 0 || c.layer >= d.L || c.n < 0) return fail(kv, FT_ERR_ARG, "append_rotated: layer or n out of range");
    if (c.rope_dim < 0 || c.rope_dim > d.head_dim || c.rope_dim % 32 || (c.rope_dim && c.n_positions < 1) ||
        (c.interleaved != 0 && c.interleaved != 1))
        return fail(kv, FT_ERR_ARG, "append_rotated: rope_dim, n_positions or interleaved");
    if ((c.q_norm || c.k_norm) && !(std::isfinite(c.eps) && c.eps > 0.f)) return fail(kv, FT_ERR_ARG, "append_rotated: eps");
    if (c.n == 0) return FT_OK;
    if (!c.q || !c.k || !c.v || !c.q_out || !c.slots || (c.rope_dim && (!c.rope || !c.positions)))
        return fail(kv, FT_ERR_ARG, "append_rotated: NULL pointer");
    if (!aligned(c.q, 16) || !aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.q_out, 16) || !aligned(c.k_out, 16) ||
        !aligned(c.q_norm, 16) || !aligned(c.k_norm, 16) || !aligned(c.rope, 16) || !words(c.slots, c.positions))
        return fail(kv, FT_ERR_ARG, "append_rotated: misaligned pointer");
    const int64_t q_row = (int64_t)d.n_q_heads * d.head_dim, k_row = (int64_t)d.n_kv_heads * d.head_dim;
    if (c.q_stride < q_row || c.q_out_stride < q_row || c.k_stride < k_row || c.v_stride < k_row || (c.k_out && c.k_out_stride < k_row) ||
        (c.q_stride | c.q_out_stride | c.k_stride | c.v_stride | (c.k_out ? c.k_out_stride : 0)) % 8)
        return fail(kv, FT_ERR_ARG, "append_rotated: token strides");
    NvtxRange r("ft_kv_append_rotated");
    RotateArgs a;
    a.kv = view(kv, c.layer);
    a.q = static_cast<const __nv_bfloat16*>(c.q);
    a.k = static_cast<const __nv_bfloat16*>(c.k);
    a.v = static_cast<const __nv_bfloat16*>(c.v);
    a.q_out = static_cast<__nv_bfloat16*>(c.q_out);
    a.k_out = static_cast<__nv_bfloat16*>(c.k_out);
    a.q_stride = (size_t)c.q_stride;
    a.k_stride = (size_t)c.k_stride;
    a.v_stride = (size_t)c.v_stride;
    a.q_out_stride = (size_t)c.q_out_stride;
    a.k_out_stride = (size_t)c.k_out_stride;
    a.q_norm = c.q_norm;
    a.k_norm = c.k_norm;
    a.rope = c.rope;
    a.positions = c.positions;
    a.slots = c.slots;
    a.n = c.n;
    a.hq = d.n_q_heads;
    a.rope_dim = c.rope_dim;
    a.n_positions = c.n_positions;
    a.eps = c.eps;
    const cudaError_t e = by_shape<Rotate>(d.head_dim, d.format, a, c.interleaved != 0, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FT_OK : cuda_fail(kv, e, "append_rotated launch");
}

}  // extern "C"
