// What the attention kernels share: which keys a row tile needs, the rule of who sees whom,
// and the numbers of the running softmax.
#pragma once
#include "ft_kv.cuh"

namespace ft {

// Softmax in base 2: a weight is exp2(t - m + kHeadroom) with t = s * scale * log2(e) and a
// reference m that is raised (and everything rescaled) only when some t exceeds it by more than
// kHeadroom.  Weights are then at most 2^(2 kHeadroom) = 2^14 and a weight 2^-20 times the
// reference's is still a normal f16.
constexpr float kHeadroom = 7.f;
constexpr float kNoRef = -1.7e38f;     // reference of a row that has seen no key: any finite t exceeds it

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The keys of a tile of rows, in blocks of kB keys: the blocks [0, a_end) (first tokens) and
// [b0, b0 + nt - a_end).  empty: no row sees a key (one block is counted, for the zeros).
struct RowTile {
    int i0, i1;          // tokens of its first and last row
    int a_end, b0, nt;
    bool empty;
    __device__ __forceinline__ int block(int v) const { return v < a_end ? v : b0 + v - a_end; }
};

// Row tile r (R rows; row = token * G + query head of the group) of a sequence of n tokens.
template <int kB>
__device__ __forceinline__ RowTile row_tile(const AttnArgs& a, const SeqInfo& s, int r, int R) {
    RowTile t;
    t.i0 = r * R / a.G;
    t.i1 = min(s.n - 1, (r * R + R - 1) / a.G);
    const int base = s.len - s.n;
    const int hi = a.tree ? s.len : min(s.len, base + t.i1 + 1);
    // a drafted token stands at base or after it
    const long long low = a.window > 0 ? (long long)base + (a.tree ? 0 : t.i0) - a.window + 1 : 0;
    const int lo = (int)max(low, 0LL);
    t.empty = hi <= 0;
    t.a_end = 0;
    t.b0 = 0;
    t.nt = 1;
    if (!t.empty) {
        t.b0 = min(lo, hi) / kB;
        t.a_end = min((min(a.n_sink, min(lo, hi)) + kB - 1) / kB, t.b0);
        t.nt = t.a_end + (hi + kB - 1) / kB - t.b0;
    }
    return t;
}

// One row's rule: key j is seen if j <= lim and (j >= low or j < n_sink), and under a tree the
// drafted keys (j >= base) go by the row's mask.
struct RowRule {
    int lim, low;
    unsigned long long mask;
};
__device__ __forceinline__ RowRule row_rule(const AttnArgs& a, const SeqInfo& s, int row) {
    RowRule r{-1, 0, 0};
    const int i = row / a.G;
    if (i >= s.n) return r;            // padding
    const int base = s.len - s.n;
    int pos = base + i;
    r.lim = min(pos, s.len - 1);
    if (a.tree) {
        r.mask = a.tree[s.q0 + i];
        pos = base + __popcll(r.mask & ~(1ull << i));
        r.lim = s.len - 1;
    }
    if (a.window > 0) r.low = (int)max((long long)pos - a.window + 1, 0LL);
    return r;
}
// The rule for a key below base or without a tree.
__device__ __forceinline__ bool sees(const AttnArgs& a, const RowRule& r, int j) {
    return j <= r.lim && (j >= r.low || j < a.n_sink);
}
// Place of a drafted key under a tree.
__device__ __forceinline__ int drafted_pos(const AttnArgs& a, const SeqInfo& s, int j) {
    const int jj = j - (s.len - s.n);
    return s.len - s.n + __popcll(a.tree[s.q0 + jj] & ~(1ull << jj));
}
// The rule for a drafted key j >= base, base <= j < len, that stands at place pos.
__device__ __forceinline__ bool sees_drafted(const AttnArgs& a, const RowRule& r, int base, int j, int pos) {
    return (r.mask >> (j - base) & 1) && (pos >= r.low || j < a.n_sink);
}

// N (2 or 4) output values, dims d.., of one row and query head from their weighted sums x, the
// reference m and the sum of weights l; a row without keys (l = 0) gives 0 and -inf.
template <int N>
__device__ __forceinline__ void store_out(const AttnArgs& a, size_t token, int h, int D, int d, const float* x, float m, float l) {
    const float f = l == 0.f ? 0.f : a.kv.v_scale / l;
    uint32_t w[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * e] * f, x[2 * e + 1] * f);
        w[e] = *reinterpret_cast<const uint32_t*>(&p);
    }
    __nv_bfloat16* dst = a.o + token * a.o_stride + (size_t)h * D + d;
    if constexpr (N == 2) *reinterpret_cast<uint32_t*>(dst) = w[0];
    else *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    if (d == 0 && a.lse)
        a.lse[token * a.hq + h] = l == 0.f ? -INFINITY : (m - kHeadroom + log2f(l)) * 0.693147180559945309417f;
}

}  // namespace ft
