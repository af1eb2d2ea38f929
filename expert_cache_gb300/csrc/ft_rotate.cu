// New queries, keys and values on their way to attention: the norm of each head, the rotation by position, queries rounded
// to bf16, keys and values quantised into the cache.
//
// A lane has 16 dims of a head (a scale block of the cache), a warp whole heads of neighbouring tokens, so that the
// mean of the squares takes two to four shuffles and the other half of a pair comes from a lane of the same warp.
// For a query the norm's weights and the angles fold into two factors per dim, which serve all heads of a run:
//   out[d] = r (x[d] A[d] + x[pair of d] B[d]),  A = w[d] c, B = -+ w[pair] s,  r = (mean x^2 + eps)^-1/2.
// A key is rounded to a few bits, and a last bit that differs can move its code by a whole step, so its values are carried as
// unevaluated sums of two fp32 (products split by a fused multiply-add, sums by Knuth's two-sum) down to the rounding.
#include <cmath>

#include "ft_kv_host.cuh"
#include "ft_kv_quant.cuh"

namespace ft {

namespace {

constexpr int kRotThreads = 128;

struct RotateArgs {
    KvView kv;
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *q_out, *k_out;
    size_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
    const float *q_norm, *k_norm, *rope;
    const int32_t *positions, *slots;
    int n, hq, rope_dim, n_positions;
    int run, q_runs, k_runs, units;      // heads of a warp; runs of q's heads, of k's (and as many of v's), of all
    float eps;
};

struct Two {
    float h, l;          // the value is h + l
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), z = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z))};
}
__device__ __forceinline__ Two two_mul(float a, float b) {
    const float p = __fmul_rn(a, b);
    return {p, __fmaf_rn(a, b, -p)};
}

// A lane's place: token, block of 16 dims, and where its pairs are.
template <int D, bool kInter>
struct Lane {
    static constexpr int kLanes = D / 16;
    int b, src;          // block of the head; lane that has the pairs' other dims (its own: within the block, or none)
    int at, angle;       // first dim of that; first pair's index
    bool turns, low;     // is rotated; its dims are the pairs' first ones
    __device__ __forceinline__ Lane(int rope_dim) {
        const int lane = threadIdx.x & 31;
        b = lane % kLanes;
        turns = 16 * b < rope_dim;
        low = 32 * b < rope_dim;
        int other = b;
        if (!kInter && turns) other = low ? b + rope_dim / 32 : b - rope_dim / 32;
        src = lane - b + other;
        at = 16 * other;
        angle = kInter ? 8 * b : 16 * (low ? b : other);
    }
};

__device__ __forceinline__ void load16(float (&f)[16], const float* p) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 v = reinterpret_cast<const float4*>(p)[j];
        f[4 * j] = v.x; f[4 * j + 1] = v.y; f[4 * j + 2] = v.z; f[4 * j + 3] = v.w;
    }
}

// Cosine and signed sine of each of a lane's dims.
template <bool kInter, int D>
__device__ __forceinline__ void load_angles(const RotateArgs& a, const Lane<D, kInter>& p, int pos, float (&c)[16], float (&s)[16]) {
    if (!p.turns || pos < 0) {
#pragma unroll
        for (int j = 0; j < 16; ++j) c[j] = 1.f, s[j] = 0.f;
        return;
    }
    const float* row = a.rope + (size_t)pos * a.rope_dim + p.angle;
    if constexpr (kInter) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 cc = reinterpret_cast<const float4*>(row)[j];
            const float4 ss = reinterpret_cast<const float4*>(row + a.rope_dim / 2)[j];
            const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[8 * j + 2 * i] = c[8 * j + 2 * i + 1] = cv[i];
                s[8 * j + 2 * i] = -sv[i];
                s[8 * j + 2 * i + 1] = sv[i];
            }
        }
    } else {
        load16(c, row);
        load16(s, row + a.rope_dim / 2);
        if (p.low)
#pragma unroll
            for (int j = 0; j < 16; ++j) s[j] = -s[j];
    }
}

// The other dims of the lane's pairs (zeros where there are none).
template <bool kInter, int D>
__device__ __forceinline__ void pairs_of(const Lane<D, kInter>& p, const uint32_t (&x)[8], uint32_t (&y)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[j] = kInter ? __byte_perm(x[j], 0, 0x1032) : __shfl_sync(0xffffffffu, x[j], p.src);
        if (!p.turns) y[j] = 0;
    }
}
template <bool kInter, int D>
__device__ __forceinline__ void load_norms(const Lane<D, kInter>& p, const float* norm, float (&w)[16], float (&wp)[16]) {
    load16(w, norm + 16 * p.b);
    if constexpr (kInter) {
#pragma unroll
        for (int j = 0; j < 16; ++j) wp[j] = w[j ^ 1];
    } else {
        load16(wp, norm + p.at);
    }
}

__device__ __forceinline__ void zero(uint32_t (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0;
}
// An infinite norm: numbers become 0 before a weight can make them infinite, infinities and NaN become NaN.
__device__ __forceinline__ void times_zero(uint32_t (&x)[8], uint32_t (&y)[8]) {
    const __nv_bfloat162 none = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        __nv_bfloat162 a = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&x[j]), none), b = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&y[j]), none);
        x[j] = *reinterpret_cast<uint32_t*>(&a);
        y[j] = *reinterpret_cast<uint32_t*>(&b);
    }
}
__device__ __forceinline__ void store_block(__nv_bfloat16* dst, const uint32_t (&x)[8]) {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}

// A run of a token's query heads.
template <int D, bool kInter>
__device__ __forceinline__ void turn_queries(const RotateArgs& a, const Lane<D, kInter>& p, int tok, int pos, bool live, int head, int end) {
    float A[16], B[16];
    load_angles(a, p, pos, A, B);
    if (a.q_norm) {
        float w[16], wp[16];
        load_norms(p, a.q_norm, w, wp);
#pragma unroll
        for (int j = 0; j < 16; ++j) A[j] *= w[j], B[j] *= wp[j];
    }
    for (; head < end; ++head) {
        uint32_t x[8], y[8];
        if (live) load_block(x, a.q + (size_t)tok * a.q_stride + head * D + 16 * p.b);
        else zero(x);
        pairs_of(p, x, y);
        float r = 1.f;
        if (a.q_norm) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) sum = fmaf(bf16_at(x, j), bf16_at(x, j), sum);
#pragma unroll
            for (int o = 1; o < D / 16; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            r = rsqrtf(sum * (1.f / D) + a.eps);
            if (r == 0.f) times_zero(x, y);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float lo = r * fmaf(bf16_at(x, 2 * j), A[2 * j], bf16_at(y, 2 * j) * B[2 * j]);
            const float hi = r * fmaf(bf16_at(x, 2 * j + 1), A[2 * j + 1], bf16_at(y, 2 * j + 1) * B[2 * j + 1]);
            x[j] = pack_bf16(lo, hi);
        }
        if (live) store_block(a.q_out + (size_t)tok * a.q_out_stride + head * D + 16 * p.b, x);
    }
}

// (mean x^2 + eps)^-1/2 of a head; squares of bf16 are exact in fp32.
template <int D>
__device__ __forceinline__ Two inverse_norm(const uint32_t (&x)[8], float eps) {
    Two sum = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const Two t = two_sum(sum.h, __fmul_rn(bf16_at(x, j), bf16_at(x, j)));
        sum = {t.h, __fadd_rn(sum.l, t.l)};
    }
#pragma unroll
    for (int o = 1; o < D / 16; o <<= 1) {
        const float h = __shfl_xor_sync(0xffffffffu, sum.h, o), l = __shfl_xor_sync(0xffffffffu, sum.l, o);
        const Two t = two_sum(sum.h, h);
        sum = {t.h, __fadd_rn(__fadd_rn(sum.l, l), t.l)};
    }
    Two m = two_sum(__fmul_rn(sum.h, 1.f / D), eps);
    m.l = __fmaf_rn(sum.l, 1.f / D, m.l);
    // one step of Newton's on the fp32 root, its residual 1 - m r^2 in two parts
    const float r = rsqrtf(m.h);
    const Two r2 = two_mul(r, r);
    float e = __fmaf_rn(-m.h, r2.h, 1.f);
    e = __fmaf_rn(-m.h, r2.l, e);
    e = __fmaf_rn(-m.l, r2.h, e);
    return {r, isinf(m.h) ? 0.f : __fmul_rn(__fmul_rn(0.5f, r), e)};
}

// r (x w c + y v s), rounded to fp32 once.
__device__ __forceinline__ float turned(float x, float w, float c, float y, float v, float s, Two r) {
    const Two xw = two_mul(x, w), yv = two_mul(y, v);
    const Two p = two_mul(xw.h, c), q = two_mul(yv.h, s), t = two_sum(p.h, q.h);
    float l = __fadd_rn(__fmaf_rn(xw.l, c, p.l), __fmaf_rn(yv.l, s, q.l));
    l = __fadd_rn(l, t.l);
    const Two o = two_mul(t.h, r.h);
    l = __fmaf_rn(t.h, r.l, __fmaf_rn(l, r.h, o.l));
    return isfinite(o.h) ? __fadd_rn(o.h, l) : o.h;
}

template <int D, int kFormat, bool kInter>
__device__ __forceinline__ void turn_keys(const RotateArgs& a, const Lane<D, kInter>& p, int tok, int pos, int slot, int head, int end,
                                          float inv_k) {
    float c[16], s[16];
    load_angles(a, p, pos, c, s);
    for (; head < end; ++head) {
        uint32_t x[8], y[8];
        if (slot >= 0) load_block(x, a.k + (size_t)tok * a.k_stride + head * D + 16 * p.b);
        else zero(x);
        pairs_of(p, x, y);
        Two r = {1.f, 0.f};
        float w[16], wp[16];
        if (a.k_norm) {
            r = inverse_norm<D>(x, a.eps);
            if (r.h == 0.f) times_zero(x, y);
            load_norms(p, a.k_norm, w, wp);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = wp[j] = 1.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float f[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int d = 2 * j + i;
                f[i] = turned(bf16_at(x, d), w[d], c[d], bf16_at(y, d), wp[d], s[d], r);
            }
            x[j] = pack_bf16(f[0], f[1]);
        }
        if (slot < 0) continue;
        if (a.k_out) store_block(a.k_out + (size_t)tok * a.k_out_stride + head * D + 16 * p.b, x);
        append_block<D, kFormat, false>(kv_tile_ptr(a.kv, slot, head, kv_tile(D, kFormat).bytes), slot & 15, p.b, x, a.kv.k_scale, inv_k);
    }
}

template <int D, int kFormat, bool kInter>
__global__ void __launch_bounds__(kRotThreads) kv_rotate_kernel(const RotateArgs a) {
    pdl_wait_and_release();
    constexpr int kTokens = 32 / (D / 16);
    const Lane<D, kInter> p(a.rope_dim);
    const long long warps = (long long)gridDim.x * (kRotThreads / 32), groups = ((long long)a.n + kTokens - 1) / kTokens;
    const long long all = groups * a.units;
    const float inv_k = __frcp_rn(a.kv.k_scale), inv_v = __frcp_rn(a.kv.v_scale);
    for (long long u = (long long)blockIdx.x * (kRotThreads / 32) + (threadIdx.x >> 5); u < all; u += warps) {
        const int unit = (int)(u % a.units);
        const long long token = u / a.units * kTokens + (threadIdx.x & 31) / Lane<D, kInter>::kLanes;
        const int tok = (int)min(token, (long long)a.n - 1);
        int slot = token < a.n ? a.slots[tok] : -1, pos = -1;
        if (slot != -1) {
            bool bad = slot < 0 || (slot >> a.kv.page_shift) >= a.kv.n_pages;
            if (a.rope_dim) {
                pos = a.positions[tok];
                bad = bad || pos < 0 || pos >= a.n_positions;
            }
            if (bad) {
                if (unit == 0 && p.b == 0) atomicOr(a.kv.status, FT_DEV_BAD_ID);
                slot = pos = -1;
            }
        }
        if (unit < a.q_runs) {
            const int head = unit * a.run;
            turn_queries(a, p, tok, pos, slot >= 0, head, min(head + a.run, a.hq));
        } else if (unit < a.q_runs + a.k_runs) {
            const int head = (unit - a.q_runs) * a.run;
            turn_keys<D, kFormat, kInter>(a, p, tok, pos, slot, head, min(head + a.run, a.kv.hkv), inv_k);
        } else {
            int head = (unit - a.q_runs - a.k_runs) * a.run;
            const int end = min(head + a.run, a.kv.hkv);
            for (; head < end && slot >= 0; ++head) {
                uint32_t x[8];
                load_block(x, a.v + (size_t)tok * a.v_stride + head * D + 16 * p.b);
                append_block<D, kFormat, true>(kv_tile_ptr(a.kv, slot, head, kv_tile(D, kFormat).bytes), slot & 15, p.b, x, a.kv.v_scale, inv_v);
            }
        }
    }
}

template <int D, int kFormat>
struct Rotate {
    static cudaError_t run(RotateArgs& a, bool inter, cudaStream_t s) {
        const cudaError_t e = inter ? prepare<kv_rotate_kernel<D, kFormat, true>>() : prepare<kv_rotate_kernel<D, kFormat, false>>();
        if (e != cudaSuccess) return e;
        const long long groups = ((long long)a.n + 32 / (D / 16) - 1) / (32 / (D / 16));
        a.run = groups * (a.hq + 2 * a.kv.hkv) >= 32LL * sm_count() ? 4 : 1;
        a.q_runs = (a.hq + a.run - 1) / a.run;
        a.k_runs = (a.kv.hkv + a.run - 1) / a.run;
        a.units = a.q_runs + 2 * a.k_runs;
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
        !aligned(c.q_norm, 16) || !aligned(c.k_norm, 16) || !aligned(c.rope, 16))
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
