// What the attention kernels share: which keys a row tile needs, the rule of who sees whom,
// and the numbers of the running softmax.
#pragma once
#include <atomic>

#include "ft_kv.cuh"

namespace ft {

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
    uint32_t d;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(smem_u32(p)), "r"(rank));
    return d;
}


// Softmax in base 2: a weight is exp2(t - m + kHeadroom) with t = s * scale * log2(e) and a
// reference m that is raised (and everything rescaled) only when some t exceeds it by more than
// kHeadroom.  Weights are then at most 2^(2 kHeadroom) = 2^14 and a weight 2^-20 times the
// reference's is still a normal f16.  They are rounded to f16 because the products with V take f16: 2^-11 of a
// weight at most, below the output's own bf16 rounding (2^-9); their sum is taken before that rounding, in
// fp32.
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
    t.i0 = div_g(a, r * R);
    t.i1 = min(s.n - 1, div_g(a, r * R + R - 1));
    const int base = s.base;
    const int hi = a.tree ? s.len : min(s.len, base + t.i1 + 1);
    // a drafted token stands at base or after it
    const long long low = a.window > 0 ? (long long)base + (a.tree ? 0 : t.i0) - a.window + 1 : 0;
    const int lo = (int)max(low, 0LL);
    t.empty = hi <= 0 || (lo >= hi && a.n_sink == 0);     // nothing cached, or the window stands past the table
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
    const int i = div_g(a, row);
    if (i >= s.n) return r;            // padding
    const int base = s.base;
    int pos = base + i;
    r.lim = min(pos, s.len - 1);
    if (a.tree) {
        r.mask = a.tree[s.q0 + i];
        pos = base + __popcll(r.mask & ~(1ull << i));
        r.lim = s.len - 1;
    }
    // keys stand at 0 or after it, drafted ones from base on, which is below 0 where fewer tokens are cached than new
    if (a.window > 0) r.low = (int)max((long long)pos - a.window + 1, (long long)min(base, 0));
    return r;
}
// The rule for a key below base or without a tree.
__device__ __forceinline__ bool sees(const AttnArgs& a, const RowRule& r, int j) {
    return j <= r.lim && (j >= r.low || j < a.n_sink);
}
// Place of the drafted key j >= base under a tree (no mask has the 64th or a later one; of one past the rows no mask is known).
__device__ __forceinline__ int drafted_pos(const AttnArgs& a, const SeqInfo& s, int j) {
    const int jj = j - s.base;
    return s.base + (jj < min(kTreeMax, a.n_tokens - s.q0) ? __popcll(a.tree[s.q0 + jj] & ~(1ull << jj)) : 0);
}
// The rule for a drafted key j >= base, base <= j < len, that stands at place pos.
__device__ __forceinline__ bool sees_drafted(const AttnArgs& a, const RowRule& r, int base, int j, int pos) {
    return j - base < kTreeMax && (r.mask >> (j - base) & 1) && (pos >= r.low || j < a.n_sink);
}

// Under a tree: whether one of the rows whose masks are m[0..n) (the sequence's tokens from i0 on) sees one of the keys j0 to
// j0 + 15 below len.  Asked only where the table has no page for them, so that one which no row needs is no error; out of line,
// since its instructions among the kernels' cost more (windowed chunk 123 us instead of 116) than it ever takes.
static __device__ __noinline__ bool tree_sees_tile(const unsigned long long* m, int i0, int n, int left, int base, int len, int j0, int window,
                                                   int n_sink) {
    const int old = min(min(j0 + kKvTile, base), len) - 1;                     // the last key of the context among them
    const int d0 = max(j0, base) - base, d1 = min(min(j0 + kKvTile, len) - base, kTreeMax);
    auto place = [&](unsigned long long mask, int i) { return __popcll(mask & ~(1ull << i)); };
    for (int i = i0; i < i0 + n; ++i) {
        const long long low = window > 0 ? (long long)base + place(m[i], i) - window + 1 : 0;
        if (old >= j0 && (old >= low || j0 < n_sink)) return true;
        for (int d = d0; d < d1; ++d)
            if ((m[i] >> d & 1) && (base + (d < left ? place(m[d], d) : 0) >= low || base + d < n_sink)) return true;
    }
    return false;
}

// Powers of two that take a row's largest magnitude to [2^13, 2^14) and back: exact in f16 down to
// 2^-27 of the largest.  A row of zeros, or with an infinity, stays as it is.
struct RowScale {
    float down, up;
};
__device__ __forceinline__ RowScale row_scale(float amax) {
    const int ex = amax > 0.f && amax < INFINITY ? max((int)(__float_as_uint(amax) >> 23) - 140, -126) : 0;
    return {__uint_as_float((uint32_t)(127 - ex) << 23), __uint_as_float((uint32_t)(127 + ex) << 23)};
}

// N (4 or 8) output values, dims d.., of one row and query head from their weighted sums x, the
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
    if constexpr (N == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    if (d == 0 && a.lse)
        a.lse[token * a.hq + h] = l == 0.f ? -INFINITY : (m - kHeadroom + log2f(l)) * 0.693147180559945309417f;
}

// ---------------------------------------------------------------------------- the line of units
// A unit is a row tile of a sequence and a kv head; its work comes in blocks of kB keys.  Units are
// laid end to end, a unit being kCost + nt places long (its own start and end cost about as much as
// kCost blocks), and every CTA takes an equal share of the places.  Within a CTA the kW workers
// split the share: its tiles of the unit where the whole share lies in one unit (the workers then
// join in the CTA), its places otherwise.
// kSplit: CTAs of the joining kernel per share.  kByRow: a thread of the first kernel has a whole row, so
// partial sums stand as [D/4][R] groups of four values and neighbouring rows are written together.
template <int kB_, int kR_, int kW_, int kMin_, int kCost_, int kSplit_, bool kByRow_>
struct Line {
    static constexpr int kB = kB_, kR = kR_, kW = kW_, kMin = kMin_, kCost = kCost_, kSplit = kSplit_;
    static constexpr bool kByRow = kByRow_;
};

constexpr int kMaxShares = 640;        // CTAs of a launch
constexpr int kJoinThreads = 128;

// The sequences' first places: prefix[0..n_seqs], in shared memory.  Called by the whole CTA.
template <typename L>
__device__ __forceinline__ void line_prefix(const AttnArgs& a, long long* prefix, long long* scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if ((long long)a.max_q * a.G > 8 * L::kR) {           // many row tiles: a warp per sequence
        for (int s = warp; s < a.n_seqs; s += blockDim.x >> 5) {
            const SeqInfo si = seq_info(a, s);
            if (lane == 0 && si.bad && blockIdx.x == 0) atomicOr(a.kv.status, FT_DEV_BAD_ID);
            const int rt = (int)(((long long)si.n * a.G + L::kR - 1) / L::kR);
            long long t = 0;
            for (int r = lane; r < rt; r += 32) t += L::kCost + row_tile<L::kB>(a, si, r, L::kR).nt;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            if (lane == 0) prefix[s + 1] = t * a.kv.hkv;
        }
    } else {
        for (int s = threadIdx.x; s < a.n_seqs; s += blockDim.x) {
            const SeqInfo si = seq_info(a, s);
            if (si.bad && blockIdx.x == 0) atomicOr(a.kv.status, FT_DEV_BAD_ID);
            const int rt = (si.n * a.G + L::kR - 1) / L::kR;
            long long t = 0;
            for (int r = 0; r < rt; ++r) t += L::kCost + row_tile<L::kB>(a, si, r, L::kR).nt;
            prefix[s + 1] = t * a.kv.hkv;
        }
    }
    __syncthreads();
    const int per = (a.n_seqs + blockDim.x - 1) / blockDim.x;
    const int s0 = min((int)threadIdx.x * per, a.n_seqs), s1 = min(s0 + per, a.n_seqs);
    long long sum = 0;
    for (int s = s0; s < s1; ++s) sum += prefix[s + 1];
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    long long at = incl - sum;
    for (int w = 0; w < warp; ++w) at += scratch[w];
    if (threadIdx.x == 0) prefix[0] = 0;
    for (int s = s0; s < s1; ++s) {
        at += prefix[s + 1];
        prefix[s + 1] = at;
    }
    __syncthreads();
}

// The shares of the CTAs: cut(c) = first place of CTA c; they differ by one at most.
struct Shares {
    int nc;
    long long q, rem;
    __device__ __forceinline__ Shares(int nc_, long long q_, long long rem_) : nc(nc_), q(q_), rem(rem_) {}
    __device__ __forceinline__ Shares(long long total, unsigned grid, int least) {
        nc = (int)min((long long)grid, max((total + least - 1) / least, 1LL));
        q = total / nc;
        rem = total - q * nc;
    }
    __device__ __forceinline__ long long cut(int c) const { return q * c + min((long long)c, rem); }
    __device__ __forceinline__ int holder(long long place) const {
        const long long wide = rem * (q + 1);
        return (int)(place < wide ? place / (q + 1) : rem + (place - wide) / q);
    }
};

// Block of a unit that stands at a place (0 before its first block, nt from its end on).
template <typename L>
__device__ __forceinline__ int block_at(long long first, int nt, long long place) {
    return (int)min(max(place - first - L::kCost, 0LL), (long long)nt);
}

struct Unit {
    int s, r, h;
    long long first, end;    // its places in the line
    SeqInfo si;
    RowTile rt;
};

// The unit that holds a place.  Called by whole warps.
template <typename L>
__device__ __forceinline__ Unit find_unit(const AttnArgs& a, const long long* prefix, long long place) {
    Unit u;
    int lo = 0, hi = a.n_seqs;
    while (hi - lo > 1) {              // largest s with prefix[s] <= place
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= place) lo = mid; else hi = mid;
    }
    u.s = lo;
    u.si = seq_info(a, lo);
    u.first = prefix[lo];
    u.r = 0;
    if (u.si.n * (long long)a.G > 4 * L::kR) {            // many row tiles: 32 at a time, one per lane
        const int lane = threadIdx.x & 31;
        for (;; u.r += 32) {
            const int r = u.r + lane;
            const bool on = (long long)r * L::kR < (long long)u.si.n * a.G;
            const long long mine = on ? (long long)(L::kCost + row_tile<L::kB>(a, u.si, r, L::kR).nt) * a.kv.hkv : 0;
            long long incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long t = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += t;
            }
            const unsigned past = __ballot_sync(0xffffffffu, u.first + incl > place);
            const int pick = past ? __ffs(past) - 1 : 31;
            const long long before = __shfl_sync(0xffffffffu, past ? incl - mine : incl, pick);
            if (!past && (long long)(u.r + 32) * L::kR >= (long long)u.si.n * a.G) break;   // lengths changed under the call
            u.first += before;
            if (past) {
                u.r += pick;
                break;
            }
        }
        u.rt = row_tile<L::kB>(a, u.si, u.r, L::kR);
    } else {
        for (;; ++u.r) {
            u.rt = row_tile<L::kB>(a, u.si, u.r, L::kR);
            const long long all = (long long)(L::kCost + u.rt.nt) * a.kv.hkv;
            if (place < u.first + all || (u.r + 1) * L::kR >= u.si.n * a.G) break;
            u.first += all;
        }
    }
    const long long len = L::kCost + u.rt.nt;
    u.h = (int)min((place - u.first) / len, (long long)a.kv.hkv - 1);
    u.first += u.h * len;
    u.end = u.first + len;
    return u;
}

// The pieces of a unit: one per CTA whose share lies in the unit, one per worker elsewhere.
struct Piece {
    int v0, v1, slot;        // blocks [v0, v1), where its partial sums stand
};
template <typename L>
__device__ __forceinline__ Piece piece_of(const Shares& sh, long long first, int nt, int c, int w) {
    const long long c0 = sh.cut(c), c1 = sh.cut(c + 1);
    Piece p{0, 0, 0};
    if (c0 >= first && c1 <= first + L::kCost + nt) {
        if (w == 0) {
            p.v0 = block_at<L>(first, nt, c0);
            p.v1 = block_at<L>(first, nt, c1);
        }
    } else {
        p.v0 = block_at<L>(first, nt, c0 + (c1 - c0) * w / L::kW);
        p.v1 = block_at<L>(first, nt, c0 + (c1 - c0) * (w + 1) / L::kW);
    }
    // a share holds at most one unit's later piece and one unit's first
    p.slot = 2 * (L::kW * c + w) + (p.v0 > 0 ? 0 : 1);
    return p;
}

// Where the four values d.. of a row stand among a piece's.
template <typename L, int D>
__device__ __forceinline__ int piece_at(int row, int d) { return L::kByRow ? d / 4 * L::kR + row : row * (D / 4) + d / 4; }

// Partial sums of one piece of a unit in the workspace: [R] (reference, sum of weights), R D values.
template <int D, int R>
__device__ __forceinline__ float* partial(const AttnArgs& a, int slot) { return a.parts + (size_t)slot * (R * (D + 2)); }

// What the second kernel needs to know of a unit that is cut (ca, cb: its first and last CTA).
struct __align__(16) JoinTask {
    long long q, rem, first;
    int nc, nt, q0, n, r, h, ca, cb, on;
};

__device__ __forceinline__ JoinTask join_task(const Shares& sh, const Unit& u, int ca, int cb) {
    JoinTask j;
    j.q = sh.q; j.rem = sh.rem; j.nc = sh.nc;
    j.first = u.first; j.nt = u.rt.nt;
    j.q0 = u.si.q0; j.n = u.si.n; j.r = u.r; j.h = u.h;
    j.ca = ca; j.cb = cb; j.on = 1;
    return j;
}

// Slice `part` of `parts` of unit u's output from its pieces, by n_threads threads (a multiple of
// 32, whole warps, `sync` between them).  A team of threads takes four values of a row: thread k of it
// the pieces k, k + team, ..., then one of them their sums in order, so the order is fixed.  Teams
// are as large as the slice leaves threads for; neighbouring threads have neighbouring values of the
// same piece, so that partial sums are read in whole sectors.  slots: shared, 2 kW + CTAs of the
// unit; sums: shared, one per thread.
struct TeamSum {
    float m, l;
    float4 x;
};
template <typename L, int D, typename Sync>
__device__ __forceinline__ void join_slice(const AttnArgs& a, const JoinTask& u, int part, int parts, int thread,
                                           int n_threads, int* slots, TeamSum* sums, Sync sync) {
    constexpr int R = L::kR;
    const Shares sh(u.nc, u.q, u.rem);
    const int ca = u.ca, cb = u.cb;
    // pieces: the workers of the first CTA, one each of the CTAs between, the workers of the last
    const int n = cb == ca ? L::kW : 2 * L::kW + cb - ca - 1;
    for (int k = thread; k < n; k += n_threads) {
        const int mid = k - L::kW, c = mid < 0 ? ca : min(ca + 1 + mid, cb);
        const Piece p = piece_of<L>(sh, u.first, u.nt, c, mid < 0 ? k : max(mid - (cb - ca - 1), 0));
        slots[k] = p.v0 == p.v1 ? -1 : p.v1 - p.v0 == u.nt ? -2 : p.slot;
    }
    sync();
    for (int w = 0; w < L::kW; ++w)
        if (slots[w] == -2 || slots[n - 1 - w] == -2) return;                // not cut: written already
    // a slice is at least 128 contiguous bytes of every piece
    const int rows = min(R, u.n * a.G - u.r * R), groups = rows * (D / 4);
    parts = min(parts, groups / 8);
    if (part >= parts) return;
    const int ga = (int)((long long)groups * part / parts), gb = (int)((long long)groups * (part + 1) / parts);
    int team = 1;
    while (team < 32 && team < n && (gb - ga) * team < n_threads) team *= 2;
    const int wide = n_threads / team, mine = thread % wide, first = thread / wide;
    for (int g0 = ga; g0 < gb; g0 += wide) {
        const int e = min(g0 + mine, gb - 1);
        const int row = L::kByRow ? e % rows : e / (D / 4), d = (L::kByRow ? e / rows : e % (D / 4)) * 4;
        float m = kNoRef, l = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kBatch = 8;                         // pieces in flight
        for (int k0 = first; k0 < n; k0 += team * kBatch) {
            float pm[kBatch], pl[kBatch];
            float4 y[kBatch];
            float mm = m;
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int k = k0 + b * team, slot = k < n ? slots[k] : -1;
                pm[b] = kNoRef;
                pl[b] = 0.f;
                y[b] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (slot >= 0) {
                    const float* src = partial<D, R>(a, slot);
                    const float2 ml = __ldcg(reinterpret_cast<const float2*>(src) + row);
                    pm[b] = ml.x;
                    pl[b] = ml.y;
                    y[b] = __ldcg(reinterpret_cast<const float4*>(src + 2 * R) + piece_at<L, D>(row, d));
                }
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) mm = fmaxf(mm, pm[b]);
            float f = ex2(m - mm);
            m = mm;
            l *= f;
            x.x *= f; x.y *= f; x.z *= f; x.w *= f;
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                f = ex2(pm[b] - mm);
                l += pl[b] * f;
                x.x += y[b].x * f; x.y += y[b].y * f; x.z += y[b].z * f; x.w += y[b].w * f;
            }
        }
        if (team > 1) {
            sums[thread] = {m, l, x};
            sync();
            if (first == 0) {
                for (int k = 1; k < team; ++k) {
                    const TeamSum o = sums[k * wide + mine];
                    const float mm = fmaxf(m, o.m), f = ex2(m - mm), of = ex2(o.m - mm);
                    m = mm;
                    l = l * f + o.l * of;
                    x.x = x.x * f + o.x.x * of; x.y = x.y * f + o.x.y * of; x.z = x.z * f + o.x.z * of; x.w = x.w * f + o.x.w * of;
                }
            }
            sync();
        }
        if (g0 + mine < gb && first == 0) {
            const int grow = u.r * R + row;
            store_out<4>(a, (size_t)(u.q0 + div_g(a, grow)), u.h * a.G + grow - div_g(a, grow) * a.G, D, d, &x.x, m, l);
        }
    }
}

// The second kernel: CTA c joins a slice of the unit that holds the first place of its share and
// began before it (the CTAs behind the one that the unit began in take a slice each), and each warp
// the unit that began and ends in the CTA's share and that its worker's place is the first cut in.
template <typename L, int D>
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(const AttnArgs a) {
    __shared__ int slots[2 * L::kW + kMaxShares], warp_slots[L::kW][L::kW];
    __shared__ TeamSum sums[kJoinThreads];
    pdl_wait_and_release();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x / L::kSplit, sub = blockIdx.x % L::kSplit;
    constexpr int kParts = L::kW == 1 ? L::kSplit : L::kSplit - 1;       // the last CTA of a share has its warps' units
    const JoinTask all = a.tasks[L::kW * cta];
    JoinTask mine;
    mine.on = 0;
    if (warp > 0 && warp < L::kW && sub == L::kSplit - 1) mine = a.tasks[L::kW * cta + warp];
    if (all.on && (L::kW == 1 || sub < L::kSplit - 1))
        join_slice<L, D>(a, all, (cta - all.ca - 1) * kParts + sub, (all.cb - all.ca) * kParts, threadIdx.x, kJoinThreads,
                         slots, sums, [] { __syncthreads(); });
    if (mine.on) {
        __syncwarp();
        join_slice<L, D>(a, mine, 0, 1, lane, 32, warp_slots[warp], sums + 32 * warp, [] { __syncwarp(); });
    }
}

// ---------------------------------------------------------------------------- launches

// Blocks of `keys` keys that a unit has at most, as far as the host knows.
inline long long most_blocks(const AttnArgs& a, int keys) {
    const long long len = (long long)a.table_stride << a.kv.page_shift, n = (len + keys - 1) / keys;
    return a.window > 0 ? min(n, ((long long)a.window + a.max_q + a.n_sink) / keys + 4) : n;
}

// The launch of a direct kernel: a cluster of a.split CTAs per unit.
struct DirectLaunch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2] = {};
    DirectLaunch(unsigned grid, int split, int threads, size_t smem, cudaStream_t s) {
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = split;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = split > 1 ? 2 : 1;
    }
    DirectLaunch(const AttnArgs& a, int threads, size_t smem, cudaStream_t s)
        : DirectLaunch((unsigned)(a.n_seqs * a.kv.hkv * a.row_tiles * a.split), a.split, threads, smem, s) {}
    DirectLaunch(const DirectLaunch&) = delete;
};

// CTAs that are resident at once: by shares, and direct by the log2 of a cluster's CTAs (clusters lie within a
// part of the GPU, so the largest leave SMs out).
struct Room {
    int grid, room[5];
};
// Looked up, with the kernels' attributes set, once per device.  direct may be NULL.
struct RoomStore {
    std::atomic<int> known[kMaxDevices][6];
    using Kernel = void (*)(AttnArgs);
    cudaError_t get(Room& r, Kernel shares, Kernel direct, Kernel join, int threads, size_t smem, int per_sm, int most) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
        std::atomic<int>(&at)[6] = known[dev];
        if (!at[0].load(std::memory_order_acquire)) {
            int n = 0;
            if ((e = cudaFuncSetAttribute(shares, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess ||
                (e = all_shared(shares)) != cudaSuccess || (e = all_shared(join)) != cudaSuccess ||
                (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, shares, threads, smem)) != cudaSuccess)
                return e;
            const int grid = min(sm_count() * min(n, per_sm), most);
            if (grid < 1) return cudaErrorInvalidConfiguration;
            at[1].store(grid, std::memory_order_relaxed);
            if (direct && ((e = cudaFuncSetAttribute(direct, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess ||
                           (e = cudaFuncSetAttribute(direct, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess ||
                           (e = all_shared(direct)) != cudaSuccess))
                return e;
            for (int x = 1; direct && x < 5; ++x) {
                DirectLaunch l((unsigned)(grid >> x << x), 1 << x, threads, smem, nullptr);
                l.cfg.attrs = l.attr + 1;
                l.cfg.numAttrs = 1;
                if ((e = cudaOccupancyMaxActiveClusters(&n, direct, &l.cfg)) != cudaSuccess) return e;
                at[1 + x].store(min(n << x, grid), std::memory_order_relaxed);
            }
            at[0].store(1, std::memory_order_release);
        }
        r.grid = at[1].load(std::memory_order_relaxed);
        for (int x = 0; x < 5; ++x) r.room[x] = at[1 + x].load(std::memory_order_relaxed);
        return cudaSuccess;
    }
};

}  // namespace ft
