// Attention over the quantised key/value cache.
//
// o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(t_ij - m_i),  t_ij = log2(e) scale q_i.k_j: one pass
// over the keys with a running reference m_i and sum; partial (m, sum, o) of two key ranges join
// by rescaling both to the larger m.
//
// Few rows share a key (a decode step has G = query heads per kv head of them), so the pass is
// bound by the bytes of the cache and by unpacking them: 9/16 byte per element is 41 elements
// per clock and SM at the copy rate.  Layout of the work:
//   * A warp owns a run of 16-token tiles.  Tiles are contiguous records; the warp streams them
//     through a ring in shared memory with one bulk copy each, several in flight, and no barrier
//     but its own.
//   * Keys stand on the m side of the matrix instruction (m16n8k16, f16 in, fp32 sums):
//     S^T = K Q^T and O^T = V^T P^T with 8 rows on the n side, so a group of 8 query heads wastes
//     nothing.  A tile's bytes are stored in the order in which the lanes' fragments need them:
//     16-byte shared-memory loads, no shuffles; P^T is the transpose (movmatrix) of S^T's
//     accumulators.
//   * Codes become f16 by the conversion instructions; code * scale is exact in f16 (2 + 4
//     significant bits, 2^-10 .. 2688); q is scaled by a power of two per row into f16's range.
//   * The (sequence, row tile, kv head) units are laid end to end, each as long as its tiles plus
//     a constant for its own start and end, and every CTA takes an equal share of the line, so
//     ragged batches balance.  A unit cut by a share's end leaves partial sums in the workspace;
//     a second kernel, a programmatic dependent, joins them in a fixed order, each of its CTAs a slice of the
//     unit that a share began inside.
//   * Short sequences go without the line: a cluster of CTAs per unit (plan_direct).
//
// 32 sequences of up to 32768 tokens, 8 heads of 128 in 8 bits (292 MB): 58 us, 5.0 TB/s; the kernel reads at 84 % of
// the copy rate while all its warps run, the rest is the start, the ragged end and the second kernel (about 10
// us).  One sequence of 262145, 2 heads of 256 in 4 bits (151 MB): 43 us, 3.5 TB/s, bound by the 633
// instructions of a tile (8192 codes; 2.0 issued per clock and SM by 8 warps, all that 238 registers leave
// room for).  One of 4096: 10 us, the latency of a launch, a tile's chain and the cluster's join.
#include <atomic>

#include "ft_kv_attn.cuh"

namespace ft {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kMaxPerSm = 4;           // CTAs
// at least 2 places of the line per warp; a unit's start and end cost about 8 tiles (a ragged batch of 32 without that
// weight: 116 us, with it 66 us)
template <int NT>
using RowsLine = Line<kKvTile, 8 * NT, kWarps, 2 * kWarps, 8, 2, false>;

// Waits give up after about two seconds.
constexpr long long kWaitClocks = 1LL << 32;
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
    if (mbar_try(bar, parity)) return true;
    const long long from = clock64();
    do {
        if (mbar_try(bar, parity)) return true;
    } while (clock64() - from < kWaitClocks);
    return false;
}

// Four f16 pairs from 8 E2M1 codes (a 32-bit word); two from 4 E4M3 codes.
__device__ __forceinline__ void e2m1_unpack(uint32_t w, uint32_t (&o)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(w));
}
__device__ __forceinline__ void e4m3_unpack(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Tiles in flight per warp, about 9 to 16 KB.
constexpr int stages(int D, int format) {
    const int b = kv_tile(D, format).bytes;
    return b <= 1152 ? 8 : b <= 2304 ? 4 : b <= 4096 ? 3 : 2;
}

// Floats of a row where the warps of a CTA join: [D/16][g 8][2] (dims g D/8 + 2 i), padded so that the
// 32 lanes of a store (8 g, 4 rows) spread over the banks.
constexpr int join_row(int D) { return D + 8; }
template <int D>
__device__ __forceinline__ int join_at(int row, int i, int g) { return row * join_row(D) + i * 16 + g * 2; }
// The e-th four values of a row block: row, first dim, place of the first two (the others: 16 floats on).
template <int D>
__device__ __forceinline__ void join_group(int e, int& row, int& d, int& at) {
    row = e / (D / 4);
    const int q = e % (D / 4), g = q & 7, i = (q >> 3) * 2;
    d = g * (D / 8) + 2 * i;
    at = join_at<D>(row, i, g);
}

// Heads of 256: q's fragments (32 registers a row tile) stay in shared memory, so that three CTAs fit.
constexpr bool q_in_smem(int D) { return D == 256; }

template <int D, int kFormat, int NT>
constexpr size_t rows_smem() {
    const size_t ring = (size_t)kWarps * stages(D, kFormat) * kv_tile(D, kFormat).bytes;
    const size_t join = (size_t)kWarps * 8 * NT * join_row(D) * 4;
    return (ring > join ? ring : join) + (q_in_smem(D) ? (size_t)kWarps * NT * D * 16 : 0);
}

// CTAs per SM that the register allocation aims at.  Heads of 256 leave three of them too few registers: 16
// sequences of 8192 with 2 heads, 4-bit, 31.6 us with three and 24.8 with two.
constexpr int rows_ctas(int D, int NT) { return D == 256 ? 2 : D == 128 ? (NT == 1 ? 3 : 2) : NT == 1 ? 4 : 3; }

// A unit's sums from the CTAs of its cluster (each has its own in x and ml): a slice of the
// values per CTA.  A team of lanes takes four values: lane k of it the ranks k, k + team, ..., then a
// butterfly, so the order of the sums is fixed.
template <int D, int R>
__device__ __forceinline__ void join_cluster(const AttnArgs& a, const Unit& u, const float* x, const float2* ml) {
    cluster_sync();
    const int rank = blockIdx.x % a.split;
    const int groups = min(R, u.si.n * a.G - u.r * R) * (D / 4);
    const int ga = groups * rank / a.split, gb = groups * (rank + 1) / a.split;
    int team = 1;
    while (team < a.split && team * 2 * (gb - ga) <= kThreads) team *= 2;
    for (int g0 = ga; g0 < gb; g0 += kThreads / team) {
        int row, d, at;
        join_group<D>(min(g0 + (int)threadIdx.x / team, gb - 1), row, d, at);
        float m = kNoRef, l = 0.f;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int c = threadIdx.x & (team - 1); c < a.split; c += team) {
            float2 p;
            float4 y;
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(p.x), "=f"(p.y) : "r"(cluster_addr(ml + row, c)));
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(y.x), "=f"(y.y) : "r"(cluster_addr(x + at, c)));
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(y.z), "=f"(y.w) : "r"(cluster_addr(x + at + 16, c)));
            const float mm = fmaxf(m, p.x), f = ex2(m - mm), g = ex2(p.x - mm);
            m = mm;
            l = l * f + p.y * g;
            sum.x = sum.x * f + y.x * g; sum.y = sum.y * f + y.y * g; sum.z = sum.z * f + y.z * g; sum.w = sum.w * f + y.w * g;
        }
        for (int o = 1; o < team; o <<= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, m, o), mm = fmaxf(m, om), f = ex2(m - mm), of = ex2(om - mm);
            const float ol = __shfl_xor_sync(0xffffffffu, l, o);
            const float4 y = make_float4(__shfl_xor_sync(0xffffffffu, sum.x, o), __shfl_xor_sync(0xffffffffu, sum.y, o),
                                         __shfl_xor_sync(0xffffffffu, sum.z, o), __shfl_xor_sync(0xffffffffu, sum.w, o));
            m = mm;
            l = l * f + ol * of;
            sum.x = sum.x * f + y.x * of; sum.y = sum.y * f + y.y * of; sum.z = sum.z * f + y.z * of; sum.w = sum.w * f + y.w * of;
        }
        if (g0 + (int)threadIdx.x / team < gb && (threadIdx.x & (team - 1)) == 0) {
            const int grow = u.r * R + row;
            store_out<4>(a, (size_t)(u.si.q0 + div_g(a, grow)), u.h * a.G + grow - div_g(a, grow) * a.G, D, d, &sum.x, m, l);
        }
    }
    cluster_sync();                                       // the others may still read this CTA's sums
}

}  // namespace

// kDirect: short sequences.  A cluster of a.split CTAs (1 to 16) takes one unit, its CTAs join through
// distributed shared memory, and there is no line of shares, no workspace and no second kernel.
template <int D, int kFormat, int NT, bool kDirect>
__global__ void __launch_bounds__(kThreads, rows_ctas(D, NT)) kv_rows_kernel(const AttnArgs a) {
    using L = RowsLine<NT>;
    constexpr int R = 8 * NT, kStages = stages(D, kFormat);
    constexpr KvTile kT = kv_tile(D, kFormat);
    constexpr bool kFour = kFormat == FT_KV_NVFP4;
    constexpr int kKW = (kFour ? D / 4 : D / 2) / 4;       // 32-bit words of K codes per lane (both tokens)
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long prefix[kDirect ? 1 : kMaxSeqs + 1], scratch[kWarps];
    __shared__ __align__(8) uint64_t bars[kWarps][kStages];
    __shared__ float join_m[kWarps][R], join_l[kWarps][R];
    __shared__ float2 row_ml[R];                          // the CTA's references and sums

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t bar0 = smem_u32(&bars[warp][0]);
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" :: "r"(bar0 + 8 * s));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    pdl_wait_and_release();
    Unit u;
    long long c0 = 0, c1 = 0, w0 = 0, w1 = 0;             // the CTA's and the warp's places in the line
    bool whole = true;                                    // the CTA's share lies in one unit: its warps split the tiles
    const int cta = blockIdx.x;
    JoinTask* task = a.tasks + kWarps * cta + warp;
    Shares shares(1, 1LL, 0LL);
    if constexpr (kDirect) {
        const int id = cta / a.split;
        u.h = id % a.kv.hkv;
        u.r = id / a.kv.hkv % a.row_tiles;
        u.s = id / a.kv.hkv / a.row_tiles;
        u.si = seq_info(a, u.s);
        if (u.si.bad && threadIdx.x == 0) atomicOr(a.kv.status, FT_DEV_BAD_ID);
        if (u.r * R >= u.si.n * a.G) return;              // the whole cluster
        u.rt = row_tile<L::kB>(a, u.si, u.r, R);
        u.first = 0;
        u.end = 1;
    } else {
        line_prefix<L>(a, prefix, scratch);
        const long long total = prefix[a.n_seqs];
        shares = Shares(total, gridDim.x, L::kMin);
        if (total == 0 || cta >= shares.nc) {
            if (lane == 0) task->on = 0;
            return;
        }
        c0 = shares.cut(cta);
        c1 = shares.cut(cta + 1);
        u = find_unit<L>(a, prefix, c0);
        whole = c1 <= u.end;
        w0 = c0 + (c1 - c0) * warp / kWarps;
        w1 = c0 + (c1 - c0) * (warp + 1) / kWarps;
    }
    uint8_t* ring = smem + (size_t)warp * kStages * kT.bytes;
    const uint32_t ring_u32 = smem_u32(ring);
    uint2* q_frag = reinterpret_cast<uint2*>(smem + rows_smem<D, kFormat, NT>()) - (kWarps - warp) * NT * (D / 16) * 32;   // heads of 256
    uint32_t parity = 0;                                  // bit s: phase of stage s to wait for
    int next = 0;                                         // stage that the next tile takes

    // The cut at the start of the CTA's share goes through unit v, or the cut at the start of the
    // warp's is the first through a unit that begins and ends in the CTA's.
    auto note_task = [&](const Unit& v) {
        if (lane != 0) return;
        if (warp == 0 ? v.first < c0 : !whole && v.first < w0 && v.first >= c0 + (c1 - c0) * (warp - 1) / kWarps && v.end <= c1)
            *task = join_task(shares, v, warp == 0 ? shares.holder(v.first) : cta, warp == 0 ? shares.holder(v.end - 1) : cta);
        else
            task->on = 0;
    };

    for (long long pos = w0; pos < w1 || whole; pos = u.end) {
        if (!whole && (pos >= u.end || pos < u.first)) u = find_unit<L>(a, prefix, pos);
        int v0 = block_at<L>(u.first, u.rt.nt, whole ? c0 : pos), v1 = block_at<L>(u.first, u.rt.nt, whole ? c1 : w1);
        if constexpr (kDirect) {
            v0 = (int)((long long)u.rt.nt * (cta % a.split) / a.split);
            v1 = (int)((long long)u.rt.nt * (cta % a.split + 1) / a.split);
        }
        const int cv0 = v0, cv1 = v1;
        if (whole) {
            v0 = cv0 + (cv1 - cv0) * warp / kWarps;
            v1 = cv0 + (cv1 - cv0) * (warp + 1) / kWarps;
        }
        if (!kDirect && cv0 == cv1) {                     // none of the unit's tiles
            if (pos == w0) note_task(u);
            if (whole) break;
            continue;
        }
        const int base = u.si.base, row0 = u.r * R;

        // ---------------------------------------------------------------- the rows' loads, the first copies
        uint4 raw[NT][D / 32];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = row0 + 8 * nt + g, i = div_g(a, row);
            const __nv_bfloat16* src = a.q + (size_t)(u.si.q0 + i) * a.q_stride + (size_t)(u.h * a.G + row - i * a.G) * D + t * (D / 4);
#pragma unroll
            for (int e = 0; e < D / 32; ++e)
                raw[nt][e] = i < u.si.n ? *reinterpret_cast<const uint4*>(src + 8 * e) : make_uint4(0, 0, 0, 0);
        }
        // lane x of the warp holds the page of tile v0 + 32 * (group of 32) + x
        const int32_t* table = a.table + (size_t)u.s * a.table_stride;
        const int per = a.kv.page_shift - 4;              // log2 of the tiles of a page
        int page = -1, group = -1;
        auto issue = [&](int v) {                         // start the copy of tile v, every lane of the warp
            const int gr = (v - v0) >> 5;
            if (gr != group) {
                group = gr;
                const int mine = v0 + 32 * gr + lane;
                page = -1;
                if (mine < v1) {
                    page = table[u.rt.block(mine) >> per];
                    if (page < 0 || page >= a.kv.n_pages) {
                        if (!a.tree || tree_sees_tile(a.tree + u.si.q0, u.rt.i0, u.rt.i1 + 1 - u.rt.i0, a.n_tokens - u.si.q0, base, u.si.len,
                                                      u.rt.block(mine) * kKvTile, a.window, a.n_sink))
                            atomicOr(a.kv.status, FT_DEV_BAD_ID);
                        page = -1;
                    }
                }
            }
            const int pg = __shfl_sync(0xffffffffu, page, (v - v0) & 31);
            if (lane == 0) {
                const uint32_t bar = bar0 + 8 * next;
                if (pg >= 0) {
                    const int blk = u.rt.block(v);
                    const uint8_t* src = a.kv.pool + ((((size_t)pg * a.kv.hkv + u.h) << per) + (blk & ((1 << per) - 1))) * kT.bytes;
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(kT.bytes) : "memory");
                    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                                 :: "r"(ring_u32 + next * kT.bytes), "l"(src), "r"(kT.bytes), "r"(bar) : "memory");
                } else {
                    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
                }
            }
            next = next + 1 == kStages ? 0 : next + 1;
            return pg >= 0;
        };
        const int vend = u.rt.empty ? v0 : v1;
        uint32_t present = 0;                             // bit of a stage: its tile's page is one of the cache's
        int cur = next;
        for (int v = v0; v < min(vend, v0 + kStages); ++v) {
            const int st = next;
            if (issue(v)) present |= 1u << st;
        }
        // ---------------------------------------------------------------- the rows
        RowRule rule[NT][2];
        uint32_t qf[NT][q_in_smem(D) ? 1 : D / 16][2];
        float coef[NT][2], m[NT][2], l[NT][2];
        int lim_min = 0x7fffffff, low_max = 0;            // keys that every row sees: below lim_min, from low_max
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float amax = 0.f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                const uint32_t wd[4] = {raw[nt][e].x, raw[nt][e].y, raw[nt][e].z, raw[nt][e].w};
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(wd[y] << 16)), fabsf(__uint_as_float(wd[y] & 0xFFFF0000u))));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const RowScale rs = row_scale(amax);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                const uint32_t wd[4] = {raw[nt][e].x, raw[nt][e].y, raw[nt][e].z, raw[nt][e].w};
                uint32_t o[4];
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    o[y] = pack_f16(__uint_as_float(wd[y] << 16) * rs.down, __uint_as_float(wd[y] & 0xFFFF0000u) * rs.down);
                if constexpr (q_in_smem(D)) {
                    q_frag[(nt * (D / 16) + 2 * e) * 32 + lane] = make_uint2(o[0], o[1]);
                    q_frag[(nt * (D / 16) + 2 * e + 1) * 32 + lane] = make_uint2(o[2], o[3]);
                } else {
                    qf[nt][2 * e][0] = o[0]; qf[nt][2 * e][1] = o[1];
                    qf[nt][2 * e + 1][0] = o[2]; qf[nt][2 * e + 1][1] = o[3];
                }
            }
            const float c = a.scale * a.kv.k_scale * 1.44269504088896340736f * rs.up;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                coef[nt][b] = __shfl_sync(0xffffffffu, c, 4 * (2 * t + b));
                const int mine = row0 + 8 * nt + 2 * t + b;
                rule[nt][b] = row_rule(a, u.si, mine);
                if (div_g(a, mine) < u.si.n) {
                    lim_min = min(lim_min, a.tree ? min(rule[nt][b].lim, base - 1) : rule[nt][b].lim);
                    low_max = max(low_max, rule[nt][b].low);
                }
                m[nt][b] = kNoRef;
                l[nt][b] = 0.f;
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, o));
            low_max = max(low_max, __shfl_xor_sync(0xffffffffu, low_max, o));
        }
        float acc[D / 16][NT][4];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.f;

        if (!kDirect && pos == w0) note_task(u);          // while the first tiles are under way

        auto q_of = [&](int nt, int x) {                  // the lane's fragment of k-step x
            if constexpr (q_in_smem(D)) return q_frag[(nt * (D / 16) + x) * 32 + lane];
            else return make_uint2(qf[nt][x][0], qf[nt][x][1]);
        };

        // ---------------------------------------------------------------- the keys
        bool gave_up = false;
        for (int v = v0; v < vend; ++v) {
            const uint32_t bar = bar0 + 8 * cur;
            if (!__all_sync(0xffffffffu, mbar_wait(bar, parity >> cur & 1))) {    // give up, once the copies in flight have had their time
                for (int x = 0; x < kStages && x < vend - v; ++x, cur = cur + 1 == kStages ? 0 : cur + 1)
                    mbar_wait(bar0 + 8 * cur, parity >> cur & 1);
                if (lane == 0) atomicOr(a.kv.status, FT_DEV_TIMEOUT);
                gave_up = true;
                break;
            }
            parity ^= 1u << cur;
            const uint8_t* tile = ring + cur * kT.bytes;
            const int j0 = u.rt.block(v) * kKvTile;
            const bool have = present >> cur & 1;

            // S^T = K Q^T
            float sc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
            {
                uint32_t kw[kKW];
#pragma unroll
                for (int x = 0; x < kKW / 4; ++x) {
                    const uint4 w = *reinterpret_cast<const uint4*>(tile + x * 512 + lane * 16);
                    kw[4 * x] = w.x; kw[4 * x + 1] = w.y; kw[4 * x + 2] = w.z; kw[4 * x + 3] = w.w;
                }
                if constexpr (kFour) {
                    uint32_t sw[2] = {0, 0};              // the D/32 scale bytes of the lane: [token 2][D/64]
                    const uint8_t* sp = tile + kT.k_scales + lane * (D / 32);
                    if constexpr (D == 64) sw[0] = *reinterpret_cast<const uint16_t*>(sp);
                    if constexpr (D == 128) sw[0] = *reinterpret_cast<const uint32_t*>(sp);
                    if constexpr (D == 256) {
                        const uint2 w = *reinterpret_cast<const uint2*>(sp);
                        sw[0] = w.x; sw[1] = w.y;
                    }
#pragma unroll
                    for (int b = 0; b < D / 64; ++b) {    // block b of the lane's dims: 4 k-steps
                        uint32_t s2[2];
#pragma unroll
                        for (int v2 = 0; v2 < 2; ++v2) {
                            const int at = v2 * (D / 64) + b;
                            const uint32_t byte = sw[at >> 2] >> (8 * (at & 3)) & 255u;
                            uint32_t hi;
                            e4m3_unpack(byte | byte << 8, s2[v2], hi);
                        }
                        uint32_t f[2][8];
#pragma unroll
                        for (int v2 = 0; v2 < 2; ++v2)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                uint32_t o[4];
                                e2m1_unpack(kw[v2 * (D / 32) + 2 * b + x], o);
#pragma unroll
                                for (int y = 0; y < 4; ++y) f[v2][4 * x + y] = hmul2(o[y], s2[v2]);
                            }
#pragma unroll
                        for (int x = 0; x < 4; ++x)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                            {
                                const uint2 q = q_of(nt, 4 * b + x);
                                mma(sc[nt], f[0][2 * x], f[1][2 * x], f[0][2 * x + 1], f[1][2 * x + 1], q.x, q.y);
                            }
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        uint32_t a0, a1, a2, a3;
                        e4m3_unpack(kw[x], a0, a2);
                        e4m3_unpack(kw[D / 16 + x], a1, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint2 q = q_of(nt, x);
                            mma(sc[nt], a0, a1, a2, a3, q.x, q.y);
                        }
                    }
                }
            }

            // weights.  sc[nt][0..1]: key j0 + g, rows 2t, 2t+1; [2..3]: key j0 + g + 8
            const bool edge = !have || j0 + 15 > lim_min || (j0 < low_max && j0 + 15 >= a.n_sink);
            bool over = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[nt][e] = __fmul_rn(sc[nt][e], coef[nt][e & 1]);   // not fused: t - m stays exact near m
            if (edge) {
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {
                    const int j = j0 + g + 8 * e2;
                    const bool drafted = a.tree && j >= base && j < u.si.len;
                    const int jp = drafted && a.window > 0 ? drafted_pos(a, u.si, j) : 0x7fffffff;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const bool ok2 = have && (drafted ? sees_drafted(a, rule[nt][b], base, j, jp) : sees(a, rule[nt][b], j));
                            if (!ok2) sc[nt][2 * e2 + b] = -INFINITY;
                        }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) over |= sc[nt][e] - m[nt][e & 1] > kHeadroom;
            if (__any_sync(0xffffffffu, over)) {          // raise the references to the rows' maxima
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        float x = fmaxf(sc[nt][b], sc[nt][2 + b]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                        x = fmaxf(x, m[nt][b]);
                        const float f = ex2(m[nt][b] - x);
                        m[nt][b] = x;
                        l[nt][b] *= f;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            acc[i][nt][b] *= f;
                            acc[i][nt][2 + b] *= f;
                        }
                    }
            }
            uint32_t pf[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = ex2(sc[nt][e] - m[nt][e & 1] + kHeadroom);
                    l[nt][e & 1] += p[e];
                }
                pf[nt][0] = transpose8x8(pack_f16(p[0], p[1]));
                pf[nt][1] = transpose8x8(pack_f16(p[2], p[3]));
            }

            // O^T += V^T P^T.  The lane holds tokens 2t, 2t+1, 2t+8, 2t+9 and dims g D/8 ..
            // A key that a row does not see has weight 0, but its slot may never have been written (or its tile be a
            // stale one), and a NaN among its bytes times 0 would be a NaN: there they count as 0.
            if constexpr (kFour) {
                uint32_t vw[D / 16];                      // [token 4][D/64 words]
                if constexpr (D == 64) {
                    const uint4 w = *reinterpret_cast<const uint4*>(tile + kT.code_bytes + lane * 16);
                    vw[0] = w.x; vw[1] = w.y; vw[2] = w.z; vw[3] = w.w;
                } else {
#pragma unroll
                    for (int x = 0; x < D / 64; ++x) {
                        const uint4 w = *reinterpret_cast<const uint4*>(tile + kT.code_bytes + x * 512 + lane * 16);
                        vw[4 * x] = w.x; vw[4 * x + 1] = w.y; vw[4 * x + 2] = w.z; vw[4 * x + 3] = w.w;
                    }
                }
                constexpr int kBlocks = D == 256 ? 2 : 1; // blocks of 16 dims that the lane's dims touch
                constexpr int kPer = D / 64 / kBlocks;    // words per token and block: 1, 2, 2
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    const int blk = D == 64 ? g >> 1 : D == 128 ? g : 2 * g + b;
                    uint32_t sw = *reinterpret_cast<const uint32_t*>(tile + kT.v_scales + (blk * 4 + t) * 4);
                    if (edge) sw = e4m3_numbers(sw);
                    uint32_t s2[4];
                    {
                        uint32_t p01, p23;
                        e4m3_unpack(sw, p01, p23);
                        s2[0] = __byte_perm(p01, 0, 0x1010); s2[1] = __byte_perm(p01, 0, 0x3232);
                        s2[2] = __byte_perm(p23, 0, 0x1010); s2[3] = __byte_perm(p23, 0, 0x3232);
                    }
#pragma unroll
                    for (int x = 0; x < kPer; ++x) {
                        uint32_t f[4][4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            e2m1_unpack(vw[q * (D / 64) + b * kPer + x], f[q]);
#pragma unroll
                            for (int y = 0; y < 4; ++y) f[q][y] = hmul2(f[q][y], s2[q]);
                        }
#pragma unroll
                        for (int y = 0; y < 4; ++y)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma(acc[(b * kPer + x) * 4 + y][nt], __byte_perm(f[0][y], f[1][y], 0x5410),
                                    __byte_perm(f[0][y], f[1][y], 0x7632), __byte_perm(f[2][y], f[3][y], 0x5410),
                                    __byte_perm(f[2][y], f[3][y], 0x7632), pf[nt][0], pf[nt][1]);
                    }
                }
            } else {
                uint32_t vw[D / 8];                       // [token 4][D/32 words]
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    const uint4 w = *reinterpret_cast<const uint4*>(tile + kT.code_bytes + x * 512 + lane * 16);
                    vw[4 * x] = w.x; vw[4 * x + 1] = w.y; vw[4 * x + 2] = w.z; vw[4 * x + 3] = w.w;
                }
                if (edge) {
#pragma unroll
                    for (int x = 0; x < D / 8; ++x) vw[x] = e4m3_numbers(vw[x]);
                }
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    uint32_t f[4][2];
#pragma unroll
                    for (int q = 0; q < 4; ++q) e4m3_unpack(vw[q * (D / 32) + x], f[q][0], f[q][1]);
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma(acc[2 * x + y][nt], __byte_perm(f[0][y], f[1][y], 0x5410), __byte_perm(f[0][y], f[1][y], 0x7632),
                                __byte_perm(f[2][y], f[3][y], 0x5410), __byte_perm(f[2][y], f[3][y], 0x7632), pf[nt][0], pf[nt][1]);
                }
            }

            __syncwarp();                                 // every lane has read the stage: refill it
            present &= ~(1u << cur);
            if (v + kStages < vend) {
                const int st = next;
                if (issue(v + kStages)) present |= 1u << st;
            }
            cur = cur + 1 == kStages ? 0 : cur + 1;
        }
        // ---------------------------------------------------------------- the sums of this run
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[nt][b] += __shfl_xor_sync(0xffffffffu, l[nt][b], o);

        if (whole) {                                      // the CTA's warps join in shared memory
            if (g == 0) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        join_m[warp][8 * nt + 2 * t + b] = m[nt][b];
                        join_l[warp][8 * nt + 2 * t + b] = l[nt][b];
                    }
            }
            __syncthreads();                              // also: no warp reads its ring any more
            float* buf = reinterpret_cast<float*>(smem);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int row = 8 * nt + 2 * t + b;
                    float mm = join_m[0][row];
#pragma unroll
                    for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, join_m[w][row]);
                    const float f = ex2(m[nt][b] - mm);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        *reinterpret_cast<float2*>(buf + warp * R * join_row(D) + join_at<D>(row, i, g)) =
                            make_float2(acc[i][nt][b] * f, acc[i][nt][2 + b] * f);
                }
            if (threadIdx.x < R) {
                const int row = threadIdx.x;
                float mm = join_m[0][row], ll = 0.f;
#pragma unroll
                for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, join_m[w][row]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) ll += join_l[w][row] * ex2(join_m[w][row] - mm);
                row_ml[row] = make_float2(mm, ll);
            }
            __syncthreads();
            const bool done = kDirect ? a.split == 1 : cv0 == 0 && cv1 == u.rt.nt;
            float* out = kDirect ? nullptr : partial<D, R>(a, 2 * kWarps * cta + (cv0 > 0 ? 0 : 1));
            const int groups = min(R, u.si.n * a.G - row0) * (D / 4);
#pragma unroll 4
            for (int e = threadIdx.x; e < groups; e += kThreads) {
                int row, d, at;
                join_group<D>(e, row, d, at);
                const float2 ml = row_ml[row];
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 y = *reinterpret_cast<const float2*>(buf + w * R * join_row(D) + at);
                    const float2 z = *reinterpret_cast<const float2*>(buf + w * R * join_row(D) + at + 16);
                    x.x += y.x; x.y += y.y; x.z += z.x; x.w += z.y;
                }
                if (done) {
                    const int i = div_g(a, row0 + row);
                    store_out<4>(a, (size_t)(u.si.q0 + i), u.h * a.G + row0 + row - i * a.G, D, d, &x.x, ml.x, ml.y);
                } else if (kDirect) {                     // for the cluster: in the place of warp 0's
                    *reinterpret_cast<float2*>(buf + at) = make_float2(x.x, x.y);
                    *reinterpret_cast<float2*>(buf + at + 16) = make_float2(x.z, x.w);
                } else {
                    *reinterpret_cast<float4*>(out + 2 * R + row * D + d) = x;
                    if (d == 0) reinterpret_cast<float2*>(out)[row] = ml;
                }
            }
            if (kDirect && a.split > 1) join_cluster<D, R>(a, u, buf, row_ml);
            break;
        }

        const bool done = v0 == 0 && v1 == u.rt.nt;
        float* out = partial<D, R>(a, 2 * (kWarps * cta + warp) + (v0 > 0 ? 0 : 1));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int row = 8 * nt + 2 * t + b, i = div_g(a, row0 + row);
                if (i >= u.si.n) continue;
                if (done) {
                    const int h = u.h * a.G + row0 + row - i * a.G;
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) {
                        const float v[4] = {acc[2 * x][nt][b], acc[2 * x][nt][2 + b], acc[2 * x + 1][nt][b],
                                            acc[2 * x + 1][nt][2 + b]};
                        store_out<4>(a, (size_t)(u.si.q0 + i), h, D, g * (D / 8) + 4 * x, v, m[nt][b], l[nt][b]);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < D / 32; ++x)
                        *reinterpret_cast<float4*>(out + 2 * R + row * D + g * (D / 8) + 4 * x) =
                            make_float4(acc[2 * x][nt][b], acc[2 * x][nt][2 + b], acc[2 * x + 1][nt][b], acc[2 * x + 1][nt][2 + b]);
                    if (g == 0) reinterpret_cast<float2*>(out)[row] = make_float2(m[nt][b], l[nt][b]);
                }
            }
        if (gave_up) break;
    }
}

namespace {

template <int D, int kFormat, int NT>
cudaError_t rows_room(Room& r) {
    static RoomStore store;
    return store.get(r, kv_rows_kernel<D, kFormat, NT, false>, kv_rows_kernel<D, kFormat, NT, true>, kv_join_kernel<RowsLine<NT>, D>,
                     kThreads, rows_smem<D, kFormat, NT>(), kMaxPerSm, kMaxShares);
}

// Direct: a.split CTAs per unit.  It saves the scan of the lengths, the partial sums and the second kernel,
// but a unit's tiles are not evened out over the SMs.  So it goes up to 24 tiles a warp where there are two
// CTAs per SM (32 sequences of 1024 with 8 heads of 256: 23 us, 36 us by shares; of 300 to 1850, 29 tiles, with
// heads of 128: 26 and 24 us), fewer where SMs stay idle, down to 12 (one sequence with 2 heads of 128: 4096
// tokens, 4 tiles, 7.6 us and 10.0 us; 16384, 16 tiles, 15.0 and 13.2 us).
bool plan_direct(AttnArgs& a, const Room& room, int rows) {
    a.row_tiles = (int)(((long long)a.max_q * a.G + rows - 1) / rows);
    const long long units = (long long)a.n_seqs * a.kv.hkv * a.row_tiles, tiles = most_blocks(a, kKvTile);
    int x = 0;
    while (x < 4 && units << (x + 1) <= room.room[x + 1] && tiles > kWarps << x) ++x;
    a.split = 1 << x;
    const long long ctas = units << x;
    return ctas <= 2LL * room.grid && tiles <= max(12LL, min(24LL, 12 * ctas / sm_count())) * kWarps << x;
}

template <int D, int kFormat, int NT>
cudaError_t launch_direct(const AttnArgs& a, cudaStream_t s) {
    DirectLaunch l(a, kThreads, rows_smem<D, kFormat, NT>(), s);
    return cudaLaunchKernelEx(&l.cfg, kv_rows_kernel<D, kFormat, NT, true>, a);
}

template <int D, int kFormat, int NT>
cudaError_t run_rows(AttnArgs a, const Room& room, cudaStream_t s) {
    if (plan_direct(a, room, 8 * NT)) return launch_direct<D, kFormat, NT>(a, s);
    const cudaError_t e = launch_pdl(kv_rows_kernel<D, kFormat, NT, false>, dim3(room.grid), dim3(kThreads), rows_smem<D, kFormat, NT>(), s, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(kv_join_kernel<RowsLine<NT>, D>, dim3(room.grid * RowsLine<NT>::kSplit), dim3(kJoinThreads), 0, s, a);
}

// Up to 32 rows of a sequence and kv head go by the rows kernel, row tiles of 8 or of 16 (8 rows over 4096
// tokens of 2 heads of 128: 7.5 us, 8.3 us in a tile of 16).  It unpacks a key once per 16 rows, the tiles
// kernel once per 128 or 256, which takes longer to start (16 sequences of 8192 with 2 heads of 128, 32 rows: 37
// us, 39 us by tiles; 48 rows: 51 and 39 us).  More rows go by it too while all the call's work is small:
// (16-row tile, key tile) products times (D + 128) up to 3 * 2^20, which take 15 to 21 us of the 20 to 27 us of
// the tiles kernel's shortest calls (512 rows over 1024 of 2 heads of 128: 10.5 and 30 us; 256 rows over
// 16384: 37 and 27 us).
template <int D, int kFormat>
cudaError_t run(AttnArgs a, cudaStream_t s) {
    const long long rows = (long long)a.max_q * a.G;
    Room room;
    cudaError_t e;
    if (rows <= 8) {
        if ((e = rows_room<D, kFormat, 1>(room)) != cudaSuccess) return e;
        return run_rows<D, kFormat, 1>(a, room, s);
    }
    const long long row_tiles = (rows + 15) / 16, most = (3LL << 20) / (D + 128);
    const bool small = row_tiles <= most && row_tiles * a.n_seqs * a.kv.hkv <= most / most_blocks(a, kKvTile);
    if (rows > 32 && !small) return launch_kv_tiles(a, D, kFormat, s);
    if ((e = rows_room<D, kFormat, 2>(room)) != cudaSuccess) return e;
    if (rows <= 32) return run_rows<D, kFormat, 2>(a, room, s);
    return plan_direct(a, room, 16) ? launch_direct<D, kFormat, 2>(a, s) : launch_kv_tiles(a, D, kFormat, s);
}

__global__ void rows_wait_check_kernel(unsigned* expired) {
    __shared__ __align__(8) uint64_t bar;
    const uint32_t b = smem_u32(&bar);
    if (threadIdx.x == 0) {
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" :: "r"(b));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    const bool done = __all_sync(0xffffffffu, mbar_wait(b, 0));
    if (threadIdx.x == 0 && !done) atomicOr(expired, 1u);
}

}  // namespace

cudaError_t check_rows_waits(unsigned* expired) {
    rows_wait_check_kernel<<<1, 32>>>(expired);
    return cudaGetLastError();
}

size_t kv_task_bytes() { return sizeof(JoinTask) * kWarps * kMaxShares; }
size_t kv_parts_bytes(int D) { return (size_t)2 * kWarps * kMaxShares * 16 * (D + 2) * sizeof(float); }

cudaError_t launch_kv_attention(const AttnArgs& a, int D, int format, cudaStream_t s) {
    if (format == FT_KV_NVFP4)
        return D == 64 ? run<64, FT_KV_NVFP4>(a, s) : D == 128 ? run<128, FT_KV_NVFP4>(a, s) : run<256, FT_KV_NVFP4>(a, s);
    return D == 64 ? run<64, FT_KV_FP8>(a, s) : D == 128 ? run<128, FT_KV_FP8>(a, s) : run<256, FT_KV_FP8>(a, s);
}

}  // namespace ft
