// Attention over the quantised cache for many rows per key: trees of drafted tokens and chunks of
// prompts (launch_kv_attention's rule says from where on).
//
// The same one-pass softmax as the rows kernel, on the 5th-generation tensor cores.  A unit is 128
// rows (token-major: row = token * G + head of the group) of a sequence and kv head; its keys come
// in blocks of 128 (64 with heads of 256).  Per block S = Q K^T (128 x 128 x D, both operands in shared
// memory, fp32 in tensor memory), P = 2^(t - m) as f16 back into tensor memory in the place of S, O += P V
// (128 x D x 128, P from tensor memory, V from shared memory with the head dim contiguous).  One CTA
// per SM:
//   warps 0-7   softmax: one row per thread, the two warpgroups taking turns with the blocks, so
//               that two blocks are under way; a block's reference follows from the one before
//               (handed over in shared memory) and O is rescaled in tensor memory only when a row's
//               maximum has grown past the headroom
//   then        K: codes -> f16 in the 128-byte swizzled layout, and at a unit's start a share of Q;
//               V: the same; four warps each with pairs and with heads of 256, else eight
//   then        one warp issues the matrix instructions: with turns S of block j + 1 before O of block
//               j, with pairs O of a tile's block and S of its next one, tile after tile (three warps
//               more only complete the warpgroup)
// Registers move between the roles at the start (the sums stand at setmaxnreg).  Codes are unpacked to
// f16, which holds them and q exactly, so the products run at the f16 rate; the codes of a warp's
// next block are loaded into registers as soon as it has stored the one before.  Within a lane's 16-byte
// vectors the order of the shared-memory stores is permuted so that the 8 lanes of a store phase hit the 8
// bank groups of a swizzle row.
// Units are laid on the line of shares like the rows kernel's (a unit's start and end cost about
// three blocks), so causal and ragged chunks balance; cut units are joined by the second kernel.
// Every wait is bounded: on expiry the CTA sets FT_DEV_TIMEOUT, leaves its loops, waits for the products under way and
// frees its tensor memory.
//
// 2048 tokens x 32 heads of 128 over 8192 keys of 8 heads, causal, 4-bit: 247 us, 975 TFLOP/s, half of what a
// large library product reaches; the tensor pipe is busy 45 % of the time.  A block's softmax
// sets the pace (two passes over tensor memory, one row per thread): 4650 clocks for 256 rows x 128 keys, of which
// the products take 2070; with blocks in halves, S one half ahead of the softmax, it took 281 us where this
// took 243.  A short call is bound by its way through the
// roles: 9 us from the launch to the first unit's last block, of which Q takes 3.5, and 5 to 8 us for the second
// kernel.
#include <atomic>

#include "ft_kv_attn.cuh"

namespace ft {

namespace {

constexpr int kRows = 128;
// Keys of a block: with heads of 256 half as many, so that two blocks of K and of V fit beside Q (one
// block of 128 each left the tensor cores waiting for every K: 10,000 clocks a block).
constexpr int keys(int D) { return D == 256 ? 64 : 128; }
// Warps of K (and again of V), their tiles of a block, first warps of the roles after the softmax's.
template <int D, bool kPair>
struct Roles {
    static constexpr int kTiles = keys(D) / kKvTile;
    static constexpr int kWide = kPair || D == 256 ? 4 : 8, kEach = kTiles / kWide;
    static constexpr int kK = 8, kV = kK + kWide, kMma = kV + kWide, kThreads = (kMma + 4) * 32;
};
constexpr int kWaitLimit = 1 << 20;
constexpr float kLeast = 1.2e-38f;
// A block's marks: the first or a later one of its unit, or none left; the unit has a second tile of
// rows; the last of the unit's.
constexpr unsigned kFirst = 0, kNext = 1, kEnd = 2, kKind = 3, kTwo = 4, kLast = 8;
// at least 2 places of the line per CTA (4: 22.2 us instead of 19.7 for 512 rows over 4096 of 2 heads of 128); a unit's
// start and end cost about 400 keys (a cost of 2 blocks: 74 us instead of 64 for 16 ragged trees)
template <int D, bool kPair>
using TilesLine = Line<keys(D), kPair ? 2 * kRows : kRows, 1, 2, D == 256 ? 6 : 3, 8, true>;

constexpr int kBufs = 2;                                                 // blocks of K and of V in shared memory
constexpr int region(int D) { return keys(D) * D * 2; }                  // bytes of one
constexpr int q_region(int D) { return kRows * D * 2; }                  // of a tile of rows of Q
constexpr size_t tiles_smem(int D, bool pair) { return (size_t)(pair ? 2 : 1) * q_region(D) + 2 * kBufs * region(D) + 1024; }

__device__ __forceinline__ void mbar_init(uint32_t b, int n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(b), "r"(n));
}
__device__ __forceinline__ void mbar_arrive(uint32_t b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(b) : "memory");
}
// Bounded wait of a whole warp for the phase of the given parity; false (for every lane) once the
// limit is hit or a role gave up.
__device__ __forceinline__ bool mbar_wait(uint32_t b, uint32_t parity, volatile int* abort_flag) {
    bool done = false;
    for (int it = 0; it < kWaitLimit && !done; ++it) {
        uint32_t ok;                                       // suspends for up to 2 us
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 2000;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(b), "r"(parity) : "memory");
        done = ok != 0;
        if (!done && *abort_flag) break;
    }
    done = __all_sync(0xffffffffu, done);
    if (!done) *abort_flag = 1;
    return done;
}
// The same for the last wait, which a role that gave up does not cut short: about two seconds by the clock.
constexpr long long kDrainClocks = 1LL << 32;
__device__ __forceinline__ bool mbar_drained(uint32_t b) {
    const long long from = clock64();
    uint32_t ok;
    do {
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], 0, 2000;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(b) : "memory");
    } while (!ok && clock64() - from < kDrainClocks);
    return __all_sync(0xffffffffu, ok != 0);
}
// One lane of a whole warp.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}

// 128-byte swizzled operand, 64 f16 per row of the swizzle, 8-row groups 1024 bytes apart.  K-major
// (Q, K: rows are the m or n index): the k index runs along the row, the next 64 of it are a region
// of 128 rows further.  MN-major (V: rows are the k index): the n index runs along the row, the next
// 64 of it 16 KB further (the leading offset).
__device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t lead) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
constexpr uint32_t idesc(int n, bool b_mn) {       // f16 x f16 -> f32, M = 128
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(id), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "l"(b), "r"(id), "r"(acc) : "memory");
}

#define FT_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
#define FT_I8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : FT_R8(r, 0), FT_R8(r, 8), FT_R8(r, 16), FT_R8(r, 24) : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
                 :: FT_I8(r, 0), FT_I8(r, 8), FT_I8(r, 16), FT_I8(r, 24), "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
                 :: FT_I8(r, 0), FT_I8(r, 8), "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four f16 pairs of 8 E2M1 codes times a scale pair; of 8 E4M3 codes (two words).
__device__ __forceinline__ uint4 unpack_e2m1(uint32_t w, uint32_t s2) {
    uint4 o;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b32 x0, x1, x2, x3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 x0, b0;\n\tcvt.rn.f16x2.e2m1x2 x1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 x2, b2;\n\tcvt.rn.f16x2.e2m1x2 x3, b3;\n\t"
        "mul.rn.f16x2 %0, x0, %5;\n\tmul.rn.f16x2 %1, x1, %5;\n\tmul.rn.f16x2 %2, x2, %5;\n\tmul.rn.f16x2 %3, x3, %5;\n\t}"
        : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w) : "r"(w), "r"(s2));
    return o;
}
__device__ __forceinline__ uint4 unpack_e4m3(uint32_t w0, uint32_t w1) {
    uint4 o;
    asm("{\n\t.reg .b16 a, b, c, d;\n\tmov.b32 {a, b}, %4;\n\tmov.b32 {c, d}, %5;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t"
        "cvt.rn.f16x2.e4m3x2 %2, c;\n\tcvt.rn.f16x2.e4m3x2 %3, d;\n\t}"
        : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w) : "r"(w0), "r"(w1));
    return o;
}

// Two fp32 at a time.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    f32x2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 unpair(f32x2 a) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(a));
    return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ void st_shared(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Byte of 16-byte chunk c (8 dims) of row r of a [kTall rows][D] operand.  Chunks that differ in the low
// three bits of c differ in the same bits of (byte >> 4): at(r, c ^ z) = at(r, c) ^ (z << 4) for z < 8.
template <int kTall>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return (c >> 3) * (kTall * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// A lane's raw bytes of a tile's K or V.  Loaded by plain loads: the read-only path is for memory that nobody writes while the
// kernel runs, and as a programmatic dependent this one starts while the kernel before may still be writing the cache.
template <int D, int kFormat>
struct Raw {
    static constexpr int kVecs = kFormat == FT_KV_NVFP4 ? D / 64 : D / 32;
    uint4 v[kVecs];
    uint2 s;                 // K: the lane's D/32 scales; V: the word of each of its blocks (NVFP4)
};

// K.  The lane (g, t) holds dims t D/4 .. of tokens g and 8 + g: chunks t D/32 + z, z < D/32.  The
// lanes t of a store phase differ in chunk z ^ perm(t).
template <int D, int kFormat>
__device__ __forceinline__ void load_k(Raw<D, kFormat>& r, const uint8_t* tile, int lane) {
    constexpr KvTile T = kv_tile(D, kFormat);
    const int t = lane & 3;
    // which vector of its token a lane loads k-th
    const int swap = kFormat == FT_KV_NVFP4 ? (D == 256 ? t >> 1 : 0) : D == 128 ? t >> 1 : D == 256 ? t : 0;
#pragma unroll
    for (int x = 0; x < r.kVecs; ++x)
        r.v[x] = *reinterpret_cast<const uint4*>(tile + (x ^ swap) * 512 + lane * 16);
    if constexpr (kFormat == FT_KV_NVFP4) {
        const uint8_t* sp = tile + T.k_scales + lane * (D / 32);
        if constexpr (D == 64) r.s.x = *reinterpret_cast<const uint16_t*>(sp);
        if constexpr (D == 128) r.s.x = *reinterpret_cast<const uint32_t*>(sp);
        if constexpr (D == 256) r.s = *reinterpret_cast<const uint2*>(sp);
    }
}
template <int D, int kFormat>
__device__ __forceinline__ void write_k(uint32_t base, const Raw<D, kFormat>& r, int row0, int lane) {
    const int g = lane >> 2, t = lane & 3;
    // the lane's first chunk of row 8 v + g: rows 8 apart are 1024 bytes apart
    const uint32_t at = base + chunk_at<keys(D)>(row0 + g, t * (D / 32));
    if constexpr (kFormat == FT_KV_NVFP4) {
        if constexpr (D == 64) {
            const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const uint32_t s2 = scale_pair(r.s.x >> (8 * v) & 255u);
#pragma unroll
                for (int i = 0; i < 2; ++i) st_shared((at ^ (i << 4)) + 1024 * v, unpack_e2m1(w[2 * v + i], s2));
            }
        } else {
            // words of a vector swapped in pairs for half of the lanes
            const bool pairs = D == 128 ? t >> 1 : t & 1;
            const uint32_t p = pairs ? 1 : 0;
#pragma unroll
            for (int x = 0; x < r.kVecs; ++x) {
                const int v = D == 128 ? x : x >> 1;
                const uint32_t half = D == 128 ? 0 : (x & 1) ^ (t >> 1);  // which 32 dims of the lane's
                const uint32_t a0 = pairs ? r.v[x].z : r.v[x].x, a1 = pairs ? r.v[x].w : r.v[x].y;
                const uint32_t b0 = pairs ? r.v[x].x : r.v[x].z, b1 = pairs ? r.v[x].y : r.v[x].w;
                const uint32_t sw = (D == 128 ? r.s.x >> (16 * v) : (v ? r.s.y : r.s.x) >> (16 * half)) & 0xFFFFu;
                const uint32_t sa = scale_pair(sw >> (8 * p) & 255u), sb = scale_pair(sw >> (8 * (p ^ 1)) & 255u);
                const uint32_t c = at ^ (half << 6) ^ (p << 5);
                st_shared(c + 1024 * v, unpack_e2m1(a0, sa));
                st_shared((c ^ 16) + 1024 * v, unpack_e2m1(a1, sa));
                st_shared((c ^ 32) + 1024 * v, unpack_e2m1(b0, sb));
                st_shared((c ^ 48) + 1024 * v, unpack_e2m1(b1, sb));
            }
        }
    } else {
        const int swap = D == 128 ? t >> 1 : D == 256 ? t : 0;
        constexpr int kPer = D / 64;                                      // vectors of a token
#pragma unroll
        for (int x = 0; x < r.kVecs; ++x) {
            const uint32_t c = at ^ ((((x ^ swap) % kPer) * 2) << 4);
            st_shared(c + 1024 * (x / kPer), unpack_e4m3(r.v[x].x, r.v[x].y));
            st_shared((c ^ 16) + 1024 * (x / kPer), unpack_e4m3(r.v[x].z, r.v[x].w));
        }
    }
}

// V.  The lane holds dims g D/8 .. of tokens 2t, 2t + 1, 2t + 8, 2t + 9: chunks g D/64 + z.  Odd g take
// neighbouring chunks in the other order.
template <int D, int kFormat>
__device__ __forceinline__ void load_v(Raw<D, kFormat>& r, const uint8_t* tile, int lane) {
    constexpr KvTile T = kv_tile(D, kFormat);
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int x = 0; x < r.kVecs; ++x) r.v[x] = *reinterpret_cast<const uint4*>(tile + T.code_bytes + x * 512 + lane * 16);
    if constexpr (kFormat == FT_KV_NVFP4) {
        const int blk = D == 64 ? g >> 1 : D == 128 ? g : 2 * g;
        r.s.x = *reinterpret_cast<const uint32_t*>(tile + T.v_scales + (blk * 4 + t) * 4);
        if constexpr (D == 256) r.s.y = *reinterpret_cast<const uint32_t*>(tile + T.v_scales + ((blk + 1) * 4 + t) * 4);
    }
}
template <int D, int kFormat>
__device__ __forceinline__ void write_v(uint32_t base, const Raw<D, kFormat>& r, int row0, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const bool odd = g & 1;
    // the lane's first chunk (odd lanes: second) of tokens 2t and 2t + 1; 8 tokens are 1024 bytes
    const uint32_t flip = odd && D > 64 ? 16 : 0;
    const uint32_t at[2] = {base + (chunk_at<keys(D)>(row0 + 2 * t, g * (D / 64)) ^ flip),
                            base + (chunk_at<keys(D)>(row0 + 2 * t + 1, g * (D / 64)) ^ flip)};
    if constexpr (kFormat == FT_KV_NVFP4) {
        if constexpr (D == 64) {
            const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) st_shared(at[q & 1] + 1024 * (q >> 1), unpack_e2m1(w[q], scale_pair(r.s.x >> (8 * q) & 255u)));
        } else if constexpr (D == 128) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint32_t w[4] = {odd ? r.v[x].y : r.v[x].x, odd ? r.v[x].x : r.v[x].y, odd ? r.v[x].w : r.v[x].z,
                                       odd ? r.v[x].z : r.v[x].w};
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint32_t s2 = scale_pair(r.s.x >> (8 * (2 * x + y)) & 255u);
                    st_shared(at[y] + 1024 * x, unpack_e2m1(w[2 * y], s2));
                    st_shared((at[y] ^ 16) + 1024 * x, unpack_e2m1(w[2 * y + 1], s2));
                }
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t w[4] = {odd ? r.v[q].y : r.v[q].x, odd ? r.v[q].x : r.v[q].y, odd ? r.v[q].w : r.v[q].z,
                                       odd ? r.v[q].z : r.v[q].w};
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint32_t s2 = scale_pair((b ? r.s.y : r.s.x) >> (8 * q) & 255u);
                    st_shared((at[q & 1] ^ (b << 5)) + 1024 * (q >> 1), unpack_e2m1(w[2 * b], s2));
                    st_shared((at[q & 1] ^ (b << 5) ^ 16) + 1024 * (q >> 1), unpack_e2m1(w[2 * b + 1], s2));
                }
            }
        }
    } else {
#pragma unroll
        for (int x = 0; x < r.kVecs; ++x) {
            const uint4 v = r.v[x];
            if constexpr (D == 64) {
                st_shared(at[0] + 1024 * x, unpack_e4m3(v.x, v.y));
                st_shared(at[1] + 1024 * x, unpack_e4m3(v.z, v.w));
            } else {
                constexpr int kPer = D / 128;                             // vectors of a token
                const int q = x / kPer;
                const uint32_t c = (at[q & 1] ^ ((x % kPer) << 5)) + 1024 * (q >> 1);
                st_shared(c, unpack_e4m3(odd ? v.z : v.x, odd ? v.w : v.y));
                st_shared((at[q & 1] ^ ((x % kPer) << 5) ^ 16) + 1024 * (q >> 1), unpack_e4m3(odd ? v.x : v.z, odd ? v.y : v.w));
            }
        }
    }
}
template <int D, int kFormat>
__device__ __forceinline__ void clear(Raw<D, kFormat>& r) {
#pragma unroll
    for (int x = 0; x < r.kVecs; ++x) r.v[x] = make_uint4(0, 0, 0, 0);
    r.s = make_uint2(0, 0);
}

// The f16 of a tile's 16 rows of V, which the warp has written, without NaNs (2688 is the largest value that a tile can
// hold; min takes the operand that is a number).  In shared memory, in a loop of a few instructions: with the same in registers, on the
// codes, the windowed chunk took 122 us instead of 115.
template <int D>
__device__ __forceinline__ void only_numbers(uint32_t base, int row0, int lane) {
    __syncwarp();
    const uint32_t at = base + row0 * 128 + lane * 16;
#pragma unroll 4
    for (int x = 0; x < D / 16; ++x) {                    // 512 bytes: 4 rows of 64 dims
        const uint32_t p = at + (x >> 2) * (keys(D) * 128) + (x & 3) * 512;
        asm volatile("{\n\t.reg .b32 a, b, c, d;\n\tld.shared.v4.b32 {a, b, c, d}, [%0];\n\t"
                     "min.f16x2 a, a, %1;\n\tmin.f16x2 b, b, %1;\n\tmin.f16x2 c, c, %1;\n\tmin.f16x2 d, d, %1;\n\t"
                     "st.shared.v4.b32 [%0], {a, b, c, d};\n\t}" :: "r"(p), "r"(0x69406940u) : "memory");
    }
}

// What the softmax warps need to know of a unit.
struct UnitInfo {
    int q0, n, len, base, r, h, i1, slot;    // slot of its partial sums, -1 when the CTA has the whole unit
    bool empty;
};

// What a CTA does of one unit: its blocks [v0, v1).
struct Run {
    Unit u;
    int v0, v1;
};

}  // namespace

// kPair: units of 256 rows, a tile of 128 per softmax warpgroup.  Both share each block of K and V, and
// neither waits for the other: S and O of a tile have their own tensor memory (2 * 128 + 2 * D columns,
// so D up to 128; a chunk of 2048 tokens: 267 us, 328 us by turns).  Otherwise units of 128 rows, the
// warpgroups taking turns with the blocks.
// kDirect: few blocks per CTA.  A cluster of a.split CTAs takes one unit, its blocks in equal runs, and joins through
// distributed shared memory: no line of shares, no workspace, no second kernel.
template <int D, int kFormat, bool kPair, bool kDirect>
__global__ void __launch_bounds__(Roles<D, kPair>::kThreads, 1) kv_tiles_kernel(const AttnArgs a) {
    using L = TilesLine<D, kPair>;
    using Role = Roles<D, kPair>;
    constexpr int kKeys = keys(D), kTiles = Role::kTiles;
    constexpr int kUnit = L::kR, kWarpK = Role::kK, kWarpV = Role::kV, kWarpMma = Role::kMma, kThreads = Role::kThreads;
    constexpr int kEach = Role::kEach;
    constexpr int kRegion = region(D), kRegionQ = q_region(D);
    constexpr KvTile kT = kv_tile(D, kFormat);
    constexpr uint32_t kColO = 256;                       // S and P: columns 0..127 and 128..255
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t sq = (smem_u32(smem_raw) + 1023) & ~1023u, sk = sq + (kPair ? 2 : 1) * kRegionQ, sv = sk + kBufs * kRegion;
    __shared__ long long prefix[kDirect ? 1 : kMaxSeqs + 1], scratch[kThreads / 32];
    __shared__ __align__(8) uint64_t bars[30];
    __shared__ uint32_t tmem_base;
    __shared__ volatile int abort_flag;
    // Written by the K warps, read by the softmax and issuing warps: by the block's number modulo 8 (a
    // softmax warpgroup may be two blocks behind the products, which are up to two blocks behind K),
    // and by the unit's number modulo 4.
    __shared__ float coef[4][kUnit];                      // t = s * coef
    __shared__ unsigned char present[8][kTiles];          // by K warp: bit x, its x-th tile is one of the cache's and some row sees a key of it
    __shared__ unsigned what[8];                          // the block's marks
    __shared__ int key0[8];                               // its first key
    __shared__ UnitInfo units[4];
    __shared__ Unit own;                                  // direct: the cluster's unit
    __shared__ int drafted[4][kTreeMax];                  // places of the drafted tokens
    __shared__ float refs[2][kRows];                      // by block parity: the rows' references
    __shared__ float halves[2][2][kRows];                 // by unit parity and warpgroup: the rows' sums

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t b0 = smem_u32(&bars[0]);
    // K full/empty, V empty by buffer; Q full; S full, V and P full, O done by the block's parity; the softmax
    // warps' references and sums; O read at a unit's end
    auto k_full = [&](int b) { return b0 + 8 * b; };
    auto k_empty = [&](int b) { return b0 + 16 + 8 * b; };
    auto v_empty = [&](int b) { return b0 + 48 + 8 * b; };
    auto s_full = [&](int b) { return b0 + 64 + 8 * b; };
    auto vp_full = [&](int b) { return b0 + 80 + 8 * b; };
    auto o_done = [&](int b) { return b0 + 96 + 8 * b; };
    auto m_full = [&](int quad, int b) { return b0 + 112 + 16 * quad + 8 * b; };    // by 32 rows
    auto l_full = [&](int quad) { return b0 + 176 + 8 * quad; };
    const uint32_t o_free = b0 + 208, drain = b0 + 216, q_full = b0 + 32;
    auto v_full = [&](int b) { return b0 + 224 + 8 * b; };    // pairs: V by buffer, P (in vp_full), S and O by tile
    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(k_full(b), Role::kWide);
            mbar_init(k_empty(b), 1);
            mbar_init(v_empty(b), 1);
            mbar_init(s_full(b), 1);
            mbar_init(vp_full(b), kPair ? 4 : 8 + Role::kWide);
            mbar_init(v_full(b), Role::kWide);
            mbar_init(o_done(b), 1);
            for (int q = 0; q < 4; ++q) mbar_init(m_full(q, b), 1);
        }
        for (int q = 0; q < 4; ++q) mbar_init(l_full(q), 2);
        mbar_init(o_free, 8);
        mbar_init(q_full, 2 * Role::kWide);
        mbar_init(drain, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(smem_u32(&tmem_base)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    pdl_wait_and_release();
    Shares shares(1, 1LL, 0LL);
    long long c0 = 0, c1 = 0;
    bool work;
    const int cta = blockIdx.x;
    if constexpr (kDirect) {
        if (threadIdx.x == 0) {
            const int id = cta / a.split;
            Unit u;
            u.h = id % a.kv.hkv;
            u.r = id / a.kv.hkv % a.row_tiles;
            u.s = id / a.kv.hkv / a.row_tiles;
            u.si = seq_info(a, u.s);
            if (u.si.bad) atomicOr(a.kv.status, FT_DEV_BAD_ID);
            u.rt = row_tile<kKeys>(a, u.si, u.r, kUnit);
            u.first = u.end = 0;
            own = u;
        }
        __syncthreads();
        work = (long long)own.r * kUnit < (long long)own.si.n * a.G;     // the whole cluster's, or none
    } else {
        line_prefix<L>(a, prefix, scratch);               // ends with a CTA barrier
        const long long total = prefix[a.n_seqs];
        shares = Shares(total, gridDim.x, L::kMin);
        work = total > 0 && cta < shares.nc;
        if (work) {
            c0 = shares.cut(cta);
            c1 = shares.cut(cta + 1);
        }
    }
    tc_after();
    const uint32_t tmem = tmem_base;

    // The runs of the CTA in order; every role walks them by itself.
    long long pos = c0;
    auto cut_of = [&](int rank) { return (int)((long long)own.rt.nt * rank / a.split); };    // direct: a CTA's first block
    auto next_run = [&](Run& r) {
        if constexpr (kDirect) {
            if (!work || pos++ > 0) return false;
            r.u = own;
            r.v0 = cut_of(cta % a.split);
            r.v1 = cut_of(cta % a.split + 1);
            return r.v0 < r.v1;
        } else {
            while (pos < c1) {
                Unit& u = r.u;
                if (pos > c0 && u.h + 1 < a.kv.hkv) {     // the same rows, the next head
                    ++u.h;
                    u.end += u.end - u.first;
                    u.first = pos;
                } else {
                    u = find_unit<L>(a, prefix, pos);
                }
                r.v0 = block_at<L>(u.first, u.rt.nt, pos);
                r.v1 = block_at<L>(u.first, u.rt.nt, c1);
                pos = u.end;
                if (r.v0 < r.v1) return true;
            }
            return false;
        }
    };
    // direct: the CTA's sums for the others, in the place of Q and the blocks (laid out like a piece in the workspace)
    float* const sums = reinterpret_cast<float*>(smem_raw + (sq - smem_u32(smem_raw)));

    Run run;
    bool ok = true;
    if constexpr (D == 256) {                             // of 20 * 96: 8 * 112 + 8 * 104 + 4 * 40
        if (warp >= kWarpMma) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        else if (warp >= kWarpK) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
    } else if constexpr (Role::kWide == 4) {              // of 20 * 96: 8 * 128 + 8 * 88 + 4 * 40
        if (warp >= kWarpMma) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        else if (warp >= kWarpK) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    } else {                                              // of 28 * 72: 8 * 104 + 16 * 64 + 4 * 40
        if (warp >= kWarpMma) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        else if (warp >= kWarpK) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    }
    if (warp < kWarpK) {
        // ------------------------------------------------------------------------ softmax
        const int quad = warp & 3, wg = warp >> 2;        // the warpgroup's tile, or the parity of its blocks
        const int row0 = kPair ? kRows * wg : 0;          // its first row of the unit
        const int row = row0 + 32 * quad + lane;
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * quad) << 16);
        const uint32_t o_addr = lane_addr + kColO + (kPair ? D * wg : 0);
        unsigned o_blocks = 0;                            // units that the warpgroup has read out of O
        SeqInfo si;
        UnitInfo u;
        RowRule rule;
        int grow = 0, base = 0, all_lim = 0, all_low = 0;
        // the reference is kept in units of s, so that s - m is exact near it however large t is
        float m = kNoRef, c = 0.f;
        f32x2 l2 = 0;                                     // the sum of this warpgroup's weights, in two halves
        // the reference that the block before was weighed with
        auto take_ref = [&](unsigned n) {
            if (!mbar_wait(m_full(quad, n & 1), n >> 1 & 1, &abort_flag)) return false;
            const float now = refs[n & 1][row];
            if (now != m) {
                const float f = m == kNoRef ? 0.f : ex2((m - now) * c);
                l2 = mul2(l2, pair(f, f));
                m = now;
            }
            return true;
        };
        unsigned un = 0;
        for (unsigned it = 0;; ++it) {                    // every block, the other warpgroup's too
            const int b = kPair ? wg : it & 1;            // S's place
            if (!mbar_wait(s_full(b), kPair ? it & 1 : it >> 1 & 1, &abort_flag)) { ok = false; break; }
            tc_after();
            const unsigned marks = what[it & 7];
            if ((marks & kKind) == kEnd) break;
            // The warpgroup whose turn it is not has seen the block too: S's barrier, of which a wait sees only the
            // phase's parity, is not used again before (it would be after this block's O).
            if (!kPair && b != wg) {
                __syncwarp();
                if (lane == 0) mbar_arrive(vp_full(b));
            }
            if ((marks & kKind) == kFirst) {
                u = units[un & 3];
                si = SeqInfo{u.q0, u.n, u.len, u.base, false};
                base = si.base;
                grow = u.r * kUnit + row;
                rule = row_rule(a, si, grow);
                // keys below all_lim and from all_low on are seen by every row of the tile (under a tree a row may stand
                // as far past base as its mask has other bits, whichever they are)
                all_lim = a.tree ? min(base, si.len) - 1 : row_rule(a, si, u.r * kUnit + row0).lim;
                const int last = kPair ? min(si.n - 1, div_g(a, u.r * kUnit + row0 + kRows - 1)) : u.i1;
                all_low = a.window > 0 ? (int)max((long long)base + (a.tree ? kTreeMax - 1 : last) - a.window + 1, 0LL) : 0;
                m = kNoRef;
                c = coef[un & 3][row];
                l2 = pair(0.f, 0.f);
            }
            if (kPair && wg == 1 && !(marks & kTwo)) {    // no rows: told, so that it keeps step
                if (lane == 0) mbar_arrive(vp_full(1));
                if (marks & kLast) ++un;
                continue;
            }
            const bool opens = (marks & kKind) == kFirst;
            if (kPair || b == wg) {
                const uint32_t s_addr = lane_addr + 128 * b;
                const int j0 = key0[it & 7];
                unsigned there = 0;                       // the block's tiles
#pragma unroll
                for (int w = 0; w < Role::kWide; ++w) there |= (unsigned)present[it & 7][w] << (w * kEach);
                const bool edge = there != (1u << kTiles) - 1 || j0 + kKeys - 1 > all_lim || (j0 < all_low && j0 + kKeys > a.n_sink) || u.empty;
                // which of 32 keys the row sees
                auto mask_of = [&](int ch) {
                    const int j = j0 + 32 * ch;
                    auto below = [&](int x) {             // bits of keys < x
                        const int n = x - j;
                        return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1;
                    };
                    const int lim1 = rule.lim + 1;
                    unsigned ok_bits = below(lim1) & (~below(rule.low) | below(a.n_sink));
                    if (a.tree && j + 31 >= base && rule.lim >= 0) {
                        const unsigned old = below(base);
                        const int sh = j - base;          // drafted token of bit 0
                        unsigned d = sh >= 64 ? 0u : sh >= 0 ? (unsigned)(rule.mask >> sh) : sh > -32 ? (unsigned)(rule.mask << -sh) : 0u;
                        d &= below(lim1) & ~old;
                        if (a.window > 0) {
                            unsigned far = 0;
                            for (unsigned x = d; x; x &= x - 1) {
                                const int e = __ffs(x) - 1;
                                if (drafted[un & 3][sh + e] < rule.low && j + e >= a.n_sink) far |= 1u << e;
                            }
                            d &= ~far;
                        }
                        ok_bits = (ok_bits & old) | d;
                    }
                    const unsigned t2 = there >> (2 * ch);
                    return ok_bits & ((t2 & 1 ? 0xFFFFu : 0u) | (t2 & 2 ? 0xFFFF0000u : 0u));
                };
                // the row's largest s.  Keys that are not seen get -inf, whatever their bytes gave (weight
                // 0: c is positive), in tensor memory too.
                float top = kNoRef;
                if (!edge) {
                    uint32_t s[2][32];
                    tmem_ld32(s_addr, s[0]);
#pragma unroll
                    for (int ch = 0; ch < kKeys / 32; ++ch) {
                        tmem_wait_ld();
                        if (ch + 1 < kKeys / 32) tmem_ld32(s_addr + 32 * (ch + 1), s[(ch + 1) & 1]);
                        float x = kNoRef, y = kNoRef;
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            x = fmaxf(x, fmaxf(__uint_as_float(s[ch & 1][e]), __uint_as_float(s[ch & 1][e + 1])));
                            y = fmaxf(y, fmaxf(__uint_as_float(s[ch & 1][e + 2]), __uint_as_float(s[ch & 1][e + 3])));
                        }
                        top = fmaxf(top, fmaxf(x, y));
                    }
                } else {
#pragma unroll 1
                    for (int ch = 0; ch < kKeys / 32; ++ch) {
                        uint32_t s[32];
                        const unsigned seen = mask_of(ch);
                        __syncwarp();
                        tmem_ld32(s_addr + 32 * ch, s);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            if (!(seen >> e & 1)) s[e] = 0xFF800000u;
                            top = fmaxf(top, __uint_as_float(s[e]));
                        }
                        tmem_st32(s_addr + 32 * ch, s);
                    }
                    tmem_wait_st();
                }
                if (!kPair && !opens && !take_ref(it - 1)) { ok = false; break; }
                const bool raise = top > m && (m == kNoRef || (top - m) * c > kHeadroom);
                float f = 1.f;
                if (raise) {
                    f = m == kNoRef ? 0.f : ex2((m - top) * c);
                    m = top;
                    l2 = mul2(l2, pair(f, f));
                }
                if constexpr (!kPair) {
                    refs[b][row] = m;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(m_full(quad, b));
                }
                if (__any_sync(0xffffffffu, raise) && !opens) {
                    // O of the block before: complete with this block's S where one tile has both
                    if (!kPair && !mbar_wait(o_done(b ^ 1), (it - 1) >> 1 & 1, &abort_flag)) { ok = false; break; }
                    tc_after();
#pragma unroll 1
                    for (int x = 0; x < D; x += 32) {
                        uint32_t o[32];
                        tmem_ld32(o_addr + x, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(o_addr + x, o);
                    }
                }
                // a row that has seen nothing keeps finite differences: its s are -inf
                const float ref = m == kNoRef ? 0.f : m;
                const f32x2 m2 = pair(-ref, -ref), c2 = pair(c, c), head2 = pair(kHeadroom, kHeadroom);
                // P over S: 32 columns of S become 16 of f16 pairs, over columns that have been read
                uint32_t s[2][32];
                tmem_ld32(s_addr, s[0]);
#pragma unroll
                for (int ch = 0; ch < kKeys / 32; ++ch) {
                    tmem_wait_ld();
                    if (ch + 1 < kKeys / 32) tmem_ld32(s_addr + 32 * (ch + 1), s[(ch + 1) & 1]);
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float2 x = unpair(fma2(add2(pair(__uint_as_float(s[ch & 1][e]), __uint_as_float(s[ch & 1][e + 1])), m2), c2, head2));
                        x.x = ex2(x.x);
                        x.y = ex2(x.y);
                        l2 = add2(l2, pair(x.x, x.y));
                        p[e >> 1] = pack_f16(x.x, x.y);
                    }
                    tmem_st16(s_addr + 16 * ch, p);
                }
                tmem_wait_st();
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(vp_full(b));
            }
            if (!(marks & kLast)) continue;
            // the unit's sums: for turns, the last block's reference and both warpgroups' weights
            float l = unpair(l2).x + unpair(l2).y;
            if constexpr (kPair) {
                if (!mbar_wait(o_done(wg), o_blocks++ & 1, &abort_flag)) { ok = false; break; }
                // the sums take the place of what the other tile's products read
                if (kDirect && marks & kTwo && !mbar_wait(o_done(1 - wg), 0, &abort_flag)) { ok = false; break; }
            } else {
                if (b != wg && !take_ref(it)) { ok = false; break; }
                halves[un & 1][wg][row] = unpair(l2).x + unpair(l2).y;
                __syncwarp();
                if (lane == 0) mbar_arrive(l_full(quad));
                if (!mbar_wait(l_full(quad), un & 1, &abort_flag)) { ok = false; break; }
                l = halves[un & 1][0][row] + halves[un & 1][1][row];
                if (!mbar_wait(o_done(it & 1), it >> 1 & 1, &abort_flag)) { ok = false; break; }
            }
            ++un;
            if (m != kNoRef) m *= c;
            tc_after();
            const int i = div_g(a, grow);
            const bool on = i < si.n, done = u.slot < 0;
            float* out = kDirect ? sums : partial<D, kUnit>(a, max(u.slot, 0));
            if (on && !done && (kPair || wg == 0)) reinterpret_cast<float2*>(out)[row] = make_float2(m, l);
#pragma unroll 1
            for (int x = kPair ? 0 : wg * (D / 2); x < (kPair ? D : (wg + 1) * (D / 2)); x += 32) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld32(o_addr + x, o);
                tmem_wait_ld();
                if (on) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float y[8];
#pragma unroll
                        for (int z = 0; z < 8; ++z) y[z] = __uint_as_float(o[e + z]);
                        if (done) {
                            store_out<8>(a, (size_t)(si.q0 + i), u.h * a.G + grow - i * a.G, D, x + e, y, m, l);
                        } else {
                            float4* dst = reinterpret_cast<float4*>(out + 2 * kUnit) + piece_at<L, D>(row, x + e);
                            dst[0] = make_float4(y[0], y[1], y[2], y[3]);
                            dst[kUnit] = make_float4(y[4], y[5], y[6], y[7]);
                        }
                    }
                }
            }
            // with turns, O is free for the next unit once both warpgroups have read their halves
            tc_before();
            __syncwarp();
            if (!kPair && lane == 0) mbar_arrive(o_free);
        }
        if (kDirect && a.split > 1) {                     // a slice of the unit's values per CTA, the ranks in order
            cluster_sync();
            const int rank = cta % a.split, rows = work ? min(kUnit, own.si.n * a.G - own.r * kUnit) : 0, groups = rows * (D / 4);
            const int ga = (int)((long long)groups * rank / a.split), gb = (int)((long long)groups * (rank + 1) / a.split);
            for (int e = ga + threadIdx.x; e < gb; e += 8 * 32) {
                const int r = e % rows, d = e / rows * 4;
                float m1 = kNoRef, l1 = 0.f;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                constexpr int kBatch = 8;                 // ranks in flight
                for (int k0 = 0; k0 < a.split; k0 += kBatch) {
                    float2 ml[kBatch];
                    float4 y[kBatch];
                    float mm = m1;
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        ml[k] = make_float2(kNoRef, 0.f);
                        y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (k0 + k < a.split && cut_of(k0 + k) < cut_of(k0 + k + 1)) {
                            const uint32_t src = cluster_addr(sums, k0 + k);
                            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(ml[k].x), "=f"(ml[k].y) : "r"(src + 8 * r));
                            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(y[k].x), "=f"(y[k].y), "=f"(y[k].z), "=f"(y[k].w)
                                         : "r"(src + 8 * kUnit + 16 * piece_at<L, D>(r, d)));
                        }
                        mm = fmaxf(mm, ml[k].x);
                    }
                    float f = ex2(m1 - mm);
                    m1 = mm;
                    l1 *= f;
                    x.x *= f; x.y *= f; x.z *= f; x.w *= f;
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        f = ex2(ml[k].x - mm);
                        l1 += ml[k].y * f;
                        x.x += y[k].x * f; x.y += y[k].y * f; x.z += y[k].z * f; x.w += y[k].w * f;
                    }
                }
                const int gr = own.r * kUnit + r, i = div_g(a, gr);
                store_out<4>(a, (size_t)(own.si.q0 + i), own.h * a.G + gr - i * a.G, D, d, &x.x, m1, l1);
            }
        }
    } else if (warp < kWarpMma) {
        // ------------------------------------------------------------------------ K (and Q), V
        const bool is_k = warp < kWarpV;
        const int w = (warp - kWarpK) & (Role::kWide - 1);       // the warp's tiles of a block: w kEach ..
        const int per = a.kv.page_shift - 4;
        unsigned it = 0;
        for (int un = 0; ok && next_run(run); ++un) {
            const SeqInfo& si = run.u.si;
            const int base = si.base;
            const int32_t* table = a.table + (size_t)run.u.s * a.table_stride;
            // keys that some row sees: below hi, from lo on or among the first tokens
            const int hi = run.u.rt.empty ? 0 : a.tree ? si.len : min(si.len, base + run.u.rt.i1 + 1);
            const int lo = a.window > 0 ? (int)max((long long)base + (a.tree ? 0 : run.u.rt.i0) - a.window + 1, 0LL) : 0;
            // V: keys that every row of the unit sees: below all_hi, from all_lo on or among the first tokens
            const int all_hi = min(a.tree ? base : base + run.u.rt.i0 + 1, si.len);
            const int all_lo = a.window > 0 ? (int)max((long long)base + (a.tree ? kTreeMax - 1 : run.u.rt.i1) - a.window + 1, 0LL) : 0;
            int group = -1, page = -1;                    // lane x: the page of its (x % kEach)-th tile of block v0 + 32 / kEach * group + x / kEach
            Raw<D, kFormat> raw[kEach];
            unsigned have = 0;                            // bit x: the tile is one of the cache's and some row sees a key of it
            auto load = [&](int v) {
                const int n = (v - run.v0) * kEach;
                if (n >> 5 != group) {
                    group = n >> 5;
                    page = -1;
                    const int mine = run.v0 + ((n & ~31) + lane) / kEach;
                    if (mine < run.v1) {
                        const int tile = run.u.rt.block(mine) * kTiles + w * kEach + lane % kEach, key = tile * 16;
                        if (key < hi && (key + 15 >= lo || key < a.n_sink)) {
                            page = table[tile >> per];
                            if (page < 0 || page >= a.kv.n_pages) {
                                if (!a.tree || tree_sees_tile(a.tree + si.q0, run.u.rt.i0, run.u.rt.i1 + 1 - run.u.rt.i0, a.n_tokens - si.q0, base, si.len,
                                                              key, a.window, a.n_sink))
                                    atomicOr(a.kv.status, FT_DEV_BAD_ID);
                                page = -1;
                            }
                        }
                    }
                }
                have = 0;
#pragma unroll
                for (int x = 0; x < kEach; ++x) {
                    const int pg = __shfl_sync(0xffffffffu, page, (n + x) & 31);
                    if (pg >= 0) {
                        have |= 1u << x;
                        const int tile = run.u.rt.block(v) * kTiles + w * kEach + x;
                        const uint8_t* src = a.kv.pool + ((((size_t)pg * a.kv.hkv + run.u.h) << per) + (tile & ((1 << per) - 1))) * kT.bytes;
                        if (is_k) load_k<D, kFormat>(raw[x], src, lane);
                        else load_v<D, kFormat>(raw[x], src, lane);
                    } else {
                        clear(raw[x]);
                    }
                }
            };
            // Q of the unit, once every product of the unit before is through with it: 8 lanes per row, a
            // tile's rows of a lane under way together
            if (it > 0 && !mbar_wait(k_empty((it - 1) % kBufs), ((it - 1) / kBufs) & 1, &abort_flag)) { ok = false; break; }
            if (warp == kWarpK && lane == 0) {
                const bool all = kDirect ? a.split == 1 : run.v0 == 0 && run.v1 == run.u.rt.nt;
                units[un & 3] = UnitInfo{si.q0, si.n, si.len, si.base, run.u.r, run.u.h, run.u.rt.i1, all ? -1 : kDirect ? 0 : 2 * cta + (run.v0 > 0 ? 0 : 1), run.u.rt.empty};
            }
            if (a.tree && warp == kWarpK)
                for (int j = lane; j < min(si.len - base, kTreeMax); j += 32)
                    drafted[un & 3][j] = drafted_pos(a, si, base + j);
            const int row_tiles = kPair && (long long)run.u.r * kUnit + kRows < (long long)si.n * a.G ? 2 : 1;
            constexpr int kLane = kRows / (8 * Role::kWide);      // rows of a lane
#pragma unroll 1
            for (int rt = 0; rt < row_tiles; ++rt) {
                const int row = 4 * kLane * (warp - kWarpK) + (lane >> 3), part = lane & 7;
                uint4 q[kLane][D / 64];
#pragma unroll
                for (int x = 0; x < kLane; ++x) {
                    const int grow = run.u.r * kUnit + kRows * rt + row + 4 * x, i = div_g(a, grow);
                    const __nv_bfloat16* src = a.q + (size_t)(si.q0 + i) * a.q_stride + (size_t)(run.u.h * a.G + grow - i * a.G) * D + part * 8;
#pragma unroll
                    for (int e = 0; e < D / 64; ++e)
                        q[x][e] = i < si.n ? *reinterpret_cast<const uint4*>(src + 64 * e) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int x = 0; x < kLane; ++x) {
                    float amax = 0.f;
#pragma unroll
                    for (int e = 0; e < D / 64; ++e) {
                        const uint32_t wd[4] = {q[x][e].x, q[x][e].y, q[x][e].z, q[x][e].w};
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(wd[y] << 16)), fabsf(__uint_as_float(wd[y] & 0xFFFF0000u))));
                    }
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    const RowScale rs = row_scale(amax);
                    // the coefficient is positive (q carries the scale's sign): times -inf it stays -inf
                    const float down = a.scale < 0.f ? -rs.down : rs.down;
                    if (part == 0) coef[un & 3][kRows * rt + row + 4 * x] = fmaxf(fabsf(a.scale) * a.kv.k_scale * 1.44269504088896340736f * rs.up, kLeast);
#pragma unroll
                    for (int e = 0; e < D / 64; ++e) {
                        const uint32_t wd[4] = {q[x][e].x, q[x][e].y, q[x][e].z, q[x][e].w};
                        uint32_t o[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            o[y] = pack_f16(__uint_as_float(wd[y] << 16) * down, __uint_as_float(wd[y] & 0xFFFF0000u) * down);
                        st_shared(sq + rt * kRegionQ + chunk_at<kRows>(row + 4 * x, e * 8 + part), make_uint4(o[0], o[1], o[2], o[3]));
                    }
                }
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            load(run.v0);
            for (int v = run.v0; v < run.v1; ++v, ++it) {
                const int b = it % kBufs;
                if (!mbar_wait(is_k ? k_empty(b) : v_empty(b), ((it / kBufs) & 1) ^ 1, &abort_flag)) { ok = false; break; }
                const uint32_t dst = (is_k ? sk : sv) + b * kRegion;
#pragma unroll
                for (int x = 0; x < kEach; ++x) {
                    const int row = 16 * (w * kEach + x);
                    if (is_k) {
                        write_k<D, kFormat>(dst, raw[x], row, lane);
                    } else {
                        // where a row does not see a key (weight 0), its slot may never have been written: no NaN may stay
                        const int j0 = run.u.rt.block(v) * kKeys + row;
                        const bool part = j0 + kKvTile > all_hi || (j0 < all_lo && j0 + kKvTile > a.n_sink);
                        if (kFormat == FT_KV_NVFP4 && part) raw[x].s = make_uint2(e4m3_numbers(raw[x].s.x), e4m3_numbers(raw[x].s.y));
                        write_v<D, kFormat>(dst, raw[x], row, lane);
                        if (kFormat == FT_KV_FP8 && part) only_numbers<D>(dst, row, lane);
                    }
                }
                if (is_k && lane == 0) {
                    present[it & 7][w] = have;
                    if (w == 0) {
                        what[it & 7] = (v == run.v0 ? kFirst : kNext) | (row_tiles > 1 ? kTwo : 0) | (v + 1 == run.v1 ? kLast : 0);
                        key0[it & 7] = run.u.rt.block(v) * kKeys;
                    }
                }
                fence_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(is_k ? k_full(b) : kPair ? v_full(b) : vp_full(it & 1));
                if (v + 1 < run.v1) load(v + 1);
            }
        }
        if (ok && is_k) {                                 // no more blocks
            ok = mbar_wait(k_empty(it % kBufs), ((it / kBufs) & 1) ^ 1, &abort_flag);
            if (w == 0 && lane == 0) what[it & 7] = what[(it + 1) & 7] = kEnd;       // the other warpgroup's turn too
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(k_full(it % kBufs));
        }
        if (!kDirect && warp == kWarpK) {                 // the unit that the cut at the CTA's first place goes through
            if (work) run.u = find_unit<L>(a, prefix, c0);
            if (lane == 0) {
                if (work && run.u.first < c0)
                    a.tasks[cta] = join_task(shares, run.u, shares.holder(run.u.first), shares.holder(run.u.end - 1));
                else
                    a.tasks[cta].on = 0;
            }
        }
    } else if (warp == kWarpMma) {
        // ------------------------------------------------------------------------ matrix instructions
        // descriptors of the regions' first bytes; an offset adds to the address field (16-byte units)
        const uint64_t q_desc = desc(sq, 16), k_desc = desc(sk, 16), v_desc = desc(sv, kKeys * 128);
        const bool lead = elect();
        unsigned units_o = 0, units_q = 0;
        // S of a tile of the block in buffer b; O of a tile of the block in buffer c, P at p
        auto products_s = [&](int tile, int b, uint32_t d) {
            if (lead) {
                const uint64_t qd = q_desc + tile * (kRegionQ >> 4), kd = k_desc + b * (kRegion >> 4);
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    const uint64_t in = ((x & 3) * 32) >> 4;
                    mma_ss(d, qd + (x >> 2) * (kRows * 128 >> 4) + in, kd + (x >> 2) * (kKeys * 128 >> 4) + in, idesc(kKeys, false), x > 0);
                }
            }
            __syncwarp();
        };
        auto products_o = [&](int tile, int c, uint32_t p, bool first) {
            if (lead) {
                const uint64_t vd = v_desc + c * (kRegion >> 4);
#pragma unroll
                for (int x = 0; x < kKeys / 16; ++x)
                    mma_ts(tmem + kColO + D * tile, p + 8 * x, vd + x * (2048 >> 4), idesc(D, true), x > 0 || !first);
            }
            __syncwarp();
        };
        auto commit = [&](uint32_t bar) {
            if (lead) tc_commit(bar);
            __syncwarp();
        };
        // O of block n, the last of its unit, without waiting for the next unit's K
        auto finish = [&](unsigned n, unsigned marks) {
            const int c = n % kBufs;
            if (kPair && !mbar_wait(v_full(c), (n / kBufs) & 1, &abort_flag)) return false;
#pragma unroll
            for (int tile = 0; tile < (kPair ? 2 : 1); ++tile) {
                const int at = kPair ? tile : n & 1;
                if (!mbar_wait(vp_full(at), (kPair ? n : n >> 1) & 1, &abort_flag)) return false;
                const bool first = (marks & kKind) == kFirst;
                if (!kPair && first && units_o++ > 0 && !mbar_wait(o_free, units_o & 1, &abort_flag)) return false;
                if (tile == 0 || marks & kTwo) {
                    tc_after();
                    products_o(tile, c, tmem + 128 * at, first);
                    commit(o_done(at));
                }
            }
            commit(v_empty(c));
            return true;
        };
        for (unsigned it = 0, before = kEnd;; ++it) {
            const int b = it % kBufs, c = (it - 1) % kBufs;
            if (before != kEnd && before & kLast) {
                ok = finish(it - 1, before);
                if (!ok) break;
                before = kEnd;
            }
            ok = mbar_wait(k_full(b), (it / kBufs) & 1, &abort_flag);
            if (!ok) break;
            tc_after();
            const unsigned now = what[it & 7];
            const bool more = (now & kKind) != kEnd, owed = before != kEnd;
            if ((now & kKind) == kFirst) {                // of a unit: its Q
                ok = mbar_wait(q_full, units_q++ & 1, &abort_flag);
                if (!ok) break;
                tc_after();
            }
            const bool first = (before & kKind) == kFirst;
            if constexpr (kPair) {
                // tile by tile: O of the block before, then S of this one over its P
                if (owed) ok = mbar_wait(v_full(c), ((it - 1) / kBufs) & 1, &abort_flag);
#pragma unroll
                for (int tile = 0; tile < 2; ++tile) {
                    if (ok && owed) {
                        ok = mbar_wait(vp_full(tile), (it - 1) & 1, &abort_flag);
                        if (ok && (tile == 0 || before & kTwo)) {
                            tc_after();
                            products_o(tile, c, tmem + 128 * tile, first);
                        }
                    }
                    if (ok && more && (tile == 0 || now & kTwo)) products_s(tile, b, tmem + 128 * tile);
                    if (ok) commit(s_full(tile));         // a tile without rows and the end are told too
                }
                if (!ok) break;
                if (more) commit(k_empty(b));
                if (owed) commit(v_empty(c));
            } else {
                // S of this block, then O of the one before
                if (more) {
                    products_s(0, b, tmem + 128 * (it & 1));
                    commit(k_empty(b));
                    commit(s_full(it & 1));
                }
                if (owed) {
                    const unsigned n = it - 1;
                    ok = mbar_wait(vp_full(n & 1), n >> 1 & 1, &abort_flag);
                    if (ok && first && units_o++ > 0)     // the unit before has been read out of O
                        ok = mbar_wait(o_free, units_o & 1, &abort_flag);
                    if (!ok) break;
                    tc_after();
                    products_o(0, c, tmem + 128 * (n & 1), first);
                    commit(v_empty(c));
                    commit(o_done(n & 1));
                }
            }
            if (!more) {
                if (!kPair) {                             // the end, for both turns
                    commit(s_full(it & 1));
                    commit(s_full((it + 1) & 1));
                }
                break;
            }
            before = now;
        }
        // what was issued reads shared memory and writes tensor memory: before the CTA's end, whether a role gave up or not
        if (lead) tc_commit(drain);
        __syncwarp();
        if (!mbar_drained(drain)) ok = false;
    }
    if (!ok && lane == 0) atomicOr(a.kv.status, FT_DEV_TIMEOUT);
    if (kDirect && a.split > 1) {
        if (warp >= kWarpK) cluster_sync();
        cluster_sync();                                   // the others may still read this CTA's sums
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == kWarpMma) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
}

namespace {

template <int D, int kFormat, bool kPair>
cudaError_t tiles_room(Room& r) {
    static RoomStore store;
    void (*direct)(AttnArgs) = nullptr;
    if constexpr (D <= 128) direct = kv_tiles_kernel<D, kFormat, kPair, true>;
    return store.get(r, kv_tiles_kernel<D, kFormat, kPair, false>, direct, kv_join_kernel<TilesLine<D, kPair>, D>,
                     Roles<D, kPair>::kThreads, tiles_smem(D, kPair), 1, kMaxShares / 4);   // two pieces of up to 256 rows each fit the workspace
}

// Direct: a.split CTAs per unit.  A CTA's start and end then come once, and there is no second kernel, but SMs
// stay idle.  So it goes where a CTA gets at most three blocks more than an even share (320 rows over 4096 of 2
// heads of 128, 4 blocks and 1: 17.7 us, 19.7 by shares; 256 rows over 16384 of one head, 8 and 1: 26 and 18 us), and
// with a CTA per unit up to 8 blocks (3 prompts of 400 over 1000, 4 heads of 128, 4 query heads each: 28 us, 44
// us by shares, whose CTAs have two or three units to start and end).  Not with heads of 256: a block takes
// them longer (320 rows over 4096: 26 us, 23 by shares).
template <int D, bool kPair>
bool plan_direct(AttnArgs& a, const Room& room) {
    constexpr int kUnit = TilesLine<D, kPair>::kR;
    const long long rows = (long long)a.max_q * a.G, row_tiles = (rows + kUnit - 1) / kUnit;
    if (row_tiles > room.grid) return false;
    const long long units = row_tiles * a.n_seqs * a.kv.hkv, blocks = most_blocks(a, keys(D));
    if (units > room.grid) return false;
    int x = 0;
    while (x < 4 && units << (x + 1) <= room.room[x + 1] && blocks > 1LL << x) ++x;
    a.row_tiles = (int)row_tiles;
    a.split = 1 << x;
    const long long each = (blocks + a.split - 1) / a.split;
    return each <= 8 && (x == 0 || each <= units * blocks / room.grid + 3);
}

template <int D, int kFormat, bool kPair>
cudaError_t run_tiles(AttnArgs a, cudaStream_t s) {
    Room room;
    cudaError_t e = tiles_room<D, kFormat, kPair>(room);
    if (e != cudaSuccess) return e;
    if constexpr (D <= 128)
        if (plan_direct<D, kPair>(a, room)) {
            DirectLaunch l(a, Roles<D, kPair>::kThreads, tiles_smem(D, kPair), s);
            return cudaLaunchKernelEx(&l.cfg, kv_tiles_kernel<D, kFormat, kPair, true>, a);
        }
    e = launch_pdl(kv_tiles_kernel<D, kFormat, kPair, false>, dim3(room.grid), dim3(Roles<D, kPair>::kThreads), tiles_smem(D, kPair), s, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(kv_join_kernel<TilesLine<D, kPair>, D>, dim3(room.grid * TilesLine<D, kPair>::kSplit), dim3(kJoinThreads), 0, s, a);
}

template <int D, int kFormat>
cudaError_t run(const AttnArgs& a, cudaStream_t s) {
    if constexpr (D <= 128) {
        // Pairs where each CTA has five blocks of 128 x 128 or more: they start and end later (512 rows over 4096 of 4
        // heads of 128: 26.6 us, 22.5 us without) but share a block's unpacking (over 16384: 34 and 38 us; 1024
        // rows over 16384: 49 and 60 us).
        const long long rows = (long long)a.max_q * a.G;
        if (rows > kRows && (rows + kRows - 1) / kRows * most_blocks(a, 128) >= 5LL * sm_count() / a.kv.hkv / a.n_seqs + 1)
            return run_tiles<D, kFormat, true>(a, s);
    }
    return run_tiles<D, kFormat, false>(a, s);
}

__global__ void tiles_wait_check_kernel(unsigned* expired) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ volatile int abort_flag;
    const uint32_t b = smem_u32(&bar);
    if (threadIdx.x == 0) {
        mbar_init(b, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    unsigned bits = 0;
    if (!mbar_wait(b, 0, &abort_flag) && abort_flag) bits |= 2u;
    const long long from = clock64();
    if (!mbar_wait(b, 0, &abort_flag) && clock64() - from < kDrainClocks / 64) bits |= 4u;     // leaves at the flag
    const long long drain = clock64();
    if (!mbar_drained(b) && clock64() - drain >= kDrainClocks) bits |= 8u;                     // does not
    if (threadIdx.x == 0) atomicOr(expired, bits);
}

}  // namespace

cudaError_t check_tiles_waits(unsigned* expired) {
    tiles_wait_check_kernel<<<1, 32>>>(expired);
    return cudaGetLastError();
}

cudaError_t launch_kv_tiles(const AttnArgs& a, int D, int format, cudaStream_t s) {
    if (format == FT_KV_NVFP4)
        return D == 64 ? run<64, FT_KV_NVFP4>(a, s) : D == 128 ? run<128, FT_KV_NVFP4>(a, s) : run<256, FT_KV_NVFP4>(a, s);
    return D == 64 ? run<64, FT_KV_FP8>(a, s) : D == 128 ? run<128, FT_KV_FP8>(a, s) : run<256, FT_KV_FP8>(a, s);
}

}  // namespace ft
