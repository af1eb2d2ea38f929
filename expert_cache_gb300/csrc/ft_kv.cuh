// Internal declarations of the quantised key/value cache and its attention.
#pragma once
#include "ft_internal.cuh"

namespace ft {

constexpr int kKvTile = 16;            // tokens per tile record
constexpr int kTreeMax = 64;           // drafted tokens of one sequence (bits of a mask)

// Byte layout of one tile record (16 tokens of one kv head).
struct KvTile {
    int code_bytes;      // of K, and again of V
    int k_scales, v_scales, bytes;
};

#ifdef __CUDACC__
__host__ __device__
#endif
inline constexpr KvTile kv_tile(int D, int format) {
    return format == FT_KV_NVFP4 ? KvTile{kKvTile * D / 2, kKvTile * D, kKvTile * D + D, kKvTile * D + 2 * D}
                                 : KvTile{kKvTile * D, 2 * kKvTile * D, 2 * kKvTile * D, 2 * kKvTile * D};
}

// One layer of a cache as the kernels see it.
struct KvView {
    uint8_t* pool;       // the layer's pages
    int n_pages, page_shift, hkv;      // page_size = 1 << page_shift
    float k_scale, v_scale;
    int* status;
};

struct JoinTask;

struct AttnArgs {
    KvView kv;
    const __nv_bfloat16* q;
    size_t q_stride;
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* table;
    int table_stride, n_seqs, n_tokens, max_q;
    int hq, G;
    unsigned g_mul;      // division by G: div_g
    int g_shift;
    const unsigned long long* tree;
    int window, n_sink;
    float scale;
    __nv_bfloat16* o;
    size_t o_stride;
    float* lse;
    int split, row_tiles;        // direct: CTAs of a unit (a cluster), row tiles of a sequence at most
    JoinTask* tasks;      // workspace: what the joining kernel has to do
    float* parts;        // workspace: partial sums of the units that a share's end cuts
};

constexpr int kMaxSeqs = 1024;         // sequences of one attention call

// The workspace: a status word, the joining kernel's tasks, partial sums.
constexpr size_t kKvHeadBytes = 256;
size_t kv_task_bytes();
size_t kv_parts_bytes(int D);

cudaError_t launch_kv_append(const KvView& kv, int D, int format, const void* k, const void* v, size_t k_stride,
                             size_t v_stride, const int32_t* slots, int n, cudaStream_t s);
cudaError_t launch_kv_read(const KvView& kv, int D, int format, const int32_t* slots, int n, void* k_out, void* v_out,
                           cudaStream_t s);
cudaError_t launch_kv_attention(const AttnArgs& a, int D, int format, cudaStream_t s);
cudaError_t launch_kv_tiles(const AttnArgs& a, int D, int format, cudaStream_t s);    // many rows per key
// The bounded waits of the two kernels against barriers that nobody arrives on; set bits of *expired (device).
cudaError_t check_rows_waits(unsigned* expired);      // 1: a tile's copy
cudaError_t check_tiles_waits(unsigned* expired);     // 2: a role's wait, 4: one after it gave up, 8: the last wait

#ifdef __CUDACC__

// Every kernel of the cache asks for the SM's largest shared memory: a kernel that follows as a
// programmatic dependent starts beside this one's last CTAs, on SMs still split as this one asked,
// and with less shared memory only a part of the attention's CTAs would fit (measured: a third of
// the grid started when the rest had finished, 84 us against 64 us for a batch of 32).
template <typename F>
inline cudaError_t all_shared(F* kern) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
}

// Byte of the tile where a lane's code byte b stands (16-byte vectors, [vector][lane][16]).
__device__ __forceinline__ int kv_lane_byte(int lane, int b) { return (b >> 4) * 512 + lane * 16 + (b & 15); }

// First byte of the run of codes of token r's dims d.. (d a multiple of 8) in K or V.
template <int D, int kFormat>
__device__ __forceinline__ int kv_k_byte(int r, int d) {
    const int in = (r >> 3) * (D / 4) + d % (D / 4);
    return kv_lane_byte(4 * (r & 7) + d / (D / 4), kFormat == FT_KV_NVFP4 ? in / 2 : in);
}
template <int D, int kFormat>
__device__ __forceinline__ int kv_v_byte(int r, int d) {
    const int in = (2 * (r >> 3) + (r & 1)) * (D / 8) + d % (D / 8);
    return kv_tile(D, kFormat).code_bytes +
           kv_lane_byte(4 * (d / (D / 8)) + ((r & 7) >> 1), kFormat == FT_KV_NVFP4 ? in / 2 : in);
}
// Scale byte of token r's block b of 16 dims (NVFP4).
template <int D>
__device__ __forceinline__ int kv_k_scale_byte(int r, int b) {
    return kv_tile(D, FT_KV_NVFP4).k_scales + (4 * (r & 7) + b / (D / 64)) * (D / 32) + (r >> 3) * (D / 64) + b % (D / 64);
}
template <int D>
__device__ __forceinline__ int kv_v_scale_byte(int r, int b) {
    return kv_tile(D, FT_KV_NVFP4).v_scales + (b * 4 + ((r & 7) >> 1)) * 4 + 2 * (r >> 3) + (r & 1);
}

// An E4M3 byte as a pair of equal f16.
__device__ __forceinline__ uint32_t scale_pair(uint32_t byte) {
    uint32_t o;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(o) : "r"(byte * 0x101u));
    return o;
}
// Two f16 of two fp32.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Four E4M3 bytes with the NaNs among them as zeros.
__device__ __forceinline__ uint32_t e4m3_numbers(uint32_t w) {
    const uint32_t nan = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    return w & ~((nan << 1) - (nan >> 7));
}

// x / G for 0 <= x < 2^31 (division by an invariant integer through a multiplication, Granlund and
// Montgomery 1994): shift = ceil(log2 G), mul = floor(2^32 (2^shift - G) / G) + 1.
__device__ __forceinline__ int div_g(const AttnArgs& a, int x) {
    return (int)((__umulhi(a.g_mul, (unsigned)x) + (unsigned)x) >> a.g_shift);
}

// Rows and cached length of sequence s, bounded as the interface says.
struct SeqInfo {
    int q0, n, len;      // first row, rows that are computed, cached tokens that the table has pages for
    int base;            // kv_len - (q_start[s + 1] - q_start[s]): the first new token's place, whatever n and len were cut to
    bool bad;
};
__device__ __forceinline__ SeqInfo seq_info(const AttnArgs& a, int s) {
    SeqInfo r;
    const int a0 = a.q_start[s], a1 = a.q_start[s + 1], len = a.kv_len[s];
    const bool in = a0 >= 0 && a0 <= a.n_tokens && a1 >= a0;                                  // otherwise no rows
    r.q0 = in ? a0 : 0;
    const int all = in ? a1 - a0 : 0;
    r.n = min(min(all, a.n_tokens - r.q0), a.max_q);
    constexpr int kMost = 0x7FFFFC00;                                                         // block ends fit 32 bits
    const long long most = min((long long)a.table_stride << a.kv.page_shift, (long long)kMost);
    r.len = (int)min((long long)max(len, 0), most);
    r.base = min(max(len, 0), kMost) - all;
    r.bad = !in || r.n != all || r.len != len;
    return r;
}

#endif  // __CUDACC__

}  // namespace ft

struct ft_kv {
    ft_kv_desc d;
    size_t layer_bytes;
    int page_shift;
    char err[256];
};
