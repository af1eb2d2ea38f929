// A step's rows, slots and positions from the sequences' lengths, with pages taken from and given back to a stack of
// free ones.
//
// Three prefix sums over the sequences (rows, pages given, pages taken) place every token without one sequence waiting
// for another: the r-th page that is taken is the r-th from the top of the stack once everything given lies on it, so a
// token finds its page from its sequence's sums alone, in the table (held before), on the old stack, or among the given ones (their
// owners' table entries, which nobody changes).
//
// Bound by latency throughout (32 bytes a sequence, 8 a token): the launch, one round of loads, the sums' barriers, a search and a
// load per token.  16 sequences of a token each: 2.2 us in a graph, 6.2 us by calls (their host time); 200 sequences over 60,000
// places for tokens, of which 12,000 are filled, 20 ending: 6.3 us.  With sums of 64 bits it was 8.0 us (every CTA executes them, and
// a CTA's instructions are its SM's); four tokens or four given pages per thread at a time were slower (8.5 and 8.2 us).
#include "ft_kv_host.cuh"

namespace ft {

namespace {

struct PlanArgs {
    ft_kv_step c;
    int n_pages, page_shift;
    int* status;
};

// Sums stop at kMost, which no number of rows or pages that is served reaches.
constexpr unsigned kMost = 1u << 30;
__device__ __forceinline__ unsigned sum_up_to(unsigned a, unsigned b) { return min(a + b, kMost); }

// Prefix sums (with the thread's own value) of each thread's values over the block; every thread calls it.
template <int N>
__device__ __forceinline__ void block_sums(const unsigned (&v)[N], unsigned (&incl)[N], unsigned (&total)[N], unsigned (*buf)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        incl[i] = v[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned t = __shfl_up_sync(0xffffffffu, incl[i], o);
            if (lane >= o) incl[i] = sum_up_to(incl[i], t);
        }
        if (lane == 31) buf[i][warp] = incl[i];
    }
    __syncthreads();
    for (int i = warp; i < N; i += warps) {
        unsigned w = lane < warps ? buf[i][lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned t = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w = sum_up_to(w, t);
        }
        buf[i][lane] = w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (warp) incl[i] = sum_up_to(incl[i], buf[i][warp - 1]);
        total[i] = buf[i][warps - 1];
    }
    __syncthreads();
}

// How many of the ascending values at[0 .. n) are at most x.
__device__ __forceinline__ int count_up_to(const int* at, int n, int x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// A thread per sequence, then threads over the tokens.  The CTAs of a launch are one cluster: each of them works
// the sums out for itself, and the state, which may be updated in place, is written once all have read it.
__global__ void __launch_bounds__(kMaxSeqs) kv_plan_kernel(const PlanArgs a) {
    __shared__ int end[kMaxSeqs], len[kMaxSeqs], held[kMaxSeqs], want[kMaxSeqs];       // end: row after a sequence's last
    __shared__ int taken[kMaxSeqs], given_end[kMaxSeqs];                                // taken: before it, -1 if it is refused
    __shared__ unsigned buf[3][32];
    __shared__ int last_taken;
    if (threadIdx.x == 0) last_taken = 0;
    pdl_wait_and_release();
    const ft_kv_step& c = a.c;
    const int s = threadIdx.x, rank = blockIdx.x, ctas = gridDim.x;
    int bits = 0;
    int n_free = *c.n_free;
    if (n_free < 0 || n_free > a.n_pages) {
        n_free = min(max(n_free, 0), a.n_pages);
        bits |= FT_DEV_BAD_ID;
    }

    // what each sequence asks for
    int n = 0, l = 0, h = 0;
    if (s < c.n_seqs) {
        n = c.n_new[s];
        l = c.len[s];
        h = c.held[s];
    }
    const bool ends = n < 0;
    const int rows = max(n, 0), old_len = l, old_held = h;
    if (ends) l = 0;
    const long long page = 1LL << a.page_shift, after = (long long)l + rows;
    const long long wants = (after + page - 1) >> a.page_shift;
    bool fine = h >= 0 && h <= c.table_stride && h <= a.n_pages;
    if (!ends)
        fine = fine && l >= 0 && (((long long)l + page - 1) >> a.page_shift) <= h && wants <= c.table_stride && after <= 0x7FFFFFFFLL &&
               (!c.tree_mask || rows <= kTreeMax);
    const unsigned lacks = wants > h ? (unsigned)min(wants - h, (long long)kMost) : 0;
    unsigned v[3] = {min((unsigned)rows, kMost), fine ? lacks : 0, fine && wants < h ? (unsigned)(h - wants) : 0}, upto[3], total[3];
    block_sums<3>(v, upto, total, buf);
    const unsigned last = upto[0], all_rows = total[0];          // of this sequence, of all
    if (all_rows > (unsigned)c.n_tokens) {                       // those whose rows do not all fit take and give nothing
        fine = fine && (rows == 0 || last <= (unsigned)c.n_tokens);
        if (!fine) v[1] = v[2] = 0;
        block_sums<3>(v, upto, total, buf);
    }
    if (!fine) bits |= FT_DEV_BAD_ID;
    const int avail = n_free + (int)total[2];
    const bool served = fine && (v[1] == 0 || upto[1] <= min((unsigned)avail, kMost - 1));
    if (fine && !served) bits |= FT_DEV_NO_PAGES;
    if (s < c.n_seqs) {
        end[s] = (int)min(last, (unsigned)c.n_tokens);
        len[s] = l;
        held[s] = h;
        want[s] = (int)wants;
        taken[s] = served ? (int)(upto[1] - v[1]) : -1;
        given_end[s] = (int)upto[2];
    }
    // the pages that leave the stack: up to those of the last sequence that is served with any
    const unsigned most = __reduce_max_sync(0xffffffffu, served && v[1] ? upto[1] : 0);
    if ((s & 31) == 0) atomicMax(&last_taken, (int)most);
    __syncthreads();
    const int left = avail - last_taken;

    // The g-th page given back.
    auto given = [&](int g) {
        const int q = count_up_to(given_end, c.n_seqs, g);
        return c.block_table[(size_t)q * c.table_stride + want[q] + (g - (q ? given_end[q - 1] : 0))];
    };
    const int at = rank * blockDim.x + threadIdx.x, step = ctas * blockDim.x;
    const int live = (int)min(all_rows, (unsigned)c.n_tokens);
    for (unsigned i = at; i < (unsigned)c.n_tokens; i += step) {
        const int t = (int)i;
        int slot = -1, pos = 0;
        if (t < live) {
            const int q = count_up_to(end, c.n_seqs, t), row = t - (q ? end[q - 1] : 0);
            if (taken[q] >= 0) {
                const int p = len[q] + row, j = p >> a.page_shift;
                int* entry = c.block_table + (size_t)q * c.table_stride + j;
                int pg;
                if (j < held[q]) {
                    pg = *entry;
                } else {
                    const int from = avail - 1 - (taken[q] + j - held[q]);
                    pg = from >= n_free ? given(from - n_free) : c.free_pages[from];
                    if ((p & (int)(page - 1)) == 0) *entry = pg;       // a page that is taken starts with a new token
                }
                if (pg >= 0 && pg < a.n_pages) slot = (int)((long long)pg << a.page_shift) + (p & (int)(page - 1));
                else bits |= FT_DEV_BAD_ID;
                pos = c.tree_mask ? len[q] + __popcll(c.tree_mask[t] & ~(1ULL << row)) : p;
            }
        }
        c.slots[t] = slot;
        if (c.positions) c.positions[t] = pos;
    }
    // what is given and not taken at once
    const int pushed = min(left, a.n_pages) - n_free;
    if (left > a.n_pages) bits |= FT_DEV_BAD_ID;
    for (int g = at; g < pushed; g += step) c.free_pages[n_free + g] = given(g);

    if (ctas > 1) {
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    } else {
        __syncthreads();
    }
    if (rank == 0) {
        if (s < c.n_seqs) {
            c.q_start[s + 1] = end[s];
            c.kv_len[s] = served ? (int)after : 0;
            c.len_out[s] = served ? (int)after : old_len;
            c.held_out[s] = served ? (int)wants : old_held;
        }
        if (s == 0) {
            c.q_start[0] = 0;
            *c.n_free_out = min(left, a.n_pages);
        }
    }
    if (bits) atomicOr(a.status, bits);
}

}  // namespace

}  // namespace ft

using namespace ft;

extern "C" ft_status ft_kv_plan(ft_kv* kv, const ft_kv_step* call, void* stream) {
    if (!kv) return FT_ERR_ARG;
    if (!call) return fail(kv, FT_ERR_ARG, "plan: NULL call");
    const ft_kv_step& c = *call;
    if (c.n_seqs < 0 || c.n_seqs > kv->d.max_seqs || c.n_tokens < 0 || c.n_tokens >= (int)kMost || c.table_stride < 1)
        return fail(kv, FT_ERR_ARG, "plan: n_seqs, n_tokens or table_stride out of range");
    if (!c.n_free || !c.free_pages || !c.q_start || !c.n_free_out || (c.n_tokens && !c.slots) ||
        (c.n_seqs && (!c.n_new || !c.len || !c.held || !c.block_table || !c.kv_len || !c.len_out || !c.held_out)))
        return fail(kv, FT_ERR_ARG, "plan: NULL pointer");
    if (!aligned(c.tree_mask, 8)) return fail(kv, FT_ERR_ARG, "plan: misaligned tree_mask");
    if (!words(c.n_new, c.len, c.held, c.n_free, c.block_table, c.free_pages, c.q_start, c.kv_len, c.slots, c.positions, c.len_out, c.held_out,
               c.n_free_out))
        return fail(kv, FT_ERR_ARG, "plan: misaligned pointer");
    NvtxRange r("ft_kv_plan");
    cudaError_t e = prepare<kv_plan_kernel>();
    if (e != cudaSuccess) return cuda_fail(kv, e, "plan");
    PlanArgs a{c, kv->d.n_pages, kv->page_shift, static_cast<int*>(kv->d.workspace)};
    int threads = c.n_tokens > kMaxSeqs ? kMaxSeqs : c.n_tokens;
    threads = ((threads > c.n_seqs ? threads : c.n_seqs) + 31) & ~31;
    if (threads < 64) threads = 64;
    int ctas = 1;
    while (ctas < 8 && (long long)ctas * 2048 < c.n_tokens) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kv_plan_kernel, a);
    return e == cudaSuccess ? FT_OK : cuda_fail(kv, e, "plan launch");
}
