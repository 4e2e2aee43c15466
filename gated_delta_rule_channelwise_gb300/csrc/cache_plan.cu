// Block tables and slots from request lengths (cgdr_cache_plan).
//
// A few kilobytes of integers: the launch itself is the time (250 requests of a token: 4.0 us; 33 prompts of
// 66,000 tokens: 6.0 us).  So there is one launch and no wait
// between blocks: every block forms the two prefix sums over the requests (new tokens, pages taken)
// again in shared memory, finds the same verdict on capacity, and then fills its share of the
// tokens and of the new table entries, finding each one's request by bisection.  What one block
// writes no block reads: a token on a new page takes the page from the free stack, not from the
// table entry that another block may be writing, and the free count that is read is another word
// than the one written.
#include "serve.cuh"

namespace cgdr {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanTokens = 1024;                     // tokens of a block
constexpr int kMaxRequests = 8192;
constexpr int kStaticBytes = 1024;                    // of shared memory at most, beside the sums

struct PlanParams {
    cgdr_plan_args a;
    int64_t e_table;                                  // footprint of the table (index-checking build)
};

__device__ __forceinline__ int pages_for(int64_t tokens, int page) { return (int)((tokens + page - 1) / page); }

// The last b in [0, B) with first[b] <= i (first is ascending, first[0] = 0).
__device__ __forceinline__ int owner(const int *first, int B, int i) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const PlanParams pp) {
    const cgdr_plan_args &p = pp.a;
    extern __shared__ int s_first[];                  // new tokens before request b, [B + 1]
    int *s_taken = s_first + p.B + 1;                 // pages taken before request b, [B + 1]
    __shared__ int64_t s_warp[2][kPlanThreads / 32];
    static_assert(sizeof(s_warp) <= kStaticBytes, "shared memory beside the sums");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int NW = kPlanThreads / 32;
    const int count = *p.free_count;

    // prefix sums in 64 bits, so that no sum of lengths wraps before it is refused
    int64_t tokens = 0, pages = 0;                    // of the requests already summed
    bool invalid = count < 0 || count > p.F, over = false;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int64_t t = 0, g = 0;
        if (b < p.B) {
            const int64_t old = p.seq_lens[b], fresh = p.new_lens[b];
            if (old < 0 || fresh < 0) invalid = true;
            else {
                const int64_t need = (old + fresh + p.page - 1) / p.page;
                if (need > p.width || old + fresh > INT32_MAX) over = true;
                t = fresh;
                g = need - (old + p.page - 1) / p.page;
            }
        }
        int64_t ti = t, gi = g;                       // inclusive sums over the warp, then over the warps
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, ti, d), y = __shfl_up_sync(0xffffffffu, gi, d);
            if (lane >= d) { ti += x; gi += y; }
        }
        if (lane == 31) { s_warp[0][warp] = ti; s_warp[1][warp] = gi; }
        __syncthreads();
        int64_t tb = tokens, gb = pages;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) { tb += s_warp[0][w]; gb += s_warp[1][w]; }
            tokens += s_warp[0][w];
            pages += s_warp[1][w];
        }
        if (b < p.B) {                                // sums past 32 bits are refused below, unread
            s_first[b] = (int)(tb + ti - t);
            s_taken[b] = (int)(gb + gi - g);
        }
        __syncthreads();
    }
    if (tokens > p.n_tokens || pages > count) over = true;
    if (!invalid && !over) {                          // the pages to be taken have to be pages of the cache
        for (int j = tid; j < pages; j += kPlanThreads) {
            const int page = p.free_pages[count - 1 - j];
            if (page < 0 || page >= p.num_pages) invalid = true;
        }
    }
    const bool wrong = __syncthreads_or(invalid), bad = __syncthreads_or(over) || wrong;
    if (tid == 0) { s_first[p.B] = (int)tokens; s_taken[p.B] = (int)pages; }
    __syncthreads();
    const int total = bad ? 0 : (int)tokens, taken = bad ? 0 : (int)pages;

    const int gtid = blockIdx.x * kPlanThreads + tid, gsize = gridDim.x * kPlanThreads;
    if (gtid == 0) {
        *p.free_count_out = count - taken;
        p.cu[p.B] = total;
        if (bad && p.status != nullptr) atomicExch(p.status, wrong ? (int)CGDR_ERR_INVALID_ARG : (int)CGDR_ERR_CAPACITY);
    }
    for (int b = gtid; b < p.B; b += gsize) {
        p.cu[b] = bad ? 0 : s_first[b];
        p.kv_lens[b] = bad ? p.seq_lens[b] : p.seq_lens[b] + p.new_lens[b];
    }
    for (int j = gtid; j < taken; j += gsize) {       // table entries of the new pages
        const int b = owner(s_taken, p.B, j);
        const int64_t e = b * p.table_sb + pages_for(p.seq_lens[b], p.page) + (j - s_taken[b]);
        if (in_bounds(e, pp.e_table, p.status, nullptr)) p.block_table[e] = p.free_pages[count - 1 - j];
    }
    for (int i = gtid; i < p.n_tokens; i += gsize) {
        int b = -1, pos = -1;
        int64_t slot = -1;
        if (i < total) {
            b = owner(s_first, p.B, i);
            const int old = p.seq_lens[b], held = pages_for(old, p.page);
            pos = old + i - s_first[b];
            const int at = pos / p.page;
            int page = -1;
            if (at >= held) page = p.free_pages[count - 1 - (s_taken[b] + at - held)];
            else if (in_bounds(b * p.table_sb + at, pp.e_table, p.status, nullptr)) page = p.block_table[b * p.table_sb + at];
            slot = (int64_t)page * p.page + pos % p.page;
        }
        p.requests[i] = b;
        p.positions[i] = pos;
        p.slots[i] = slot < 0 ? -1 : slot;
    }
}

cgdr_status check(const cgdr_plan_args *a) {
    if (!a) return CGDR_ERR_INVALID_ARG;
    if (a->B < 0 || a->width < 0 || a->n_tokens < 0 || a->F < 0 || a->num_pages < 0) return CGDR_ERR_INVALID_ARG;
    if (!page_ok(a->page) || a->B > kMaxRequests || a->n_tokens > kMaxTokens) return CGDR_ERR_UNSUPPORTED;
    if (!a->free_count || !a->free_count_out || !a->cu) return CGDR_ERR_INVALID_ARG;
    if (a->F > 0 && !a->free_pages) return CGDR_ERR_INVALID_ARG;
    if (a->B > 0 && (!a->seq_lens || !a->new_lens || !a->kv_lens || (a->width > 0 && !a->block_table)))
        return CGDR_ERR_INVALID_ARG;
    if (a->n_tokens > 0 && (!a->requests || !a->positions || !a->slots)) return CGDR_ERR_INVALID_ARG;
    if (a->free_count == a->free_count_out || (a->B > 0 && a->seq_lens == a->kv_lens)) return CGDR_ERR_INVALID_ARG;
    if (a->table_sb < (a->B > 1 ? a->width : 0)) return CGDR_ERR_INVALID_ARG;
    const void *words[] = {a->block_table, a->seq_lens, a->new_lens, a->free_pages, a->free_count, a->free_count_out,
                           a->kv_lens, a->cu, a->requests, a->positions, a->status};
    for (const void *w : words)
        if (!aligned_to(w, 4)) return CGDR_ERR_ALIGNMENT;
    return aligned_to(a->slots, 8) ? CGDR_OK : CGDR_ERR_ALIGNMENT;
}

}  // namespace
}  // namespace cgdr

extern "C" cgdr_status cgdr_cache_plan(const cgdr_plan_args *a, void *stream) {
    using namespace cgdr;
    const cgdr_status st = check(a);
    if (st != CGDR_OK) return st;
    static SmemOnce smem_once;
    const int bytes = 2 * (a->B + 1) * (int)sizeof(int);
    if (bytes + kStaticBytes > 48 * 1024 &&           // the limit without it covers both kinds
        !smem_limit_once(smem_once, reinterpret_cast<const void *>(cache_plan_kernel), 2 * (kMaxRequests + 1) * (int)sizeof(int)))
        return CGDR_ERR_CUDA;
    const int work = a->n_tokens > a->B ? a->n_tokens : a->B;
    int grid = (work + kPlanTokens - 1) / kPlanTokens;
    grid = grid < 1 ? 1 : grid > 256 ? 256 : grid;
    PlanParams p{*a, a->B > 0 ? (a->B - 1) * a->table_sb + a->width : 0};
    cache_plan_kernel<<<grid, kPlanThreads, bytes, static_cast<cudaStream_t>(stream)>>>(p);
    return launched();
}
