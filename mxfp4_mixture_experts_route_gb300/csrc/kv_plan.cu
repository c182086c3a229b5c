// Block tables, slot maps, positions and tree masks from request lengths.
//
// With c_b cached and n_b new tokens of request b and pages of P tokens:
//   row_start_b = sum_{a<b} n_a
//   old_b = ceil(c_b / P), new_b = ceil((c_b + n_b) / P)
//   entry j in [old_b, new_b) of row b = free[sum_{a<b} (new_a - old_a) + j - old_b],
//   the list of free pages ending at its length or its first negative entry
//   slot of row i = entry((c_b + i) / P) * P + (c_b + i) % P
//   mask row i = {i} + its ancestors, position c_b + (ancestors of i)
//
// Bound: latency (a step's lengths and tables are kilobytes).  So it is one
// launch in which no CTA waits for another: every CTA scans all the lengths
// itself (two counts packed into one 64-bit word, one block scan per 256
// requests) and then writes its own share, taking a fresh page's id from the
// free list rather than from the table entry another CTA writes.  Measured: 3.3 us
// for 8 requests of 8 drafted tokens, 6.5 us for 512 of 64, 5.9 us for 64 prompts of
// up to 4096, of which the launch and the scan are 2.5 to 3.
#include "kv.cuh"

namespace moe {
namespace {

constexpr int PLAN_THREADS = 256;

struct PlanShared {
    int row[KV_MAX_B + 1];      // first row of each request (clamped to T), then their total
    int page[KV_MAX_B + 1];     // free pages taken before each request
    unsigned long long warp_sum[PLAN_THREADS / 32];
    int parent[32 * KV_MAX_W];
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// a request's new tokens (0 when it does not fit) and the free pages it takes
struct PlanReq {
    int c, n, old_pages, new_pages;
};
__device__ __forceinline__ PlanReq plan_request(const KvDims& d, const PlanArgs& a, int b, bool report) {
    PlanReq r;
    r.c = ld_dep(a.ctx_len + b);
    r.n = ld_dep(a.n_new + b);
    const bool ok = r.c >= 0 && r.n >= 0 && (int64_t)r.c + r.n <= (int64_t)d.max_pages * d.page && r.n <= (1 << 20) &&
                    (d.W == 0 || r.n <= 32 * d.W);
    if (!ok) {
        if (report) latch_status(a.sb, MOE_ERR_BAD_LENGTHS, b);
        r.c = r.n = 0;
    }
    r.old_pages = ceil_div(r.c, d.page);
    r.new_pages = ceil_div(r.c + r.n, d.page);
    return r;
}

// the page that holds token `at` of request b; -1 when there is none
__device__ __forceinline__ int page_of(const KvDims& d, const PlanArgs& a, const PlanReq& r, int b, int taken, int j) {
    int id;
    if (j < r.old_pages) {
        id = ld_dep(a.block_table + (int64_t)b * d.max_pages + j);
    } else {
        const int64_t f = (int64_t)taken + (j - r.old_pages);
        if (f >= a.n_free) return -1;
        id = ld_dep(a.free_pages + f);
        if (id < 0) return -1;               // the list's end
    }
    if (id < 0 || id >= d.n_pages) {
        latch_status(a.sb, MOE_ERR_BAD_PAGE, id);
        return -1;
    }
    return id;
}

template <bool TREE>
__global__ void __launch_bounds__(PLAN_THREADS) k_kv_plan(const KvDims d, const PlanArgs a) {
    __shared__ PlanShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    KT_MARK(K_KV_PLAN, 0);
    pdl_wait();
    KT_MARK(K_KV_PLAN, 1);
    // prefix sums of rows (low 33 bits: at most 2^12 requests of 2^20 rows) and pages
    unsigned long long base = 0;
    for (int b0 = 0; b0 < d.B; b0 += PLAN_THREADS) {
        const int b = b0 + tid;
        unsigned long long v = 0;
        if (b < d.B) {
            const PlanReq r = plan_request(d, a, b, blockIdx.x == 0);
            v = (unsigned long long)(r.new_pages - r.old_pages) << 33 | (unsigned)r.n;
        }
        unsigned long long s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        if (lane == 31) sh.warp_sum[warp] = s;
        __syncthreads();
        unsigned long long before = base;
#pragma unroll
        for (int w = 0; w < PLAN_THREADS / 32; ++w) {
            const unsigned long long u = sh.warp_sum[w];
            if (w < warp) before += u;
            base += u;
        }
        if (b < d.B) {
            const unsigned long long ex = before + s - v, rows = ex & ((1ull << 33) - 1);
            sh.row[b] = rows < (unsigned long long)d.T ? (int)rows : d.T;
            sh.page[b] = (int)(ex >> 33);
        }
        __syncthreads();
    }
    const unsigned long long rows = base & ((1ull << 33) - 1);
    const int pages = (int)(base >> 33);
    const int total = rows < (unsigned long long)d.T ? (int)rows : d.T;
    if (tid == 0) sh.row[d.B] = total;
    __syncthreads();
    const int listed = pages < a.n_free ? pages : a.n_free;   // entries of the free list that are taken, if it has them
    const bool reports = blockIdx.x == 0 && tid == PLAN_THREADS - 1;   // (of the warp with the fewest rows)
    // (looked at when the rows are done)
    const int last = reports && listed > 0 ? ld_dep(a.free_pages + listed - 1) : 0;
    if (blockIdx.x == 0) {
        for (int b = tid; b <= d.B; b += PLAN_THREADS) a.row_start[b] = sh.row[b];
        if (reports) {
            a.used[0] = total;
            if (rows > (unsigned long long)d.T) latch_status(a.sb, MOE_ERR_BAD_LENGTHS, d.B);
        }
    }
    // fresh table entries, a request a CTA at a time
    for (int b = blockIdx.x; b < d.B; b += gridDim.x) {
        const PlanReq r = plan_request(d, a, b, false);
        for (int j = r.old_pages + tid; j < r.new_pages; j += PLAN_THREADS) {
            const int id = page_of(d, a, r, b, sh.page[b], j);
            a.block_table[(int64_t)b * d.max_pages + j] = id;
            const int f = sh.page[b] + (j - r.old_pages);
            // a negative entry with a page behind it: not the list's end
            if (id < 0 && f + 1 < listed && ld_dep(a.free_pages + f) < 0 && ld_dep(a.free_pages + f + 1) >= 0)
                latch_status(a.sb, MOE_ERR_BAD_PAGE, ld_dep(a.free_pages + f));
        }
        if (TREE) {
            // the rows of this request: the walk up from each, parents in shared memory
            const int r0 = sh.row[b], n = sh.row[b + 1] - r0;
            __syncthreads();
            for (int i = tid; i < n; i += PLAN_THREADS) sh.parent[i] = ld_dep(a.parents + r0 + i);
            __syncthreads();
            for (int i = tid; i < n; i += PLAN_THREADS) {
                const int at = r.c + i;
                const int pg = page_of(d, a, r, b, sh.page[b], at / d.page);
                a.slots[r0 + i] = pg < 0 ? -1 : (int64_t)pg * d.page + at % d.page;
                int cur = i, depth = -1;
                for (int w = d.W - 1; w >= 0; --w) {
                    uint32_t bits = 0;
                    while (cur >= 0 && (cur >> 5) == w) {
                        bits |= 1u << (cur & 31);
                        ++depth;
                        const int up = sh.parent[cur];
                        if (up >= cur || up < -1) {
                            latch_status(a.sb, MOE_ERR_BAD_PARENT, r0 + cur);
                            cur = -1;
                        } else {
                            cur = up;
                        }
                    }
                    a.mask[(int64_t)(r0 + i) * d.W + w] = bits;
                }
                a.positions[r0 + i] = r.c + depth;
            }
        }
    }
    // chains: rows by position in the batch; and the rows that no request owns
    const int first = TREE ? total : 0;
    for (int t = first + blockIdx.x * PLAN_THREADS + tid; t < d.T; t += gridDim.x * PLAN_THREADS) {
        if (t >= total) {
            a.slots[t] = -1;
            a.positions[t] = -1;
            for (int w = 0; w < d.W; ++w) a.mask[(int64_t)t * d.W + w] = 0;
            continue;
        }
        int lo = 0, hi = d.B;   // the last request with row[b] <= t
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (sh.row[m] <= t) lo = m; else hi = m;
        }
        const PlanReq r = plan_request(d, a, lo, false);
        const int at = r.c + (t - sh.row[lo]);
        const int pg = page_of(d, a, r, lo, sh.page[lo], at / d.page);
        a.slots[t] = pg < 0 ? -1 : (int64_t)pg * d.page + at % d.page;
        a.positions[t] = at;
    }
    if (reports) {
        int taken = listed;
        if (last < 0) {   // the list ends before: entries below lo are pages, hi is none
            int lo = 0, hi = listed - 1;
            while (lo < hi) {
                const int m = (lo + hi) >> 1;
                if (ld_dep(a.free_pages + m) < 0) hi = m; else lo = m + 1;
            }
            taken = hi;
        }
        a.used[1] = taken;
        if (pages > taken) latch_status(a.sb, MOE_ERR_NO_PAGES, pages - taken);
    }
    KT_MARK(K_KV_PLAN, 2);
}

}  // namespace

cudaError_t launch_kv_plan(const KvDims& d, const PlanArgs& a, cudaStream_t st) {
    KT_BIND();
    timing_begin(K_KV_PLAN, st);
    // a request a CTA in trees; a CTA's width of rows a CTA in chains
    const int want = a.parents ? d.B : (d.T + PLAN_THREADS - 1) / PLAN_THREADS;
    const int most = 4 * num_sms();
    const dim3 grid(want < most ? want : most);
    const cudaError_t e = a.parents ? launch_pdl(k_kv_plan<true>, grid, dim3(PLAN_THREADS), 0, st, d, a)
                                    : launch_pdl(k_kv_plan<false>, grid, dim3(PLAN_THREADS), 0, st, d, a);
    timing_end(st);
    return e;
}

}  // namespace moe
