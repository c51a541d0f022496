// Pages and rows of a step from the requests' lengths: reserve (pages for the new tokens,
// block tables, first rows of q, slots of the tokens) and release (pages behind the rows that
// a request keeps).
//
//   need_c = ceil((old_c + new_c) / page) - ceil(old_c / page)
//
// pages come from the end of a stack of free ones, in the order of the requests; a request is
// granted when its need and its tokens fit what those before it left. The work is a few words
// a request and 16 bytes a token, so a call is a launch and a chain of dependent loads: one
// cluster of up to eight CTAs, each of which scans the requests, PP_NT at a time, and does its
// share of the pages and tokens (a grid would need a second launch before n_free may change).
// Where the requests of a turn do not all fit, one warp goes through them, 32 at a time: those
// that want more than is left can never fit and drop out, the others are granted up to the
// first whose prefix does not fit; a few rounds a group.
// 64 trees of 65 slots 5.4 us in a graph (10.6 with the host's time of calls one after another), 512 requests of up to
// 128 tokens, a quarter refused, 13.6 (13.5), 64 releases 3.5 (8.5).
#include "paged.cuh"

namespace dartree {

constexpr int PP_NT = 512;
constexpr int PP_CLUSTER = 8;

struct ReserveArgs {
    int C, T, S, log2_page, n_pages, max_pages;
    int32_t* table;
    const int32_t* n_ctx;
    const int32_t* n_new;
    const int32_t* free_pages;
    const int32_t* n_free;
    int32_t* q_start;   // null: S rows to a request
    int32_t* granted;
    int32_t* n_free_out;
    int64_t* slot;
    int32_t* pos;
    int32_t* request;
    int* status;
};

// Last entry of off[0 .. n) that is at most i (off ascending, off[0] <= i).
__device__ __forceinline__ int pp_find(const int* off, int n, int i) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (off[m] <= i) lo = m;
        else hi = m - 1;
    }
    return lo;
}

// Inclusive sum over the lanes.
__device__ __forceinline__ int pp_scan(int v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

__global__ void __launch_bounds__(PP_NT) paged_reserve_kernel(const __grid_constant__ ReserveArgs a) {
    __shared__ int need[PP_NT], want[PP_NT];            // of the turn's requests; want < 0: none to grant
    __shared__ int pages_at[PP_NT], rows_at[PP_NT];     // sums before a request
    __shared__ int old_s[PP_NT], held_s[PP_NT], got[PP_NT];
    __shared__ int wtot[PP_NT / 32], total;
    const int tid = threadIdx.x, lane = tid & 31;
    const int cta = int(cluster_ctarank()), ctas = int(cluster_nctarank());
    const int share = cta * PP_NT + tid, step = ctas * PP_NT;
    griddep_launch_dependents();
    griddep_wait();
    const int page = 1 << a.log2_page;
    const int64_t cap = int64_t(a.max_pages) << a.log2_page;
    const int stack0 = *a.n_free, stack = min(max(stack0, 0), a.n_pages);
    if (stack != stack0 && share == 0) set_status(a.status, DARTREE_EINTERNAL);
    int pages_used = 0, rows_used = 0;                  // by the turns before
    for (int c0 = 0; c0 < a.C; c0 += PP_NT) {
        const int n = min(PP_NT, a.C - c0), c = c0 + tid;
        int old = 0, held = 0, nd = 0, wt = -1;
        if (tid < n) {
            const int o = a.n_ctx[c], w = a.n_new[c];
            const bool bad = o < 0 || o > cap || w < 0 || w > a.S;
            if (bad) {
                if (cta == 0) set_status(a.status, DARTREE_EINTERNAL);
            } else {
                old = o;
                held = (o + page - 1) >> a.log2_page;   // (rows + S + 1024 < 2^31)
                nd = ((o + w + page - 1) >> a.log2_page) - held;
                if (int64_t(o) + w <= cap) wt = w;
            }
        }
        if (wt < 0) nd = 0;
        old_s[tid] = old, held_s[tid] = held, need[tid] = nd, want[tid] = wt;
        // (sums of a turn: at most 512 (S / 16 + 1) pages and 512 S tokens; those of all C by
        // C * S below 2^31)
        int pb = block_exclusive_scan<PP_NT>(nd, wtot, &total);
        const int all_pages = total;
        __syncthreads();
        int rb = block_exclusive_scan<PP_NT>(max(wt, 0), wtot, &total);
        const int all_rows = total;
        __syncthreads();
        int turn_pages = all_pages, turn_rows = all_rows;
        if (all_pages <= stack - pages_used && (!a.q_start || all_rows <= a.T - rows_used)) {
            pages_at[tid] = pb, rows_at[tid] = rb, got[tid] = max(wt, 0);
        } else {
            if (tid < 32) {
                int left = stack - pages_used, room = a.q_start ? a.T - rows_used : 0x7fffffff;
                int pu = 0, ru = 0;
                for (int g = 0; g < PP_NT; g += 32) {
                    const int my_need = need[g + lane], my_want = want[g + lane];
                    bool in = my_want >= 0, given = false;
                    while (true) {
                        in = in && my_need <= left && my_want <= room;
                        if (!__any_sync(0xffffffffu, in)) break;
                        const int sp = pp_scan(in ? my_need : 0), sr = pp_scan(in ? my_want : 0);
                        const unsigned over = __ballot_sync(0xffffffffu, in && (sp > left || sr > room));
                        const int first = over ? __ffs(over) - 1 : 32;
                        const bool now = in && lane < first;
                        given |= now;
                        if (now) in = false;
                        // (the sums of the last lane before `first`; lane `first` fits alone, so first > 0)
                        left -= __shfl_sync(0xffffffffu, sp, first - 1);
                        room -= __shfl_sync(0xffffffffu, sr, first - 1);
                        if (!over) break;
                    }
                    const int ep = pp_scan(given ? my_need : 0), er = pp_scan(given ? my_want : 0);
                    pages_at[g + lane] = pu + ep - (given ? my_need : 0);
                    rows_at[g + lane] = ru + er - (given ? my_want : 0);
                    got[g + lane] = given ? my_want : -1;
                    pu += __shfl_sync(0xffffffffu, ep, 31);
                    ru += __shfl_sync(0xffffffffu, er, 31);
                }
                if (lane == 0) wtot[0] = pu, wtot[1] = ru;
            }
            __syncthreads();
            turn_pages = wtot[0], turn_rows = wtot[1];
            if (got[tid] < 0) need[tid] = 0, got[tid] = 0;
        }
        __syncthreads();
        if (cta == 0 && tid < n) {
            a.granted[c] = got[tid];
            if (a.q_start) a.q_start[c] = rows_used + rows_at[tid];
        }
        // page i of the turn
        auto taken = [&](int i) -> int { return a.free_pages[stack - 1 - pages_used - i]; };
        for (int i = share; i < turn_pages; i += step) {
            const int r = pp_find(pages_at, n, i), p = taken(i);
            if (unsigned(p) >= unsigned(a.n_pages)) set_status(a.status, DARTREE_EINTERNAL);
            a.table[size_t(c0 + r) * a.max_pages + held_s[r] + (i - pages_at[r])] = p;
        }
        if (a.slot || a.pos || a.request) {
            const int rows = a.q_start ? turn_rows : n * a.S;
            for (int i = share; i < rows; i += step) {
                const int r = a.q_start ? pp_find(rows_at, n, i) : i / a.S;
                const int k = i - (a.q_start ? rows_at[r] : r * a.S);
                const size_t at = a.q_start ? size_t(rows_used) + i : size_t(c0) * a.S + i;
                const bool live = k < got[r];
                const int j = old_s[r] + k, pi = j >> a.log2_page;
                if (a.slot) {
                    int64_t s = -1;
                    if (live) {
                        const int p = pi < held_s[r] ? a.table[size_t(c0 + r) * a.max_pages + pi]
                                                     : taken(pages_at[r] + pi - held_s[r]);
                        if (unsigned(p) < unsigned(a.n_pages)) s = (int64_t(p) << a.log2_page) + (j & (page - 1));
                        else set_status(a.status, DARTREE_EINTERNAL);
                    }
                    a.slot[at] = s;
                }
                if (a.pos) a.pos[at] = live ? j : -1;
                if (a.request) a.request[at] = live ? c0 + r : -1;
            }
        }
        pages_used += turn_pages, rows_used += turn_rows;
        __syncthreads();                                // (the next turn writes what this one reads)
    }
    if (a.q_start) {
        for (int i = rows_used + share; i < a.T; i += step) {
            if (a.slot) a.slot[i] = -1;
            if (a.pos) a.pos[i] = -1;
            if (a.request) a.request[i] = -1;
        }
        if (share == 0) a.q_start[a.C] = rows_used;
    }
    cluster_sync();                                     // every CTA has read n_free
    if (share == 0) *a.n_free_out = stack - pages_used;
}

struct ReleaseArgs {
    int C, log2_page, n_pages, max_pages;
    const int32_t* table;
    const int32_t* n_held;
    const int32_t* n_keep;
    const int32_t* n_shared;  // or null
    int32_t* free_pages;
    const int32_t* n_free;
    int32_t* n_free_out;
    int* status;
};

__global__ void __launch_bounds__(PP_NT) paged_release_kernel(const __grid_constant__ ReleaseArgs a) {
    __shared__ int first[PP_NT], at[PP_NT];
    __shared__ int wtot[PP_NT / 32], total;
    const int tid = threadIdx.x;
    const int cta = int(cluster_ctarank()), ctas = int(cluster_nctarank());
    const int share = cta * PP_NT + tid, step = ctas * PP_NT;
    griddep_launch_dependents();
    griddep_wait();
    const int page = 1 << a.log2_page;
    const int64_t cap = int64_t(a.max_pages) << a.log2_page;
    const int stack0 = *a.n_free, stack = min(max(stack0, 0), a.n_pages);
    if (stack != stack0 && share == 0) set_status(a.status, DARTREE_EINTERNAL);
    int64_t used = stack;
    for (int c0 = 0; c0 < a.C; c0 += PP_NT) {
        const int n = min(PP_NT, a.C - c0), c = c0 + tid;
        int lo = 0, count = 0;
        if (tid < n) {
            const int h0 = a.n_held[c], k0 = a.n_keep[c], s0 = a.n_shared ? a.n_shared[c] : 0;
            const int h = int(min(int64_t(max(h0, 0)), cap)), k = int(min(int64_t(max(max(k0, s0), 0)), cap));
            if (cta == 0 && (h != h0 || k0 < 0 || s0 < 0)) set_status(a.status, DARTREE_EINTERNAL);
            lo = (k + page - 1) >> a.log2_page;
            count = max(((h + page - 1) >> a.log2_page) - lo, 0);
        }
        first[tid] = lo;
        const int before = block_exclusive_scan<PP_NT>(count, wtot, &total);
        at[tid] = before;
        const int turn = total;
        __syncthreads();
        for (int i = share; i < turn; i += step) {
            const int r = pp_find(at, n, i);
            const int p = a.table[size_t(c0 + r) * a.max_pages + first[r] + (i - at[r])];
            const bool fits = used + i < a.n_pages;     // (more pages than the pool has: given back twice)
            if (!fits || unsigned(p) >= unsigned(a.n_pages)) set_status(a.status, DARTREE_EINTERNAL);
            if (fits) a.free_pages[used + i] = p;
        }
        used += turn;
        __syncthreads();
    }
    cluster_sync();
    if (share == 0) *a.n_free_out = int(min(used, int64_t(a.n_pages)));
}

// One cluster: a CTA for about every 2048 tokens (16 requests' pages), at most eight.
template <typename Args>
static int launch_pages(int id, void (*kernel)(const Args), const Args& a, int64_t work, cudaStream_t stream) {
    int n = 1;
    while (n < PP_CLUSTER && int64_t(n) * 2048 < work) n *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(n));
    cfg.blockDim = dim3(PP_NT);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2] = {pdl_attribute()};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(n);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    KTimer kt_(id, stream);
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? DARTREE_OK : DARTREE_ECUDA;
}

int launch_paged_reserve(const PagedArgs& p, const dartree_paged_step& x, cudaStream_t stream) {
    const ReserveArgs a{p.C, p.T, p.S, p.log2_page, p.n_pages, p.max_pages, x.table, x.n_ctx, x.n_new, x.free_pages,
                        x.n_free, x.q_start, x.granted, x.n_free_out, x.slot, x.pos, x.request, p.status};
    const bool tokens = x.slot || x.pos || x.request;
    return launch_pages(KID_PAGED_RESERVE, paged_reserve_kernel, a, tokens ? int64_t(p.T) : int64_t(p.C) * 16, stream);
}

int launch_paged_release(const PagedArgs& p, const int32_t* table, const int32_t* n_held, const int32_t* n_keep,
                         const int32_t* n_shared, int32_t* free_pages, const int32_t* n_free, int32_t* n_free_out,
                         cudaStream_t stream) {
    const ReleaseArgs a{p.C, p.log2_page, p.n_pages, p.max_pages, table, n_held, n_keep, n_shared, free_pages, n_free,
                        n_free_out, p.status};
    return launch_pages(KID_PAGED_RELEASE, paged_release_kernel, a, int64_t(p.C) * 16, stream);
}

}  // namespace dartree
