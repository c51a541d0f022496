// Device helpers of the paged key/value cache: a request's lengths and the place of a
// cached row, both checked against the buffers before anything is read or written.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace dartree {

struct PagedRequest {
    int q0;      // first row of q
    int n_new;   // new tokens (used tree slots)
    int n_old;   // rows cached before them
    int n_keys;  // rows the block table holds of n_old + n_new
};

// Lengths of request c, clamped to what the buffers hold; `bad` is set when a clamp
// changed one.
__device__ __forceinline__ PagedRequest paged_request(const PagedArgs& a, int c, bool& bad) {
    PagedRequest r;
    const long cap = long(a.max_pages) << a.log2_page;  // <= 2^31 - 1 (checked on the host)
    if (a.q_start) {
        const int s0 = a.q_start[c], s1 = a.q_start[c + 1];
        r.q0 = min(max(s0, 0), a.T);
        const int e = min(max(s1, r.q0), a.T);
        r.n_new = min(e - r.q0, a.S);
        bad = r.q0 != s0 || e != s1 || r.n_new != e - r.q0;
    } else {
        const int n = a.n_nodes ? a.n_nodes[c] : a.S;
        r.q0 = c * a.S;
        r.n_new = min(max(n, 0), a.S);
        bad = r.n_new != n;
    }
    const long old = a.n_ctx[c];
    r.n_old = int(min(max(old, 0l), cap));
    const long keys = long(r.n_old) + r.n_new;
    r.n_keys = int(min(keys, cap));
    bad |= r.n_old != old || r.n_keys != keys;
    return r;
}
__device__ __forceinline__ PagedRequest paged_request(const PagedArgs& a, int c) {
    bool bad;
    return paged_request(a, c, bad);
}

// Page of cached row j of request c, -1 when the table's entry is no page of the pool.
__device__ __forceinline__ int paged_page(const int32_t* table, int width, int n_pages, int c, int j, int log2_page) {
    const int p = table[size_t(c) * width + (j >> log2_page)];
    return unsigned(p) < unsigned(n_pages) ? p : -1;
}
// Element offset of row j (in its page) of head g.
__device__ __forceinline__ size_t paged_offset(const PagedArgs& a, int page, int g, int j) {
    return (((size_t(page) * a.Hkv + g) << a.log2_page) + (j & (a.page - 1))) * a.D;
}

}  // namespace dartree
