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

// ----------------------------------------------------------------------------- arithmetic of the scores

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two fp32 values per instruction (fma, add) and the larger of three.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) { return pair(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

}  // namespace dartree
