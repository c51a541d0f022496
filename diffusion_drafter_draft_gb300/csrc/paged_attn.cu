// Attention of new tokens over the paged cache and the attention weight each cached row
// receives: the plain kernels (CUDA cores, fp32).
#include <cuda_bf16.h>
#include <math.h>

#include "paged.cuh"

namespace dartree {

// Whether new token i of request c sees row j of it (j < n_keys).
__device__ __forceinline__ bool paged_sees(const PagedArgs& a, const PagedRequest& r, int c, int i, int j) {
    if (j < r.n_old) return true;
    const int s = j - r.n_old;
    return a.mask ? a.mask[(size_t(c) * a.S + i) * a.S + s] != 0 : s <= i;
}

// ----------------------------------------------------------------------------- attention
//
// One warp per (row of q, query head): 32 keys a step, one score per lane, the running
// maximum and sum of the softmax across the warp; each lane holds D / 32 values of the
// output.

constexpr int PG_NT = 256;

template <int D>
__global__ void __launch_bounds__(PG_NT) paged_attn_kernel(PagedArgs a, const bf16_t* __restrict__ q, float scale,
                                                           bf16_t* __restrict__ out, float* __restrict__ lse) {
    __shared__ float sq[PG_NT / 32][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const size_t id = size_t(blockIdx.x) * (PG_NT / 32) + warp;  // (request, token, head)
    if (id >= size_t(a.C) * a.S * a.Hq) return;
    const int h = int(id % a.Hq), i = int(id / a.Hq % a.S), c = int(id / a.Hq / a.S);
    bool bad;
    const PagedRequest r = paged_request(a, c, bad);
    if (bad && h == 0 && i == 0 && lane == 0) set_status(a.status, DARTREE_EINTERNAL);
    if (i >= r.n_new) {
        if (!a.q_start) {  // a slot without a node
            const size_t row = size_t(c) * a.S + i;
            for (int d = lane; d < D; d += 32) out[(row * a.Hq + h) * D + d] = bf16_t{0};
            if (lse && lane == 0) lse[row * a.Hq + h] = -INFINITY;
        }
        return;
    }
    const size_t row = size_t(r.q0) + i;
    const int g = h / (a.Hq / a.Hkv);
    for (int d = lane; d < D; d += 32) sq[warp][d] = to_float(q[(row * a.Hq + h) * D + d]);
    __syncwarp();
    const bf16_t* kp = static_cast<const bf16_t*>(a.k);
    const bf16_t* vp = static_cast<const bf16_t*>(a.v);
    float m = -INFINITY, l = 0.f, acc[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
    for (int j0 = 0; j0 < r.n_keys; j0 += 32) {
        const int j = j0 + lane;
        long long off = -1;
        float s = -INFINITY;
        if (j < r.n_keys && paged_sees(a, r, c, i, j)) {
            const int pg = paged_page(a.table, a.max_pages, a.n_pages, c, j, a.log2_page);
            if (pg < 0) {
                set_status(a.status, DARTREE_EINTERNAL);
            } else {
                off = (long long)paged_offset(a, pg, g, j);
                float x = 0.f;
                for (int d = 0; d < D; ++d) x = fmaf(sq[warp][d], to_float(kp[off + d]), x);
                s = x * scale;
            }
        }
        const float mx = fmaxf(m, warp_max(s));
        if (mx == -INFINITY) continue;
        const float f = expf(m - mx), p = expf(s - mx);
        l = l * f + warp_sum(p);
        m = mx;
        const float pb = to_float(from_float<bf16_t>(p));
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[e] *= f;
        for (int t = 0; t < 32; ++t) {
            const float w = __shfl_sync(0xffffffffu, pb, t);
            const long long o = __shfl_sync(0xffffffffu, off, t);
            if (o < 0) continue;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(w, to_float(vp[o + lane + 32 * e]), acc[e]);
        }
    }
    const float inv = l > 0.f ? 1.0f / l : 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) out[(row * a.Hq + h) * D + lane + 32 * e] = from_float<bf16_t>(acc[e] * inv);
    if (lse && lane == 0) lse[row * a.Hq + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

size_t paged_attention_part_bytes(const PagedArgs&) { return 0; }

int launch_paged_attention(const PagedArgs& a, const void* q, float scale, void* out, float* lse, void*,
                           cudaStream_t stream) {
    const size_t warps = size_t(a.C) * a.S * a.Hq;
    const unsigned grid = unsigned((warps + PG_NT / 32 - 1) / (PG_NT / 32));
    KTimer kt_(KID_PAGED_ATTN, stream);
    if (a.D == 64)
        paged_attn_kernel<64><<<grid, PG_NT, 0, stream>>>(a, static_cast<const bf16_t*>(q), scale,
                                                          static_cast<bf16_t*>(out), lse);
    else
        paged_attn_kernel<128><<<grid, PG_NT, 0, stream>>>(a, static_cast<const bf16_t*>(q), scale,
                                                           static_cast<bf16_t*>(out), lse);
    return cudaGetLastError() == cudaSuccess ? DARTREE_OK : DARTREE_ECUDA;
}

// ----------------------------------------------------------------------------- weights
//
// One thread per cached row of a (request, key/value head): the key in registers, the
// query rows of the group one after the other in shared memory.

constexpr int PW_NT = 128;

template <int D>
__global__ void __launch_bounds__(PW_NT) paged_weights_kernel(PagedArgs a, const bf16_t* __restrict__ q,
                                                              const float* __restrict__ lse, float scale, float decay,
                                                              float* __restrict__ weights, int blocks) {
    __shared__ float sq[D];
    const int cg = int(blockIdx.x / blocks), c = cg / a.Hkv, g = cg - c * a.Hkv;
    const int j = int(blockIdx.x % blocks) * PW_NT + threadIdx.x;
    bool bad;
    const PagedRequest r = paged_request(a, c, bad);
    if (bad && threadIdx.x == 0) set_status(a.status, DARTREE_EINTERNAL);
    const bool real = j < r.n_keys;
    float key[D];
    bool held = false;
    if (real) {
        const int pg = paged_page(a.table, a.max_pages, a.n_pages, c, j, a.log2_page);
        if (pg < 0) {
            set_status(a.status, DARTREE_EINTERNAL);
        } else {
            held = true;
            const bf16_t* kp = static_cast<const bf16_t*>(a.k) + paged_offset(a, pg, g, j);
#pragma unroll
            for (int d = 0; d < D; ++d) key[d] = to_float(kp[d]);
        }
    }
    const int grp = a.Hq / a.Hkv;
    float sum = 0.f;
    for (int i = 0; i < r.n_new; ++i)
        for (int hg = 0; hg < grp; ++hg) {
            const size_t row = (size_t(r.q0) + i) * a.Hq + g * grp + hg;
            __syncthreads();
            for (int d = threadIdx.x; d < D; d += PW_NT) sq[d] = to_float(q[row * D + d]);
            __syncthreads();
            if (!held || !paged_sees(a, r, c, i, j)) continue;
            float x = 0.f;
#pragma unroll
            for (int d = 0; d < D; ++d) x = fmaf(sq[d], key[d], x);
            const float l = lse[row];
            if (l > -INFINITY) sum += expf(x * scale - l);
        }
    if (real) {
        float* w = weights + size_t(cg) * (size_t(a.max_pages) << a.log2_page) + j;
        *w = j < r.n_old ? fmaf(decay, *w, sum) : sum;
    }
}

int launch_paged_weights(const PagedArgs& a, const void* q, const float* lse, float scale, float decay,
                         float* weights, cudaStream_t stream) {
    const int blocks = ((a.max_pages << a.log2_page) + PW_NT - 1) / PW_NT;
    const unsigned grid = unsigned(a.C) * a.Hkv * blocks;
    KTimer kt_(KID_PAGED_WEIGHTS, stream);
    if (a.D == 64)
        paged_weights_kernel<64><<<grid, PW_NT, 0, stream>>>(a, static_cast<const bf16_t*>(q), lse, scale, decay,
                                                             weights, blocks);
    else
        paged_weights_kernel<128><<<grid, PW_NT, 0, stream>>>(a, static_cast<const bf16_t*>(q), lse, scale, decay,
                                                              weights, blocks);
    return cudaGetLastError() == cudaSuccess ? DARTREE_OK : DARTREE_ECUDA;
}

}  // namespace dartree
