// Attention weight each cached row of the paged cache receives (eviction's input).
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
