// What the kernels of the paged attention share: arguments, the merge of chunks that are
// a cluster.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include "paged.cuh"

namespace dartree {

constexpr float PG_MOST = 16384.0f;    // weights from which a new maximum is taken
constexpr float LOG2E = 1.4426950408889634f;
constexpr int PG_CLUSTER = 8;         // chunks that merge through shared memory

struct PgArgs {
    PagedArgs a;
    int grp, tt, tiles, nchunk, rows;
    int inner;                        // a head's tiles follow one another
    float sl2;                        // scale * log2(e)
    bf16_t* out;
    float* lse;
    float* part_o;
    float2* part_ml;
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// The chunks of a tile are a cluster: CTA `chunk` merges every nchunk-th of `rows` rows (warp `warp`
// of `warps` every warps-th of them, at most 32) from all CTAs' O (ob, `pitch` floats a row) and
// (maximum, sum) (ml), and writes output and lse. places[row]: token * heads + head, -2 - that for a
// tree slot without a node (zeros), -1: no row.
// Lane i has the place of the warp's row i and, from one round of reads, its factors
// 2^(m_j - m) / sum (four trees of 65 slots: 27.1 us, 29.9 with a round of reads for every row); the
// first row's O is on its way before they are known. One row in hand: two take 26.7, but a single
// token then 11.0 instead of 10.7 (more code, run once out of a cold cache).
template <int D>
__device__ __forceinline__ void paged_merge(const PgArgs& x, const float* ob, int pitch, const float2* ml,
                                            const int* places, int rows, int chunk, int warp, int warps) {
    constexpr int V = D / 32;                            // values of a row per lane
    const int lane = threadIdx.x & 31;
    const int k0 = chunk + x.nchunk * warp, step = x.nchunk * warps, kl = k0 + step * lane;
    const int place = kl < rows ? places[kl] : -1;
    float f[PG_CLUSTER], lj[PG_CLUSTER], o[PG_CLUSTER][V];
#pragma unroll
    for (int j = 0; j < PG_CLUSTER; ++j) {
        f[j] = -INFINITY, lj[j] = 0.f;
        if (j < x.nchunk && place != -1) ld_dsmem_f32x2(dsmem_addr(ml + kl, j), f[j], lj[j]);
    }
    bool known = false;
    unsigned left = __ballot_sync(0xffffffffu, place != -1);
#pragma unroll 1
    while (left) {
        const int i = __ffs(left) - 1;
        left &= left - 1;
#pragma unroll
        for (int j = 0; j < PG_CLUSTER; ++j)
            if (j < x.nchunk) {
                const uint32_t src = dsmem_addr(ob + (k0 + step * i) * pitch + lane * V, j);
                if (V == 4) ld_dsmem_f32x4(src, o[j][0], o[j][1], o[j][V - 2], o[j][V - 1]);
                else ld_dsmem_f32x2(src, o[j][0], o[j][1]);
            }
        if (!known) {
            known = true;
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int j = 0; j < PG_CLUSTER; ++j) top = fmaxf(top, f[j]);
#pragma unroll
            for (int j = 0; j < PG_CLUSTER; ++j) {
                f[j] = lj[j] > 0.f ? ex2(f[j] - top) : 0.f;
                sum = fmaf(f[j], lj[j], sum);
            }
            const float inv = sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
            for (int j = 0; j < PG_CLUSTER; ++j) f[j] *= inv;
            if (x.lse && place != -1)
                x.lse[place >= 0 ? place : -2 - place] =
                    sum > 0.f ? (top + log2f(sum)) * 0.6931471805599453f : place >= 0 ? -INFINITY : 0.f;
        }
        float acc[V];
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll
        for (int j = 0; j < PG_CLUSTER; ++j) {
            const float fj = __shfl_sync(0xffffffffu, f[j], i);
            if (j < x.nchunk && fj > 0.f)                // (nothing seen there: O may be anything)
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] = fmaf(fj, o[j][e], acc[e]);
        }
        const int to = __shfl_sync(0xffffffffu, place, i);
        uint32_t* dst = reinterpret_cast<uint32_t*>(x.out + size_t(to >= 0 ? to : -2 - to) * D) + lane * (V / 2);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) dst[e] = pack2(acc[2 * e], acc[2 * e + 1]);
    }
}

// Few rows (paged_few.cu): tiles of 16 rows, one per request and key/value head.
int launch_paged_few(const PgArgs& x, bool cluster, bool alone, const CUtensorMap& tq,
                     const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream);

}  // namespace dartree
