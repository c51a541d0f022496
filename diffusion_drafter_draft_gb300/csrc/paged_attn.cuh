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

// Groups of requests that share their first rows (a call with shared prefixes): the new tokens of a whole
// group are attended over the shared rows together, in `np` chunks of the rows; then each request's over its
// own rows in `nchunk`. The partial results of a row of q lie at chunk * rows + row, the prefix's chunks first.
struct PgGroups {
    int G, np;
    unsigned units, ctas;             // CTAs' worth of tiles of all groups (a bound), CTAs of the prefix
    const int32_t* start;             // [G + 1] first requests
    const int32_t* rows;              // [G] rows shared
    int early, early_items;           // own rows: the first CTAs take early_items (request, head) pairs each
};

struct PgArgs {
    PagedArgs a;
    int grp, tt, tiles, nchunk, rows;
    int inner;                        // a head's tiles follow one another
    float sl2;                        // scale * log2(e)
    bf16_t* out;
    float* lse;
    float* part_o;
    float2* part_ml;
    PgGroups s;
};

// Whether request c is in a group.
__device__ __forceinline__ bool paged_in_group(const PgArgs& x, int c) {
    return c >= x.s.start[0] && c < x.s.start[x.s.G];
}

// Rows that request c shares with its group, in whole pages (0: no group); `bad` is set where the group's are past the
// request's `n_old` cached ones. By a whole warp, the same for all lanes.
__device__ __forceinline__ int paged_shared_rows(const PgArgs& x, int c, int n_old, bool& bad) {
    const int lane = threadIdx.x & 31;
    int n = 0, rows = 0;                                  // starts up to c; the last one's rows
    for (int j = 0; j <= x.s.G; j += 32) {                // (starts and rows at once: one round of loads for 31 groups)
        const int s = j + lane <= x.s.G ? x.s.start[j + lane] : 0x7fffffff;
        const int r = j + lane < x.s.G ? x.s.rows[j + lane] : 0;
        const unsigned b = __ballot_sync(0xffffffffu, s <= c);
        if (b) rows = __shfl_sync(0xffffffffu, r, 31 - __clz(b));
        n += __popc(b);
        if (b != 0xffffffffu) break;
    }
    if (n == 0 || n > x.s.G) return 0;
    bad |= rows > n_old;
    const int64_t cap = int64_t(x.a.max_pages) << x.a.log2_page;
    return int(min(int64_t(max(rows, 0)), cap)) & ~(x.a.page - 1);
}

// The `unit`-th run of `per` tokens of the groups' tokens: its group's first request, rows of q, tokens, shared
// rows, and its first token among them. False past the last. By a whole warp, the same for all lanes.
struct PgUnit {
    int c, q0, n, t0, keys;
};
__device__ __forceinline__ bool paged_shared_unit(const PgArgs& x, unsigned unit, int per, PgUnit& u, bool& bad) {
    const int lane = threadIdx.x & 31;
    const PagedArgs& a = x.a;
    const int64_t cap = int64_t(a.max_pages) << a.log2_page;
    bad = false;
    bool found = false;
    unsigned before = 0;
    for (int j0 = 0; j0 < x.s.G; j0 += 32) {
        const int j = j0 + lane;
        int c = 0, f0 = 0, f1 = 0;
        bool wrong = false;
        if (j < x.s.G) {
            const int s0 = x.s.start[j], s1 = x.s.start[j + 1];
            c = min(max(s0, 0), a.C);
            const int e = min(max(s1, c), a.C);
            wrong = c != s0 || e != s1 || x.s.rows[j] < 0 || x.s.rows[j] > cap;
            if (a.q_start) {
                f0 = min(max(a.q_start[c], 0), a.T);
                f1 = min(max(a.q_start[e], f0), a.T);
            } else {
                f0 = c * a.S, f1 = e * a.S;
            }
        }
        bad |= __any_sync(0xffffffffu, wrong) != 0;
        const unsigned mine = unsigned((f1 - f0 + per - 1) / per);
        unsigned inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, unit < before + inc);
        if (hit && !found) {
            const int l = __ffs(hit) - 1;
            u.c = __shfl_sync(0xffffffffu, c, l);
            u.q0 = __shfl_sync(0xffffffffu, f0, l);
            u.n = __shfl_sync(0xffffffffu, f1, l) - u.q0;
            u.t0 = int(unit - before - __shfl_sync(0xffffffffu, inc - mine, l)) * per;
            u.keys = int(min(int64_t(max(x.s.rows[j0 + l], 0)), cap)) & ~(a.page - 1);
            if (unit != 0) return true;                   // (the first unit's CTAs look at all groups)
            found = true;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    return found;
}

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

constexpr int PF_BM = 128;           // few rows: keys of a block
constexpr int PF_N = 16;             // rows

// Column-wise reduction of 16 values per lane over a warp: lane i gets column i % 16.
template <class F>
__device__ __forceinline__ float warp_columns(float (&v)[PF_N], int lane, F op) {
#pragma unroll
    for (int w = PF_N / 2; w > 0; w >>= 1) {
        const bool up = lane & w;
#pragma unroll
        for (int k = 0; k < w; ++k) {
            const float mine = up ? v[k + w] : v[k], other = up ? v[k] : v[k + w];
            v[k] = op(mine, __shfl_xor_sync(0xffffffffu, other, w));
        }
    }
    return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
}

// Few rows (paged_few.cu): tiles of 16 rows, one per request and key/value head.
int launch_paged_few(const PgArgs& x, bool cluster, bool alone, const CUtensorMap& tq,
                     const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream);
// Their own rows in a call with shared prefixes, and the join (paged_own.cu).
int launch_paged_own(const PgArgs& x, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t stream);

}  // namespace dartree
