// Writing the paged key/value cache: append (head norms, rotation and store of new
// tokens), eviction (selection by accumulated weight and the copy of the kept rows) and
// commit (the accepted path of a verified tree moved behind the root's row).
#include <cuda_bf16.h>
#include <math.h>

#include "paged.cuh"

namespace dartree {

// ----------------------------------------------------------------------------- append
//
// y = x * g / sqrt(mean(x^2) + eps) per head, then (y_i, y_i+D/2) turned by the angle
// position * theta^(-2i/D); queries to q_out, keys and (unchanged) values to their page
// rows. A CTA takes TOK consecutive rows of q: their angles (reduced to [-pi, pi] in
// double, sine and cosine in float) go to shared memory once and serve all heads. A head
// belongs to D/16 lanes, each with 8 pairs (16-byte loads and stores; the mean square by
// shuffles). Everything in fp32, rounded once when stored.

constexpr int PA_NT = 256;

struct PagedFreq {
    double inv[64];  // theta^(-2i/D), i < D/2 (host, double)
};

struct AppendArgs {
    const void* q;
    const void* k;
    const void* v;
    int64_t ldq, ldk, ldv;
    const void* gq;
    const void* gk;
    const int32_t* pos_base;
    float eps;
    void* q_out;
};

// 8 consecutive values as 16-byte loads / stores
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const float4 a = reinterpret_cast<const float4*>(p)[w];
        x[4 * w] = a.x, x[4 * w + 1] = a.y, x[4 * w + 2] = a.z, x[4 * w + 3] = a.w;
    }
}
__device__ __forceinline__ void load8(const bf16_t* p, float (&x)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        x[2 * w] = bf16_bits_to_float(u[w] & 0xffffu);
        x[2 * w + 1] = bf16_bits_to_float(u[w] >> 16);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
#pragma unroll
    for (int w = 0; w < 2; ++w)
        reinterpret_cast<float4*>(p)[w] = make_float4(x[4 * w], x[4 * w + 1], x[4 * w + 2], x[4 * w + 3]);
}
__device__ __forceinline__ void store8(bf16_t* p, const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * w], x[2 * w + 1]);
        u[w] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// The request that row r of q belongs to by q_start (its last entry <= r).
__device__ __forceinline__ int paged_row_request(const int32_t* q_start, int C, int r) {
    int lo = 0, hi = C - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (q_start[m] <= r) lo = m;
        else hi = m - 1;
    }
    return lo;
}

template <typename T, int D, int TOK>
__global__ void __launch_bounds__(PA_NT) paged_append_kernel(PagedArgs a, AppendArgs x,
                                                             const __grid_constant__ PagedFreq fr) {
    constexpr int HALF = D / 2, LANES = D / 16;
    __shared__ float cs[TOK][HALF], sn[TOK][HALF];
    __shared__ int state[TOK];      // 0: not a row of the batch, 1: a slot without a node, 2: a token
    __shared__ long long at[TOK];   // element offset of head 0's row in the pages, -1: not stored
    const int r0 = int(blockIdx.x) * TOK;
    if (blockIdx.x == 0)            // every request's lengths are checked once
        for (int c = threadIdx.x; c < a.C; c += PA_NT) {
            bool bad;
            paged_request(a, c, bad);
            if (bad) set_status(a.status, DARTREE_EINTERNAL);
        }
    for (int e = threadIdx.x; e < TOK * HALF; e += PA_NT) {
        const int t = e / HALF, i = e - t * HALF, r = r0 + t;
        int st = 0;
        if (r < a.T) {
            const int c = a.q_start ? paged_row_request(a.q_start, a.C, r) : r / a.S;
            const PagedRequest q = paged_request(a, c);
            const int j = r - q.q0;
            if (j >= 0 && j < q.n_new) {
                st = 2;
                const double p = double(x.pos_base ? x.pos_base[c] : q.n_old) +
                                 double(a.pos ? a.pos[size_t(c) * a.S + j] : j);
                const double ang = p * fr.inv[i];
                const double k = rint(ang * 0.15915494309189535);       // 1 / (2 pi)
                sincosf(float(fma(-k, 6.283185307179586, ang)), &sn[t][i], &cs[t][i]);
                if (i == 0) {
                    const int row = q.n_old + j;
                    long long o = -1;
                    if (row < q.n_keys) {
                        const int pg = paged_page(a.table, a.max_pages, a.n_pages, c, row, a.log2_page);
                        if (pg < 0) set_status(a.status, DARTREE_EINTERNAL);
                        else o = (long long)paged_offset(a, pg, 0, row);
                    }
                    at[t] = o;
                }
            } else if (!a.q_start) {
                st = 1;
            }
        }
        if (i == 0) state[t] = st;
    }
    __syncthreads();
    const int l = threadIdx.x % LANES, i0 = 8 * l;
    const int units = a.Hq + 2 * a.Hkv;
    const size_t head = size_t(a.page) * D;  // elements between a page's heads
    // (whole lane groups enter or leave the loop; the shuffles stay within a group)
    const unsigned group = ((1u << LANES) - 1u) << ((threadIdx.x & 31) / LANES * LANES);
    for (int w = threadIdx.x / LANES; w < TOK * units; w += PA_NT / LANES) {
        const int t = w / units, u = w - t * units, r = r0 + t;
        if (state[t] == 0) continue;
        const bool isq = u < a.Hq, isv = u >= a.Hq + a.Hkv;
        const int g = isq ? u : isv ? u - a.Hq - a.Hkv : u - a.Hq;
        T* dst;
        if (isq) {
            dst = static_cast<T*>(x.q_out) + (size_t(r) * a.Hq + g) * D;
        } else {
            if (state[t] != 2 || at[t] < 0) continue;
            dst = static_cast<T*>(isv ? a.v : a.k) + at[t] + size_t(g) * head;
        }
        float lo[8], hi[8];
        if (state[t] == 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) lo[e] = hi[e] = 0.f;
        } else {
            const T* src = isq   ? static_cast<const T*>(x.q) + size_t(r) * x.ldq
                           : isv ? static_cast<const T*>(x.v) + size_t(r) * x.ldv
                                 : static_cast<const T*>(x.k) + size_t(r) * x.ldk;
            src += size_t(g) * D;
            load8(src + i0, lo);
            load8(src + HALF + i0, hi);
            if (!isv) {
                const T* gain = static_cast<const T*>(isq ? x.gq : x.gk);
                if (gain) {
                    float s = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) s = fmaf(lo[e], lo[e], fmaf(hi[e], hi[e], s));
#pragma unroll
                    for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(group, s, o);
                    const float f = rsqrtf(s * (1.0f / D) + x.eps);
                    float gl[8], gh[8];
                    load8(gain + i0, gl);
                    load8(gain + HALF + i0, gh);
#pragma unroll
                    for (int e = 0; e < 8; ++e) lo[e] *= f * gl[e], hi[e] *= f * gh[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float c = cs[t][i0 + e], s = sn[t][i0 + e], p = lo[e], q = hi[e];
                    lo[e] = p * c - q * s;
                    hi[e] = q * c + p * s;
                }
            }
        }
        store8(dst + i0, lo);
        store8(dst + HALF + i0, hi);
    }
}

template <typename T, int D>
static void launch_append_t(const PagedArgs& a, const AppendArgs& x, const PagedFreq& fr, cudaStream_t stream) {
    // four rows per CTA share the set-up once every SM has a CTA that way
    if (a.T >= 4 * num_sms())
        paged_append_kernel<T, D, 4><<<(a.T + 3) / 4, PA_NT, 0, stream>>>(a, x, fr);
    else
        paged_append_kernel<T, D, 1><<<a.T, PA_NT, 0, stream>>>(a, x, fr);
}

int launch_paged_append(const PagedArgs& a, const void* q, const void* k, const void* v, int64_t ldq, int64_t ldk,
                        int64_t ldv, const void* gq, const void* gk, const int32_t* pos_base, float eps, double theta,
                        void* q_out, cudaStream_t stream) {
    AppendArgs x{q, k, v, ldq, ldk, ldv, gq, gk, pos_base, eps, q_out};
    PagedFreq fr{};
    for (int i = 0; i < a.D / 2; ++i) fr.inv[i] = pow(theta, -2.0 * double(i) / double(a.D));
    KTimer kt_(KID_PAGED_APPEND, stream);
    if (a.dtype == DARTREE_BF16) {
        if (a.D == 64) launch_append_t<bf16_t, 64>(a, x, fr, stream);
        else launch_append_t<bf16_t, 128>(a, x, fr, stream);
    } else {
        if (a.D == 64) launch_append_t<float, 64>(a, x, fr, stream);
        else launch_append_t<float, 128>(a, x, fr, stream);
    }
    return cudaGetLastError() == cudaSuccess ? DARTREE_OK : DARTREE_ECUDA;
}

// ----------------------------------------------------------------------------- eviction
//
// paged_select_kernel, one CTA per (request, key/value head): the rows between `sink`
// and n - recent are ranked by (weight desc, row asc). The weight of the last kept row
// is found digit by digit (four 8-bit radix passes over order-preserving 32-bit keys);
// of the rows that carry exactly it the lowest are kept. A scan in row order then writes
// the kept rows ascending.
// paged_move_kernel: 16 bytes of one kept row per thread.

constexpr int PS_NT = 1024;

__device__ __forceinline__ uint32_t evict_key(float w) { return isnan(w) ? 0u : ord_f32(w); }

__global__ void __launch_bounds__(PS_NT) paged_select_kernel(PagedArgs a, const float* __restrict__ weights,
                                                             int budget, int sink, int recent,
                                                             int32_t* __restrict__ keep, int32_t* __restrict__ counts) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_prefix, s_left;
    __shared__ int warp_tot[PS_NT / 32], s_total;
    const int cg = int(blockIdx.x), c = cg / a.Hkv;
    const long cap = long(a.max_pages) << a.log2_page;
    const int n0 = a.n_ctx[c];
    const int n = int(min(max(long(n0), 0l), cap));
    if (threadIdx.x == 0 && n != n0) set_status(a.status, DARTREE_EINTERNAL);
    int32_t* out = keep + size_t(cg) * budget;
    if (threadIdx.x == 0 && cg == c * a.Hkv) counts[c] = min(n, budget);
    if (n <= budget) {
        for (int i = threadIdx.x; i < budget; i += PS_NT) out[i] = i < n ? i : -1;
        return;
    }
    const float* w = weights + size_t(cg) * cap;
    const int lo = sink, hi = n - recent;
    const uint32_t need = uint32_t(budget - sink - recent);  // < hi - lo
    if (threadIdx.x == 0) s_prefix = 0, s_left = need;
    uint32_t mask = 0;
    for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += PS_NT) hist[i] = 0;
        __syncthreads();
        const uint32_t prefix = s_prefix, left = s_left;
        for (int i = lo + int(threadIdx.x); i < hi; i += PS_NT) {
            const uint32_t k = evict_key(w[i]);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x < 32) {  // the digit of the left-th largest key with this prefix
            uint32_t rem = left, digit = 0;
            pick_digit_warp(hist, rem, digit);
            if (threadIdx.x == 0) s_prefix = prefix | (digit << shift), s_left = rem;
        }
        mask |= 255u << shift;
        __syncthreads();
    }
    const uint32_t last = s_prefix, ties = s_left;  // `ties` rows of key `last` are kept, the lowest ones
    // rows in order, one per thread and step: (keys above, keys equal) counted before each
    int base_gt = 0, base_eq = 0;
    for (int i = threadIdx.x; i < sink; i += PS_NT) out[i] = i;
    for (int i = threadIdx.x; i < recent; i += PS_NT) out[budget - recent + i] = hi + i;
    if (need == 0) return;
    for (int i0 = lo; i0 < hi; i0 += PS_NT) {
        const int i = i0 + int(threadIdx.x);
        const uint32_t k = i < hi ? evict_key(w[i]) : 0u;
        const bool gt = i < hi && k > last, eq = i < hi && k == last;
        const int pre = block_exclusive_scan<PS_NT>((gt ? 1 : 0) | (eq ? 1 << 16 : 0), warp_tot, &s_total);
        const int total = s_total;
        const int g = base_gt + (pre & 0xffff), e = base_eq + (pre >> 16);
        if (gt || (eq && e < int(ties))) out[sink + g + min(e, int(ties))] = i;
        base_gt += total & 0xffff;
        base_eq += total >> 16;
    }
}

constexpr int PM_NT = 256;

__global__ void __launch_bounds__(PM_NT) paged_move_kernel(PagedArgs a, const float* __restrict__ weights, int budget,
                                                           const int32_t* __restrict__ dst_table, int dst_pages,
                                                           const int32_t* __restrict__ keep,
                                                           const int32_t* __restrict__ counts,
                                                           int32_t* __restrict__ n_out,
                                                           float* __restrict__ weights_out, int row_vecs) {
    // row_vecs: 16-byte vectors of one row; a row's keys come first, then its values
    const size_t id = size_t(blockIdx.x) * PM_NT + threadIdx.x;
    if (id < size_t(a.C)) n_out[id] = counts[id];
    const int vec = int(id % (2 * row_vecs));
    const size_t rr = id / (2 * row_vecs);
    if (rr >= size_t(a.C) * a.Hkv * budget) return;
    const int r = int(rr % budget), cg = int(rr / budget), c = cg / a.Hkv, g = cg - c * a.Hkv;
    const int src = keep[rr];
    if (src < 0) return;
    const size_t cap = size_t(a.max_pages) << a.log2_page;
    if (vec == 0 && weights_out)
        weights_out[size_t(cg) * (size_t(dst_pages) << a.log2_page) + r] = weights[size_t(cg) * cap + src];
    const int sp = paged_page(a.table, a.max_pages, a.n_pages, c, src, a.log2_page);
    const int dp = paged_page(dst_table, dst_pages, a.n_pages, c, r, a.log2_page);
    if (sp < 0 || dp < 0) {
        if (vec == 0) set_status(a.status, DARTREE_EINTERNAL);
        return;
    }
    uint4* pool = static_cast<uint4*>(vec < row_vecs ? a.k : a.v);
    const int v = vec < row_vecs ? vec : vec - row_vecs;
    const size_t per = size_t(a.D) / row_vecs;  // elements of a vector
    pool[paged_offset(a, dp, g, r) / per + v] = pool[paged_offset(a, sp, g, src) / per + v];
}

int launch_paged_evict(const PagedArgs& a, const float* weights, int budget, int sink, int recent,
                       const int32_t* dst_table, int dst_pages, int32_t* keep, int32_t* n_out, float* weights_out,
                       int32_t* counts, cudaStream_t stream) {
    {
        KTimer kt_(KID_PAGED_SELECT, stream);
        paged_select_kernel<<<a.C * a.Hkv, PS_NT, 0, stream>>>(a, weights, budget, sink, recent, keep, counts);
    }
    if (cudaGetLastError() != cudaSuccess) return DARTREE_ECUDA;
    const int row_vecs = a.D * (a.dtype == DARTREE_BF16 ? 2 : 4) / 16;
    const size_t threads = size_t(a.C) * a.Hkv * budget * 2 * row_vecs;  // >= C: every n_out is written
    {
        KTimer kt_(KID_PAGED_MOVE, stream);
        paged_move_kernel<<<unsigned((threads + PM_NT - 1) / PM_NT), PM_NT, 0, stream>>>(
            a, weights, budget, dst_table, dst_pages, keep, counts, n_out, weights_out, row_vecs);
    }
    return cudaGetLastError() == cudaSuccess ? DARTREE_OK : DARTREE_ECUDA;
}

// ----------------------------------------------------------------------------- commit
//
// One CTA per request. A destination row may be the source of another row, so all rows
// of a batch of heads are read into registers before any is written: a batch holds
// PC_NT * PC_V 16-byte vectors and whole heads only.

constexpr int PC_NT = 512;
constexpr int PC_V = 8;

__global__ void __launch_bounds__(PC_NT) paged_commit_kernel(PagedArgs a, const int32_t* __restrict__ path,
                                                             const int32_t* accepted_len, int L, int32_t* n_out,
                                                             int row_vecs) {
    __shared__ long long s_src[DARTREE_MAX_L], s_dst[DARTREE_MAX_L];  // element offsets of head 0, -1: not moved
    const int c = int(blockIdx.x);
    const long cap = long(a.max_pages) << a.log2_page;
    const int n0 = a.n_ctx[c], acc0 = accepted_len[c];
    const int old = int(min(max(long(n0), 0l), cap));
    const int acc = min(max(acc0, 0), min(L, a.S - 1));
    const long end = long(old) + 1 + acc;
    if (threadIdx.x == 0 && (old != n0 || acc != acc0 || end > cap)) set_status(a.status, DARTREE_EINTERNAL);
    if (int(threadIdx.x) < acc) {
        const int slot = path[size_t(c) * L + threadIdx.x];
        const long src = long(old) + slot, dst = long(old) + 1 + threadIdx.x;
        long long so = -1, d_o = -1;
        if (slot < 1 || slot >= a.S || src >= cap || dst >= cap) {
            set_status(a.status, DARTREE_EINTERNAL);
        } else if (src != dst) {
            const int sp = paged_page(a.table, a.max_pages, a.n_pages, c, int(src), a.log2_page);
            const int dp = paged_page(a.table, a.max_pages, a.n_pages, c, int(dst), a.log2_page);
            if (sp < 0 || dp < 0) {
                set_status(a.status, DARTREE_EINTERNAL);
            } else {
                so = (long long)paged_offset(a, sp, 0, int(src));
                d_o = (long long)paged_offset(a, dp, 0, int(dst));
            }
        }
        s_src[threadIdx.x] = so;
        s_dst[threadIdx.x] = d_o;
    }
    __syncthreads();
    if (threadIdx.x == 0) n_out[c] = int(min(end, cap));
    if (acc == 0) return;
    const int per = a.D / row_vecs;                     // elements of a vector
    const int head_vecs = acc * row_vecs;               // of one head of keys or values
    const int heads = min(2 * a.Hkv, PC_NT * PC_V / head_vecs);  // >= 2: 64 rows x 32 vectors at most
    for (int h0 = 0; h0 < 2 * a.Hkv; h0 += heads) {
        const int total = min(heads, 2 * a.Hkv - h0) * head_vecs;
        uint4 x[PC_V];
        size_t to[PC_V];
        bool put[PC_V];
#pragma unroll
        for (int u = 0; u < PC_V; ++u) {
            const int e = u * PC_NT + int(threadIdx.x);
            put[u] = false;
            if (e < total) {
                const int h = h0 + e / head_vecs, f = e % head_vecs, r = f / row_vecs, v = f % row_vecs;
                if (s_src[r] >= 0) {
                    const size_t off = size_t(h >> 1) * (size_t(a.page) * a.D);
                    const uint4* pool = static_cast<const uint4*>(h & 1 ? a.v : a.k);
                    x[u] = pool[(size_t(s_src[r]) + off) / per + v];
                    to[u] = (size_t(s_dst[r]) + off) / per + v;
                    put[u] = true;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < PC_V; ++u) {
            const int e = u * PC_NT + int(threadIdx.x);
            if (put[u]) static_cast<uint4*>((h0 + e / head_vecs) & 1 ? a.v : a.k)[to[u]] = x[u];
        }
        // (the next batch holds other heads: no row of this one)
    }
}

int launch_paged_commit(const PagedArgs& a, const int32_t* path, const int32_t* accepted_len, int L, int32_t* n_out,
                        cudaStream_t stream) {
    const int row_vecs = a.D * (a.dtype == DARTREE_BF16 ? 2 : 4) / 16;
    KTimer kt_(KID_PAGED_COMMIT, stream);
    paged_commit_kernel<<<a.C, PC_NT, 0, stream>>>(a, path, accepted_len, L, n_out, row_vecs);
    return cudaGetLastError() == cudaSuccess ? DARTREE_OK : DARTREE_ECUDA;
}

}  // namespace dartree
