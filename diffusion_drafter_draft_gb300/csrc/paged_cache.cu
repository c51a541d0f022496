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
// rows. A row of q belongs to WPT warps, each with the row's angles in shared memory
// (reduced to [-pi, pi] in double, sine and cosine in float) and gain times sine and
// cosine of its lanes' pairs in registers: a head belongs to D/16 lanes, each with 8
// pairs (16-byte loads and stores, the mean square by shuffles). Everything in fp32,
// rounded once when stored. Bound by memory once there are rows enough: 13.5 k rows of 48
// heads of 128 (150 MB each way) take 58 us, a plain copy 52; one head in hand per lane
// instead of four took 68 (24 KB in flight an SM). A few rows are latency (65 rows 5.6 us).

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
template <typename T> struct Raw8 { uint4 v[sizeof(T) / 2]; };
template <typename T>
__device__ __forceinline__ Raw8<T> raw8(const T* p) {
    Raw8<T> r;
#pragma unroll
    for (int w = 0; w < int(sizeof(T) / 2); ++w) r.v[w] = reinterpret_cast<const uint4*>(p)[w];
    return r;
}
template <typename T>
__device__ __forceinline__ void put8(T* p, const Raw8<T>& r) {
#pragma unroll
    for (int w = 0; w < int(sizeof(T) / 2); ++w) reinterpret_cast<uint4*>(p)[w] = r.v[w];
}
__device__ __forceinline__ void widen8(const Raw8<float>& r, float (&x)[8]) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        x[4 * w] = __uint_as_float(r.v[w].x), x[4 * w + 1] = __uint_as_float(r.v[w].y);
        x[4 * w + 2] = __uint_as_float(r.v[w].z), x[4 * w + 3] = __uint_as_float(r.v[w].w);
    }
}
__device__ __forceinline__ void widen8(const Raw8<bf16_t>& r, float (&x)[8]) {
    const uint32_t u[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        x[2 * w] = bf16_bits_to_float(u[w] & 0xffffu);
        x[2 * w + 1] = __uint_as_float(u[w] & 0xffff0000u);
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

template <typename T, int D, int WPT>
__global__ void __launch_bounds__(PA_NT, 2) paged_append_kernel(PagedArgs a, AppendArgs x,
                                                             const __grid_constant__ PagedFreq fr) {
    constexpr int HALF = D / 2, LANES = D / 16, HEADS = 32 / LANES;  // heads a warp has in hand
    constexpr int STEP = HEADS * WPT;
    constexpr int U = sizeof(T) == 2 ? 4 : 2;                        // heads of a lane fetched together
    __shared__ __align__(16) float cs[PA_NT / 32][HALF], sn[PA_NT / 32][HALF];
    griddep_launch_dependents();
    griddep_wait();
    if (blockIdx.x == 0)            // every request's lengths are checked once
        for (int c = threadIdx.x; c < a.C; c += PA_NT) {
            bool bad;
            paged_request(a, c, bad);
            if (bad) set_status(a.status, DARTREE_EINTERNAL);
        }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = int((blockIdx.x * (PA_NT / 32) + warp) / WPT);
    if (r >= a.T) return;
    const int l = lane % LANES, i0 = 8 * l, h0 = (warp % WPT) * HEADS + lane / LANES;
    const T* qrow = static_cast<const T*>(x.q) + size_t(r) * x.ldq + i0;
    // the first heads are on their way while the row's place and angles are found
    Raw8<T> rl[U], rh[U];
    auto fetch = [&](int h) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (h + u * STEP < a.Hq) {
                rl[u] = raw8(qrow + size_t(h + u * STEP) * D);
                rh[u] = raw8(qrow + size_t(h + u * STEP) * D + HALF);
            }
    };
    fetch(h0);
    const int c = a.q_start ? paged_row_request(a.q_start, a.C, r) : r / a.S;
    const PagedRequest q = paged_request(a, c);
    const int j = r - q.q0;
    T* qout = static_cast<T*>(x.q_out) + size_t(r) * a.Hq * D + i0;
    if (j < 0 || j >= q.n_new) {
        if (!a.q_start) {           // a slot without a node
            const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            for (int h = h0; h < a.Hq; h += STEP) {
                store8(qout + size_t(h) * D, zero);
                store8(qout + size_t(h) * D + HALF, zero);
            }
        }
        return;
    }
    const double p = double(x.pos_base ? x.pos_base[c] : q.n_old) + double(a.pos ? a.pos[size_t(c) * a.S + j] : j);
#pragma unroll
    for (int i = lane; i < HALF; i += 32) {
        const double ang = p * fr.inv[i];
        const double k = rint(ang * 0.15915494309189535);       // 1 / (2 pi)
        sincosf(float(fma(-k, 6.283185307179586, ang)), &sn[warp][i], &cs[warp][i]);
    }
    __syncwarp();
    // y_lo = f (lo ac - hi bs), y_hi = f (hi bc + lo as): gains and angles of this lane's pairs
    float ac[8], bs[8], bc[8], as[8];
    auto factors = [&](const T* gain) {
        float gl[8], gh[8];
        if (gain) {
            widen8(raw8(gain + i0), gl);
            widen8(raw8(gain + HALF + i0), gh);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float co = cs[warp][i0 + e], si = sn[warp][i0 + e];
            const float g = gain ? gl[e] : 1.f, h = gain ? gh[e] : 1.f;
            ac[e] = g * co, as[e] = g * si, bc[e] = h * co, bs[e] = h * si;
        }
    };
    // (the lanes of a head enter or leave a loop together: the shuffles stay among them)
    const unsigned group = ((1u << LANES) - 1u) << (lane / LANES * LANES);
    float lo[8], hi[8];
    auto turn = [&](const Raw8<T>& xl, const Raw8<T>& xh, bool norm) {
        widen8(xl, lo);
        widen8(xh, hi);
        float f = 1.f;
        if (norm) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(lo[e], lo[e], fmaf(hi[e], hi[e], s));
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(group, s, o);
            f = rsqrtf(s * (1.0f / D) + x.eps);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = lo[e], v = hi[e];
            lo[e] = f * (u * ac[e] - v * bs[e]);
            hi[e] = f * (v * bc[e] + u * as[e]);
        }
    };
    factors(static_cast<const T*>(x.gq));
    for (int h = h0; h < a.Hq; h += U * STEP) {
        if (h != h0) fetch(h);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (h + u * STEP < a.Hq) {
                turn(rl[u], rh[u], x.gq != nullptr);
                store8(qout + size_t(h + u * STEP) * D, lo);
                store8(qout + size_t(h + u * STEP) * D + HALF, hi);
            }
    }
    const int row = q.n_old + j;
    if (row >= q.n_keys) return;
    const int pg = paged_page(a.table, a.max_pages, a.n_pages, c, row, a.log2_page);
    if (pg < 0) {
        set_status(a.status, DARTREE_EINTERNAL);
        return;
    }
    const size_t at = paged_offset(a, pg, 0, row) + i0, head = size_t(a.page) * D;
    factors(static_cast<const T*>(x.gk));
    const T* krow = static_cast<const T*>(x.k) + size_t(r) * x.ldk + i0;
    const T* vrow = static_cast<const T*>(x.v) + size_t(r) * x.ldv + i0;
    for (int g = h0; g < a.Hkv; g += U / 2 * STEP) {
        Raw8<T> vl[U / 2], vh[U / 2];
#pragma unroll
        for (int u = 0; u < U / 2; ++u)
            if (g + u * STEP < a.Hkv) {
                const size_t o = size_t(g + u * STEP) * D;
                rl[u] = raw8(krow + o);
                rh[u] = raw8(krow + o + HALF);
                vl[u] = raw8(vrow + o);
                vh[u] = raw8(vrow + o + HALF);
            }
#pragma unroll
        for (int u = 0; u < U / 2; ++u)
            if (g + u * STEP < a.Hkv) {
                T* kd = static_cast<T*>(a.k) + at + size_t(g + u * STEP) * head;
                T* vd = static_cast<T*>(a.v) + at + size_t(g + u * STEP) * head;
                turn(rl[u], rh[u], x.gk != nullptr);
                store8(kd, lo);
                store8(kd + HALF, hi);
                put8(vd, vl[u]);
                put8(vd + HALF, vh[u]);
            }
    }
}

template <typename T, int D>
static cudaError_t launch_append_t(const PagedArgs& a, const AppendArgs& x, const PagedFreq& fr, cudaStream_t stream) {
    // a warp per row once that gives every SM two CTAs of eight warps; below, a CTA per row
    const bool wide = a.T < 16 * num_sms();
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(wide ? unsigned(a.T) : unsigned((a.T + 7) / 8));
    cfg.blockDim = dim3(PA_NT);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    KTimer kt_(KID_PAGED_APPEND, stream);
    return wide ? cudaLaunchKernelEx(&cfg, paged_append_kernel<T, D, 8>, a, x, fr)
                : cudaLaunchKernelEx(&cfg, paged_append_kernel<T, D, 1>, a, x, fr);
}

int launch_paged_append(const PagedArgs& a, const void* q, const void* k, const void* v, int64_t ldq, int64_t ldk,
                        int64_t ldv, const void* gq, const void* gk, const int32_t* pos_base, float eps, double theta,
                        void* q_out, cudaStream_t stream) {
    AppendArgs x{q, k, v, ldq, ldk, ldv, gq, gk, pos_base, eps, q_out};
    PagedFreq fr{};
    for (int i = 0; i < a.D / 2; ++i) fr.inv[i] = pow(theta, -2.0 * double(i) / double(a.D));
    const cudaError_t e = a.dtype == DARTREE_BF16
                              ? (a.D == 64 ? launch_append_t<bf16_t, 64>(a, x, fr, stream)
                                           : launch_append_t<bf16_t, 128>(a, x, fr, stream))
                              : (a.D == 64 ? launch_append_t<float, 64>(a, x, fr, stream)
                                           : launch_append_t<float, 128>(a, x, fr, stream));
    return e == cudaSuccess ? DARTREE_OK : DARTREE_ECUDA;
}

// ----------------------------------------------------------------------------- eviction
//
// paged_select_kernel, one CTA per (request, key/value head): the rows between `sink`
// and n - recent are ranked by (weight desc, row asc). Their weights become
// order-preserving 32-bit keys, held in shared memory when they fit (PS_KEYS); the key of
// the last kept row is found digit by digit (radix 2^11, 2^11, 2^10: three passes, the
// first one spread over 8 exponent and 2 mantissa bits); of the rows that carry exactly
// it the lowest are kept. Each thread then counts its own run of rows, one scan gives
// every run its place, and the kept rows are written ascending.
// paged_move_kernel: PM_U rows' 16-byte vectors per thread, their addresses looked up
// before the first is read (one vector per thread, a chain of four dependent loads each,
// took 91 us where this takes 48 for 134 MB each way, 5.6 TB/s; eight rows 67). From
// PM_STREAM bytes on neither side is meant to stay in the L2: with and without that,
// selection included, 8 MB 15.1 and 14.4 us, 17 MB 17.8 and 18.5, 34 MB 23.9 and 25.1, 134
// MB 56.7 and 60.8, and an attention over the copies that follows keeps the gain.
// 128 heads of 8192-16384 rows to 2048, 61 us: selection 14-16 us, bound by its passes' latency (one
// CTA per head), then the copy, bound by memory.

constexpr int PS_NT = 1024;
constexpr int PS_KEYS = 48 * 1024;      // keys kept in shared memory
constexpr int PS_BINS = 2048;

__device__ __forceinline__ uint32_t evict_key(float w) { return isnan(w) ? 0u : ord_f32(w); }

__global__ void __launch_bounds__(PS_NT) paged_select_kernel(PagedArgs a, const float* __restrict__ weights,
                                                             int budget, int sink, int recent, int held,
                                                             int32_t* __restrict__ keep, int32_t* __restrict__ counts) {
    extern __shared__ uint32_t keys[];              // [held]
    __shared__ uint32_t hist[PS_BINS];
    __shared__ uint32_t s_digit, s_left;
    __shared__ int warp_tot[PS_NT / 32], s_total;
    griddep_launch_dependents();
    griddep_wait();
    const int cg = int(blockIdx.x), c = cg / a.Hkv, tid = int(threadIdx.x);
    const long cap = long(a.max_pages) << a.log2_page;
    const int n0 = a.n_ctx[c];
    const int n = int(min(max(long(n0), 0l), cap));
    if (tid == 0 && n != n0) set_status(a.status, DARTREE_EINTERNAL);
    int32_t* out = keep + size_t(cg) * budget;
    if (tid == 0 && cg == c * a.Hkv) counts[c] = min(n, budget);
    if (n <= budget) {
        for (int i = tid; i < budget; i += PS_NT) out[i] = i < n ? i : -1;
        return;
    }
    for (int i = tid; i < sink; i += PS_NT) out[i] = i;
    for (int i = tid; i < recent; i += PS_NT) out[budget - recent + i] = n - recent + i;
    const uint32_t need = uint32_t(budget - sink - recent);
    if (need == 0) return;
    const float* w = weights + size_t(cg) * cap + sink;
    const int m = n - recent - sink;                // rows ranked, > need
    const bool in_smem = m <= held;
    auto key = [&](int i) -> uint32_t { return in_smem ? keys[i] : evict_key(w[i]); };
    uint32_t prefix = 0, mask = 0, left = need;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digits = pass == 2 ? 1023u : 2047u;
        for (int i = tid; i < PS_BINS; i += PS_NT) hist[i] = 0;
        __syncthreads();
        if (pass == 0 && in_smem) {
            auto take = [&](int i, float f) {
                const uint32_t k = evict_key(f);
                keys[i] = k;
                atomicAdd(&hist[k >> 21], 1u);
            };
            if ((reinterpret_cast<uintptr_t>(weights) & 15) == 0) {  // (a head's rows start 16-byte aligned)
                const int first = sink & ~3;
                const float4* w4 = reinterpret_cast<const float4*>(w - sink + first);
#pragma unroll 4
                for (int q = tid; first + 4 * q < n - recent; q += PS_NT) {
                    const float4 f = w4[q];
                    const int i = first + 4 * q - sink;
                    if (i >= 0) take(i, f.x);
                    if (i + 1 >= 0 && i + 1 < m) take(i + 1, f.y);
                    if (i + 2 >= 0 && i + 2 < m) take(i + 2, f.z);
                    if (i + 3 < m) take(i + 3, f.w);
                }
            } else {
                for (int i = tid; i < m; i += PS_NT) take(i, w[i]);
            }
        } else {
#pragma unroll 4
            for (int i = tid; i < m; i += PS_NT) {
                const uint32_t k = key(i);
                if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & digits], 1u);
            }
        }
        __syncthreads();
        // thread t: digits 2047 - 2t and 2046 - 2t; the one that holds the left-th largest key
        const uint32_t d0 = PS_BINS - 1 - 2 * tid, h0 = hist[d0], h1 = hist[d0 - 1];
        const uint32_t before = uint32_t(block_exclusive_scan<PS_NT>(int(h0 + h1), warp_tot, &s_total));
        if (before < left && left <= before + h0) {
            s_digit = d0;
            s_left = left - before;
        } else if (before + h0 < left && left <= before + h0 + h1) {
            s_digit = d0 - 1;
            s_left = left - before - h0;
        }
        __syncthreads();
        prefix |= s_digit << shift;
        left = s_left;
        mask |= digits << shift;
    }
    // rows above the last key are kept, and the lowest `left` of those that carry it (runs of
    // an odd length: the threads' shared-memory reads fall into different banks)
    const int run = ((m + PS_NT - 1) / PS_NT) | 1, i0 = min(m, tid * run), i1 = min(m, i0 + run);
    int gt = 0, eq = 0;
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = key(i);
        gt += k > prefix;
        eq += k == prefix;
    }
    const int g0 = block_exclusive_scan<PS_NT>(gt, warp_tot, &s_total);
    int e = block_exclusive_scan<PS_NT>(eq, warp_tot, &s_total);
    int o = sink + g0 + min(e, int(left));
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = key(i);
        if (k > prefix || (k == prefix && e++ < int(left))) out[o++] = sink + i;
    }
}

constexpr int PM_NT = 128;
constexpr int PM_U = 3;
constexpr int64_t PM_STREAM = int64_t(16) << 20;  // bytes copied

template <int VECS, bool STREAM>  // 16-byte vectors of a row; a row's keys come first, then its values
__global__ void __launch_bounds__(PM_NT) paged_move_kernel(PagedArgs a, const float* __restrict__ weights, int budget,
                                                           const int32_t* __restrict__ dst_table, int dst_pages,
                                                           const int32_t* __restrict__ keep,
                                                           const int32_t* __restrict__ counts,
                                                           int32_t* __restrict__ n_out,
                                                           float* __restrict__ weights_out, int per) {
    constexpr int TPR = 2 * VECS, RP = PM_NT / TPR;  // threads of a row, rows of a pass
    griddep_launch_dependents();
    griddep_wait();
    const int cg = int(blockIdx.x / per), c = cg / a.Hkv, g = cg - c * a.Hkv;
    const int r0 = int(blockIdx.x % per) * (RP * PM_U) + int(threadIdx.x) / TPR;
    const int vec = int(threadIdx.x) % TPR;
    if (threadIdx.x == 0 && blockIdx.x % per == 0 && g == 0) n_out[c] = counts[c];
    uint4* pool = static_cast<uint4*>(vec < VECS ? a.k : a.v);
    const int v = vec < VECS ? vec : vec - VECS;
    int src[PM_U], sp[PM_U], dp[PM_U];
#pragma unroll
    for (int u = 0; u < PM_U; ++u) {
        const int r = r0 + u * RP;
        src[u] = r < budget ? keep[size_t(cg) * budget + r] : -1;
    }
#pragma unroll
    for (int u = 0; u < PM_U; ++u) {
        sp[u] = dp[u] = -1;
        if (src[u] >= 0) {
            sp[u] = paged_page(a.table, a.max_pages, a.n_pages, c, src[u], a.log2_page);
            dp[u] = paged_page(dst_table, dst_pages, a.n_pages, c, r0 + u * RP, a.log2_page);
        }
    }
    uint4 x[PM_U];
    auto vector = [&](int page, int row) -> uint4& {
        return pool[((((size_t(page) * a.Hkv + g) << a.log2_page) + (row & (a.page - 1))) * VECS) + v];
    };
#pragma unroll
    for (int u = 0; u < PM_U; ++u)
        if (sp[u] >= 0 && dp[u] >= 0) x[u] = STREAM ? __ldcs(&vector(sp[u], src[u])) : vector(sp[u], src[u]);
#pragma unroll
    for (int u = 0; u < PM_U; ++u) {
        if (src[u] < 0) continue;
        const int r = r0 + u * RP;
        if (sp[u] >= 0 && dp[u] >= 0) {
            if (STREAM) __stcs(&vector(dp[u], r), x[u]);
            else vector(dp[u], r) = x[u];
        } else if (vec == 0) {
            set_status(a.status, DARTREE_EINTERNAL);
        }
        if (vec == 0 && weights_out)
            weights_out[size_t(cg) * (size_t(dst_pages) << a.log2_page) + r] =
                weights[size_t(cg) * (size_t(a.max_pages) << a.log2_page) + src[u]];
    }
}

template <int VECS>
static cudaError_t launch_move(const PagedArgs& a, const float* weights, int budget, const int32_t* dst_table,
                               int dst_pages, const int32_t* keep, const int32_t* counts, int32_t* n_out,
                               float* weights_out, cudaStream_t stream) {
    const int rows = PM_NT / (2 * VECS) * PM_U, per = (budget + rows - 1) / rows;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(a.C) * a.Hkv * per);
    cfg.blockDim = dim3(PM_NT);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    KTimer kt_(KID_PAGED_MOVE, stream);
    const bool stream_it = int64_t(a.C) * a.Hkv * budget * (2 * VECS * 16) >= PM_STREAM;
    return cudaLaunchKernelEx(&cfg, stream_it ? paged_move_kernel<VECS, true> : paged_move_kernel<VECS, false>, a,
                              weights, budget, dst_table, dst_pages, keep, counts, n_out, weights_out, per);
}

int launch_paged_evict(const PagedArgs& a, const float* weights, int budget, int sink, int recent,
                       const int32_t* dst_table, int dst_pages, int32_t* keep, int32_t* n_out, float* weights_out,
                       int32_t* counts, cudaStream_t stream) {
    {
        const int64_t cap = int64_t(a.max_pages) << a.log2_page;
        const int held = int(cap < PS_KEYS ? cap : PS_KEYS);
        static std::atomic<uint64_t> raised{0};
        if (!raise_smem(paged_select_kernel, PS_KEYS * 4, raised)) return DARTREE_ECUDA;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(unsigned(a.C) * a.Hkv);
        cfg.blockDim = dim3(PS_NT);
        cfg.dynamicSmemBytes = size_t(held) * 4;
        cfg.stream = stream;
        cudaLaunchAttribute attr[1] = {pdl_attribute()};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        KTimer kt_(KID_PAGED_SELECT, stream);
        if (cudaLaunchKernelEx(&cfg, paged_select_kernel, a, weights, budget, sink, recent, held, keep, counts) !=
            cudaSuccess)
            return DARTREE_ECUDA;
    }
    auto move = [&](auto f) {
        return f(a, weights, budget, dst_table, dst_pages, keep, counts, n_out, weights_out, stream);
    };
    const int vecs = a.D * (a.dtype == DARTREE_BF16 ? 2 : 4) / 16;
    const cudaError_t e = vecs == 8 ? move(launch_move<8>) : vecs == 16 ? move(launch_move<16>) : move(launch_move<32>);
    return e == cudaSuccess ? DARTREE_OK : DARTREE_ECUDA;
}

// ----------------------------------------------------------------------------- commit
//
// One CTA per request. A destination row may be the source of another row, so all rows
// of a batch of heads are read into registers before any is written: a batch holds
// PC_NT * PC_V 16-byte vectors and whole heads only. The rows' accumulated weights, when given,
// go with them the same way, PC_NT of them a batch. Bound by four dependent loads and the
// launch: one request 4.8 us, 64 requests 6.9; with weights, kernels of their own, 5.6 and 7.6.

constexpr int PC_NT = 512;
constexpr int PC_V = 8;

template <int VECS, bool WEIGHTS>  // 16-byte vectors of a row
__global__ void __launch_bounds__(PC_NT) paged_commit_kernel(PagedArgs a, const int32_t* __restrict__ path,
                                                             const int32_t* accepted_len, int L,
                                                             float* __restrict__ weights, int32_t* n_out) {
    __shared__ int s_row[WEIGHTS ? DARTREE_MAX_L : 1];                // cached row that moves to n_ctx + 1 + i
    __shared__ long long s_src[DARTREE_MAX_L], s_dst[DARTREE_MAX_L];  // element offsets of head 0, -1: not moved
    griddep_launch_dependents();
    griddep_wait();
    const int c = int(blockIdx.x);
    const long cap = long(a.max_pages) << a.log2_page;
    const int n0 = a.n_ctx[c], acc0 = accepted_len[c];  // (these and the path in one round trip)
    const int slot = int(threadIdx.x) < L ? path[size_t(c) * L + threadIdx.x] : 0;
    const int old = int(min(max(long(n0), 0l), cap));
    const int acc = min(max(acc0, 0), min(L, a.S - 1));
    const long end = long(old) + 1 + acc;
    if (threadIdx.x == 0 && (old != n0 || acc != acc0 || end > cap)) set_status(a.status, DARTREE_EINTERNAL);
    if (int(threadIdx.x) < acc) {
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
        if constexpr (WEIGHTS) s_row[threadIdx.x] = int(src);
        s_src[threadIdx.x] = so;
        s_dst[threadIdx.x] = d_o;
    }
    __syncthreads();
    if (threadIdx.x == 0) n_out[c] = int(min(end, cap));
    if (acc == 0) return;
    const int per = a.D / VECS;                         // elements of a vector
    const int heads = min(2 * a.Hkv, PC_NT * PC_V / (acc * VECS));  // >= 2: 64 rows x 32 vectors at most
    const uint32_t inv = 0xffffffffu / uint32_t(acc) + 1u;  // q / acc = high word of q * inv (q < 2^16, acc > 1)
    const size_t head = size_t(a.page) * a.D / per;     // vectors between a page's heads
    for (int h0 = 0; h0 < 2 * a.Hkv; h0 += heads) {
        const int total = min(heads, 2 * a.Hkv - h0) * acc * VECS;
        uint4 x[PC_V];
        uint4* to[PC_V];
#pragma unroll
        for (int u = 0; u < PC_V; ++u) {
            const int e = u * PC_NT + int(threadIdx.x);
            to[u] = nullptr;
            if (e < total) {
                const int q = e / VECS, v = e % VECS;
                const int hq = acc == 1 ? q : int(__umulhi(uint32_t(q), inv)), r = q - hq * acc, h = h0 + hq;
                if (s_src[r] >= 0) {
                    uint4* pool = static_cast<uint4*>(h & 1 ? a.v : a.k) + size_t(h >> 1) * head + v;
                    x[u] = pool[size_t(s_src[r]) / per];
                    to[u] = pool + size_t(s_dst[r]) / per;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < PC_V; ++u)
            if (to[u]) *to[u] = x[u];
        // (the next batch holds other heads: no row of this one)
    }
    if constexpr (WEIGHTS) {
        const int hb = PC_NT / acc, hq = int(threadIdx.x) / acc, r = int(threadIdx.x) - hq * acc;  // heads of a batch
        for (int g0 = 0; g0 < a.Hkv; g0 += hb) {
            const bool move = hq < hb && g0 + hq < a.Hkv && s_src[r] >= 0;
            float* const w = weights + (size_t(c) * a.Hkv + g0 + hq) * size_t(cap);
            float x = 0.f;
            if (move) x = w[s_row[r]];
            __syncthreads();
            if (move) w[old + 1 + r] = x;
        }
    }
}

template <int VECS, bool WEIGHTS>
static cudaError_t launch_commit_t(const cudaLaunchConfig_t& cfg, const PagedArgs& a, const int32_t* path,
                                   const int32_t* accepted_len, int L, float* weights, int32_t* n_out) {
    return cudaLaunchKernelEx(&cfg, paged_commit_kernel<VECS, WEIGHTS>, a, path, accepted_len, L, weights, n_out);
}

int launch_paged_commit(const PagedArgs& a, const int32_t* path, const int32_t* accepted_len, int L, float* weights,
                        int32_t* n_out, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(a.C));
    cfg.blockDim = dim3(PC_NT);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    KTimer kt_(KID_PAGED_COMMIT, stream);
    const int vecs = a.D * (a.dtype == DARTREE_BF16 ? 2 : 4) / 16;
    const auto f = weights ? (vecs == 8    ? launch_commit_t<8, true>
                              : vecs == 16 ? launch_commit_t<16, true>
                                           : launch_commit_t<32, true>)
                           : (vecs == 8    ? launch_commit_t<8, false>
                              : vecs == 16 ? launch_commit_t<16, false>
                                           : launch_commit_t<32, false>);
    return f(cfg, a, path, accepted_len, L, weights, n_out) == cudaSuccess ? DARTREE_OK : DARTREE_ECUDA;
}

}  // namespace dartree
