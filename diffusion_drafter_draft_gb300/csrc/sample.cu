// Tokens drawn under temperature, top-k, top-p and min-p from given uniform numbers, and the
// walk of a verification tree on such draws.
//
//   w_v = exp((x_v - max x) / T)
//   kept: the k first in the order (x descending, token ascending); of those the smallest
//         leading set that holds top_p of their weight; of those w_v >= min_p (the first
//         always stays)
//   token: the lowest with  sum of kept w_0 .. w_v  >  u * sum of all kept w
//
// A token hangs on the last digits of these sums: a sum over 150 thousand fp32 weights, off by
// 1e-7 of itself, lands on a neighbour wherever weights are smaller than that. So weights are
// integers, 2^42 for the largest, off by half a unit and about 2^-42 of themselves (float pairs:
// the difference exact, a table of 2^(-j/128), a cubic), and sums are exact 64-bit integers, the
// same in any order and for any split of the row.
//
// One cluster per row; each CTA keeps its slice in shared memory, so the logits are read once.
//   load    slice to shared memory, maximum and minimum
//   select  (top-k, top-p) a histogram of 2048 bins of x between maximum and minimum, counts or
//           weights; the bin in which k, or top_p of the weight, is reached; then finer bins of that
//           bin's keys, until it holds at most 256 elements or one value. Those go to a list in
//           CTA 0, which finds the last one kept by comparing all pairs (equal values: the r-th
//           by token). If all that top-k keeps fits the list, CTA 0 finishes there.
//   draw    sums of each warp's stretch of the row; the warp that holds the goal walks its own.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace dartree {

constexpr int SP_NT = 512;
constexpr int SP_WARPS = SP_NT / 32;
constexpr int SP_BINS = 2048;
constexpr int SP_LIST = 256;
constexpr int SP_MAXC = 8;        // CTAs of a cluster
constexpr int SP_Q = 42;          // a weight of 1 is 2^42; 2^20 of them stay below 2^63

struct SampleArgs {
    const void* x;
    int64_t ld;                   // elements between rows
    int V, seg;                   // seg: elements of a CTA's slice
    float temperature, top_p, min_p;
    int top_k;
    const float* temperatures;    // per request, or null
    const int32_t* top_ks;
    const float* top_ps;
    const float* min_ps;
    const float* u;
    int32_t* tok;                 // rows
    int* status;
    // walk of a tree
    int L, B, per;                // per: rows of logits (and of u) to a request
    const int32_t* t_tok;
    const int32_t* t_par;
    const int32_t* t_depth;       // null: a row for each slot
    const int32_t* n_nodes;
    int32_t* accepted;
    int32_t* path;
    int32_t* bonus;
    float2 table[129];            // 2^(-j/128) as a pair of floats
};

// The settings of a request, and what the weights need of them.
struct Filter {
    float T, p, least, u;
    int k;
    float ch, cl;                 // log2(e) / T as a pair
    uint64_t wmin;                // least weight that min-p keeps
    bool greedy;
};

struct Crossing {                 // where a measure summed from the top reaches its goal
    uint64_t above, mass;         // measure of the bins before the bin, and of all
    uint32_t bin, cnt_above, cnt;
    uint32_t pad;
};

struct SpShared {
    uint32_t cnt[SP_BINS];        // histogram: elements,
    uint32_t lo[SP_BINS], hi[SP_BINS];   // weights (64 bits in two words)
    float2 table[129];            // SampleArgs::table
    uint64_t list[SP_LIST];       // CTA 0: (key, ~token)
    uint64_t lw[SP_LIST], kw[SP_LIST];
    uint64_t sums[SP_MAXC][SP_WARPS];    // of every warp of the cluster
    uint64_t tot_mass[SP_MAXC];
    uint32_t tot_cnt[SP_MAXC];
    uint64_t red[SP_WARPS];
    uint32_t redc[SP_WARPS];
    float top[SP_MAXC], low[SP_MAXC];
    uint32_t first[SP_MAXC];
    Filter f;
    Crossing x;
    uint32_t list_n, kthr, ithr, token;
    uint64_t rest, total;
};

__device__ __forceinline__ uint64_t sp_warp_sum(uint64_t v) {
#pragma unroll
    for (int m = 16; m; m >>= 1) v += shfl_xor_u64(v, m);
    return v;
}
__device__ __forceinline__ uint64_t sp_warp_scan(uint64_t v) {   // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t a = __shfl_up_sync(0xffffffffu, uint32_t(v), o);
        const uint32_t b = __shfl_up_sync(0xffffffffu, uint32_t(v >> 32), o);
        if (lane >= o) v += (uint64_t(b) << 32) | a;
    }
    return v;
}
__device__ __forceinline__ void st_dsmem_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(addr), "r"(v) : "memory");
}

// The weight of x in units of 2^-42.
//   t = (m - x) log2(e) / T = n + f; j = round(128 f), r = f - j / 128, z = r ln 2
//   2^-t = 2^-n 2^(-j/128) (1 - z + z^2/2 - z^3/6 + z^4/24),  |z| < 0.0028
// The difference, t, -z and the product are pairs of floats (errors below 2^-43 of the weight);
// the powers from z^2 on are below 2^-18, in single precision.
__device__ __forceinline__ uint64_t sp_weight(float x, float m, const Filter& f, const float2* table) {
    if (x == m) return uint64_t(1) << SP_Q;
    const float d = __fsub_rn(m, x);
    const float bb = __fsub_rn(d, m);
    const float e = __fsub_rn(__fsub_rn(m, __fsub_rn(d, bb)), __fadd_rn(x, bb));
    const float th = __fmul_rn(d, f.ch);
    if (!(th < float(SP_Q + 2))) return 0;            // below half a unit (also x = -inf)
    const float tl = __fmaf_rn(d, f.ch, -th) + __fmaf_rn(d, f.cl, e * f.ch);
    const float n = floorf(th), fr = __fsub_rn(th, n);
    const float j = rintf(fr * 128.0f);
    const float r = __fmaf_rn(j, -0.0078125f, fr);     // exact
    constexpr float LH = 0.693147182464599609375f, LL = -1.904654323148236017e-9f;   // ln 2
    const float zh = __fmul_rn(r, LH);
    const float zl = __fmaf_rn(r, LH, -zh) + __fmaf_rn(r, LL, tl * LH);
    const float z2 = zh * zh;
    const float q = z2 * __fmaf_rn(zh, __fmaf_rn(zh, 1.0f / 24.0f, -1.0f / 6.0f), 0.5f);
    const float el = q - zl;                           // e^-z - 1 = -zh + el
    const float2 t = table[int(j)];
    const float ph = __fmul_rn(t.x, -zh), pl = __fmaf_rn(t.x, -zh, -ph);
    const float rest = (t.y + pl) + __fmaf_rn(t.x, el, -t.y * zh);
    const float wh = __fadd_rn(t.x, ph);
    const float wl = __fadd_rn(__fadd_rn(__fsub_rn(t.x, wh), ph), rest);
    const int64_t w = (int64_t(__float2int_rn(wh * 16777216.0f)) << (SP_Q - 24)) +
                      __float2int_rn(wl * float(int64_t(1) << SP_Q));   // wh in [1/2, 1]: exact; |wl| < 2^-23
    const int s = int(n);
    return s ? uint64_t((w + (int64_t(1) << (s - 1))) >> s) : uint64_t(w);
}

template <typename T> struct SpElem;
template <> struct SpElem<float> {
    static constexpr int VEC = 4;
    static __device__ __forceinline__ void widen(const uint4& v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float clean(float x) { return fmaxf(x, -INFINITY); }   // NaN: never drawn
    static __device__ __forceinline__ uint4 clean4(uint4 v) {
        float x[4];
        widen(v, x);
        return make_uint4(__float_as_uint(clean(x[0])), __float_as_uint(clean(x[1])), __float_as_uint(clean(x[2])),
                          __float_as_uint(clean(x[3])));
    }
    static __device__ __forceinline__ float none() { return -INFINITY; }
    static __device__ __forceinline__ float get(const float* p) { return clean(*p); }
    static __device__ __forceinline__ void put(float* p, float x) { *p = x; }
};
template <> struct SpElem<bf16_t> {
    static constexpr int VEC = 8;
    static __device__ __forceinline__ void widen(const uint4& v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint32_t clean2(uint32_t w) {
        const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162*>(&w);
        const __nv_bfloat162 low = __halves2bfloat162(__ushort_as_bfloat16(0xff80), __ushort_as_bfloat16(0xff80));
        const __nv_bfloat162 r = __hmax2(a, low);      // (the operand that is a number)
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    static __device__ __forceinline__ uint4 clean4(uint4 v) {
        return make_uint4(clean2(v.x), clean2(v.y), clean2(v.z), clean2(v.w));
    }
    static __device__ __forceinline__ float get(const bf16_t* p) { return fmaxf(to_float(*p), -INFINITY); }
    static __device__ __forceinline__ void put(bf16_t* p, float x) { *p = bf16_t{uint16_t(__float_as_uint(x) >> 16)}; }
};

// A CTA's slice of a row: `nv` vectors in shared memory, element e of vector v being token
// first + v * VEC + e (first may lie before the slice; what is no element of it is -inf).
template <typename T>
struct Slice {
    const uint4* v;
    int nv, first, lo, hi;
};

// Elements that are still in question: bin1 of the first histogram and a range of keys.
struct Range {
    float m, s;                   // bin of x: (m - x) * s
    int bin;                      // -1: no bin chosen yet
    uint32_t khi, klo;
    int shift;
};
__device__ __forceinline__ int sp_bin(float x, const Range& g) {
    return int(fminf(__fmul_rn(__fsub_rn(g.m, x), g.s), float(SP_BINS - 1)));
}

struct Kept {                     // the last element kept, (key, token)
    uint32_t key, idx;
    __device__ __forceinline__ bool has(uint32_t k, uint32_t i) const { return k > key || (k == key && i <= idx); }
};

// Everything a row needs of the cluster. All functions are called by all threads of the cluster.
template <typename T>
struct Sampler {
    using E = SpElem<T>;
    static constexpr int VEC = E::VEC;
    SpShared& sh;
    Slice<T> sl;
    uint32_t S, cr;               // CTAs, this one
    int* status;

    template <typename F>
    __device__ __forceinline__ void each(F f) const {          // f(x, token), this thread's elements
        for (int i = threadIdx.x; i < sl.nv; i += SP_NT) {
            float x[VEC];
            E::widen(sl.v[i], x);
#pragma unroll
            for (int e = 0; e < VEC; ++e) f(x[e], sl.first + i * VEC + e);
        }
    }

    __device__ __forceinline__ bool real(int tok) const { return tok >= sl.lo && tok < sl.hi; }

    // (count, mass) summed over the block, to all threads
    __device__ void block_sum(uint32_t& c, uint64_t& w) {
        const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
        c = __reduce_add_sync(0xffffffffu, c);
        w = sp_warp_sum(w);
        __syncthreads();
        if (lane == 0) sh.redc[wid] = c, sh.red[wid] = w;
        __syncthreads();
        c = 0, w = 0;
#pragma unroll
        for (int i = 0; i < SP_WARPS; ++i) c += sh.redc[i], w += sh.red[i];
    }

    // Histogram of the kept elements in g and the bin where the goal is reached: count k (MASS false) or
    // the share p of the whole weight (first histogram) or the weight `goal` (finer ones).
    template <bool MASS>
    __device__ Crossing crossing(const Range& g, const Kept& kept, const Filter& f, float m, bool share, uint64_t goal) {
        for (int i = threadIdx.x; i < SP_BINS; i += SP_NT) {
            sh.cnt[i] = 0;
            if (MASS) sh.lo[i] = 0, sh.hi[i] = 0;
        }
        __syncthreads();
        each([&](float x, int tok) {
            if (!real(tok)) return;
            const uint32_t key = ord_f32(x);
            if (!kept.has(key, uint32_t(tok))) return;
            int b = sp_bin(x, g);
            if (g.bin >= 0) {
                if (b != g.bin || key > g.khi || key < g.klo) return;
                b = int((g.khi - key) >> g.shift);
            }
            atomicAdd(&sh.cnt[b], 1u);
            if (MASS) {
                const uint64_t w = sp_weight(x, m, f, sh.table);
                if (!w) return;
                const uint32_t wl = uint32_t(w);
                const uint32_t before = atomicAdd(&sh.lo[b], wl);
                const uint32_t up = uint32_t(w >> 32) + (before + wl < wl ? 1u : 0u);
                if (up) atomicAdd(&sh.hi[b], up);
            }
        });
        cluster_sync();
        // CTA r sums bins [r * nb, (r + 1) * nb) over the cluster, consecutive bins to a thread
        const int nb = SP_BINS / int(S), per = (nb + SP_NT - 1) / SP_NT;   // 1, 2 or 4
        uint32_t c[4] = {0, 0, 0, 0};
        uint64_t w[4] = {0, 0, 0, 0};
        const int b0 = int(cr) * nb + int(threadIdx.x) * per;
        const bool mine = int(threadIdx.x) * per < nb;
        uint32_t cs = 0;
        uint64_t ws = 0;
        if (mine)
            for (uint32_t q = 0; q < S; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < per) {
                        const uint32_t n = ld_dsmem_u32(dsmem_addr(&sh.cnt[b0 + i], q));
                        c[i] += n, cs += n;
                        if (MASS) {
                            const uint64_t v = (uint64_t(ld_dsmem_u32(dsmem_addr(&sh.hi[b0 + i], q))) << 32) +
                                               ld_dsmem_u32(dsmem_addr(&sh.lo[b0 + i], q));
                            w[i] += v, ws += v;
                        }
                    }
        // sums before this thread's bins: over the warps, then the CTAs
        const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
        const uint32_t ci = uint32_t(sp_warp_scan(cs));
        const uint64_t wi = MASS ? sp_warp_scan(ws) : 0;
        if (lane == 31) sh.redc[wid] = ci, sh.red[wid] = wi;
        __syncthreads();
        uint32_t cb = ci - cs, ct = 0;
        uint64_t wb = wi - ws, wt = 0;
#pragma unroll
        for (int i = 0; i < SP_WARPS; ++i) {
            if (i < wid) cb += sh.redc[i], wb += sh.red[i];
            ct += sh.redc[i], wt += sh.red[i];
        }
        if (threadIdx.x < S) {
            st_dsmem_u32(dsmem_addr(&sh.tot_cnt[cr], threadIdx.x), ct);
            st_dsmem_u64(dsmem_addr(&sh.tot_mass[cr], threadIdx.x), wt);
        }
        cluster_sync();
        uint64_t all = 0;
        for (uint32_t q = 0; q < S; ++q) {
            const uint64_t tw = MASS ? sh.tot_mass[q] : sh.tot_cnt[q];
            all += tw;
            if (q < cr) cb += sh.tot_cnt[q], wb += sh.tot_mass[q];
        }
        if (share) {                                   // before_i < p Z  <=>  before_i < ceil(p Z)
            goal = uint64_t(ceil(double(f.p) * double(all)));
            goal = goal < 1 ? 1 : goal;
        }
        goal = goal > all ? all : goal;                // (k of fewer elements: all of them)
        if (mine) {
            uint32_t cc = cb;
            uint64_t ww = wb;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < per) {
                    const uint64_t a = MASS ? ww : cc, d = MASS ? w[i] : c[i];
                    if (a < goal && goal <= a + d)
                        for (uint32_t q = 0; q < S; ++q) {
                            st_dsmem_u64(dsmem_addr(&sh.x.above, q), a);
                            st_dsmem_u64(dsmem_addr(&sh.x.mass, q), goal);
                            st_dsmem_u32(dsmem_addr(&sh.x.bin, q), uint32_t(b0 + i));
                            st_dsmem_u32(dsmem_addr(&sh.x.cnt_above, q), cc);
                            st_dsmem_u32(dsmem_addr(&sh.x.cnt, q), c[i]);
                        }
                    cc += c[i], ww += w[i];
                }
        }
        cluster_sync();
        return sh.x;
    }

    // Adds the elements that pred takes to CTA 0's list (list_n is zero before).
    template <typename F>
    __device__ void gather(F pred) {
        const uint32_t n = dsmem_addr(&sh.list_n, 0);
        each([&](float x, int tok) {
            if (real(tok) && pred(x, tok)) {
                const uint32_t at = atom_add_dsmem_u32(n, 1u);
                if (at < SP_LIST)
                    st_dsmem_u64(dsmem_addr(&sh.list[at], 0), (uint64_t(ord_f32(x)) << 32) | (0xffffffffu - uint32_t(tok)));
            }
        });
        cluster_sync();
    }

    // Sums of measure(x, token) in token order: the token at which the running sum passes `goal` (or u times
    // the whole, SHARE), -1 if none.
    template <bool SHARE, typename F>
    __device__ int draw(F measure, uint64_t goal, float u) {
        const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
        const int per = ((sl.nv + SP_WARPS - 1) / SP_WARPS + 31) / 32 * 32;    // vectors of a warp's stretch
        const int v0 = min(wid * per, sl.nv), v1 = min(v0 + per, sl.nv);
        auto of = [&](int i, uint64_t (&w)[VEC]) -> uint64_t {
            uint64_t s = 0;
            float x[VEC];
            if (i < v1) E::widen(sl.v[i], x);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int tok = sl.first + i * VEC + e;
                w[e] = i < v1 && real(tok) ? measure(x[e], tok) : 0;
                s += w[e];
            }
            return s;
        };
        uint64_t w[VEC], sum = 0;
        for (int i = v0 + lane; i < v1; i += 32) sum += of(i, w);
        sum = sp_warp_sum(sum);
        if (lane < int(S)) st_dsmem_u64(dsmem_addr(&sh.sums[cr][wid], lane), sum);
        cluster_sync();
        uint64_t before = 0, all = 0;
        for (uint32_t q = 0; q < S; ++q)
            for (int i = 0; i < SP_WARPS; ++i) {
                const uint64_t s = sh.sums[q][i];
                if (q < cr || (q == cr && i < wid)) before += s;
                all += s;
            }
        if (SHARE) {
            goal = uint64_t(double(u) * double(all));
            if (goal >= all) goal = all ? all - 1 : 0;   // (u below 1: only by rounding)
        }
        // (none: fewer than the goal; the token then stays -1)
        if (goal >= all && cr == 0 && threadIdx.x < S) st_dsmem_u32(dsmem_addr(&sh.token, threadIdx.x), 0xffffffffu);
        if (before <= goal && goal < before + sum) {     // this warp's stretch
            uint64_t run = before;
            for (int i0 = v0; i0 < v1; i0 += 32) {
                const uint64_t s = of(i0 + lane, w), inc = sp_warp_scan(s), end = shfl_idx_u64(inc, 31);
                if (goal < run + end) {
                    uint64_t a = run + inc - s;
                    if (a <= goal && goal < a + s) {
                        int tok = -1;
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            if (tok < 0 && goal < a + w[e]) tok = sl.first + (i0 + lane) * VEC + e;
                            a += w[e];
                        }
                        for (uint32_t q = 0; q < S; ++q) st_dsmem_u32(dsmem_addr(&sh.token, q), uint32_t(tok));
                    }
                    break;
                }
                run += end;
            }
        }
        cluster_sync();
        return int(sh.token);
    }

    // CTA 0: of the list's elements, the last one kept when `above` lies before them and the goal is
    // reached among them, to all CTAs' (kthr, ithr).
    template <bool MASS>
    __device__ void last_of_list(uint64_t above, uint64_t goal, const Filter& f, float m) {
        if (cr == 0) {
            const int n = min(int(sh.list_n), SP_LIST);
            if (MASS) {
                for (int i = threadIdx.x; i < n; i += SP_NT)
                    sh.lw[i] = sp_weight(f32_from_ord(uint32_t(sh.list[i] >> 32)), m, f, sh.table);
                __syncthreads();
            }
            const int i = threadIdx.x;
            if (i < n) {
                const uint64_t e = sh.list[i];
                uint64_t a = above;
                for (int j = 0; j < n; ++j)
                    if (sh.list[j] > e) a += MASS ? sh.lw[j] : 1;
                if (a < goal && goal <= a + (MASS ? sh.lw[i] : 1))
                    for (uint32_t q = 0; q < S; ++q) {
                        st_dsmem_u32(dsmem_addr(&sh.kthr, q), uint32_t(e >> 32));
                        st_dsmem_u32(dsmem_addr(&sh.ithr, q), 0xffffffffu - uint32_t(e));
                    }
            }
        }
        cluster_sync();
    }

    // The last element of `kept` before the goal: count k, or the share p of the weight. With `small`, stops
    // when all that is above and in the bin fits the list, gathers it and returns true.
    template <bool MASS>
    __device__ bool select(Kept& kept, const Filter& f, float m, float low, bool small) {
        const float range = MASS ? fminf(m - low, 31.0f * f.T) : m - low;
        Range g{m, range > 0.f ? float(SP_BINS) / range : 0.f, -1, 0u, 0u, 0};
        if (!(g.s < 3.0e38f)) g.s = 3.0e38f;
        Crossing c = crossing<MASS>(g, kept, f, m, MASS, uint64_t(f.k));
        uint64_t above = c.above;
        const uint64_t goal = c.mass;
        uint32_t cnt_above = c.cnt_above, cnt = c.cnt;
        // keys of the bin: its ends in x, with room for the roundings of (m - x) * s
        g.bin = int(c.bin);
        {
            const float a = g.s > 0.f ? float(c.bin) / g.s : 0.f, b = g.s > 0.f ? float(c.bin + 1) / g.s : 0.f;
            const float slack = (fabsf(m) + b) * 1.9073486e-6f;    // 2^-19
            const bool open = int(c.bin) == SP_BINS - 1;
            g.khi = c.bin == 0 ? ord_f32(m) : ord_f32(fminf(m, (m - a) + slack));
            g.klo = open || g.s == 0.f ? ord_f32(-INFINITY) : ord_f32((m - b) - slack);
            if (low > -INFINITY && m == low) g.khi = ord_f32(m), g.klo = g.khi;
        }
        const Kept old = kept;
        while (true) {
            // (what is above fits the list together with the bin: the last step can be taken there)
            const bool whole = small && cnt_above + cnt <= uint32_t(SP_LIST);
            if (whole || cnt <= uint32_t(SP_LIST)) {
                const Range h = g;
                gather([&](float x, int tok) -> bool {
                    const uint32_t key = ord_f32(x);
                    if (!old.has(key, uint32_t(tok))) return false;
                    const int b = sp_bin(x, h);
                    if (b == h.bin && key >= h.klo) return whole || key <= h.khi;
                    return whole && b < h.bin;
                });
                if (whole) return true;
                last_of_list<MASS>(above, goal, f, m);
                kept = Kept{sh.kthr, sh.ithr};
                if (threadIdx.x == 0) sh.list_n = 0;       // (the next list is behind cluster barriers)
                return false;
            }
            if (g.khi == g.klo) {                          // one value: the r-th of its tokens
                const uint32_t key = g.khi;
                uint64_t r = goal - above;                 // >= 1
                if (MASS) {
                    const uint64_t w = sp_weight(f32_from_ord(key), m, f, sh.table);
                    r = (r + w - 1) / w;
                }
                const int t = draw<false>(
                    [&](float x, int tok) -> uint64_t { return ord_f32(x) == key && old.has(key, uint32_t(tok)); }, r - 1,
                    0.f);
                kept = Kept{key, uint32_t(t)};
                return false;
            }
            g.shift = 0;
            while (((g.khi - g.klo) >> g.shift) >= uint32_t(SP_BINS)) ++g.shift;
            c = crossing<MASS>(g, kept, f, m, false, goal - above);
            above += c.above, cnt_above += c.cnt_above, cnt = c.cnt;
            const uint32_t hi = g.khi - (c.bin << g.shift), span = (1u << g.shift) - 1u;
            g.klo = hi - g.klo > span ? hi - span : g.klo;
            g.khi = hi;
        }
    }

    // CTA 0: top-k, top-p, min-p and the draw among the list's elements.
    __device__ int finish_in_list(const Filter& f, float m) {
        if (cr == 0) {
            const int n = min(int(sh.list_n), SP_LIST), i = threadIdx.x;
            const uint64_t e = i < n ? sh.list[i] : 0;
            if (i < n) sh.lw[i] = sp_weight(f32_from_ord(uint32_t(e >> 32)), m, f, sh.table);
            __syncthreads();
            const int k = f.k > 0 ? min(f.k, n) : n;
            int rank = 0;
            uint64_t before = 0;
            if (i < n)
                for (int j = 0; j < n; ++j)
                    if (sh.list[j] > e) ++rank, before += sh.lw[j];
            uint32_t c = 0;
            uint64_t z = i < n && rank < k ? sh.lw[i] : 0;
            const uint64_t mine = z;
            block_sum(c, z);
            uint64_t goal = z;
            if (f.p < 1.f) {
                goal = uint64_t(ceil(double(f.p) * double(z)));
                goal = goal < 1 ? 1 : goal > z ? z : goal;
            }
            const bool keep = i < n && rank < k && (rank == 0 || (before < goal && mine >= f.wmin));
            uint64_t w = keep ? mine : 0;
            const uint64_t kw = w;
            if (i < n) sh.kw[i] = kw;
            block_sum(c, w);                               // (its barriers also order kw)
            uint64_t at = uint64_t(double(f.u) * double(w));
            if (at >= w) at = w - 1;
            if (kw) {
                uint64_t a = 0;
                for (int j = 0; j < n; ++j)
                    if (uint32_t(sh.list[j]) > uint32_t(e)) a += sh.kw[j];   // lower tokens
                if (a <= at && at < a + kw)
                    for (uint32_t q = 0; q < S; ++q)
                        st_dsmem_u32(dsmem_addr(&sh.token, q), 0xffffffffu - uint32_t(e));
            }
        }
        cluster_sync();
        return int(sh.token);
    }
};

// The token of one row, to every thread of the cluster; -1 for a row that holds nothing but -inf and NaN.
// `data`: the CTA's shared memory for its slice. sh.f is set and seen by all threads.
template <typename T>
__device__ int sp_row(const T* row, int V, int seg, SpShared& sh, uint4* data, int* status) {
    using E = SpElem<T>;
    constexpr int VEC = E::VEC;
    const uint32_t S = cluster_nctarank(), cr = cluster_ctarank();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int lo = min(int(cr) * seg, V), hi = min(lo + seg, V);
    // ---------------------------------------------------------------- load
    const T* p = row + lo;
    const int shift = int((reinterpret_cast<uintptr_t>(p) % 16) / sizeof(T));
    const int nv = hi > lo ? (shift + (hi - lo) + VEC - 1) / VEC : 0;
    const T* base = p - shift;
    float top = -INFINITY, low = INFINITY;
    auto see = [&](const uint4& v) {
        float x[VEC];
        E::widen(v, x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            top = fmaxf(top, x[e]);
            low = x[e] > -INFINITY ? fminf(low, x[e]) : low;
        }
    };
    const int i0 = shift ? 1 : 0, i1 = (shift + (hi - lo)) / VEC;       // whole vectors
    constexpr int U = 4;
    for (int i = i0 + int(threadIdx.x); i < i1; i += U * SP_NT) {
        uint4 v[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i + k * SP_NT < i1) v[k] = __ldg(reinterpret_cast<const uint4*>(base) + i + k * SP_NT);
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i + k * SP_NT < i1) {
                v[k] = E::clean4(v[k]);
                data[i + k * SP_NT] = v[k];
                see(v[k]);
            }
    }
    if (threadIdx.x < 2 && nv > 0) {                                    // the ends, element by element
        const int i = threadIdx.x == 0 ? 0 : nv - 1;
        if ((i < i0 || i >= i1) && (threadIdx.x == 0 || nv > 1 || i0 == 0))
            for (int e = 0; e < VEC; ++e) {
                const int at = i * VEC + e;
                const float x = at >= shift && at < shift + (hi - lo) ? E::get(base + at) : -INFINITY;
                E::put(reinterpret_cast<T*>(data) + at, x);
                top = fmaxf(top, x);
                low = x > -INFINITY ? fminf(low, x) : low;
            }
    }
    top = warp_max(top);
    low = -warp_max(-low);
    if (lane == 0) sh.red[wid] = (uint64_t(__float_as_uint(top)) << 32) | __float_as_uint(low);
    if (threadIdx.x == 0) sh.list_n = 0;
    __syncthreads();
    for (int i = 0; i < SP_WARPS; ++i) {
        top = fmaxf(top, __uint_as_float(uint32_t(sh.red[i] >> 32)));
        low = fminf(low, __uint_as_float(uint32_t(sh.red[i])));
    }
    if (threadIdx.x < S) {
        st_dsmem_u32(dsmem_addr(&sh.top[cr], threadIdx.x), __float_as_uint(top));
        st_dsmem_u32(dsmem_addr(&sh.low[cr], threadIdx.x), __float_as_uint(low));
    }
    cluster_sync();
    for (uint32_t q = 0; q < S; ++q) top = fmaxf(top, sh.top[q]), low = fminf(low, sh.low[q]);
    const Filter f = sh.f;
    Sampler<T> s{sh, Slice<T>{data, nv, lo - shift, lo, hi}, S, cr, status};
    int tok = -1;
    if (top > -INFINITY) {
        // ------------------------------------------------------------ the maximum's lowest token
        if (f.greedy) {
            uint32_t best = 0xffffffffu;
            s.each([&](float x, int t) { if (x == top) best = min(best, uint32_t(t)); });
            best = __reduce_min_sync(0xffffffffu, best);
            __syncthreads();
            if (lane == 0) sh.redc[wid] = best;
            __syncthreads();
            for (int i = 0; i < SP_WARPS; ++i) best = min(best, sh.redc[i]);
            if (threadIdx.x < S) st_dsmem_u32(dsmem_addr(&sh.first[cr], threadIdx.x), best);
            cluster_sync();
            for (uint32_t q = 0; q < S; ++q) best = min(best, sh.first[q]);
            tok = int(best);
        } else {
            // (a maximum of +inf holds all the weight: nothing else is kept)
            Kept kept{0u, 0xffffffffu};
            if (top == INFINITY) kept.key = ord_f32(top), low = top;
            bool listed = false;
            if (f.k > 0 && f.k < V) listed = s.template select<false>(kept, f, top, low, f.k <= SP_LIST);
            if (!listed && f.p < 1.f) listed = s.template select<true>(kept, f, top, low, false);
            if (listed) {
                tok = s.finish_in_list(f, top);
            } else {
                const float2* table = sh.table;
                tok = s.template draw<true>(
                    [&](float x, int t) -> uint64_t {
                        if (!kept.has(ord_f32(x), uint32_t(t))) return 0;
                        const uint64_t w = sp_weight(x, top, f, table);
                        return w >= f.wmin ? w : 0;
                    },
                    0, f.u);
            }
        }
    }
    cluster_sync();                                        // (what the next row writes has been read)
    return tok;
}

// Settings of request r for the row with uniform number ui; what is no setting is an error and taken for none.
__device__ __forceinline__ void sp_filter(const SampleArgs& a, int r, float u, SpShared& sh) {
    Filter f;
    bool bad = false;
    f.T = a.temperatures ? a.temperatures[r] : a.temperature;
    f.k = a.top_ks ? a.top_ks[r] : a.top_k;
    f.p = a.top_ps ? a.top_ps[r] : a.top_p;
    f.least = a.min_ps ? a.min_ps[r] : a.min_p;
    f.u = u;
    if (!(f.T >= 0.f && f.T < INFINITY)) bad = true, f.T = 0.f;
    if (f.k < 0) bad = true, f.k = 0;
    if (!(f.p >= 0.f && f.p <= 1.f)) bad = true, f.p = 1.f;
    if (!(f.least >= 0.f && f.least <= 1.f)) bad = true, f.least = 0.f;
    if (!(f.u >= 0.f && f.u < 1.f)) bad = true, f.u = 0.f;
    if (bad) set_status(a.status, DARTREE_EINTERNAL);
    f.greedy = f.T == 0.f || f.k == 1 || f.p == 0.f;
    const double c = fmin(1.4426950408889634 / double(f.T > 0.f ? f.T : 1.f), 1e37);
    f.ch = float(c), f.cl = float(c - double(f.ch));
    f.wmin = uint64_t(ceil(double(f.least) * double(uint64_t(1) << SP_Q)));
    sh.f = f;
}

template <typename T, bool TREE>
__global__ void __launch_bounds__(SP_NT, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
    extern __shared__ __align__(16) uint4 sp_data[];
    __shared__ SpShared sh;
    __shared__ int found_s;
    const uint32_t S = cluster_nctarank(), cr = cluster_ctarank();
    const int r = int(blockIdx.x / S);
    for (int i = threadIdx.x; i < 129; i += SP_NT) sh.table[i] = a.table[i];
    griddep_launch_dependents();
    griddep_wait();
    const T* x = static_cast<const T*>(a.x);
    if constexpr (!TREE) {
        if (threadIdx.x == 0) sp_filter(a, r, a.u[r], sh);
        const int tok = sp_row<T>(x + size_t(r) * a.ld, a.V, a.seg, sh, sp_data, a.status);
        if (cr == 0 && threadIdx.x == 0) a.tok[r] = tok;
    } else {
        const int SL = a.B + 1, n = min(SL, a.n_nodes[r]);
        const int32_t* tk = a.t_tok + size_t(r) * SL;
        const int32_t* pr = a.t_par + size_t(r) * SL;
        int cur = 0, acc = 0, bon = -1;
        while (true) {
            const int row = a.t_depth ? a.t_depth[size_t(r) * SL + cur] : cur;
            if (row < 0 || row >= a.per) break;            // no row for this depth
            const size_t at = size_t(r) * a.per + row;
            if (threadIdx.x == 0) sp_filter(a, r, a.u[at], sh), found_s = 0x7fffffff;
            const int t = sp_row<T>(x + at * a.V, a.V, a.seg, sh, sp_data, a.status);
            for (int j = 1 + int(threadIdx.x); j < n; j += SP_NT)
                if (pr[j] == cur && tk[j] == t) atomicMin(&found_s, j);
            __syncthreads();
            const int next = found_s;
            __syncthreads();
            if (next == 0x7fffffff) {
                bon = t;
                break;
            }
            if (acc >= a.L) {                              // more steps than depths: malformed tree
                if (cr == 0 && threadIdx.x == 0) set_status(a.status, DARTREE_EINTERNAL);
                break;
            }
            if (cr == 0 && threadIdx.x == 0) a.path[size_t(r) * a.L + acc] = next;
            ++acc;
            cur = next;
        }
        if (cr == 0) {
            for (int q = acc + int(threadIdx.x); q < a.L; q += SP_NT) a.path[size_t(r) * a.L + q] = -1;
            if (threadIdx.x == 0) a.accepted[r] = acc, a.bonus[r] = bon;
        }
    }
}

// ----------------------------------------------------------------------------- host

constexpr int SP_SLICE = 80 * 1024;        // bytes of a slice beside which a second CTA fits
constexpr int SP_MOST = 190 * 1024;

// Elements of a CTA's slice with S CTAs to a row, and its bytes with the ends of an unaligned row.
static int sp_seg(int V, int S) { return ((V + S - 1) / S + 7) / 8 * 8; }
static int sp_bytes(int V, int S, int es) { return sp_seg(V, S) * es + 32; }

bool sample_supported(int V, int dtype) {
    return V <= (1 << 20) && sp_bytes(V, SP_MAXC, dtype == DARTREE_BF16 ? 2 : 4) <= SP_MOST;
}

template <typename T, bool TREE>
static int launch_sample_t(SampleArgs a, int rows, cudaStream_t stream) {
    const int es = int(sizeof(T));
    // as few CTAs as leave room for two on an SM, more while that does not fill the SMs
    int S = 1;
    while (S < SP_MAXC && (sp_bytes(a.V, S, es) > SP_SLICE ||
                           (int64_t(rows) * S * 2 <= 2 * num_sms() && a.V / (2 * S) >= 1024)))
        S *= 2;
    a.seg = sp_seg(a.V, S);
    const int bytes = sp_bytes(a.V, S, es);
    auto kern = sample_kernel<T, TREE>;
    static std::atomic<uint64_t> raised{0};
    if (!raise_smem(kern, SP_MOST, raised)) return DARTREE_ECUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(rows) * unsigned(S));
    cfg.blockDim = dim3(SP_NT);
    cfg.dynamicSmemBytes = size_t(bytes);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2] = {pdl_attribute()};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(S);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    KTimer kt_(TREE ? KID_SAMPLE_WALK : KID_SAMPLE, stream);
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? DARTREE_OK : DARTREE_ECUDA;
}

static SampleArgs sample_args(const void* x, int V, const dartree_filter& f, const float* u, int* status) {
    SampleArgs a{};
    a.x = x, a.V = V, a.ld = V, a.u = u, a.status = status;
    a.temperature = f.temperature, a.top_k = f.top_k, a.top_p = f.top_p, a.min_p = f.min_p;
    a.temperatures = f.temperatures, a.top_ks = f.top_ks, a.top_ps = f.top_ps, a.min_ps = f.min_ps;
    for (int j = 0; j <= 128; ++j) {
        const double t = exp2(double(j) / -128.0);
        a.table[j].x = float(t);
        a.table[j].y = float(t - double(a.table[j].x));
    }
    return a;
}

int launch_sample(const void* logits, int rows, int V, int64_t ld, int dtype, const dartree_filter& f, const float* u,
                  int32_t* tok, int* status, cudaStream_t stream) {
    SampleArgs a = sample_args(logits, V, f, u, status);
    a.ld = ld, a.tok = tok;
    return dtype == DARTREE_BF16 ? launch_sample_t<bf16_t, false>(a, rows, stream)
                                 : launch_sample_t<float, false>(a, rows, stream);
}

int launch_sample_walk(int C, int L, int B, const int32_t* tok, const int32_t* par, const int32_t* depth,
                       const int32_t* n_nodes, const void* target, int rows_mode, int V, int dtype,
                       const dartree_filter& f, const float* u, int32_t* accepted, int32_t* path, int32_t* bonus,
                       int* status, cudaStream_t stream) {
    SampleArgs a = sample_args(target, V, f, u, status);
    const bool node = rows_mode == DARTREE_ROWS_PER_NODE;
    a.L = L, a.B = B, a.per = node ? B + 1 : L;
    a.t_tok = tok, a.t_par = par, a.t_depth = node ? nullptr : depth, a.n_nodes = n_nodes;
    a.accepted = accepted, a.path = path, a.bonus = bonus;
    return dtype == DARTREE_BF16 ? launch_sample_t<bf16_t, true>(a, C, stream)
                                 : launch_sample_t<float, true>(a, C, stream);
}

}  // namespace dartree
