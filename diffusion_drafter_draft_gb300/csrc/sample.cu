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
// integers, 2^43 for the largest, off by about half a unit and 2^-34 of themselves at random (Weigher
// below), and sums are exact 64-bit integers, the same in any order and for any split of the row.
//
// One cluster per row; each CTA keeps its slice in shared memory, so the logits are read once.
//   load    slice to shared memory, maximum and minimum, each thread's largest
//   top-k   up to 1024: what reaches the j-th largest of the threads' largest, j = ceil(k / CTAs), in
//           every CTA holds the k first (and few others): a list in CTA 0, sorted, which finishes
//           there
//   top-p   a histogram of 2048 bins of x between maximum and minimum, of counts and places in the bin, tells
//           within 1e-3 of the weight which x hold the border; one pass takes the weights of all, of what
//           lies above and of each warp's stretch, and lists what lies between; CTA 0 finds the border and the
//           warp that holds the goal
//   select  (where that is not enough: larger k, top-p of what it left, runs of equal values) the same histogram of
//           weights or counts; the bin in which the goal is reached, as a list in CTA 0, sorted and summed; while a
//           bin holds more than the list, finer bins of its keys (one value: the r-th by token)
//   draw    sums of each warp's stretch of the row; the warp that holds the goal walks its own
#include <math.h>

#include "paged.cuh"

namespace dartree {

constexpr int SP_NT = 512;
constexpr int SP_WARPS = SP_NT / 32;
constexpr int SP_BINS = 2048;
constexpr int SP_LIST = 1024;     // elements of CTA 0's list
constexpr int SP_FEW = 256;       // twice the elements that are compared with one another
constexpr int SP_MAXC = 8;        // CTAs of a cluster
constexpr int SP_FLUSH = 512;     // elements whose weights' sums fit 32 bits each (Weigher::add)
constexpr int SP_Q = 43;          // a weight of 1 is 2^43; 2^20 of them stay below 2^64

// 2^(i/256) as a pair of floats, i < 256 (evaluated by the compiler in double).
struct SpTable {
    float2 t[256];
};
constexpr SpTable sp_make_table() {
    SpTable r{};
    for (int i = 0; i < 256; ++i) {
        const double y = double(i) / 256.0 * 0.6931471805599453;
        double sum = 1.0, term = 1.0;
        for (int k = 1; k < 20; ++k) {
            term *= y / k;
            sum += term;
        }
        r.t[i].x = float(sum);
        r.t[i].y = float(sum - double(r.t[i].x));
    }
    return r;
}
__device__ const SpTable sp_table = sp_make_table();

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
};

// The settings of a request.
struct Filter {
    float T, p, least;
    int k;
    float up;                     // 2^64 for a T below 2^-64, 2^-64 for one above 2^64 (the next would lose bits), else 1
    float ch, cl;                 // 256 log2(e) / (T up) as a pair
    uint64_t u, share;            // u and (below 1) p times 2^64
    uint64_t wmin;                // least weight that min-p keeps
    uint64_t cut;                 // weights below it cannot be reached by p of the whole
    bool greedy;
};
// x in [0, 1) times 2^bits, rounded down (or up): doubles are slow here. (-0 is 0.)
__device__ __forceinline__ uint64_t sp_fixed(float x, int bits, bool up) {
    const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
    const int e = int(b >> 23);
    uint64_t m = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;      // x = m 2^(e - 150)
    const int s = (e ? e : 1) - 150 + bits;
    if (s >= 0) return m << s;
    if (s <= -24) return up && m ? 1 : 0;
    return (m >> -s) + (up && (m & ((1u << -s) - 1u)) ? 1 : 0);
}

struct Crossing {                 // where a measure summed from the top reaches its goal
    uint64_t above, goal;         // measure of the bins before the bin
    uint32_t bin;
    uint32_t pad;
};

struct SpShared {
    float2 table[256 * 8];        // sp_table, a copy for every eighth lane
    uint32_t lo[SP_BINS];         // histogram: counts, or weights (64 bits in two words)
    union {
        uint32_t hi[SP_BINS];
        uint64_t list[SP_LIST];   // (key, ~token): a CTA's own, then (CTA 0) all; never while hi is in use
    };
    uint64_t lw[SP_FEW];
    uint64_t sums[SP_MAXC][SP_WARPS];    // of every warp of the cluster
    uint64_t tot[SP_MAXC], rest[SP_MAXC];
    uint64_t red[SP_WARPS];
    uint32_t redc[SP_WARPS];
    float top[SP_MAXC], low[SP_MAXC];
    uint32_t first[SP_MAXC], reach[SP_MAXC], count[SP_MAXC];
    uint64_t above[SP_MAXC][SP_WARPS];   // CTA 0
    uint32_t b_lo, b_hi, owner;
    uint64_t left;
    uint64_t strip[2 * SP_WARPS];
    Filter f;
    Crossing x;
    uint32_t list_n, token, done;
    float kx;
    int ki;
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

// The weight of x in units of 2^-43: with t = (m - x) 256 log2(e) / T, K = -round(t), rho = -t - K,
//   w = 2^(K div 256) 2^(K mod 256 / 256) (1 + rho L + (rho L)^2 / 2 + (rho L)^3 / 6),   L = ln 2 / 256, |rho L| < 2^-9.5
// The difference, t and the table are pairs of floats, so what is left is the rounding of rho L and of its product with
// the table, 2^-34 of the weight, different for every x: no bias. (bf16 values, too: the difference of a large maximum
// and a value near zero, or the other way round, is no float.) A weight is then rounded twice to integers of 2^-22 and,
// what remains, of 2^-43, by adding 3 and 1.5 * 2^-20: the sums' low bits are the integers. Two elements at a time
// (fma.rn.f32x2): 22 issue slots an element. The table has a copy for every eighth lane, so that a look-up costs three
// accesses of the shared memory's banks (one copy of 1024 entries: six, and 25 instead of 20 slots' time an element).
// Below xlo, where the weight is none, x counts as xlo (t of at least 62 * 256). Rows in which xlo cannot lie between
// two floats, or differences overflow, and temperatures beyond 2^-64 .. 2^64, with which differences are scaled, take the
// same steps one element at a time (`slow`).
constexpr uint32_t SP_C1 = 0x40400000u;   // 3.0
constexpr uint32_t SP_C2 = 0x35c00000u;   // 1.5 * 2^-20
struct Weigher {
    float m, ch, cl, xlo, up;
    bool slow;
    const float2* table;
    static constexpr float L = 2.7076061740622863e-3f, L2 = 3.6655656e-6f, L3 = 3.3083027e-9f;   // ln 2 / 256, L^2/2, L^3/6

    __device__ __forceinline__ static uint64_t whole(uint32_t i1, uint32_t i2) {
        return (uint64_t(i1) << 21) + uint64_t(int64_t(int32_t(i2)));
    }
    // integers of 2^-22 and of 2^-43 of d = m - x, off by e
    __device__ __forceinline__ void core1(float d, float e, uint32_t& i1, uint32_t& i2) const {
        const float th = __fmul_rn(d, -ch);
        const float tl = __fmaf_rn(e, ch, __fmaf_rn(d, cl, __fmaf_rn(d, ch, th)));
        const float y = __fadd_rn(th, 12582912.0f);
        const float rho = __fadd_rn(__fadd_rn(th, __fsub_rn(12582912.0f, y)), -tl);
        const float em = __fmul_rn(rho, __fmaf_rn(rho, __fmaf_rn(rho, L3, L2), L));
        const uint32_t k = __float_as_uint(y);
        const float2 t = table[(k & 255u) * 8];
        const float s = __uint_as_float(((k & ~255u) << 15) + 0x3f800000u);
        const float c = __fmaf_rn(t.x, em, t.y);
        const float vt = __fmul_rn(t.x, s), vc = __fmul_rn(c, s);
        const float h = __fadd_rn(vt, 3.0f), g = __fadd_rn(vc, 3.0f);
        const float l = __fadd_rn(__fadd_rn(vt, __fsub_rn(3.0f, h)), __fadd_rn(vc, __fsub_rn(3.0f, g)));
        i1 = __float_as_uint(h) + __float_as_uint(g) - 2u * SP_C1;
        i2 = __float_as_uint(__fadd_rn(l, __uint_as_float(SP_C2))) - SP_C2;
    }
    __device__ __forceinline__ uint64_t one(float x) const {
        if (x == m) return uint64_t(1) << SP_Q;
        float d = __fsub_rn(m, x);
        if (slow && !(d * up * ch < 15872.0f)) return 0;
        if (!slow) x = fmaxf(x, xlo), d = __fsub_rn(m, x);
        const float bb = __fsub_rn(d, m);
        const float e = __fsub_rn(__fsub_rn(m, __fsub_rn(d, bb)), __fadd_rn(x, bb));
        uint32_t i1, i2;
        core1(d * up, e * up, i1, i2);
        return whole(i1, i2);
    }
    __device__ __noinline__ uint64_t one_call(float x) const { return one(x); }   // (rare places)
    // two elements, each at least xlo: their integers (from SP_C1 and SP_C2 on)
    __device__ __forceinline__ void two(float x0, float x1, uint32_t (&h)[2], uint32_t (&g)[2], uint32_t (&q)[2]) const {
        const uint64_t M = pair(m, m), N1 = pair(-1.0f, -1.0f), CH = pair(ch, ch), NCH = pair(-ch, -ch), CL = pair(cl, cl);
        const uint64_t X = pair(x0, x1), MG = pair(12582912.0f, 12582912.0f), C1 = pair(SP_C1, SP_C1);
        const uint64_t d = fma2(X, N1, M);
        const uint64_t th = mul2(d, NCH);
        const uint64_t bb = fma2(M, N1, d), e1 = fma2(fma2(bb, N1, d), N1, M);
        const uint64_t tl = fma2(fma2(add2(X, bb), N1, e1), CH, fma2(d, CL, fma2(d, CH, th)));
        const uint64_t y = add2(th, MG);
        const uint64_t rho = fma2(tl, N1, add2(th, fma2(y, N1, MG)));
        const uint64_t em = mul2(rho, fma2(rho, fma2(rho, pair(L3, L3), pair(L2, L2)), pair(L, L)));
        const uint32_t k0 = uint32_t(y), k1 = uint32_t(y >> 32);
        const float2 t0 = table[(k0 & 255u) * 8], t1 = table[(k1 & 255u) * 8];
        const uint64_t th2 = pair(t0.x, t1.x);
        const uint64_t s = pair(((k0 & ~255u) << 15) + 0x3f800000u, ((k1 & ~255u) << 15) + 0x3f800000u);
        const uint64_t c = fma2(th2, em, pair(t0.y, t1.y));
        const uint64_t vt = mul2(th2, s), vc = mul2(c, s);
        const uint64_t hh = add2(vt, C1), gg = add2(vc, C1);
        const uint64_t l = add2(add2(vt, fma2(hh, N1, C1)), add2(vc, fma2(gg, N1, C1)));
        const uint64_t qq = add2(l, pair(SP_C2, SP_C2));
        h[0] = uint32_t(hh), h[1] = uint32_t(hh >> 32);
        g[0] = uint32_t(gg), g[1] = uint32_t(gg >> 32);
        q[0] = uint32_t(qq), q[1] = uint32_t(qq >> 32);
    }
    // Weights of N elements (below xlo: none).
    template <int N>
    __device__ __forceinline__ void each(const float (&x)[N], uint64_t (&w)[N]) const {
        if (slow) {
#pragma unroll
            for (int e = 0; e < N; ++e) w[e] = one_call(x[e]);
            return;
        }
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            uint32_t h[2], g[2], q[2];
            two(fmaxf(x[e], xlo), fmaxf(x[e + 1], xlo), h, g, q);
            w[e] = whole(h[0] + g[0] - 2u * SP_C1, q[0] - SP_C2);
            w[e + 1] = whole(h[1] + g[1] - 2u * SP_C1, q[1] - SP_C2);
        }
    }
    // Sums of weights, 2^-22 and 2^-43 apart; SP_FLUSH elements fit (a thread's share of a held slice is below that).
    // add_above: of all, and of those above `bound`.
    template <int N>
    __device__ __forceinline__ void add_above(const float (&x)[N], float bound, uint32_t& i1, uint32_t& i2, uint32_t& a1,
                                              uint32_t& a2) const {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            uint32_t h[2], g[2], q[2];
            two(fmaxf(x[e], xlo), fmaxf(x[e + 1], xlo), h, g, q);
            h[0] += g[0] - 2u * SP_C1, h[1] += g[1] - 2u * SP_C1, q[0] -= SP_C2, q[1] -= SP_C2;
            i1 += h[0] + h[1], i2 += q[0] + q[1];
            if (x[e] > bound) a1 += h[0], a2 += q[0];
            if (x[e + 1] > bound) a1 += h[1], a2 += q[1];
        }
    }
    template <int N>
    __device__ __forceinline__ void add(const float (&x)[N], uint32_t& i1, uint32_t& i2) const {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            uint32_t h[2], g[2], q[2];
            two(fmaxf(x[e], xlo), fmaxf(x[e + 1], xlo), h, g, q);
            i1 += h[0] + g[0] + h[1] + g[1] - 4u * SP_C1;
            i2 += q[0] + q[1] - 2u * SP_C2;
        }
    }
};
// Of row maximum m under f.
__device__ __forceinline__ Weigher sp_weigher(float m, const Filter& f, const float2* table) {
    const float below = __uint_as_float(m > 0.f ? __float_as_uint(m) - 1u : m < 0.f ? __float_as_uint(m) + 1u : 0x80000001u);
    const float reach = 15872.0f / f.ch;                   // 62 * 256
    Weigher w{m, f.ch, f.cl, fminf(m - reach, below), f.up, false, table + (threadIdx.x & 7)};
    w.slow = !(f.up == 1.f && fabsf(m) < 1e30f && reach < 1e30f && (m - below) * f.ch < 15872.0f);
    return w;
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
    static __device__ __forceinline__ float get(const float* p) { return clean(*p); }
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
};

// A CTA's slice [lo, hi) of a row as `nv` vectors of 16 bytes, element e of vector v being token first + v * VEC + e
// (first may lie before the slice; what is no element of it reads as -inf, which is never kept, like NaN).
// HELD: in shared memory; else read again from memory (the L2, mostly) by every pass, for batches of more rows
// than fit.
template <typename T, bool HELD>
struct Slice {
    using E = SpElem<T>;
    static constexpr int VEC = E::VEC;
    const uint4* v;               // HELD: the CTA's shared memory; else the row from `first` on, aligned
    const T* row;
    int nv, first, lo, hi;
    bool only_inf;                // the maximum is +inf: it counts as 0 and all else as -inf

    // Vector i as it lies, its ends cleared.
    __device__ __forceinline__ uint4 raw(int i) const {
        if (HELD) return v[i];
        const int t = first + i * VEC;
        if (t >= lo && t + VEC <= hi) return __ldg(v + i);
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (sizeof(T) == 4) {
                w[k] = t + k >= lo && t + k < hi ? __float_as_uint(row[t + k]) : 0xff800000u;
            } else {
                const int a = t + 2 * k;
                w[k] = (a >= lo && a < hi ? uint32_t(row[a].bits) : 0xff80u) |
                       (a + 1 >= lo && a + 1 < hi ? uint32_t(row[a + 1].bits) : 0xff80u) << 16;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void values(uint4 r, float (&x)[VEC]) const {
        if (!HELD) r = E::clean4(r);
        E::widen(r, x);
        if (only_inf)
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] = x[e] == INFINITY ? 0.f : -INFINITY;
    }
    __device__ __forceinline__ void values(int i, float (&x)[VEC]) const { values(raw(i), x); }
    // One element of the slice.
    __device__ __forceinline__ float value(int tok) const {
        float x;
        if (HELD) x = E::get(reinterpret_cast<const T*>(v) + (tok - first));
        else x = tok >= lo && tok < hi ? E::get(row + tok) : -INFINITY;
        return only_inf ? (x == INFINITY ? 0.f : -INFINITY) : x;
    }
    // f(i, x) for vectors i0, i0 + step, ... below i1; read ahead where that takes long.
    template <typename F>
    __device__ __forceinline__ void over(int i0, int i1, int step, F f) const {
        float x[VEC];
        if (HELD) {
            for (int i = i0; i < i1; i += step) {
                values(i, x);
                f(i, x);
            }
        } else {
            constexpr int A = 3;                           // vectors ahead
            uint4 r[A];
#pragma unroll
            for (int k = 0; k < A; ++k)
                if (i0 + k * step < i1) r[k] = raw(i0 + k * step);
            for (int i = i0; i < i1; i += step) {
                const uint4 now = r[0];
#pragma unroll
                for (int k = 0; k + 1 < A; ++k) r[k] = r[k + 1];
                if (i + A * step < i1) r[A - 1] = raw(i + A * step);
                values(now, x);
                f(i, x);
            }
        }
    }
};

// Elements that are still in question: bin of the first histogram and a range of keys.
struct Range {
    float m, s;                   // bin of x: (m - x) * s
    int bin;                      // -1: no bin chosen yet
    uint32_t khi, klo;
    int shift;
};
__device__ __forceinline__ int sp_bin(float x, const Range& g) {
    return int(fminf(__fmul_rn(__fsub_rn(g.m, x), g.s), float(SP_BINS - 1)));
}

struct Kept {                     // the last element kept
    float x;
    int tok;
    __device__ __forceinline__ bool has(float v, int t) const { return v > x || (v == x && t <= tok); }
};
// Everything but -inf: what lies around the row reads as that, with tokens below 0 ahead of a row that does not start on
// 16 bytes.
constexpr Kept SP_ALL{-INFINITY, -0x7fffffff - 1};

// What a row needs of the cluster. All functions are called by all threads of the cluster.
template <typename T, bool HELD>
struct Sampler {
    using E = SpElem<T>;
    static constexpr int VEC = E::VEC;
    SpShared& sh;
    Slice<T, HELD> sl;
    uint32_t S, cr;               // CTAs, this one
    Weigher wg;

    template <typename F>
    __device__ __forceinline__ void each(F f) const {          // f(x, token), this thread's elements
        sl.over(threadIdx.x, sl.nv, SP_NT, [&](int i, const float (&x)[VEC]) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) f(x[e], sl.first + i * VEC + e);
        });
    }

    // Sum over the block, and the sum before this thread (exclusive, in thread order).
    __device__ uint64_t block_scan(uint64_t v, uint64_t& before) {
        const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
        const uint64_t inc = sp_warp_scan(v);
        __syncthreads();
        if (lane == 31) sh.red[wid] = inc;
        __syncthreads();
        before = inc - v;
        uint64_t all = 0;
#pragma unroll
        for (int i = 0; i < SP_WARPS; ++i) {
            const uint64_t r = sh.red[i];
            if (i < wid) before += r;
            all += r;
        }
        return all;
    }

    // Histogram of the kept elements in g and the bin where the goal is reached: count `goal` (MASS false), the
    // share p of the whole weight (share) or the weight `goal`. Weights below `cut`, which cannot be
    // reached, only count for the whole.
    template <bool MASS>
    __device__ Crossing crossing(const Range& g, const Kept& kept, const Filter& f, uint64_t cut, bool share, uint64_t goal) {
        for (int i = threadIdx.x; i < SP_BINS; i += SP_NT) {
            sh.lo[i] = 0;
            if (MASS) sh.hi[i] = 0;
        }
        __syncthreads();
        uint64_t rest = 0;
        auto bin_of = [&](float x) -> int {                // -1: not in question
            int b = sp_bin(x, g);
            if (g.bin >= 0) {
                const uint32_t key = ord_f32(x);
                b = b != g.bin || key > g.khi || key < g.klo ? -1 : int((g.khi - key) >> g.shift);
            }
            return b;
        };
        sl.over(threadIdx.x, sl.nv, SP_NT, [&](int i, const float (&x)[VEC]) {
            bool in[VEC], any = false;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                in[e] = kept.has(x[e], sl.first + i * VEC + e) && (g.bin < 0 || bin_of(x[e]) >= 0);
                any |= in[e];
            }
            if (!any) return;
            if constexpr (!MASS) {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (in[e]) atomicAdd(&sh.lo[bin_of(x[e])], 1u);
            } else {
                uint64_t w[VEC];
                wg.template each<VEC>(x, w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    if (!in[e]) continue;
                    if (w[e] < cut) {
                        rest += w[e];
                        continue;
                    }
                    const int b = bin_of(x[e]);
                    const uint32_t wl = uint32_t(w[e]);
                    const uint32_t before = atomicAdd(&sh.lo[b], wl);
                    const uint32_t up = uint32_t(w[e] >> 32) + (before + wl < wl ? 1u : 0u);
                    if (up) atomicAdd(&sh.hi[b], up);
                }
            }
        });
        if (MASS && share) {
            uint64_t before;
            rest = block_scan(rest, before);
            if (threadIdx.x < S) st_dsmem_u64(dsmem_addr(&sh.rest[cr], threadIdx.x), rest);
        }
        cluster_sync();
        // CTA r sums bins [r * nb, (r + 1) * nb) over the cluster, consecutive bins to a thread
        const int nb = SP_BINS / int(S), per = (nb + SP_NT - 1) / SP_NT;   // 1, 2 or 4
        uint64_t w[4] = {0, 0, 0, 0}, ws = 0, wb;
        const int b0 = int(cr) * nb + int(threadIdx.x) * per;
        const bool mine = int(threadIdx.x) * per < nb;
        if (mine)
            for (uint32_t q = 0; q < S; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < per) {
                        uint64_t v = ld_dsmem_u32(dsmem_addr(&sh.lo[b0 + i], q));
                        if (MASS) v += uint64_t(ld_dsmem_u32(dsmem_addr(&sh.hi[b0 + i], q))) << 32;
                        w[i] += v, ws += v;
                    }
        const uint64_t wt = block_scan(ws, wb);
        if (threadIdx.x < S) st_dsmem_u64(dsmem_addr(&sh.tot[cr], threadIdx.x), wt);
        cluster_sync();
        uint64_t all = 0, more = 0;
        for (uint32_t q = 0; q < S; ++q) {
            all += sh.tot[q];
            if (q < cr) wb += sh.tot[q];
            if (MASS && share) more += sh.rest[q];
        }
        if (share) {                                   // before_i < p Z  <=>  before_i < ceil(p Z)
            goal = share_of(all + more, f);
        }
        goal = goal > all ? all : goal;                // (k of fewer elements: all of them)
        if (mine) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < per) {
                    if (wb < goal && goal <= wb + w[i])
                        for (uint32_t q = 0; q < S; ++q) {
                            st_dsmem_u64(dsmem_addr(&sh.x.above, q), wb);
                            st_dsmem_u64(dsmem_addr(&sh.x.goal, q), goal);
                            st_dsmem_u32(dsmem_addr(&sh.x.bin, q), uint32_t(b0 + i));
                        }
                    wb += w[i];
                }
        }
        cluster_sync();
        return sh.x;
    }

    // Takes an element into the CTA's own list.
    __device__ __forceinline__ void take(float x, int tok) {
        const uint32_t at = atomicAdd(&sh.list_n, 1u);
        if (at < SP_LIST) sh.list[at] = (uint64_t(ord_f32(x)) << 32) | (0xffffffffu - uint32_t(tok));
    }
    // The CTAs' lists are made: how many elements there are in all, to every CTA.
    __device__ uint32_t listed() {
        __syncthreads();
        if (threadIdx.x < S) st_dsmem_u32(dsmem_addr(&sh.count[cr], threadIdx.x), sh.list_n);
        cluster_sync();
        uint32_t n = 0;
        for (uint32_t q = 0; q < S; ++q) n += sh.count[q];
        if (threadIdx.x == 0) sh.list_n = 0;               // (the next list is behind a barrier)
        return n;
    }
    template <typename F>
    __device__ uint32_t gather(F pred) {
        each([&](float x, int tok) {
            if (pred(x, tok)) take(x, tok);
        });
        return listed();
    }

    // CTA 0: all CTAs' lists, n elements (at most SP_LIST), together in its own.
    __device__ void pull_list(int n) {
        static_assert(SP_LIST == 2 * SP_NT, "two entries to a thread");
        uint64_t v[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            int k = int(threadIdx.x) + j * SP_NT;
            if (k < n)
                for (uint32_t q = 0; q < S; ++q) {
                    const int c = int(sh.count[q]);
                    if (k < c) {
                        v[j] = ld_dsmem_u64(dsmem_addr(&sh.list[k], q));
                        break;
                    }
                    k -= c;
                }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j) sh.list[threadIdx.x + j * SP_NT] = v[j];     // (zeros behind the n-th)
        __syncthreads();
    }
    template <int EPL>
    __device__ __forceinline__ void sort_warp() {
        const int at = EPL * int(threadIdx.x & 31);
        uint64_t v[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) v[j] = sh.list[at + j];
        warp_bitonic_desc<EPL>(v);
#pragma unroll
        for (int j = 0; j < EPL; ++j) sh.list[at + j] = v[j];
    }
    // The same, sorted, largest first: by one warp while they are few, else a bitonic network over two elements a
    // thread, 64 a warp: distances below 64 by shuffles, the others through shared memory.
    __device__ void sort_list(int n) {
        pull_list(n);
        if (n <= 256) {
            if (threadIdx.x < 32) {
                if (n <= 64) sort_warp<2>();
                else sort_warp<8>();
            }
            __syncthreads();
            return;
        }
        const int i0 = 2 * int(threadIdx.x);
        uint64_t v[2] = {sh.list[i0], sh.list[i0 + 1]};
        int P = 512;
        while (P < n) P *= 2;
        for (int k = 2; k <= P; k <<= 1)
            for (int d = k >> 1; d >= 1; d >>= 1) {
                const bool desc = (i0 & k) == 0;
                if (d == 1) {
                    const uint64_t a = v[0], b = v[1];
                    if (desc ? a < b : a > b) v[0] = b, v[1] = a;
                    continue;
                }
                if (d >= 64) {
                    __syncthreads();
                    sh.list[i0] = v[0], sh.list[i0 + 1] = v[1];
                    __syncthreads();
                }
                const bool keep_max = ((i0 & d) == 0) == desc;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint64_t o = d >= 64 ? sh.list[(i0 + j) ^ d] : shfl_xor_u64(v[j], d / 2);
                    v[j] = (v[j] > o) == keep_max ? v[j] : o;
                }
            }
        __syncthreads();
        sh.list[i0] = v[0], sh.list[i0 + 1] = v[1];
        __syncthreads();
    }
    static __device__ __forceinline__ float list_x(uint64_t e) { return f32_from_ord(uint32_t(e >> 32)); }
    static __device__ __forceinline__ int list_tok(uint64_t e) { return int(0xffffffffu - uint32_t(e)); }

    __device__ __forceinline__ void post_kept(uint64_t e) {
        for (uint32_t q = 0; q < S; ++q) {
            st_dsmem_u32(dsmem_addr(&sh.kx, q), __float_as_uint(list_x(e)));
            st_dsmem_u32(dsmem_addr(&sh.ki, q), uint32_t(list_tok(e)));
        }
    }

    // Vectors of a warp's stretch of the slice (whole strips of 32).
    static __device__ __forceinline__ int stretch(int nv) { return ((nv + SP_WARPS - 1) / SP_WARPS + 31) / 32 * 32; }

    // What the draw takes of the elements: above `sure` all, below `never` none, between by has() and the weight.
    struct Take {
        Kept kept;
        float sure, never;
    };
    __device__ Take take_of(const Kept& kept, const Filter& f) const {
        Take t{kept, kept.x, kept.x};
        if (f.wmin) {
            // (a few steps of the smallest floats, where the products are none)
            const float mid = wg.m + f.T * logf(f.least), slack = 1e-4f * f.T + 4e-7f * fabsf(wg.m) + 1e-44f;
            t.sure = fmaxf(t.sure, mid + slack), t.never = fmaxf(t.never, mid - slack);
        }
        return t;
    }
    // The elements x of vector i, what is not taken as -inf; false: none is.
    __device__ __forceinline__ bool taken(int i, const Take& t, uint64_t wmin, float (&x)[VEC]) const {
        float top = x[0];
        bool near = false;
#pragma unroll
        for (int e = 1; e < VEC; ++e) top = fmaxf(top, x[e]);
        if (top < t.never) return false;
#pragma unroll
        for (int e = 0; e < VEC; ++e) near |= x[e] <= t.sure && x[e] >= t.never && x[e] > -INFINITY;
        if (near) {
            uint32_t in = 0;                               // (by shared memory: x[] stays in registers)
#pragma unroll 1
            for (int e = 0; e < VEC; ++e) {
                const float y = sl.value(sl.first + i * VEC + e);
                if (t.kept.has(y, sl.first + i * VEC + e) &&
                    (y > t.sure || y == wg.m || !wmin || wg.one_call(y) >= wmin))
                    in |= 1u << e;
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] = (in >> e) & 1u ? x[e] : -INFINITY;
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] = x[e] > t.sure ? x[e] : -INFINITY;
        }
        return true;
    }

    // The sum over the lane's vectors of a warp's stretch.
    __device__ __forceinline__ uint64_t lane_sum(int v0, int v1, const Take& t, uint64_t wmin) const {
        uint64_t sum = 0;
        uint32_t i1 = 0, i2 = 0;
        int n = 0;
        sl.over(v0 + int(threadIdx.x & 31), v1, 32, [&](int i, float (&x)[VEC]) {
            if (!taken(i, t, wmin, x)) return;
            if (wg.slow) {
                uint64_t w[VEC];
                wg.template each<VEC>(x, w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) sum += x[e] > -INFINITY ? w[e] : 0;
            } else {
                wg.template add<VEC>(x, i1, i2);
                if (!HELD && ++n == SP_FLUSH / VEC) sum += Weigher::whole(i1, i2), i1 = i2 = 0, n = 0;
            }
        });
        return sum + Weigher::whole(i1, i2);
    }

    // The stretch of sums[S][SP_WARPS] that holds the goal-th unit (u of the whole, when u is not null), and the units
    // left in it. By each warp for itself: lane l has entries 4 l .. 4 l + 3.
    __device__ __forceinline__ int find_stretch(const uint64_t* sums, const uint64_t* u, uint64_t goal, uint64_t& left) const {
        const int lane = threadIdx.x & 31;
        uint64_t v[4], mine = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = 4 * lane + e < int(S) * SP_WARPS ? sums[4 * lane + e] : 0;
            mine += v[e];
        }
        const uint64_t inc = sp_warp_scan(mine), all = shfl_idx_u64(inc, 31);
        if (u) goal = __umul64hi(*u, all);                   // below `all`
        if (goal >= all) goal = all ? all - 1 : 0;
        uint64_t b = inc - mine;
        const unsigned hit = __ballot_sync(0xffffffffu, b <= goal && goal < b + mine);
        int at = 4 * lane;
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (goal >= b + v[e] && at == 4 * lane + e) b += v[e], ++at;
        const int l = hit ? __ffs(hit) - 1 : 0;
        left = shfl_idx_u64(goal - b, l);
        return __shfl_sync(0xffffffffu, at, l);
    }

    // The CTA that holds stretch `owner`: its strips, a warp each, then the strip that holds the unit `left`; the
    // token to all CTAs. measure(i, x, w): the weights of vector i's elements x.
    template <typename F>
    __device__ int walk(int owner, uint64_t left, F measure) {
        if (owner / SP_WARPS == int(cr)) {
            const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
            const int per = stretch(sl.nv), v0 = owner % SP_WARPS * per, v1 = min(v0 + per, sl.nv);
            uint64_t base = 0;
            for (int r0 = v0; r0 < v1; r0 += 32 * SP_WARPS) {
                const int i = r0 + 32 * wid + lane;
                uint64_t w[VEC], s = 0;
#pragma unroll
                for (int e = 0; e < VEC; ++e) w[e] = 0;
                if (i < v1) {
                    float x[VEC];
                    sl.values(i, x);
                    measure(i, x, w);
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) s += w[e];
                const uint64_t inc = sp_warp_scan(s), end = shfl_idx_u64(inc, 31);
                __syncthreads();
                if (lane == 0) sh.strip[wid] = end;
                __syncthreads();
                uint64_t all = 0, run = base;
#pragma unroll
                for (int k = 0; k < SP_WARPS; ++k) {
                    if (k < wid) run += sh.strip[k];
                    all += sh.strip[k];
                }
                uint64_t a = run + inc - s;
                if (a <= left && left < a + s) {
                    int tok = -1;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        if (tok < 0 && left < a + w[e]) tok = sl.first + i * VEC + e;
                        a += w[e];
                    }
                    for (uint32_t q = 0; q < S; ++q) st_dsmem_u32(dsmem_addr(&sh.token, q), uint32_t(tok));
                }
                base += all;
                if (left < base) break;
            }
        }
        cluster_sync();
        return int(sh.token);
    }
    __device__ int walk_kept(int owner, uint64_t left, const Kept& kept, const Filter& f) {
        const Take t = take_of(kept, f);
        return walk(owner, left, [&](int i, float (&x)[VEC], uint64_t (&w)[VEC]) {
            if (!taken(i, t, f.wmin, x)) return;
            wg.template each<VEC>(x, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[e] = x[e] > -INFINITY ? w[e] : 0;
        });
    }

    // The token at which the running sum of the kept elements' weights passes u times the whole.
    __device__ int draw(const Kept& kept, const Filter& f) {
        const int wid = threadIdx.x >> 5, per = stretch(sl.nv);
        const Take t = take_of(kept, f);
        const uint64_t sum = sp_warp_sum(lane_sum(min(wid * per, sl.nv), min(wid * per + per, sl.nv), t, f.wmin));
        if ((threadIdx.x & 31) < S) st_dsmem_u64(dsmem_addr(&sh.sums[cr][wid], threadIdx.x & 31), sum);
        cluster_sync();
        uint64_t left;
        const int owner = find_stretch(&sh.sums[0][0], &f.u, 0, left);
        return walk_kept(owner, left, kept, f);
    }

    // The (goal + 1)-th token whose value is `value`, of those in `kept`.
    __device__ int nth_equal(const Kept& kept, float value, uint64_t goal) {
        const int wid = threadIdx.x >> 5, per = stretch(sl.nv), v1 = min(wid * per + per, sl.nv);
        auto measure = [&](int i, const float (&x)[VEC], uint64_t (&w)[VEC]) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[e] = x[e] == value && kept.has(x[e], sl.first + i * VEC + e);
        };
        uint64_t sum = 0;
        sl.over(wid * per + int(threadIdx.x & 31), v1, 32, [&](int i, const float (&x)[VEC]) {
            uint64_t w[VEC];
            measure(i, x, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum += w[e];
        });
        sum = sp_warp_sum(sum);
        if ((threadIdx.x & 31) < S) st_dsmem_u64(dsmem_addr(&sh.sums[cr][wid], threadIdx.x & 31), sum);
        cluster_sync();
        uint64_t left;
        const int owner = find_stretch(&sh.sums[0][0], nullptr, goal, left);
        return walk(owner, left, measure);
    }

    // top-p of the whole row. 0: not found this way; 1: the token; 2: the last one kept (min-p comes behind it).
    // (row, V, seg: where a token's stretch is)
    __device__ int nucleus(const Filter& f, float low, const T* row, int V, int seg, Kept& kept, int& tok) {
        // (a little more than the range: the lowest value stays below the last place's end)
        const float m = wg.m, range = fminf(1.0001f * (m - low), 31.0f * f.T);
        const float s = range > 0.f ? 256.0f * SP_BINS / range : 0.f;
        if (!(s > 1e-30f && s < 1e30f) || wg.slow) return 0;
        const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
        for (int i = threadIdx.x; i < SP_BINS; i += SP_NT) sh.lo[i] = 0;
        if (threadIdx.x == 0) sh.b_lo = sh.b_hi = SP_BINS - 1;
        __syncthreads();
        // a bin's word: elements in the upper 12 bits, their 256ths of the bin (8 bits each) in the lower 20. (More than
        // 4095 of a CTA's elements in a bin: the elements do not add up, and the other way is taken.)
        uint32_t n = 0;
        sl.over(threadIdx.x, sl.nv, SP_NT, [&](int, const float (&x)[VEC]) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                // (beyond the range, 31 T: no weight; the sum's low bits are the nearest whole number)
                const float v = __fmul_rn(__fsub_rn(m, x[e]), s);
                if (v < 256.0f * SP_BINS - 0.5f) {
                    const uint32_t q = __float_as_uint(v + 8388608.0f);
                    atomicAdd(&sh.lo[(q >> 8) & (SP_BINS - 1)], (1u << 20) + (q & 255u));
                    ++n;
                }
            }
        });
        n = block_count(int(n));
        if (threadIdx.x < S) st_dsmem_u32(dsmem_addr(&sh.count[cr], threadIdx.x), n);
        cluster_sync();
        // the weights that the bins' counts and mean places stand for, in 2^-40; CTA r has bins [r nb, (r + 1) nb)
        const int nb = SP_BINS / int(S), per = (nb + SP_NT - 1) / SP_NT;   // 1, 2 or 4
        const int b0 = int(cr) * nb + int(threadIdx.x) * per;
        const bool mine = int(threadIdx.x) * per < nb;
        uint32_t c[4] = {0, 0, 0, 0}, fr[4] = {0, 0, 0, 0}, cs = 0;
        if (mine)
            for (uint32_t q = 0; q < S; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < per) {
                        const uint32_t v = ld_dsmem_u32(dsmem_addr(&sh.lo[b0 + i], q));
                        c[i] += v >> 20, fr[i] += v & 0xfffffu;
                    }
        uint64_t w[4] = {0, 0, 0, 0}, ws = 0, wb;
        const float scale = -1.4426950408889634f / (s * f.T);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c[i]) {
                const float at = float(256 * (b0 + i)) + float(fr[i]) / float(c[i]);
                w[i] = __float2ull_rn(float(c[i]) * ex2(fmaf(at, scale, 40.0f)));
                ws += w[i], cs += c[i];
            }
        const uint64_t wt = block_scan(ws, wb);
        const uint32_t ct = block_count(int(cs));
        if (threadIdx.x < S) {
            st_dsmem_u64(dsmem_addr(&sh.tot[cr], threadIdx.x), wt);
            st_dsmem_u32(dsmem_addr(&sh.first[cr], threadIdx.x), ct);
        }
        cluster_sync();
        uint64_t all = 0;
        uint32_t there = 0;
        for (uint32_t q = 0; q < S; ++q) {
            all += sh.tot[q], there += sh.count[q] - sh.first[q];
            if (q < cr) wb += sh.tot[q];
        }
        if (there != 0) return 0;
        // A bin is at most 31/2048 = 0.0151 wide in the exponent: its weight by the mean place is off by 0.0151^2 / 8
        // = 2.9e-5 of itself, by the places' rounding (half a 256th) 3e-5, by arithmetic 1e-6 at most. So the border
        // lies where the sums come within 2^-11 of p Z.
        const uint64_t pz = share_of(all, f), t1 = pz - (pz >> 11), t2 = pz + (pz >> 11);
        if (mine)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < per) {
                    const bool l = wb < t1 && t1 <= wb + w[i], h = wb < t2 && t2 <= wb + w[i];
                    for (uint32_t q = 0; q < S && (l || h); ++q) {
                        if (l) st_dsmem_u32(dsmem_addr(&sh.b_lo, q), uint32_t(b0 + i));
                        if (h) st_dsmem_u32(dsmem_addr(&sh.b_hi, q), uint32_t(b0 + i));
                    }
                    wb += w[i];
                }
        cluster_sync();
        const float lo_at = (float(256 * sh.b_lo) - 0.5f) / s, hi_at = (float(256 * (sh.b_hi + 1)) - 0.5f) / s;
        const float slack = (fabsf(m) + hi_at) * 1.9073486e-6f;            // 2^-19: roundings of (m - x) * s
        const float x_hi = sh.b_lo == 0 ? INFINITY : (m - lo_at) + slack;
        const float x_lo = sh.b_hi == SP_BINS - 1 ? -3.402823466e38f : (m - hi_at) - slack;
        if (f.wmin && take_of(kept, f).never > x_hi) return 2;             // (min-p keeps less than top-p)
        // weights of all and of what lies above x_hi, by stretches; x_lo .. x_hi to the list
        const int sv = stretch(sl.nv), v1 = min(wid * sv + sv, sl.nv);
        uint32_t i1 = 0, i2 = 0, a1 = 0, a2 = 0;
        uint64_t t_sum = 0, a_sum = 0;
        int held = 0;
        sl.over(wid * sv + lane, v1, 32, [&](int i, const float (&x)[VEC]) {
            uint32_t near = 0;
#pragma unroll
            for (int e = 0; e < VEC; ++e) near |= x[e] >= x_lo && x[e] <= x_hi ? 1u << e : 0u;
            wg.template add_above<VEC>(x, x_hi, i1, i2, a1, a2);
            while (near) {                                 // (by shared memory: x[] stays in registers)
                const int e = __ffs(near) - 1;
                near &= near - 1;
                take(sl.value(sl.first + i * VEC + e), sl.first + i * VEC + e);
            }
            if (!HELD && ++held == SP_FLUSH / VEC) {
                t_sum += Weigher::whole(i1, i2), a_sum += Weigher::whole(a1, a2);
                i1 = i2 = a1 = a2 = 0, held = 0;
            }
        });
        const uint64_t total = sp_warp_sum(t_sum + Weigher::whole(i1, i2));
        const uint64_t above = sp_warp_sum(a_sum + Weigher::whole(a1, a2));
        if (lane == 0) {
            st_dsmem_u64(dsmem_addr(&sh.sums[cr][wid], 0), total);
            st_dsmem_u64(dsmem_addr(&sh.above[cr][wid], 0), above);
        }
        const int ln0 = int(listed());
        if (cr == 0) {
            bool found = ln0 <= SP_LIST;
            if (found) {
                uint64_t z = 0, a = 0;
                if (wid == 0) {
                    for (int k = lane; k < int(S) * SP_WARPS; k += 32) z += (&sh.sums[0][0])[k], a += (&sh.above[0][0])[k];
                    z = sp_warp_sum(z), a = sp_warp_sum(a);
                    if (lane == 0) sh.strip[0] = z, sh.strip[1] = a;
                }
                // The weights of SP_NT slices of x_lo .. x_hi, in the histogram's place, the slice of the border, and its
                // elements compared with one another. Where they are many and of one value (bf16), slices of the
                // tokens first.
                unsigned long long* const slices = reinterpret_cast<unsigned long long*>(sh.lo);
                static_assert(SP_NT * 8 <= sizeof(sh.lo), "a slice for each thread");
                pull_list(ln0);
                const float top = x_hi == INFINITY ? m : x_hi, wide = top - x_lo;
                const float by_x = wide > 0.f ? float(SP_NT) / wide : 0.f, by_tok = float(SP_NT) / float(V);
                uint64_t lw[2] = {0, 0};
                bool in[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = int(threadIdx.x) + k * SP_NT;
                    in[k] = i < ln0;
                    if (in[k]) lw[k] = wg.one_call(list_x(sh.list[i]));
                }
                const uint64_t goal = share_of(sh.strip[0], f);
                uint64_t base = sh.strip[1];
                uint64_t* const some = sh.lw;
                int ns = 0;
                for (int level = 0; level < 2 && found; ++level) {
                    int at[2];
                    slices[threadIdx.x] = 0;
                    if (threadIdx.x == 0) sh.first[0] = 0, sh.first[1] = 0xffffffffu, sh.first[2] = 0;
                    __syncthreads();
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (in[k]) {
                            const uint64_t e = sh.list[threadIdx.x + k * SP_NT];
                            const float v = level == 0 ? (top - list_x(e)) * by_x : float(list_tok(e)) * by_tok;
                            at[k] = int(fminf(fmaxf(v, 0.f), float(SP_NT - 1)));
                            atomicAdd(&slices[at[k]], (unsigned long long)lw[k]);
                        }
                    __syncthreads();
                    const uint64_t own = slices[threadIdx.x];
                    uint64_t before;
                    const uint64_t all_in = block_scan(own, before);
                    before += base;
                    found = base < goal && goal <= base + all_in;
                    if (before < goal && goal <= before + own) sh.x.bin = threadIdx.x, sh.x.above = before;
                    __syncthreads();
                    base = sh.x.above;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        in[k] = in[k] && found && at[k] == int(sh.x.bin);
                        if (in[k]) {
                            const uint64_t e = sh.list[threadIdx.x + k * SP_NT];
                            atomicMin(&sh.first[1], uint32_t(e >> 32));
                            atomicMax(&sh.first[2], uint32_t(e >> 32));
                            const uint32_t i = atomicAdd(&sh.first[0], 1u);
                            if (i < SP_FEW / 2) some[2 * i] = e, some[2 * i + 1] = lw[k];
                        }
                    }
                    __syncthreads();
                    ns = int(sh.first[0]);
                    const bool one_value = sh.first[1] == sh.first[2];
                    __syncthreads();
                    if (ns <= SP_FEW / 2 || !one_value) break;
                }
                found = found && ns <= SP_FEW / 2;
                if (found && int(threadIdx.x) < ns) {
                    const uint64_t me = some[2 * threadIdx.x], w = some[2 * threadIdx.x + 1];
                    uint64_t b = base;
                    for (int i = 0; i < ns; ++i) b += some[2 * i] > me ? some[2 * i + 1] : 0;
                    if (b < goal && goal <= b + w) {
                        sh.x.goal = me;
                        post_kept(me);
                    }
                }
                __syncthreads();
                if (found) {
                    const uint64_t last = sh.x.goal;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (lw[k] && sh.list[threadIdx.x + k * SP_NT] >= last)
                            atomicAdd(reinterpret_cast<unsigned long long*>(&sh.above[0][0]) +
                                          stretch_of(list_tok(sh.list[threadIdx.x + k * SP_NT]), row, V, seg),
                                      (unsigned long long)lw[k]);
                    __syncthreads();
                    uint64_t left;
                    const int owner = wid == 0 ? find_stretch(&sh.above[0][0], &f.u, 0, left) : 0;
                    if (threadIdx.x == 0)
                        for (uint32_t q = 0; q < S; ++q) {
                            st_dsmem_u32(dsmem_addr(&sh.owner, q), uint32_t(owner));
                            st_dsmem_u64(dsmem_addr(&sh.left, q), left);
                        }
                }
            }
            if (threadIdx.x == 0) {
                for (uint32_t q = 0; q < S; ++q) st_dsmem_u32(dsmem_addr(&sh.done, q), found ? 1u : 0u);
            }
        }
        cluster_sync();
        if (!sh.done) return 0;
        kept = Kept{sh.kx, sh.ki};
        if (f.wmin) return 2;
        tok = walk_kept(int(sh.owner), sh.left, kept, f);
        return 1;
    }
    // Which of the cluster's stretches token t is in.
    __device__ int stretch_of(int t, const T* row, int V, int seg) const {
        const int q = t / seg, lo = q * seg, hi = min(lo + seg, V);
        const int shift = int((reinterpret_cast<uintptr_t>(row + lo) % 16) / sizeof(T));
        const int nv = (shift + (hi - lo) + VEC - 1) / VEC;
        return q * SP_WARPS + (t - lo + shift) / VEC / stretch(nv);
    }

    // CTA 0: of the list's n elements, the last one kept when `above` lies before them and the goal is
    // reached among them.
    template <bool MASS>
    __device__ Kept last_of_list(int n, uint64_t above, uint64_t goal) {
        if (cr == 0) {
            sort_list(n);
            const int i = 2 * int(threadIdx.x);
            uint64_t w[2] = {0, 0}, before;
            for (int e = 0; e < 2; ++e)
                if (i + e < n) w[e] = MASS ? wg.one(list_x(sh.list[i + e])) : 1;
            block_scan(w[0] + w[1], before);
            before += above;
            for (int e = 0; e < 2; ++e) {
                if (before < goal && goal <= before + w[e]) post_kept(sh.list[i + e]);
                before += w[e];
            }
        }
        cluster_sync();
        return Kept{sh.kx, sh.ki};
    }

    // Smallest count or weight that is at least p of z.
    static __device__ __forceinline__ uint64_t share_of(uint64_t z, const Filter& f) {
        const uint64_t g = __umul64hi(z, f.share) + (z * f.share != 0);
        return g < 1 ? 1 : g;
    }

    // The last element of `kept` before the goal: count k, or the share p of the weight.
    template <bool MASS>
    __device__ Kept select(const Kept& kept, const Filter& f, float low) {
        const float m = wg.m;
        // (below 31 T a weight is nothing; and what is below (1 - p) / V of the largest cannot be reached: all
        // of it together is less than 1 - p of the whole)
        const float range = MASS ? fminf(m - low, 31.0f * f.T) : m - low;
        Range g{m, range > 0.f ? float(SP_BINS) / range : 0.f, -1, 0u, 0u, 0};
        if (!(g.s < 3.0e38f)) g.s = 3.0e38f;
        Crossing c = crossing<MASS>(g, kept, f, MASS ? f.cut : 0, MASS, uint64_t(f.k));
        uint64_t above = c.above;
        const uint64_t goal = c.goal;
        // keys of the bin: its ends in x, with room for the roundings of (m - x) * s
        g.bin = int(c.bin);
        {
            const float a = g.s > 0.f ? float(c.bin) / g.s : 0.f, b = g.s > 0.f ? float(c.bin + 1) / g.s : 0.f;
            const float slack = (fabsf(m) + b) * 1.9073486e-6f;    // 2^-19
            const bool open = int(c.bin) == SP_BINS - 1;
            g.khi = c.bin == 0 ? ord_f32(m) : ord_f32(fminf(m, (m - a) + slack));
            g.klo = open || g.s == 0.f ? ord_f32(-3.402823466e38f) : ord_f32((m - b) - slack);
            if (m == low) g.khi = ord_f32(m), g.klo = g.khi;
        }
        while (true) {
            const Range h = g;
            const uint32_t n = gather([&](float x, int tok) -> bool {
                if (!kept.has(x, tok) || sp_bin(x, h) != h.bin) return false;
                const uint32_t key = ord_f32(x);
                return key <= h.khi && key >= h.klo;
            });
            if (n <= uint32_t(SP_LIST)) return last_of_list<MASS>(int(n), above, goal);
            if (g.khi == g.klo) {                          // one value: the r-th of its tokens
                const float x = f32_from_ord(g.khi);
                uint64_t r = goal - above;                 // >= 1
                if (MASS) {
                    const uint64_t w = wg.one(x);
                    r = (r + w - 1) / w;
                }
                return Kept{x, nth_equal(kept, x, r - 1)};
            }
            g.shift = 0;
            while (((g.khi - g.klo) >> g.shift) >= uint32_t(SP_BINS)) ++g.shift;
            c = crossing<MASS>(g, kept, f, 0, false, goal - above);
            above += c.above;
            const uint32_t hi = g.khi - (c.bin << g.shift), span = (1u << g.shift) - 1u;
            g.klo = hi - g.klo > span ? hi - span : g.klo;
            g.khi = hi;
        }
    }

    // CTA 0: top-k, top-p and min-p on the list's n elements, and the draw (true: the token); false: the last
    // one kept.
    __device__ bool finish_in_list(int n, const Filter& f, int V, Kept& kept, int& tok) {
        if (cr == 0) {
            sort_list(n);
            const int k = min(f.k, n), i = 2 * int(threadIdx.x);
            uint64_t w[2] = {0, 0}, before;
            for (int e = 0; e < 2; ++e)
                if (i + e < k) w[e] = wg.one(list_x(sh.list[i + e]));
            const uint64_t z = block_scan(w[0] + w[1], before);
            uint64_t goal = z;
            if (f.p < 1.f) {
                goal = share_of(z, f);
            }
            uint64_t kw = 0;                               // what is kept is a leading part of the list
            int kn = 0;
            for (int e = 0; e < 2; ++e) {
                const bool keep = i + e < k && (i + e == 0 || (before < goal && w[e] >= f.wmin && w[e] > 0));
                before += w[e];
                if (keep) kw += w[e], ++kn;
                else w[e] = 0;
            }
            const uint64_t total = block_scan(kw, before);
            const int n_kept = int(block_count(kn));
            // the draw: the kept weights by slices of the tokens, the slice of the goal, its elements compared
            unsigned long long* const slices = reinterpret_cast<unsigned long long*>(sh.lo);
            const float by_tok = float(SP_NT) / float(V);
            slices[threadIdx.x] = 0;
            if (threadIdx.x == 0) sh.first[0] = 0;
            __syncthreads();
            int at[2] = {-1, -1};
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (i + e < n_kept) {
                    at[e] = min(int(float(list_tok(sh.list[i + e])) * by_tok), SP_NT - 1);
                    atomicAdd(&slices[at[e]], (unsigned long long)w[e]);
                }
            __syncthreads();
            const uint64_t own = slices[threadIdx.x], pick = __umul64hi(f.u, total);
            block_scan(own, before);
            if (before <= pick && pick < before + own) sh.x.bin = threadIdx.x, sh.x.above = before;
            __syncthreads();
            uint64_t* const some = sh.lw;
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (at[e] >= 0 && at[e] == int(sh.x.bin)) {
                    const uint32_t q = atomicAdd(&sh.first[0], 1u);
                    if (q < SP_FEW / 2) some[2 * q] = uint64_t(list_tok(sh.list[i + e])), some[2 * q + 1] = w[e];
                }
            __syncthreads();
            const int ns = int(sh.first[0]);
            if (ns <= SP_FEW / 2) {
                if (int(threadIdx.x) < ns) {
                    const uint64_t me = some[2 * threadIdx.x];
                    uint64_t a = sh.x.above;
                    for (int q = 0; q < ns; ++q) a += some[2 * q] < me ? some[2 * q + 1] : 0;
                    if (a <= pick && pick < a + some[2 * threadIdx.x + 1])
                        for (uint32_t q = 0; q < S; ++q) {
                            st_dsmem_u32(dsmem_addr(&sh.token, q), uint32_t(me));
                            st_dsmem_u32(dsmem_addr(&sh.done, q), 1u);
                        }
                }
            } else if (threadIdx.x == 0) {                 // (more neighbouring tokens than that: by a pass over the row)
                post_kept(sh.list[n_kept - 1]);
                for (uint32_t q = 0; q < S; ++q) st_dsmem_u32(dsmem_addr(&sh.done, q), 0u);
            }
        }
        cluster_sync();
        kept = Kept{sh.kx, sh.ki}, tok = int(sh.token);
        return sh.done != 0;
    }
    __device__ uint32_t block_count(int n) {
        const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
        const uint32_t c = __reduce_add_sync(0xffffffffu, uint32_t(n));
        if (lane == 0) sh.redc[wid] = c;
        __syncthreads();
        uint32_t all = 0;
#pragma unroll
        for (int i = 0; i < SP_WARPS; ++i) all += sh.redc[i];
        return all;
    }
};

// The token of one row, to every thread of the cluster; -1 for a row that holds nothing but -inf and NaN.
// `data`: the CTA's shared memory for its slice. sh.f is set by a thread before.
template <typename T, bool HELD>
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
    // (thread t has vectors t, t + SP_NT, ..., as every pass over the slice by single vectors)
    const Slice<T, false> mem{reinterpret_cast<const uint4*>(base), row, nv, lo - shift, lo, hi, false};
    constexpr int U = 4;
    for (int i = threadIdx.x; i < nv; i += U * SP_NT) {
        uint4 v[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i + k * SP_NT < nv) v[k] = mem.raw(i + k * SP_NT);
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i + k * SP_NT < nv) {
                v[k] = E::clean4(v[k]);
                if (HELD) data[i + k * SP_NT] = v[k];
                see(v[k]);
            }
    }
    __syncthreads();
    const Filter f = sh.f;
    const float mine = top;
    top = warp_max(top);
    low = -warp_max(-low);
    if (lane == 0) sh.red[wid] = (uint64_t(__float_as_uint(top)) << 32) | __float_as_uint(low);
    if (threadIdx.x == 0) sh.list_n = 0;
    // the j-th largest of the threads' largest, its upper 16 bits
    const bool short_k = !f.greedy && f.k > 0 && f.k < V && f.k <= SP_LIST;
    uint32_t reach = 0;
    if (short_k) {
        const uint32_t o = ord_f32(mine);
        const int j = (f.k + int(S) - 1) / int(S);
        for (uint32_t bit = 0x80000000u; bit >= 0x10000u; bit >>= 1)
            if (__syncthreads_count(o >= (reach | bit)) >= j) reach |= bit;
    }
    __syncthreads();
    for (int i = 0; i < SP_WARPS; ++i) {
        top = fmaxf(top, __uint_as_float(uint32_t(sh.red[i] >> 32)));
        low = fminf(low, __uint_as_float(uint32_t(sh.red[i])));
    }
    if (threadIdx.x < S) {
        st_dsmem_u32(dsmem_addr(&sh.top[cr], threadIdx.x), __float_as_uint(top));
        st_dsmem_u32(dsmem_addr(&sh.low[cr], threadIdx.x), __float_as_uint(low));
        st_dsmem_u32(dsmem_addr(&sh.reach[cr], threadIdx.x), reach);
    }
    cluster_sync();
    for (uint32_t q = 0; q < S; ++q) {
        top = fmaxf(top, sh.top[q]), low = fminf(low, sh.low[q]);
        reach = min(reach, sh.reach[q]);
    }
    int tok = -1;
    if (top > -INFINITY) {
        Sampler<T, HELD> s{sh, Slice<T, HELD>{HELD ? data : mem.v, row, nv, lo - shift, lo, hi, false}, S, cr,
                           Weigher{}};
        if (f.greedy) {                                    // the maximum's lowest token
            uint32_t best = 0xffffffffu;
            if (mine == top) s.each([&](float x, int t) { if (x == top) best = min(best, uint32_t(t)); });
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
            if (top == INFINITY) {                         // it holds all the weight: nothing else is kept
                s.sl.only_inf = true;
                top = low = 0.f, reach = 0;
            }
            s.wg = sp_weigher(top, f, sh.table);
            Kept kept = SP_ALL;
            bool done = false, cut = f.p < 1.f;
            if (short_k) {
                if (s.sl.only_inf || ord_f32(mine) >= reach)           // (the thread has some)
                    s.each([&](float x, int t) {
                        if (x > -INFINITY && ord_f32(x) >= reach) s.take(x, t);
                    });
                const uint32_t n = s.listed();
                if (n <= uint32_t(SP_LIST)) {
                    done = s.finish_in_list(int(n), f, V, kept, tok);
                    cut = false;
                } else {
                    kept = s.template select<false>(kept, f, low);
                }
            } else if (f.k > 0 && f.k < V) {
                kept = s.template select<false>(kept, f, low);
            }
            if (!done && cut) {
                const int how = f.k > 0 && f.k < V ? 0 : s.nucleus(f, low, row, V, seg, kept, tok);
                done = how == 1;
                if (how == 0) kept = s.template select<true>(kept, f, low);
            }
            if (!done) tok = s.draw(kept, f);
        }
    }
    return tok;                                            // (behind a cluster barrier and what is read of others)
}

// Settings of request r for the row with uniform number ui; what is no setting is an error and taken for none.
__device__ __forceinline__ void sp_filter(const SampleArgs& a, int r, float u, SpShared& sh) {
    Filter f;
    bool bad = false;
    f.T = a.temperatures ? a.temperatures[r] : a.temperature;
    f.k = a.top_ks ? a.top_ks[r] : a.top_k;
    f.p = a.top_ps ? a.top_ps[r] : a.top_p;
    f.least = a.min_ps ? a.min_ps[r] : a.min_p;
    if (!(f.T >= 0.f && f.T < INFINITY)) bad = true, f.T = 0.f;
    if (f.k < 0) bad = true, f.k = 0;
    if (!(f.p >= 0.f && f.p <= 1.f)) bad = true, f.p = 1.f;
    if (!(f.least >= 0.f && f.least <= 1.f)) bad = true, f.least = 0.f;
    if (!(u >= 0.f && u < 1.f)) bad = true, u = 0.f;
    if (bad) set_status(a.status, DARTREE_EINTERNAL);
    f.greedy = f.T == 0.f || f.k == 1 || f.p == 0.f;
    // 256 / ln 2 (a pair) by T: the quotient, and the remainder's
    constexpr float KH = 369.329925537109375f, KL = 4.9304653e-6f;
    constexpr float BIG = 18446744073709551616.0f;         // 2^64
    f.up = f.T < 1.0f / BIG ? BIG : f.T > BIG ? 1.0f / BIG : 1.0f;
    const float T = f.T > 0.f ? f.T * f.up : 1.f;
    f.ch = __fdiv_rn(KH, T);
    f.cl = __fdiv_rn(__fmaf_rn(-f.ch, T, KH) + KL, T);
    f.u = sp_fixed(u, 64, false), f.share = f.p < 1.f ? sp_fixed(f.p, 64, true) : 0;
    f.wmin = f.least < 1.f ? sp_fixed(f.least, SP_Q, true) : uint64_t(1) << SP_Q;
    f.cut = sp_fixed(0.99f * (1.0f - f.p) / float(a.V), SP_Q, false);
    sh.f = f;
}

template <typename T, bool TREE, bool HELD>
__global__ void __launch_bounds__(SP_NT, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
    extern __shared__ __align__(16) uint4 sp_data[];
    __shared__ SpShared sh;
    __shared__ int found_s;
    const uint32_t S = cluster_nctarank(), cr = cluster_ctarank();
    const int r = int(blockIdx.x / S);
    cluster_arrive_release();
    for (int i = threadIdx.x; i < 256 * 8; i += SP_NT) sh.table[i] = sp_table.t[i >> 3];
    griddep_launch_dependents();
    griddep_wait();
    cluster_wait_acquire();                                // every CTA has started: its shared memory may be written
    const T* x = static_cast<const T*>(a.x);
    if constexpr (!TREE) {
        if (threadIdx.x == SP_NT - 1) sp_filter(a, r, a.u[r], sh);
        const int tok = sp_row<T, HELD>(x + size_t(r) * a.ld, a.V, a.seg, sh, sp_data, a.status);
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
            if (threadIdx.x == SP_NT - 1) sp_filter(a, r, a.u[at], sh), found_s = 0x7fffffff;
            const int t = sp_row<T, HELD>(x + at * a.V, a.V, a.seg, sh, sp_data, a.status);
            for (int j = 1 + int(threadIdx.x); j < n; j += SP_NT)
                if (t >= 0 && pr[j] == cur && tk[j] == t) atomicMin(&found_s, j);
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

constexpr int SP_SLICE = 76 * 1024;        // bytes of a slice beside which a second CTA fits
constexpr int SP_MOST = 190 * 1024;

// Elements of a CTA's slice with S CTAs to a row, and its bytes with the ends of an unaligned row.
static int sp_seg(int V, int S) { return ((V + S - 1) / S + 7) / 8 * 8; }
static int sp_bytes(int V, int S, int es) { return sp_seg(V, S) * es + 32; }

bool sample_supported(int V, int dtype) {
    return V <= (1 << 20) && sp_bytes(V, SP_MAXC, dtype == DARTREE_BF16 ? 2 : 4) <= SP_MOST;
}

template <typename T, bool TREE, bool HELD>
static int launch_sample_t(SampleArgs& a, int rows, int S, cudaStream_t stream) {
    a.seg = sp_seg(a.V, S);
    auto kern = sample_kernel<T, TREE, HELD>;
    static std::atomic<uint64_t> raised{0};
    if (HELD && !raise_smem(kern, SP_MOST, raised)) return DARTREE_ECUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(rows) * unsigned(S));
    cfg.blockDim = dim3(SP_NT);
    cfg.dynamicSmemBytes = HELD ? size_t(sp_bytes(a.V, S, int(sizeof(T)))) : 0;
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

// Rows held in shared memory: as few CTAs to a row as leave room for two on an SM, more while that does not fill
// the SMs. Batches that do not run at once that way are read again by each pass instead, by as many CTAs as fill
// the SMs.
template <typename T, bool TREE>
static int launch_sample_rows(SampleArgs& a, int rows, cudaStream_t stream) {
    const int es = int(sizeof(T));
    const int64_t slots = 2 * num_sms();
    int S = 1;
    while (S < SP_MAXC &&
           (sp_bytes(a.V, S, es) > SP_SLICE || (int64_t(rows) * S * 2 <= slots && a.V / (2 * S) >= 1024)))
        S *= 2;
    if constexpr (!TREE) {
        if (int64_t(rows) * S > slots && S > 1) {
            S = 1;
            while (S < SP_MAXC && int64_t(rows) * S * 2 <= slots) S *= 2;
            return launch_sample_t<T, false, false>(a, rows, S, stream);
        }
    }
    return launch_sample_t<T, TREE, true>(a, rows, S, stream);
}

static SampleArgs sample_args(const void* x, int V, const dartree_filter& f, const float* u, int* status) {
    SampleArgs a{};
    a.x = x, a.V = V, a.ld = V, a.u = u, a.status = status;
    a.temperature = f.temperature, a.top_k = f.top_k, a.top_p = f.top_p, a.min_p = f.min_p;
    a.temperatures = f.temperatures, a.top_ks = f.top_ks, a.top_ps = f.top_ps, a.min_ps = f.min_ps;
    return a;
}

int launch_sample(const void* logits, int rows, int V, int64_t ld, int dtype, const dartree_filter& f, const float* u,
                  int32_t* tok, int* status, cudaStream_t stream) {
    SampleArgs a = sample_args(logits, V, f, u, status);
    a.ld = ld, a.tok = tok;
    return dtype == DARTREE_BF16 ? launch_sample_rows<bf16_t, false>(a, rows, stream)
                                 : launch_sample_rows<float, false>(a, rows, stream);
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
    return dtype == DARTREE_BF16 ? launch_sample_rows<bf16_t, true>(a, C, stream)
                                 : launch_sample_rows<float, true>(a, C, stream);
}

}  // namespace dartree
