// The own rows of requests that share a prefix, and the join with it: at most 16 rows of q (tokens times heads of a
// key/value head) to a request, as in paged_few.cu and with its transposed products,
//
//   S^T = K Q^T,  O^T += V^T P^T,   out = (O 2^(m - M) + sum_k O_k 2^(m_k - M)) / (l 2^(m - M) + sum_k l_k 2^(m_k - M)),
//
// O_k, m_k and l_k being the shared rows' chunks, which the launch before leaves in memory. Own rows are few (what a
// request has beside a document that all have), so that a CTA for each (request, key/value head) would
// be mostly its own start: 64 requests of 8 heads are 512 CTAs, two waves of 10 us. So one wave of CTAs goes through
// them: tensor memory, barriers and descriptors are set up once, the next ones' keys and values are on their way
// while one is finished. The shared rows' launch lets this one start when all its CTAs have waited for what came before, and
// only the join waits for that launch: CTAs that find an SM free beside it take more requests than the others.
//
// CTA = some (request, key/value head) pairs, one after another, then their join:
//   warps 0..3  softmax, one thread per key, and the products with V (warp 0); O, maximum and sum as one more chunk,
//               in memory and the last pair's in shared memory; then, a warp to a row of q, the join
//   warp 4      producer: keys and values through a ring of ST stages; q when the scores before are done
//   warp 5      issues S^T, a block ahead of the softmax, into one of two buffers
// Blocks are numbered through all of a CTA's requests, so that the barriers' phases go on. Rows past the end may hold
// anything: their scores are masked and their values zeroed. P is rounded to bf16 as in paged_attn.cu and for its reason
// (outputs 2.3e-3 from 64 bits, relative, where one rounding to bf16 is 1.7e-3); everything else is fp32. Every wait is
// bounded; one that runs out records DARTREE_ETIMEOUT and ends the CTA's work.
// 64 tokens behind 16384 shared rows and up to 512 of their own (134 MB, 20 us at the memory's rate): 51.3 us with the
// shared rows in 64 CTAs (38 us) and three pairs to each of 171 others; 55.6 before the joins fetched the chunks' O ahead of
// their weights, 61.5 with the shared rows on 128 SMs, 65 with a CTA for each request and head. A CTA of one pair keeps
// no chunk in memory and is compiled by itself (51 tokens behind 3496 rows 17.6 us, 21 with the loops). Bound by the
// chain of a pair's lookups, blocks (1.7 us each), sums and chunks, two CTAs to an SM.
#include <cuda.h>

#include <algorithm>

#include "paged_attn.cuh"
#include "tc.cuh"

namespace dartree {

constexpr int PO_NT = 192;

template <int D, int ST>
struct PoSmem {
    static constexpr int PANELS = D / 64;
    static constexpr size_t PANEL = size_t(PF_BM) * 128;
    static constexpr size_t TILE = PANELS * PANEL;              // a block's keys or values
    static constexpr size_t QPANEL = PF_N * 128;
    static constexpr size_t Q_OFF = ST * TILE;
    static constexpr size_t P_OFF = Q_OFF + PANELS * QPANEL;    // [2][128 keys][16] bf16; then O [16][D] fp32
    static constexpr size_t PBUF = size_t(PF_BM) * PF_N * 2;
    static_assert(size_t(PF_N) * D * 4 <= 2 * PBUF, "O fits in P's place");
    static constexpr size_t RED_OFF = P_OFF + 2 * PBUF;         // float [4 warps][16]
    static constexpr size_t ML_OFF = RED_OFF + 4 * PF_N * 4;    // (maximum, sum) [16]
    static constexpr size_t BAR_OFF = ML_OFF + PF_N * 8;
    // qfull, qfree, full[ST], empty[ST], sfull[2], sfree[2], pdone[2]
    static constexpr size_t SLOT_OFF = BAR_OFF + 8 * (2 + 2 * ST + 6);
    static constexpr size_t TOTAL = SLOT_OFF + 16 + 1024;
    static_assert(2 * (TOTAL + 1024) <= 228 * 1024, "two CTAs fit in shared memory");
};

// ONE: each CTA has one pair
template <int D, int ST, bool ONE>
__global__ void __launch_bounds__(PO_NT, 2)
    paged_own_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PgArgs x) {
    using L = PoSmem<D, ST>;
    static_assert(ST == 3 || ST % 2 == 0, "what a stage of keys held before");
    constexpr uint32_t OCOL = 2 * PF_N, TCOLS = 64;          // TMEM: S^T at 16 b, O^T at 32
    const PagedArgs& a = x.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* qfull = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
    uint64_t* qfree = qfull + 1;      // the scores that read q are done
    uint64_t* full = qfree + 1;       // [ST] stage landed
    uint64_t* empty = full + ST;      // [ST] the MMAs that read it are done
    uint64_t* sfull = empty + ST;     // [2] scores written
    uint64_t* sfree = sfull + 2;      // [2] scores read
    uint64_t* pdone = sfree + 2;      // [2] the product with V that reads the buffer of P done
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + L::SLOT_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(qfull, 1);
        mbar_init(qfree, 1);
        for (int s = 0; s < ST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sfull[b], 1);
            mbar_init(&sfree[b], 4);
            mbar_init(&pdone[b], 1);
        }
        fence_mbar_init();
    }
    if (warp == 5) tc::tmem_alloc(slot, TCOLS);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *slot;
    griddep_launch_dependents();     // (what comes before the shared rows' launch is done: that waited for it)

    // this CTA's pairs: the first CTAs' early_items each, of the others an equal share (one more in the first of them)
    const int items = a.C * a.Hkv, cta = int(blockIdx.x), first = min(x.s.early * x.s.early_items, items);
    int it0, it1;
    if (ONE) {
        it0 = cta, it1 = cta + 1;
    } else if (cta < x.s.early) {
        it0 = min(cta * x.s.early_items, items), it1 = min(it0 + x.s.early_items, items);
    } else {
        const int others = int(gridDim.x) - x.s.early, i = cta - x.s.early, each = (items - first) / others,
                  extra = (items - first) - each * others;
        it0 = first + i * each + min(i, extra), it1 = it0 + each + int(i < extra);
    }
    struct Item {
        int c, g, kb, nblk;
        PagedRequest r;
        bool bad;
    };
    // request, head, first own row and blocks of an item (by a whole warp)
    auto item_of = [&](int it) -> Item {
        Item t;
        t.c = it / a.Hkv, t.g = it - t.c * a.Hkv;
        t.r = paged_request(a, t.c, t.bad);
        t.kb = paged_shared_rows(x, t.c, t.r.n_old, t.bad);
        t.nblk = t.r.n_new > 0 ? (max(t.r.n_keys - t.kb, 0) + PF_BM - 1) / PF_BM : 0;
        return t;
    };
    bool ok = true;
    int B = 0;                       // blocks of the items before

    if (warp == 4) {
        // ---------------------------------------------------------------- producer
        const int pr = min(a.page, PF_BM), sub = PF_BM / pr;              // rows and copies per panel of a block
        const int su = lane % sub, pn = lane / sub;                       // this lane's page and panel
        const bool mine = pn < L::PANELS;
        int n = 0, issued = 0;                                            // items with blocks so far; stages filled
        for (int it = it0; it < it1 && ok; ++it) {
            const Item t = item_of(it);
            if (t.bad && t.g == 0 && lane == 0) set_status(a.status, DARTREE_EINTERNAL);
            if (t.nblk == 0) continue;
            const int32_t* table = a.table + size_t(t.c) * a.max_pages;
            // this lane's table entry of block b (looked up two blocks ahead, checked when it is used), and
            // the page to fetch: n_pages, beyond the pool and so all zeros, past the end and for no page
            auto entry_of = [&](int b) -> int {
                const int j = t.kb + b * PF_BM + su * pr;
                return mine && j < t.r.n_keys ? table[j >> a.log2_page] : a.n_pages;
            };
            auto page_of = [&](int e, int b) -> int {
                if (unsigned(e) < unsigned(a.n_pages)) return e;
                if (mine && t.kb + b * PF_BM + su * pr < t.r.n_keys) set_status(a.status, DARTREE_EINTERNAL);
                return a.n_pages;
            };
            int e0 = entry_of(0), e1 = entry_of(1);
            if (lane == 0) {
                if (n > 0) ok = mbar_wait_bounded(qfree, uint32_t(n - 1) & 1u, a.status);
                if (ok) {
                    mbar_arrive_expect_tx(qfull, uint32_t(L::PANELS * x.tt * x.grp * 128));
                    for (int p = 0; p < L::PANELS; ++p)
                        tc::tma_load_3d(smem + L::Q_OFF + p * L::QPANEL, &tmQ, 64 * p, t.g * x.grp, t.r.q0, qfull);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            ++n;
            for (int i = 0; i < t.nblk && ok; ++i) {
                const int pg = page_of(e0, i);
                e0 = e1;
                e1 = entry_of(i + 2);
                for (int kv = 0; kv < 2; ++kv) {
                    const int idx = 2 * (B + i) + kv, s = idx % ST;
                    if (lane == 0 && idx >= ST)
                        ok = mbar_wait_bounded(&empty[s], uint32_t((idx / ST) & 1) ^ 1u, a.status);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&full[s], uint32_t(L::TILE));
                    __syncwarp();
                    if (mine)
                        tc::tma_load_4d(smem + s * L::TILE + pn * L::PANEL + size_t(su) * pr * 128, kv ? &tmV : &tmK,
                                        64 * pn, (t.kb + i * PF_BM + su * pr) & (a.page - 1), t.g, pg, &full[s]);
                    issued = idx + 1;
                }
            }
            B += t.nblk;
        }
        // copies issued and not yet seen complete land before the CTA can exit
        if (lane == 0) {
            if (n > 0) mbar_wait_bounded(qfull, uint32_t(n - 1) & 1u, a.status);
            for (int q = max(issued - ST, 0); q < issued; ++q)
                mbar_wait_bounded(&full[q % ST], uint32_t(q / ST) & 1u, a.status);
        }
    } else if (warp == 5) {
        // ---------------------------------------------------------------- scores
        // (warp-uniform values, one elected lane: descriptors stay in uniform registers)
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        int n = 0;
        for (int it = it0; it < it1 && ok; ++it) {
            const Item t = item_of(it);
            const int nb = __shfl_sync(0xffffffffu, t.nblk, 0), b0 = __shfl_sync(0xffffffffu, B, 0);
            if (nb == 0) continue;
            if (tc::elect_one()) {
                constexpr uint32_t id = tc::idesc_bf16_f32(PF_BM, PF_N);
                constexpr uint32_t HI = uint32_t(tc::DESC_SW128_KMAJOR >> 32), LO = uint32_t(tc::DESC_SW128_KMAJOR);
                const uint32_t r0 = (smem_u32(smem) >> 4) & 0x3fffu, q0 = (smem_u32(smem + L::Q_OFF) >> 4) & 0x3fffu;
                auto desc = [&](uint32_t at) { return (uint64_t(HI) << 32) | (LO | at); };
                ok = mbar_wait_bounded(qfull, uint32_t(n) & 1u, a.status);
                for (int i = 0; i < nb && ok; ++i) {
                    // A wait for a phase that is two ahead would take the one before for it, one for a phase that is
                    // two behind would not end. A stage of keys in a ring of three held the values of block gi - 2
                    // before, which are waited for elsewhere: once they were read, the keys' phase is the next. In
                    // an even ring it held keys.
                    const int gi = b0 + i, ki = 2 * gi, s = ki % ST;
                    if (ST == 3 && gi >= 2) ok = mbar_wait_bounded(&pdone[gi & 1], uint32_t((gi >> 1) - 1) & 1u, a.status);
                    ok = ok && mbar_wait_bounded(&full[s], uint32_t(ki / ST) & 1u, a.status);
                    if (ok && gi >= 2) ok = mbar_wait_bounded(&sfree[gi & 1], uint32_t((gi >> 1) - 1) & 1u, a.status);
                    if (!ok) break;
                    tc::fence_after_sync();
                    const uint32_t da = r0 + uint32_t(s) * uint32_t(L::TILE >> 4);
#pragma unroll
                    for (int p = 0; p < L::PANELS; ++p)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc::mma_bf16(tm + uint32_t((gi & 1) * PF_N), desc(da + p * uint32_t(L::PANEL >> 4) + 2u * kk),
                                         desc(q0 + p * uint32_t(L::QPANEL >> 4) + 2u * kk), id, p > 0 || kk > 0);
                    // (before the scores' barrier: these arrive while the CTA still waits for that one)
                    tc::mma_commit(&empty[s]);
                    if (i + 1 == nb) tc::mma_commit(qfree);
                    tc::mma_commit(&sfull[gi & 1]);
                }
            }
            ok = __any_sync(0xffffffffu, !ok) == 0;
            B += nb;
            ++n;
        }
    } else {
        // ---------------------------------------------------------------- softmax
        const int key = threadIdx.x;                                 // row of a block (TMEM lane)
        const uint32_t head1 = (1u << x.grp) - 1u;                   // (grp <= 16)
        const uint32_t by_grp = 65535u / uint32_t(x.grp) + 1u;
        // row of q of column n < 16 behind column 0's: the token n / grp, its head (exact; a division here is 40 instructions)
        auto row_at = [&](int n) -> size_t {
            const uint32_t t = uint32_t(n) * by_grp >> 16;
            return size_t(t) * a.Hq + (uint32_t(n) - t * uint32_t(x.grp));
        };
        const uint32_t trow = tmem + (uint32_t(warp * 32) << 16);
        float* const red = reinterpret_cast<float*>(smem + L::RED_OFF);
        float2* const ml = reinterpret_cast<float2*>(smem + L::ML_OFF);
        float* const ob = reinterpret_cast<float*>(smem + L::P_OFF);
        const size_t step = size_t(a.T) * a.Hq;                      // (chunk k of a row of q: part[k * step + row])
        // the 128 threads' barrier, with their vote
        auto vote = [](bool v) -> bool {
            uint32_t any;
            __syncwarp();
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                         "barrier.cta.red.or.pred.aligned q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                         : "=r"(any) : "r"(uint32_t(v)) : "memory");
            return any != 0;
        };
        for (int it = it0; it < it1 && ok; ++it) {
            const Item t = item_of(it);
            const PagedRequest& r = t.r;
            const int nblk = t.nblk, cols = r.n_new * x.grp;         // rows of q with a token
            const uint32_t live = (1u << cols) - 1u;                 // (cols <= 16)
            float m[PF_N], l[PF_N], p[PF_N];
#pragma unroll
            for (int n = 0; n < PF_N; ++n) m[n] = -INFINITY, l[n] = 0.f;
            for (int i = 0; i < nblk; ++i) {
                const int gi = B + i, j = t.kb + i * PF_BM + key, s = j - r.n_old, vi = 2 * gi + 1;
                uint32_t seen = j < r.n_keys ? live : 0u;
                if (s >= 0 && seen) {                                // a new row
                    if (!a.mask) {
                        seen &= ~((1u << s * x.grp) - 1u);           // (s < n_new)
                    } else {
                        const uint8_t* col = a.mask + size_t(t.c) * a.S * a.S + s;
                        uint8_t v[PF_N];
#pragma unroll
                        for (int n = 0; n < PF_N; ++n) v[n] = col[size_t(min(n, r.n_new - 1)) * a.S];
                        seen = 0;
#pragma unroll
                        for (int n = 0; n < PF_N; ++n)
                            if (n < r.n_new && v[n]) seen |= head1 << n * x.grp;
                    }
                }
                ok = ok && mbar_wait_bounded(&sfull[gi & 1], uint32_t(gi >> 1) & 1u, a.status);
                if (gi >= 2) ok = ok && mbar_wait_bounded(&pdone[gi & 1], uint32_t((gi >> 1) - 1) & 1u, a.status);
                if (i + 1 == nblk && r.n_keys < t.kb + nblk * PF_BM) {
                    // rows past the end may hold anything: their values are zeroed (0 * NaN is NaN)
                    ok = ok && mbar_wait_bounded(&full[vi % ST], uint32_t(vi / ST) & 1u, a.status);
                    if (ok && j >= r.n_keys) {
                        uint4* vrow = reinterpret_cast<uint4*>(smem + (vi % ST) * L::TILE + size_t(key) * 128);
#pragma unroll
                        for (int e = 0; e < 8 * L::PANELS; ++e)
                            vrow[(e >> 3) * (L::PANEL / 16) + (e & 7)] = make_uint4(0, 0, 0, 0);
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                uint32_t sc[PF_N];
                if (ok) {
                    tc::fence_after_sync();
                    tc::tmem_ld16(trow + uint32_t((gi & 1) * PF_N), sc);
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sfree[gi & 1]);
                }
                // P of the block against the maxima in use, to shared memory; the largest weight. (No maximum yet:
                // the weight of a key that is seen is infinite.)
                uint8_t* const pb = smem + L::P_OFF + (gi & 1) * L::PBUF + key * 32;
                const int flip = (key >> 2) & 1;
                auto weigh = [&]() -> float {
                    float big = 0.f;
                    uint32_t pk[PF_N / 2];
#pragma unroll
                    for (int n = 0; n < PF_N; ++n) {
                        p[n] = (seen >> n) & 1u ? ex2(fmaf(__uint_as_float(sc[n]), x.sl2, -m[n])) : 0.f;
                        big = fmaxf(big, p[n]);
                        if (n & 1) pk[n / 2] = pack2(p[n - 1], p[n]);
                    }
                    reinterpret_cast<uint4*>(pb)[flip] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    reinterpret_cast<uint4*>(pb)[flip ^ 1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                    fence_proxy_async_smem();
                    return big;
                };
                bool redo = i == 0;
                if (!redo) {
                    float big = 0.f;
                    if (ok) big = weigh();
                    redo = vote(ok && !(big <= PG_MOST));
                }
                if (redo) {
                    float v[PF_N];
#pragma unroll
                    for (int n = 0; n < PF_N; ++n)
                        v[n] = ok && (seen >> n) & 1u ? __uint_as_float(sc[n]) : -INFINITY;
                    const float top = warp_columns(v, lane, [](float u, float w) { return fmaxf(u, w); });
                    if (lane < PF_N) red[warp * PF_N + lane] = top * x.sl2;  // (sl2 > 0: -inf stays)
                    vote(false);
                    float f[PF_N];
#pragma unroll
                    for (int n = 0; n < PF_N; ++n) {
                        const float mx = fmaxf(fmaxf(red[n], red[PF_N + n]), fmaxf(red[2 * PF_N + n], red[3 * PF_N + n]));
                        f[n] = mx > m[n] && m[n] > -INFINITY ? ex2(m[n] - mx) : 1.f;
                        m[n] = fmaxf(m[n], mx);
                        l[n] *= f[n];
                    }
                    if (i > 0) {                                     // the products so far
                        ok = ok && mbar_wait_bounded(&pdone[(gi - 1) & 1], uint32_t((gi - 1) >> 1) & 1u, a.status);
                        ok = __all_sync(0xffffffffu, ok);
                        if (ok) {
                            uint32_t o[PF_N];
                            tc::fence_after_sync();
                            tc::tmem_ld16(trow + OCOL, o);
#pragma unroll
                            for (int n = 0; n < PF_N; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * f[n]);
                            tc::tmem_st16_async(trow + OCOL, o);
                            tc::tmem_wait_st();
                            tc::fence_before_sync();
                        }
                    }
                    if (ok) weigh();
                    vote(false);
                }
#pragma unroll
                for (int n = 0; n < PF_N; ++n) l[n] += ok ? p[n] : 0.f;
                if (warp == 0 && ok) {
                    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
                    const int u = __shfl_sync(0xffffffffu, gi, 0), u0 = __shfl_sync(0xffffffffu, i, 0);
                    if (tc::elect_one()) {
                        constexpr uint32_t id = tc::idesc_bf16_f32(PF_BM, PF_N) | tc::IDESC_A_MNMAJOR | tc::IDESC_B_MNMAJOR;
                        // (heads of 64 fill both halves of the 128 rows: a step of zero bytes to the next panel)
                        constexpr uint64_t VD = tc::desc_sw128_mnmajor_base(D == 128 ? uint32_t(L::PANEL) : 0u);
                        constexpr uint64_t PD = tc::DESC_SW32_MNMAJOR;
                        const int w = 2 * u + 1, sv = w % ST;
                        if (mbar_wait_bounded(&full[sv], uint32_t(w / ST) & 1u, a.status)) {
                            tc::fence_after_sync();
                            const uint32_t da = ((smem_u32(smem) >> 4) & 0x3fffu) + uint32_t(sv) * uint32_t(L::TILE >> 4);
                            const uint32_t db = (smem_u32(smem + L::P_OFF + (u & 1) * L::PBUF) >> 4) & 0x3fffu;
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                tc::mma_bf16(tm + OCOL, VD | (da + 128u * kk), PD | (db + 32u * kk), id, u0 > 0 || kk > 0);
                            tc::mma_commit(&empty[sv]);
                            tc::mma_commit(&pdone[u & 1]);
                        }
                    }
                    __syncwarp();
                }
            }
            // ------------------------------------------------------------ end of the own rows
            if (nblk > 0) {
                const int gl = B + nblk - 1;
                ok = ok && mbar_wait_bounded(&pdone[gl & 1], uint32_t(gl >> 1) & 1u, a.status);
                ok = __all_sync(0xffffffffu, ok);
            }
            float v[PF_N];
#pragma unroll
            for (int n = 0; n < PF_N; ++n) v[n] = l[n];
            const float part = warp_columns(v, lane, [](float u, float w) { return u + w; });
            vote(false);                                             // (red: the last maxima are read)
            if (lane < PF_N) red[warp * PF_N + lane] = part;
            ok = !vote(!ok);
            if (!ok) break;                                          // (all 128 threads)
            uint32_t o[PF_N];
            if (nblk > 0) {
                tc::fence_after_sync();
                tc::tmem_ld16(trow + OCOL, o);
                tc::fence_before_sync();
            }
            // one more chunk of the rows of q: in memory, the last pair's in P's place (every product is done)
            const bool last = ONE || it + 1 == it1;
            const size_t own = size_t(x.s.np) * step + size_t(r.q0) * a.Hq + size_t(t.g) * x.grp;
#pragma unroll
            for (int n = 0; n < PF_N; ++n) {
                const float sum = nblk > 0 ? (red[n] + red[PF_N + n]) + (red[2 * PF_N + n] + red[3 * PF_N + n]) : 0.f;
                const size_t at = own + row_at(n);
                const float2 own_ml = sum > 0.f ? make_float2(m[n], sum) : make_float2(-INFINITY, 0.f);
                if (last) {
                    if (n == key) ml[n] = own_ml;
                    if (key < D && n < cols && nblk > 0) ob[n * D + key] = __uint_as_float(o[n]);
                } else if (n < cols) {
                    if (n == key) x.part_ml[at] = own_ml;
                    if (key < D && nblk > 0) x.part_o[at * D + key] = __uint_as_float(o[n]);
                }
            }
            vote(false);                                             // (red is read)
            B += nblk;
        }
        // ------------------------------------------------------------ join: a warp to a row of q
        PagedRequest r{};
        bool shares = false;                                         // (looked up before the waits)
        auto look = [&](int it) {
            if (!ONE && it < it0) return;
            r = paged_request(a, it / a.Hkv);
            shares = paged_in_group(x, it / a.Hkv);
        };
        look(it1 - 1);
        griddep_wait();                                              // the shared rows' launch
        for (int it = it1 - 1; it >= it0 && ok; --it) {
            const bool last = ONE || it + 1 == it1;
            const int g = it % a.Hkv;
            const int cols = r.n_new * x.grp, rows = a.q_start ? cols : x.rows;   // (slots without a node get zeros)
            const int np = shares ? x.s.np : 0;
            const size_t o0 = size_t(r.q0) * a.Hq + size_t(g) * x.grp;
            auto row_of = [&](int n) -> size_t { return o0 + row_at(n); };
            constexpr int V = D / 32, RW = PF_N / 4;
            float2 pm[RW][3];                                        // chunks `lane` and `lane` + 32 (np <= 64), own rows
#pragma unroll
            for (int q = 0; q < RW; ++q) {
                const int n = warp + 4 * q;
#pragma unroll
                for (int h = 0; h < 3; ++h) {
                    const int k = h == 2 ? x.s.np : lane + 32 * h;
                    pm[q][h] = make_float2(-INFINITY, 0.f);
                    if (n < cols && (h == 2 || k < np)) pm[q][h] = h == 2 && last ? ml[n] : __ldcg(x.part_ml + k * step + row_of(n));
                }
            }
            if (!ONE) look(it - 1);
#pragma unroll
            for (int q = 0; q < RW; ++q) {
                const int n = warp + 4 * q;
                if (n >= rows) break;
                const size_t row = row_of(n);
                // the chunks' O, eight at a time; the first are on their way before the weights (a chunk in which
                // nothing was seen has no O: what is read has no weight)
                float y[8][V];
                auto fetch = [&](int k0) {
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
#pragma unroll
                        for (int e = 0; e < V; ++e) y[u][e] = 0.f;
                        if (k0 + u < np && n < cols) {
                            const float* src = x.part_o + (size_t(k0 + u) * step + row) * D + lane * V;
                            if (V == 4) {
                                const float4 z = __ldcg(reinterpret_cast<const float4*>(src));
                                y[u][0] = z.x, y[u][1] = z.y, y[u][V - 2] = z.z, y[u][V - 1] = z.w;
                            } else {
                                const float2 z = __ldcg(reinterpret_cast<const float2*>(src));
                                y[u][0] = z.x, y[u][1] = z.y;
                            }
                        }
                    }
                };
                fetch(0);
                float top = -INFINITY, fk[3];
#pragma unroll
                for (int h = 0; h < 3; ++h)
                    if (pm[q][h].y > 0.f) top = fmaxf(top, pm[q][h].x);
                top = warp_max(top);
#pragma unroll
                for (int h = 0; h < 3; ++h) fk[h] = pm[q][h].y > 0.f ? ex2(pm[q][h].x - top) : 0.f;
                const float sum = fmaf(fk[2], pm[q][2].y, warp_sum(fmaf(fk[0], pm[q][0].y, fk[1] * pm[q][1].y)));
                const float inv = sum > 0.f ? 1.0f / sum : 0.f;
                float acc[V];
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] = 0.f;
                if (fk[2] > 0.f) {
                    const float* src = x.part_o + (x.s.np * step + row) * D + lane * V;
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] = (last ? ob[n * D + lane * V + e] : __ldcg(src + e)) * (fk[2] * inv);
                }
                for (int k0 = 0; k0 < np && n < cols; k0 += 8) {
                    if (k0 > 0) fetch(k0);
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const int k = k0 + u;
                        const float w = __shfl_sync(0xffffffffu, k < 32 ? fk[0] : fk[1], k & 31) * inv;
#pragma unroll
                        for (int e = 0; e < V; ++e) acc[e] = w > 0.f ? fmaf(w, y[u][e], acc[e]) : acc[e];
                    }
                }
                uint32_t* dst = reinterpret_cast<uint32_t*>(x.out + row * D) + lane * (V / 2);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) dst[e] = pack2(acc[2 * e], acc[2 * e + 1]);
                if (x.lse && lane == 0)
                    x.lse[row] = sum > 0.f ? (top + log2f(sum)) * 0.6931471805599453f : n < cols ? -INFINITY : 0.f;
            }
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 5) tc::tmem_dealloc(tmem, TCOLS);
}

template <int D, int ST>
static int launch_own_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PgArgs& x,
                        cudaStream_t stream) {
    const size_t smem = PoSmem<D, ST>::TOTAL;
    cudaLaunchConfig_t cfg{};
    // the early CTAs, and of others as many as the fewest rounds need
    const int64_t items = int64_t(x.a.C) * x.a.Hkv, slots = 2 * num_sms();
    const int64_t left = items - std::min(items, int64_t(x.s.early) * x.s.early_items);
    const int64_t rounds = (left + slots - 1) / slots;
    const bool one = (x.s.early == 0 || x.s.early_items == 1) && rounds <= 1;
    auto kern = one ? paged_own_kernel<D, ST, true> : paged_own_kernel<D, ST, false>;
    static std::atomic<uint64_t> raised[2];
    if (!raise_smem(kern, int(smem), raised[one])) return DARTREE_ECUDA;
    cfg.gridDim = dim3(unsigned(one ? items : x.s.early + (rounds > 0 ? (left + rounds - 1) / rounds : 0)));
    cfg.blockDim = dim3(PO_NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    KTimer kt_(KID_PAGED_OWN, stream);
    return cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, x) == cudaSuccess ? DARTREE_OK : DARTREE_ECUDA;
}

int launch_paged_own(const PgArgs& x, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t stream) {
    return x.a.D == 64 ? launch_own_t<64, 6>(tq, tk, tv, x, stream) : launch_own_t<128, 3>(tq, tk, tv, x, stream);
}

}  // namespace dartree
