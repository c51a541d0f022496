// Attention of few rows over the paged key/value cache: tokens times heads of a key/value
// head at most 16 (single tokens, short drafts). The mathematics, the chunks of key blocks
// and their merge are the general kernel's; the products are transposed,
//
//   S^T = K Q^T  (128 keys x 16 rows),   O^T += V^T P^T  (D x 16 rows),
//
// so that a block costs the tensor cores and the softmax 16 rows, not 128: there a block of
// a lone CTA takes 1.5 us however few rows live. One token over 2048 rows: 9.0 us (10.5 there), 64
// tokens over 4096-8192 rows: 236 us (260), 6.8 TB/s. P is rounded to bf16 as there: a token's
// output has the same bound whichever kernel its batch goes to.
//
// CTA = (chunk of key blocks, (request, key/value head)):
//   warps 0..3  softmax, one thread per key: its 16 scores, P in bf16 to shared memory (an
//               MN-major operand, 32-byte swizzle); warp 0 issues O^T += V^T P^T (V as
//               it lies in its pages, MN-major)
//   warp 4      producer, as in the general kernel
//   warp 5      issues S^T, a block ahead of the softmax, into one of two buffers
// Sums stay with the threads until the end. Weights are formed against the rows' maxima of the
// blocks before; the threads' vote of a block (the barrier that P needs anyway) finds a
// weight above 2^14, and then, and in the first block, the maxima are taken across the keys and O is
// rescaled. Every wait is bounded; one that runs out records DARTREE_ETIMEOUT.
#include <cuda.h>

#include "paged_attn.cuh"
#include "tc.cuh"

namespace dartree {

constexpr int PF_NT = 192;

template <int D, int ST>
struct PfSmem {
    static constexpr int PANELS = D / 64;
    static constexpr size_t PANEL = size_t(PF_BM) * 128;
    static constexpr size_t TILE = PANELS * PANEL;              // a block's keys or values
    static constexpr size_t QPANEL = PF_N * 128;
    static constexpr size_t Q_OFF = ST * TILE;
    static constexpr size_t P_OFF = Q_OFF + PANELS * QPANEL;    // [2][128 keys][16] bf16
    static constexpr size_t PBUF = size_t(PF_BM) * PF_N * 2;
    static constexpr size_t RED_OFF = P_OFF + 2 * PBUF;         // float [4 warps][16]
    static constexpr size_t ML_OFF = RED_OFF + 4 * PF_N * 4;    // (maximum, sum) [16]
    static constexpr size_t PLACE_OFF = ML_OFF + PF_N * 8;      // int [16]
    static constexpr size_t BAR_OFF = PLACE_OFF + PF_N * 4;
    // qfull, full[ST], empty[ST], sfull[2], sfree[2], pdone[2]
    static constexpr size_t SLOT_OFF = BAR_OFF + 8 * (1 + 2 * ST + 6);
    static constexpr size_t TOTAL = SLOT_OFF + 16 + 1024;
    static_assert(TOTAL <= 227 * 1024, "fits in shared memory");
    static constexpr int PITCH = D + 4;                         // merge of a cluster's chunks, over the ring: O [16][PITCH]
    static_assert(PF_N * PITCH * 4 <= ST * TILE, "merge fits in the ring's place");
};

template <int D, int ST, bool CL>
__global__ void __launch_bounds__(PF_NT, 2)
    paged_few_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PgArgs x) {
    static_assert(ST == 3 || ST % 2 == 0, "what a stage of keys held before");
    using L = PfSmem<D, ST>;
    constexpr uint32_t OCOL = 2 * PF_N, TCOLS = 64;          // TMEM: S^T at 16 b, O^T at 32
    const PagedArgs& a = x.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* qfull = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
    uint64_t* full = qfull + 1;       // [ST] stage landed
    uint64_t* empty = full + ST;      // [ST] the MMAs that read it are done
    uint64_t* sfull = empty + ST;     // [2] scores written
    uint64_t* sfree = sfull + 2;      // [2] scores read
    uint64_t* pdone = sfree + 2;      // [2] the product with V that reads the buffer of P done
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + L::SLOT_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(qfull, 1);
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
    griddep_launch_dependents();
    griddep_wait();

    const int chunk = int(blockIdx.x % x.nchunk), cg = int(blockIdx.x / x.nchunk);
    const int c = cg / a.Hkv, g = cg - c * a.Hkv;
    bool bad;
    const PagedRequest r = paged_request(a, c, bad);
    if (bad && threadIdx.x == 0 && g == 0) set_status(a.status, DARTREE_EINTERNAL);
    const int blocks = r.n_new > 0 ? (r.n_keys + PF_BM - 1) / PF_BM : 0;
    const int per = (blocks + x.nchunk - 1) / x.nchunk;
    const int b0 = chunk * per, nblk = max(min(blocks, b0 + per) - b0, 0);

    if (warp == 4) {
        // ---------------------------------------------------------------- producer
        if (nblk > 0) {
            const int pr = min(a.page, PF_BM), sub = PF_BM / pr;          // rows and copies per panel of a block
            if (lane == 0) {
                mbar_arrive_expect_tx(qfull, uint32_t(L::PANELS * x.tt * x.grp * 128));
                for (int p = 0; p < L::PANELS; ++p)
                    tc::tma_load_3d(smem + L::Q_OFF + p * L::QPANEL, &tmQ, 64 * p, g * x.grp, r.q0, qfull);
            }
            const int su = lane % sub, pn = lane / sub;                   // this lane's page and panel
            const bool mine = pn < L::PANELS;
            const int32_t* table = a.table + size_t(c) * a.max_pages;
            // this lane's table entry of block b (looked up two blocks ahead, checked when it is used), and
            // the page to fetch: n_pages, beyond the pool and so all zeros, past the end and for no page
            auto entry_of = [&](int b) -> int {
                const int j = b * PF_BM + su * pr;
                return mine && j < r.n_keys ? table[j >> a.log2_page] : a.n_pages;
            };
            auto page_of = [&](int e, int b) -> int {
                if (unsigned(e) < unsigned(a.n_pages)) return e;
                if (mine && b * PF_BM + su * pr < r.n_keys) set_status(a.status, DARTREE_EINTERNAL);
                return a.n_pages;
            };
            int e0 = entry_of(b0), e1 = entry_of(b0 + 1), issued = 0;
            bool ok = true;
            for (int i = 0; i < nblk && ok; ++i) {
                const int pg = page_of(e0, b0 + i);
                e0 = e1;
                e1 = entry_of(b0 + i + 2);
                for (int kv = 0; kv < 2; ++kv) {
                    const int idx = 2 * i + kv, s = idx % ST;
                    if (lane == 0 && idx >= ST)
                        ok = mbar_wait_bounded(&empty[s], uint32_t((idx / ST) & 1) ^ 1u, a.status);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&full[s], uint32_t(L::TILE));
                    __syncwarp();
                    if (mine)
                        tc::tma_load_4d(smem + s * L::TILE + pn * L::PANEL + size_t(su) * pr * 128, kv ? &tmV : &tmK,
                                        64 * pn, ((b0 + i) * PF_BM + su * pr) & (a.page - 1), g, pg, &full[s]);
                    issued = idx + 1;
                }
            }
            // copies issued and not yet seen complete land before the CTA can exit
            if (lane == 0) {
                mbar_wait_bounded(qfull, 0, a.status);
                for (int q = max(issued - ST, 0); q < issued; ++q)
                    mbar_wait_bounded(&full[q % ST], uint32_t(q / ST) & 1u, a.status);
            }
        }
    } else if (warp == 5) {
        // ---------------------------------------------------------------- scores
        // (warp-uniform values, one elected lane: descriptors stay in uniform registers)
        const int nb = __shfl_sync(0xffffffffu, nblk, 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        if (nb > 0 && tc::elect_one()) {
            constexpr uint32_t id = tc::idesc_bf16_f32(PF_BM, PF_N);
            constexpr uint32_t HI = uint32_t(tc::DESC_SW128_KMAJOR >> 32), LO = uint32_t(tc::DESC_SW128_KMAJOR);
            const uint32_t r0 = (smem_u32(smem) >> 4) & 0x3fffu, q0 = (smem_u32(smem + L::Q_OFF) >> 4) & 0x3fffu;
            auto desc = [&](uint32_t at) { return (uint64_t(HI) << 32) | (LO | at); };
            bool ok = mbar_wait_bounded(qfull, 0, a.status);
            for (int i = 0; i < nb && ok; ++i) {
                // A wait for a phase that is two ahead would take the one before for it, one for a phase that is two
                // behind would not end. A stage of keys in a ring of three held the values of block i - 2 before, which
                // are waited for elsewhere: once they were read, the keys' phase is the next. In an even ring it held
                // keys.
                const int ki = 2 * i, s = ki % ST;
                if (ST == 3 && i >= 2) ok = mbar_wait_bounded(&pdone[i & 1], uint32_t((i >> 1) - 1) & 1u, a.status);
                ok = ok && mbar_wait_bounded(&full[s], uint32_t(ki / ST) & 1u, a.status);
                if (ok && i >= 2) ok = mbar_wait_bounded(&sfree[i & 1], uint32_t((i >> 1) - 1) & 1u, a.status);
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t da = r0 + uint32_t(s) * uint32_t(L::TILE >> 4);
#pragma unroll
                for (int p = 0; p < L::PANELS; ++p)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc::mma_bf16(tm + uint32_t((i & 1) * PF_N), desc(da + p * uint32_t(L::PANEL >> 4) + 2u * kk),
                                     desc(q0 + p * uint32_t(L::QPANEL >> 4) + 2u * kk), id, p > 0 || kk > 0);
                tc::mma_commit(&sfull[i & 1]);
                if (ki + ST < 2 * nb) tc::mma_commit(&empty[s]);    // (handed back only when it is filled again)
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- softmax
        const int key = threadIdx.x;                                 // row of a block (TMEM lane)
        const int cols = r.n_new * x.grp;                            // rows of q with a token
        const uint32_t live = (1u << cols) - 1u, head1 = (1u << x.grp) - 1u;   // (cols, grp <= 16)
        const uint32_t trow = tmem + (uint32_t(warp * 32) << 16);
        float* const red = reinterpret_cast<float*>(smem + L::RED_OFF);
        float m[PF_N], l[PF_N], p[PF_N];
#pragma unroll
        for (int n = 0; n < PF_N; ++n) m[n] = -INFINITY, l[n] = 0.f;
        bool ok = true;
        // the 128 threads' barrier, with their vote
        auto vote = [](bool v) -> bool {
            uint32_t any;
            __syncwarp();
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                         "barrier.cta.red.or.pred.aligned q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                         : "=r"(any) : "r"(uint32_t(v)) : "memory");
            return any != 0;
        };
        for (int i = 0; i < nblk; ++i) {
            const int j = (b0 + i) * PF_BM + key, s = j - r.n_old, vi = 2 * i + 1;
            uint32_t seen = j < r.n_keys ? live : 0u;
            if (s >= 0 && seen) {                                    // a new row
                if (!a.mask) {
                    seen &= ~((1u << s * x.grp) - 1u);               // (s < n_new)
                } else {
                    const uint8_t* col = a.mask + size_t(c) * a.S * a.S + s;
                    uint8_t v[PF_N];
#pragma unroll
                    for (int t = 0; t < PF_N; ++t) v[t] = col[size_t(min(t, r.n_new - 1)) * a.S];
                    seen = 0;
#pragma unroll
                    for (int t = 0; t < PF_N; ++t)
                        if (t < r.n_new && v[t]) seen |= head1 << t * x.grp;
                }
            }
            ok = ok && mbar_wait_bounded(&sfull[i & 1], uint32_t(i >> 1) & 1u, a.status);
            if (i >= 2) ok = ok && mbar_wait_bounded(&pdone[i & 1], uint32_t((i >> 1) - 1) & 1u, a.status);
            if (i + 1 == nblk && r.n_keys < (b0 + nblk) * PF_BM) {
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
                tc::tmem_ld16(trow + uint32_t((i & 1) * PF_N), sc);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sfree[i & 1]);
            }
            // P of the block against the maxima in use, to shared memory; the largest weight. (No maximum yet:
            // the weight of a key that is seen is infinite.)
            uint8_t* const pb = smem + L::P_OFF + (i & 1) * L::PBUF + key * 32;
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
                if (i > 0) {                                         // the products so far
                    ok = ok && mbar_wait_bounded(&pdone[(i - 1) & 1], uint32_t((i - 1) >> 1) & 1u, a.status);
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
                const int u = __shfl_sync(0xffffffffu, i, 0), nb = __shfl_sync(0xffffffffu, nblk, 0);
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
                            tc::mma_bf16(tm + OCOL, VD | (da + 128u * kk), PD | (db + 32u * kk), id, u > 0 || kk > 0);
                        tc::mma_commit(&pdone[u & 1]);
                        if (w + ST < 2 * nb) tc::mma_commit(&empty[sv]);
                    }
                }
                __syncwarp();
            }
        }
        // ---------------------------------------------------------------- end
        if (nblk > 0) {
            ok = ok && mbar_wait_bounded(&pdone[(nblk - 1) & 1], uint32_t((nblk - 1) >> 1) & 1u, a.status);
            ok = __all_sync(0xffffffffu, ok);
        }
        float v[PF_N];
#pragma unroll
        for (int n = 0; n < PF_N; ++n) v[n] = l[n];
        const float part = warp_columns(v, lane, [](float u, float w) { return u + w; });
        vote(false);                                                 // (red: the last maxima are read)
        if (lane < PF_N) red[warp * PF_N + lane] = part;
        const bool all_ok = !vote(!ok);
        float inv[PF_N];                                             // sums, then what O is scaled by
#pragma unroll
        for (int n = 0; n < PF_N; ++n)
            inv[n] = all_ok && nblk > 0 ? (red[n] + red[PF_N + n]) + (red[2 * PF_N + n] + red[3 * PF_N + n]) : 0.f;
        uint32_t o[PF_N];
        if (all_ok && nblk > 0) {
            tc::fence_after_sync();
            tc::tmem_ld16(trow + OCOL, o);
        }
        // row n of q: token n / grp, head n % grp; tree slots without a node get zeros, of ragged batches
        // only tokens are written
        const size_t o0 = size_t(r.q0) * a.Hq + size_t(g) * x.grp;
        auto row_of = [&](int n) -> size_t { return o0 + size_t(n / x.grp) * a.Hq + n % x.grp; };
        const int rows = a.q_start ? cols : x.rows;
        if (!CL && x.nchunk == 1) {
            if (key < rows) {                                        // (a row's sum: by its number among the threads)
                float lk = 0.f, mk = -INFINITY;
#pragma unroll
                for (int n = 0; n < PF_N; ++n)
                    if (n == key) lk = inv[n], mk = m[n];
                if (x.lse) x.lse[row_of(key)] = lk > 0.f ? (mk + log2f(lk)) * 0.6931471805599453f
                                                         : key < cols ? -INFINITY : 0.f;
            }
#pragma unroll
            for (int n = 0; n < PF_N; ++n)
                if (n < rows && key < D) {
                    const bool has = inv[n] > 0.f && n < cols;
                    const __nv_bfloat16 h = __float2bfloat16_rn(has ? __uint_as_float(o[n]) / inv[n] : 0.f);
                    reinterpret_cast<__nv_bfloat16*>(x.out)[row_of(n) * D + key] = h;
                }
        } else {
            float2* const ml = reinterpret_cast<float2*>(smem + L::ML_OFF);
            int* const places = reinterpret_cast<int*>(smem + L::PLACE_OFF);
            const size_t pr = (size_t(cg) * x.nchunk + chunk) * x.rows;
            if (key < PF_N) {
                float2 mine = make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int n = 0; n < PF_N; ++n)
                    if (n == key && inv[n] > 0.f && n < cols) mine = make_float2(m[n], inv[n]);
                if constexpr (CL) {
                    ml[key] = mine;
                    places[key] = key < cols ? int(row_of(key)) : key < rows ? -2 - int(row_of(key)) : -1;
                } else if (key < cols) {
                    x.part_ml[pr + key] = mine;
                }
            }
            float* const ob = reinterpret_cast<float*>(smem);
#pragma unroll
            for (int n = 0; n < PF_N; ++n)
                if (n < cols && inv[n] > 0.f && key < D) {
                    if constexpr (CL) ob[n * L::PITCH + key] = __uint_as_float(o[n]);
                    else x.part_o[(pr + n) * D + key] = __uint_as_float(o[n]);
                }
            if constexpr (CL) {
                __syncwarp();
                cluster_sync();
                paged_merge<D>(x, ob, L::PITCH, ml, places, PF_N, chunk, warp, 4);
                __syncwarp();
                cluster_sync();                                      // (no CTA leaves while its rows are read)
            }
        }
    }
    if constexpr (CL)
        if (warp >= 4) {
            __syncwarp();
            cluster_sync();
            cluster_sync();
        }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 5) tc::tmem_dealloc(tmem, TCOLS);
}

template <int D, int ST, bool CL>
static int launch_few_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PgArgs& x,
                        cudaStream_t stream) {
    auto kern = paged_few_kernel<D, ST, CL>;
    const size_t smem = PfSmem<D, ST>::TOTAL;
    static std::atomic<uint64_t> raised{0};
    if (!raise_smem(kern, int(smem), raised)) return DARTREE_ECUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(x.nchunk) * unsigned(x.a.C) * x.a.Hkv);
    cfg.blockDim = dim3(PF_NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2] = {pdl_attribute()};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(x.nchunk);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CL ? 2 : 1;
    KTimer kt_(KID_PAGED_ATTN, stream);
    return cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, x) == cudaSuccess ? DARTREE_OK : DARTREE_ECUDA;
}

// Alone on its SM a CTA has room for three blocks' keys and values (heads of 64: six), else two share the SM with half of that.
int launch_paged_few(const PgArgs& x, bool cluster, bool alone, const CUtensorMap& tq, const CUtensorMap& tk,
                     const CUtensorMap& tv, cudaStream_t stream) {
    if (x.a.D == 64)
        return cluster ? launch_few_t<64, 12, true>(tq, tk, tv, x, stream)
               : alone ? launch_few_t<64, 12, false>(tq, tk, tv, x, stream)
                       : launch_few_t<64, 6, false>(tq, tk, tv, x, stream);
    return cluster ? launch_few_t<128, 6, true>(tq, tk, tv, x, stream)
           : alone ? launch_few_t<128, 6, false>(tq, tk, tv, x, stream)
                   : launch_few_t<128, 3, false>(tq, tk, tv, x, stream);
}

}  // namespace dartree
