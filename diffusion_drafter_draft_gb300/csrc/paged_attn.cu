// Attention of new tokens over the paged key/value cache.
//
//   out_i = sum_j softmax_j(scale <q_i, k_j>) v_j,   lse_i = log sum_j exp(scale <q_i, k_j>)
//
// over the cached rows j < n_old and the new rows up to token i's own (or those a tree
// mask marks). The query heads of a key/value head are stacked: a tile holds TT = 128 / grp
// tokens, row (token, head) at token * grp + head, so that one TMA box brings it and a
// tile's rows end at nearly the same key. One pass over 128-key blocks with the running
// maximum and sum of the softmax.
//
// CTA = (chunk of a tile's key blocks, NT tiles, (request, key/value head)):
//   warp 0      producer: a block's keys, then its values, page by page (TMA, 128-byte
//               swizzle) through a ring of ST stages; a row past the request's last is
//               fetched from beyond the pool, which TMA fills with zeros
//   warp 1      issues S = Q K^T (both operands in shared memory) and O += P V (P in
//               tensor memory over S's columns, V as an MN-major operand straight from
//               its pages: nothing is transposed)
//   warp 2      passes on the landing of a group's keys and values
//   warps 4..   softmax, one thread per row: the row's 128 scores in registers, P in bf16
//               back to tensor memory, weighted against the maximum of the blocks before:
//               bf16 and fp32 carry 2^14 as well as 1, so only a half block whose weights
//               add up to more (and the first, and masked ones) takes its own and rescales O
// P is rounded to bf16, the type of the values it is multiplied with (a weight is off by 2^-8 of itself at
// most; maxima, sums and O stay fp32, the sums add the weights before they are rounded). The remainders as a
// second operand would double the work of P V, which bounds prompts, for an output that is bf16 itself:
// against 64 bits it is 2.3e-3 off in norm, the exact one rounded 1.7e-3.
// With NT = 2 the tensor cores work on one tile while the other tile's softmax runs.
// Rows of a partly used page may hold anything: the last block's value rows past the end
// are zeroed in shared memory (0 * NaN is NaN), its scores are masked.
//
// Up to eight chunks of a tile may be a cluster (CL) and merge through shared memory; else
// their partial rows go through memory to a second launch.
//
// Long chunks are bound by the tensor cores (8192 tokens over 8192 rows, 32/8 heads of 128:
// 1.0 ms, 1.66 PFLOP/s), trees by the chain of a block (scores, weights, product: ~1.6 us) and the
// merge (four trees of 65 slots over 1024-2048 rows: 24.7 us). At most 16 rows of a key/value head
// (single tokens) have a kernel of their own, paged_few.cu.
// Every mbarrier wait is bounded; one that runs out records DARTREE_ETIMEOUT.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "paged_attn.cuh"
#include "tc.cuh"

namespace dartree {

constexpr int PG_BM = 128;            // rows of a tile
constexpr int PG_BN = 128;            // keys of a block

template <int D, int NT, int ST>
struct PgSmem {
    static constexpr int PANELS = D / 64;                       // 64 values of D per 128-byte row
    static constexpr size_t PANEL = size_t(PG_BN) * 128;
    static constexpr size_t TILE = PANELS * PANEL;              // a query tile, or a block's keys or values
    static constexpr size_t RING_OFF = NT * TILE;
    static constexpr size_t BAR_OFF = RING_OFF + ST * TILE;
    // qfull, vclean, full[ST], empty[ST], sfull[NT], pfull[NT], phalf[NT], pdone[NT], ofull[NT]
    static constexpr size_t SLOT_OFF = BAR_OFF + 8 * (2 + 2 * ST + 5 * NT);
    static constexpr size_t TOTAL = SLOT_OFF + 16 + 1024;       // (+ alignment of the base to 1024)
    static_assert(TOTAL <= 227 * 1024, "tiles and ring fit in shared memory");
    // merge of a cluster's chunks, over tiles and ring: O of each row in fp32 (a row's 16 extra bytes
    // keep the rows of a warp in different banks), (maximum, sum), its place
    static constexpr int PITCH = D + 4;
    static constexpr size_t ML_OFF = size_t(NT) * PG_BM * PITCH * 4;
    static constexpr size_t ROW_OFF = ML_OFF + NT * PG_BM * 8;  // int [NT][128]: a row's place in the output
    static_assert(ROW_OFF + NT * PG_BM * 4 <= BAR_OFF, "merge fits in the tiles' place");
};

struct PgPlan {
    int tt, tiles, nt, nchunk, rows;  // tokens per tile, tiles, tiles per CTA, chunks, rows kept per partial tile
    bool cluster, few, alone;         // the chunks merge through shared memory; at most 16 rows; a CTA per SM and tile
    size_t part_ml, total;            // workspace (partials): offset of the maxima and sums, bytes
    double us;                        // expected time
    int64_t most_rows;                // partial rows of any plan for at most these sizes, their bytes
    size_t most;
};

// SH: a call with shared prefixes. CTAs below x.s.ctas take runs of a group's tokens over the rows that the group
// shares (all seen by all), the others a request's tokens over its own rows, from row `kb` on.
template <int D, int NT, int ST, bool CL, bool SH>
__global__ void __launch_bounds__(128 + 128 * NT, NT == 1 ? 2 : 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PgArgs x) {
    using L = PgSmem<D, NT, ST>;
    constexpr uint32_t OCOL = NT * PG_BN;                    // TMEM: S/P of tile t at 128 t, O at OCOL + D t
    constexpr uint32_t TCOLS = NT == 2 ? 512 : 256;
    const PagedArgs& a = x.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* qfull = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
    uint64_t* vclean = qfull + 1;     // value rows past the end zeroed (last block)
    uint64_t* full = qfull + 2;       // [ST] stage landed
    uint64_t* empty = full + ST;      // [ST] the MMAs that read it are done
    uint64_t* sfull = empty + ST;     // [NT] scores written (and every earlier MMA done)
    uint64_t* phalf = sfull + NT;     // [NT] P of the block's first 64 keys written, what the group reads landed
    uint64_t* pfull = phalf + NT;     // [NT] P of the others written
    uint64_t* pdone = pfull + NT;     // [NT] the product of the first 64 keys done
    uint64_t* ofull = pdone + NT;     // [NT] the last product with V done
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + L::SLOT_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(qfull, 1);
        mbar_init(vclean, 1);
        for (int s = 0; s < ST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int t = 0; t < NT; ++t) {
            mbar_init(&sfull[t], 1);
            mbar_init(&phalf[t], 5);  // four softmax warps and warp 2
            mbar_init(&pfull[t], 4);
            mbar_init(&pdone[t], 1);
            mbar_init(&ofull[t], 1);
        }
        fence_mbar_init();
    }
    if (warp == 1) tc::tmem_alloc(slot, TCOLS);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *slot;
    // (SH: the launch behind may start before this one ends and does not wait itself until its merge, so what
    // came before has to be done by then)
    if (!SH) griddep_launch_dependents();
    griddep_wait();
    if (SH) griddep_launch_dependents();

    // the last tiles (the most keys of a causal batch) first, of all heads or (x.inner) head by head
    const bool whole = SH && blockIdx.x < x.s.ctas;                       // (over shared rows)
    const int nchunk = whole ? x.s.np : x.nchunk;
    const unsigned cta = SH && !whole ? blockIdx.x - x.s.ctas : blockIdx.x;
    const int ntile = (x.tiles + NT - 1) / NT;
    const int chunk = int(cta % nchunk);
    const unsigned rest = cta / nchunk, heads = a.C * a.Hkv, in = x.inner ? ntile : heads;
    const int high = int(rest / in), low = int(rest - high * in);
    const int cg = x.inner ? high : low, tp = ntile - 1 - (x.inner ? low : high);
    int c = cg / a.Hkv, g = cg - c * a.Hkv;
    int t0 = tp * NT * x.tt;                                              // first token
    int kb = 0;                                                           // first key
    bool bad;
    PagedRequest r;
    if (whole) {
        const unsigned unit = rest % x.s.units;
        g = int(rest / x.s.units);
        PgUnit u{0, 0, 0, 0, 0};
        paged_shared_unit(x, unit, NT * x.tt, u, bad);
        bad = bad && unit == 0;
        c = u.c, t0 = u.t0;
        r = PagedRequest{u.q0, u.n, u.keys, u.keys};
    } else {
        r = paged_request(a, c, bad);
        if (SH) kb = paged_shared_rows(x, c, r.n_old, bad);
        bad = bad && tp == 0;
    }
    if (bad && threadIdx.x == 0 && g == 0) set_status(a.status, DARTREE_EINTERNAL);
    const uint8_t* const mask = whole ? nullptr : a.mask;
    const int live = min(max(r.n_new - t0, 0), NT * x.tt);                // tokens
    const int nact = NT == 1 ? (live > 0) : (live + x.tt - 1) / x.tt;     // tiles with a token
    const int end = mask || whole ? r.n_keys : min(r.n_keys, r.n_old + t0 + live);
    const int blocks = live > 0 ? (max(end - kb, 0) + PG_BN - 1) / PG_BN : 0;
    const int per = (blocks + nchunk - 1) / nchunk;
    const int b0 = chunk * per, nblk = max(min(blocks, b0 + per) - b0, 0);

    // the softmax holds a row of scores in registers: its warpgroups take over registers that the
    // first one was launched with (NT = 2: 384 x 168 >= 128 x 80 + 256 x 208; NT = 1: 256 x 128 =
    // 128 x 56 + 128 x 200)
    if (warp < 4) {
    if (NT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
        // ---------------------------------------------------------------- producer
        if (nblk > 0) {
            const int pr = min(a.page, PG_BN), sub = PG_BN / pr;          // rows and copies per panel of a block
            if (lane == 0) {
                mbar_arrive_expect_tx(qfull, uint32_t(nact * L::PANELS * x.tt * x.grp * 128));
                for (int t = 0; t < nact; ++t)
                    for (int p = 0; p < L::PANELS; ++p)
                        tc::tma_load_3d(smem + t * L::TILE + p * L::PANEL, &tmQ, 64 * p, g * x.grp,
                                        r.q0 + t0 + t * x.tt, qfull);
            }
            const int su = lane % sub, pn = lane / sub;                   // this lane's page and panel
            const bool mine = sub <= 32 && pn < L::PANELS;
            const int32_t* table = a.table + size_t(c) * a.max_pages;
            // this lane's table entry of block b (looked up two blocks ahead, checked when it is used), and
            // the page to fetch: n_pages, beyond the pool and so all zeros, past the end and for no page
            auto entry_of = [&](int b) -> int {
                const int j = kb + b * PG_BN + su * pr;
                return mine && j < r.n_keys ? table[j >> a.log2_page] : a.n_pages;
            };
            auto page_of = [&](int e, int b) -> int {
                if (unsigned(e) < unsigned(a.n_pages)) return e;
                if (mine && kb + b * PG_BN + su * pr < r.n_keys) set_status(a.status, DARTREE_EINTERNAL);
                return a.n_pages;
            };
            int e0 = entry_of(b0), e1 = entry_of(b0 + 1), issued = 0;
            for (int i = 0; i < nblk; ++i) {
                const int pg = page_of(e0, b0 + i);
                e0 = e1;
                e1 = entry_of(b0 + i + 2);
                bool ok = true;
                for (int kv = 0; kv < 2 && ok; ++kv) {
                    const int idx = 2 * i + kv, s = idx % ST;
                    if (lane == 0 && idx >= ST)
                        ok = mbar_wait_bounded(&empty[s], uint32_t((idx / ST) & 1) ^ 1u, a.status);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&full[s], uint32_t(L::TILE));
                    __syncwarp();
                    if (mine)
                        tc::tma_load_4d(smem + L::RING_OFF + s * L::TILE + pn * L::PANEL + size_t(su) * pr * 128,
                                        kv ? &tmV : &tmK, 64 * pn, (kb + (b0 + i) * PG_BN + su * pr) & (a.page - 1), g, pg,
                                        &full[s]);
                    issued = idx + 1;
                }
                if (!ok) break;
            }
            // the last block's value rows past the end are zeroed once they have landed
            const int have = r.n_keys - kb - (b0 + nblk - 1) * PG_BN, vl = 2 * nblk - 1;
            if (have < PG_BN && issued > vl) {
                bool ok = true;
                if (lane == 0) ok = mbar_wait_bounded(&full[vl % ST], uint32_t(vl / ST) & 1u, a.status);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (ok) {
                    uint8_t* vb = smem + L::RING_OFF + (vl % ST) * L::TILE + size_t(have) * 128;
                    for (int e = lane; e < (PG_BN - have) * 8; e += 32)
#pragma unroll
                        for (int p = 0; p < L::PANELS; ++p)
                            reinterpret_cast<uint4*>(vb + p * L::PANEL)[e] = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(vclean);
                }
            }
            // copies issued and not yet seen complete land before the CTA can exit
            if (lane == 0) {
                mbar_wait_bounded(qfull, 0, a.status);
                for (int q = max(issued - ST, 0); q < issued; ++q)
                    mbar_wait_bounded(&full[q % ST], uint32_t(q / ST) & 1u, a.status);
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issue
        // The tensor cores take MMAs about as fast as one thread issues them, and a barrier
        // test costs that thread a few hundred cycles beside two softmax warps: so a group
        // (O += P V of a tile in two halves of the keys, the first while the other's weights
        // are formed, then the tile's next S) waits for the two halves of P alone; the first
        // also counts the landing of what the group reads (warp 2), and the next group's is
        // tested while this group's last MMAs are issued.
        // (warp-uniform values, one elected lane: descriptors stay in uniform registers)
        const int nb = __shfl_sync(0xffffffffu, nblk, 0), na = __shfl_sync(0xffffffffu, nact, 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        if (nb > 0 && tc::elect_one()) {
            constexpr uint32_t idS = tc::idesc_bf16_f32(PG_BM, PG_BN);
            constexpr uint32_t idO = tc::idesc_bf16_f32(PG_BM, D) | tc::IDESC_B_MNMAJOR;
            constexpr uint32_t PSTEP = L::PANEL >> 4, TSTEP = L::TILE >> 4;  // descriptor steps (low word)
            // (14 bits: in a cluster the address carries the rank of the CTA above them)
            const uint32_t q0 = (smem_u32(smem) >> 4) & 0x3fffu, r0 = (smem_u32(smem + L::RING_OFF) >> 4) & 0x3fffu;
            constexpr uint32_t KHI = uint32_t(tc::DESC_SW128_KMAJOR >> 32), KLO = uint32_t(tc::DESC_SW128_KMAJOR);
            constexpr uint64_t VD = tc::desc_sw128_mnmajor_base(uint32_t(L::PANEL));
            auto kdesc = [&](uint32_t at) { return (uint64_t(KHI) << 32) | (KLO | at); };
            auto score = [&](int t, int s, int p) {   // 64 values of D
                const uint32_t da = q0 + t * TSTEP + p * PSTEP, db = r0 + s * TSTEP + p * PSTEP;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc::mma_bf16(tm + uint32_t(t * PG_BN), kdesc(da + 2u * kk), kdesc(db + 2u * kk), idS,
                                 p > 0 || kk > 0);
            };
            bool ok = mbar_wait_bounded(qfull, 0, a.status) && mbar_wait_bounded(&full[0], 0, a.status);
            if (ok) {
                tc::fence_after_sync();
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (t < na) {
#pragma unroll
                        for (int p = 0; p < L::PANELS; ++p) score(t, 0, p);
                        tc::mma_commit(&sfull[t]);
                    }
                if (ST < 2 * nb) tc::mma_commit(&empty[0]);
            }
            int vs = 1 % ST, ks = 2 % ST;             // stages of block i's values and block i + 1's keys
            bool ready = false;
            for (int i = 0; i < nb && ok; ++i) {
                const bool last = i + 1 == nb;
                // (a stage is handed back only when it is filled again)
                const bool back_v = 2 * i + 1 + ST < 2 * nb, back_k = 2 * i + 2 + ST < 2 * nb;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (t >= na) break;
                    const uint32_t db = r0 + vs * TSTEP;
                    auto product = [&](int h) {       // 64 keys
#pragma unroll
                        for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
                            tc::mma_bf16_ts(tm + OCOL + uint32_t(t * D), tm + uint32_t(t * PG_BN + 8 * kk),
                                            (VD & ~0xffffffffull) | (uint32_t(VD) | (db + 128u * kk)), idO,
                                            i > 0 || kk > 0);
                    };
                    if (!ready) ok = mbar_wait_bounded(&phalf[t], uint32_t(i) & 1u, a.status);
                    if (!ok) break;
                    tc::fence_after_sync();
                    product(0);
                    tc::mma_commit(&pdone[t]);
                    ok = mbar_wait_bounded(&pfull[t], uint32_t(i) & 1u, a.status);
                    if (!ok) break;
                    tc::fence_after_sync();
                    product(1);
                    const bool end_v = t == na - 1;
                    if (end_v && back_v) tc::mma_commit(&empty[vs]);
                    if (last) {
                        ready = false;
                        tc::mma_commit(&ofull[t]);
                    } else {
#pragma unroll
                        for (int p = 0; p + 1 < L::PANELS; ++p) score(t, ks, p);
                        ready = mbar_try_wait(end_v ? &phalf[0] : &phalf[NT - 1], uint32_t(end_v ? i + 1 : i) & 1u);
                        score(t, ks, L::PANELS - 1);
                        tc::mma_commit(&sfull[t]);
                        if (end_v && back_k) tc::mma_commit(&empty[ks]);
                    }
                }
                vs += 2;
                if (vs >= ST) vs -= ST;
                ks += 2;
                if (ks >= ST) ks -= ST;
            }
        }
    } else if (warp == 2) {
        // ---------------------------------------------------------------- landing of the groups' operands
        if (nblk > 0 && lane == 0) {
            // (every phase of a stage is waited for, block 0's keys' too: a wait two phases ahead would
            // take the phase before for its own)
            bool ok = mbar_wait_bounded(&full[0], 0, a.status);
            for (int i = 0; i < nblk && ok; ++i) {
                const int vi = 2 * i + 1, ki = 2 * i + 2;
                const bool last = i + 1 == nblk;
                ok = mbar_wait_bounded(&full[vi % ST], uint32_t(vi / ST) & 1u, a.status) &&
                     (last || mbar_wait_bounded(&full[ki % ST], uint32_t(ki / ST) & 1u, a.status));
                if (ok && last && r.n_keys < kb + (b0 + nblk) * PG_BN) ok = mbar_wait_bounded(vclean, 0, a.status);
                for (int t = 0; t < nact && ok; ++t) {
                    if (i > 0) ok = mbar_wait_bounded(&phalf[t], uint32_t(i - 1) & 1u, a.status);
                    if (ok) mbar_arrive(&phalf[t]);
                }
            }
        }
    }
    if constexpr (CL) {                            // (the softmax warps merge between these)
        __syncwarp();
        cluster_sync();
        cluster_sync();
    }
    } else {
        // ---------------------------------------------------------------- softmax
        if (NT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int t = (warp - 4) >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;                     // row of the tile (TMEM lane)
        const int ti = row / x.grp, hg = row - ti * x.grp;
        const int i_tok = t0 + t * x.tt + ti;                    // token of the request
        const bool slot_ok = ti < x.tt && (whole || i_tok < a.S);
        const bool real = slot_ok && i_tok < r.n_new;
        const int limit = !real ? 0 : mask || whole ? r.n_keys : min(r.n_keys, r.n_old + i_tok + 1);
        const bool work = __any_sync(0xffffffffu, real);         // a warp without a token forms no weights
        const uint32_t trow = tmem + (uint32_t(quarter * 32) << 16);
        const uint32_t scol = trow + uint32_t(t * PG_BN), ocol = trow + OCOL + uint32_t(t * D);
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        // the tree's mask for the 128 keys from `key` on: lane q reads slot q of a 32-key word of a token
        // of this warp's, and the vote is the word (eight tokens' four words are loaded together)
        auto tree_bits = [&](int key, uint32_t (&bits)[4]) {
            const int tok0 = (quarter * 32) / x.grp, tok1 = (quarter * 32 + 31) / x.grp;
            const int sl = key + lane - r.n_old;
#pragma unroll
            for (int w = 0; w < 4; ++w) bits[w] = 0;
            // (every load is in range by its clamped indices and needs no other's outcome: a tree of 64 slots
            // of one head 15.2 us, 25.0 with loads by need)
            for (int q0 = tok0; q0 <= tok1; q0 += 8) {
                uint8_t v[8][4];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int i_q = min(t0 + t * x.tt + q0 + u, r.n_new - 1);
                    const uint8_t* mrow = mask + (size_t(c) * a.S + i_q) * a.S;
#pragma unroll
                    for (int w = 0; w < 4; ++w) v[u][w] = mrow[min(max(sl + 32 * w, 0), r.n_new - 1)];
                }
#pragma unroll
                for (int u = 0; u < 8; ++u)
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int j = sl + 32 * w;
                        const uint32_t word = __ballot_sync(0xffffffffu, j < 0 || (j < r.n_new && v[u][w] != 0));
                        if (q0 + u == ti) bits[w] = word;
                    }
            }
        };
        if (t < nact) {
            for (int i = 0; i < nblk; ++i) {
                const int key0 = kb + (b0 + i) * PG_BN;
                const bool tree = mask && key0 + PG_BN > r.n_old;
                uint32_t bits[4];
                if (tree && work) tree_bits(key0, bits);
                ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(&sfull[t], uint32_t(i) & 1u, a.status));
                if (ok && work) {
                    tc::fence_after_sync();
                    uint32_t s[128];
                    tc::tmem_ld128(scol, s);
                    const int lim = limit - key0;                // columns from `lim` on are hidden
                    const bool cut = tree || __any_sync(0xffffffffu, real && lim < PG_BN);
                    // 32 scores weighted against the maximum in use: P to tensor memory over the scores;
                    // sums of a half
                    const uint64_t sl = pair(x.sl2, x.sl2);
                    uint64_t ls[4];
                    auto weigh = [&](int w, uint64_t off) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float y0, y1;
                            unpair(fma2(pair(s[32 * w + e], s[32 * w + e + 1]), sl, off), y0, y1);
                            const float p0 = ex2(y0), p1 = ex2(y1);
                            const bool first = w % 2 == 0 && e < 8;
                            ls[(e >> 1) & 3] = first ? pair(p0, p1) : add2(ls[(e >> 1) & 3], pair(p0, p1));
                            pk[e / 2] = pack2(p0, p1);
                        }
                        tc::tmem_st16_async(scol + 16u * w, pk);
                    };
                    auto weigh_half = [&](int h) -> float {          // 64 keys
                        const float ms = m > -INFINITY ? -m : 0.f;   // (a row that has seen nothing: 2^-inf = 0)
                        const uint64_t off = pair(ms, ms);
                        weigh(2 * h, off);
                        weigh(2 * h + 1, off);
                        float s0, s1;
                        unpair(add2(add2(ls[0], ls[1]), add2(ls[2], ls[3])), s0, s1);
                        return s0 + s1;
                    };
                    auto hand_over = [&](uint64_t* bar) {
                        tc::tmem_wait_st();
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar);
                    };
                    // whether a half's weights are too large, in any row (or there is no maximum yet)
                    auto too_large = [&](float v) -> bool {
                        return __any_sync(0xffffffffu, real && !(v <= PG_MOST && m > -INFINITY));
                    };
                    // takes the maximum of the scores from `e0` on and rescales what was added up so far
                    auto own_maximum = [&](int e0) {
                        float p[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int e = 0; e < 128; e += 2)
                            if (e >= e0)
                                p[(e >> 1) & 3] =
                                    max3(p[(e >> 1) & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                        const float mx = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])) * x.sl2;   // (sl2 > 0: -inf stays)
                        const bool grow = real && mx > m, resc = grow && m > -INFINITY;
                        if (__any_sync(0xffffffffu, resc)) {
                            const float f = resc ? ex2(m - mx) : 1.0f;
#pragma unroll 1
                            for (int c0 = 0; c0 < D; c0 += 32) {
                                uint32_t o[32];
                                tc::tmem_ld32(ocol + uint32_t(c0), o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tc::tmem_st32(ocol + uint32_t(c0), o);
                            }
                            l *= f;
                        }
                        if (grow) m = mx;
                    };
                    bool first = false;                          // the first half is handed over
                    if (i > 0 && !cut) {
                        const float sum = weigh_half(0);
                        if (!too_large(sum)) {
                            l += sum;
                            hand_over(&phalf[t]);
                            first = true;
                        }
                    } else if (cut) {
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t seen = tree ? bits[w] : 0xffffffffu;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((seen >> e) & 1u) || 32 * w + e >= lim) s[32 * w + e] = 0xff800000u;  // -inf
                        }
                    }
                    if (!first) {                                // O's products up to block i - 1 are done
                        own_maximum(0);
                        l += weigh_half(0);
                        hand_over(&phalf[t]);
                    }
                    float sum = weigh_half(1);
                    if (first && too_large(sum)) {               // O's product of the first half has to be, too
                        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&pdone[t], uint32_t(i) & 1u, a.status));
                        tc::fence_after_sync();
                        own_maximum(64);
                        sum = weigh_half(1);
                    }
                    l += sum;
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                } else if (ok) {
                    if (lane == 0) mbar_arrive(&phalf[t]);
                }
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(&pfull[t]);
            }
            if (nblk > 0) {
                ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(&ofull[t], 0, a.status));
                if (ok) tc::fence_after_sync();
            }
        }
        const bool has = ok && t < nact && nblk > 0 && real && l > 0.f;
        const bool load = ok && t < nact && nblk > 0 && work;    // (TMEM loads are warp-wide)
        const size_t orow = (size_t(r.q0) + i_tok) * a.Hq + size_t(g) * x.grp + hg;
        if (!CL && !SH && x.nchunk == 1) {
            // tree slots without a node get zeros; rows of ragged batches only their own tokens
            const bool write = real || (slot_ok && !a.q_start);
            const float inv = has ? 1.0f / l : 0.f;
            uint4* dst = reinterpret_cast<uint4*>(x.out + orow * D);
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t o[32];
                __syncwarp();
                if (load) tc::tmem_ld32(ocol + uint32_t(c0), o);
                if (write)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t pk[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            pk[e] = has ? pack2(__uint_as_float(o[8 * q + 2 * e]) * inv,
                                                __uint_as_float(o[8 * q + 2 * e + 1]) * inv)
                                        : 0u;
                        dst[c0 / 8 + q] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
            }
            if (x.lse && write) x.lse[orow] = has ? (m + log2f(l)) * 0.6931471805599453f : real ? -INFINITY : 0.f;
        } else if constexpr (CL) {
            // the chunks of a tile are a cluster: every CTA puts its rows' O, maximum and sum into its
            // shared memory and merges every nchunk-th row from all of them
            float* const ob = reinterpret_cast<float*>(smem);
            float2* const ml = reinterpret_cast<float2*>(smem + L::ML_OFF);
            // (over the tiles' place: once the last MMA of the CTA is done, the other tile's too)
            if (nblk > 0) mbar_wait_bounded(&ofull[nact - 1], 0, a.status);
            __syncwarp();
            const int rr = t * PG_BM + row;
            int* const places = reinterpret_cast<int*>(smem + L::ROW_OFF);
            ml[rr] = has ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
            // (token * heads + head: below 2^31; -2 - place: a slot without a node; -1: no row)
            places[rr] = real ? int(orow) : slot_ok && !a.q_start ? -2 - int(orow) : -1;
            if (load)
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    __syncwarp();
                    tc::tmem_ld32(ocol + uint32_t(c0), o);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        reinterpret_cast<uint4*>(ob + rr * L::PITCH + c0)[q] =
                            make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                }
            __syncwarp();
            cluster_sync();
            paged_merge<D>(x, ob, L::PITCH, ml, places, NT * PG_BM, chunk, warp - 4, 4 * NT);
            __syncwarp();
            cluster_sync();                                      // (no CTA leaves while its rows are read)
        } else {
            const size_t pr = SH ? size_t(whole ? chunk : x.s.np + chunk) * (size_t(a.T) * a.Hq) + orow
                                 : ((size_t(cg) * x.tiles + tp * NT + t) * x.nchunk + chunk) * x.rows + row;
            if (real) x.part_ml[pr] = has ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
            float4* dst = reinterpret_cast<float4*>(x.part_o + pr * D);
            if (load)
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    __syncwarp();
                    tc::tmem_ld32(ocol + uint32_t(c0), o);
                    if (has)
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            dst[c0 / 4 + q] =
                                make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]),
                                            __uint_as_float(o[4 * q + 2]), __uint_as_float(o[4 * q + 3]));
                }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tmem, TCOLS);
}

// ----------------------------------------------------------------------------- combine
//
// Chunks that are no cluster. One warp per (request, token, query head): the chunks' (max, sum) pairs by the lanes in
// parallel, then their rows of O eight at a time.

// SH: the chunks of the shared rows (a request without a group has none), then those of its own.
template <int D, bool SH>
__global__ void __launch_bounds__(256) paged_combine_kernel(const __grid_constant__ PgArgs x) {
    constexpr int V = D / 32;
    const PagedArgs& a = x.a;
    const int lane = threadIdx.x & 31;
    const size_t id = size_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    griddep_launch_dependents();
    griddep_wait();
    if (id >= size_t(a.C) * a.S * a.Hq) return;
    const int h = int(id % a.Hq), i = int(id / a.Hq % a.S), c = int(id / a.Hq / a.S);
    const PagedRequest r = paged_request(a, c);
    const bool real = i < r.n_new;
    if (!real && a.q_start) return;
    const size_t orow = (size_t(r.q0) + i) * a.Hq + h;
    const int g = h / x.grp, tile = i / x.tt, row = (i - tile * x.tt) * x.grp + (h - g * x.grp);
    // (chunk k of this row lies at p0 + k * step)
    int first = 0, n = x.nchunk;
    size_t step = x.rows, p0 = ((size_t(c) * a.Hkv + g) * x.tiles + tile) * x.nchunk * size_t(x.rows) + row;
    if (SH) {
        step = size_t(a.T) * a.Hq, p0 = orow;
        first = paged_in_group(x, c) ? 0 : x.s.np;
        n = x.s.np + x.nchunk;
    }
    float mx = -INFINITY;
    if (real)
        for (int k = first + lane; k < n; k += 32) {
            const float2 ml = x.part_ml[p0 + size_t(k) * step];
            if (ml.y > 0.f) mx = fmaxf(mx, ml.x);
        }
    mx = warp_max(mx);
    float acc[V], sum = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    if (mx > -INFINITY)
        for (int k0 = first; k0 < n; k0 += 32) {
            float f = 0.f;  // lane t: chunk k0 + t's factor 2^(m - mx)
            if (k0 + lane < n) {
                const float2 ml = x.part_ml[p0 + size_t(k0 + lane) * step];
                if (ml.y > 0.f) {
                    f = ex2(ml.x - mx);
                    sum += f * ml.y;
                }
            }
            const int nk = min(32, n - k0);
            for (int u0 = 0; u0 < nk; u0 += 8) {
                float o[8][V];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float fu = __shfl_sync(0xffffffffu, f, (u0 + u) & 31);
                    const float* src = x.part_o + (p0 + size_t(k0 + u0 + u) * step) * D + lane * V;
#pragma unroll
                    for (int e = 0; e < V; ++e) o[u][e] = 0.f;
                    if (u0 + u < nk && fu > 0.f) {
                        if (V == 4) {
                            const float4 y = *reinterpret_cast<const float4*>(src);
                            o[u][0] = y.x, o[u][1] = y.y, o[u][V - 2] = y.z, o[u][V - 1] = y.w;
                        } else {
                            const float2 y = *reinterpret_cast<const float2*>(src);
                            o[u][0] = y.x, o[u][1] = y.y;
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float fu = __shfl_sync(0xffffffffu, f, (u0 + u) & 31);
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] = fmaf(fu, o[u][e], acc[e]);
                }
            }
        }
    sum = warp_sum(sum);
    const float inv = sum > 0.f ? 1.0f / sum : 0.f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(x.out + orow * D) + lane * (V / 2);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) dst[e] = pack2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if (x.lse && lane == 0)
        x.lse[orow] = sum > 0.f ? (mx + log2f(sum)) * 0.6931471805599453f : real ? -INFINITY : 0.f;
}

// ----------------------------------------------------------------------------- host

// Tiles per CTA and chunks of a tile's key blocks: the least time, in us, fitted to sweeps of
// 18 shapes with caches that were not in the L2. A CTA's start and end, then a block: two
// tiles 6 and 1.7 (heads of 128; of 64, 6 and 1.45, which two CTAs of one tile, 5 and 1.4,
// always beat); one tile beside another CTA, with a ring of one block, 5 and 2.5; alone on
// its SM with two and a half blocks in flight 4 and 1.55 (both less where many tiles read
// the same keys). Merging in a cluster, where all CTAs run at once, 2 and 3 for a whole
// tile; through memory 6 and the partial results' bytes at 4 TB/s.
// Against the best of all ways: one tree of 65 slots over 2048 rows 18.9 -> 13.9 us with
// CTAs alone, 16 over 4096 rows 120 us with two tiles a CTA (169 with one).
// Chunks that meet in memory are for tables of PG_PART_BLOCKS blocks on (their launch costs more than a
// few blocks) and keep within PG_PART_BYTES of partial rows, part_rows of them at most: so a workspace's
// size grows with batch, tokens and table, and one that serves a batch serves every smaller one. (Tables
// of up to 16384 rows are planned as without these limits; of random batches over up to 131072 rows 3 in
// 100 lose 1.4 % by the same times, 7 % at most.)
constexpr int PG_PART_BLOCKS = 8;
constexpr int64_t PG_PART_BYTES = int64_t(128) << 20;

// Most chunks of `ctas` tiles that are worth their merge: enough to fill the SMs, or 16.
static int64_t most_chunks(int64_t ctas, int64_t slots) { return slots / ctas > 16 ? slots / ctas : 16; }

// Upper bound of the partial rows (chunks times rows) of any plan for these tiles: grows with each argument.
// (`tiles` of all heads; two tiles a CTA, on half the slots, have the same bound.)
static int64_t part_rows(int64_t tiles, int64_t blocks, int64_t rows, int D) {
    if (tiles == 0 || blocks < PG_PART_BLOCKS) return 0;
    const int64_t fill = 2 * int64_t(num_sms()), ways = 16 * tiles > fill ? 16 * tiles : fill;
    const int64_t all = (ways < tiles * blocks ? ways : tiles * blocks) * rows, cap = PG_PART_BYTES / (4 * D);
    return all < cap ? all : cap;
}

// `keys`: rows that a request may have, 0: what its row of the table holds.
static PgPlan paged_plan(const PagedArgs& a, int64_t keys = 0) {
    PgPlan p{};
    const int grp = a.Hq / a.Hkv;
    p.tt = PG_BM / grp;
    p.tiles = (a.S + p.tt - 1) / p.tt;
    p.rows = p.tiles > 1 ? PG_BM : a.S * grp;
    const int64_t heads = int64_t(a.C) * a.Hkv;
    const int64_t blocks = ((keys ? keys : int64_t(a.max_pages) << a.log2_page) + PG_BN - 1) / PG_BN;
    p.nt = 1, p.nchunk = 1;
    double best = 1e300;
    p.most_rows = part_rows(heads * p.tiles, blocks, p.rows, a.D);
    auto stored = [&](int64_t n) { return n == 1 || heads * p.tiles * n * p.rows <= p.most_rows; };
    // whether clusters of n all run at once: each of the eight groups of SMs may have n - 1 places over
    auto fits = [](int64_t ctas, int64_t n, int64_t slots) { return n <= PG_CLUSTER && ctas <= slots - 8 * (n - 1); };
    if (a.S * grp <= 16) {
        p.few = true, p.tt = a.S;
        const int64_t sms = num_sms();
        // In us: start and end of a CTA 3, a block 0.9 alone on its SM and 1.25 beside another, or its share of
        // the memory (a wave of two per SM; the last one's part); a second launch 4.5, the merge in a
        // cluster 2. (Equal clusters: the more chunks, since requests may be shorter than their tables.)
        const double tile = 2.0 * PG_BN * a.D * 2 * double(sms) / 6.7e6;   // a block per SM, at the memory's rate
        for (int64_t n = 1; n <= blocks && n <= 64 && heads > 0 && n <= most_chunks(heads, 2 * sms); ++n) {
            const double per = double((blocks + n - 1) / n), load = double(heads * n) / double(sms);
            const double waves = floor(load / 2.0), rest = load - 2.0 * waves;
            const double shared = double(heads) * double(blocks) * tile / double(sms);
            double t = n > 1 ? 4.5 : 0.0;
            if (load <= 2.0) t += 3.0 + fmax(per * (load <= 1.0 ? 0.9 : 1.25), shared);
            else t += waves * (3.0 + per * 2.0 * tile) + (rest > 0.0 ? 3.0 + per * fmax(1.25, rest * tile) : 0.0);
            if (t < best && stored(n)) best = t, p.nchunk = int(n), p.cluster = false;
            const double tc = 5.0 + fmax(per * 0.9, shared);
            if (n > 1 && fits(heads * n, n, sms) && tc <= best) best = tc, p.nchunk = int(n), p.cluster = true;
        }
        p.alone = heads * p.nchunk <= sms;
    }
    const double shared = double(heads) * double(blocks) * 4.0 * PG_BN * a.D / 6.7e6;   // the memory's share
    for (int way = 0; way < 3 && heads > 0 && !p.few; ++way) {
        if (way == 2 && (p.tiles == 1 || a.D == 64)) break;
        const int nt = way == 2 ? 2 : 1;
        const bool alone = way == 1, many = p.tiles >= 4;
        const int64_t base = heads * ((p.tiles + nt - 1) / nt), slots = int64_t(num_sms()) * (way == 0 ? 2 : 1);
        const double ends = way == 0 ? 5.0 : alone ? 4.0 : 6.0;
        const double block = a.D == 128 ? (way == 0 ? (many ? 2.1 : 2.5) : alone ? (many ? 1.36 : 1.55) : 1.7)
                                        : (way == 0 ? 1.4 : 1.5);
        for (int64_t n = 1; n <= blocks && n <= most_chunks(base, slots); ++n) {
            const double load = double(base * n) / double(slots);
            const double waves = load <= 1.0 ? 1.0 : load < 3.0 ? ceil(load) : load + 0.5;
            const bool cluster = n > 1 && nt == 1 && fits(base * n, n, slots);
            const double merge = n == 1 ? 0.0 : cluster ? 2.0 + 3.0 * p.rows / PG_BM
                                 : 6.0 + double(heads) * p.tiles * double(n) * p.rows * a.D * 8.0 / 4e6;
            const double t = fmax(waves * (ends + block * double((blocks + n - 1) / n)), shared + 3.0) + merge;
            if (t < best && (cluster || stored(n)))
                best = t, p.nt = nt, p.nchunk = int(n), p.cluster = cluster, p.alone = alone;
        }
    }
    p.us = best;
    auto bytes = [&](int64_t rows, size_t* ml) {
        auto up = [](size_t b) { return (b + 255) / 256 * 256; };
        *ml = up(size_t(rows) * a.D * 4);
        return *ml + up(size_t(rows) * 8);
    };
    size_t most_ml;
    p.most = bytes(p.most_rows, &most_ml);
    if (p.nchunk > 1 && !p.cluster) p.total = bytes(heads * p.tiles * p.nchunk * p.rows, &p.part_ml);
    return p;
}

size_t paged_attention_part_bytes(const PagedArgs& a, bool most) {
    if (a.dtype != DARTREE_BF16) return 0;
    const PgPlan p = paged_plan(a);
    return most ? p.most : p.total;
}

void paged_attention_plan(const PagedArgs& a, dartree_paged_plan* out) {
    const PgPlan p = paged_plan(a);
    *out = dartree_paged_plan{p.few, p.few ? 1 : p.nt, p.nchunk, p.cluster, p.alone, p.total};
}

bool make_page_map(CUtensorMap* m, const PagedArgs& a, const void* pool) {
    const uint64_t d[4] = {uint64_t(a.D), uint64_t(a.page), uint64_t(a.Hkv), uint64_t(a.n_pages)};
    const uint64_t st[3] = {uint64_t(a.D) * 2, uint64_t(a.page) * a.D * 2, uint64_t(a.Hkv) * a.page * a.D * 2};
    const uint32_t box[4] = {64, uint32_t(a.page < PG_BN ? a.page : PG_BN), 1, 1};
    return make_tensor_map_bf16_nd(m, pool, 4, d, st, box);
}
bool make_query_map(CUtensorMap* m, const PagedArgs& a, const void* q, int tt) {
    const uint64_t d[3] = {uint64_t(a.D), uint64_t(a.Hq), uint64_t(a.T > 0 ? a.T : 1)};
    const uint64_t st[2] = {uint64_t(a.D) * 2, uint64_t(a.Hq) * a.D * 2};
    const uint32_t box[3] = {64, uint32_t(a.Hq / a.Hkv), uint32_t(tt)};
    return make_tensor_map_bf16_nd(m, q, 3, d, st, box);
}

template <int D, int NT, int ST, bool CL = false, bool SH = false>
static int launch_attn_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PgArgs& x,
                         cudaStream_t stream) {
    auto kern = paged_attn_kernel<D, NT, ST, CL, SH>;
    const size_t smem = PgSmem<D, NT, ST>::TOTAL;
    static std::atomic<uint64_t> raised{0};
    if (!raise_smem(kern, int(smem), raised)) return DARTREE_ECUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(x.s.ctas + unsigned(x.nchunk) * unsigned(x.a.C) * x.a.Hkv * ((x.tiles + NT - 1) / NT));
    cfg.blockDim = dim3(128 + 128 * NT);
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

int launch_paged_attention(const PagedArgs& a, const void* q, float scale, void* out, float* lse, void* part,
                           cudaStream_t stream) {
    const PgPlan p = paged_plan(a);
    CUtensorMap tq, tk, tv;
    if (!make_query_map(&tq, a, q, p.tt) || !make_page_map(&tk, a, a.k) || !make_page_map(&tv, a, a.v))
        return DARTREE_ECUDA;
    uint8_t* w = static_cast<uint8_t*>(part);
    // Tiles of nearly the same length (few new tokens beside the table's rows) follow one another head by
    // head and find their keys and values in the L2 (16 trees of 65 slots over 4096 rows, three tiles: 170 us
    // against 197); tiles of very different lengths go by length, the longest first. (Not for a grid that runs
    // at once: 28 against 27 us for four trees over 2048 rows.)
    const int64_t ctas = int64_t(a.C) * a.Hkv * ((p.tiles + p.nt - 1) / p.nt) * p.nchunk;
    const bool inner = 4 * int64_t(a.S) <= int64_t(a.max_pages) << a.log2_page &&
                       ctas > num_sms() * (p.nt == 1 && !p.alone ? 2 : 1);
    PgArgs x{a, a.Hq / a.Hkv, p.tt, p.tiles, p.nchunk, p.rows, inner, scale * LOG2E, static_cast<bf16_t*>(out), lse,
             reinterpret_cast<float*>(w), reinterpret_cast<float2*>(w + p.part_ml), PgGroups{}};
    int e;
    if (p.few)
        e = launch_paged_few(x, p.cluster, p.alone, tq, tk, tv, stream);
    else if (a.D == 64)
        e = (p.alone ? (p.cluster ? launch_attn_t<64, 1, 8, true> : launch_attn_t<64, 1, 8>)
                     : (p.cluster ? launch_attn_t<64, 1, 4, true> : launch_attn_t<64, 1, 4>))(tq, tk, tv, x, stream);
    else
        e = (p.nt == 2 ? launch_attn_t<128, 2, 5>
             : p.alone ? (p.cluster ? launch_attn_t<128, 1, 5, true> : launch_attn_t<128, 1, 5>)
                       : (p.cluster ? launch_attn_t<128, 1, 2, true> : launch_attn_t<128, 1, 2>))(tq, tk, tv, x, stream);
    if (e != DARTREE_OK || p.nchunk == 1 || p.cluster) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((size_t(a.C) * a.S * a.Hq + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    KTimer kt_(KID_PAGED_COMBINE, stream);
    const cudaError_t ce = a.D == 64 ? cudaLaunchKernelEx(&cfg, paged_combine_kernel<64, false>, x)
                                     : cudaLaunchKernelEx(&cfg, paged_combine_kernel<128, false>, x);
    return ce == cudaSuccess ? DARTREE_OK : DARTREE_ECUDA;
}

// ----------------------------------------------------------------------------- shared prefixes
//
// Requests that share their first rows: those rows are read once for a tile of 128 rows of q instead of once for
// each request. The new tokens of a group lie together in q, so the general kernel takes them as one request's, all
// of which see all shared rows, and leaves (maximum, sum, O) of each chunk in memory. Own rows of at most 16 rows of q
// to a request are the launch behind it (paged_own.cu), which joins; others are CTAs of the same launch, from the
// first row behind the shared pages on, and paged_combine_kernel joins.

struct PgSharedPlan {
    int early, early_items;           // own rows of few: CTAs beside the shared rows' and what each takes
    bool use, few, alone;             // shared at all; own rows by the transposed kernel; one CTA to an SM
    int tt, tiles, nt, np, ns;
    unsigned units;
    size_t ml, total;
};

// In us, fitted to sweeps like paged_plan's times. Shared rows: CTAs as there, and the partial results at 5 TB/s.
// Own rows of few (paged_own.cu): 5, a (request, head) pair 3, a block 1.1 and the join's loads 1.2 for every eight
// chunks, in rounds of two CTAs to an SM; pairs of CTAs that find room beside the shared rows' cost their joins only. Other
// own rows: as in paged_plan, behind the shared rows' CTAs in the same launch; the join is a launch, 4.
constexpr int64_t PG_SHARED_BYTES = int64_t(512) << 20;  // of partial rows, as long as there is a choice

static PgSharedPlan shared_plan(const PagedArgs& a, const dartree_paged_groups& s) {
    PgSharedPlan p{};
    const int G = s.G;
    int64_t most_rows = s.most_rows, most_rest = s.most_rest;
    const int64_t cap = int64_t(a.max_pages) << a.log2_page;
    if (most_rows <= 0 || most_rows > cap) most_rows = cap;
    if (most_rest <= 0 || most_rest > cap) most_rest = cap;
    const int grp = a.Hq / a.Hkv;
    const int64_t sms = num_sms(), heads = int64_t(a.C) * a.Hkv;
    const int64_t pb = (most_rows + PG_BN - 1) / PG_BN, rb = (most_rest + PG_BN - 1) / PG_BN;
    p.tt = PG_BM / grp;
    p.tiles = (a.S + p.tt - 1) / p.tt;
    p.few = a.S * grp <= 16;
    const int64_t row_bytes = int64_t(a.T) * a.Hq * a.D * 4;
    const double chunk = double(row_bytes) * 2.0 / 5e6;
    auto waves_of = [](double load) { return load <= 1.0 ? 1.0 : load < 3.0 ? ceil(load) : load + 0.5; };
    double best = 1e300;
    for (int way = 0; way < 3; ++way) {
        if (way == 2 && a.D == 64) break;
        const int nt = way == 2 ? 2 : 1;
        const int64_t per = int64_t(nt) * p.tt;
        const int64_t units = (a.T + G * (per - 1)) / per, base = units * a.Hkv;
        const double slots = double(sms) * (way == 0 ? 2.0 : 1.0);
        const bool many = units >= 4 * G;
        const double ends = way == 0 ? 5.0 : way == 1 ? 4.0 : 6.0;
        const double block = a.D == 128 ? (way == 0 ? (many ? 2.1 : 2.5) : way == 1 ? (many ? 1.36 : 1.55) : 1.7)
                                        : (way == 0 ? 1.4 : 1.5);
        const double pair = 3.0 + 1.1 * double(rb);
        double own = 0.0;
        int ns = 1;
        const double ctas = double(heads * ((p.tiles + nt - 1) / nt));
        for (int64_t n = 1; !p.few && n <= rb && n <= 4; ++n) {
            const double t = ctas * double(n) / slots * (ends + block * double((rb + n - 1) / n)) + chunk * double(n) + 4.0;
            if (n == 1 || t < own) own = t, ns = int(n);
        }
        // (of the chunks that leave equally many blocks to each, the fewest)
        for (int64_t n = 1, k = pb; n <= 64; n = (pb + k - 2) / (k - 1)) {
            if (n > 1 && (n + ns) * row_bytes > PG_SHARED_BYTES) break;
            k = (pb + n - 1) / n;
            const double cta = ends + block * double(k), load = double(base * n) / slots;
            const double prefix = waves_of(load) * cta + chunk * double(n);
            double t = prefix + own;
            if (p.few) {
                // own CTAs that find room beside the shared rows' serve pairs for as long as these last
                const int64_t left = load < 1.0 ? int64_t(2.0 * (1.0 - load) * double(sms)) : 0;
                const int64_t most = left > 0 ? (heads + left - 1) / left : 0;
                const int64_t early = std::min(most, std::max(int64_t(cta / pair), int64_t(1)));
                const int64_t rest = heads - left * early;
                const double join = 1.2 * ceil(double(n) / 8.0);
                t = fmax(prefix, double(early) * pair) + 5.0 + join * double(std::max(early, int64_t(1)));
                if (rest > 0) t += ceil(double(rest) / double(2 * sms)) * (pair + join);
                // (pairs that run at once hold each other up, and own rows pass the memory)
                t += 2.5 * double(heads) / double(2 * sms) + (heads > 2 * sms ? 3.0 : 0.0);
                t = fmax(t, 10.0 + double(heads) * double(most_rest) * a.D * 4.0 / 5.3e6);
                if (t < best) p.early = int(std::min(left, (heads + most - 1) / std::max(most, int64_t(1)))), p.early_items = int(early);
            }
            if (t < best) {
                best = t;
                p.nt = nt, p.np = int(n), p.ns = ns, p.alone = way == 1, p.units = unsigned(units);
            }
            if (k == 1) break;
        }
    }
    // Where sharing pays, from sweeps of 63 batches of few rows and 26 of more (both ways' times for each). The plain call's
    // requests find the shared rows in the L2, so that of its expected time over 25 about half comes true. Few rows: 64
    // tokens behind 16384 rows 52 us against 357, 8 behind 2048 12.4 against 15.3, 64 behind 442 27 against 25, 128 with 998
    // of their own behind 470 96 against 71. More rows than that only save what the requests' own tiles leave empty: ten
    // trees of 34 slots (136 rows) behind 6932 rows 63 against 82, sixteen of 65 (260 rows) behind 8192 141 against 111.
    const double plain = paged_plan(a, most_rows + most_rest).us, met = plain < 25.0 ? plain : 25.0 + 0.5 * (plain - 25.0);
    p.use = s.always || (p.few ? best < 0.97 * met : a.S * grp < 2 * PG_BM && best < 0.75 * plain);
    const int64_t rows = int64_t(a.T) * a.Hq * (p.np + p.ns);
    p.ml = (size_t(rows) * a.D * 4 + 255) / 256 * 256;
    p.total = p.ml + (size_t(rows) * 8 + 255) / 256 * 256;
    return p;
}

size_t paged_shared_part_bytes(const PagedArgs& a, const dartree_paged_groups& s) {
    const PgSharedPlan p = shared_plan(a, s);
    return p.use ? p.total : paged_plan(a).total;
}

void paged_shared_plan(const PagedArgs& a, const dartree_paged_groups& s, dartree_paged_shared_plan_t* out) {
    const PgSharedPlan p = shared_plan(a, s);
    *out = dartree_paged_shared_plan_t{p.use, p.few, p.nt, p.np, p.ns, p.alone, p.use ? p.total : paged_plan(a).total};
}

int launch_paged_shared(const PagedArgs& a, const void* q, const dartree_paged_groups& s, float scale, void* out,
                        float* lse, void* part, size_t part_bytes, cudaStream_t stream) {
    const PgSharedPlan p = shared_plan(a, s);
    if (part_bytes < (p.use ? p.total : paged_plan(a).total)) return DARTREE_EWORKSPACE;
    if (!p.use) return launch_paged_attention(a, q, scale, out, lse, part, stream);
    CUtensorMap tq, tk, tv;
    if (!make_query_map(&tq, a, q, p.tt) || !make_page_map(&tk, a, a.k) || !make_page_map(&tv, a, a.v))
        return DARTREE_ECUDA;
    uint8_t* w = static_cast<uint8_t*>(part);
    const int grp = a.Hq / a.Hkv;
    // (own rows by the other kernel: no CTAs for them in this launch)
    PgArgs x{a, grp, p.tt, p.few ? 0 : p.tiles, p.ns, 0, 0, scale * LOG2E, static_cast<bf16_t*>(out), lse,
             reinterpret_cast<float*>(w), reinterpret_cast<float2*>(w + p.ml),
             PgGroups{s.G, p.np, p.units, p.units * unsigned(a.Hkv) * unsigned(p.np), s.start, s.rows,
                      p.early, p.early_items}};
    int e;
    if (a.D == 64)
        e = (p.alone ? launch_attn_t<64, 1, 8, false, true> : launch_attn_t<64, 1, 4, false, true>)(tq, tk, tv, x, stream);
    else
        e = (p.nt == 2 ? launch_attn_t<128, 2, 5, false, true>
             : p.alone ? launch_attn_t<128, 1, 5, false, true>
                       : launch_attn_t<128, 1, 2, false, true>)(tq, tk, tv, x, stream);
    if (e != DARTREE_OK) return e;
    if (p.few) {
        CUtensorMap tf;
        if (!make_query_map(&tf, a, q, a.S)) return DARTREE_ECUDA;
        PgArgs y = x;
        y.tt = a.S, y.tiles = 1, y.rows = a.S * grp;
        return launch_paged_own(y, tf, tk, tv, stream);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((size_t(a.C) * a.S * a.Hq + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    KTimer kt_(KID_PAGED_COMBINE, stream);
    const cudaError_t ce = a.D == 64 ? cudaLaunchKernelEx(&cfg, paged_combine_kernel<64, true>, x)
                                     : cudaLaunchKernelEx(&cfg, paged_combine_kernel<128, true>, x);
    return ce == cudaSuccess ? DARTREE_OK : DARTREE_ECUDA;
}

}  // namespace dartree
