// Attention weight each cached row of the paged cache receives (eviction's input):
//
//   w_j <- decay * w_j + sum over the new tokens i that see j, and the query heads of the
//          key/value head, of exp(scale <q_i, k_j> - lse_i)
//
// The scores are formed transposed, S^T = K Q^T: a block's 128 keys are the tile's rows
// (tensor-memory lanes) and the queries its columns, so each thread owns a key and adds up
// a row of its own: no reduction across threads, no atomics, a fixed order of addition.
//
// CTA = (chunk of key blocks, (request, key/value head)), over all query tiles of TT
// tokens x grp heads (columns token * grp + head), or (SPLIT: few key blocks under many
// query tiles) over a part of them, the parts' CTAs a cluster that adds its sums:
//   warp 0      producer: key blocks and query tiles by TMA through two rings (a single
//               query tile is fetched once)
//   warp 1      issues S^T into one of two tensor-memory buffers
//   warps 2..9  two groups of 128 threads, one per buffer: while one adds up a tile the
//               other's is formed; the groups' sums of a block meet in shared memory
// Single tokens are bound by reading the keys once (16 tokens over 4096-8192 rows: 39 us,
// 5.4 TB/s); chunks by the sums, an exponential per score and ~4.5 instructions (two chunks
// of 256-511 tokens over 4000-8000 rows, 16/4 heads of 64: 32 us, the exponentials alone 12).
// Every mbarrier wait is bounded; one that runs out records DARTREE_ETIMEOUT.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include "paged.cuh"
#include "tc.cuh"

namespace dartree {

constexpr int PW_BM = 128;   // keys of a block
constexpr int PW_NT = 320;   // producer, MMA, two groups of four warps

template <int D>
struct PwSmem {
    static constexpr int PANELS = D / 64;
    static constexpr size_t PANEL = size_t(PW_BM) * 128;
    static constexpr size_t TILE = PANELS * PANEL;
    // stages of the two rings: a single query tile stays, and the keys have the longer ring;
    // otherwise the queries stream past a block of keys. A tile of at most 16 columns (single
    // tokens) has a place of its own, and the keys all stages. 100 KB: two CTAs per SM
    static constexpr int SHORT = D == 64 ? 2 : 1, LONG = D == 64 ? 4 : 2, ALL = SHORT + LONG;
    static constexpr int FEW = 16;
    static constexpr size_t FEW_PANEL = FEW * 128;
    static constexpr int MAXS = ALL;                                     // barriers per ring
    static constexpr size_t FEW_OFF = ALL * TILE;
    static constexpr size_t LSE_OFF = FEW_OFF + PANELS * FEW_PANEL;     // float [2 groups][2][128]
    static constexpr size_t SUM_OFF = LSE_OFF + 4 * 128 * 4;            // float [2 blocks][128]
    static constexpr size_t BAR_OFF = SUM_OFF + 2 * 128 * 4;
    // kfull, kempty, qfull, qempty [MAXS], sfull, sfree [2]
    static constexpr size_t SLOT_OFF = BAR_OFF + 8 * (4 * MAXS + 4);
    static constexpr size_t TOTAL = SLOT_OFF + 16 + 1024;
    static_assert(2 * (TOTAL + 1024) <= 228 * 1024, "two CTAs fit in shared memory");
};

struct PwArgs {
    PagedArgs a;
    int grp, tt, tiles, nchunk;
    int split;                // CTAs of a cluster that share a chunk's query tiles
    float sl2, decay;
    const float* lse;
    float* weights;
};

template <int D, bool SPLIT>
__global__ void __launch_bounds__(PW_NT, 2)
    paged_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ PwArgs x) {
    using L = PwSmem<D>;
    const PagedArgs& a = x.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
    uint64_t* kempty = kfull + L::MAXS;
    uint64_t* qfull = kempty + L::MAXS;
    uint64_t* qempty = qfull + L::MAXS;
    uint64_t* sfull = qempty + L::MAXS;   // [2] scores written, by buffer
    uint64_t* sfree = sfull + 2;        // [2] scores read
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + L::SLOT_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::MAXS; ++s) {
            mbar_init(&kfull[s], 1);
            mbar_init(&kempty[s], 1);
            mbar_init(&qfull[s], 1);
            mbar_init(&qempty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sfull[s], 1);
            mbar_init(&sfree[s], 4);
        }
        fence_mbar_init();
    }
    const bool once = x.tiles == 1;                       // one query tile: it stays in stage 0
    const bool few = once && x.tt * x.grp <= L::FEW;
    const int ks_n = few ? L::ALL : once ? L::LONG : L::SHORT, qs_n = few ? 1 : once ? L::SHORT : L::LONG;
    uint8_t* const kring = smem;
    uint8_t* const qring = few ? smem + L::FEW_OFF : smem + ks_n * L::TILE;
    const uint32_t qpanel = uint32_t(few ? L::FEW_PANEL : L::PANEL);
    // columns that pad a tile to 16 are rows of zeros (no copy writes them): their scores are 0 and, with an lse of
    // -inf, add nothing, so a tile whose tokens are all there needs no masks
    const int used = x.tt * x.grp, pad = (16 - used % 16) % 16;
    for (int e = threadIdx.x; e < pad * qs_n * L::PANELS * 8; e += PW_NT) {
        const int row = e / 8 % pad, pnl = e / 8 / pad;        // (panel of all stages)
        uint8_t* const at = qring + (pnl / L::PANELS) * L::TILE + (pnl % L::PANELS) * qpanel;
        reinterpret_cast<uint4*>(at + size_t(used + row) * 128)[e % 8] = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    if (warp == 1) tc::tmem_alloc(slot, 256);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *slot;
    griddep_launch_dependents();
    griddep_wait();

    const unsigned split = SPLIT ? x.split : 1u, rest = blockIdx.x / split;
    const int part = int(blockIdx.x % split);                // (rank in the cluster)
    const int chunk = int(rest % x.nchunk), cg = int(rest / x.nchunk);
    const int c = cg / a.Hkv, g = cg - c * a.Hkv;
    bool bad;
    const PagedRequest r = paged_request(a, c, bad);
    if (bad && threadIdx.x == 0 && g == 0) set_status(a.status, DARTREE_EINTERNAL);
    const int blocks = (r.n_keys + PW_BM - 1) / PW_BM;
    const int per = (blocks + x.nchunk - 1) / x.nchunk;
    const int b0 = chunk * per, b1 = min(blocks, b0 + per);
    const int ntile = (r.n_new + x.tt - 1) / x.tt;
    // the tiles that see a row of block b, this CTA's part of them
    auto first_tile = [&](int b) -> int {
        const int ahead = b * PW_BM - r.n_old, first = a.mask || ahead <= 0 ? 0 : ahead / x.tt;
        return SPLIT ? first + max(ntile - first, 0) * part / int(split) : first;
    };
    auto last_tile = [&](int b) -> int {                     // one behind it
        if (!SPLIT) return ntile;
        const int ahead = b * PW_BM - r.n_old, first = a.mask || ahead <= 0 ? 0 : ahead / x.tt;
        return first + max(ntile - first, 0) * (part + 1) / int(split);
    };
    float total = 0.f, kept = 0.f;                           // (split: a key's sum here, its weight before)

    if (warp == 0) {
        // ---------------------------------------------------------------- producer
        if (b0 < b1 && ntile > 0) {
            const int pr = min(a.page, PW_BM), sub = PW_BM / pr;
            const int su = lane % sub, pn = lane / sub;
            const bool mine = pn < L::PANELS;
            const int32_t* table = a.table + size_t(c) * a.max_pages;
            // this lane's table entry of block b (looked up two blocks ahead, checked when it is used), and
            // the page to fetch: n_pages, beyond the pool and so all zeros, past the end and for no page
            auto entry_of = [&](int b) -> int {
                const int j = b * PW_BM + su * pr;
                return mine && j < r.n_keys ? table[j >> a.log2_page] : a.n_pages;
            };
            auto page_of = [&](int e, int b) -> int {
                if (unsigned(e) < unsigned(a.n_pages)) return e;
                if (mine && b * PW_BM + su * pr < r.n_keys) set_status(a.status, DARTREE_EINTERNAL);
                return a.n_pages;
            };
            const uint32_t qbytes = uint32_t(L::PANELS * x.tt * x.grp * 128);
            int e0 = entry_of(b0), e1 = entry_of(b0 + 1), nk = 0, nq = 0;
            // single tokens: the keys pass by the L2 (45.2 -> 41.8 us; chunks 31.8 -> 32.5)
            const uint64_t policy = tc::evict_first();
            bool ok = true;
            for (int b = b0; b < b1 && ok; ++b) {
                const int pg = page_of(e0, b);
                e0 = e1;
                e1 = entry_of(b + 2);
                if (lane == 0 && nk >= ks_n)
                    ok = mbar_wait_bounded(&kempty[nk % ks_n], uint32_t((nk / ks_n) & 1) ^ 1u, a.status);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                const int ks = nk % ks_n;
                if (lane == 0) mbar_arrive_expect_tx(&kfull[ks], uint32_t(L::TILE));
                __syncwarp();
                if (mine) {
                    uint8_t* const to = kring + ks * L::TILE + pn * L::PANEL + size_t(su) * pr * 128;
                    const int row = (b * PW_BM + su * pr) & (a.page - 1);
                    if (once) tc::tma_load_4d(to, &tmK, 64 * pn, row, g, pg, &kfull[ks], policy);
                    else tc::tma_load_4d(to, &tmK, 64 * pn, row, g, pg, &kfull[ks]);
                }
                ++nk;
                if (lane == 0 && !(once && nq > 0))
                    for (int t = first_tile(b), end = last_tile(b); t < end && ok; ++t) {
                        const int qs = nq % qs_n;
                        if (nq >= qs_n)
                            ok = mbar_wait_bounded(&qempty[qs], uint32_t((nq / qs_n) & 1) ^ 1u, a.status);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&qfull[qs], qbytes);
                        for (int p = 0; p < L::PANELS; ++p)
                            tc::tma_load_3d(qring + qs * L::TILE + p * qpanel, &tmQ, 64 * p, g * x.grp,
                                            r.q0 + t * x.tt, &qfull[qs]);
                        ++nq;
                    }
                ok = __shfl_sync(0xffffffffu, ok, 0);
            }
            // copies issued and not yet seen complete land before the CTA can exit
            if (lane == 0) {
                for (int q = max(nk - ks_n, 0); q < nk; ++q)
                    mbar_wait_bounded(&kfull[q % ks_n], uint32_t(q / ks_n) & 1u, a.status);
                for (int q = max(nq - qs_n, 0); q < nq; ++q)
                    mbar_wait_bounded(&qfull[q % qs_n], uint32_t(q / qs_n) & 1u, a.status);
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issue
        // (warp-uniform values, one elected lane: descriptors stay in uniform registers)
        const int n_t = __shfl_sync(0xffffffffu, ntile, 0), u0 = __shfl_sync(0xffffffffu, b0, 0),
                  u1 = __shfl_sync(0xffffffffu, b1, 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        if (n_t > 0 && tc::elect_one()) {
            const uint32_t id = tc::idesc_bf16_f32(PW_BM, (x.tt * x.grp + 15) / 16 * 16);
            constexpr uint32_t PSTEP = L::PANEL >> 4, TSTEP = L::TILE >> 4;  // descriptor steps (low word)
            const uint32_t k0 = (smem_u32(kring) >> 4) & 0x3fffu, q0 = (smem_u32(qring) >> 4) & 0x3fffu,
                           qstep = qpanel >> 4;
            constexpr uint32_t HI = uint32_t(tc::DESC_SW128_KMAJOR >> 32), LO = uint32_t(tc::DESC_SW128_KMAJOR);
            auto desc = [&](uint32_t at) { return (uint64_t(HI) << 32) | (LO | at); };
            int ks = 0, qs = 0, n = 0;
            uint32_t kp = 0, qp = 0;
            bool ok = true;
            for (int b = u0; b < u1 && ok; ++b) {
                ok = mbar_wait_bounded(&kfull[ks], kp, a.status);
                for (int t = first_tile(b), end = last_tile(b); t < end && ok; ++t, ++n) {
                    if (!once || n == 0) ok = mbar_wait_bounded(&qfull[qs], qp, a.status);
                    if (ok && n >= 2) ok = mbar_wait_bounded(&sfree[n & 1], uint32_t((n >> 1) - 1) & 1u, a.status);
                    if (!ok) break;
                    tc::fence_after_sync();
                    const uint32_t da = k0 + ks * TSTEP, db = q0 + qs * TSTEP;
#pragma unroll
                    for (int p = 0; p < L::PANELS; ++p)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc::mma_bf16(tm + uint32_t((n & 1) * 128), desc(da + p * PSTEP + 2u * kk),
                                         desc(db + p * qstep + 2u * kk), id, p > 0 || kk > 0);
                    if (!once) {
                        tc::mma_commit(&qempty[qs]);
                        if (++qs == qs_n) qs = 0, qp ^= 1u;
                    }
                    if (t + 1 == end) tc::mma_commit(&kempty[ks]);
                    tc::mma_commit(&sfull[n & 1]);
                }
                if (++ks == ks_n) ks = 0, kp ^= 1u;
            }
        }
    } else {
        // ---------------------------------------------------------------- sums
        const int group = (warp - 2) >> 2, quarter = warp & 3;
        const int key = quarter * 32 + lane;
        const uint32_t trow = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(group * 128);
        float* slse = reinterpret_cast<float*>(smem + L::LSE_OFF) + group * 256;   // [2][128]
        float* ssum = reinterpret_cast<float*>(smem + L::SUM_OFF);
        const int kti = key / x.grp, khg = key - kti * x.grp;   // token and head of column `key` of a tile
        const float* const lrow = x.lse + (size_t(r.q0) + kti) * a.Hq + size_t(g) * x.grp + khg;
        const size_t lstep = size_t(x.tt) * a.Hq;
        const int lmax = kti < x.tt ? r.n_new - kti : 0;        // tiles with t * tt below it have a token here
        // lse of column `key` of tile t (-inf: no token)
        auto lse_of = [&](int t) -> float { return t * x.tt < lmax ? lrow[t * lstep] : -INFINITY; };
        float* const wrow = x.weights + size_t(cg) * (size_t(a.max_pages) << a.log2_page);
        const uint64_t sl = pair(x.sl2, x.sl2);
        int n = 0, buf = 0;
        bool ok = true;
        // this group's next tile's values are fetched while the current one is added up
        int next_t = -1;
        float next_lse = 0.f;
        for (int b = b0; b < b1; ++b) {
            const int j = b * PW_BM + key;
            const bool owner = ntile == 1 ? (n & 1) == group : group == 0;   // writes the block's weights
            float before = 0.f;
            if (owner && j < r.n_old) before = wrow[j];
            float sum = 0.f;
            const int end = last_tile(b);
            for (int t = first_tile(b); t < end; ++t, ++n) {
                if ((n & 1) != group) continue;
                const float mine = next_t == t ? next_lse : lse_of(t);
                if (ntile > 1 || next_t != t) {                               // (a lone tile's stay)
                    buf ^= 1;                                                 // (the last tile's may still be read)
                    // minus it, in the log2 domain; a row that saw nothing adds nothing
                    slse[buf * 128 + key] = mine > -INFINITY ? mine * -1.4426950408889634f : -INFINITY;
                    asm volatile("bar.sync %0, 128;" :: "r"(2 + group) : "memory");
                }
                next_t = t;
                next_lse = mine;
                if (ntile > 1) {
                    next_t = t + 2;
                    if (next_t >= end && b + 1 < b1)                          // (then no split: end = ntile)
                        next_t = first_tile(b + 1) + (((n + end - t) & 1) != group ? 1 : 0);
                    if (next_t < end) next_lse = lse_of(next_t);
                }
                // a tree's new rows: bit i of tok, whether the tile's token i sees this key (a batch of loads is
                // independent and on its way at once: loads by need took a block of 33 slots 18 us longer)
                uint32_t tok[4] = {0, 0, 0, 0};
                const bool tree = a.mask && __any_sync(0xffffffffu, j >= r.n_old);
                if (tree) {
                    const int s = j - r.n_old, nt = min(r.n_new - t * x.tt, x.tt);
                    const uint8_t* row = a.mask + (size_t(c) * a.S + t * x.tt) * a.S + (s >= 0 && s < r.n_new ? s : 0);
#pragma unroll
                    for (int w = 0; w < 4; ++w)
#pragma unroll 1
                        for (int q = 0; q < 32 && 32 * w + q < nt; q += 8) {
                            uint8_t m[8];
#pragma unroll
                            for (int u = 0; u < 8; ++u) m[u] = row[size_t(min(32 * w + q + u, nt - 1)) * a.S];
#pragma unroll
                            for (int u = 0; u < 8; ++u) tok[w] |= m[u] ? 1u << (q + u) : 0u;
                        }
#pragma unroll
                    for (int w = 0; w < 4; ++w) tok[w] = s < 0 ? 0xffffffffu : s < r.n_new ? tok[w] : 0u;
                }
                ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(&sfull[group], uint32_t(n >> 1) & 1u, a.status));
                if (ok) {
                    tc::fence_after_sync();
                    const int t0 = t * x.tt, cols = min(r.n_new - t0, x.tt) * x.grp;   // columns with a token
                    // causal: a new row is seen by the tokens from its own on
                    const int s = j - r.n_old, from = a.mask || s <= t0 ? 0 : (s - t0) * x.grp;
                    uint64_t part[4] = {0, 0, 0, 0};
                    const float* z = slse + buf * 128;
                    // 2^(s sl2 - lse2) of 16 columns
                    auto add = [&](const uint32_t* v, int c0) {
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(z + c0 + e);
                            float y0, y1, y2, y3;
                            unpair(fma2(pair(v[e], v[e + 1]), sl, w.x), y0, y1);
                            unpair(fma2(pair(v[e + 2], v[e + 3]), sl, w.y), y2, y3);
                            const int k = (e >> 1) & 2;
                            part[k] = add2(part[k], pair(ex2(y0), ex2(y1)));
                            part[k + 1] = add2(part[k + 1], pair(ex2(y2), ex2(y3)));
                        }
                    };
                    // hidden columns get a score of -inf (what lies behind the last token may be anything)
                    if (__all_sync(0xffffffffu, used > 112 && cols == used && from <= 0 && !tree)) {
#pragma unroll
                        for (int c0 = 0; c0 < 128; c0 += 32) {
                            uint32_t v[32];
                            tc::tmem_ld32(trow + uint32_t(c0), v);
                            add(v, c0);
                            add(v + 16, c0 + 16);
                        }
                    } else if (!tree) {
#pragma unroll 1
                        for (int c0 = 0; c0 < cols; c0 += 16) {
                            uint32_t v[16];
                            tc::tmem_ld16(trow + uint32_t(c0), v);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (c0 + e >= cols || c0 + e < from) v[e] = 0xff800000u;
                            add(v, c0);
                        }
                    } else {
                        // a tree's rows: bit i of `see` is token c0 / grp + i's
#pragma unroll 1
                        for (int c0 = 0; c0 < cols; c0 += 16) {
                            uint32_t v[16];
                            const int ti = c0 / x.grp, w = ti >> 5;
                            const uint32_t lo = w == 0 ? tok[0] : w == 1 ? tok[1] : w == 2 ? tok[2] : tok[3];
                            const uint32_t up = w == 0 ? tok[1] : w == 1 ? tok[2] : w == 2 ? tok[3] : 0u;
                            uint32_t see = __funnelshift_r(lo, up, ti & 31);
                            int hg = c0 - ti * x.grp;
                            tc::tmem_ld16(trow + uint32_t(c0), v);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                if (!(see & 1u) || c0 + e >= cols) v[e] = 0xff800000u;
                                if (++hg == x.grp) hg = 0, see >>= 1;
                            }
                            add(v, c0);
                        }
                    }
                    float s0, s1;
                    unpair(add2(add2(part[0], part[1]), add2(part[2], part[3])), s0, s1);
                    sum += s0 + s1;
                    tc::fence_before_sync();
                }
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(&sfree[group]);
            }
            if (ntile > 1) {  // the groups' sums of the block: group 1 hands over its own, by block parity
                if (group == 1) ssum[(b & 1) * 128 + key] = sum;
                asm volatile("bar.sync 1, 256;" ::: "memory");
                if (group == 0) sum += ssum[(b & 1) * 128 + key];
            }
            if (SPLIT) total = ok ? sum : 0.f, kept = before;
            else if (owner && j < r.n_keys && ok) wrow[j] = j < r.n_old ? fmaf(x.decay, before, sum) : sum;
        }
    }
    if constexpr (SPLIT) {
        // (one block: its sums, group 0's, go to shared memory, and the first CTA adds the parts in their order)
        const int key = (warp & 3) * 32 + lane, j = b0 * PW_BM + key;
        float* const xs = reinterpret_cast<float*>(smem + L::SUM_OFF) + ((b0 & 1) ^ 1) * 128;
        const bool mine = warp >= 2 && warp < 6;
        if (mine) xs[key] = total;
        __syncwarp();
        cluster_sync();
        if (mine && part == 0 && b0 < b1 && j < r.n_keys) {
            float sum = 0.f;
            for (int q = 0; q < int(split); ++q) sum += __uint_as_float(ld_dsmem_u32(dsmem_addr(xs + key, q)));
            x.weights[size_t(cg) * (size_t(a.max_pages) << a.log2_page) + j] = j < r.n_old ? fmaf(x.decay, kept, sum) : sum;
        }
        __syncwarp();
        cluster_sync();                                      // (no CTA leaves while its sums are read)
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tmem, 256);
}

// ----------------------------------------------------------------------------- host

template <int D, bool SPLIT>
static int launch_weights_t(const CUtensorMap& tq, const CUtensorMap& tk, const PwArgs& x, cudaStream_t stream) {
    auto kern = paged_weights_kernel<D, SPLIT>;
    const size_t smem = PwSmem<D>::TOTAL;
    static std::atomic<uint64_t> raised{0};
    if (!raise_smem(kern, int(smem), raised)) return DARTREE_ECUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(x.split) * x.nchunk * unsigned(x.a.C) * x.a.Hkv);
    cfg.blockDim = dim3(PW_NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2] = {pdl_attribute()};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(x.split);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = SPLIT ? 2 : 1;
    KTimer kt_(KID_PAGED_WEIGHTS, stream);
    return cudaLaunchKernelEx(&cfg, kern, tq, tk, x) == cudaSuccess ? DARTREE_OK : DARTREE_ECUDA;
}

int launch_paged_weights(const PagedArgs& a, const void* q, const float* lse, float scale, float decay,
                         float* weights, cudaStream_t stream) {
    PwArgs x{a, a.Hq / a.Hkv, 0, 0, 0, 1, scale * 1.4426950408889634f, decay, lse, weights};
    x.tt = 128 / x.grp < a.S ? 128 / x.grp : a.S;
    x.tiles = (a.S + x.tt - 1) / x.tt;
    const int64_t heads = int64_t(a.C) * a.Hkv;
    const int64_t blocks = ((int64_t(a.max_pages) << a.log2_page) + PW_BM - 1) / PW_BM;
    // Chunks of key blocks, in us. More query tiles than one: two CTAs an SM hardly slow each other, and a CTA
    // takes 3 and 1.4 (heads of 64: 1.2) for each tile of each of its blocks; so many waves. One query tile: start
    // and end of a CTA 2, a block 0.56 alone on its SM and 0.75 beside another, or its share of the memory (a
    // wave of two per SM; the last one's part). Of equals (several tiles: of those within 8 %) the most chunks,
    // since requests may be shorter than their tables: two chunks of 256-511 tokens, 32 us with 67 chunks and 38
    // with 34, where equal lengths take 41.8 and 40.3. 16 requests of 8192 rows, 8 heads: two chunks 43.0 us, one
    // 49.5, five 51.1; 16 trees of 65 slots over 4096 rows: seven 74 us, three 102.
    const int64_t sms = num_sms(), most = 4 * sms / heads > 64 ? 4 * sms / heads : 64;
    const double tile = double(PW_BM) * a.D * 2 * double(sms) / 6.7e6;     // a block per SM, at the memory's rate
    const double shared = double(heads) * double(blocks) * tile / double(sms);
    auto time = [&](int64_t n) -> double {
        const double per = double((blocks + n - 1) / n), load = double(heads * n) / double(sms);
        const double waves = floor(load / 2.0), rest = load - 2.0 * waves;
        if (x.tiles > 1)
            return (load <= 8.0 ? ceil(load / 2.0) : load / 2.0 + 0.5) * (3.0 + per * x.tiles * (a.D == 64 ? 1.2 : 1.4));
        if (load <= 2.0) return 2.0 + fmax(per * (load <= 1.0 ? 0.56 : 0.75), shared);
        return waves * (2.0 + per * 2.0 * tile) + (rest > 0.0 ? 2.0 + per * fmax(0.75, rest * tile) : 0.0);
    };
    double best = 1e300;
    for (int64_t n = 1; n <= blocks && n <= most; ++n) best = fmin(best, time(n));
    x.nchunk = 1;
    for (int64_t n = 1; n <= blocks && n <= most; ++n)
        if (time(n) <= best * (x.tiles > 1 ? 1.08 : 1.0)) x.nchunk = int(n);
    // Few key blocks under many query tiles (prompts with little before them): a block to a CTA, and two, four or
    // eight CTAs, a cluster, share its tiles; start, end and merge 5 then. The longest CTA, or all waves and half
    // of the longest (of new rows only the tokens from their own on see them). A prompt of 512 tokens 20.9 -> 9.1
    // us, 2048 76 -> 42, 378 of three requests, 16 heads of a group, 53 -> 16; over more waves than its tiles are
    // worth it loses (two chunks of 511 tokens over 8000 rows: 42 us whole, 50 by two).
    if (x.tiles > 1) {
        const double seen = double(x.tiles) * (a.mask ? 1.0 : 1.0 - 0.5 * fmin(1.0, a.S / double(blocks * PW_BM)));
        const double tile_us = a.D == 64 ? 1.2 : 1.4;
        auto shared_time = [&](int64_t q, double ends) -> double {
            const double part = ceil(double(x.tiles) / double(q)), w = double(heads * blocks * q) / double(2 * sms);
            return fmax(ends + part * tile_us, w * (ends + seen / double(q) * tile_us) + 0.5 * part * tile_us);
        };
        best = fmin(best, shared_time(1, 3.0));
        for (int64_t q = 2; q <= 8; q *= 2)
            if (shared_time(q, 5.0) < 0.95 * best) best = shared_time(q, 5.0), x.nchunk = int(blocks), x.split = int(q);
    }
    CUtensorMap tq, tk;
    // (a batch without tokens has no queries: its map is never used)
    if (!make_query_map(&tq, a, a.T > 0 ? q : a.k, x.tt) || !make_page_map(&tk, a, a.k)) return DARTREE_ECUDA;
    if (x.split > 1)
        return a.D == 64 ? launch_weights_t<64, true>(tq, tk, x, stream) : launch_weights_t<128, true>(tq, tk, x, stream);
    return a.D == 64 ? launch_weights_t<64, false>(tq, tk, x, stream) : launch_weights_t<128, false>(tq, tk, x, stream);
}

}  // namespace dartree
