// Paged-cache attention for few rows: single tokens and short query sets (bf16).
//
// A row tile holds at most 16 packed rows (tokens x grouped heads), so every key byte meets
// at most 16 multiply-adds: the kernel is a stream of K and V at memory speed, and everything
// else has to hide under it.  Stages of 32 KB (K and V of 64 keys, or of 128 at head_dim 64;
// one TMA box per page and 128-byte column block) pass through a ring of 96 KB per CTA, two
// CTAs per SM; one warp issues the loads, four warps take a quarter of each stage's keys.
// The products are m16n8k16 tensor-core instructions on operands read by ldmatrix: at 16 rows a
// 128-row accumulator tile would be seven-eighths padding, and the arithmetic is a small part of
// the time either way.
//   S = Q K^T (Q in registers), online softmax per warp with a lazily moved maximum, O += P V.
// P is rounded to bf16 for the product (its sum is taken before, in fp32).  The warps work on
// separate keys with separate (m, l, O) and merge at the end of the item, so no step of the
// stream waits for another warp.  The work split, and the merge of an item split over CTAs,
// are those of cache_common.cuh.
// Measured, one token each of 32 query and 8 key heads of 128: 64 sequences of 200-16k keys
// (1.06 GB) 175 us, 6.07 TB/s, 0.90 of the copy rate; one history of 131k keys (537 MB) 97 us,
// 0.82; 200 sequences of up to 2k keys, 8 heads, with a bias table (454 MB) 95 us, 0.70; one
// sequence of 1k keys 10.9 us.  What is not the stream: 3 us until the first keys arrive (launch,
// offsets, page), 2.5 us an item's end (four warps' results, and its part's way to memory), 3 us
// for the last CTA's merge of an item's parts, and equal ranges that end up to 10% apart (131k
// keys: 71 to 85 us, at a mean of 77).
#include "cache_common.cuh"
#include "tilemath.cuh"

namespace jfa {

namespace {

constexpr int kDecBM = 16, kDecWarps = 4, kDecThreads = 32 * (kDecWarps + 1), kDecCtasPerSm = 2;

template <int D>
struct DecCfg {
    static constexpr int BN = 8192 / D;                      // keys of a stage: 32 KB of K and V
    static constexpr int KG = BN / 64;                       // groups of 16 keys that a warp takes of it
    static constexpr int kCB = D / 64;                       // 128-byte column blocks of a row
    static constexpr int kBlock = BN * 128;                  // one column block of a stage's keys
    static constexpr int kStage = 2 * kCB * kBlock;          // K blocks, then V blocks
    static constexpr int kStages = 98304 / kStage;
    static constexpr int kOffSlots = kStages * kStage;       // two tiles of 8 fp32 rows of the merge (8 KB kept)
    static constexpr int kOffML = kOffSlots + 2 * 16 * 64 * 4;   // [2 buffers][m, l][warp][row]
    static constexpr int kOffBias = kOffML + 2 * 2 * kDecWarps * 16 * 4;  // [row][32 buckets + 1], log2 units
    static constexpr int kOffBar = kOffBias + 16 * 33 * 4;
    static constexpr int kOffMisc = kOffBar + 2 * kStages * 8;
    static constexpr int kOffBase = (kOffMisc + 16 + int(sizeof(CacheStart)) + 15) / 16 * 16;  // lists: position of each box
    static constexpr int kBoxes = BN / 16;
    static constexpr int kBytes = kOffBase + kStages * kBoxes * 4 + 1024;
    static_assert(kDecCtasPerSm * (kBytes + 1024) <= 228 * 1024, "shared memory of an SM");
    static constexpr int kPart = kDecBM * (D + 2);           // floats of a partial result: O, m, l
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// c += a b, m16n8k16, bf16 operands, fp32 accumulator.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kDecWarps) : "memory"); }

template <int D, bool BIAS, bool LIST>
__global__ void __launch_bounds__(kDecThreads, kDecCtasPerSm)
    jfa_cache_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                            const CacheFwdParams p) {
    using C = DecCfg<D>;
    constexpr int BM = kDecBM, BN = C::BN, KG = C::KG, NS = 2 * KG, NT = D / 8;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto full = [&](uint32_t s) -> uint32_t { return sbase + C::kOffBar + 8u * s; };
    auto empty = [&](uint32_t s) -> uint32_t { return sbase + C::kOffBar + 8u * (C::kStages + s); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc);
    volatile int* last_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < uint32_t(C::kStages); ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kDecWarps);
        }
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    CacheStart* start = reinterpret_cast<CacheStart*>(smem + C::kOffMisc + 16);
    CacheCursor<BN, LIST> cur(p, cache_start<BN, LIST>(p, reinterpret_cast<int*>(smem)));  // (the ring's memory as scratch)
    if (threadIdx.x == 0) *start = cur.st;
    __syncthreads();
    if (LIST) launch_dependents();  // (the join kernel waits for this one to end)
    CacheSeg g;
    int* bases = reinterpret_cast<int*>(smem + C::kOffBase);  // [stage][box]

    if (warp == kDecWarps) {
        // ---------------------------------------------------------------- producer
        // A lane loads one box of each stage: K or V, column block, page.
        fence_proxy_async_smem();  // the scratch's writes before the first loads into it
        const int rows = min(1 << p.page_log2, 64);          // keys of a box
        const int per = BN / rows;                           // pages (or parts of one) in a stage
        const bool mine = lane < 2 * C::kCB * per;
        const int pg = lane % per, cb = (lane / per) % C::kCB, isv = lane / (per * C::kCB);
        const uint32_t box = uint32_t(isv * C::kCB * C::kBlock + cb * C::kBlock + pg * rows * 128);
        const CUtensorMap* map = isv ? &tmV : &tmK;
        uint32_t it = 0;
        bool ok = true, have = cur.next(p, g);
        int kt = g.k0;
        // A stage's page: -1 outside the item's keys (not loaded); past the cache (read as
        // zeros) for a bad entry.
        auto page_of = [&](const CacheSeg& s, int k) -> int {
            const int j = (s.r.f + k) * BN + pg * rows;
            if (!mine || j >= s.r.hi || j + rows <= s.r.lo) return -1;
            const int page = p.table[size_t(s.b) * size_t(p.max_pages) + size_t(j >> p.page_log2)];
            if (page >= 0 && page < p.n_pages) return page;
            atomicOr(p.status, kStatusBounds);
            return p.n_pages;
        };
        // Lists: a stage, as this lane sees it (its block; whether to load it; that block's page, the
        // slot and the position of the first key).  Its entry is asked for two stages before it is loaded,
        // its page one stage, so that the stream waits for neither; whether the entry counts is seen when it is loaded, the
        // first time while its page is on the way.
        struct Stage {
            bool have, read, met, head, starts, ends;  // an entry, the first, a new list, an entry's last stage
            int hk, block, last, slot, base, page, at;  // last: the entry before
            size_t row;                                // of the page table
        };
        CacheListScan scan;
        bool starts = false;
        auto list_of = [&](const CacheSeg& s) {
            return p.lists + (size_t(s.s.q0 + s.tile) * size_t(p.Hkv) + size_t(s.hk)) * size_t(p.n_list);
        };
        auto step = [&](Stage& s) {
            while (have && (g.r.n == 0 || kt >= g.k1)) {
                have = cur.next(p, g);
                kt = g.k0;
                starts = true;
            }
            s.have = have;
            s.block = -1;
            if (!have) return;
            const int j0 = kt++ * BN, j = j0 + pg * rows, e = j >> p.page_log2;
            s.hk = g.hk;
            s.slot = j & ((1 << p.page_log2) - 1);
            s.row = size_t(g.b) * size_t(p.max_pages);
            s.at = g.s.kv_len - g.s.q_len + g.tile;  // the token's position
            s.met = j < g.r.hi;
            s.head = e == 0;
            if (s.met) {
                s.block = list_of(g)[e];
                s.last = list_of(g)[max(e - 1, 0)];
            }
            s.ends = ((j0 + BN) & ((1 << p.page_log2) - 1)) == 0;
            s.starts = starts;
            starts = false;
        };
        auto look = [&](Stage& s) {  // (blocks past the token's own hold no key that it may see)
            s.base = int(uint32_t(s.block) << p.page_log2) + s.slot;
            s.read = mine && s.block >= 0 && s.block <= s.at >> p.page_log2 && s.base <= s.at;
            s.page = s.read ? p.table[s.row + size_t(s.block)] : -1;
        };
        if constexpr (LIST) {
            Stage now, next;
            step(now);
            if (now.have) {
                look(now);
                scan.start(list_of(g), (g.k0 * BN) >> p.page_log2, lane);
            }
            step(next);
            while (now.have) {
                const Stage s = now;
                now = next;
                if (now.have) {
                    look(now);
                    step(next);
                }
                if (s.starts) scan = CacheListScan();
                const bool counts = scan.counts(s.block, s.met, s.head ? 0u : CacheListScan::key(s.last), p.page_log2 <= 6, s.ends, per, pg, p.status);
                const bool in = s.read && counts;
                const uint32_t st = it % C::kStages, ph = (it / C::kStages) & 1;
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(empty(st), ph ^ 1, abort_flag))) {
                    ok = false;
                    break;
                }
                const int n = __popc(__ballot_sync(0xffffffffu, in));
                if (lane < per) bases[st * C::kBoxes + pg] = in ? s.base : kNoBlock;
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(full(st), uint32_t(n * rows * 128));
                __syncwarp();
                if (in) {
                    int page = s.page;
                    if (page < 0 || page >= p.n_pages) {
                        atomicOr(p.status, kStatusBounds);
                        page = p.n_pages;  // past the cache: read as zeros
                    }
                    tma_load_4d(sbase + st * C::kStage + box, map, full(st), cb * 64, s.slot, s.hk, page);
                }
                ++it;
            }
            have = false;
        }
        while (have && (g.r.n == 0)) have = cur.next(p, g), kt = g.k0;
        int page = have ? page_of(g, kt) : -1;
        while (have) {
            const int at = page, j0 = (g.r.f + kt) * BN + pg * rows, hk = g.hk;
            if (++kt >= g.k1) {
                do {
                    have = cur.next(p, g);
                    kt = g.k0;
                } while (have && g.r.n == 0);
            }
            if (have) page = page_of(g, kt);
            const uint32_t st = it % C::kStages, ph = (it / C::kStages) & 1;
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(empty(st), ph ^ 1, abort_flag))) {
                ok = false;
                break;
            }
            const int n = __popc(__ballot_sync(0xffffffffu, at >= 0));
            if (lane == 0) mbar_arrive_expect_tx(full(st), uint32_t(n * rows * 128));
            __syncwarp();
            if (at >= 0)
                tma_load_4d(sbase + st * C::kStage + box, map, full(st), cb * 64, j0 & ((1 << p.page_log2) - 1), hk, at);
            ++it;
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0) atomicOr(p.status, kStatusTimeout);
        }
        drain_ring(full(0), it, C::kStages);
        wait_previous();
        return;
    }

    // -------------------------------------------------------------------- consumers
    float* slots = reinterpret_cast<float*>(smem + C::kOffSlots);
    float* ml = reinterpret_cast<float*>(smem + C::kOffML);
    float* btab = reinterpret_cast<float*>(smem + C::kOffBias);
    const int quad = lane & 3, qrow = lane >> 2;
    uint32_t it = 0, seg_no = 0;
    bool ok = true;
    CacheCut cut = cache_no_cut();  // lists: parts are added up by the join kernel
    // ldmatrix source: row of this warp's 16 keys and 16-byte piece, for K and (transposed) V
    const int krow = 16 * KG * warp + (lane & 7) + ((lane >> 4) << 3), kpc = (lane >> 3) & 1;
    const int vrow = 16 * KG * warp + (lane & 7) + (((lane >> 3) & 1) << 3), vpc = lane >> 4;
    while (cur.next(p, g)) {
        const int bm = LIST ? p.bm : BM;
        const int R = g.s.q_len * p.g, diag = g.s.kv_len - g.s.q_len, r0 = g.tile * bm;
        const int nr = min(bm, R - r0);
        const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(p.Q);
        // this lane's rows qrow and qrow + 8: queries, limits, heads
        uint32_t qa[D / 16][4];
        int lim[2], low[2], rel[2];
        if (BIAS) {  // the rows' bias, for this item's heads
            for (int e = threadIdx.x; e < nr * 32; e += 32 * kDecWarps) {
                const int r = r0 + (e >> 5);
                btab[(e >> 5) * 33 + (e & 31)] =
                    p.bias[(g.hk * p.g + r - div_g(p, r) * p.g) * 32 + (e & 31)] * 1.4426950408889634f;
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rr = qrow + 8 * i;
            const bool in = rr < nr;
            const int r = r0 + (in ? rr : 0), tok = div_g(p, r), head = g.hk * p.g + r - tok * p.g;
            rel[i] = tok + diag;
            lim[i] = p.causal ? min(g.s.kv_len, rel[i] + 1) : g.s.kv_len;
            low[i] = p.window >= 0 ? rel[i] - p.window : 0;
            const __nv_bfloat16* src = Q + (g.s.q0 + tok) * p.q_stride + int64_t(head) * D + 2 * quad;
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                qa[s][i] = in ? *reinterpret_cast<const uint32_t*>(src + 16 * s) : 0u;
                qa[s][2 + i] = in ? *reinterpret_cast<const uint32_t*>(src + 16 * s + 8) : 0u;
            }
        }
        if (BIAS) consumer_sync();
        const float* brow[2] = {btab + qrow * 33, btab + (qrow + 8 < nr ? qrow + 8 : 0) * 33};
        // keys that every row of the tile sees: no mask in [all_lo, all_hi)
        const int t_first = div_g(p, r0), t_last = div_g(p, r0 + nr - 1);
        const int all_hi = p.causal ? min(g.s.kv_len, t_first + diag + 1) : g.s.kv_len;
        const int all_lo = p.window >= 0 ? max(0, t_last + diag - p.window) : 0;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
        int bucket = -1;
        float bcur[2] = {0.f, 0.f};
        const int k_end = g.r.n > 0 ? g.k1 : g.k0;
        for (int kt = g.k0; kt < k_end; ++kt, ++it) {
            const uint32_t st = it % C::kStages, ph = (it / C::kStages) & 1;
            if (ok && !__all_sync(0xffffffffu, mbar_wait_bounded(full(st), ph, abort_flag))) {
                ok = false;
                *abort_flag = 1;
                if (lane == 0) atomicOr(p.status, kStatusTimeout);
            }
            if (!ok) continue;
            const int w0 = (g.r.f + kt) * BN + 16 * KG * warp;  // this warp's keys [w0, w0 + 16 KG)
            const uint32_t sK = sbase + st * C::kStage, sV = sK + C::kCB * C::kBlock;
            // Values that no row may see are undefined, and 0 * NaN is not 0: clear them.
            bool edge = w0 < g.r.lo || w0 + 16 * KG > g.r.hi;
            int at16[KG];  // lists: the positions of each 16 keys
            if constexpr (LIST) {
                const int brows = min(1 << p.page_log2, 64);
                edge = false;
                bool none = true;
#pragma unroll
                for (int q = 0; q < KG; ++q) {
                    const int c = 16 * (KG * warp + q);
                    at16[q] = bases[st * C::kBoxes + c / brows] + (c & (brows - 1));
                    edge = edge || at16[q] + 16 > all_hi;
                    none = none && at16[q] >= all_hi;
                }
                if (none) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(empty(st));
                    continue;
                }
                if (edge) {
                    for (int e = lane; e < 16 * KG * C::kCB * 8; e += 32) {
                        const int row = e / (C::kCB * 8), c = e % (C::kCB * 8);
                        if (at16[KG == 2 ? row >> 4 : 0] + (row & 15) >= all_hi)
                            st_shared_v4(sV + uint32_t((c >> 3) * C::kBlock + (16 * KG * warp + row) * 128 + (c & 7) * 16), 0, 0, 0, 0);
                    }
                    __syncwarp();
                }
            }
            if (!LIST && edge) {
                for (int e = lane; e < 16 * KG * C::kCB * 8; e += 32) {
                    const int row = e / (C::kCB * 8), c = e % (C::kCB * 8), j = w0 + row;
                    if (j < g.r.lo || j >= g.r.hi)
                        st_shared_v4(sV + uint32_t((c >> 3) * C::kBlock + (16 * KG * warp + row) * 128 + (c & 7) * 16), 0, 0, 0, 0);
                }
                __syncwarp();
            }
            float s[NS][4];
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int q = 0; q < KG; ++q) {
                    uint32_t b[4];
                    ldsm4(b, sK + uint32_t((k >> 2) * C::kBlock + (16 * q + krow) * 128 + (((((k & 3) << 1) + kpc) ^ (krow & 7)) << 4)));
                    mma16816(s[2 * q], qa[k], b[0], b[1]);
                    mma16816(s[2 * q + 1], qa[k], b[2], b[3]);
                }
            // scores of rows qrow (i = 0) and qrow + 8 (i = 1) at keys w0 + 8 n + 2 quad + e
            if constexpr (LIST) {
#pragma unroll
                for (int q = 0; q < KG; ++q) {
                    const int far = rel[0] - at16[q];  // (the rows are one token's)
                    const int bk = relpos_bucket(far);
                    const bool one = far >= 15 && bk == relpos_bucket(far - 15);
#pragma unroll
                    for (int n = 2 * q; n < 2 * q + 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int j = 8 * (n & 1) + 2 * quad + (i & 1);  // key of the 16
                            float b = 0.f;
                            if (BIAS) b = brow[i >> 1][one ? bk : relpos_bucket(far - j)];
                            s[n][i] = BIAS ? fmaf(s[n][i], p.scale_log2, b) : s[n][i] * p.scale_log2;
                            if (j > far) s[n][i] = -INFINITY;
                        }
                }
            } else if (BIAS) {
                const int far = t_last + diag - w0, near = t_first + diag - (w0 + 16 * KG - 1);
                const int bk = relpos_bucket(far);
                if ((near >= 0 || far <= 0) && bk == relpos_bucket(near)) {
                    if (bk != bucket) {
                        bucket = bk;
#pragma unroll
                        for (int i = 0; i < 2; ++i) bcur[i] = brow[i][bk];
                    }
#pragma unroll
                    for (int n = 0; n < NS; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[n][i] = fmaf(s[n][i], p.scale_log2, bcur[i >> 1]);
                } else {
#pragma unroll
                    for (int n = 0; n < NS; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int j = w0 + 8 * n + 2 * quad + (i & 1);
                            s[n][i] = fmaf(s[n][i], p.scale_log2, brow[i >> 1][relpos_bucket(rel[i >> 1] - j)]);
                        }
                }
            } else {
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[n][i] *= p.scale_log2;
            }
            if (!LIST && (w0 < all_lo || w0 + 16 * KG > all_hi)) {
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = w0 + 8 * n + 2 * quad + (i & 1);
                        if (j >= lim[i >> 1] || j < low[i >> 1]) s[n][i] = -INFINITY;
                    }
            }
            float mx[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mx[i] = fmaxf(s[0][2 * i], s[0][2 * i + 1]);
#pragma unroll
                for (int n = 1; n < NS; ++n) mx[i] = fmax3(mx[i], s[n][2 * i], s[n][2 * i + 1]);
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            }
            // The maximum moves only when it would grow by more than 2^8: sums and O stay in
            // its units, and P stays below 2^8.
            const bool grow0 = mx[0] > m[0] + 8.f, grow1 = mx[1] > m[1] + 8.f;
            if (__any_sync(0xffffffffu, grow0 || grow1)) {
                const float n0 = grow0 ? mx[0] : m[0], n1 = grow1 ? mx[1] : m[1];
                const float a0 = m[0] == -INFINITY ? 0.f : ex2_approx(m[0] - n0);
                const float a1 = m[1] == -INFINITY ? 0.f : ex2_approx(m[1] - n1);
                m[0] = n0;
                m[1] = n1;
                l[0] *= a0;
                l[1] *= a1;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    o[n][0] *= a0;
                    o[n][1] *= a0;
                    o[n][2] *= a1;
                    o[n][3] *= a1;
                }
            }
            const float u0 = m[0] == -INFINITY ? 0.f : m[0], u1 = m[1] == -INFINITY ? 0.f : m[1];
            uint32_t pa[KG][4];
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const float e0 = ex2_approx(s[n][0] - u0), e1 = ex2_approx(s[n][1] - u0);
                const float e2 = ex2_approx(s[n][2] - u1), e3 = ex2_approx(s[n][3] - u1);
                l[0] += e0 + e1;
                l[1] += e2 + e3;
                pa[n >> 1][2 * (n & 1)] = pack_bf16x2(e0, e1);
                pa[n >> 1][2 * (n & 1) + 1] = pack_bf16x2(e2, e3);
            }
#pragma unroll
            for (int q = 0; q < KG; ++q)
#pragma unroll
                for (int n = 0; n < NT / 2; ++n) {
                    uint32_t b[4];
                    ldsm4_t(b, sV + uint32_t((n >> 2) * C::kBlock + (16 * q + vrow) * 128 + (((((n & 3) << 1) + vpc) ^ (vrow & 7)) << 4)));
                    mma16816(o[2 * n], pa[q], b[0], b[1]);
                    mma16816(o[2 * n + 1], pa[q], b[2], b[3]);
                }
            if (edge) fence_proxy_async_smem();  // the cleared rows before the ring's next load
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(st));
        }
        // ------------------------------------------------------------ end of the item's part
        // Merge the four warps: m and l of every row, then O, 8 rows at a time (most items have
        // no more), warps 2 and 3 into the slots, warps 0 and 1 onto them, and the two slots'
        // sum out.
        float* mw = ml + (seg_no & 1) * (2 * kDecWarps * 16);
        float* lw = mw + kDecWarps * 16;
        ++seg_no;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (quad == 0) {
                mw[warp * 16 + qrow + 8 * i] = m[i];
                lw[warp * 16 + qrow + 8 * i] = l[i];
            }
        }
        consumer_sync();
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = qrow + 8 * i;
            const float mm = fmaxf(fmaxf(mw[r], mw[16 + r]), fmaxf(mw[32 + r], mw[48 + r]));
            f[i] = m[i] == -INFINITY ? 0.f : ex2_approx(m[i] - mm);
        }
        const bool whole = g.whole();
        int first = 0, last = 0;
        if (!whole) {
            first = cache_first_cta(p, *start, g);
            last = cache_last_cta(p, *start, g);
        }
        float* part = p.part + size_t(cache_slot(blockIdx.x, first)) * C::kPart;
        constexpr int CW = D / 16;  // columns of a thread: 16 threads a row
        const int ocol = CW * (threadIdx.x & 15);
        float2* slot = reinterpret_cast<float2*>(slots) + (warp & 1) * (4 * D) + lane;  // [D / 8][8 rows][4]
#pragma unroll 1
        for (int h = 0; 8 * h < nr; ++h) {
            if (h) consumer_sync();
            const float fh = h ? f[1] : f[0];
            if (warp >= 2) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    slot[n * 32] = make_float2((h ? o[n][2] : o[n][0]) * fh, (h ? o[n][3] : o[n][1]) * fh);
            }
            consumer_sync();
            if (warp < 2) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float2 x = slot[n * 32];
                    slot[n * 32] = make_float2(fmaf(h ? o[n][2] : o[n][0], fh, x.x), fmaf(h ? o[n][3] : o[n][1], fh, x.y));
                }
            }
            // this thread's row: its maximum and sum
            const int orow = 8 * h + (threadIdx.x >> 4);
            float om = -INFINITY, ol = 0.f;
#pragma unroll
            for (int w = 0; w < kDecWarps; ++w) om = fmaxf(om, mw[16 * w + orow]);
#pragma unroll
            for (int w = 0; w < kDecWarps; ++w) {
                const float mm = mw[16 * w + orow];
                ol = fmaf(mm == -INFINITY ? 0.f : ex2_approx(mm - om), lw[16 * w + orow], ol);
            }
            consumer_sync();
            const float* a = slots + (ocol >> 3) * 64 + (orow & 7) * 8 + (ocol & 7);
            float v[CW];
#pragma unroll
            for (int e = 0; e < CW; e += 4) {
                const float4 x = *reinterpret_cast<const float4*>(a + e), y = *reinterpret_cast<const float4*>(a + 8 * D + e);
                v[e] = x.x + y.x;
                v[e + 1] = x.y + y.y;
                v[e + 2] = x.z + y.z;
                v[e + 3] = x.w + y.w;
            }
            if (orow >= nr || !ok) continue;
            if (!whole) {
#pragma unroll
                for (int e = 0; e < CW; e += 4)
                    *reinterpret_cast<float4*>(part + orow * D + ocol + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                if (ocol == 0) {
                    part[BM * D + orow] = om;
                    part[BM * D + BM + orow] = ol;
                }
                continue;
            }
            const int r = r0 + orow, tok = div_g(p, r);
            const size_t grow = size_t(g.s.q0 + tok) * size_t(p.H) + size_t(g.hk * p.g + r - tok * p.g);
            const float inv = ol > 0.f ? 1.f / ol : 0.f;
#pragma unroll
            for (int e = 0; e < CW; e += 4) {
                if (p.o_f32)
                    *reinterpret_cast<float4*>(static_cast<float*>(p.O) + grow * D + ocol + e) =
                        make_float4(v[e] * inv, v[e + 1] * inv, v[e + 2] * inv, v[e + 3] * inv);
                else
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + grow * D + ocol + e) =
                        make_uint2(pack_bf16x2(v[e] * inv, v[e + 1] * inv), pack_bf16x2(v[e + 2] * inv, v[e + 3] * inv));
            }
            if (ocol == 0 && p.lse) p.lse[grow] = ol > 0.f ? (om + __log2f(ol)) * 0.6931471805599453f : -INFINITY;
        }
        if (LIST && !whole && g.k0 == 0 && ok) cut = CacheCut{g.s.q0, nr, r0, g.hk * p.g, first, last, {0, 0}};
        if (LIST || whole) continue;
        __threadfence();
        consumer_sync();
        if (threadIdx.x == 0) {
            int done = 0;
            if (ok) {
                done = atomicAdd(p.counters + kCtrSplit + first, 1u) == uint32_t(last - first);
                if (done) p.counters[kCtrSplit + first] = 0u;  // every part has arrived: ready for the next call
                __threadfence();
            }
            *last_flag = done;
        }
        consumer_sync();
        if (!*last_flag) continue;
        // The last part to arrive adds them all up, in the order of the keys.  A warp takes a
        // row's maxima and sums, its lanes the parts; the weights go to the slots' memory, at
        // most kBatch parts at a time, and then a thread takes four columns of a row over the
        // parts, with the parts dealt to several threads where there are few columns.
        const int parts = last - first + 1, cols = nr * (D / 4);
        constexpr int kBatch = 96;           // parts x 16 rows of weights: 6 of the slots' 8 KB
        constexpr int kCols = BM * (D / 4) / (32 * kDecWarps);
        float* wts = slots;                  // [part][16]
        float* row_m = slots + kBatch * 16;  // [16], and the sums [16]
        float* row_l = row_m + 16;
        auto part_of = [&](int c) { return p.part + size_t(cache_slot(first + c, first)) * C::kPart; };
        // columns: up to 4 per thread (nr = 16); threads per column: as many as fit
        const int share = cols > 64 ? 1 : 32 * kDecWarps / cols, who = share > 1 ? threadIdx.x / cols : 0;
        const int col0 = share > 1 ? threadIdx.x % cols : threadIdx.x;
        constexpr int kAhead = 8;            // parts of the first column loaded before the weights are known
        float4 ahead[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (who + k * share < parts && col0 < cols && who < share)
                ahead[k] = __ldcg(reinterpret_cast<const float4*>(part_of(who + k * share)) + col0);
        const bool few = parts <= 64;        // a row's m and l in two registers of a lane
        for (int rr = warp; rr < nr; rr += kDecWarps) {
            float mm, ll;
            if (few) {
                float mc[2], lc[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int c = lane + 32 * k;
                    mc[k] = c < parts ? __ldcg(part_of(c) + BM * D + rr) : -INFINITY;
                    lc[k] = c < parts ? __ldcg(part_of(c) + BM * D + BM + rr) : 0.f;
                }
                mm = fmaxf(mc[0], mc[1]);
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, s));
                ll = 0.f;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int c = lane + 32 * k;
                    const float w = mc[k] == -INFINITY ? 0.f : ex2_approx(mc[k] - mm);
                    ll = fmaf(w, lc[k], ll);
                    if (c < parts) wts[c * 16 + rr] = w;
                }
            } else {
                mm = -INFINITY;
                for (int c = lane; c < parts; c += 32) mm = fmaxf(mm, __ldcg(part_of(c) + BM * D + rr));
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, s));
                ll = 0.f;
                for (int c = lane; c < parts; c += 32) {
                    const float mc = __ldcg(part_of(c) + BM * D + rr);
                    ll = fmaf(mc == -INFINITY ? 0.f : ex2_approx(mc - mm), __ldcg(part_of(c) + BM * D + BM + rr), ll);
                }
            }
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, s);
            if (lane == 0) {
                row_m[rr] = mm;
                row_l[rr] = ll;
            }
        }
        consumer_sync();
        float4 acc[kCols];
#pragma unroll
        for (int k = 0; k < kCols; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c0 = 0; c0 < parts; c0 += kBatch) {
            const int n = min(kBatch, parts - c0);
            for (int e = threadIdx.x; !few && e < n * 16; e += 32 * kDecWarps) {
                const int rr = e & 15;
                const float mc = rr < nr ? __ldcg(part_of(c0 + (e >> 4)) + BM * D + rr) : -INFINITY;
                wts[e] = mc == -INFINITY ? 0.f : ex2_approx(mc - row_m[rr]);
            }
            if (!few) consumer_sync();
            if (who < share) {
#pragma unroll
                for (int k = 0; k < kCols; ++k) {
                    const int col = col0 + k * 32 * kDecWarps, rr = col / (D / 4);
                    if (col >= cols) break;
                    const float* w = wts + rr;
                    auto add = [&](const float4 u, int c) {
                        const float f0 = w[c * 16];
                        acc[k].x = fmaf(u.x, f0, acc[k].x);
                        acc[k].y = fmaf(u.y, f0, acc[k].y);
                        acc[k].z = fmaf(u.z, f0, acc[k].z);
                        acc[k].w = fmaf(u.w, f0, acc[k].w);
                    };
                    int c = who;
                    if (k == 0 && c0 == 0) {
#pragma unroll
                        for (int a = 0; a < kAhead; ++a)
                            if (who + a * share < n) add(ahead[a], who + a * share);
                        c = who + kAhead * share;
                    }
#pragma unroll 8
                    for (; c < n; c += share) add(__ldcg(reinterpret_cast<const float4*>(part_of(c0 + c)) + col), c);
                }
            }
            consumer_sync();
        }
        if (share > 1) {  // the threads of a column, added in their order
            float4* sums = reinterpret_cast<float4*>(slots);  // (over the weights, read by now; row_l lies behind)
            if (who < share) sums[threadIdx.x] = acc[0];
            consumer_sync();
            if (who == 0)
                for (int k = 1; k < share; ++k) {
                    const float4 u = sums[k * cols + col0];
                    acc[0].x += u.x;
                    acc[0].y += u.y;
                    acc[0].z += u.z;
                    acc[0].w += u.w;
                }
        }
        if (who == 0) {
#pragma unroll
            for (int k = 0; k < kCols; ++k) {
                const int col = col0 + k * 32 * kDecWarps, rr = col / (D / 4), c = 4 * (col % (D / 4));
                if (col >= cols) break;
                const int r2 = r0 + rr, t2 = div_g(p, r2);
                const size_t orow2 = size_t(g.s.q0 + t2) * size_t(p.H) + size_t(g.hk * p.g + r2 - t2 * p.g);
                const float ll = row_l[rr], li = ll > 0.f ? 1.f / ll : 0.f;
                if (p.o_f32)
                    *reinterpret_cast<float4*>(static_cast<float*>(p.O) + orow2 * D + c) =
                        make_float4(acc[k].x * li, acc[k].y * li, acc[k].z * li, acc[k].w * li);
                else
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + orow2 * D + c) =
                        make_uint2(pack_bf16x2(acc[k].x * li, acc[k].y * li), pack_bf16x2(acc[k].z * li, acc[k].w * li));
                if (p.lse && c == 0)
                    p.lse[orow2] = ll > 0.f ? (row_m[rr] + __log2f(ll)) * 0.6931471805599453f : -INFINITY;
            }
        }
    }
    if (LIST && threadIdx.x == 0) p.cuts[blockIdx.x] = ok ? cut : cache_no_cut();
}

template <int D, bool BIAS, bool LIST = false>
cudaError_t launch(const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, bool early, int num_sms,
                   cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(jfa_cache_decode_kernel<D, BIAS, LIST>, DecCfg<D>::kBytes, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms * kDecCtasPerSm);
    cfg.blockDim = dim3(kDecThreads);
    cfg.dynamicSmemBytes = DecCfg<D>::kBytes;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = early ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, jfa_cache_decode_kernel<D, BIAS, LIST>, mk, mv, p);
    return e == cudaSuccess && LIST ? launch_cache_join(D, p, num_sms * kDecCtasPerSm, st) : e;
}

}  // namespace

size_t cache_decode_part_bytes(int D, int num_sms) {
    return size_t(num_sms) * kDecCtasPerSm * 2 * kDecBM * size_t(D + 2) * 4;
}

cudaError_t launch_cache_decode(int D, const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, bool early,
                                int num_sms, cudaStream_t st) {
    if (D == 128)
        return p.bias ? launch<128, true>(mk, mv, p, early, num_sms, st) : launch<128, false>(mk, mv, p, early, num_sms, st);
    return p.bias ? launch<64, true>(mk, mv, p, early, num_sms, st) : launch<64, false>(mk, mv, p, early, num_sms, st);
}

cudaError_t launch_cache_decode_lists(int D, const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, int num_sms,
                                      cudaStream_t st) {
    if (D == 128)
        return p.bias ? launch<128, true, true>(mk, mv, p, false, num_sms, st) : launch<128, false, true>(mk, mv, p, false, num_sms, st);
    return p.bias ? launch<64, true, true>(mk, mv, p, false, num_sms, st) : launch<64, false, true>(mk, mv, p, false, num_sms, st);
}

}  // namespace jfa
