// Paged-cache attention for chunks of new tokens (bf16): tcgen05 products, TMEM accumulators.
//
// An item is up to 256 packed rows (tokens x grouped heads) of one (sequence, key head): two
// 128-row tiles that share every key and value tile, so that one tile's softmax runs while
// the tensor core works on the other.  Key tiles of 128 positions are gathered by TMA, one
// box per page and 128-byte column block; a box of a short page lands at its rows of the
// tile, whose swizzle repeats every 8 rows (the smallest page).
// CTA = 18 warps, one CTA per SM, each on an equal share of the batch's key-tile steps
// (cache_common.cuh).  Two warps share each row (thread = row = TMEM lane): one takes score
// columns [0, 64) and O columns [0, D/2), the other the rest; they exchange row maxima and
// sums through shared memory.
//   warps 0-3, 8-11    tile A, columns [0, 64) and [64, 128): softmax, rescaling, epilogue
//   warps 4-7, 12-15   tile B
//   warp 16            loads: Q rows (cp.async, swizzled by hand: packed rows of grouped
//                      heads are not a box), K and V boxes through 2-stage rings
//   warp 17            tcgen05.mma issuer and TMEM owner; clears V rows no query may see
// TMEM (512 columns): S_A [0,128), S_B [128,256), O_A [256,256+D), O_B [384,384+D); P
// overwrites its own S columns as packed bf16 and is read from TMEM by O += P V.
// An item with a single row tile runs its steps alternately as tile A and tile B (both on
// the same query rows, each with its own maximum, sum and O), so it keeps the overlap; the
// two are merged at the end.
#include "cache_common.cuh"
#include "tilemath.cuh"

namespace jfa {

namespace {

template <int D>
struct ChkCfg {
    static constexpr int BM = 128, BN = 128, kPair = 2 * BM;
    static constexpr int kCB = D / 64;
    static constexpr int kQBytes = BM * D * 2, kKVBytes = BN * D * 2;
    static constexpr int kOffQ = 0, kOffK = kOffQ + 2 * kQBytes, kOffV = kOffK + 2 * kKVBytes;
    static constexpr int kOffBar = kOffV + 2 * kKVBytes;
    static constexpr int kNumBars = 32;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;   // tmem slot, abort flag, merge flag
    static constexpr int kOffStart = kOffMisc + 16;
    static constexpr int kOffComb = kOffStart + 64;           // tile B's m and l halves of a split item, two buffers
    static constexpr int kOffXch = kOffComb + 2 * 3 * BM * 4; // pair exchanges [2][2][8][32]
    static constexpr int kSmemNeed = kOffXch + 2 * 2 * 8 * 32 * 4 + 1024;
    // at least 120 KB: one CTA per SM, as the CTA allocates all 512 TMEM columns
    static constexpr int kSmemBytes = kSmemNeed > 120 * 1024 ? kSmemNeed : 120 * 1024;
    static constexpr int kSoftWarps = 16, kProdWarp = 16, kMmaWarp = 17, kThreads = 18 * 32;
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kIdescQK = make_idesc(kFmtBF16, BM, BN, false, false);
    static constexpr uint32_t kIdescPV = make_idesc(kFmtBF16, BM, D, false, true);
    static constexpr int kPart = kPair * (D + 2);  // floats of a partial result: O (four columns of all rows at a time), m, l
    __host__ __device__ static constexpr uint32_t tmem_s(int x) { return x ? 128u : 0u; }
    __host__ __device__ static constexpr uint32_t tmem_o(int x) { return x ? 384u : 256u; }
};

enum {
    B_Q_FULL = 0,
    B_Q_EMPTY = 1,
    B_K_FULL = 2,   // +stage
    B_K_EMPTY = 4,
    B_V_FULL = 6,
    B_V_EMPTY = 8,
    B_S_FULL = 10,  // +tile
    B_P_FULL = 12,
    B_O_DONE = 14,
    B_O_EMPTY = 16,
    B_DRAIN = 18,
    B_COMBINE = 19,  // split item: tile B's last P V done and its m and l written
    B_XCH = 20,      // +pair of warps
    B_PART = 28,     // partial result written by every softmax warp
    B_FLAG = 29,     // and its arrival counted
};

// TMEM column (within a tile's S/P columns) of the 16 P values of P V step s.
__device__ __forceinline__ uint32_t p_col(int s) { return uint32_t(32 * (s >> 1) + 8 * (s & 1)); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// What every role derives from an item's part: the steps [k0, k1) of the pair's key tiles,
// and those of them that each tile takes.
struct Steps {
    int k0, k1;      // none when the item has no key
    int a[2], b[2];  // tile x: steps [a, b)
    bool split;      // one row tile, its steps taken alternately by both tiles
    __device__ int count(int x) const {
        if (split) return (k1 - k0 + 1 - x) / 2;
        return b[x] > a[x] ? b[x] - a[x] : 0;
    }
};
__device__ __forceinline__ Steps steps_of(const CacheFwdParams& p, const CacheSeg& g) {
    Steps s;
    s.k0 = g.k0;
    s.k1 = g.r.n > 0 ? g.k1 : g.k0;
    s.split = (2 * g.tile + 1) * 128 >= g.s.q_len * p.g;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        CacheRange r{0, 0, 0, 0};
        if ((2 * g.tile + x) * 128 < g.s.q_len * p.g) r = cache_range<128, 128>(p, g.s, 2 * g.tile + x);
        s.a[x] = max(s.k0, r.f - g.r.f);
        s.b[x] = r.n > 0 ? min(s.k1, r.f - g.r.f + r.n) : s.a[x];
    }
    return s;
}

template <int D, bool BIAS>
__global__ void __launch_bounds__(576, 1)
    jfa_cache_chunk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                           const CacheFwdParams p) {
    using C = ChkCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t sQ = sbase + C::kOffQ, sK = sbase + C::kOffK, sV = sbase + C::kOffV;
    auto bar = [&](int i) -> uint32_t { return sbase + C::kOffBar + 8u * uint32_t(i); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    volatile int* last_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
    CacheStart* start = reinterpret_cast<CacheStart*>(smem + C::kOffStart);
    static_assert(sizeof(CacheStart) <= 64, "start record");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(bar(B_Q_FULL), 1);
        mbar_init(bar(B_Q_EMPTY), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(B_K_FULL + s), 1);
            mbar_init(bar(B_K_EMPTY + s), 1);
            mbar_init(bar(B_V_FULL + s), 1);
            mbar_init(bar(B_V_EMPTY + s), 1);
            mbar_init(bar(B_S_FULL + s), 1);
            mbar_init(bar(B_P_FULL + s), 8);
            mbar_init(bar(B_O_DONE + s), 1);
            mbar_init(bar(B_O_EMPTY + s), 8);
        }
        mbar_init(bar(B_DRAIN), 1);
        mbar_init(bar(B_COMBINE), 8);
        for (int q = 0; q < 8; ++q) mbar_init(bar(B_XCH + q), 2);
        mbar_init(bar(B_PART), C::kSoftWarps);
        mbar_init(bar(B_FLAG), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == C::kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    cache_start<C::kPair, C::BN>(p, start, reinterpret_cast<long long*>(smem));  // (Q's memory as scratch)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    CacheCursor<C::kPair, C::BN> cur(*start);
    CacheSeg g;

    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(p.status, kStatusTimeout);
    };

    if (warp == C::kProdWarp) {
        // ------------------------------------------------------------ loads
        // One box of K and one of V per lane and tile: column block, page (or 64 keys of one).
        const int rows = min(1 << p.page_log2, 64), per = C::BN / rows;
        const bool mine = lane < C::kCB * per;
        const int pg = lane % per, cb = (lane / per) % C::kCB;
        const uint32_t box = uint32_t(cb * C::BN * 128 + pg * rows * 128);
        uint32_t kv_it = 0, item_it = 0, k_extra = 0;
        bool ok = true;
        auto page_of = [&](const CacheSeg& s, int k) -> int {
            const int j = (s.r.f + k) * C::BN + pg * rows;
            if (!mine || j >= s.r.hi || j + rows <= s.r.lo) return -1;
            const int page = p.table[size_t(s.b) * size_t(p.max_pages) + size_t(j >> p.page_log2)];
            if (page >= 0 && page < p.n_pages) return page;
            atomicOr(p.status, kStatusBounds);
            return p.n_pages;  // past the cache: read as zeros
        };
        auto wwait = [&](int b, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait_bounded(bar(b), parity, abort_flag));
        };
        while (ok && cur.next(p, g)) {
            if (g.r.n == 0) continue;
            if (!wwait(B_Q_EMPTY, (item_it & 1) ^ 1)) { ok = false; break; }
            {
                // Q: row r of the pair (token r / g, head r % g) to row r % 128 of its tile
                constexpr int kChunks = D / 8, kStep = 32 / kChunks;  // 16-byte pieces of a row; rows per pass
                const int c = lane % kChunks, R = g.s.q_len * p.g, r0 = g.tile * C::kPair;
                const int n = min(C::kPair, (min(R - r0, C::kPair) + C::BM - 1) / C::BM * C::BM);
                int r = lane / kChunks, tok = (r0 + r) / p.g, h = r0 + r - tok * p.g;
                const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.Q);
                for (; r < n; r += kStep) {
                    const bool in = r0 + r < R;
                    const __nv_bfloat16* src =
                        in ? q + (g.s.q0 + tok) * p.q_stride + int64_t(g.hk * p.g + h) * D + 8 * c : q;
                    const int row = r & (C::BM - 1);
                    cp_async16(sQ + uint32_t((r / C::BM) * C::kQBytes + (c >> 3) * C::BM * 128 + row * 128 +
                                             (((c & 7) ^ (row & 7)) << 4)),
                               src, in);
                    h += kStep;
                    while (h >= p.g) {
                        h -= p.g;
                        ++tok;
                    }
                }
            }
            ++item_it;
            int page = page_of(g, g.k0);
            for (int k = g.k0; k < g.k1; ++k, ++kv_it) {
                const uint32_t st = kv_it & 1, ph = (kv_it >> 1) & 1;
                const int at = page, slot = ((g.r.f + k) * C::BN + pg * rows) & ((1 << p.page_log2) - 1);
                const uint32_t bytes = uint32_t(__popc(__ballot_sync(0xffffffffu, at >= 0)) * rows * 128);
                if (k + 1 < g.k1) page = page_of(g, k + 1);
                if (!wwait(B_K_EMPTY + st, ph ^ 1)) { ok = false; break; }
                if (lane == 0) mbar_arrive_expect_tx(bar(B_K_FULL + st), bytes);
                __syncwarp();
                if (at >= 0) tma_load_4d(sK + st * C::kKVBytes + box, &tmK, bar(B_K_FULL + st), cb * 64, slot, g.hk, at);
                if (!wwait(B_V_EMPTY + st, ph ^ 1)) { k_extra = 1; ok = false; break; }
                if (lane == 0) mbar_arrive_expect_tx(bar(B_V_FULL + st), bytes);
                __syncwarp();
                if (at >= 0) tma_load_4d(sV + st * C::kKVBytes + box, &tmV, bar(B_V_FULL + st), cb * 64, slot, g.hk, at);
                if (k == g.k0) {  // Q has arrived by now, or nearly
                    cp_async_wait_all();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_Q_FULL));
                }
            }
        }
        if (!ok && lane == 0) fail();
        cp_async_wait_all();
        __syncwarp();
        drain_ring(bar(B_K_FULL), kv_it + k_extra, 2);
        drain_ring(bar(B_V_FULL), kv_it, 2);
    } else if (warp == C::kMmaWarp) {
        // ------------------------------------------------------------ MMA issuer
        auto wwait = [&](int b, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait_bounded(bar(b), parity, abort_flag));
        };
        uint32_t kv_it = 0, item_it = 0, pv_cnt0 = 0, pv_cnt1 = 0, items_x0 = 0, items_x1 = 0;
        bool ok = true;
        const SDesc dQ0 = sdesc_sw128(sQ, 16, 1024), dQ1 = sdesc_sw128(sQ + C::kQBytes, 16, 1024);
        const SDesc dK0 = sdesc_sw128(sK, 16, 1024), dK1 = sdesc_sw128(sK + C::kKVBytes, 16, 1024);
        const SDesc dV0 = sdesc_sw128(sV, C::BN * 128, 1024), dV1 = sdesc_sw128(sV + C::kKVBytes, C::BN * 128, 1024);
        // S_x = Q K^T, after the tile's previous P V product, which reads P from those columns
        auto issue_s = [&](int x, uint32_t st, int qx) -> bool {
            const uint32_t pc = x ? pv_cnt1 : pv_cnt0;
            if (pc > 0 && !wwait(B_O_DONE + x, (pc - 1) & 1)) return false;
            tc_fence_after();
            const SDesc dq = qx ? dQ1 : dQ0, dk = st ? dK1 : dK0;
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
                    mma_ss(tmem + C::tmem_s(x), dq, ((s * 32) >> 7) * C::BM * 128 + ((s * 32) & 127), dk,
                           ((s * 32) >> 7) * C::BN * 128 + ((s * 32) & 127), C::kIdescQK, s > 0);
                tc_commit(bar(B_S_FULL + x));
            }
            __syncwarp();
            return true;
        };
        // O_x += P_x V
        auto issue_pv = [&](int x, uint32_t st, bool first) -> bool {
            const uint32_t pc = x ? pv_cnt1 : pv_cnt0, ix = x ? items_x1 : items_x0;
            if (!wwait(B_P_FULL + x, pc & 1)) return false;
            if (first && !wwait(B_O_EMPTY + x, (ix & 1) ^ 1)) return false;
            tc_fence_after();
            const SDesc dv = st ? dV1 : dV0;
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < C::BN / 16; ++s)
                    mma_ts(tmem + C::tmem_o(x), tmem + C::tmem_s(x) + p_col(s), dv, s * 16 * 128, C::kIdescPV,
                           (!first || s > 0));
                tc_commit(bar(B_O_DONE + x));
            }
            __syncwarp();
            if (x) ++pv_cnt1; else ++pv_cnt0;
            return true;
        };
        auto commit = [&](int b) {
            if (elect_one()) tc_commit(bar(b));
            __syncwarp();
        };
        // V rows that no query of the item may see are undefined, and 0 * NaN is not 0: the
        // first and last key tile's are cleared before the product reads them.
        auto clear_v = [&](uint32_t st, int k) {
            const int c0 = (g.r.f + k) * C::BN;
            const int lo = max(0, g.r.lo - c0), hi = min(C::BN, g.r.hi - c0);
            if (lo == 0 && hi == C::BN) return;
            for (int e = lane; e < C::BN * C::kCB * 8; e += 32) {
                const int row = e / (C::kCB * 8), c = e % (C::kCB * 8);
                if (row < lo || row >= hi)
                    st_shared_v4(sV + st * C::kKVBytes + uint32_t((c >> 3) * C::BN * 128 + row * 128 + (c & 7) * 16), 0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
        };
        while (ok && cur.next(p, g)) {
            if (g.r.n == 0) continue;
            const Steps s = steps_of(p, g);
            const int n = s.k1 - s.k0;
            if (!wwait(B_Q_FULL, item_it & 1)) { ok = false; break; }
            if (!s.split) {
                auto act = [&](int x, int j) { return j >= s.a[x] && j < s.b[x]; };
                {
                    const uint32_t st = kv_it & 1, ph = (kv_it >> 1) & 1;
                    if (!wwait(B_K_FULL + st, ph)) { ok = false; break; }
                    if (act(0, s.k0) && !issue_s(0, st, 0)) { ok = false; break; }
                    if (act(1, s.k0) && !issue_s(1, st, 1)) { ok = false; break; }
                    commit(B_K_EMPTY + st);
                    if (n == 1) commit(B_Q_EMPTY);
                }
                for (int i = 0; i < n && ok; ++i) {
                    const int j = s.k0 + i;
                    const uint32_t t = kv_it + i, st = t & 1, ph = (t >> 1) & 1;
                    const uint32_t t1 = t + 1, st1 = t1 & 1, ph1 = (t1 >> 1) & 1;
                    if (!wwait(B_V_FULL + st, ph)) { ok = false; break; }
                    clear_v(st, j);
                    if (act(0, j) && !issue_pv(0, st, j == s.a[0])) { ok = false; break; }
                    if (i + 1 < n && !wwait(B_K_FULL + st1, ph1)) { ok = false; break; }
                    if (act(0, j + 1) && !issue_s(0, st1, 0)) { ok = false; break; }
                    if (act(1, j) && !issue_pv(1, st, j == s.a[1])) { ok = false; break; }
                    commit(B_V_EMPTY + st);
                    if (act(1, j + 1) && !issue_s(1, st1, 1)) { ok = false; break; }
                    if (i + 1 < n) {
                        commit(B_K_EMPTY + st1);
                        if (i + 2 == n) commit(B_Q_EMPTY);
                    }
                }
            } else {
                // step i: tile x = i & 1 computes P V of step i, then S of step i + 2
                for (int i = 0; i < 2 && i < n && ok; ++i) {
                    const uint32_t t = kv_it + i, st = t & 1, ph = (t >> 1) & 1;
                    if (!wwait(B_K_FULL + st, ph) || !issue_s(i, st, 0)) { ok = false; break; }
                    commit(B_K_EMPTY + st);
                    if (i + 1 == n) commit(B_Q_EMPTY);
                }
                for (int i = 0; i < n && ok; ++i) {
                    const int x = i & 1;
                    const uint32_t t = kv_it + i, st = t & 1, ph = (t >> 1) & 1;
                    const uint32_t t2 = t + 2, st2 = t2 & 1, ph2 = (t2 >> 1) & 1;
                    if (!wwait(B_V_FULL + st, ph)) { ok = false; break; }
                    clear_v(st, s.k0 + i);
                    if (!issue_pv(x, st, i < 2)) { ok = false; break; }
                    commit(B_V_EMPTY + st);
                    if (i + 2 < n) {
                        if (!wwait(B_K_FULL + st2, ph2) || !issue_s(x, st2, 0)) { ok = false; break; }
                        commit(B_K_EMPTY + st2);
                        if (i + 3 == n) commit(B_Q_EMPTY);
                    }
                }
            }
            kv_it += n;
            ++item_it;
            items_x0 += s.count(0) > 0 ? 1 : 0;
            items_x1 += s.count(1) > 0 ? 1 : 0;
        }
        if (!ok && lane == 0) fail();
        commit(B_DRAIN);  // every issued product, before TMEM is released
        mbar_wait_bounded(bar(B_DRAIN), 0, nullptr);
    } else {
        // ------------------------------------------------------------ softmax / epilogue
        const int x = (warp >> 2) & 1, hf = warp >> 3, pair = warp & 7;
        const int t = (warp & 3) * 32 + lane;  // row in the tile == TMEM lane
        constexpr int HC = C::BN / 2, OC = D / 2;
        const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
        const uint32_t tSt = tmem + lane_base + C::tmem_s(x);
        const uint32_t tS = tSt + uint32_t(HC * hf);
        const uint32_t tO = tmem + lane_base + C::tmem_o(x) + uint32_t(OC * hf);
        uint32_t s_cnt = 0, split_cnt = 0, x_cnt = 0, part_cnt = 0;
        float* comb_s = reinterpret_cast<float*>(smem + C::kOffComb);
        float* xch_s = reinterpret_cast<float*>(smem + C::kOffXch);
        auto wwait = [&](int b, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait_bounded(bar(b), parity, abort_flag));
        };
        // The partner warp's value of a per-row float this warp also passes in (spun for
        // inline, bounded, rather than parked: the live scores would be saved around a call).
        auto exchange = [&](float v, float& other) -> bool {
            float* buf = xch_s + (x_cnt & 1) * 512 + pair * 32;
            buf[hf * 256 + lane] = v;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_XCH + pair));
            bool done = false;
            for (uint32_t spin = 0; spin < (1u << 26) && !done; ++spin) {
                done = mbar_try_wait(bar(B_XCH + pair), x_cnt & 1);
                if (!done && (spin & 1023u) == 1023u && *abort_flag) break;
            }
            const bool good = __all_sync(0xffffffffu, done);
            ++x_cnt;
            if (good) other = buf[(hf ^ 1) * 256 + lane];
            return good;
        };
        const float xs = p.scale_log2;
        bool ok = true;
        while (ok && cur.next(p, g)) {
            const Steps sp = steps_of(p, g);
            const int R = g.s.q_len * p.g, diag = g.s.kv_len - g.s.q_len;
            const int n = sp.count(x);
            const int first_k = sp.split ? sp.k0 + x : sp.a[x], stride_k = sp.split ? 2 : 1;
            const int row = (2 * g.tile + (sp.split ? 0 : x)) * C::BM + t;  // packed row
            const bool row_valid = row < R;
            const int rc = min(row, R - 1), tok = rc / p.g, head = g.hk * p.g + rc - tok * p.g;
            const int rel = tok + diag;  // position of the row: rows past the end repeat the last one's masks
            const int t0 = __shfl_sync(0xffffffffu, tok, 0), t31 = __shfl_sync(0xffffffffu, tok, 31);
            const float* brow = BIAS ? p.bias + head * 32 : nullptr;
            const size_t orow = size_t(g.s.q0 + tok) * size_t(p.H) + size_t(head);
            float bmax = 0.f;
            if (BIAS) {
                bmax = -INFINITY;
#pragma unroll 8
                for (int i = 0; i < 32; ++i) bmax = fmaxf(bmax, __ldg(brow + i));
                bmax *= 1.4426950408889634f;
            }
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < n; ++i) {
                const int col0 = (g.r.f + first_k + i * stride_k) * C::BN;
                int lim = g.s.kv_len - col0;
                if (p.causal) lim = min(lim, rel + 1 - col0);
                const int lo = p.window >= 0 ? rel - p.window - col0 : 0;
                const bool full = __all_sync(0xffffffffu, lim >= C::BN && lo <= 0);
                // Bias per 32-column chunk: one value per row when every row's positions of
                // the chunk share a bucket, else looked up per element.
                uint32_t hmask = 3u;
                float cb[2] = {0.f, 0.f};
                if (BIAS) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int c = col0 + 32 * (2 * hf + k);
                        const int far = t31 + diag - c, near = t0 + diag - c - 31;
                        const int bk = relpos_bucket(far);
                        const bool one = (near >= 0 || far <= 0) && bk == relpos_bucket(near);
                        if (!one) hmask &= ~(1u << k);
                        cb[k] = __ldg(brow + bk) * 1.4426950408889634f;
                    }
                }
                if (!wwait(B_S_FULL + x, s_cnt & 1)) { ok = false; break; }
                tc_fence_after();
                uint32_t sr[2][32];
                tmem_ld32(tS, sr[0]);
                tmem_ld32(tS + 32u, sr[1]);
                // in place: scaled, biased and masked scores of chunk k, minus `shift`
                auto to_x = [&](uint32_t (&r)[32], int k, float shift) {
                    const int kk = 2 * hf + k;
                    if (!BIAS || (hmask & (1u << k))) {
                        const float2 sc = make_float2(xs, xs), add = make_float2(cb[k] - shift, cb[k] - shift);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float2 t2 = fma2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), sc, add);
                            r[e] = __float_as_uint(t2.x);
                            r[e + 1] = __float_as_uint(t2.y);
                        }
                    } else {
                        const int rk = rel - col0 - 32 * kk;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float bv = __ldg(brow + relpos_bucket(rk - e));
                            r[e] = __float_as_uint(fmaf(__uint_as_float(r[e]), xs, fmaf(bv, 1.4426950408889634f, -shift)));
                        }
                    }
                    if (!full) {
                        const int lk = lim - 32 * kk, lok = lo - 32 * kk;
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[e] = (e >= lok && e < lk) ? r[e] : __float_as_uint(-INFINITY);
                    }
                };
                tmem_ld_wait(sr[0]);
                tmem_ld_wait(sr[1]);
                // pass 1: an upper bound of this half's row maximum from the raw scores
                float mx = -INFINITY;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int kk = 2 * hf + k;
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    if (full) {
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], __uint_as_float(sr[k][e]), __uint_as_float(sr[k][e + 1]));
                    } else {
                        const int lk = lim - 32 * kk, lok = lo - 32 * kk;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            m4[e & 3] = fmaxf(m4[e & 3], (e >= lok && e < lk) ? __uint_as_float(sr[k][e]) : -INFINITY);
                    }
                    const float mk = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    mx = fmaxf(mx, fmaf(mk, xs, (hmask & (1u << k)) ? cb[k] : bmax));
                }
                float mo;
                if (!exchange(mx, mo)) { ok = false; break; }
                mx = fmaxf(mx, mo);
                // the running maximum moves only when it would grow by more than 2^8
                float m_new = m;
                if (mx > m + 8.f) m_new = mx;
                const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
                const float alpha = (m == -INFINITY) ? 0.f : ex2_approx(m - m_use);
                const bool need_rescale = (m_new != m) && i > 0;
                m = m_new;
                if (__any_sync(0xffffffffu, need_rescale)) {
#pragma unroll 1
                    for (int c = 0; c < OC / 8; ++c) {
                        uint32_t r[8];
                        tmem_ld8(tO + c * 8u, r);
                        tmem_ld_wait(r);
#pragma unroll
                        for (int e = 0; e < 8; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
                        tmem_st8(tO + c * 8u, r);
                    }
                }
                // pass 2: P = exp2(x - m), its sum in fp32, and bf16 P over the scores
                float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                tmem_ld32(tS, sr[0]);  // the raw scores again: cheaper than 64 live registers
                tmem_ld32(tS + 32u, sr[1]);
                tmem_ld_wait(sr[0]);
                tmem_ld_wait(sr[1]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int kk = 2 * hf + k;
                    uint32_t pk[16];
                    if (full && (!BIAS || (hmask & (1u << k)))) {
                        const float2 xs2 = make_float2(xs, xs), add = make_float2(cb[k] - m_use, cb[k] - m_use);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float2 t2 = fma2(make_float2(__uint_as_float(sr[k][e]), __uint_as_float(sr[k][e + 1])), xs2, add);
                            const float2 e2 = make_float2(ex2_approx(t2.x), ex2_approx(t2.y));
                            rs[(e >> 1) & 1] = add2(rs[(e >> 1) & 1], e2);
                            pk[e >> 1] = pack_bf16x2(e2.x, e2.y);
                        }
                    } else {
                        to_x(sr[k], k, m_use);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float2 e2 = make_float2(ex2_approx(__uint_as_float(sr[k][e])), ex2_approx(__uint_as_float(sr[k][e + 1])));
                            rs[(e >> 1) & 1] = add2(rs[(e >> 1) & 1], e2);
                            pk[e >> 1] = pack_bf16x2(e2.x, e2.y);
                        }
                    }
                    tmem_st16(tSt + 32u * kk, pk);
                }
                const float2 r01 = add2(rs[0], rs[1]);
                l = l * alpha + (r01.x + r01.y);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_P_FULL + x));
                ++s_cnt;
            }
            if (!ok) break;
            const bool whole = g.whole();
            if (n > 0) {
                if (!wwait(B_O_DONE + x, (s_cnt - 1) & 1)) { ok = false; break; }
                tc_fence_after();
            }
            // m, lt: the row's maximum and sum; O is O_A c0 (+ O_B c1 for a split item)
            float lt = l, c0 = 1.f, c1 = 0.f;
            if (n > 0) {
                float other;
                if (!exchange(l, other)) { ok = false; break; }
                lt = l + other;
            }
            const bool two = sp.split && sp.count(1) > 0;
            if (two) {
                float* comb = comb_s + (split_cnt & 1) * 2 * C::BM;
                ++split_cnt;
                if (x == 1) {
                    if (hf == 0) {
                        comb[t] = m;
                        comb[C::BM + t] = lt;
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_COMBINE));
                } else {
                    if (!wwait(B_COMBINE, (split_cnt - 1) & 1)) { ok = false; break; }
                    tc_fence_after();
                    const float m1 = comb[t], l1 = comb[C::BM + t], mm = fmaxf(m, m1);
                    c0 = m == -INFINITY ? 0.f : ex2_approx(m - mm);
                    c1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - mm);
                    lt = fmaf(lt, c0, l1 * c1);
                    m = mm;
                }
            }
            const bool owner = !sp.split || x == 0;  // tile B of a split item hands over to tile A
            // this row's values of columns OC hf + 32 c .. + 32, times mul
            auto load_o = [&](int c, float mul, float (&v)[32]) {
                if (n == 0) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.f;
                    return;
                }
                uint32_t r0[32];
                tmem_ld32(tO + c * 32u, r0);
                tmem_ld_wait(r0);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r0[e]) * (c0 * mul);
                if (two) {
                    tmem_ld32(tO + (C::tmem_o(1) - C::tmem_o(0)) + c * 32u, r0);
                    tmem_ld_wait(r0);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = fmaf(__uint_as_float(r0[e]), c1 * mul, v[e]);
                }
            };
            auto release = [&]() {
                if (n == 0) return;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(B_O_EMPTY + x));
                    if (two) mbar_arrive(bar(B_O_EMPTY + 1));
                }
            };
            auto put = [&](int col, const float* v, int cnt) {  // this row's output columns col .. col + cnt
                if (!row_valid) return;
                if (p.o_f32) {
                    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.O) + orow * D + col);
#pragma unroll
                    for (int e = 0; e < cnt / 4; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.O) + orow * D + col);
#pragma unroll
                    for (int e = 0; e < cnt / 8; ++e)
                        dst[e] = make_uint4(pack_bf16x2(v[8 * e], v[8 * e + 1]), pack_bf16x2(v[8 * e + 2], v[8 * e + 3]),
                                            pack_bf16x2(v[8 * e + 4], v[8 * e + 5]), pack_bf16x2(v[8 * e + 6], v[8 * e + 7]));
                }
            };
            if (whole) {
                if (!owner) continue;
                const float inv = lt > 0.f ? 1.f / lt : 0.f;
#pragma unroll
                for (int c = 0; c < OC / 32; ++c) {
                    float v[32];
                    load_o(c, inv, v);
                    put(OC * hf + 32 * c, v, 32);
                }
                release();
                if (row_valid && p.lse && hf == 0)
                    p.lse[orow] = lt > 0.f ? (m + __log2f(lt)) * 0.6931471805599453f : -INFINITY;
                continue;
            }
            // An item split over CTAs: leave this part, count it, and the last one to arrive
            // adds them all up in the order of the keys.
            const int first = cache_cta_of(*start, g.first), last = cache_cta_of(*start, g.first + g.units - 1);
            const int prow = sp.split ? t : x * C::BM + t;  // row of the pair
            if (owner) {
                float* part = p.part + size_t(cache_slot(blockIdx.x, first)) * C::kPart;
                float4* po = reinterpret_cast<float4*>(part);
                if (n > 0) {
#pragma unroll
                    for (int c = 0; c < OC / 32; ++c) {
                        float v[32];
                        load_o(c, 1.f, v);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            po[((OC * hf + 32 * c) / 4 + e) * C::kPair + prow] =
                                make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    }
                    release();
                }
                if (hf == 0) {
                    part[C::kPair * D + prow] = m;
                    part[C::kPair * D + C::kPair + prow] = n > 0 ? lt : 0.f;
                }
                __threadfence();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_PART));
            if (threadIdx.x == 0) {
                int done = 0;
                if (mbar_wait_bounded(bar(B_PART), part_cnt & 1, abort_flag)) {
                    __threadfence();
                    done = atomicAdd(p.counters + first, 1u) == uint32_t(last - first);
                    if (done) p.counters[first] = 0u;  // every part has arrived: ready for the next call
                    __threadfence();
                }
                *last_flag = done;
                mbar_arrive(bar(B_FLAG));
            }
            __syncwarp();
            if (!wwait(B_FLAG, part_cnt & 1)) { ok = false; break; }
            ++part_cnt;
            if (!*last_flag || !owner) continue;
            const float* pm = p.part + C::kPair * D + prow;
            float mm = -INFINITY, ll = 0.f;
#pragma unroll 4
            for (int c = first; c <= last; ++c) mm = fmaxf(mm, __ldcg(pm + size_t(cache_slot(c, first)) * C::kPart));
#pragma unroll 4
            for (int c = first; c <= last; ++c) {
                const float* q = pm + size_t(cache_slot(c, first)) * C::kPart;
                const float mc = __ldcg(q);
                ll = fmaf(__ldcg(q + C::kPair), mc == -INFINITY ? 0.f : ex2_approx(mc - mm), ll);
            }
            const float inv = ll > 0.f ? 1.f / ll : 0.f;
#pragma unroll 1
            for (int c8 = 0; c8 < OC / 16; ++c8) {
                float v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = 0.f;
#pragma unroll 2
                for (int c = first; c <= last; ++c) {
                    const float* q = p.part + size_t(cache_slot(c, first)) * C::kPart;
                    const float mc = __ldcg(q + C::kPair * D + prow);
                    if (mc == -INFINITY) continue;  // no key of this part: its O is not set
                    const float w = ex2_approx(mc - mm) * inv;
                    const float4* q4 = reinterpret_cast<const float4*>(q) + ((OC * hf) / 4 + 4 * c8) * C::kPair + prow;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 u = __ldcg(q4 + e * C::kPair);
                        v[4 * e] = fmaf(u.x, w, v[4 * e]);
                        v[4 * e + 1] = fmaf(u.y, w, v[4 * e + 1]);
                        v[4 * e + 2] = fmaf(u.z, w, v[4 * e + 2]);
                        v[4 * e + 3] = fmaf(u.w, w, v[4 * e + 3]);
                    }
                }
                put(OC * hf + 16 * c8, v, 16);
            }
            if (row_valid && p.lse && hf == 0)
                p.lse[orow] = ll > 0.f ? (mm + __log2f(ll)) * 0.6931471805599453f : -INFINITY;
        }
        if (!ok && lane == 0) fail();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == C::kMmaWarp) tmem_dealloc(tmem, C::kTmemCols);
}

template <int D, bool BIAS>
cudaError_t launch(const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, int num_sms, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(jfa_cache_chunk_kernel<D, BIAS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         ChkCfg<D>::kSmemBytes);
    if (e != cudaSuccess) return e;
    jfa_cache_chunk_kernel<D, BIAS><<<num_sms, ChkCfg<D>::kThreads, ChkCfg<D>::kSmemBytes, st>>>(mk, mv, p);
    return cudaGetLastError();
}

}  // namespace

size_t cache_chunk_part_bytes(int D, int num_sms) { return size_t(num_sms) * 2 * 256 * size_t(D + 2) * 4; }

cudaError_t launch_cache_chunk(int D, const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, int num_sms,
                               cudaStream_t st) {
    if (D == 128) return p.bias ? launch<128, true>(mk, mv, p, num_sms, st) : launch<128, false>(mk, mv, p, num_sms, st);
    return p.bias ? launch<64, true>(mk, mv, p, num_sms, st) : launch<64, false>(mk, mv, p, num_sms, st);
}

}  // namespace jfa
