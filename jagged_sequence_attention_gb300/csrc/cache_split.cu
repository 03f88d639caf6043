// Paged-cache attention for chunks of new tokens, fp32: tensor-core products of operands split
// into three bf16 parts each.
//
// x = x0 + x1 + x2 with x0 = bf16(x), x1 = bf16(x - x0), x2 = bf16(x - x0 - x1): both
// differences are exact in fp32, |x1| <= 2^-8 and |x2| <= 2^-17 of x's power of two, and the
// three parts hold x exactly (8 + 8 + 7 of its 24 bits and the signs).  A product of two split
// values keeps
//   x0 y0 + (x0 y1 + x1 y0) + (x1 y1 + x0 y2 + x2 y0),
// leaving out x1 y2 + x2 y1 + x2 y2, together at most 2^-24 of the product (two terms of 2^-25):
// each product is as exact as fp32's own rounding.  The tensor core accumulates in fp32, but not
// with rounding to nearest, so two things keep its sums at fp32's level: the small terms go first,
// while the accumulator is small, and leave only the x0 y0 steps (4 for a score, 8 for an output)
// to the full-size accumulator; and the output of each key tile starts from zero and is added to
// the running one in registers.
// Six bf16 products at 16 times and more the rate of the FMA units.  A step of 128 rows x 128
// keys takes 2.5 us: 2.1 of products (24 + 48 instructions of M = 128, those of P V at the half
// rate of N = 64), the rest the chain output -> P -> output of a step, as TMEM holds one P and
// one output.  Measured: 20 sequences of 200-4000 keys, 5 of them prompts of 100-600 tokens (8
// query, 4 key heads of 64) 75 us, of which this kernel 47 (its 1788 steps over 152 CTAs are 29),
// the single tokens' 20 and the merge 8.
//
// An item is 128 packed rows of one (sequence, key head); a step is 128 keys.  Head dimension
// 32 runs as 64 with zeros.  CTA = 16 warps, one CTA per SM:
//   warps 0-7    softmax: two warps share a row, 64 score columns and 32 output columns each
//   warps 8-13   split Q (from global memory) and the K and V tiles that TMA left in shared
//                memory, and write the parts' swizzled tiles; K a step ahead of V, since each
//                step's K parts wait for the step before's scores and its V parts for the
//                step before's output (in the order of the steps: 4.4 us a step)
//   warp 14      tcgen05.mma issuer and TMEM owner
//   warp 15      TMA loads of K and V, a tile of each ahead (one box per page and 128 bytes of a
//               row): 64 KB in flight, which loads through registers would not reach
// TMEM (512 columns): scores twice [0,128), [128,256), so that a tile's scores form during the
// previous one's softmax; P's parts [256,448); the tile's output [448,512).
#include "cache_common.cuh"
#include "tilemath.cuh"

namespace jfa {

namespace {

constexpr int kSpBM = 128, kSpBN = 128, kSpD = 64;

struct SpCfg {
    static constexpr int kPlane = 128 * 128;        // one part of a tile: 128 rows of 64 bf16
    static constexpr int kTile = 3 * kPlane;
    static constexpr int kOffQ = 0, kOffK = kTile, kOffV = kOffK + kTile;
    static constexpr int kStageBlock = 128 * 128;   // fp32 tile as loaded: 128 rows of 32 floats, twice
    static constexpr int kOffKS = kOffV + kTile, kOffVS = kOffKS + 2 * kStageBlock;
    static constexpr int kOffBar = kOffVS + 2 * kStageBlock;
    static constexpr int kOffMisc = kOffBar + 32 * 8;
    static constexpr int kOffXch = kOffMisc + 16;   // pair exchanges [2][2][4][32]
    static constexpr int kOffSums = kOffXch + 2 * 2 * 4 * 32 * 4;  // scratch of the work split
    static constexpr int kBytes = kOffSums + kCacheMaxGroups * 4 + 1024;
    static constexpr int kSoftWarps = 8, kSplitWarps = 6, kMmaWarp = 14, kTmaWarp = 15,
                         kThreads = 16 * 32;
    static constexpr uint32_t kTmemCols = 512, kP = 256, kO = 448;
    static constexpr uint32_t kIdescQK = make_idesc(kFmtBF16, 128, 128, false, false);
    static constexpr uint32_t kIdescPV = make_idesc(kFmtBF16, 128, kSpD, false, true);
};

enum {
    P_Q_FULL = 0,
    P_Q_EMPTY,
    P_K_FULL,
    P_K_EMPTY,
    P_V_FULL,
    P_V_EMPTY,
    P_P_FULL,
    P_O_DONE,
    P_DRAIN,
    P_S_FULL,                // +buffer
    P_S_EMPTY = P_S_FULL + 2,
    P_XCH = P_S_EMPTY + 2,   // +pair of warps
    P_KS_FULL = P_XCH + 4,   // K as loaded
    P_KS_EMPTY,
    P_VS_FULL,
    P_VS_EMPTY,
};

// The six products of split operands, the small ones first: (part of A, part of B).
__device__ __forceinline__ constexpr int term_a(int t) { return t == 0 ? 1 : t == 1 ? 0 : t == 2 ? 2 : t == 3 ? 0 : t == 4 ? 1 : 0; }
__device__ __forceinline__ constexpr int term_b(int t) { return t == 0 ? 1 : t == 1 ? 2 : t == 2 ? 0 : t == 3 ? 1 : 0; }

// Two values' three parts, each pair packed.
__device__ __forceinline__ void split2(float x, float y, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
    p0 = pack_bf16x2(x, y);
    const float rx = x - __uint_as_float(p0 << 16), ry = y - __uint_as_float(p0 & 0xffff0000u);
    p1 = pack_bf16x2(rx, ry);
    p2 = pack_bf16x2(rx - __uint_as_float(p1 << 16), ry - __uint_as_float(p1 & 0xffff0000u));
}

// The steps of a CTA's range, one key tile after the other.
struct SplitStream {
    CacheCursor<kSpBN> cur;
    CacheSeg g;
    int k;         // the step's key tile of its item
    uint32_t it;   // steps and items begun before it
    uint32_t item;
    bool have;
    __device__ explicit SplitStream(const CacheCursor<kSpBN>& c) : cur(c), k(0), it(0), item(0), have(false) {}
    __device__ void advance(const CacheFwdParams& p) {  // to the next step; its number is counted by the caller
        if (have && ++k < g.k1) return;
        if (have) ++item;
        do {
            have = cur.next(p, g);
        } while (have && g.r.n == 0);
        if (have) k = g.k0;
    }
};

// Four elements of row r, the piece-th four, to the parts' tiles at `dst`.
__device__ __forceinline__ void put_parts(uint32_t dst, int r, int piece, const float4& v) {
    uint32_t w[3][2];
    split2(v.x, v.y, w[0][0], w[1][0], w[2][0]);
    split2(v.z, v.w, w[0][1], w[1][1], w[2][1]);
    const uint32_t at = dst + uint32_t(r * 128 + (((piece >> 1) ^ (r & 7)) << 4) + (piece & 1) * 8);
#pragma unroll
    for (int q = 0; q < 3; ++q)
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + uint32_t(q * SpCfg::kPlane)), "r"(w[q][0]), "r"(w[q][1])
                     : "memory");
}

// A thread's rows of a loaded tile at `src`, in parts to `dst`; zeros but for rows [lo, hi), as
// no row of the item may look there.  Three rows' loads at once, ahead of the stores that the
// compiler keeps them in order with.  (Not inlined: the warps of an SM fetch code from many
// places at a time.)
template <int D>
__device__ __noinline__ void split_rows(uint32_t src, uint32_t dst, int lo, int hi, int row0, int c) {
    constexpr int kStep = 4 * SpCfg::kSplitWarps;
#pragma unroll 1
    for (int r0 = row0; r0 < 128; r0 += 3 * kStep) {
        uint4 u[3][D / 32];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int r = min(r0 + i * kStep, 127);
#pragma unroll
            for (int h = 0; h < D / 32; ++h)
                u[i][h] = ld_shared_v4(src + uint32_t(h * SpCfg::kStageBlock + r * 128 + ((c ^ (r & 7)) << 4)));
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int r = r0 + i * kStep;
            if (r >= 128) break;
            const bool in = r >= lo && r < hi;
#pragma unroll
            for (int h = 0; h < D / 32; ++h)
                put_parts(dst, r, c + 8 * h,
                          in ? make_float4(__uint_as_float(u[i][h].x), __uint_as_float(u[i][h].y), __uint_as_float(u[i][h].z),
                                           __uint_as_float(u[i][h].w))
                             : make_float4(0.f, 0.f, 0.f, 0.f));
        }
    }
}

template <int D, bool BIAS>
__global__ void __launch_bounds__(SpCfg::kThreads, 1)
    jfa_cache_split_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                           const CacheFwdParams p) {
    using C = SpCfg;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) -> uint32_t { return sbase + C::kOffBar + 8u * uint32_t(i); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(bar(P_Q_FULL), C::kSplitWarps);
        mbar_init(bar(P_Q_EMPTY), 1);
        mbar_init(bar(P_K_FULL), C::kSplitWarps);
        mbar_init(bar(P_K_EMPTY), 1);
        mbar_init(bar(P_V_FULL), C::kSplitWarps);
        mbar_init(bar(P_V_EMPTY), 1);
        mbar_init(bar(P_P_FULL), C::kSoftWarps);
        mbar_init(bar(P_O_DONE), 1);
        mbar_init(bar(P_DRAIN), 1);
        mbar_init(bar(P_KS_FULL), 1);
        mbar_init(bar(P_KS_EMPTY), C::kSplitWarps);
        mbar_init(bar(P_VS_FULL), 1);
        mbar_init(bar(P_VS_EMPTY), C::kSplitWarps);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(P_S_FULL + s), 1);
            mbar_init(bar(P_S_EMPTY + s), C::kSoftWarps);
        }
        for (int q = 0; q < 4; ++q) mbar_init(bar(P_XCH + q), 2);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (D == 32)  // the parts' upper columns stay zero
        for (int e = threadIdx.x; e < 9 * 128 * 4; e += C::kThreads) {
            const int row = e >> 2, c = 4 + (e & 3);
            st_shared_v4(sbase + uint32_t(row * 128 + ((c ^ (row & 7)) << 4)), 0, 0, 0, 0);
        }
    if (warp == C::kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    CacheCursor<kSpBN> cur(p, cache_start<kSpBN>(p, reinterpret_cast<int*>(smem + C::kOffSums)));
    const CacheStart start = cur.st;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    launch_dependents();  // the kernel for few rows may fill SMs as they come free
    CacheSeg g;
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(p.status, kStatusTimeout);
    };
    auto wwait = [&](int b, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_bounded(bar(b), parity, abort_flag));
    };
    bool ok = true;

    if (warp == C::kMmaWarp) {
        // ------------------------------------------------------------ MMA issuer
        uint32_t it = 0, item_it = 0;  // steps and items so far
        const SDesc dQ = sdesc_sw128(sbase + C::kOffQ, 16, 1024), dK = sdesc_sw128(sbase + C::kOffK, 16, 1024);
        const SDesc dV = sdesc_sw128(sbase + C::kOffV, 128 * 128, 1024);
        auto commit = [&](int b) {
            if (elect_one()) tc_commit(bar(b));
            __syncwarp();
        };
        auto issue_s = [&](uint32_t i) -> bool {  // scores of step i into buffer i & 1
            const uint32_t x = i & 1, use = i >> 1;
            if (!wwait(P_K_FULL, i & 1) || !wwait(P_S_EMPTY + x, (use & 1) ^ 1)) return false;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int t = 0; t < 6; ++t)
#pragma unroll
                    for (int s = 0; s < kSpD / 16; ++s)
                        mma_ss(tmem + 128u * x, dQ, term_a(t) * C::kPlane + s * 32, dK, term_b(t) * C::kPlane + s * 32,
                               C::kIdescQK, t > 0 || s > 0);
                tc_commit(bar(P_S_FULL + x));
            }
            __syncwarp();
            commit(P_K_EMPTY);
            return true;
        };
        while (ok && cur.next(p, g)) {
            const int n = g.r.n > 0 ? g.k1 - g.k0 : 0;
            if (n == 0) continue;
            if (!wwait(P_Q_FULL, item_it & 1) || !issue_s(it)) { ok = false; break; }
            if (n == 1) commit(P_Q_EMPTY);
            for (int j = 0; j < n && ok; ++j) {
                const uint32_t i = it + j;
                if (j + 1 < n) {
                    if (!issue_s(i + 1)) { ok = false; break; }
                    if (j + 2 == n) commit(P_Q_EMPTY);
                }
                if (!wwait(P_V_FULL, i & 1) || !wwait(P_P_FULL, i & 1)) { ok = false; break; }
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int t = 0; t < 6; ++t)
#pragma unroll
                        for (int s = 0; s < kSpBN / 16; ++s)
                            mma_ts(tmem + C::kO, tmem + C::kP + 64u * term_a(t) + 8u * s, dV,
                                   term_b(t) * C::kPlane + s * 16 * 128, C::kIdescPV, t > 0 || s > 0);
                    tc_commit(bar(P_O_DONE));
                }
                __syncwarp();
                commit(P_V_EMPTY);
            }
            it += n;
            ++item_it;
        }
        if (!ok && lane == 0) fail();
        commit(P_DRAIN);  // every issued product, before TMEM is released
        mbar_wait_bounded(bar(P_DRAIN), 0, nullptr);
    } else if (warp == C::kTmaWarp) {
        // ------------------------------------------------------------ loads
        const int rows = min(1 << p.page_log2, 64), per = kSpBN / rows;  // keys of a box, boxes of a column block
        const int mask = (1 << p.page_log2) - 1;
        // K and V are loaded in turn, K a step ahead: its tile is split, and its memory free
        // again, before V's.
        auto issue = [&](SplitStream& s, int full, int empty, int stage, const CUtensorMap* map) -> bool {
            // lane: a page of the tile (two column blocks of it)
            const int j = (s.g.r.f + s.k) * kSpBN + lane * rows;
            int page = -1;
            if (lane < per && j < s.g.r.hi && j + rows > s.g.r.lo) {
                page = p.table[size_t(s.g.b) * size_t(p.max_pages) + size_t(j >> p.page_log2)];
                if (page < 0 || page >= p.n_pages) {
                    atomicOr(p.status, kStatusBounds);
                    page = p.n_pages;  // past the cache: read as zeros
                }
            }
            const uint32_t bytes = uint32_t(__popc(__ballot_sync(0xffffffffu, page >= 0)) * rows * 128 * (D / 32));
            if (!wwait(empty, (s.it & 1) ^ 1)) return false;
            if (lane == 0) mbar_arrive_expect_tx(bar(full), bytes);
            __syncwarp();
            if (page >= 0)
#pragma unroll
                for (int h = 0; h < D / 32; ++h)
                    tma_load_4d(sbase + uint32_t(stage + h * C::kStageBlock + lane * rows * 128), map, bar(full), 32 * h, j & mask,
                                s.g.hk, page);
            ++s.it;
            return true;
        };
        SplitStream ks{cur}, vs{cur};
        ks.advance(p);
        vs.advance(p);
        for (bool first = true; vs.have && ok; first = false) {
            if (ks.have) {
                ok = issue(ks, P_KS_FULL, P_KS_EMPTY, C::kOffKS, &tmK);
                ks.advance(p);
                if (first) continue;
            }
            if (ok) ok = issue(vs, P_VS_FULL, P_VS_EMPTY, C::kOffVS, &tmV);
            vs.advance(p);
        }
        if (!ok && lane == 0) fail();
        drain_ring(bar(P_KS_FULL), ks.it, 1);
        drain_ring(bar(P_VS_FULL), vs.it, 1);
    } else if (warp >= C::kSoftWarps) {
        // ------------------------------------------------------------ splits
        const int tid = threadIdx.x - 32 * C::kSoftWarps;
        constexpr int kStep = 4 * C::kSplitWarps;
        const int c = tid & 7, row0 = tid >> 3;  // elements 4 c .. and 32 + 4 c .. of rows row0 + kStep i
        auto arrive = [&](int full) {
            fence_proxy_async_smem();  // before the products read them
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(full));
        };
        auto split_tile = [&](SplitStream& s, int staged, int full, int stage, int off) {
            const uint32_t ph = s.it & 1;
            if (!wwait(staged, ph) || !wwait(full + 1, ph ^ 1)) return false;
            const int c0 = (s.g.r.f + s.k) * kSpBN;
            split_rows<D>(sbase + uint32_t(stage), sbase + uint32_t(off), s.g.r.lo - c0, s.g.r.hi - c0, row0, c);
            arrive(full);
            if (lane == 0) mbar_arrive(bar(staged + 1));
            ++s.it;
            s.advance(p);
            return true;
        };
        auto split_q = [&](const SplitStream& s) {
            const int R = s.g.s.q_len * p.g, r0 = s.g.tile * kSpBM;
            if (!wwait(P_Q_EMPTY, (s.item & 1) ^ 1)) return false;
#pragma unroll 3
            for (int r = row0; r < 128; r += kStep) {
                float4 v[D / 32];
#pragma unroll
                for (int h = 0; h < D / 32; ++h) v[h] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r0 + r < R) {
                    const int tok = div_g(p, r0 + r);
                    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.Q) + (s.g.s.q0 + tok) * p.q_stride +
                                                                        int64_t(s.g.hk * p.g + r0 + r - tok * p.g) * D);
#pragma unroll
                    for (int h = 0; h < D / 32; ++h) v[h] = src[c + 8 * h];
                }
#pragma unroll
                for (int h = 0; h < D / 32; ++h) put_parts(sbase + C::kOffQ, r, c + 8 * h, v[h]);
            }
            arrive(P_Q_FULL);
            return true;
        };
        SplitStream ks(cur), vs(cur);
        ks.advance(p);
        vs.advance(p);
        if (vs.have) ok = split_q(vs);
        for (bool first = true; vs.have && ok; first = false) {
            if (ks.have) {
                ok = split_tile(ks, P_KS_FULL, P_K_FULL, C::kOffKS, C::kOffK);
                if (first) continue;
            }
            const uint32_t item = vs.item;
            if (ok) ok = split_tile(vs, P_VS_FULL, P_V_FULL, C::kOffVS, C::kOffV);
            if (ok && vs.have && vs.item != item) ok = split_q(vs);
        }
        if (!ok && lane == 0) fail();
    } else {
        // ------------------------------------------------------------ softmax / output
        const int hf = warp >> 2, pair = warp & 3, t = pair * 32 + lane;
        const uint32_t lane_base = uint32_t(pair * 32) << 16;
        const uint32_t tO = tmem + lane_base + C::kO + 32u * hf, tP = tmem + lane_base + C::kP;
        float* xch_s = reinterpret_cast<float*>(smem + C::kOffXch);
        uint32_t it = 0, x_cnt = 0;
        auto exchange = [&](float v, float& other) -> bool {
            float* buf = xch_s + (x_cnt & 1) * 256 + pair * 32;
            buf[hf * 128 + lane] = v;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(P_XCH + pair));
            const bool good = wwait(P_XCH + pair, x_cnt & 1);
            ++x_cnt;
            if (good) other = buf[(hf ^ 1) * 128 + lane];
            return good;
        };
        while (ok && cur.next(p, g)) {
            const int n = g.r.n > 0 ? g.k1 - g.k0 : 0;
            const int R = g.s.q_len * p.g, diag = g.s.kv_len - g.s.q_len, r0 = g.tile * kSpBM;
            const bool row_valid = r0 + t < R;
            const int rc = min(r0 + t, R - 1), tok = div_g(p, rc), head = g.hk * p.g + rc - tok * p.g;
            const int rel = tok + diag;  // rows past the end repeat the last one's masks
            const int t0 = __shfl_sync(0xffffffffu, tok, 0), t31 = __shfl_sync(0xffffffffu, tok, 31);
            const float* brow = BIAS ? p.bias + head * 32 : nullptr;
            const size_t orow = size_t(g.s.q0 + tok) * size_t(p.H) + size_t(head);
            float m = -INFINITY, l = 0.f, o[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.f;
            // the output of the step before, added and brought to the new maximum
            auto add_o = [&](float alpha) {
                uint32_t r[32];
                tmem_ld32(tO, r);
                tmem_ld_wait(r);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = (o[e] + __uint_as_float(r[e])) * alpha;
            };
            for (int j = 0; j < n; ++j) {
                const uint32_t i = it + j, x = i & 1;
                const int col0 = (g.r.f + g.k0 + j) * kSpBN + 64 * hf;  // this warp's first key
                int lim = g.s.kv_len - col0;
                if (p.causal) lim = min(lim, rel + 1 - col0);
                const int lo = p.window >= 0 ? rel - p.window - col0 : 0;
                const bool full = __all_sync(0xffffffffu, lim >= 64 && lo <= 0);
                if (!wwait(P_S_FULL + x, (i >> 1) & 1)) { ok = false; break; }
                tc_fence_after();
                const uint32_t tS = tmem + lane_base + 128u * x + 64u * hf;
                // scaled, biased and masked scores of columns 32 k .. + 32 of this half; read twice
                // (for the maximum, then for P), so that 32 are held at a time
                auto scores = [&](int k, uint32_t (&r)[32]) {
                    tmem_ld32(tS + 32u * k, r);
                    const int rk = rel - col0 - 32 * k;
                    const int far = t31 + diag - col0 - 32 * k, near = t0 + diag - col0 - 32 * k - 31;
                    const int bk = BIAS ? relpos_bucket(far) : 0;
                    const bool one = !BIAS || ((near >= 0 || far <= 0) && bk == relpos_bucket(near));
                    const float b1 = BIAS ? __ldg(brow + bk) * 1.4426950408889634f : 0.f;
                    tmem_ld_wait(r);
                    if (one) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            r[e] = __float_as_uint(BIAS ? fmaf(__uint_as_float(r[e]), p.scale_log2, b1) : __uint_as_float(r[e]) * p.scale_log2);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            r[e] = __float_as_uint(fmaf(__uint_as_float(r[e]), p.scale_log2,
                                                        __ldg(brow + relpos_bucket(rk - e)) * 1.4426950408889634f));
                    }
                    if (!full) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (e + 32 * k < lo || e + 32 * k >= lim) r[e] = __float_as_uint(-INFINITY);
                    }
                };
                float mx = -INFINITY;
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    uint32_t r[32];
                    scores(k, r);
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
                    mx = fmaxf(mx, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
                }
                float mo;
                if (!exchange(mx, mo)) { ok = false; break; }
                const float m_new = fmaxf(m, fmaxf(mx, mo)), m_use = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = m == -INFINITY ? 0.f : ex2_approx(m - m_use);
                m = m_new;
                if (j > 0) {  // P's columns and the output are free once the product before is done
                    if (!wwait(P_O_DONE, (i - 1) & 1)) { ok = false; break; }
                    tc_fence_after();
                    add_o(alpha);
                }
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    uint32_t r[32];
                    scores(k, r);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t w[3][8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float2 y = make_float2(ex2_approx(__uint_as_float(r[16 * h + 2 * e]) - m_use),
                                                         ex2_approx(__uint_as_float(r[16 * h + 2 * e + 1]) - m_use));
                            sum = add2(sum, y);
                            split2(y.x, y.y, w[0][e], w[1][e], w[2][e]);
                        }
#pragma unroll
                        for (int q = 0; q < 3; ++q) tmem_st8(tP + 64u * q + 32u * hf + 16u * k + 8u * h, w[q]);
                    }
                }
                l = fmaf(l, alpha, sum.x + sum.y);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(P_S_EMPTY + x));
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(P_P_FULL));
            }
            if (!ok) break;
            it += n;
            float lt = l;
            if (n > 0) {
                if (!wwait(P_O_DONE, (it - 1) & 1)) { ok = false; break; }
                tc_fence_after();
                add_o(1.f);
                // (the next item's first product waits for its P, which these warps write)
                tc_fence_before();
                float other;
                if (!exchange(l, other)) { ok = false; break; }
                lt = l + other;
            }
            if (g.whole()) {
                const float inv = lt > 0.f ? 1.f / lt : 0.f;
                if (32 * hf < D && row_valid) {
                    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.O) + orow * D + 32 * hf);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e] = make_float4(o[4 * e] * inv, o[4 * e + 1] * inv, o[4 * e + 2] * inv, o[4 * e + 3] * inv);
                }
                if (p.lse && hf == 0 && row_valid) p.lse[orow] = lt > 0.f ? (m + log2f(lt)) * 0.6931471805599453f : -INFINITY;
                continue;
            }
            // an item cut between CTAs: this part, and with the first one the merge's record
            const int first = cache_first_cta(p, start, g), last = cache_last_cta(p, start, g);
            float* part = p.part + size_t(cache_slot(blockIdx.x, first)) * cache_merge_part(D);
            if (row_valid) {
                if (32 * hf < D) {
                    float4* po = reinterpret_cast<float4*>(part);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        po[(8 * hf + e) * kMergeRows + t] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
                if (hf == 0) {
                    part[kMergeRows * D + t] = m;
                    part[kMergeRows * D + kMergeRows + t] = lt;
                }
            }
            const int rows = min(kSpBM, R - r0);
            if (int(threadIdx.x) * 64 < rows && g.k0 == 0) {
                if (threadIdx.x == 0) p.cuts[first] = CacheCut{g.s.q0, rows, r0, g.hk * p.g, first, last, {0, 0}};
                p.cut_flags[first * kMergeCtas + threadIdx.x] = 1u;
            }
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
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(jfa_cache_split_kernel<D, BIAS>, SpCfg::kBytes, done);
    if (e != cudaSuccess) return e;
    jfa_cache_split_kernel<D, BIAS><<<num_sms, SpCfg::kThreads, SpCfg::kBytes, st>>>(mk, mv, p);
    return cudaGetLastError();
}

}  // namespace

size_t cache_split_part_bytes(int D, int num_sms) { return size_t(num_sms) * 2 * cache_merge_part(D) * 4; }

cudaError_t launch_cache_split(int D, const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, int num_sms,
                               cudaStream_t st) {
    if (D == 32) return p.bias ? launch<32, true>(mk, mv, p, num_sms, st) : launch<32, false>(mk, mv, p, num_sms, st);
    return p.bias ? launch<64, true>(mk, mv, p, num_sms, st) : launch<64, false>(mk, mv, p, num_sms, st);
}

}  // namespace jfa
