// Paged-cache attention for chunks of new tokens (bf16): tcgen05 products, TMEM accumulators.
//
// An item is up to 256 packed rows (tokens x grouped heads) of one (sequence, key head): two
// tiles of floor(128 / g) tokens' rows (so that a tile is one box of Q) that share every key and
// value tile, so that one tile's softmax runs while the tensor core works on the other.  Key
// tiles of 128 positions are gathered by TMA, one box per page and 128-byte column block; a box
// of a short page lands at its rows of the tile, whose swizzle repeats every 8 rows (the
// smallest page).
// A cache held in 4 bits: codes and scales come through rings of their own, and warps 18-21 load and
// unpack them to fp16 tiles in the layout that TMA would have written; queries are taken to fp16
// with a power of two per row, and P is 2^6 times the weights in fp16 (as in
// cache_decode4.cu).  Measured, the prompts below over 4 bits: 786 us, 1093 TFLOP/s, 0.56 of the burst
// rate: the unpacking hides beside the products, but leaves the softmax warps 80 registers and
// one chunk of scores at a time.  (Unpacking by one warp each for K and V 855 us, by four from
// global memory one tile ahead 1478, the few-rows kernel for all 4099.)
// CTA = 19 warps (22 over 4 bits), one CTA per SM; the CTAs draw their work from a counter (cache_common.cuh).
// Two warps share each row (thread = row = TMEM lane): one takes score columns [0, 64) and O
// columns [0, D/2), the other the rest; they exchange row maxima and sums through shared
// memory.
//   warps 0-3, 8-11    tile A, columns [0, 64) and [64, 128): softmax, rescaling, epilogue
//   warps 4-7, 12-15   tile B
//   warp 18            TMA loads: Q once per item, K and V boxes through rings
//   warp 16            tcgen05.mma issuer and TMEM owner; clears V rows no query may see
//   warp 17            draws pieces of work when the loads near the end of what was drawn, and
//                      hands out their items
// TMEM (512 columns): S_A [0,128), S_B [128,256), O_A [256,256+D), O_B [384,384+D); P
// overwrites its own S columns as packed bf16 and is read from TMEM by O += P V.
// An item with a single row tile runs its steps alternately as tile A and tile B (both on
// the same query rows, each with its own maximum, sum and O), so it keeps the overlap; the
// two are merged at the end.
// The parts of an item cut between blocks go to the workspace in fp32, and a second kernel
// adds them up: the last part's CTA alone would read them at one SM's rate (about 2 us a
// part of 132 KB), and a long history under one chunk has tens of parts.
// Measured: 8 prompts of 700-1024 tokens (32 query, 8 key heads of 128) over 3k-14k keys, 859
// GFLOP, 708 us with the merge, 1213 TFLOP/s, 0.64 of the measured matrix-product burst rate (874 us
// with a bias).  A step of 256 x 128 scores takes 1.8 us, its products 1.1 and its exponentials 0.5
// (32 a clock): what is left is each tile's own chain S -> softmax -> P V -> S, since at head_dim
// 128 TMEM holds no second score tile per row tile.  P is rounded to bf16 for its product, as in
// the packed forward, after its sum is taken in fp32: 2^-8 of each weight, at most.  256 sets of 1-64 rows over 100-8000 keys (8
// heads of 64, 947 MB) 243 us, 0.57 of the copy rate: long items stream 128 keys in 0.86 us on
// each SM (5.7 TB/s in all), an item's end and start cost 3 us more, a single short item 5-8 us
// from its draw to its stored rows, and the sets of up to 16 rows follow in the decode kernel
// (53 us).  Slower, and not kept: two key tiles in one score tile for sets of up to 64 rows
// (254 -> 290 us), two key heads in one item (262 -> 279 us), the decode kernel first (254 ->
// 266 us), drawing an item ahead of time (738 -> 796 us for the prompts, whose last items then
// wait in CTAs that are busy).
#include "cache_common.cuh"
#include "quant.cuh"
#include "tilemath.cuh"

#include <limits.h>

namespace jfa {

namespace {

// A part of an item, as handed to the other warps (b < 0: the end).
struct alignas(16) SegRec {
    int b, hk, tile, k0, k1;
    int q0, q_len, kv_len;
    int first, last, slot;  // split item: blocks of its first and last part, this part's slot
    int pad;
};

// From this many positions back on, 32 consecutive positions lie in three buckets at most:
// r in [62, ..) and r - 31 differ by a factor of at most 2 in 1 + r, two buckets' width.
// (and r <= -31 likewise, from the other side).  Chunks between the two touch |r| <= 93 and
// read the bias from a table by position; a stride of 4 mod 32 spreads the heads of a warp's
// rows over the banks.
constexpr int kThreeBuckets = 62, kNear = 96, kNearStride = 100, kNearHeads = 32;

template <int D, bool Q4>
struct ChkCfg {
    static constexpr int BM = 128, BN = 128, kPair = kMergeRows;
    static constexpr int kCB = D / 64;
    static constexpr int kQBytes = BM * D * 2, kKVBytes = BN * D * 2;
    // K and V rings: what shared memory holds (a short item's keys come from DRAM, and two
    // stages of 16 KB in flight would not keep up with it)
    // 4 bits: one ring of unpacked tiles, K and V in turn, and of packed ones a ring each
    static constexpr int kStages = D == 128 ? 2 : 5, kRing = D == 128 ? 3 : 6, kRaw = 2;
    static constexpr int kRawCodes = BN * D / 2, kRawBytes = kRawCodes + BN * D / 16;
    static constexpr int kOffQ = 0, kOffK = kOffQ + 2 * kQBytes, kOffV = kOffK + (Q4 ? 0 : kStages * kKVBytes);
    static constexpr int kOffRaw = kOffK + kRing * kKVBytes;
    static constexpr int kOffBar = Q4 ? kOffRaw + 2 * kRaw * kRawBytes : kOffV + kStages * kKVBytes;
    static constexpr int kNumBars = 60;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;   // tmem slot, abort flag
    static constexpr int kSlots = 4;                          // parts of items handed out and not yet taken by all
    static constexpr int kAsk = 3;                            // key tiles of a part left to load when the next is asked for
    static constexpr int kOffSeg = kOffMisc + 16;
    static constexpr int kOffStarts = kOffSeg + kSlots * int(sizeof(SegRec));  // first position of each bias bucket
    static constexpr int kOffComb = kOffStarts + 32 * 4;      // tile B's m and l of a split item, two buffers
    static constexpr int kOffXch = kOffComb + 2 * 3 * BM * 4; // pair exchanges [2][2][8][32]
    static constexpr int kOffGroups = kOffXch + 2 * 2 * 8 * 32 * 4;
    // bias by relative position |r| < kNear, log2 units, of the first kNearHeads heads
    static constexpr int kOffNear = kOffGroups + (int(sizeof(CacheGroups)) + 15) / 16 * 16;
    static constexpr int kStride = Q4 ? kNear + 1 : kNearStride;  // (shared memory is short by 400 bytes)
    // 4 bits: what takes a row's scores back to its queries' size [2 BM], behind the m and l in use
    static constexpr int kOffDown = kOffComb + 2 * 2 * BM * 4;
    static constexpr int kSmemNeed = kOffNear + kNearHeads * kStride * 4 + 1024;
    // at least 120 KB: one CTA per SM, as the CTA allocates all 512 TMEM columns
    static constexpr int kSmemBytes = kSmemNeed > 120 * 1024 ? kSmemNeed : 120 * 1024;
    // 4 bits: two warps unpack K's tiles and two V's, half of the rows each, and the first of each two
    // loads.  One warp each left a thread 96 registers instead of 80, but took longer than a step
    // (8 prompts 841 us instead of 788); four warps on each tile in turn and a loading one 815.
    static constexpr int kShare = 2, kWriters = Q4 ? 2 * kShare : 1;
    static constexpr int kSoftWarps = 16, kMmaWarp = 16, kDrawWarp = 17, kProdWarp = 18, kThreads = (kProdWarp + kWriters) * 32;
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kIdescQK = make_idesc(Q4 ? kFmtF16 : kFmtBF16, BM, BN, false, false);
    static constexpr uint32_t kIdescPV = make_idesc(Q4 ? kFmtF16 : kFmtBF16, BM, D, false, true);
    static constexpr int kPart = cache_merge_part(D);  // floats of a partial result: O (four columns of all rows at a time), m, l
    __host__ __device__ static constexpr uint32_t tmem_s(int x) { return x ? 128u : 0u; }
    __host__ __device__ static constexpr uint32_t tmem_o(int x) { return x ? 384u : 256u; }
};

enum {
    B_Q_FULL = 0,
    B_Q_EMPTY = 1,
    B_S_FULL = 2,    // +tile
    B_P_FULL = 4,
    B_O_DONE = 6,
    B_O_EMPTY = 8,
    B_DRAIN = 10,
    B_COMBINE = 11,  // split item: tile B's last P V done and its m and l written
    B_ASK = 12,      // the producer is near the end of its part
    B_XCH = 14,      // +pair of warps
    B_K_FULL = 22,   // +stage (up to 6)
    B_K_EMPTY = 28,
    B_V_FULL = 34,
    B_V_EMPTY = 40,
    B_SEG_FULL = 46,   // +slot: a part of an item handed out
    B_SEG_EMPTY = 50,  // +slot: and read by every other warp
    B_Q_RAW = 54,      // 4 bits: queries as they are given
    B_RAW_EMPTY = 55,  // +stage: packed tiles read, K's, then V's
};

// TMEM column (within a tile's S/P columns) of the 16 P values of P V step s.
__device__ __forceinline__ uint32_t p_col(int s) { return uint32_t(32 * (s >> 1) + 8 * (s & 1)); }

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
    const int rt = p.tile_tokens * p.g;  // packed rows of a tile
    s.split = (2 * g.tile + 1) * rt >= g.s.q_len * p.g;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        CacheRange r{0, 0, 0, 0};
        if ((2 * g.tile + x) * rt < g.s.q_len * p.g) r = cache_range<128>(p, g.s, 2 * g.tile + x, rt);
        s.a[x] = max(s.k0, r.f - g.r.f);
        s.b[x] = r.n > 0 ? min(s.k1, r.f - g.r.f + r.n) : s.a[x];
    }
    return s;
}

template <int D, bool BIAS, bool Q4>
__global__ void __launch_bounds__((ChkCfg<D, Q4>::kThreads), 1)
    jfa_cache_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const CacheFwdParams p) {
    using C = ChkCfg<D, Q4>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t sQ = sbase + C::kOffQ, sK = sbase + C::kOffK, sV = sbase + C::kOffV;
    auto bar = [&](int i) -> uint32_t { return sbase + C::kOffBar + 8u * uint32_t(i); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    SegRec* handed = reinterpret_cast<SegRec*>(smem + C::kOffSeg);
    int* starts = reinterpret_cast<int*>(smem + C::kOffStarts);
    CacheGroups* groups = reinterpret_cast<CacheGroups*>(smem + C::kOffGroups);
    static_assert(C::kSmemNeed <= 227 * 1024, "shared memory of a CTA");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(bar(B_Q_FULL), C::kWriters);
        mbar_init(bar(B_Q_EMPTY), Q4 ? 1 + C::kSoftWarps : 1);
        if (Q4) {  // K_*: the ring of unpacked tiles; V_FULL: of packed ones, K's, then V's
            for (int s = 0; s < C::kRing; ++s) {
                mbar_init(bar(B_K_FULL + s), C::kShare);
                mbar_init(bar(B_K_EMPTY + s), 1);
            }
            for (int s = 0; s < 2 * C::kRaw; ++s) {
                mbar_init(bar(B_V_FULL + s), 1);
                mbar_init(bar(B_RAW_EMPTY + s), C::kShare);
            }
            for (int s = 0; s < 3; ++s) mbar_init(bar(B_V_EMPTY + s), 1);  // every third V read
            mbar_init(bar(B_Q_RAW), 1);
        }
        for (int s = 0; !Q4 && s < C::kStages; ++s) {
            mbar_init(bar(B_K_FULL + s), 1);
            mbar_init(bar(B_K_EMPTY + s), 1);
            mbar_init(bar(B_V_FULL + s), 1);
            mbar_init(bar(B_V_EMPTY + s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(B_S_FULL + s), 1);
            mbar_init(bar(B_P_FULL + s), 8);
            mbar_init(bar(B_O_DONE + s), 1);
            mbar_init(bar(B_O_EMPTY + s), 8);
        }
        mbar_init(bar(B_DRAIN), 1);
        mbar_init(bar(B_COMBINE), 8);
        for (int q = 0; q < 8; ++q) mbar_init(bar(B_XCH + q), 2);
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(bar(B_SEG_FULL + s), 1);
            mbar_init(bar(B_SEG_EMPTY + s), C::kSoftWarps + 1 + C::kWriters);
        }
        mbar_init(bar(B_ASK), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == C::kProdWarp && lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (threadIdx.x >= 64 && threadIdx.x < 96) {
        // the smallest r with (1 + r)^2 >= 2^b: the root's integer part is within one of it
        int r = int(sqrtf(exp2f(float(lane))));
        r = max(r - 2, 0);
        while ((long long)(1 + r) * (1 + r) < (1LL << lane)) ++r;
        starts[lane] = r;
    }
    if (warp == C::kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    float* near_tab = reinterpret_cast<float*>(smem + C::kOffNear);
    const bool near_ok = BIAS && p.H <= kNearHeads;
    if (near_ok)
        for (int e = threadIdx.x; e < p.H * kNear; e += C::kThreads)
            near_tab[(e / kNear) * C::kStride + e % kNear] = p.bias[(e / kNear) * 32 + relpos_bucket(e % kNear)] * 1.4426950408889634f;
    cache_pieces<C::BN>(p, groups);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    launch_dependents();  // the decode kernel may fill SMs as they come free
    CacheSeg g;
    int first = 0, last = 0, part_slot = 0;
    uint32_t seg_no = 0;
    // The next part of an item (false: no more, or the CTA gave up).
    auto next = [&]() -> bool {
        const uint32_t slot = seg_no % C::kSlots;
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar(B_SEG_FULL + slot), (seg_no / C::kSlots) & 1, abort_flag)))
            return false;
        const SegRec r = handed[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_SEG_EMPTY + slot));
        ++seg_no;
        if (r.b < 0) return false;
        g.b = r.b;
        g.hk = r.hk;
        g.tile = r.tile;
        g.s = CacheSeq{r.q0, r.q_len, r.kv_len};
        g.r = cache_range<C::BN>(p, g.s, g.tile);
        g.n = max(1, g.r.n);
        g.k0 = r.k0;
        g.k1 = r.k1;
        first = r.first;
        last = r.last;
        part_slot = r.slot;
        return true;
    };

    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(p.status, kStatusTimeout);
    };

    if (Q4 && warp >= C::kProdWarp) {
        if constexpr (Q4) {
            // -------------------------------------------------------- loads and unpacking
            // Two warps each for K and V; the queries are taken to fp16 by all.  A thread takes 32
            // neighbouring elements of a row at a time, `kPer` lanes a row: queries from bf16, in
            // place, with a power of two of their row that brings their largest magnitude to
            // 2^14, keys and values from 16 bytes of codes and two scales.  What it writes are four
            // of the eight 16-byte pieces of a 128-byte row of the tile; the lanes of a row's second
            // half write theirs in another order, so that eight lanes meet all banks.  (Codes
            // loaded by address, a tile ahead, came too late: 1478 us for the 8 prompts.)
            constexpr int kPer = D / 32, kRows = 32 / kPer, NP = 4, kGroups = C::BN / (NP * kRows);
            const int v = (warp - C::kProdWarp) & 1, share = (warp - C::kProdWarp) >> 1, quarter = lane % kPer, row0 = lane / kPer;
            const int turn = D == 128 ? 2 * (quarter >> 1) : 0;  // its order: pieces c ^ turn
            float* down_s = reinterpret_cast<float*>(smem + C::kOffDown);
            // (rows of a thread are 8 or 16 apart: their pieces lie alike)
            uint32_t piece[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                piece[c] = uint32_t((quarter >> 1) * C::BM * 128 + row0 * 128 + (((4 * (quarter & 1) + (c ^ turn)) ^ (row0 & 7)) << 4));
            auto wwait = [&](int b, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait_bounded(bar(b), parity, abort_flag));
            };
            auto publish = [&](int b) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(b));
            };
            uint32_t done = 0, item_it = 0;  // tiles unpacked, items
            bool ok = true;
            // Loads: a lane takes one box of each tile, the codes of a page (or of 64 keys of one), and
            // its scales.
            const CUtensorMap* map = v ? &tmV : &tmK;
            const uint8_t* scales = v ? p.v_scales : p.k_scales;
            const int64_t s_page = v ? p.vss[0] : p.kss[0], s_head = v ? p.vss[1] : p.kss[1];
            const int rows = min(1 << p.page_log2, 64), per = C::BN / rows;
            const uint32_t raw0 = sbase + C::kOffRaw + v * C::kRaw * C::kRawBytes;
            uint32_t issued = 0;
            int lk = 0, page = -1;           // the next key tile to load, and its page
            auto page_of = [&](int k) -> int {
                const int j = (g.r.f + k) * C::BN + lane * rows;
                if (lane >= per || k >= g.k1 || j >= g.r.hi || j + rows <= g.r.lo) return -1;
                const int at = p.table[size_t(g.b) * size_t(p.max_pages) + size_t(j >> p.page_log2)];
                if (at >= 0 && at < p.n_pages) return at;
                atomicOr(p.status, kStatusBounds);
                return p.n_pages;  // past the cache: codes read as zeros (with any scales)
            };
            // The next tile into its place, which this warp has read.
            auto load_tile = [&]() {
                if (share || lk >= g.k1) return;
                const uint32_t st = issued % C::kRaw, dst = raw0 + st * C::kRawBytes;
                const uint32_t full_b = bar(B_V_FULL + v * C::kRaw + int(st));
                if (!v && g.k1 - lk == min(C::kAsk, g.k1 - g.k0) && lane == 0) mbar_arrive(bar(B_ASK));
                if (!wwait(B_RAW_EMPTY + v * C::kRaw + int(st), ((issued / C::kRaw) & 1) ^ 1)) { ok = false; return; }
                const uint32_t bytes = uint32_t(__popc(__ballot_sync(0xffffffffu, page >= 0)) * rows * (D / 2 + D / 16));
                if (lane == 0) mbar_arrive_expect_tx(full_b, bytes);
                __syncwarp();
                if (page >= 0) {
                    const int slot = ((g.r.f + lk) * C::BN + lane * rows) & ((1 << p.page_log2) - 1);
                    tma_load_4d(dst + lane * rows * (D / 2), map, full_b, 0, slot, g.hk, page);
                    bulk_load(dst + C::kRawCodes + lane * rows * (D / 16),
                              scales + (page < p.n_pages ? page : 0) * s_page + g.hk * s_head + slot * (D / 16), uint32_t(rows * (D / 16)), full_b);
                }
                ++issued;
                page = page_of(++lk);
            };
            // The next tile, of key tile k; keys outside the item's become zeros (what lies there is
            // undefined, and 0 * NaN is not 0).
            auto unpack = [&](int k) -> bool {
                const uint32_t rs = done % C::kRaw, at = 2 * done + v, st = at % C::kRing;
                const uint32_t raw = raw0 + rs * C::kRawBytes, tile = sK + st * C::kKVBytes;
                const int c0 = (g.r.f + k) * C::BN, lo = g.r.lo - c0, hi = g.r.hi - c0;
                const bool edge = lo > 0 || hi < C::BN;
                uint4 w[2][NP];
                uint32_t sc[2][NP];
                auto fetch = [&](int n) {
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        const int row = kRows * (NP * (C::kShare * n + share) + i) + row0;
                        w[n & 1][i] = ld_shared_v4(raw + uint32_t(row * (D / 2) + 16 * quarter));
                        uint16_t two;
                        asm volatile("ld.shared.b16 %0, [%1];" : "=h"(two) : "r"(raw + uint32_t(C::kRawCodes + row * (D / 16) + 2 * quarter)));
                        sc[n & 1][i] = two;
                        if (edge && (row < lo || row >= hi)) sc[n & 1][i] = 0u;
                    }
                };
                if (!wwait(B_V_FULL + v * C::kRaw + int(rs), (done / C::kRaw) & 1)) return false;
                fetch(0);
                // (A place's barrier tells its last use from the one before by parity alone, and V may
                // run ahead of K by two: a split item's keys are read up to two tiles before its
                // values.  So V's third last tile, which had this place two uses ago, is seen read first.)
                if (v && done >= 3 && !wwait(B_V_EMPTY + int(done % 3), (done / 3 - 1) & 1)) return false;
                if (!wwait(B_K_EMPTY + int(st), ((at / C::kRing) & 1) ^ 1)) return false;
#pragma unroll
                for (int n = 0; n < kGroups / C::kShare; ++n) {
                    if (n + 1 < kGroups / C::kShare) {
                        fetch(n + 1);
                    } else {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(B_RAW_EMPTY + v * C::kRaw + int(rs)));
                    }
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        const uint32_t two = e4m3_to_f16(sc[n & 1][i]);
                        const uint32_t s0 = __byte_perm(two, 0u, turn ? 0x3232 : 0x1010), s1 = __byte_perm(two, 0u, turn ? 0x1010 : 0x3232);
                        const uint4 u = w[n & 1][i];
                        const uint32_t x[4] = {turn ? u.z : u.x, turn ? u.w : u.y, turn ? u.x : u.z, turn ? u.y : u.w};
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t h[4];
                            e2m1_to_f16(x[c], h);
                            const uint32_t s = c < 2 ? s0 : s1;
                            st_shared_v4(tile + piece[c] + uint32_t(kRows * (NP * (C::kShare * n + share) + i) * 128), f16_mul2(h[0], s), f16_mul2(h[1], s),
                                         f16_mul2(h[2], s), f16_mul2(h[3], s));
                        }
                    }
                }
                publish(B_K_FULL + int(st));
                ++done;
                return true;
            };
            auto convert_q = [&](int tiles) {
#pragma unroll 1
                for (int r0 = kRows * (warp - C::kProdWarp); r0 < tiles * C::BM; r0 += C::kWriters * kRows) {
                    const uint32_t tile = sQ + uint32_t((r0 >= C::BM ? C::kQBytes : 0) + (r0 & (C::BM - 1)) * 128);
                    uint4 q[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) q[c] = ld_shared_v4(tile + piece[c]);
                    float top = 0.f;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t v[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            top = fmax3(top, fabsf(__uint_as_float(v[e] << 16)), fabsf(__uint_as_float(v[e] & 0xffff0000u)));
                    }
#pragma unroll
                    for (int d = 1; d < kPer; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    const uint32_t e = min(max(__float_as_uint(top) >> 23, 15u), 254u);  // (rows past the tile's hold anything)
                    const float up = __uint_as_float((268u - e) << 23);
                    if (quarter == 0) down_s[r0 + row0] = __uint_as_float((e - 14u) << 23);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t v[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
                        uint32_t h[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            h[k] = pack_f16x2(__uint_as_float(v[k] << 16) * up, __uint_as_float(v[k] & 0xffff0000u) * up);
                        st_shared_v4(tile + piece[c], h[0], h[1], h[2], h[3]);
                    }
                }
            };
            while (ok && next()) {
                if (g.r.n == 0) {
                    if (warp == C::kProdWarp && lane == 0) mbar_arrive(bar(B_ASK));
                    continue;
                }
                lk = g.k0;
                page = share ? -1 : page_of(lk);
#pragma unroll 1
                for (int i = 0; i < C::kRaw; ++i) load_tile();
                if (!wwait(B_Q_EMPTY, (item_it & 1) ^ 1)) { ok = false; break; }
                const int tiles = (2 * g.tile + 1) * p.tile_tokens < g.s.q_len ? 2 : 1;
                if (warp == C::kProdWarp) {  // a box per tile and column block; tokens past the sequence's are not stored
                    if (lane == 0) mbar_arrive_expect_tx(bar(B_Q_RAW), uint32_t(tiles * C::kCB * p.tile_tokens * p.g * 128));
                    __syncwarp();
                    if (lane < tiles * C::kCB)
                        tma_load_3d(sQ + (lane / C::kCB) * C::kQBytes + (lane % C::kCB) * C::BM * 128, &tmQ, bar(B_Q_RAW),
                                    (lane % C::kCB) * 64, g.hk * p.g, g.s.q0 + (2 * g.tile + lane / C::kCB) * p.tile_tokens);
                }
                ++item_it;
                if (!wwait(B_Q_RAW, (item_it - 1) & 1)) { ok = false; break; }
                convert_q(tiles);
                publish(B_Q_FULL);
#pragma unroll 1
                for (int k = g.k0; k < g.k1 && ok; ++k) {
                    ok = unpack(k);
                    if (ok) load_tile();
                }
            }
            if (!ok && lane == 0) fail();
            if (warp == C::kProdWarp && item_it > 0) mbar_wait_bounded(bar(B_Q_RAW), (item_it - 1) & 1, nullptr);
            drain_ring(bar(B_V_FULL + v * C::kRaw), issued, C::kRaw);
        }
    } else if (!Q4 && warp == C::kProdWarp) {
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
        auto ask = [&]() {
            if (lane == 0) mbar_arrive(bar(B_ASK));
        };
        while (ok && next()) {
            if (g.r.n == 0) {
                ask();
                continue;
            }
            auto load_q = [&]() {
                // a box per tile and column block; tokens past the sequence's are not stored
                const int tiles = (2 * g.tile + 1) * p.tile_tokens < g.s.q_len ? 2 : 1;
                if (lane == 0)
                    mbar_arrive_expect_tx(bar(B_Q_FULL), uint32_t(tiles * C::kCB * p.tile_tokens * p.g * 128));
                __syncwarp();
                if (lane < tiles * C::kCB)
                    tma_load_3d(sQ + (lane / C::kCB) * C::kQBytes + (lane % C::kCB) * C::BM * 128, &tmQ, bar(B_Q_FULL),
                                (lane % C::kCB) * 64, g.hk * p.g, g.s.q0 + (2 * g.tile + lane / C::kCB) * p.tile_tokens);
                ++item_it;
            };
            // Q's memory is free when the last part's scores are done; its first key tiles may
            // be in flight by then
            bool have_q = __all_sync(0xffffffffu, mbar_try_wait(bar(B_Q_EMPTY), (item_it & 1) ^ 1));
            if (have_q) load_q();
            int page = page_of(g, g.k0);
            for (int k = g.k0; k < g.k1; ++k, ++kv_it) {
                if (g.k1 - k == min(C::kAsk, g.k1 - g.k0)) ask();
                if (!have_q && k - g.k0 == C::kStages / 2) {
                    if (!wwait(B_Q_EMPTY, (item_it & 1) ^ 1)) { ok = false; break; }
                    load_q();
                    have_q = true;
                }
                const uint32_t st = kv_it % C::kStages, ph = (kv_it / C::kStages) & 1;
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
            }
            if (ok && !have_q) {
                if (!wwait(B_Q_EMPTY, (item_it & 1) ^ 1)) { ok = false; break; }
                load_q();
            }
        }
        if (!ok && lane == 0) fail();
        if (item_it > 0) mbar_wait_bounded(bar(B_Q_FULL), (item_it - 1) & 1, nullptr);
        drain_ring(bar(B_K_FULL), kv_it + k_extra, C::kStages);
        drain_ring(bar(B_V_FULL), kv_it, C::kStages);
    } else if (warp == C::kDrawWarp) {
        // ------------------------------------------------------------ work
        const int ng = (p.B + 31) >> 5, pieces = groups->pieces, whole = groups->whole, blk = groups->blk;
        const int cut = groups->cut;
        bool ok = true;
        uint32_t asked = 0;
        auto wwait = [&](int b, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar(b), parity, abort_flag));
            return ok;
        };
        // A CTA draws when the loads of all it was handed are near their end: no more than it
        // can work off, however long, and as many short parts as keep the loads in flight.
        // (Waited for before every part handed out, so that the barrier is never two phases
        // ahead of the wait.)
        auto wanted = [&]() {
            for (; asked < seg_no && ok; ++asked) wwait(B_ASK, asked & 1);
            return ok;
        };
        auto hand_out = [&](const SegRec& r) {
            const uint32_t slot = seg_no % C::kSlots;
            if (!wanted() || !wwait(B_SEG_EMPTY + int(slot), ((seg_no / C::kSlots) & 1) ^ 1)) return false;
            if (lane == 0) {
                handed[slot] = r;
                mbar_arrive(bar(B_SEG_FULL + slot));
            }
            __syncwarp();
            ++seg_no;
            return true;
        };
        int w = blockIdx.x;
        while (w < pieces) {
            CacheStart st;
            if (w < whole) {
                st = cache_find_item(p, *groups, ng, w, lane);
                st.u_end = INT_MAX;  // (one item, all of its units)
            } else {
                const int u = cut + (w - whole) * blk;
                st = cache_find_unit<C::BN>(p, *groups, ng, u, lane);
                st.u_end = min(groups->total, u + blk);
            }
            CacheCursor<C::BN> cur(p, st, groups->order);
            while (ok && cur.next(p, g)) {
                SegRec r{g.b, g.hk, g.tile, g.k0, g.k1, g.s.q0, g.s.q_len, g.s.kv_len, 0, 0, 0, 0};
                if (w >= whole) {
                    r.first = int(uint32_t(g.first + p.item_cost - cut) / uint32_t(blk));
                    r.last = int(uint32_t(g.first + p.item_cost + g.n - 1 - cut) / uint32_t(blk));
                    r.slot = cache_slot(w - whole, r.first);
                }
                hand_out(r);
                if (w < whole) break;
            }
            if (!wanted()) break;
            if (lane == 0) w = int(gridDim.x + atomicAdd(p.counters + kCtrDrawn, 1u));
            w = __shfl_sync(0xffffffffu, w, 0);
        }
        hand_out(SegRec{-1, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0});
        if (!ok && lane == 0) fail();
        // the last CTA to have drawn its last piece leaves the counters zero
        if (lane == 0 && atomicAdd(p.counters + kCtrDone, 1u) == gridDim.x - 1) {
            p.counters[kCtrDrawn] = 0u;
            p.counters[kCtrDone] = 0u;
        }
    } else if (warp == C::kMmaWarp) {
        // ------------------------------------------------------------ MMA issuer
        auto wwait = [&](int b, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait_bounded(bar(b), parity, abort_flag));
        };
        uint32_t kv_it = 0, item_it = 0, pv_cnt0 = 0, pv_cnt1 = 0, items_x0 = 0, items_x1 = 0;
        bool ok = true;
        const SDesc dQ0 = sdesc_sw128(sQ, 16, 1024), dQ1 = sdesc_sw128(sQ + C::kQBytes, 16, 1024);
        const SDesc dK0 = sdesc_sw128(sK, 16, 1024), dV0 = sdesc_sw128(sV, C::BN * 128, 1024);
        // stage and phase of key tile t's K and V: rings of their own, or one ring in turn
        constexpr int kVFull = Q4 ? B_K_FULL : B_V_FULL, kVEmpty = Q4 ? B_K_EMPTY : B_V_EMPTY;
        auto k_stage = [](uint32_t t) { return Q4 ? (2 * t) % C::kRing : t % C::kStages; };
        auto k_phase = [](uint32_t t) { return (Q4 ? (2 * t) / C::kRing : t / C::kStages) & 1; };
        auto v_stage = [](uint32_t t) { return Q4 ? (2 * t + 1) % C::kRing : t % C::kStages; };
        auto v_phase = [](uint32_t t) { return (Q4 ? (2 * t + 1) / C::kRing : t / C::kStages) & 1; };
        auto stage = [&](const SDesc& d, uint32_t st) { return SDesc{d.lo + st * (C::kKVBytes >> 4), d.hi}; };
        // S_x = Q K^T, after the tile's previous P V product, which reads P from those columns
        auto issue_s = [&](int x, uint32_t st, int qx) -> bool {
            const uint32_t pc = x ? pv_cnt1 : pv_cnt0;
            if (pc > 0 && !wwait(B_O_DONE + x, (pc - 1) & 1)) return false;
            tc_fence_after();
            const SDesc dq = qx ? dQ1 : dQ0, dk = stage(dK0, st);
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
            const SDesc dv = stage(dV0, st);
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
        while (ok && next()) {
            if (g.r.n == 0) continue;
            const Steps s = steps_of(p, g);
            const int n = s.k1 - s.k0;
            if (!wwait(B_Q_FULL, item_it & 1)) { ok = false; break; }
            if (!s.split) {
                auto act = [&](int x, int j) { return j >= s.a[x] && j < s.b[x]; };
                {
                    const uint32_t st = k_stage(kv_it), ph = k_phase(kv_it);
                    if (!wwait(B_K_FULL + st, ph)) { ok = false; break; }
                    if (act(0, s.k0) && !issue_s(0, st, 0)) { ok = false; break; }
                    if (act(1, s.k0) && !issue_s(1, st, 1)) { ok = false; break; }
                    commit(B_K_EMPTY + st);
                    if (n == 1) commit(B_Q_EMPTY);
                }
                for (int i = 0; i < n && ok; ++i) {
                    const int j = s.k0 + i;
                    const uint32_t t = kv_it + i, st = v_stage(t), ph = v_phase(t);
                    const uint32_t t1 = t + 1, st1 = k_stage(t1), ph1 = k_phase(t1);
                    if (!wwait(kVFull + st, ph)) { ok = false; break; }
                    if (!Q4) clear_v(st, j);
                    if (act(0, j) && !issue_pv(0, st, j == s.a[0])) { ok = false; break; }
                    if (i + 1 < n && !wwait(B_K_FULL + st1, ph1)) { ok = false; break; }
                    if (act(0, j + 1) && !issue_s(0, st1, 0)) { ok = false; break; }
                    if (act(1, j) && !issue_pv(1, st, j == s.a[1])) { ok = false; break; }
                    commit(kVEmpty + st);
                    if (Q4) commit(B_V_EMPTY + t % 3);
                    if (act(1, j + 1) && !issue_s(1, st1, 1)) { ok = false; break; }
                    if (i + 1 < n) {
                        commit(B_K_EMPTY + st1);
                        if (i + 2 == n) commit(B_Q_EMPTY);
                    }
                }
            } else {
                // step i: tile x = i & 1 computes P V of step i, then S of step i + 2
                for (int i = 0; i < 2 && i < n && ok; ++i) {
                    const uint32_t t = kv_it + i, st = k_stage(t), ph = k_phase(t);
                    if (!wwait(B_K_FULL + st, ph) || !issue_s(i, st, 0)) { ok = false; break; }
                    commit(B_K_EMPTY + st);
                    if (i + 1 == n) commit(B_Q_EMPTY);
                }
                for (int i = 0; i < n && ok; ++i) {
                    const int x = i & 1;
                    const uint32_t t = kv_it + i, st = v_stage(t), ph = v_phase(t);
                    const uint32_t t2 = t + 2, st2 = k_stage(t2), ph2 = k_phase(t2);
                    if (!wwait(kVFull + st, ph)) { ok = false; break; }
                    if (!Q4) clear_v(st, s.k0 + i);
                    if (!issue_pv(x, st, i < 2)) { ok = false; break; }
                    commit(kVEmpty + st);
                    if (Q4) commit(B_V_EMPTY + t % 3);
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
    } else if (warp < C::kSoftWarps) {
        // ------------------------------------------------------------ softmax / epilogue
        const int x = (warp >> 2) & 1, hf = warp >> 3, pair = warp & 7;
        const int t = (warp & 3) * 32 + lane;  // row in the tile == TMEM lane
        constexpr int HC = C::BN / 2, OC = D / 2;
        const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
        const uint32_t tSt = tmem + lane_base + C::tmem_s(x);
        const uint32_t tS = tSt + uint32_t(HC * hf);
        const uint32_t tO = tmem + lane_base + C::tmem_o(x) + uint32_t(OC * hf);
        uint32_t s_cnt = 0, split_cnt = 0, x_cnt = 0;
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
        float xs = p.scale_log2;
        // 4 bits: P = 2^6 times the weights, in fp16, where small ones keep more of their bits
        constexpr float kLift = Q4 ? 6.f : 0.f;
        uint32_t item_it = 0;
        bool ok = true;
        while (ok && next()) {
            const Steps sp = steps_of(p, g);
            const int R = g.s.q_len * p.g, diag = g.s.kv_len - g.s.q_len;
            const int n = sp.count(x);
            const int first_k = sp.split ? sp.k0 + x : sp.a[x], stride_k = sp.split ? 2 : 1;
            const int rt = p.tile_tokens * p.g;                      // packed rows of a tile
            const int row = (2 * g.tile + (sp.split ? 0 : x)) * rt + t;  // packed row
            const bool row_valid = t < rt && row < R;
            const int rc = min(row, R - 1), tok = div_g(p, rc), head = g.hk * p.g + rc - tok * p.g;
            const int rel = tok + diag;  // position of the row: rows past the end repeat the last one's masks
            const int t0 = __shfl_sync(0xffffffffu, tok, 0), t31 = __shfl_sync(0xffffffffu, tok, 31);
            const float* brow = BIAS ? p.bias + head * 32 : nullptr;
            const size_t orow = size_t(g.s.q0 + tok) * size_t(p.H) + size_t(head);
            float m = -INFINITY, l = 0.f;
            if (Q4 && g.r.n > 0) {
                if (!wwait(B_Q_FULL, item_it & 1)) { ok = false; break; }
                // (not 0, which would not leave a masked score at -inf; scores are below 2^33)
                xs = fmaxf(p.scale_log2 * reinterpret_cast<const float*>(smem + C::kOffDown)[(sp.split ? 0 : x) * C::BM + t], 1e-37f);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_Q_EMPTY));
                ++item_it;
            }
            for (int i = 0; i < n; ++i) {
                const int col0 = (g.r.f + first_k + i * stride_k) * C::BN;
                int lim = g.s.kv_len - col0;
                if (p.causal) lim = min(lim, rel + 1 - col0);
                const int lo = p.window >= 0 ? rel - p.window - col0 : 0;
                const bool full = __all_sync(0xffffffffu, lim >= C::BN && lo <= 0);
                // Bias per 32-column chunk: one value per row when every row's positions of
                // the chunk share a bucket, else three values a row, or near the row's own
                // position a table's.
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
                // Without a bias both chunks' scores are held at a time, with one (and over 4 bits, where a
                // thread has 80 registers: 916 -> 788 us for the prompts) they are taken one
                // by one in rolled loops: the three ways of its lookup would otherwise be laid out
                // four times, and a short item pays for every line of code it fetches.  (A path for
                // two plain chunks beside it made steps with a bias slower: 67 -> 73 us for nine prompts
                // of 200-800 tokens among single ones, short items.  It was not measured on long
                // prompts, which pay 708 -> 874 us for a bias in this form.)
                constexpr bool plain = !BIAS && !Q4;
                uint32_t sr[2][32];
                if (plain) {
                    tmem_ld32(tS, sr[0]);
                    tmem_ld32(tS + 32u, sr[1]);
                }
                auto mask = [&](uint32_t (&r)[32], int kk) {
                    const int lk = lim - 32 * kk, lok = lo - 32 * kk;
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = (e >= lok && e < lk) ? r[e] : __float_as_uint(-INFINITY);
                };
                // in place: scaled, biased and masked scores of chunk k, minus `shift`
                auto to_x = [&](uint32_t (&r)[32], int k, float shift) {
                    const int kk = 2 * hf + k;
                    if (hmask & (1u << k)) {
                        const float c1k = k ? cb[1] : cb[0];
                        const float2 sc = make_float2(xs, xs), add = make_float2(c1k - shift, c1k - shift);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float2 t2 = fma2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), sc, add);
                            r[e] = __float_as_uint(t2.x);
                            r[e + 1] = __float_as_uint(t2.y);
                        }
                    } else {
                        const int rk = rel - col0 - 32 * kk;  // relative position of the chunk's first column
                        const bool back = __all_sync(0xffffffffu, rk >= kThreeBuckets);
                        if (back || __all_sync(0xffffffffu, rk <= -31)) {
                            const int b0 = relpos_bucket(rk), s = back ? -1 : 1;
                            const int b1 = min(b0 + s, 31), b2 = min(b0 + 2 * s, 31);
                            // columns before e1 lie in b0, before e2 in b1
                            const int e1 = back ? rk - starts[b0] + 1 : starts[b1] + rk;
                            const int e2 = back ? rk - starts[b1] + 1 : (b1 == b0 ? 32 : starts[b2] + rk);
                            const float v0 = fmaf(__ldg(brow + b0), 1.4426950408889634f, -shift);
                            const float v1 = fmaf(__ldg(brow + b1), 1.4426950408889634f, -shift);
                            const float v2 = fmaf(__ldg(brow + b2), 1.4426950408889634f, -shift);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                r[e] = __float_as_uint(fmaf(__uint_as_float(r[e]), xs, e < e1 ? v0 : e < e2 ? v1 : v2));
                        } else if (near_ok) {
                            const float* tab = near_tab + head * C::kStride;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                r[e] = __float_as_uint(fmaf(__uint_as_float(r[e]), xs, tab[abs(rk - e)] - shift));
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float bv = __ldg(brow + relpos_bucket(rk - e));
                                r[e] = __float_as_uint(fmaf(__uint_as_float(r[e]), xs, fmaf(bv, 1.4426950408889634f, -shift)));
                            }
                        }
                    }
                    if (!full) mask(r, kk);
                };
                // raw scores' maximum, of those the row sees
                auto raw_max = [&](const uint32_t (&r)[32], int kk) {
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    if (full) {
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
                    } else {
                        const int lk = lim - 32 * kk, lok = lo - 32 * kk;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            m4[e & 3] = fmaxf(m4[e & 3], (e >= lok && e < lk) ? __uint_as_float(r[e]) : -INFINITY);
                    }
                    return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                };
                // pass 1: this half's row maximum, from the raw scores where the bias is one value
                float mx = -INFINITY;
                if (plain) {
                    tmem_ld_wait(sr[0]);
                    tmem_ld_wait(sr[1]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) mx = fmaxf(mx, fmaf(raw_max(sr[k], 2 * hf + k), xs, cb[k]));
                } else {
#pragma unroll 1
                    for (int k = 0; k < 2; ++k) {
                        uint32_t(&r)[32] = sr[0];
                        tmem_ld32(tS + 32u * k, r);
                        tmem_ld_wait(r);
                        if (hmask & (1u << k)) {
                            mx = fmaxf(mx, fmaf(raw_max(r, 2 * hf + k), xs, (k ? cb[1] : cb[0])));
                        } else {
                            to_x(r, k, 0.f);
#pragma unroll
                            for (int e = 0; e < 32; e += 2) mx = fmax3(mx, __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
                        }
                    }
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
                auto exps = [&](const uint32_t (&r)[32], int kk) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 e2 = make_float2(ex2_approx(__uint_as_float(r[e])), ex2_approx(__uint_as_float(r[e + 1])));
                        rs[(e >> 1) & 1] = add2(rs[(e >> 1) & 1], e2);
                        pk[e >> 1] = Q4 ? pack_f16x2(e2.x, e2.y) : pack_bf16x2(e2.x, e2.y);
                    }
                    tmem_st16(tSt + 32u * kk, pk);
                };
                if (plain) {
                    tmem_ld32(tS, sr[0]);  // the raw scores again: cheaper than 64 live registers
                    tmem_ld32(tS + 32u, sr[1]);
                    tmem_ld_wait(sr[0]);
                    tmem_ld_wait(sr[1]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float2 xs2 = make_float2(xs, xs), add = make_float2(cb[k] - m_use + kLift, cb[k] - m_use + kLift);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float2 t2 = fma2(make_float2(__uint_as_float(sr[k][e]), __uint_as_float(sr[k][e + 1])), xs2, add);
                            sr[k][e] = __float_as_uint(t2.x);
                            sr[k][e + 1] = __float_as_uint(t2.y);
                        }
                        if (!full) mask(sr[k], 2 * hf + k);
                        exps(sr[k], 2 * hf + k);
                    }
                } else {
#pragma unroll 1
                    for (int k = 0; k < 2; ++k) {
                        tmem_ld32(tS + 32u * k, sr[0]);
                        tmem_ld_wait(sr[0]);
                        to_x(sr[0], k, m_use - kLift);
                        exps(sr[0], 2 * hf + k);
                    }
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
            m -= kLift;
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
                const float inv = lt > 0.f ? (Q4 ? p.o_mul : 1.f) / lt : 0.f;
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
            // An item cut between blocks: leave this part, and with the first one the record
            // by which the merge kernel finds the item.
            const int prow = sp.split ? t : x * rt + t;  // row of the item
            if (owner) {
                float* part = p.part + size_t(part_slot) * C::kPart;
                float4* po = reinterpret_cast<float4*>(part);
                if (n > 0) {
#pragma unroll
                    for (int c = 0; c < OC / 32; ++c) {
                        float v[32];
                        load_o(c, 1.f, v);
                        if (row_valid) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                po[((OC * hf + 32 * c) / 4 + e) * C::kPair + prow] =
                                    make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                        }
                    }
                    release();
                }
                if (hf == 0 && row_valid) {
                    part[C::kPair * D + prow] = m;
                    part[C::kPair * D + C::kPair + prow] = n > 0 ? lt : 0.f;
                }
            }
            const int rows = min(2 * rt, R - 2 * g.tile * rt);
            if (int(threadIdx.x) * 64 < rows && g.k0 == 0) {
                if (threadIdx.x == 0) p.cuts[first] = CacheCut{g.s.q0, rows, 2 * g.tile * rt, g.hk * p.g, first, last, {0, 0}};
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

// Adds up the parts of the items cut between blocks.  A task is 64 rows of the item that starts
// in a block and goes on past it; its flag says whether there is one.  Bound by the latency of
// its few loads for most calls, and by the parts' bytes for long prompts (42 MB for the 8 prompts
// above: 17 us from DRAM, less from L2).  The grid is small and a
// CTA looks at the flags of all its tasks at once, clearing them for the next call: most calls
// cut few items, and a CTA for each possible task would cost 10 us to find nothing to do.
// A thread takes one row and a quarter of the columns, some parts at a time against a running
// maximum; a warp's loads are whole lines, since parts are stored four columns of all rows at a
// time.
constexpr int kMergeThreads = 256;
template <int D>
__device__ __forceinline__ void merge_rows(const CacheFwdParams& p, const CacheCut& cut, int row, int group) {
    constexpr int kPart = cache_merge_part(D), NV = D / 16, kAtOnce = D == 128 ? 2 : 4;  // NV: float4s of a thread
    if (row >= cut.rows) return;
    float m = -INFINITY, l = 0.f;
    float4 v[NV];
#pragma unroll
    for (int e = 0; e < NV; ++e) v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = cut.first; c <= cut.last; c += kAtOnce) {
        float mc[kAtOnce], lc[kAtOnce], top = m;
        float4 u[kAtOnce][NV];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            mc[k] = -INFINITY;
            if (c + k > cut.last) continue;
            const float* q = p.part + size_t(cache_slot(c + k, cut.first)) * kPart;
            const float4* q4 = reinterpret_cast<const float4*>(q) + group * NV * kMergeRows + row;
            mc[k] = q[kMergeRows * D + row];
            lc[k] = q[kMergeRows * D + kMergeRows + row];
#pragma unroll
            for (int e = 0; e < NV; ++e) u[k][e] = q4[e * kMergeRows];
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, mc[k]);
        if (top == -INFINITY) continue;
        const float keep = m == -INFINITY ? 0.f : ex2_approx(m - top);
        m = top;
        l *= keep;
#pragma unroll
        for (int e = 0; e < NV; ++e) v[e] = make_float4(v[e].x * keep, v[e].y * keep, v[e].z * keep, v[e].w * keep);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (mc[k] == -INFINITY) continue;  // no key of this part (or no part): its O is not set
            const float w = ex2_approx(mc[k] - top);
            l = fmaf(lc[k], w, l);
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                v[e].x = fmaf(u[k][e].x, w, v[e].x);
                v[e].y = fmaf(u[k][e].y, w, v[e].y);
                v[e].z = fmaf(u[k][e].z, w, v[e].z);
                v[e].w = fmaf(u[k][e].w, w, v[e].w);
            }
        }
    }
    const float inv = l > 0.f ? p.o_mul / l : 0.f;
    const int r = cut.row0 + row, tok = div_g(p, r);
    const size_t orow = size_t(cut.q0 + tok) * size_t(p.H) + size_t(cut.head0 + r - tok * p.g);
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        const size_t at = orow * D + group * (D / 4) + 4 * e;
        if (p.o_f32)
            *reinterpret_cast<float4*>(static_cast<float*>(p.O) + at) =
                make_float4(v[e].x * inv, v[e].y * inv, v[e].z * inv, v[e].w * inv);
        else
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + at) =
                make_uint2(pack_bf16x2(v[e].x * inv, v[e].y * inv), pack_bf16x2(v[e].z * inv, v[e].w * inv));
    }
    if (p.lse && group == 0) p.lse[orow] = l > 0.f ? (m + __log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// Whether a record is one of this call's: one that an earlier call left (in a workspace that was
// not zero) may name rows, heads or parts that this call does not have.
__device__ __forceinline__ bool cut_fits(const CacheFwdParams& p, const CacheCut& c, int blocks) {
    return c.q0 >= 0 && c.q0 < p.T && c.rows >= 1 && c.rows <= kMergeRows && c.row0 >= 0 && c.row0 <= INT_MAX - kMergeRows &&
           div_g(p, c.row0 + c.rows - 1) < p.T - c.q0 && c.head0 >= 0 && c.head0 <= p.H - p.g && c.first >= 0 &&
           c.first <= c.last && c.last < blocks;
}

template <int D>
__global__ void __launch_bounds__(kMergeThreads) jfa_cache_merge_kernel(const CacheFwdParams p, int blocks) {
    const int tasks = blocks * kMergeCtas;
    __shared__ uint32_t there;
    for (int base = blockIdx.x; base < tasks; base += 32 * gridDim.x) {  // 32 tasks of this CTA
        if (threadIdx.x < 32) {
            const int i = base + threadIdx.x * gridDim.x;
            const bool set = i < tasks && p.cut_flags[i] != 0u;
            if (set) p.cut_flags[i] = 0u;
            const uint32_t m = __ballot_sync(0xffffffffu, set);
            if (threadIdx.x == 0) there = m;
        }
        __syncthreads();
        for (uint32_t m = there; m; m &= m - 1) {
            const int i = base + (__ffs(m) - 1) * gridDim.x;
            const CacheCut cut = p.cuts[i / kMergeCtas];
            if (!cut_fits(p, cut, blocks)) {
                if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
                continue;
            }
            merge_rows<D>(p, cut, 64 * (i % kMergeCtas) + (threadIdx.x & 63), threadIdx.x >> 6);
        }
        __syncthreads();
    }
}

template <int D, bool BIAS, bool Q4>
cudaError_t launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, int num_sms, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    using C = ChkCfg<D, Q4>;
    cudaError_t e = allow_smem(jfa_cache_chunk_kernel<D, BIAS, Q4>, C::kSmemBytes, done);
    if (e != cudaSuccess) return e;
    jfa_cache_chunk_kernel<D, BIAS, Q4><<<num_sms, C::kThreads, C::kSmemBytes, st>>>(mq, mk, mv, p);
    return cudaGetLastError();
}

}  // namespace

size_t cache_chunk_part_bytes(int D, int num_sms) { return size_t(num_sms) * kBlocksPerCta * 2 * 256 * size_t(D + 2) * 4; }

cudaError_t launch_cache_chunk(int D, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                               const CacheFwdParams& p, int num_sms, cudaStream_t st) {
    if (D == 128)
        return p.bias ? launch<128, true, false>(mq, mk, mv, p, num_sms, st) : launch<128, false, false>(mq, mk, mv, p, num_sms, st);
    return p.bias ? launch<64, true, false>(mq, mk, mv, p, num_sms, st) : launch<64, false, false>(mq, mk, mv, p, num_sms, st);
}

cudaError_t launch_cache_chunk4(int D, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p,
                                int num_sms, cudaStream_t st) {
    if (D == 128)
        return p.bias ? launch<128, true, true>(mq, mk, mv, p, num_sms, st) : launch<128, false, true>(mq, mk, mv, p, num_sms, st);
    return p.bias ? launch<64, true, true>(mq, mk, mv, p, num_sms, st) : launch<64, false, true>(mq, mk, mv, p, num_sms, st);
}

cudaError_t launch_cache_merge(int D, const CacheFwdParams& p, int blocks, int num_sms, cudaStream_t st) {
    const int grid = num_sms * 4;
    if (D == 128)
        jfa_cache_merge_kernel<128><<<grid, kMergeThreads, 0, st>>>(p, blocks);
    else if (D == 32)
        jfa_cache_merge_kernel<32><<<grid, kMergeThreads, 0, st>>>(p, blocks);
    else
        jfa_cache_merge_kernel<64><<<grid, kMergeThreads, 0, st>>>(p, blocks);
    return cudaGetLastError();
}

}  // namespace jfa
