// Attention over a 4-bit paged cache for few rows: single tokens and short query sets.
//
// A position's key and value are 64 + 8 bytes a head of 128 each, so the stream that bounds the
// 16-bit decode kernel is 3.6 times shorter here, and what a CTA does with each byte shows.  The
// products are m16n8k16 with the keys on the 16 side and up to 8 (or two times 8) packed rows on the 8
// side,
//   S^T = K Q^T,   O^T += V^T P^T,
// so a code is unpacked once into the register it is multiplied from, and a token of up to 8
// grouped heads pays for 8 rows.  Unpacking is two codes an instruction to fp16 pairs, and one
// multiplication by the scale (exact: quant.cuh).
//   K^T: a lane reads a quarter of a key's row (D/8 bytes, one or two groups); the order of the
//        contraction is free, and the queries are laid out in the same one.
//   V^T: a lane reads an eighth of the rows of four keys, and pairs the codes of two keys by
//        exchanging half bytes before they are unpacked.  The 16 (or 8) columns that it gets are
//        neighbours, so its outputs are too.
//   P^T: the scores' fragment, transposed across the warp eight by eight.
// Which of 16 keys is which row of the product is free as well, and chosen so that the reads of V
// spread over the banks.
// Queries are taken to fp16 with a power of two per row that brings their largest magnitude to
// 2^14: they keep all of their bits down to 2^-28 of it (2^-39 of it is lost at most).
// P = 2^6 softmax weights against a maximum that moves lazily (at most 2^14), in fp16: 2^-11 of each
// weight, and 2^-31 of the largest.  Sums are taken in fp32 before.
// Stages of 128 keys pass through a ring of 54 KB per CTA, three CTAs an SM (two for 16 rows); one warp
// issues the loads (codes and scales of each page, by plain copies where a head's slots lie in one
// piece, else by tensor maps), four warps take 32 keys of each stage.  The warps merge at the end of an item;
// the parts of an item cut between CTAs are added by a kernel of their own (cache_join.cu).
// Measured, one token each of 32 query and 8 key heads of 128: 64 sequences of 200-16k keys (300 MB)
// 66 us, 4.5 TB/s, 0.68 of the copy rate; one history of 131k keys (151 MB) 37.6 us, 0.60; 64 lists of 64
// blocks of 32 keys (104 MB) 35.4 us, 0.44; one sequence of 1k keys 9.1 us.  The same stream with no
// arithmetic takes 52 us of the 66: the rest is instructions, 620 a warp for 32 keys (128 conversions and as many
// multiplications by scales among them), which fill half the issue slots; the warps wait for their own
// chains and, a fifth of the time, for code.  More warps do not help: four CTAs an SM at 96
// registers (which spill) 86 us instead of 69 then, two CTAs 73, 16 keys at a time in half the code 73.
#include "cache_common.cuh"
#include "quant.cuh"
#include "tilemath.cuh"

namespace jfa {

cudaError_t launch_cache_decode4(int D, const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, bool early,
                                 int num_sms, cudaStream_t st);
size_t cache_decode4_part_bytes(int D, int num_sms);

namespace {

constexpr float kLift = 6.f;  // log2 of the weights' factor

template <int D, int NT>
struct Cfg {
    // (eight consumer warps a CTA, two CTAs an SM, at 96 registers: 64 histories of 4-bit keys 84 us
    // instead of 75)
    static constexpr int kWarps = 4, kThreads = 32 * (kWarps + 1), kCtas = NT == 1 ? 3 : 2;
    static constexpr int BN = 32 * kWarps, BM = 8 * NT;
    static constexpr int kSlotsN = kWarps / 2;               // tiles of 8 rows in the merge of the warps
    static constexpr int kRow = D / 2, kScales = D / 16;     // bytes of a key's codes and scales
    static constexpr int kCodes = BN * kRow;
    static constexpr int kOffKS = 2 * kCodes, kOffVS = kOffKS + BN * kScales;
    static constexpr int kStage = kOffVS + BN * kScales;
    static constexpr int kStages = 55296 / kStage;
    static constexpr int kPitch = D + 4;                     // floats of a row in the merge's slots
    static constexpr int kSlot = 8 * kPitch;
    static constexpr int kOffSlots = kStages * kStage;
    static constexpr int kSlots = kSlotsN * kSlot * 4 > 8192 ? kSlotsN * kSlot * 4 : 8192;
    static constexpr int kOffML = kOffSlots + kSlots;        // [2 buffers][m, l][warp][row]
    static constexpr int kOffBias = kOffML + 2 * 2 * kWarps * 16 * 4;
    static constexpr int kOffBar = kOffBias + 16 * 33 * 4;
    static constexpr int kOffMisc = kOffBar + 2 * kStages * 8;
    static constexpr int kOffBase = (kOffMisc + 16 + int(sizeof(CacheStart)) + 15) / 16 * 16;  // lists: position of each box
    static constexpr int kBoxes = BN / 16;
    static constexpr int kBytes = kOffBase + kStages * kBoxes * 4 + 1024;
    static_assert(kCtas * (kBytes + 1024) <= 228 * 1024, "shared memory of an SM");
    static constexpr int kPart = 16 * (D + 2);               // floats of a partial result: O, m, l
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
template <int WARPS>
__device__ __forceinline__ void consumer_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(32 * WARPS) : "memory");
}

// Key of 16 that is row i of the product.
__device__ __forceinline__ int key_of(int i) {
    return (i & 8) | ((i & 1) << 2) | ((i >> 1) & 3);
}

template <int D, bool BIAS, bool LIST, int NT>
__global__ void __launch_bounds__((Cfg<D, NT>::kThreads), (Cfg<D, NT>::kCtas))
    jfa_cache_decode4_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                             const CacheFwdParams p) {
    using C = Cfg<D, NT>;
    constexpr int kWarps = C::kWarps, BM = C::BM, BN = C::BN, KG = 2, MT = D / 16, KS = D / 16, NR = 2 * NT;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto full = [&](uint32_t s) -> uint32_t { return sbase + C::kOffBar + 8u * s; };
    auto empty = [&](uint32_t s) -> uint32_t { return sbase + C::kOffBar + 8u * (C::kStages + s); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc);
    int* bases = reinterpret_cast<int*>(smem + C::kOffBase);  // [stage][box]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < uint32_t(C::kStages); ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kWarps);
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
    launch_dependents();  // (the join kernel waits for this one to end)
    CacheSeg g;

    if (warp == kWarps) {
        // ---------------------------------------------------------------- producer
        // A lane loads a page's (or 64 keys' of one) part of each stage: K and V, codes and scales.
        fence_proxy_async_smem();  // the scratch's writes before the first loads into it
        const int rows = min(1 << p.page_log2, 64);          // keys of a box
        const int per = BN / rows;                           // pages (or parts of one) in a stage
        const int pg = LIST ? lane & (per - 1) : lane;
        const bool mine = lane < per;
        const uint32_t box = uint32_t(pg * rows * C::kRow), sbox = uint32_t(C::kOffKS + pg * rows * C::kScales);
        uint32_t it = 0;
        bool ok = true, more = cur.next(p, g);
        int kt = g.k0;
        // A stage, as this lane sees it: its block of the sequence (-1: nothing to load), that block's page,
        // the slot and the position of the first key.  Its list entry is asked for two stages before it
        // is loaded, its page one stage, so that the stream waits for neither; whether the entry counts is seen when it
        // is loaded, the first time while its page is on the way.
        struct Stage {
            bool have, read, met, head, starts, ends;  // read: a page; lists: an entry, the first, a new list, an entry's last stage
            int hk, block, last, slot, base, page, at;  // last: the entry before
            size_t row;                                // of the page table
        };
        CacheListScan scan;
        bool starts = false;
        auto list_of = [&](const CacheSeg& s) {
            return p.lists + (size_t(s.s.q0 + s.tile) * size_t(p.Hkv) + size_t(s.hk)) * size_t(p.n_list);
        };
        auto step = [&](Stage& s) {
            while (more && (g.r.n == 0 || kt >= g.k1)) {
                more = cur.next(p, g);
                kt = g.k0;
                starts = true;
            }
            s.have = more;
            s.block = -1;
            s.base = kNoBlock;
            if (!more) return;
            const int j0 = (g.r.f + kt++) * BN, j = j0 + pg * rows;
            s.hk = g.hk;
            s.slot = j & ((1 << p.page_log2) - 1);
            s.row = size_t(g.b) * size_t(p.max_pages);
            if constexpr (LIST) {
                const int e = j >> p.page_log2;
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
            } else if (mine && j < g.r.hi && j + rows > g.r.lo) {
                s.block = j >> p.page_log2;
            }
        };
        auto look = [&](Stage& s) {
            bool in = s.block >= 0;
            if constexpr (LIST) {  // (blocks past the token's own hold no key that it may see)
                in = in && mine && s.block <= s.at >> p.page_log2;
                s.base = int(uint32_t(s.block) << p.page_log2) + s.slot;
                in = in && s.base <= s.at;
            }
            s.page = in ? p.table[s.row + size_t(s.block)] : -1;
            s.read = in;
        };
        Stage now, next;
        step(now);
        if (now.have) {
            look(now);
            if constexpr (LIST) scan.start(list_of(g), (g.k0 * BN) >> p.page_log2, lane);
        }
        step(next);
        while (now.have) {
            const Stage s = now;
            now = next;
            if (now.have) {
                look(now);
                step(next);
            }
            bool in = s.read;
            if constexpr (LIST) {
                if (s.starts) scan = CacheListScan();
                const bool counts = scan.counts(s.block, s.met, s.head ? 0u : CacheListScan::key(s.last), p.page_log2 <= 6, s.ends, per, pg, p.status);
                in = in && counts;
            }
            const uint32_t st = it % C::kStages, ph = (it / C::kStages) & 1;
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(empty(st), ph ^ 1, abort_flag))) {
                ok = false;
                break;
            }
            const int n = __popc(__ballot_sync(0xffffffffu, in));
            if constexpr (LIST) {
                if (mine) bases[st * C::kBoxes + pg] = in ? s.base : kNoBlock;
                __syncwarp();
            }
            if (lane == 0) mbar_arrive_expect_tx(full(st), uint32_t(n * rows * 2 * (C::kRow + C::kScales)));
            __syncwarp();
            if (in) {
                const uint32_t dst = sbase + st * C::kStage, bytes = uint32_t(rows * C::kScales), codes = uint32_t(rows * C::kRow);
                // (a bad entry is reported; any page will do for it)
                const bool bad = s.page < 0 || s.page >= p.n_pages;
                if (bad) atomicOr(p.status, kStatusBounds);
                const int page = bad ? 0 : s.page;
                if (p.dense) {
                    bulk_load(dst + box, static_cast<const uint8_t*>(p.K) + page * p.ks[0] + s.hk * p.ks[2] + s.slot * C::kRow, codes, full(st));
                    bulk_load(dst + C::kCodes + box, static_cast<const uint8_t*>(p.V) + page * p.vs[0] + s.hk * p.vs[2] + s.slot * C::kRow, codes,
                              full(st));
                } else {
                    tma_load_4d(dst + box, &tmK, full(st), 0, s.slot, s.hk, page);
                    tma_load_4d(dst + C::kCodes + box, &tmV, full(st), 0, s.slot, s.hk, page);
                }
                bulk_load(dst + sbox, p.k_scales + page * p.kss[0] + s.hk * p.kss[1] + s.slot * C::kScales, bytes, full(st));
                bulk_load(dst + (C::kOffVS - C::kOffKS) + sbox, p.v_scales + page * p.vss[0] + s.hk * p.vss[1] + s.slot * C::kScales, bytes,
                          full(st));
            }
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
    CacheCut cut = cache_no_cut();
    const int kkey = key_of(qrow);                        // this lane's key of a fragment's first 8 (and 8 on)
    int vkey[4];                                             // its four keys of V^T
#pragma unroll
    for (int c = 0; c < 4; ++c) vkey[c] = key_of(2 * quad + (c & 1) + 8 * (c >> 1));
    // where they lie in 16 keys: K's row, V's of vkey[0] and vkey[1]
    constexpr int kR = C::kRow, kSc = C::kScales;
    const uint32_t k_at = uint32_t(kkey * kR + (D == 128 ? 16 : 8) * quad);
    const uint32_t ks_at = uint32_t(kkey * kSc + (D == 128 ? 2 * quad : quad));
    uint32_t v_at[2];
#pragma unroll
    for (int c = 0; c < 2; ++c)
        v_at[c] = uint32_t(vkey[c] * kR + (D == 128 ? 8 : 4) * qrow);
    const uint32_t vs_at = uint32_t(  // (vkey[1] is 4 keys on)
        vkey[0] * kSc + (D == 128 ? qrow : qrow >> 1));
    while (cur.next(p, g)) {
        const int R = g.s.q_len * p.g, diag = g.s.kv_len - g.s.q_len, r0 = g.tile * p.bm;
        const int nr = min(LIST ? p.bm : BM, R - r0);
        if (BIAS) {  // the rows' bias, for this item's heads
            for (int e = threadIdx.x; e < nr * 32; e += 32 * kWarps) {
                const int r = r0 + (e >> 5);
                btab[(e >> 5) * 33 + (e & 31)] =
                    p.bias[(g.hk * p.g + r - div_g(p, r) * p.g) * 32 + (e & 31)] * 1.4426950408889634f;
            }
        }
        // queries: row 8 x + qrow, columns D/4 quad .. in the order of the keys' codes
        uint32_t qb[NT][KS][2];
        float rs[NR];  // what takes a score of row 8 x + 2 quad + e to log2 units
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            const int rr = 8 * x + qrow;
            const bool in = rr < nr;
            const int r = r0 + (in ? rr : 0), tok = div_g(p, r), head = g.hk * p.g + r - tok * p.g;
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.Q) + (g.s.q0 + tok) * p.q_stride +
                                                              int64_t(head) * D + (D / 4) * quad);
            uint32_t raw[D / 8];
#pragma unroll
            for (int v = 0; v < D / 32; ++v) {
                const uint4 u = in ? src[v] : make_uint4(0u, 0u, 0u, 0u);
                raw[4 * v] = u.x;
                raw[4 * v + 1] = u.y;
                raw[4 * v + 2] = u.z;
                raw[4 * v + 3] = u.w;
            }
            float top = 0.f;
#pragma unroll
            for (int v = 0; v < D / 8; ++v)
                top = fmax3(top, fabsf(__uint_as_float(raw[v] << 16)), fabsf(__uint_as_float(raw[v] & 0xffff0000u)));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const uint32_t e = max(__float_as_uint(top) >> 23, 15u);
            const float up = __uint_as_float((268u - e) << 23), down = __uint_as_float((e - 14u) << 23);  // 2^(14 - log2 top), and back
#pragma unroll
            for (int v = 0; v < D / 8; ++v)
                qb[x][v >> 1][v & 1] = pack_f16x2(__uint_as_float(raw[v] << 16) * up, __uint_as_float(raw[v] & 0xffff0000u) * up);
#pragma unroll
            for (int i = 0; i < 2; ++i)  // (not 0, which would not leave a masked score at -inf; scores are below 2^33)
                rs[2 * x + i] = fmaxf(p.scale_log2 * __shfl_sync(0xffffffffu, down, 4 * (2 * quad + i)), 1e-37f);
        }
        // the rows of this lane's scores
        int lim[NR], low[NR], rel[NR];
        const float* brow[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int rr = 8 * (i >> 1) + 2 * quad + (i & 1);
            rel[i] = div_g(p, r0 + (rr < nr ? rr : 0)) + diag;
            lim[i] = p.causal ? min(g.s.kv_len, rel[i] + 1) : g.s.kv_len;
            low[i] = p.window >= 0 ? rel[i] - p.window : 0;
            brow[i] = btab + (rr < nr ? rr : 0) * 33;
        }
        if (BIAS) consumer_sync<kWarps>();
        // keys that every row of the tile sees: no mask in [all_lo, all_hi)
        const int t_first = div_g(p, r0), t_last = div_g(p, r0 + nr - 1);
        const int all_hi = p.causal ? min(g.s.kv_len, t_first + diag + 1) : g.s.kv_len;
        const int all_lo = p.window >= 0 ? max(0, t_last + diag - p.window) : 0;
        float m[NR], l[NR], o[MT][NT][4];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < MT; ++n)
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][x][i] = 0.f;
        const int k_end = g.r.n > 0 ? g.k1 : g.k0;
        for (int kt = g.k0; kt < k_end; ++kt, ++it) {
            const uint32_t st = it % C::kStages, ph = (it / C::kStages) & 1;
            if (ok && !__all_sync(0xffffffffu, mbar_wait_bounded(full(st), ph, abort_flag))) {
                ok = false;
                *abort_flag = 1;
                if (lane == 0) atomicOr(p.status, kStatusTimeout);
            }
            if (!ok) continue;
            const uint32_t sK = sbase + st * C::kStage + 16 * KG * warp * C::kRow, sV = sK + C::kCodes;
            const uint32_t sKS = sbase + st * C::kStage + C::kOffKS + 16 * KG * warp * C::kScales, sVS = sKS + (C::kOffVS - C::kOffKS);
            int at16[KG];  // the position of each 16 keys
            int hi = g.r.hi;
            const int lo = g.r.lo;
            if constexpr (LIST) {
                const int brows = min(1 << p.page_log2, 64);
#pragma unroll
                for (int q = 0; q < KG; ++q) {
                    const int c = 16 * (KG * warp + q);
                    at16[q] = bases[st * C::kBoxes + c / brows] + (c & (brows - 1));
                }
                hi = all_hi;
            } else {
#pragma unroll
                for (int q = 0; q < KG; ++q) at16[q] = (g.r.f + kt) * BN + 16 * (KG * warp + q);
            }
            if (at16[0] >= hi && at16[KG - 1] >= hi) {  // nothing of this warp's to see
                __syncwarp();
                if (lane == 0) mbar_arrive(empty(st));
                continue;
            }
            float s[KG][NT][4];
#pragma unroll
            for (int q = 0; q < KG; ++q)
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[q][x][i] = 0.f;
#pragma unroll
            for (int q = 0; q < KG; ++q) {
                uint32_t w[2][D / 32], sc[2][D / 64];  // codes and scales of keys kkey, kkey + 8
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t row = uint32_t((16 * q + 8 * i) * kR), srow = uint32_t((16 * q + 8 * i) * kSc);
                    if constexpr (D == 128) {
                        const uint4 u = ld_shared_v4(sK + k_at + row);
                        w[i][0] = u.x;
                        w[i][1] = u.y;
                        w[i][2] = u.z;
                        w[i][3] = u.w;
                        const uint32_t two = e4m3_to_f16(lds16(sKS + ks_at + srow));
                        sc[i][0] = __byte_perm(two, 0u, 0x1010);
                        sc[i][1] = __byte_perm(two, 0u, 0x3232);
                    } else {
                        const uint2 u = lds64(sK + k_at + row);
                        w[i][0] = u.x;
                        w[i][1] = u.y;
                        sc[i][0] = e4m3_to_f16(lds8(sKS + ks_at + srow) * 0x101u);
                    }
                }
#pragma unroll
                for (int v = 0; v < D / 32; ++v) {
                    uint32_t a0[4], a1[4];
                    e2m1_to_f16(w[0][v], a0);
                    e2m1_to_f16(w[1][v], a1);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a[4] = {f16_mul2(a0[2 * h], sc[0][v >> 1]), f16_mul2(a1[2 * h], sc[1][v >> 1]),
                                               f16_mul2(a0[2 * h + 1], sc[0][v >> 1]), f16_mul2(a1[2 * h + 1], sc[1][v >> 1])};
#pragma unroll
                        for (int x = 0; x < NT; ++x) mma_f16(s[q][x], a, qb[x][2 * v + h][0], qb[x][2 * v + h][1]);
                    }
                }
            }
            // scores of rows 2 quad + (i & 1) of each 8, at keys kkey (i < 2) and kkey + 8
#pragma unroll
            for (int q = 0; q < KG; ++q) {
                const int a16 = at16[q];
                if (BIAS) {
                    const int far = t_last + diag - a16, near = t_first + diag - (a16 + 15);
                    const int bk = relpos_bucket(far);
                    const bool one = (near >= 0 || far <= 0) && bk == relpos_bucket(near);
#pragma unroll
                    for (int x = 0; x < NT; ++x)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int ri = 2 * x + (i & 1);
                            const int b = one ? bk : relpos_bucket(rel[ri] - (a16 + kkey + 8 * (i >> 1)));
                            s[q][x][i] = fmaf(s[q][x][i], rs[ri], brow[ri][b]);
                        }
                }
                if (a16 < all_lo || a16 + 16 > all_hi) {
#pragma unroll
                    for (int x = 0; x < NT; ++x)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int ri = 2 * x + (i & 1), j = a16 + kkey + 8 * (i >> 1);
                            if (j >= lim[ri] || j < low[ri]) s[q][x][i] = -INFINITY;
                        }
                }
            }
            // The maximum moves only when it would grow by more than 2^8: sums and O stay in its
            // units, and P stays below 2^14.
            float mx[NR];
            bool grow = false;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int x = i >> 1, e = i & 1;
                mx[i] = fmaxf(fmaxf(s[0][x][e], s[0][x][e + 2]), fmaxf(s[1][x][e], s[1][x][e + 2]));
                if (!BIAS) mx[i] *= rs[i];  // (with a bias the scores are in log2 units already)
                grow = grow || mx[i] > m[i] + 8.f;
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int i = 0; i < NR; ++i) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], d));
                    const float to = mx[i] > m[i] + 8.f ? mx[i] : m[i];
                    const float a = m[i] == -INFINITY ? 0.f : ex2_approx(m[i] - to);
                    m[i] = to;
                    l[i] *= a;
#pragma unroll
                    for (int n = 0; n < MT; ++n) {
                        o[n][i >> 1][i & 1] *= a;
                        o[n][i >> 1][2 + (i & 1)] *= a;
                    }
                }
            }
            uint32_t pb[KG][NT][2];
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                const float u0 = m[2 * x] == -INFINITY ? 0.f : m[2 * x] - kLift, u1 = m[2 * x + 1] == -INFINITY ? 0.f : m[2 * x + 1] - kLift;
#pragma unroll
                for (int q = 0; q < KG; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float e0 = ex2_approx(BIAS ? s[q][x][2 * h] - u0 : fmaf(s[q][x][2 * h], rs[2 * x], -u0));
                        const float e1 = ex2_approx(BIAS ? s[q][x][2 * h + 1] - u1 : fmaf(s[q][x][2 * h + 1], rs[2 * x + 1], -u1));
                        l[2 * x] += e0;
                        l[2 * x + 1] += e1;
                        pb[q][x][h] = transposed(pack_f16x2(e0, e1));
                    }
            }
#pragma unroll
            for (int q = 0; q < KG; ++q) {
                uint32_t w[4][D / 64], sb[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t row = uint32_t((16 * q + 8 * (c >> 1)) * kR), srow = uint32_t((16 * q + 8 * (c >> 1)) * kSc);
                    if constexpr (D == 128) {
                        const uint2 u = lds64(sV + v_at[c & 1] + row);
                        w[c][0] = u.x;
                        w[c][1] = u.y;
                    } else {
                        w[c][0] = lds32(sV + v_at[c & 1] + row);
                    }
                    sb[c] = lds8(sVS + vs_at + (c & 1 ? uint32_t(4 * kSc) : 0u) + srow);
                }
                // Scales of keys that no row may see are undefined, and 0 * NaN is not 0.
                if (at16[q] < lo || at16[q] + 16 > hi) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int j = at16[q] + vkey[c];
                        if (j < lo || j >= hi) sb[c] = 0u;
                    }
                }
                const uint32_t s01 = e4m3_to_f16(sb[0] | (sb[1] << 8)), s23 = e4m3_to_f16(sb[2] | (sb[3] << 8));
#pragma unroll
                for (int v = 0; v < D / 64; ++v) {
                    // half bytes of keys 0, 1 and 2, 3 side by side: even columns, odd columns
                    constexpr uint32_t L = 0x0f0f0f0fu;
                    uint32_t e01[4], o01[4], e23[4], o23[4];
                    e2m1_to_f16((w[0][v] & L) | ((w[1][v] << 4) & ~L), e01);
                    e2m1_to_f16(((w[0][v] >> 4) & L) | (w[1][v] & ~L), o01);
                    e2m1_to_f16((w[2][v] & L) | ((w[3][v] << 4) & ~L), e23);
                    e2m1_to_f16(((w[2][v] >> 4) & L) | (w[3][v] & ~L), o23);
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const uint32_t a[4] = {f16_mul2(e01[n], s01), f16_mul2(o01[n], s01), f16_mul2(e23[n], s23), f16_mul2(o23[n], s23)};
#pragma unroll
                        for (int x = 0; x < NT; ++x) mma_f16(o[4 * v + n][x], a, pb[q][x][0], pb[q][x][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(st));
        }
        // ------------------------------------------------------------ end of the item's part
        // Merge the warps: m and l of every row, then O, 8 rows at a time: the second half of the
        // warps into slots, the first onto them, and the slots' sum out.
        float* mw = ml + (seg_no & 1) * (2 * kWarps * 16);
        float* lw = mw + kWarps * 16;
        ++seg_no;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
            if (qrow == 0) {
                mw[warp * 16 + 8 * (i >> 1) + 2 * quad + (i & 1)] = m[i] - kLift;
                lw[warp * 16 + 8 * (i >> 1) + 2 * quad + (i & 1)] = l[i];
            }
        }
        consumer_sync<kWarps>();
        const bool whole = g.whole();
        int first = 0, last = 0;
        if (!whole) {
            first = cache_first_cta(p, *start, g);
            last = cache_last_cta(p, *start, g);
        }
        float* part = p.part + size_t(cache_slot(blockIdx.x, first)) * C::kPart;
        constexpr int CW = D / 16;  // columns of a thread: 16 threads a row
        const int ocol = CW * (threadIdx.x & 15);
        float* slot = slots + (warp % C::kSlotsN) * C::kSlot + (D / 8) * qrow;
#pragma unroll
        for (int h = 0; h < NT; ++h) {
            if (8 * h >= nr) break;
            if (h) consumer_sync<kWarps>();
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * h + 2 * quad + e;
                float mm = mw[r];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, mw[16 * w + r]);
                f[e] = m[2 * h + e] == -INFINITY ? 0.f : ex2_approx(m[2 * h + e] - kLift - mm);
            }
            auto put = [&](bool add) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int n = 0; n < MT; n += 2) {
                        float4* dst = reinterpret_cast<float4*>(slot + (2 * quad + e) * C::kPitch + 2 * n);
                        float4 x = make_float4(o[n][h][e] * f[e], o[n][h][2 + e] * f[e], o[n + 1][h][e] * f[e], o[n + 1][h][2 + e] * f[e]);
                        if (add) {
                            const float4 y = *dst;
                            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                        }
                        *dst = x;
                    }
            };
            if (warp >= C::kSlotsN) put(false);
            consumer_sync<kWarps>();
            if (warp < C::kSlotsN) put(true);
            // this thread's row: its maximum and sum
            const int orow = 8 * h + ((threadIdx.x & 127) >> 4);
            float om = -INFINITY, ol = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) om = fmaxf(om, mw[16 * w + orow]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mm = mw[16 * w + orow];
                ol = fmaf(mm == -INFINITY ? 0.f : ex2_approx(mm - om), lw[16 * w + orow], ol);
            }
            consumer_sync<kWarps>();
            const float* a = slots + (orow & 7) * C::kPitch + ocol;
            float v[CW];
#pragma unroll
            for (int e = 0; e < CW; e += 4) {
                float4 x = *reinterpret_cast<const float4*>(a + e);
#pragma unroll
                for (int k = 1; k < C::kSlotsN; ++k) {
                    const float4 y = *reinterpret_cast<const float4*>(a + k * C::kSlot + e);
                    x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                }
                v[e] = x.x;
                v[e + 1] = x.y;
                v[e + 2] = x.z;
                v[e + 3] = x.w;
            }
            if (threadIdx.x >= 128 || orow >= nr || !ok) continue;
            if (!whole) {
#pragma unroll
                for (int e = 0; e < CW; e += 4)
                    *reinterpret_cast<float4*>(part + orow * D + ocol + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                if (ocol == 0) {
                    part[16 * D + orow] = om;
                    part[16 * D + 16 + orow] = ol;
                }
                continue;
            }
            const int r = r0 + orow, tok = div_g(p, r);
            const size_t at = size_t(g.s.q0 + tok) * size_t(p.H) + size_t(g.hk * p.g + r - tok * p.g);
            const float inv = ol > 0.f ? p.o_mul / ol : 0.f;
#pragma unroll
            for (int e = 0; e < CW; e += 4) {
                if (p.o_f32)
                    *reinterpret_cast<float4*>(static_cast<float*>(p.O) + at * D + ocol + e) =
                        make_float4(v[e] * inv, v[e + 1] * inv, v[e + 2] * inv, v[e + 3] * inv);
                else
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + at * D + ocol + e) =
                        make_uint2(pack_bf16x2(v[e] * inv, v[e + 1] * inv), pack_bf16x2(v[e + 2] * inv, v[e + 3] * inv));
            }
            if (ocol == 0 && p.lse) p.lse[at] = ol > 0.f ? (om + __log2f(ol)) * 0.6931471805599453f : -INFINITY;
        }
        // (an item cut between CTAs: the first part's CTA leaves the record)
        if (!whole && g.k0 == 0 && ok) cut = CacheCut{g.s.q0, nr, r0, g.hk * p.g, first, last, {0, 0}};
    }
    if (threadIdx.x == 0) p.cuts[blockIdx.x] = ok ? cut : cache_no_cut();
}

template <int D, bool BIAS, bool LIST, int NT>
cudaError_t launch(const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, bool early, int num_sms,
                   cudaStream_t st) {
    using C = Cfg<D, NT>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(jfa_cache_decode4_kernel<D, BIAS, LIST, NT>, C::kBytes, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms * C::kCtas);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kBytes;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = early ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, jfa_cache_decode4_kernel<D, BIAS, LIST, NT>, mk, mv, p);
    return e == cudaSuccess ? launch_cache_join(D, p, num_sms * C::kCtas, st) : e;
}

template <int D, bool LIST>
cudaError_t launch(const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, bool early, int num_sms,
                   cudaStream_t st) {
    if (p.bm <= 8)
        return p.bias ? launch<D, true, LIST, 1>(mk, mv, p, early, num_sms, st) : launch<D, false, LIST, 1>(mk, mv, p, early, num_sms, st);
    return p.bias ? launch<D, true, LIST, 2>(mk, mv, p, early, num_sms, st) : launch<D, false, LIST, 2>(mk, mv, p, early, num_sms, st);
}

}  // namespace

// The records, then the parts.
constexpr size_t kRecordBytes = size_t(3) * kMaxSms * sizeof(CacheCut);

size_t cache_decode4_part_bytes(int D, int num_sms) { return kRecordBytes + size_t(num_sms) * 3 * 2 * 16 * size_t(D + 2) * 4; }

cudaError_t launch_cache_decode4(int D, const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& call, bool early,
                                 int num_sms, cudaStream_t st) {
    CacheFwdParams p = call;  // (the chunk kernel, which may run at the same time, has records of its own)
    p.cuts = reinterpret_cast<CacheCut*>(p.part);
    p.part += kRecordBytes / sizeof(float);
    if (p.lists)
        return D == 128 ? launch<128, true>(mk, mv, p, early, num_sms, st) : launch<64, true>(mk, mv, p, early, num_sms, st);
    return D == 128 ? launch<128, false>(mk, mv, p, early, num_sms, st) : launch<64, false>(mk, mv, p, early, num_sms, st);
}

}  // namespace jfa
