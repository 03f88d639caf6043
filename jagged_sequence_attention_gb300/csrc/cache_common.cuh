// Paged-cache attention: what the kernels share.
//
// The new tokens of sequence b and the g = H / Hkv query heads of one key head hk form
// R_b = q_len_b * g packed rows (row r: token r / g, head hk * g + r % g), so grouped heads
// share every key and value read.  Rows are cut into tiles of p.bm, keys into tiles of BN; an
// item is a (sequence, key head, row tile) and its units are the key tiles it visits (at
// least one, so that rows without a key still get their zeros).
//
// Work split: all units of the batch, in the order (sequence, key head, row tile, key tile),
// are cut into equal contiguous ranges, one per CTA.  Lengths live on the device only (a
// captured graph is replayed on new ones), so each CTA finds its range itself from the
// arrays: one read of the lengths, a scan, and a search.  An item whose units fall to several CTAs
// is finished by the last of them to arrive (a counter per item), which adds their partial
// results in unit order, so the result does not depend on who arrives last.
#pragma once

#include "jfa_internal.h"
#include "ptx.cuh"

#include <atomic>
#include <climits>

namespace jfa {

constexpr int kCacheMaxB = 1 << 13, kCacheMaxGroups = kCacheMaxB / 32;
constexpr int kBlocksPerCta = 4;  // chunk kernel: blocks of the last part of the work, per CTA
constexpr int kMergeCtas = 4;     // merge tasks of a cut item of it, 64 rows each
constexpr int kMaxSms = 320;
// Words of the workspace's zeroed part: pieces drawn and CTAs done (chunk kernel), arrivals of
// split items (the other kernels, at most 3 CTAs an SM), flags of cut items (chunk kernel).
constexpr int kCtrDrawn = 0, kCtrDone = 1, kCtrSplit = 64, kCtrCuts = kCtrSplit + 3 * kMaxSms,
              kCtrEnd = kCtrCuts + kMaxSms * kBlocksPerCta * kMergeCtas;
static_assert(kCtrEnd * 4 <= JFA_CACHE_ZERO_BYTES, "counters fit the zeroed part");

// An item cut between blocks: `rows` packed rows from row0 on of the sequence at q0, heads
// from head0 on, blocks first .. last.
struct CacheCut {
    int q0, rows, row0, head0, first, last;
    int pad[2];
};

struct CacheFwdParams {
    const int32_t* q_off;    // [B+1]
    const int32_t* kv_lens;  // [B]
    const int32_t* table;    // [B, max_pages]
    int B, max_pages, T, max_kv;
    int H, Hkv, g;
    uint32_t g_mul, g_shift; // division by g (div_g)
    int page_log2, n_pages;
    int causal, window;      // window: -1 none
    float scale_log2;        // scale * log2(e)
    const float* bias;       // [H,32] or nullptr
    const void* Q;
    int64_t q_stride;        // elements between tokens
    void* O;
    int o_f32;
    float* lse;              // or nullptr
    const void* K;
    const void* V;
    int64_t ks[3], vs[3];    // page, slot, head strides (elements)
    uint32_t* counters;      // workspace: arrivals per split item, pieces drawn (zero between calls)
    uint32_t* cut_flags;     // workspace (zero between calls): [block][kMergeCtas]
    CacheCut* cuts;          // workspace: [block]
    float* part;             // workspace: partial results, two slots per CTA or block
    int* status;
    int min_units;           // units a CTA takes at least
    int item_cost;           // units that stand for an item's start and end (cache_units)
    int row_lo, row_hi;      // sequences this launch works on: row_lo < q_len * g <= row_hi
    int bm;                  // packed rows of an item
    int tile_tokens;         // chunk kernel: tokens of one of an item's two tiles
};

struct CacheSeq {
    int q0, q_len, kv_len;
};

// r / g for 0 <= r < 2^31, by a multiplication: with l = ceil(log2 g) and
// g_mul = floor(2^32 (2^l - g) / g) + 1, floor(r / g) = (hi32(r g_mul) + r) >> l exactly
// (Granlund and Montgomery 1994; the sum fits 32 bits since r < 2^31).
__host__ inline void set_div_g(CacheFwdParams& p) {
    uint32_t l = 0;
    while ((1u << l) < uint32_t(p.g)) ++l;
    p.g_shift = l;
    p.g_mul = uint32_t((uint64_t(1) << 32) * ((uint64_t(1) << l) - uint64_t(p.g)) / uint64_t(p.g)) + 1u;
}
__device__ __forceinline__ int div_g(const CacheFwdParams& p, int r) {
    return int((__umulhi(uint32_t(r), p.g_mul) + uint32_t(r)) >> p.g_shift);
}
// Sequence b's lengths; a bad sequence reads as empty.  In bad: whether it is one.
__device__ __forceinline__ CacheSeq cache_seq(const CacheFwdParams& p, int b, bool& bad) {
    const int q0 = p.q_off[b], q1 = p.q_off[b + 1], kv = p.kv_lens[b];
    bad = q0 < 0 || q1 < q0 || q1 > p.T || kv < 0 || kv > p.max_kv;
    if (bad) return CacheSeq{0, 0, 0};
    const int rows = (q1 - q0) * p.g;
    return CacheSeq{q0, rows > p.row_lo && rows <= p.row_hi ? q1 - q0 : 0, kv};
}

// Keys [lo, hi) that some row of the row tile may see, and the key tiles [f, f + n) they lie in.
struct CacheRange {
    int lo, hi, f, n;
};
template <int BN>
__device__ __forceinline__ CacheRange cache_range(const CacheFwdParams& p, const CacheSeq& s, int tile, int bm) {
    const int r0 = tile * bm, r1 = min(s.q_len * p.g, r0 + bm) - 1;
    const int diag = s.kv_len - s.q_len;
    CacheRange k;
    k.hi = p.causal ? max(0, min(s.kv_len, div_g(p, r1) + diag + 1)) : s.kv_len;
    k.lo = p.window >= 0 ? max(0, div_g(p, r0) + diag - p.window) : 0;
    k.f = k.lo / BN;
    k.n = k.hi > k.lo ? (k.hi - 1) / BN + 1 - k.f : 0;
    return k;
}

template <int BN>
__device__ __forceinline__ CacheRange cache_range(const CacheFwdParams& p, const CacheSeq& s, int tile) {
    return cache_range<BN>(p, s, tile, p.bm);
}

__device__ __forceinline__ int cache_tiles(const CacheFwdParams& p, const CacheSeq& s) {
    return int(uint32_t(s.q_len * p.g + p.bm - 1) / uint32_t(p.bm));
}

// Units of an item: its key tiles, and p.item_cost more that stand for its start and end, so
// that equal ranges of units take equal times.  (Unit counts fit 31 bits: cache.cu checks.)
template <int BN>
__device__ __forceinline__ int cache_units(const CacheFwdParams& p, const CacheSeq& s, int tile) {
    return max(1, cache_range<BN>(p, s, tile).n) + p.item_cost;
}

__device__ __forceinline__ int warp_scan(int v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    return v;
}

// Sum over the warp of values below 2^31 that lanes have added up mod 2^32 (w) and in their
// upper 16 bits (hi); -1 unless it is below 2^31 - 2^16.  One sequence's units fit (cache.cu
// checks), but offsets that go back and forth make many sequences of the same rows.
__device__ __forceinline__ int cache_sum(uint32_t w, int hi) {
    const int s = int(__reduce_add_sync(0xffffffffu, w));
    return __reduce_add_sync(0xffffffffu, hi) >= 0x7fff || s < 0 ? -1 : s;  // (hi: within 256 of the sum's)
}
__device__ __forceinline__ int cache_sum(int v) { return cache_sum(uint32_t(v), v >> 16); }

// Units of one key head of a lane's sequence, by the whole warp: a lane counts the tiles of
// its own short sequence, and the warp together those of a long one.
template <int BN>
__device__ __forceinline__ int cache_seq_units(const CacheFwdParams& p, const CacheSeq& s, int lane) {
    const int nt = cache_tiles(p, s);
    int u = 0;
    const bool heavy = nt > 32;
    if (!heavy)
        for (int t = 0; t < nt; ++t) u += cache_units<BN>(p, s, t);
    uint32_t todo = __ballot_sync(0xffffffffu, heavy);
    while (todo) {
        const int l = __ffs(todo) - 1;
        todo &= todo - 1;
        const CacheSeq h{0, __shfl_sync(0xffffffffu, s.q_len, l), __shfl_sync(0xffffffffu, s.kv_len, l)};
        const int hn = cache_tiles(p, h);
        int v = 0;
        for (int t = lane; t < hn; t += 32) v += cache_units<BN>(p, h, t);
        v = __reduce_add_sync(0xffffffffu, v);
        if (lane == l) u = v;
    }
    return u;
}

// The sequence at place b of an order (a lane number within each group of 32).
__device__ __forceinline__ int cache_ordered(const uint8_t* order, int b) { return order ? (b & ~31) + order[b] : b; }

// The sequence of a lane in group c (32 sequences, in the batch's order or a given one); the
// first CTA reports bad ones.
__device__ __forceinline__ CacheSeq cache_lane_seq(const CacheFwdParams& p, int c, int lane, bool report,
                                                   const uint8_t* order = nullptr) {
    const int b = 32 * c + lane;
    bool bad = false;
    CacheSeq s{0, 0, 0};
    if (b < p.B) s = cache_seq(p, cache_ordered(order, b), bad);
    if (bad && report) atomicOr(p.status, kStatusBounds);
    return s;
}

// Where a CTA's range of units starts, and how the ranges are cut.
struct CacheStart {
    int b, hk, tile, kt;
    int u, u_end;       // this CTA's units [u, u_end)
    int base, rem;      // units per CTA, the first `rem` CTAs one more
    CacheSeq s;         // sequence b
};

// The item of the `left`-th unit (one that they have) of the sequences that a warp's lanes hold
// (s: a lane's sequence 32 c + lane, one: its units per key head), into b, hk, tile and kt of `st`.
template <int BN>
__device__ __forceinline__ void cache_locate(const CacheFwdParams& p, int c, const CacheSeq& s, int one, int left, int lane,
                                             CacheStart& st) {
    const int inc = warp_scan(one * p.Hkv, lane);
    const int l = __ffs(__ballot_sync(0xffffffffu, inc > left)) - 1;
    left -= __shfl_sync(0xffffffffu, inc - one * p.Hkv, l);
    const int per = __shfl_sync(0xffffffffu, one, l);
    const CacheSeq q{__shfl_sync(0xffffffffu, s.q0, l), __shfl_sync(0xffffffffu, s.q_len, l),
                     __shfl_sync(0xffffffffu, s.kv_len, l)};
    st.s = q;
    st.b = 32 * c + l;
    st.hk = int(uint32_t(left) / uint32_t(per));
    left -= st.hk * per;
    const int nt = cache_tiles(p, q);
    st.tile = 0;
    st.kt = left;
    if (nt == 1) return;
    for (int t0 = 0; t0 < nt; t0 += 32) {
        const int n = t0 + lane < nt ? cache_units<BN>(p, q, t0 + lane) : 0;
        const int in = warp_scan(n, lane);
        const uint32_t m = __ballot_sync(0xffffffffu, in > left);
        if (m) {
            const int t = __ffs(m) - 1;
            st.tile = t0 + t;
            st.kt = left - __shfl_sync(0xffffffffu, in - n, t);
            break;
        }
        left -= __shfl_sync(0xffffffffu, in, 31);
    }
}

// total < 0: more units than can be counted, none is worked on.
__device__ __forceinline__ void cache_cut(const CacheFwdParams& p, int total, CacheStart& st) {
    if (total < 0) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
        total = 0;
    }
    const int want = int((uint32_t(total) + uint32_t(p.min_units) - 1u) / uint32_t(p.min_units));
    const int G = min(int(gridDim.x), max(want, 1)), cta = blockIdx.x;
    st = CacheStart{};
    if (cta < G && total > 0) {
        st.base = int(uint32_t(total) / uint32_t(G));
        st.rem = total - st.base * G;
        st.u = cta * st.base + min(cta, st.rem);
        st.u_end = st.u + st.base + (cta < st.rem ? 1 : 0);
    }
}

// This CTA's range, by every thread of the CTA; each warp gets it in registers.  sums: shared
// scratch of ceil(B / 32) values (unused up to 32 sequences, which every warp looks over
// itself); the caller synchronises before it is used for anything else.
template <int BN>
__device__ __forceinline__ CacheStart cache_start(const CacheFwdParams& p, int* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int groups = (p.B + 31) >> 5;
    CacheStart st;
    if (groups <= 1) {
        const CacheSeq s = cache_lane_seq(p, 0, lane, blockIdx.x == 0 && warp == 0);
        const int one = cache_seq_units<BN>(p, s, lane);
        cache_cut(p, cache_sum(one * p.Hkv), st);
        if (st.u < st.u_end) cache_locate<BN>(p, 0, s, one, st.u, lane, st);
        return st;
    }
    for (int c = warp; c < groups; c += warps) {
        const CacheSeq s = cache_lane_seq(p, c, lane, blockIdx.x == 0);
        const int v = cache_sum(cache_seq_units<BN>(p, s, lane) * p.Hkv);
        if (lane == 0) sums[c] = v < 0 ? INT_MAX : v;
    }
    __syncthreads();
    uint32_t total = 0;
    int hi = 0;
    for (int c = lane; c < groups; c += 32) {
        total += uint32_t(sums[c]);
        hi += sums[c] >> 16;
    }
    cache_cut(p, cache_sum(total, hi), st);
    if (st.u < st.u_end) {
        int left = st.u, c = 0;
        for (int c0 = 0; c0 < groups; c0 += 32) {
            const int v = c0 + lane < groups ? sums[c0 + lane] : 0;
            const int inc = warp_scan(v, lane);
            const uint32_t m = __ballot_sync(0xffffffffu, inc > left);
            if (m) {
                const int l = __ffs(m) - 1;
                c = c0 + l;
                left -= __shfl_sync(0xffffffffu, inc - v, l);
                break;
            }
            left -= __shfl_sync(0xffffffffu, inc, 31);
        }
        const CacheSeq s = cache_lane_seq(p, c, lane, false);
        cache_locate<BN>(p, c, s, cache_seq_units<BN>(p, s, lane), left, lane, st);
    }
    return st;
}

// A CTA's part of one item: key tiles [k0, k1) of its n (at least one), the item's units from
// number `first` of the batch on.
struct CacheSeg {
    int b, hk, tile;
    CacheSeq s;
    CacheRange r;
    int k0, k1, n;
    int first;
    __device__ bool whole() const { return k0 == 0 && k1 == n; }
};

// Walks a range of units, sequences in the batch's order or a given one (st.b then counts
// places in that order).  Every role of a CTA walks its own copy.
template <int BN>
struct CacheCursor {
    CacheStart st;
    CacheSeq s;
    int nt;
    const uint8_t* order;
    __device__ CacheCursor(const CacheFwdParams& p, const CacheStart& start, const uint8_t* ord = nullptr)
        : st(start), s(start.s), nt(cache_tiles(p, start.s)), order(ord) {}  // (nt = 0: an empty range)
    __device__ bool next(const CacheFwdParams& p, CacheSeg& g) {
        while (st.u < st.u_end) {
            while (nt <= 0) {
                if (nt == 0) ++st.b;
                if (st.b >= p.B) return false;
                bool bad;
                s = cache_seq(p, cache_ordered(order, st.b), bad);
                nt = cache_tiles(p, s);
            }
            g.b = cache_ordered(order, st.b);
            g.hk = st.hk;
            g.tile = st.tile;
            g.s = s;
            g.r = cache_range<BN>(p, s, st.tile);
            g.n = max(1, g.r.n);
            // the units before the first key tile are the item's cost
            const int v1 = min(g.n + p.item_cost, st.kt + (st.u_end - st.u));
            g.k0 = max(0, st.kt - p.item_cost);
            g.k1 = max(0, v1 - p.item_cost);
            g.first = st.u - st.kt;
            st.u += v1 - st.kt;
            st.kt = 0;
            if (++st.tile == nt) {
                st.tile = 0;
                if (++st.hk == p.Hkv) {
                    st.hk = 0;
                    nt = 0;
                }
            }
            if (g.k1 > g.k0) return true;
        }
        return false;
    }
};

// The CTA that holds unit u, and the first and last CTA with a part of an item.
__device__ __forceinline__ int cache_cta_of(const CacheStart& st, int u) {
    const int head = st.rem * (st.base + 1);
    return u < head ? int(uint32_t(u) / uint32_t(st.base + 1)) : st.rem + int(uint32_t(u - head) / uint32_t(st.base));
}
__device__ __forceinline__ int cache_first_cta(const CacheFwdParams& p, const CacheStart& st, const CacheSeg& g) {
    return cache_cta_of(st, g.first + p.item_cost);
}
__device__ __forceinline__ int cache_last_cta(const CacheFwdParams& p, const CacheStart& st, const CacheSeg& g) {
    return cache_cta_of(st, g.first + p.item_cost + g.n - 1);
}

// ------------------------------------------------------------------ work drawn in order
//
// The chunk kernel's CTAs draw their work one piece at a time from a counter, so that the
// pieces in flight are neighbours (row tiles of one key head, reading the same keys out of
// L2) and no CTA is left with more than its share.  The pieces are whole items, in order,
// while much work remains, and near the end blocks of `blk` units, which may cut items; the
// cut items' parts, numbered by block, are merged by a second kernel.  Which units form a piece
// depends on the lengths alone, so results do not depend on who draws what.
// The sequences of a group of 32 are taken longest first, so that what is drawn late is short.
struct CacheGroups {      // shared memory
    uint8_t order[kCacheMaxB];   // sequences in the order they are worked on, within their group
    int units[kCacheMaxGroups];  // units before the group of 32 sequences
    int items[kCacheMaxGroups];  // items before it
    int total, cut;        // units; the first `whole` items are units [0, cut)
    int whole, blk, pieces;
    int longest;           // units of the longest item
};

// The group of unit u (or item u): the last one starting at or before it.  (A group without
// any shares its start with the next one that has some, which comes later.)
__device__ __forceinline__ int cache_find_group(const int* before, int groups, int u, int lane) {
    int c = 0;
    for (int c0 = 0; c0 < groups; c0 += 32) {
        const uint32_t m = __ballot_sync(0xffffffffu, c0 + lane < groups && before[c0 + lane] <= u);
        if (!m) break;
        c = c0 + 31 - __clz(int(m));
    }
    return c;
}

// Unit u of the batch, by a whole warp: its item and unit within it.
template <int BN>
__device__ __forceinline__ CacheStart cache_find_unit(const CacheFwdParams& p, const CacheGroups& G, int groups, int u,
                                                      int lane) {
    CacheStart st{};
    st.u = st.u_end = u;
    const int c = cache_find_group(G.units, groups, u, lane);
    const CacheSeq s = cache_lane_seq(p, c, lane, false, G.order);
    cache_locate<BN>(p, c, s, cache_seq_units<BN>(p, s, lane), u - G.units[c], lane, st);
    return st;
}

// Item i of the batch, by a whole warp.
__device__ __forceinline__ CacheStart cache_find_item(const CacheFwdParams& p, const CacheGroups& G, int groups, int i,
                                                      int lane) {
    CacheStart st{};
    const int c = cache_find_group(G.items, groups, i, lane);
    const CacheSeq s = cache_lane_seq(p, c, lane, false, G.order);
    const int tiles = cache_tiles(p, s);
    const int inc = warp_scan(tiles * p.Hkv, lane);
    int left = i - G.items[c];
    const int l = __ffs(__ballot_sync(0xffffffffu, inc > left)) - 1;
    left -= __shfl_sync(0xffffffffu, inc - tiles * p.Hkv, l);
    const int nt = __shfl_sync(0xffffffffu, tiles, l);
    st.s = CacheSeq{__shfl_sync(0xffffffffu, s.q0, l), __shfl_sync(0xffffffffu, s.q_len, l),
                    __shfl_sync(0xffffffffu, s.kv_len, l)};
    st.b = 32 * c + l;
    st.hk = int(uint32_t(left) / uint32_t(nt));
    st.tile = left - st.hk * nt;
    return st;
}

// The batch's pieces, by every thread of the CTA.  G.pieces is 0 for a batch without rows.
template <int BN>
__device__ __forceinline__ void cache_pieces(const CacheFwdParams& p, CacheGroups* G) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int groups = (p.B + 31) >> 5;
    if (threadIdx.x == 0) G->longest = 1;
    __syncthreads();
    for (int c = warp; c < groups; c += warps) {
        const CacheSeq s = cache_lane_seq(p, c, lane, blockIdx.x == 0);
        const int tiles = cache_tiles(p, s);
        int rank = 0;
#pragma unroll 8
        for (int l = 0; l < 32; ++l) {
            const int kv = __shfl_sync(0xffffffffu, s.kv_len, l);
            rank += kv > s.kv_len || (kv == s.kv_len && l < lane);
        }
        // (lanes past the last sequence hold length 0 and come after every other's tie)
        if (32 * c + lane < p.B) G->order[32 * c + rank] = uint8_t(lane);
        // a sequence's last item sees the most keys (but for a window's odd tile)
        const int n = __reduce_max_sync(0xffffffffu, tiles > 0 ? cache_units<BN>(p, s, tiles - 1) : 0);
        const int u = cache_sum(cache_seq_units<BN>(p, s, lane) * p.Hkv);
        const int t = __reduce_add_sync(0xffffffffu, tiles);
        if (lane == 0) {
            G->units[c] = u < 0 ? INT_MAX : u;
            G->items[c] = t * p.Hkv;
            atomicMax(&G->longest, n);
        }
    }
    __syncthreads();
    if (warp == 0) {
        int u = 0, items = 0, hi = 0;
        for (int c0 = 0; c0 < groups; c0 += 32) {  // sums to exclusive prefixes
            const bool in = c0 + lane < groups;
            const int v = in ? G->units[c0 + lane] : 0, w = in ? G->items[c0 + lane] : 0;
            const int vi = warp_scan(v, lane), wi = warp_scan(w, lane);
            if (in) {
                G->units[c0 + lane] = u + vi - v;
                G->items[c0 + lane] = items + wi - w;
            }
            u += __shfl_sync(0xffffffffu, vi, 31);
            items += __shfl_sync(0xffffffffu, wi, 31);
            hi += __reduce_add_sync(0xffffffffu, v >> 16);
        }
        __syncwarp();
        if (hi >= 0x7fff || u < 0) {  // more units than can be counted: none is worked on
            if (blockIdx.x == 0 && lane == 0) atomicOr(p.status, kStatusBounds);
            u = items = 0;
        }
        const int grid = gridDim.x, longest = G->longest;
        // The last part, cut in blocks, covers the spread with which the CTAs come out of the
        // whole items: a quarter of an item each (half: more parts to merge, 8 prompts 726 us
        // against 709; an eighth: 5 equal prompts 648 us against 575).  Never none, so that the
        // unit the blocks start at exists: without one the search below would look for unit `u`,
        // past the last, and find no lane that holds it.  Where the longest item is over half a
        // CTA's share, everything is cut.
        const int mean = int(uint32_t(u) / uint32_t(max(items, 1)));
        const int rest = (long long)(longest) * 2 * grid > u ? u : min(u, grid * max(1, (mean + 1) / 4));
        int cut = 0, whole = 0;
        if (u > rest) {
            const CacheStart st = cache_find_unit<BN>(p, *G, groups, u - rest, lane);
            cut = u - rest - st.kt;
            const int c = st.b >> 5;
            const int tiles = cache_tiles(p, cache_lane_seq(p, c, lane, false, G->order));
            const int before = __reduce_add_sync(0xffffffffu, 32 * c + lane < st.b ? tiles : 0);
            whole = G->items[c] + before * p.Hkv + st.hk * __shfl_sync(0xffffffffu, tiles, st.b & 31) + st.tile;
        }
        const int left = u - cut;
        // few units: one block a CTA, of at least min_units (or an item); else up to
        // kBlocksPerCta of at least eight units
        const int per = max(1, min(kBlocksPerCta, left / (8 * grid))) * grid;
        const int blk = max((left + per - 1) / per, min(p.min_units, longest));
        if (lane == 0) {
            G->total = u;
            G->cut = cut;
            G->whole = whole;
            G->blk = blk;
            G->pieces = whole + (left + blk - 1) / blk;
        }
    }
    __syncthreads();
}

// Partial results of split items: slot 0 of a CTA for the item that started in an earlier
// CTA, slot 1 for one that goes on in the next.  An item split over CTAs first..last has its
// first part in slot 1 of `first`, the others in slot 0.
__device__ __forceinline__ int cache_slot(int cta, int first_cta) { return 2 * cta + (cta == first_cta ? 1 : 0); }

// Programmatic launch: let the next kernel of the stream start (when it was launched so), and
// wait for the previous one to have finished.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
// One box of the pages: elements x .., slots y .., head z, page w.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// Lets `kernel` use `bytes` of shared memory per CTA, once per device (done: a bit for each).
template <typename Kernel>
cudaError_t allow_smem(Kernel* kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_acquire) >> dev) & 1u)) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    return e;
}

// fp32, items of 128 packed rows: tensor-core products of operands in three bf16 parts each.
cudaError_t launch_cache_split(int D, const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, int num_sms,
                               cudaStream_t st);
size_t cache_split_part_bytes(int D, int num_sms);
// fp32, items of p.bm = 4 or 16 packed rows; early: as launch_cache_decode's.
cudaError_t launch_cache_simt(int D, const CacheFwdParams& p, bool early, int num_sms, cudaStream_t st);
size_t cache_simt_part_bytes(int D, int num_sms);
// bf16, row tiles of 16 packed rows: bound by the stream of K and V.
// early: start while the chunk kernel before it in the stream still runs (they share no
// memory that either writes), and end after it.
cudaError_t launch_cache_decode(int D, const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, bool early,
                                int num_sms, cudaStream_t st);
size_t cache_decode_part_bytes(int D, int num_sms);
// bf16, items of 256 packed rows: bound by the tensor cores and the exponentials.
// mq: the queries as (D, head, token), boxes of 128 bytes x g heads x tile_tokens.
cudaError_t launch_cache_chunk(int D, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                               const CacheFwdParams& p, int num_sms, cudaStream_t st);
size_t cache_chunk_part_bytes(int D, int num_sms);
// Parts of cut items as the merge kernel reads them: O four columns of kMergeRows rows at a
// time, then the rows' m and l.
constexpr int kMergeRows = 256;
__host__ __device__ constexpr int cache_merge_part(int D) { return kMergeRows * (D + 2); }  // floats
// blocks: how many the items may be cut between (num_sms of the split kernel, kBlocksPerCta times
// as many of the chunk kernel).
cudaError_t launch_cache_merge(int D, const CacheFwdParams& p, int blocks, int num_sms, cudaStream_t st);

struct CacheAppendParams {
    const int32_t* q_off;
    const int32_t* kv_lens;
    const int32_t* table;
    int B, max_pages, T, max_kv;
    int H, Hkv, D;            // H: rotated query heads (0: none)
    int page_log2, n_pages;
    const void* K;
    const void* V;
    const void* Q;
    void* Q_out;
    int64_t k_stride, v_stride, q_stride, qo_stride;
    void* Kc;
    void* Vc;
    int64_t ks[3], vs[3];
    const float* rot;
    int rot_dim, rot_len, pairs;
    int* status;
};
cudaError_t launch_cache_append(int dtype, const CacheAppendParams& p, cudaStream_t st);

}  // namespace jfa
