// Paged-cache attention: what the kernels share.
//
// The new tokens of sequence b and the g = H / Hkv query heads of one key head hk form
// R_b = q_len_b * g packed rows (row r: token r / g, head hk * g + r % g), so grouped heads
// share every key and value read.  Rows are cut into tiles of BM, keys into tiles of BN; an
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

namespace jfa {

struct CacheFwdParams {
    const int32_t* q_off;    // [B+1]
    const int32_t* kv_lens;  // [B]
    const int32_t* table;    // [B, max_pages]
    int B, max_pages, T, max_kv;
    int H, Hkv, g;
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
    uint32_t* counters;      // workspace: arrivals per split item (zero between calls)
    float* part;             // workspace: partial results, two slots per CTA
    int* status;
    int min_units;           // units a CTA takes at least
    int row_lo, row_hi;      // sequences this launch works on: row_lo < q_len * g <= row_hi
};

struct CacheSeq {
    int q0, q_len, kv_len;
};

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
template <int BM, int BN>
__device__ __forceinline__ CacheRange cache_range(const CacheFwdParams& p, const CacheSeq& s, int tile) {
    const int r0 = tile * BM, r1 = min(s.q_len * p.g, r0 + BM) - 1;
    const int diag = s.kv_len - s.q_len;
    CacheRange k;
    k.hi = p.causal ? max(0, min(s.kv_len, r1 / p.g + diag + 1)) : s.kv_len;
    k.lo = p.window >= 0 ? max(0, r0 / p.g + diag - p.window) : 0;
    k.f = k.lo / BN;
    k.n = k.hi > k.lo ? (k.hi - 1) / BN + 1 - k.f : 0;
    return k;
}

template <int BM>
__device__ __forceinline__ int cache_tiles(const CacheFwdParams& p, const CacheSeq& s) {
    return (s.q_len * p.g + BM - 1) / BM;
}

__device__ __forceinline__ long long warp_sum_ll(long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ long long warp_scan_ll(long long v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    return v;
}

// Units of one key head of sequence 32 c + lane, by the whole warp: a lane counts the tiles
// of its own short sequence, and the warp together those of a long one.
template <int BM, int BN>
__device__ long long cache_seq_units(const CacheFwdParams& p, int c, int lane, bool report) {
    const int b = 32 * c + lane;
    CacheSeq s{0, 0, 0};
    bool bad = false;
    if (b < p.B) s = cache_seq(p, b, bad);
    if (bad && report) atomicOr(p.status, kStatusBounds);
    const int nt = cache_tiles<BM>(p, s);
    long long u = 0;
    const bool heavy = nt > 4;
    if (!heavy)
        for (int t = 0; t < nt; ++t) u += max(1, cache_range<BM, BN>(p, s, t).n);
    uint32_t todo = __ballot_sync(0xffffffffu, heavy);
    while (todo) {
        const int l = __ffs(todo) - 1;
        todo &= todo - 1;
        const CacheSeq h{0, __shfl_sync(0xffffffffu, s.q_len, l), __shfl_sync(0xffffffffu, s.kv_len, l)};
        const int hn = cache_tiles<BM>(p, h);
        long long v = 0;
        for (int t = lane; t < hn; t += 32) v += max(1, cache_range<BM, BN>(p, h, t).n);
        v = warp_sum_ll(v);
        if (lane == l) u = v;
    }
    return u;
}

// Where a CTA's range of units starts, and how the ranges are cut.
struct CacheStart {
    int b, hk, tile, kt;
    long long u, u_end;       // this CTA's units [u, u_end)
    long long base;           // units per CTA, the first `rem` CTAs one more
    int rem;
};

// By every thread of the CTA (blockDim.x a multiple of 32).  sums: shared scratch of
// ceil(B / 32) values.
template <int BM, int BN>
__device__ void cache_start(const CacheFwdParams& p, CacheStart* out, long long* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int chunks = (p.B + 31) >> 5;
    for (int c = warp; c < chunks; c += warps) {
        const long long v = warp_sum_ll(cache_seq_units<BM, BN>(p, c, lane, blockIdx.x == 0));
        if (lane == 0) sums[c] = v * p.Hkv;
    }
    __syncthreads();
    if (warp == 0) {
        long long total = 0;
        for (int c = lane; c < chunks; c += 32) total += sums[c];
        total = warp_sum_ll(total);
        CacheStart st{0, 0, 0, 0, 0, 0, 0, 0};
        const long long want = (total + p.min_units - 1) / p.min_units;
        const int G = int(min((long long)(gridDim.x), max(want, 1LL)));
        const int cta = blockIdx.x;
        if (cta < G && total > 0) {
            st.base = total / G;
            st.rem = int(total - st.base * G);
            st.u = cta * st.base + min(cta, st.rem);
            st.u_end = st.u + st.base + (cta < st.rem ? 1 : 0);
        }
        if (st.u < st.u_end) {
            long long left = st.u;  // units before the range, from the search's position on
            int c = 0;
            for (int c0 = 0; c0 < chunks; c0 += 32) {
                const long long v = c0 + lane < chunks ? sums[c0 + lane] : 0;
                const long long inc = warp_scan_ll(v, lane);
                const uint32_t m = __ballot_sync(0xffffffffu, inc > left);
                if (m) {
                    const int l = __ffs(m) - 1;
                    c = c0 + l;
                    left -= __shfl_sync(0xffffffffu, inc - v, l);
                    break;
                }
                left -= __shfl_sync(0xffffffffu, inc, 31);
            }
            const long long one = cache_seq_units<BM, BN>(p, c, lane, false);
            const long long inc = warp_scan_ll(one * p.Hkv, lane);
            const int l = __ffs(__ballot_sync(0xffffffffu, inc > left)) - 1;
            left -= __shfl_sync(0xffffffffu, inc - one * p.Hkv, l);
            st.b = 32 * c + l;
            const long long per = __shfl_sync(0xffffffffu, one, l);
            st.hk = int(left / per);
            left -= st.hk * per;
            bool bad;
            const CacheSeq s = cache_seq(p, st.b, bad);
            const int nt = cache_tiles<BM>(p, s);
            for (int t0 = 0; t0 < nt; t0 += 32) {
                const long long n = t0 + lane < nt ? max(1, cache_range<BM, BN>(p, s, t0 + lane).n) : 0;
                const long long in = warp_scan_ll(n, lane);
                const uint32_t m = __ballot_sync(0xffffffffu, in > left);
                if (m) {
                    const int t = __ffs(m) - 1;
                    st.tile = t0 + t;
                    st.kt = int(left - __shfl_sync(0xffffffffu, in - n, t));
                    break;
                }
                left -= __shfl_sync(0xffffffffu, in, 31);
            }
        }
        if (lane == 0) *out = st;
    }
    __syncthreads();
}

// A CTA's part of one item: units [k0, k1) of its `units`, from unit number `first` of the batch.
struct CacheSeg {
    int b, hk, tile;
    CacheSeq s;
    CacheRange r;
    int k0, k1, units;
    long long first;
    __device__ bool whole() const { return k0 == 0 && k1 == units; }
};

// Walks a CTA's range.  Every role of a CTA walks its own copy.
template <int BM, int BN>
struct CacheCursor {
    CacheStart st;
    CacheSeq s;
    int nt;
    __device__ explicit CacheCursor(const CacheStart& start) : st(start), s{0, 0, 0}, nt(-1) {}
    __device__ bool next(const CacheFwdParams& p, CacheSeg& g) {
        if (st.u >= st.u_end) return false;
        while (nt <= 0) {
            if (nt == 0) ++st.b;
            if (st.b >= p.B) return false;
            bool bad;
            s = cache_seq(p, st.b, bad);
            nt = cache_tiles<BM>(p, s);
        }
        g.b = st.b;
        g.hk = st.hk;
        g.tile = st.tile;
        g.s = s;
        g.r = cache_range<BM, BN>(p, s, st.tile);
        g.units = max(1, g.r.n);
        g.k0 = st.kt;
        g.k1 = int(min((long long)(g.units), st.kt + (st.u_end - st.u)));
        g.first = st.u - st.kt;
        st.u += g.k1 - g.k0;
        st.kt = 0;
        if (++st.tile == nt) {
            st.tile = 0;
            if (++st.hk == p.Hkv) {
                st.hk = 0;
                nt = 0;
            }
        }
        return true;
    }
};

// The CTA that holds unit u.
__device__ __forceinline__ int cache_cta_of(const CacheStart& st, long long u) {
    const long long head = st.rem * (st.base + 1);
    return u < head ? int(u / (st.base + 1)) : st.rem + int((u - head) / st.base);
}

// Partial results of split items: slot 0 of a CTA for the item that started in an earlier
// CTA, slot 1 for one that goes on in the next.  An item split over CTAs first..last has its
// first part in slot 1 of `first`, the others in slot 0.
__device__ __forceinline__ int cache_slot(int cta, int first_cta) { return 2 * cta + (cta == first_cta ? 1 : 0); }

// One box of the pages: elements x .., slots y .., head z, page w.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// fp32, row tiles of 128 (chunk) or 16 packed rows.
cudaError_t launch_cache_simt(int D, bool chunk, const CacheFwdParams& p, int num_sms, cudaStream_t st);
size_t cache_simt_part_bytes(int D, int num_sms);
// bf16, row tiles of 16 packed rows: bound by the stream of K and V.
cudaError_t launch_cache_decode(int D, const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, int num_sms,
                                cudaStream_t st);
size_t cache_decode_part_bytes(int D, int num_sms);
// bf16, items of 256 packed rows: bound by the tensor cores and the exponentials.
cudaError_t launch_cache_chunk(int D, const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, int num_sms,
                               cudaStream_t st);
size_t cache_chunk_part_bytes(int D, int num_sms);

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
