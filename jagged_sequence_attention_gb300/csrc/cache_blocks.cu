// Attention over selected blocks of a paged cache: the blocks' bounds, the selection, and the
// attention call.  A block is a page.  Semantics are documented in include/jfa.h.
//
// The score of a block for a token and key head is the sum over the group's heads h of an upper
// bound of <q_h, k> over the block's keys,
//   sum_h sum_d max(q_hd lo_d, q_hd hi_d) = <u, hi> + <w, lo>,  u = sum_h max(q_h, 0), w = sum_h min(q_h, 0),
// with lo and hi the block's least and largest elements, so the group costs what one head does.
//
// The selection is that of exact arithmetic.  Scores are taken in fp32: u and w are sums of g values of
// one sign, and a dot product adds n products one after the other (a lane's D / 4, joined in 3 steps; of
// a tile, see there), so a score is off by less than
//   slack = (g + n + 4) 2^-24 max|lo, hi| sum_d (u_d - w_d),
// and 2^-116 times as much as these for what falls below fp32's (or bf16's) numbers.
// With t the k-th largest fp32 score, the exact k-th largest lies within slack of t: a block above
// t + 2 slack is in, one below t - 2 slack is out, and those between, mostly one, are scored
// again in 64 bits and taken in order, of equal ones the lower index.
#include <cuda_bf16.h>

#include "cache_handle.h"
#include "cache_rows.cuh"
#include "quant.cuh"

using namespace jfa;

namespace jfa {

cudaError_t launch_cache_decode4(int D, const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, bool early,
                                 int num_sms, cudaStream_t st);

namespace {

constexpr int kChunk = 64;          // blocks that a CTA scores
constexpr int kSumThreads = 512, kScoreThreads = 256, kTileThreads = 256;
constexpr int kTileTokens = 32;     // tokens that a CTA scores, where a sequence has many
constexpr int kSelWarps = 32;       // warps that choose for one item, where more than 1024 blocks may compete

struct BlockParams {
    CacheAppendParams a;            // the batch and the cache
    const uint8_t* k_scales;
    int64_t kss[2];
    __nv_bfloat16* bounds;          // [n_pages, Hkv, 2, D]: least, largest
    const __nv_bfloat16* Q;
    int64_t q_stride;
    int g, n_blocks, n_first, n_last;
    int32_t* blocks;                // [T, Hkv, n_blocks]
    float* scores;                  // [T, Hkv, max_pages]
    float* slack;                   // [T, Hkv, chunks]
    int chunks;
    int tile;                       // summarize: tokens that a CTA looks over; tiles' scores: chunks of a CTA
};

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t c;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
    return c;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t c;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
    return c;
}

// The bounds of every page that got new tokens, over all its positions below kv_len, by the CTA that
// has the page's first new token among its `tile` tokens.  A thread takes eight elements of a head
// of every so many-th slot (as many threads a vector as the CTA has room for), so that a page is a
// few loads deep.
template <bool FOUR>
__global__ void __launch_bounds__(kSumThreads) jfa_cache_summarize_kernel(const BlockParams z) {
    const CacheAppendParams& p = z.a;
    __shared__ uint4 red[2][kSumThreads];
    const int lane = threadIdx.x & 31, size = 1 << p.page_log2;
    const int t0 = blockIdx.x * z.tile, t1 = min(t0 + z.tile, p.T);
    const int vl = p.D == 128 ? 4 : 3, vecs = p.Hkv << vl, share = max(1, kSumThreads / vecs);
    int b = find_sequence(p.q_off, p.B, t0, lane);
    if (b < 0) b = 0;  // (tokens before the first sequence)
    for (; b < p.B; ++b) {
        const int q0 = p.q_off[b], q1 = p.q_off[b + 1], kv = p.kv_lens[b];
        if (q0 >= t1) break;
        const int ta = max(q0, t0), tb = min(q1, t1);  // its tokens here
        if (ta >= tb) continue;
        if (q0 < 0 || q1 > p.T || kv < q1 - q0 || kv > p.max_kv) {
            if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
            continue;
        }
        // its pages that have their first new token here
        const int pa = kv - q1 + ta, pb = kv - q1 + tb - 1;
        int k = pa >> p.page_log2;
        if (ta > q0 && (pa & (size - 1))) ++k;
        for (; k <= pb >> p.page_log2; ++k) {
            const int page = p.table[size_t(b) * size_t(p.max_pages) + size_t(k)];
            if (page < 0 || page >= p.n_pages) {
                if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
                continue;
            }
            const int n = min(size, kv - (k << p.page_log2));
            for (int v0 = 0; v0 < vecs; v0 += kSumThreads) {
                const int vn = min(vecs - v0, kSumThreads), who = threadIdx.x / vn, v = v0 + threadIdx.x % vn, h = v >> vl, u = v & ((1 << vl) - 1);
                const bool in = who < share;
                uint4 lo = make_uint4(0x7f807f80u, 0x7f807f80u, 0x7f807f80u, 0x7f807f80u), hi = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
                auto take = [&](const uint4 l, const uint4 x) {
                    lo = make_uint4(min_bf16x2(lo.x, l.x), min_bf16x2(lo.y, l.y), min_bf16x2(lo.z, l.z), min_bf16x2(lo.w, l.w));
                    hi = make_uint4(max_bf16x2(hi.x, x.x), max_bf16x2(hi.y, x.y), max_bf16x2(hi.z, x.z), max_bf16x2(hi.w, x.w));
                };
                if constexpr (FOUR) {
                    const uint8_t* codes = static_cast<const uint8_t*>(p.Kc) + page * p.ks[0] + h * p.ks[2] + 4 * u;
                    const uint8_t* scales = z.k_scales + page * z.kss[0] + h * z.kss[1] + (u >> 1);
#pragma unroll 8
                    for (int j = in ? who : n; j < n; j += share) {
                        const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + j * p.ks[1]);
                        const float s = f16_to_float(e4m3_to_f16(scales[j << (vl - 1)])).x;
                        uint32_t e[4], o[4];
                        e2m1_to_f16(w, e);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 x = f16_to_float(e[i]);
                            o[i] = pack_bf16x2(x.x * s, x.y * s);
                        }
                        const uint4 x = make_uint4(o[0], o[1], o[2], o[3]);
                        take(x, x);
                    }
                } else {
                    const __nv_bfloat16* key = static_cast<const __nv_bfloat16*>(p.Kc) + page * p.ks[0] + h * p.ks[2] + 8 * u;
#pragma unroll 8
                    for (int j = in ? who : n; j < n; j += share) {
                        const uint4 x = *reinterpret_cast<const uint4*>(key + j * p.ks[1]);
                        take(x, x);
                    }
                }
                red[0][threadIdx.x] = lo;
                red[1][threadIdx.x] = hi;
                __syncthreads();
                if (threadIdx.x < vn) {
                    for (int i = 1; i < share; ++i) take(red[0][threadIdx.x + i * vn], red[1][threadIdx.x + i * vn]);
                    __nv_bfloat16* dst = z.bounds + (size_t(page) * p.Hkv + h) * 2 * p.D + 8 * u;
                    *reinterpret_cast<uint4*>(dst) = lo;
                    *reinterpret_cast<uint4*>(dst + p.D) = hi;
                }
                __syncthreads();
            }
        }
    }
}

// A token of a selection: its sequence and own block, or b < 0.  A row before its sequence's first
// position sees nothing (own = -1).
struct Chooser {
    int b, own;
};
__device__ __forceinline__ Chooser chooser(const CacheAppendParams& p, int t, int lane, bool report = false) {
    Chooser c{find_sequence(p.q_off, p.B, t, lane), -1};
    if (c.b >= p.B) c.b = -1;
    if (c.b < 0) return c;
    const int q0 = p.q_off[c.b], q1 = p.q_off[c.b + 1], kv = p.kv_lens[c.b];
    if (q0 < 0 || q1 > p.T || t < q0 || t >= q1 || kv < 0 || kv > p.max_kv) {
        if (report) atomicOr(p.status, kStatusBounds);
        c.b = -1;
        return c;
    }
    const int pos = kv - q1 + t;
    if (pos >= 0) c.own = pos >> p.page_log2;
    return c;
}

// u and w of a token and key head into sums [2 D] (lo's factors w, then hi's u), by `threads` threads.
template <typename F>
__device__ __forceinline__ void query_sums(const BlockParams& z, int t, int hk, F* sums, int thread, int threads) {
    const int D = z.a.D;
    for (int d = thread; d < D; d += threads) {
        F u = 0, w = 0;
        const __nv_bfloat16* q = z.Q + t * z.q_stride + hk * z.g * D + d;
        for (int h = 0; h < z.g; ++h) {
            const F x = F(__bfloat162float(q[h * D]));
            u += x > F(0) ? x : F(0);
            w += x < F(0) ? x : F(0);
        }
        sums[d] = w;
        sums[D + d] = u;
    }
}

// What an fp32 score may be off by (infinite where it may be no number at all): m the largest magnitude
// among the bounds, norm the sums' norm (which is itself a sum of 2 D values, hence the 1.01).  A product or sum
// may leave fp32's range, and so may a sum of queries by itself: from 2^128 - 2^119 on its first bf16 part is
// infinite, whatever the bounds.  An operand
// below 2^-126 may count as 0, and a product or sum may lose 2^-126: 2 D and a few times that is below 2^-116.
__device__ __forceinline__ float slack_of(const BlockParams& z, int steps, float m, float norm) {
    if (!(m * norm < 3e38f && norm < 3e38f)) return INFINITY;
    if (m == 0.f || norm == 0.f) return 0.f;   // all scores are 0
    return fmaf(float(z.g + steps) * (1.01f * 0x1p-24f) * m, norm, 0x1p-116f * (m + norm) + 0x1p-116f);
}

// Page of block k of sequence b, or -1.
__device__ __forceinline__ int block_page(const CacheAppendParams& p, int b, int k) {
    const int page = p.table[size_t(b) * size_t(p.max_pages) + size_t(k)];
    return page >= 0 && page < p.n_pages ? page : -1;
}

// Scores of kChunk blocks for one token and key head: eight lanes a block.  Bound by the latency of
// the chain sequence -> page -> bounds, with the queries' sums beside it, and for many blocks by the
// bounds' bytes, 4 D of them a block, all of a CTA's in flight at once.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) jfa_cache_score_kernel(const BlockParams z) {
    const CacheAppendParams& p = z.a;
    constexpr int kLanes = 8, kAt = kScoreThreads / kLanes, kTimes = kChunk / kAt, NV = D / 32;  // vectors of a lane: 2 D / 64
    const int t = blockIdx.x, hk = blockIdx.z, lane = threadIdx.x & 31;
    launch_dependents();  // (the choice waits for this kernel to end)
    const Chooser c = chooser(p, t, lane);
    const int first = z.n_first, end = c.own + 1 - z.n_last, k0 = blockIdx.y * kChunk;  // the blocks that compete
    if (c.b < 0 || c.own + 1 <= z.n_blocks || k0 >= end) return;
    __shared__ __align__(16) float sums[2 * D];
    __shared__ float red[kScoreThreads / 32];
    const int part = threadIdx.x % kLanes;
    uint4 x[kTimes][NV];
    bool in[kTimes];
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
        const int k = k0 + threadIdx.x / kLanes + kAt * i;
        in[i] = k >= first && k < end;
        const int page = in[i] ? block_page(p, c.b, k) : -1;
        if (in[i] && page < 0) atomicOr(p.status, kStatusBounds);
        const uint4* src = reinterpret_cast<const uint4*>(z.bounds + (size_t(max(page, 0)) * p.Hkv + hk) * 2 * D) + part;
#pragma unroll
        for (int v = 0; v < NV; ++v) x[i][v] = page >= 0 ? src[kLanes * v] : make_uint4(0u, 0u, 0u, 0u);
    }
    query_sums<float>(z, t, hk, sums, threadIdx.x, kScoreThreads);
    __syncthreads();
    float f[8 * NV], norm = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[8 * v + j] = sums[8 * (kLanes * v + part) + j];
            norm += fabsf(f[8 * v + j]);
        }
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) norm += __shfl_xor_sync(0xffffffffu, norm, d);
    uint32_t top = 0u;  // the largest magnitudes
    float* out = z.scores + (size_t(t) * p.Hkv + hk) * size_t(p.max_pages);
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const uint32_t r[4] = {x[i][v].x, x[i][v].y, x[i][v].z, x[i][v].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                top = max_bf16x2(top, r[j] & 0x7fff7fffu);
                s = fmaf(__uint_as_float(r[j] << 16), f[8 * v + 2 * j], s);
                s = fmaf(__uint_as_float(r[j] & 0xffff0000u), f[8 * v + 2 * j + 1], s);
            }
        }
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (in[i] && part == 0) out[k0 + threadIdx.x / kLanes + kAt * i] = s;
    }
    float m = fmaxf(__uint_as_float(top << 16), __uint_as_float(top & 0xffff0000u));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kScoreThreads / 32; ++w) m = fmaxf(m, red[w]);
        z.slack[(size_t(t) * p.Hkv + hk) * size_t(z.chunks) + blockIdx.y] = slack_of(z, 8 * NV + 4, m, norm);
    }
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const __nv_bfloat16* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p))
                 : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Scores for kTileTokens tokens and one key head, kChunk blocks at a time: a matrix product on the tensor
// cores, the sums as three bf16 parts each.  16 of the 2 D products are added at a time, the small
// parts' first, by instructions that add to no less than fp32's precision, and the 16s' sums in
// fp32: in all within 35 + D / 8 + 1 steps of 2^-24 of the products' magnitudes.  A warp has 16 tokens by 16 blocks.
// Bound by the chain page table -> bounds -> products of each chunk, the next one's loads under way
// meanwhile; chunks are dealt to as many CTAs as there is room for.  The product on the CUDA cores in fp32,
// a CTA a chunk with the sums anew, took 41 us of 82 for four prompts of 100-500 tokens over up to 20k
// keys; this one about 18 of 58.  The tile's sequences come one after the other: it is taken where they are long.
template <int D>
__global__ void __launch_bounds__(kTileThreads, 2) jfa_cache_score_tile_kernel(const BlockParams z) {
    const CacheAppendParams& p = z.a;
    constexpr int kRow = 2 * D, kPitch = kRow + 8;  // (rows end 16 bytes apart in the banks)
    constexpr int kVecs = kRow / 8, kLoads = kChunk * kVecs / kTileThreads;
    extern __shared__ __align__(16) uint8_t tile_smem[];
    __nv_bfloat16* sums = reinterpret_cast<__nv_bfloat16*>(tile_smem);  // [3][kTileTokens][kPitch]
    __nv_bfloat16* bounds = sums + 3 * kTileTokens * kPitch;            // [kChunk][kPitch]
    __shared__ float norms[kTileTokens];
    __shared__ uint32_t top[2];  // this chunk's largest magnitude, and the next one's
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, hk = blockIdx.z;
    const int t0 = blockIdx.x * kTileTokens, t1 = min(t0 + kTileTokens, p.T);
    const int m0 = 16 * (warp & 1), n0 = 16 * (warp >> 1);  // this warp's tokens and blocks
    launch_dependents();  // (the choice waits for this kernel to end)
    int b = find_sequence(p.q_off, p.B, t0, lane);
    if (b < 0) b = 0;
    bool have_sums = false;
    uint32_t odd = 0u;
    for (; b < p.B; ++b) {
        const int q0 = p.q_off[b], q1 = p.q_off[b + 1], kv = p.kv_lens[b];
        if (q0 >= t1) break;
        const int ta = max(q0, t0), tb = min(q1, t1);
        if (ta >= tb) continue;
        if (q0 < 0 || q1 > p.T || kv < 0 || kv > p.max_kv) {
            if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
            continue;
        }
        const int last = kv - q1 + tb - 1;  // the last token's position
        const int most = last >= 0 ? (last >> p.page_log2) + 1 : 0, end = most - z.n_last;
        if (most <= z.n_blocks) continue;
        int ch = max(int(blockIdx.y) * z.tile, z.n_first / kChunk);
        const int ch_end = min((int(blockIdx.y) + 1) * z.tile, (end + kChunk - 1) / kChunk);
        if (ch >= ch_end) continue;
        uint4 x[kLoads];
        auto load = [&](int chunk) {
            int page[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int k = chunk * kChunk + (threadIdx.x + kTileThreads * i) / kVecs;
                page[i] = -1;
                if (k >= z.n_first && k < end) {
                    page[i] = block_page(p, b, k);
                    if (page[i] < 0) atomicOr(p.status, kStatusBounds);
                }
            }
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                x[i] = page[i] < 0 ? make_uint4(0u, 0u, 0u, 0u)
                                   : *reinterpret_cast<const uint4*>(z.bounds + (size_t(page[i]) * p.Hkv + hk) * kRow + 8 * (threadIdx.x % kVecs));
        };
        load(ch);
        if (!have_sums) {
            have_sums = true;
            if (threadIdx.x < 2) top[threadIdx.x] = 0u;
            // eight columns of a token a thread, the lanes of a token side by side
            for (int e = threadIdx.x; e < kTileTokens * D / 8; e += kTileThreads) {
                const int i = e / (D / 8), v = e % (D / 8);
                float u[2][8], n = 0.f;  // w, u
#pragma unroll
                for (int j = 0; j < 8; ++j) u[0][j] = u[1][j] = 0.f;
                if (t0 + i < t1) {
                    const __nv_bfloat16* q = z.Q + (t0 + i) * z.q_stride + hk * z.g * D + 8 * v;
#pragma unroll 4
                    for (int h = 0; h < z.g; ++h) {
                        Vec<__nv_bfloat16> q8;
                        q8.load(q + h * D);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            u[0][j] += fminf(q8.v[j], 0.f);
                            u[1][j] += fmaxf(q8.v[j], 0.f);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) n += u[1][j] - u[0][j];
#pragma unroll
                for (int d = 1; d < D / 8; d <<= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
                if (v == 0) norms[i] = n;
#pragma unroll
                for (int part = 0; part < 3; ++part)
#pragma unroll
                    for (int side = 0; side < 2; ++side) {
                        uint32_t r[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float &a = u[side][2 * j], &c = u[side][2 * j + 1];
                            r[j] = pack_bf16x2(a, c);
                            a -= __uint_as_float(r[j] << 16);
                            c -= __uint_as_float(r[j] & 0xffff0000u);
                        }
                        *reinterpret_cast<uint4*>(sums + (part * kTileTokens + i) * kPitch + side * D + 8 * v) = make_uint4(r[0], r[1], r[2], r[3]);
                    }
            }
        }
        for (; ch < ch_end; ++ch, odd ^= 1u) {
            __syncthreads();  // (the last chunk's products are done)
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                m = max_bf16x2(max_bf16x2(m, x[i].x & 0x7fff7fffu), x[i].y & 0x7fff7fffu);
                m = max_bf16x2(max_bf16x2(m, x[i].z & 0x7fff7fffu), x[i].w & 0x7fff7fffu);
                const int e = threadIdx.x + kTileThreads * i;
                *reinterpret_cast<uint4*>(bounds + (e / kVecs) * kPitch + 8 * (e % kVecs)) = x[i];
            }
            m = max(m & 0xffffu, m >> 16);  // (magnitudes compare like whole numbers)
            m = __reduce_max_sync(0xffffffffu, m);
            if (lane == 0) atomicMax(&top[odd], m);
            __syncthreads();
            if (threadIdx.x == 0) top[odd ^ 1u] = 0u;
            if (ch + 1 < ch_end) load(ch + 1);
            float acc[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
            // ldmatrix sources: rows of this warp's tokens and blocks, and 16-byte pieces
            const __nv_bfloat16* pa = sums + (m0 + (lane & 15)) * kPitch + 8 * (lane >> 4);
            const __nv_bfloat16* pb = bounds + (n0 + (lane & 7) + 8 * (lane >> 4)) * kPitch + 8 * ((lane >> 3) & 1);
#pragma unroll 4
            for (int d = 0; d < kRow; d += 16) {
                uint32_t bb[4];
                ldmatrix4(bb, pb + d);
                float c[2][4] = {};
#pragma unroll
                for (int part = 2; part >= 0; --part) {
                    uint32_t a[4];
                    ldmatrix4(a, pa + part * kTileTokens * kPitch + d);
                    mma_bf16(c[0], a, bb[0], bb[1]);
                    mma_bf16(c[1], a, bb[2], bb[3]);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][i] += c[j][i];
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int t = t0 + m0 + (lane >> 2) + 8 * r, pos = kv - q1 + t, n = (pos >> p.page_log2) + 1;
                if (t < ta || t >= tb || pos < 0 || n <= z.n_blocks) continue;
                float* out = z.scores + (size_t(t) * p.Hkv + hk) * size_t(p.max_pages);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = ch * kChunk + n0 + 8 * (j >> 1) + 2 * (lane & 3) + (j & 1);
                    if (k >= z.n_first && k < n - z.n_last) out[k] = acc[j >> 1][2 * r + (j & 1)];
                }
            }
            if (threadIdx.x < kTileTokens) {
                const int t = t0 + int(threadIdx.x), pos = kv - q1 + t;
                if (t >= ta && t < tb && pos >= 0 && (pos >> p.page_log2) + 1 > z.n_blocks)
                    z.slack[(size_t(t) * p.Hkv + hk) * size_t(z.chunks) + ch] =
                        slack_of(z, 35 + D / 8 + 1, __uint_as_float(top[odd] << 16), norms[threadIdx.x]);
            }
        }
    }
}

__device__ __forceinline__ uint32_t ordered(float x) {  // larger scores, larger keys
    const uint32_t b = __float_as_uint(x + 0.f);        // (-0 is 0)
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// The score of block k in 64 bits, by a warp.
__device__ __forceinline__ double exact_score(const BlockParams& z, int b, int hk, int k, const double* sums, int lane) {
    const CacheAppendParams& p = z.a;
    const int page = block_page(p, b, k);
    double s = 0.0;
    if (page >= 0) {
        const __nv_bfloat16* src = z.bounds + (size_t(page) * p.Hkv + hk) * 2 * p.D;
        for (int d = lane; d < 2 * p.D; d += 32) s = fma(double(__bfloat162float(src[d])), sums[d], s);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
}

__device__ __forceinline__ unsigned long long ordered64(double x) {
    const unsigned long long b = __double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | (1ull << 63);
}

// The threads that choose for one token and key head: a warp of a CTA, or a CTA (of 4 or 32 warps).  Their kernels run
// alone and cold, so what they cost beside latencies is the code they fetch: scores lie in shared
// memory and loops stay rolled, and what few items need is a call (scores in registers, every pass laid
// out: 37.7 us for a step over one history of 131k keys instead of 27.1).
template <int WARPS>
struct Choosers {
    static constexpr int kThreads = 32 * WARPS, kItems = WARPS == 1 ? 4 : 1;
    static constexpr int kHeld = WARPS == 1 ? 512 : WARPS <= 4 ? 1024 : 8192, kCands = WARPS <= 4 ? 128 : 1024;
    struct Smem {
        float held[kHeld];
        unsigned long long keys[kCands];
        double sums[2 * 128];
        int cand[kCands];
        unsigned long long prefix;
        float ends[3][WARPS > 2 ? WARPS : 2];
        int hist[256];
        int parts[2][WARPS];
        int left, found;
    };
    Smem* m;
    int thread, lane, warp, turn;

    __device__ void sync() const {
        if (WARPS == 1)
            __syncwarp();
        else
            __syncthreads();
    }
    __device__ int total(int a) {  // (two buffers: one synchronisation a sum)
        a = __reduce_add_sync(0xffffffffu, a);
        if (WARPS == 1) return a;
        turn ^= 1;
        if (lane == 0) m->parts[turn][warp] = a;
        __syncthreads();
        return __reduce_add_sync(0xffffffffu, lane < WARPS ? m->parts[turn][lane] : 0);
    }
    // a's sum over the threads before this one, and over all of them
    __device__ int before(bool a, int& all) {
        const uint32_t votes = __ballot_sync(0xffffffffu, a);
        const int mine = __popc(votes & ((1u << lane) - 1u));
        all = __popc(votes);
        if (WARPS == 1) return mine;
        turn ^= 1;
        if (lane == 0) m->parts[turn][warp] = all;
        __syncthreads();
        const int p = lane < WARPS ? m->parts[turn][lane] : 0;
        all = __reduce_add_sync(0xffffffffu, p);
        return __reduce_add_sync(0xffffffffu, lane < warp ? p : 0) + mine;
    }
};

// Settles the candidates, scores in [low, above], of which the best `need` are chosen: their scores become
// +inf or -inf.  In 64 bits, on arithmetic units that are few here, so only what settle leaves.
template <int WARPS>
__device__ __noinline__ void settle_exactly(Choosers<WARPS>& g, const BlockParams& z, const int t, const int b, const int hk, const int first,
                                            float* sc, const int n, const float low, const float above, const int need, const int nc) {
    using C = Choosers<WARPS>;
    auto is_cand = [&](int i) { return i < n && sc[i] >= low && sc[i] <= above; };
    query_sums<double>(z, t, hk, g.m->sums, g.thread, C::kThreads);
    if (g.thread == 0) g.m->found = 0;
    g.sync();
    if (nc <= C::kCands) {
        for (int i = g.thread; i < n; i += C::kThreads)
            if (is_cand(i)) g.m->cand[atomicAdd(&g.m->found, 1)] = i;
        g.sync();
        for (int i = g.warp; i < nc; i += WARPS) {
            const double s = exact_score(z, b, hk, first + g.m->cand[i], g.m->sums, g.lane);
            if (g.lane == 0) g.m->keys[i] = ordered64(s);
        }
        g.sync();
        for (int i = g.thread; i < nc; i += C::kThreads) {
            const unsigned long long mine = g.m->keys[i];
            const int at = g.m->cand[i];
            int rank = 0;
            for (int j = 0; j < nc; ++j) rank += g.m->keys[j] > mine || (g.m->keys[j] == mine && g.m->cand[j] < at);
            sc[at] = rank < need ? INFINITY : -INFINITY;
        }
        g.sync();
        return;
    }
    // Very many nearly equal scores: the need-th largest exact score, eight bits at a time, each
    // pass scoring all candidates again; then equal ones by their index.
    if (g.thread == 0) {
        g.m->prefix = 0ull;
        g.m->left = need;
    }
    auto key_of = [&](int i) { return ordered64(exact_score(z, b, hk, first + i, g.m->sums, g.lane)); };
    for (int shift = 56; shift >= 0; shift -= 8) {
        for (int i = g.thread; i < 256; i += C::kThreads) g.m->hist[i] = 0;
        g.sync();
        const unsigned long long mask = shift == 56 ? 0ull : ~0ull << (shift + 8), want = g.m->prefix;
        for (int i = g.warp; i < n; i += WARPS) {
            if (!is_cand(i)) continue;
            const unsigned long long key = key_of(i);
            if (g.lane == 0 && (key & mask) == want) atomicAdd(&g.m->hist[int((key >> shift) & 255u)], 1);
        }
        g.sync();
        if (g.thread == 0) {
            int higher = 0, d = 255;
            while (d > 0 && higher + g.m->hist[d] < g.m->left) higher += g.m->hist[d--];
            g.m->left -= higher;
            g.m->prefix |= (unsigned long long)(d) << shift;
        }
        g.sync();
    }
    const unsigned long long border = g.m->prefix;
    int equal = g.m->left;  // of those at the border, the first so many
    for (int i0 = 0; i0 < n; i0 += WARPS) {
        const int i = i0 + g.warp;
        const bool is = is_cand(i);
        const unsigned long long key = is ? key_of(i) : 0ull;
        int all;
        // (one vote a warp: thread 0 of each)
        const int at = g.before(g.lane == 0 && is && key == border, all);
        if (g.lane == 0 && is) sc[i] = key > border || (key == border && at < equal) ? INFINITY : -INFINITY;
        equal -= all;
    }
    g.sync();
}

// a + b = s + e exactly (Knuth).
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
    s = __fadd_rn(a, b);
    const float v = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, v)), __fsub_rn(b, v));
}

// The same in pairs of floats: sums and products with their rounding errors carried along (Ogita, Rump
// and Oishi, SIAM J. Sci. Comput. 26, 2005).  A lane's 8 terms and 5 steps between lanes leave an error below
// 2^-40 of the products' magnitudes, less than slack / 2^20.  What even that leaves open goes on
// to settle_exactly.  slack 0: all bounds or all queries are zero, the candidates' scores exact and equal.
template <int WARPS>
__device__ __noinline__ void settle(Choosers<WARPS>& g, const BlockParams& z, const int t, const int b, const int hk, const int first, float* sc,
                                    const int n, const float low, const float above, const float slack, const int need, const int nc) {
    using C = Choosers<WARPS>;
    const CacheAppendParams& p = z.a;
    auto is_cand = [&](int i) { return i < n && sc[i] >= low && sc[i] <= above; };
    if (slack == 0.f) {
        int seen = 0, all;
        for (int i0 = 0; i0 < n; i0 += C::kThreads) {
            const int i = i0 + g.thread;
            const bool is = is_cand(i);
            const int at = seen + g.before(is, all);
            if (is) sc[i] = at < need ? INFINITY : -INFINITY;
            seen += all;
        }
        g.sync();
        return;
    }
    if (nc > C::kCands) {
        settle_exactly<WARPS>(g, z, t, b, hk, first, sc, n, low, above, need, nc);
        return;
    }
    float2* pairs = reinterpret_cast<float2*>(g.m->keys);
    // A lane has 8 (or 4) of a block's 2 D bounds, lo's in the first half of the lanes, and their queries' sums.
    const int per = p.D / 16, d0 = (g.lane & 15) * per;
    float hi8[8], lo8[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) hi8[j] = lo8[j] = 0.f;
    const __nv_bfloat16* q = z.Q + t * z.q_stride + hk * z.g * p.D + d0;
    auto eight = [&](const __nv_bfloat16* src, float (&v)[8]) {
        const uint2 a = *reinterpret_cast<const uint2*>(src), b = per == 8 ? *reinterpret_cast<const uint2*>(src + 4) : make_uint2(0u, 0u);
        Vec<__nv_bfloat16> x;
        x.set(make_uint4(a.x, a.y, b.x, b.y));
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = x.v[j];
    };
#pragma unroll(WARPS == 1 ? 4 : 1)
    for (int h = 0; h < z.g; ++h) {
        float x[8], e;
        eight(q + h * p.D, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            two_sum(hi8[j], g.lane < 16 ? fminf(x[j], 0.f) : fmaxf(x[j], 0.f), hi8[j], e);
            lo8[j] += e;
        }
    }
    if (g.thread == 0) g.m->found = 0;
    g.sync();
    for (int i = g.thread; i < n; i += C::kThreads)
        if (is_cand(i)) g.m->cand[atomicAdd(&g.m->found, 1)] = i;
    g.sync();
    constexpr int kAtOnce = WARPS == 1 ? 4 : 1;  // candidates whose pages and bounds a warp asks for together
    for (int i0 = g.warp * kAtOnce; i0 < nc; i0 += WARPS * kAtOnce) {
        int page[kAtOnce];
        float x[kAtOnce][8];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) page[k] = i0 + k < nc ? block_page(p, b, first + g.m->cand[i0 + k]) : -1;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (page[k] >= 0) eight(z.bounds + (size_t(page[k]) * p.Hkv + hk) * 2 * p.D + per * g.lane, x[k]);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (i0 + k >= nc) break;
            float s = 0.f, c = 0.f, e;
            if (page[k] >= 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float m = __fmul_rn(x[k][j], hi8[j]), r = __fmaf_rn(x[k][j], hi8[j], -m);
                    two_sum(s, m, s, e);
                    c += e + (r + x[k][j] * lo8[j]);
                }
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                const float other = __shfl_xor_sync(0xffffffffu, s, d);
                c += __shfl_xor_sync(0xffffffffu, c, d);
                two_sum(s, other, s, e);
                c += e;
            }
            two_sum(s, c, s, e);
            if (g.lane == 0) pairs[i0 + k] = make_float2(s, e);
        }
    }
    g.sync();
    // the need-th and the next, by pairs
    float2* border = reinterpret_cast<float2*>(g.m->ends);
    uint8_t* chosen = reinterpret_cast<uint8_t*>(g.m->sums);
    static_assert(C::kCands <= sizeof(g.m->sums));
    for (int i = g.thread; i < nc; i += C::kThreads) {
        const float2 mine = pairs[i];
        const int at = g.m->cand[i];
        int rank = 0;
        for (int j = 0; j < nc; ++j) {
            const float2 o = pairs[j];
            rank += o.x > mine.x || (o.x == mine.x && (o.y > mine.y || (o.y == mine.y && g.m->cand[j] < at)));
        }
        if (rank == need - 1 || rank == need) border[rank - need + 1] = mine;
        chosen[i] = rank < need;
    }
    g.sync();
    const bool open = (border[0].x - border[1].x) + (border[0].y - border[1].y) <= 0x1p-14f * slack;
    g.sync();
    if (open) {
        settle_exactly<WARPS>(g, z, t, b, hk, first, sc, n, low, above, need, nc);
        return;
    }
    for (int i = g.thread; i < nc; i += C::kThreads) sc[g.m->cand[i]] = chosen[i] ? INFINITY : -INFINITY;
    g.sync();
}

// The k-th largest score where very many are nearly equal (or all are): halves the values between the least and
// the largest, after 16 steps their bit patterns.
template <int WARPS>
__device__ __noinline__ float search(Choosers<WARPS>& g, const float* sc, const int n, const int k, const float small, const float large) {
    uint32_t lo = ordered(small), hi = ordered(large) + 1u;  // k scores or more are at least lo, fewer at least hi
    for (int step = 0; hi - lo > 1u && step < 64; ++step) {
        uint32_t mid = lo + (hi - lo) / 2u;
        if (step < 16) {
            const uint32_t m = ordered(0.5f * unordered(lo) + 0.5f * unordered(hi - 1u));
            if (m > lo && m < hi) mid = m;
        }
        const float c = unordered(mid);
        int a = 0;
        for (int i = g.thread; i < n; i += Choosers<WARPS>::kThreads) a += sc[i] >= c;
        if (g.total(a) >= k)
            lo = mid;
        else
            hi = mid;
    }
    return unordered(lo);
}

// The chosen blocks of one token and key head, from its scores.
template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS * Choosers<WARPS>::kItems, WARPS <= 4 ? 5 : 1) jfa_cache_choose_kernel(const BlockParams z) {
    using C = Choosers<WARPS>;
    const CacheAppendParams& p = z.a;
    extern __shared__ __align__(16) uint8_t choose_smem[];
    const int item = blockIdx.x * C::kItems + threadIdx.x / C::kThreads, t = item / p.Hkv, hk = item - t * p.Hkv;
    C g{reinterpret_cast<typename C::Smem*>(choose_smem) + threadIdx.x / C::kThreads, int(threadIdx.x % C::kThreads), int(threadIdx.x & 31),
        int(threadIdx.x % C::kThreads) >> 5, 0};
    // (every thread waits for the scores' kernel, also those with nothing to choose: what follows in the stream
    // starts once this kernel has ended, and must find that one's reads done)
    const Chooser c = t < p.T ? chooser(p, t, g.lane, g.thread == 0) : Chooser{-1, 0};
    if (c.b < 0) {
        wait_previous();
        return;
    }
    int32_t* out = z.blocks + (size_t(t) * p.Hkv + hk) * size_t(z.n_blocks);
    const int all = c.own + 1, first = z.n_first, k = z.n_blocks - z.n_first - z.n_last, n = all - z.n_last - first;  // n compete for k places
    const bool few = all <= z.n_blocks;
    // the blocks that are chosen in any case, or all that there are
#pragma unroll 1
    for (int i = g.thread; i < z.n_blocks; i += C::kThreads) {
        if (few)
            out[i] = i < all ? i : -1;
        else if (i < first || i >= first + k)
            out[i] = i < first ? i : all - z.n_blocks + i;
    }
    wait_previous();
    if (few || k == 0) return;
    float* sc = z.scores + (size_t(t) * p.Hkv + hk) * size_t(p.max_pages) + first;
    const float* sl = z.slack + (size_t(t) * p.Hkv + hk) * size_t(z.chunks);
    float small = INFINITY, large = -INFINITY, slack = 0.f;
    const bool held = n <= C::kHeld;
#pragma unroll 4
    for (int i = g.thread; i < n; i += C::kThreads) {
        const float x = sc[i] + 0.f;  // (-0 is 0)
        small = fminf(small, x);
        large = fmaxf(large, x);
        if (held) g.m->held[i] = x;
    }
    if (held) sc = g.m->held;
#pragma unroll 1
    for (int i = first / kChunk + g.thread; i <= (first + n - 1) / kChunk; i += C::kThreads) slack = fmaxf(slack, sl[i]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        small = fminf(small, __shfl_xor_sync(0xffffffffu, small, d));
        large = fmaxf(large, __shfl_xor_sync(0xffffffffu, large, d));
        slack = fmaxf(slack, __shfl_xor_sync(0xffffffffu, slack, d));
    }
    if (WARPS > 1) {
        if (g.lane == 0) {
            g.m->ends[0][g.warp] = small;
            g.m->ends[1][g.warp] = large;
            g.m->ends[2][g.warp] = slack;
        }
        __syncthreads();
#pragma unroll 1
        for (int w = 0; w < WARPS; ++w) {
            small = fminf(small, g.m->ends[0][w]);
            large = fmaxf(large, g.m->ends[1][w]);
            slack = fmaxf(slack, g.m->ends[2][w]);
        }
    } else {
        __syncwarp();
    }
    // The k-th largest score, `up`, and the next, `down`: the scores by 256 steps of their range, then
    // those of the step that holds the k-th by their rank.
    float up, down = -INFINITY, kth;
    const bool wild = slack == INFINITY;  // (the scores are of no use: all are taken again in 64 bits)
    if (wild) {
#pragma unroll 1
        for (int i = g.thread; i < n; i += C::kThreads) sc[i] = 0.f;
        g.sync();
        settle_exactly<WARPS>(g, z, t, c.b, hk, first, sc, n, -INFINITY, INFINITY, k, n);
        up = INFINITY;
    }
    bool found = !wild && large > small;
    if (found) {
        const float per = 255.f / (large - small);
        auto step_of = [&](float x) { return max(0, min(int((x - small) * per), 255)); };
#pragma unroll 1
        for (int i = g.thread; i < 256; i += C::kThreads) g.m->hist[i] = 0;
        if (g.thread == 0) {
            g.m->found = g.m->left = 0;
            g.m->prefix = 0ull;
        }
        g.sync();
#pragma unroll 4
        for (int i = g.thread; i < n; i += C::kThreads) atomicAdd(&g.m->hist[step_of(sc[i])], 1);
        g.sync();
        if (g.warp == 0) {  // a lane eight steps, from the top
            int mine = 0;
#pragma unroll 1
            for (int j = 0; j < 8; ++j) mine += g.m->hist[255 - (8 * g.lane + j)];
            int higher = warp_scan(mine, g.lane) - mine;
            if (higher < k && higher + mine >= k) {
                int j = 255 - 8 * g.lane;
                while (higher + g.m->hist[j] < k) higher += g.m->hist[j--];
                g.m->left = j;
                g.m->prefix = higher;
            }
        }
        g.sync();
        const int step = g.m->left, rank = k - 1 - int(g.m->prefix), here = g.m->hist[step];
        float* list = reinterpret_cast<float*>(g.m->keys);
        found = here <= C::kCands;
        if (found) {
#pragma unroll 4
            for (int i = g.thread; i < n; i += C::kThreads) {
                const float x = sc[i];
                const int at = step_of(x);
                if (at == step)
                    list[atomicAdd(&g.m->found, 1)] = x;
                else if (at < step)
                    down = fmaxf(down, x);
            }
            g.sync();
#pragma unroll 1
            for (int i = g.thread; i < here; i += C::kThreads) {
                const float x = list[i];
                int r = 0;
#pragma unroll 4
                for (int j = 0; j < here; ++j) r += list[j] > x || (list[j] == x && j < i);
                if (r == rank) g.m->ends[0][0] = x;
                if (r == rank + 1) g.m->ends[0][1] = x;
            }
            g.sync();
            up = g.m->ends[0][0];
            if (rank + 1 < here) {
                down = g.m->ends[0][1];
            } else {  // the largest of the lower steps
                down = unordered(__reduce_max_sync(0xffffffffu, ordered(down)));
                if (WARPS > 1) {
                    if (g.lane == 0) g.m->ends[1][g.warp] = down;
                    __syncthreads();
#pragma unroll 1
                    for (int w = 0; w < WARPS; ++w) down = fmaxf(down, g.m->ends[1][w]);
                }
            }
        }
    }
    if (!found && !wild) up = down = search<WARPS>(g, sc, n, k, small, large);
    kth = up;
    float cut = kth;  // chosen: scores of at least this
    // Scores further apart than twice the slack are in the order of the exact ones: then the k largest
    // are the chosen ones.
    if (!wild && up - down <= 2.01f * slack) {
        const float above = __fadd_ru(kth, 2.f * slack), low = __fadd_rd(kth, -2.f * slack);
        int sure = 0, maybe = 0;
#pragma unroll 1
        for (int i = g.thread; i < n; i += C::kThreads) {
            sure += sc[i] > above;
            maybe += sc[i] >= low && sc[i] <= above;
        }
        sure = g.total(sure);
        maybe = g.total(maybe);
        cut = low;
        if (sure + maybe != k) {
            settle<WARPS>(g, z, t, c.b, hk, first, sc, n, low, above, slack, k - sure, maybe);
            // (chosen candidates are +inf now, the others -inf)
            cut = above;
        }
    }
    int done = 0;  // the chosen ones, ascending
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += C::kThreads) {
        const int i = i0 + g.thread;
        const bool in = i < n && sc[i] >= cut;
        int here;
        const int to = done + g.before(in, here);
        if (in && to < k) out[first + to] = first + i;
        done += here;
    }
}

constexpr int kMaxChunks = 65535;  // of a grid's second dimension
int chunks_of(int32_t max_pages) { return max_pages > 0 ? (max_pages - 1) / kChunk + 1 : 1; }

void batch_params(CacheAppendParams& p, jfa_cache c, int32_t B, int64_t T, const int32_t* q_offsets, const int32_t* kv_lens,
                  const int32_t* page_table, int32_t max_pages) {
    p.q_off = q_offsets;
    p.kv_lens = kv_lens;
    p.table = page_table;
    p.B = B;
    p.max_pages = max_pages;
    p.T = int(T);
    p.Hkv = c->Hkv;
    p.D = c->D;
    p.page_log2 = c->page_log2;
    p.n_pages = c->n_pages;
    p.Kc = c->K;
    p.Vc = c->V;
    for (int i = 0; i < 3; ++i) {
        p.ks[i] = c->ks[i];
        p.vs[i] = c->vs[i];
    }
    p.status = c->d_status;
}

// Started while the scores are still computed, whose end it waits for.
template <int WARPS>
cudaError_t launch_choice(const BlockParams& z, int64_t items, cudaStream_t st) {
    using C = Choosers<WARPS>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(jfa_cache_choose_kernel<WARPS>, int(sizeof(typename C::Smem)) * C::kItems, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((items + C::kItems - 1) / C::kItems));
    cfg.blockDim = dim3(C::kThreads * C::kItems);
    cfg.dynamicSmemBytes = sizeof(typename C::Smem) * C::kItems;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = z.a.max_pages > z.n_blocks ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, jfa_cache_choose_kernel<WARPS>, z);
}

// Blocks are those of bf16 and 4-bit caches with pages of at least 16 positions.
jfa_status check_blocks(jfa_cache c) { return c->dtype == JFA_BF16 && c->page_log2 >= 4 ? JFA_OK : JFA_ERR_UNSUPPORTED; }

}  // namespace

}  // namespace jfa

extern "C" {

jfa_status jfa_cache_summarize(jfa_cache cache, int32_t B, int64_t T, const int32_t* q_offsets, const int32_t* kv_lens,
                               const int32_t* page_table, int32_t max_pages, void* bounds, void* stream) {
    BlockParams z{};
    jfa_status s = check_batch(cache, B, T, q_offsets, kv_lens, page_table, max_pages, &z.a.max_kv);
    if (s == JFA_OK) s = check_blocks(cache);
    if (s != JFA_OK) return s;
    if (!bounds || !aligned(bounds, 16)) return JFA_ERR_INVALID_ARG;
    if (!on_device(cache)) return JFA_ERR_PLAN_MISMATCH;
    if (B == 0 || T == 0) return JFA_OK;
    batch_params(z.a, cache, B, T, q_offsets, kv_lens, page_table, max_pages);
    z.bounds = static_cast<__nv_bfloat16*>(bounds);
    z.k_scales = cache->k_scales;
    for (int i = 0; i < 2; ++i) z.kss[i] = cache->kss[i];
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // A CTA for as many tokens as a sequence has on average, at most a page's: about a page each.  (A page's
    // worth always: 16 x 8 tokens on pages of 32 9.0 us instead of 3.5, 512 single ones 61 instead of 7.4; a CTA
    // for each token: 16 x 64 tokens 5.9 instead of 3.6, 512 of one sequence 4.3 instead of 3.5.)
    for (z.tile = 1; z.tile < 1 << cache->page_log2 && 2 * int64_t(z.tile) * B <= T;) z.tile *= 2;
    const int grid = int((T + z.tile - 1) / z.tile);
    if (cache->ops)
        jfa_cache_summarize_kernel<true><<<grid, kSumThreads, 0, st>>>(z);
    else
        jfa_cache_summarize_kernel<false><<<grid, kSumThreads, 0, st>>>(z);
    return cudaGetLastError() == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

size_t jfa_cache_select_workspace_size(jfa_cache cache, int64_t T, int32_t max_pages) {
    // (sizes that jfa_cache_select refuses have no workspace: it would not always fit 64 bits)
    if (!cache || T < 0 || T > (1 << 30) || max_pages < 0 || T * cache->Hkv > INT32_MAX || chunks_of(max_pages) > kMaxChunks) return 0;
    return 256 + size_t(T) * size_t(cache->Hkv) * (size_t(max_pages) + size_t(chunks_of(max_pages))) * 4;
}

jfa_status jfa_cache_select(jfa_cache cache, int32_t B, int64_t T, int32_t max_q_len, const int32_t* q_offsets,
                            const int32_t* kv_lens, const int32_t* page_table, int32_t max_pages, const void* bounds,
                            const void* Q, int64_t q_stride, int32_t H, int32_t n_blocks, int32_t n_first, int32_t n_last,
                            int32_t* blocks, void* workspace, size_t workspace_bytes, void* stream) {
    BlockParams z{};
    jfa_status s = check_batch(cache, B, T, q_offsets, kv_lens, page_table, max_pages, &z.a.max_kv);
    if (s == JFA_OK) s = check_blocks(cache);
    if (s != JFA_OK) return s;
    if (H < 1 || H > 65535 || H % cache->Hkv != 0 || T * H > INT32_MAX - 256 || max_q_len < 0) return JFA_ERR_INVALID_ARG;
    if (H / cache->Hkv > 128 || chunks_of(max_pages) > kMaxChunks) return JFA_ERR_UNSUPPORTED;
    if (n_first < 0 || n_last < 1 || n_blocks < 1 || n_first > n_blocks - n_last ||
        (int64_t(n_blocks) << cache->page_log2) > (1 << 30))
        return JFA_ERR_INVALID_ARG;
    if (!bounds || !aligned(bounds, 16) || (T > 0 && (!row_ok(cache, Q, q_stride, H) || !blocks || !aligned(blocks, 4))))
        return JFA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < jfa_cache_select_workspace_size(cache, T, max_pages))
        return JFA_ERR_INVALID_ARG;
    if (!on_device(cache)) return JFA_ERR_PLAN_MISMATCH;
    if (B == 0 || T == 0) return JFA_OK;
    batch_params(z.a, cache, B, T, q_offsets, kv_lens, page_table, max_pages);
    z.bounds = static_cast<__nv_bfloat16*>(const_cast<void*>(bounds));
    z.Q = static_cast<const __nv_bfloat16*>(Q);
    z.q_stride = q_stride;
    z.g = H / cache->Hkv;
    z.n_blocks = n_blocks;
    z.n_first = n_first;
    z.n_last = n_last;
    z.blocks = blocks;
    z.chunks = chunks_of(max_pages);
    z.scores = static_cast<float*>(workspace);
    z.slack = z.scores + size_t(T) * size_t(cache->Hkv) * size_t(max_pages);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (max_pages > n_blocks) {
        // Many tokens a sequence (as far as the host knows): 32 of them share the bounds' reads.  On 8 key
        // heads of 128 over 250 blocks, token by token against in tiles: 4 x 8 tokens 18.6 and 28.7 us, 16 x 8
        // 32.4 and 30.8, 64 x 8 (125 blocks) 55.5 and 39.1, 1 x 16 15.4 and 17.6, 16 x 16 49.9 and 25.7, 1 x 512 87.8 and 34.3.
        const bool tiles = (max_q_len == 0 || max_q_len > 4) && T >= 8 * int64_t(B) && T >= 128;
        cudaError_t e = cudaSuccess;
        if (tiles) {
            const int D = cache->D, bytes = (3 * kTileTokens + kChunk) * (2 * D + 8) * 2, tiles_of_tokens = (z.a.T + kTileTokens - 1) / kTileTokens;
            // four times as many CTAs as run at a time, where the chunks allow: 58 us for the prompts of the kernel's
            // comment, against 61 for twice as many, 63 for as many (with a few of them in a second wave)
            const int64_t ctas = int64_t(tiles_of_tokens) * cache->Hkv, parts = std::max<int64_t>(1, std::min<int64_t>(z.chunks, (8 * cache->num_sms + ctas - 1) / ctas));
            z.tile = int((z.chunks + parts - 1) / parts);
            const dim3 grid(tiles_of_tokens, (z.chunks + z.tile - 1) / z.tile, cache->Hkv);
            static std::atomic<uint64_t> done[2];
            e = D == 128 ? allow_smem(jfa_cache_score_tile_kernel<128>, bytes, done[0]) : allow_smem(jfa_cache_score_tile_kernel<64>, bytes, done[1]);
            if (e == cudaSuccess) {
                if (D == 128)
                    jfa_cache_score_tile_kernel<128><<<grid, kTileThreads, bytes, st>>>(z);
                else
                    jfa_cache_score_tile_kernel<64><<<grid, kTileThreads, bytes, st>>>(z);
            }
        } else {
            const dim3 grid(z.a.T, z.chunks, cache->Hkv);
            if (cache->D == 128)
                jfa_cache_score_kernel<128><<<grid, kScoreThreads, 0, st>>>(z);
            else
                jfa_cache_score_kernel<64><<<grid, kScoreThreads, 0, st>>>(z);
        }
        if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return JFA_ERR_CUDA;
    }
    // As many warps an item as hold its scores and fill the SMs: one where there are many items, four, or a
    // CTA's 32.  On 8 heads, 250 blocks, with one, four and 32: 8 items 8.6, 6.4 and 8.5 us, 64 14.8, 9.9 and
    // 9.5, 128 15.4, 8.4 and 10.7, 512 24.4, 20.0 and 36, 1024 30.7, 29.5 and 63, 2048 25.9, 28.6 and 94 (in tiles),
    // 4096 (125 blocks) 42, 53 and 203.
    const int64_t items = T * cache->Hkv;
    cudaError_t e;
    if (max_pages <= Choosers<1>::kHeld && items > 8 * cache->num_sms)
        e = launch_choice<1>(z, items, st);
    else if (max_pages <= Choosers<4>::kHeld)
        e = launch_choice<4>(z, items, st);
    else
        e = launch_choice<kSelWarps>(z, items, st);
    return e == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

jfa_status jfa_cache_fwd_blocks(jfa_cache cache, int32_t B, int64_t T, const int32_t* q_offsets, const int32_t* kv_lens,
                                const int32_t* page_table, int32_t max_pages, const void* Q, int64_t q_stride, int32_t H,
                                const int32_t* blocks, int32_t n_blocks, int32_t bias_kind, const float* bias_table, float scale,
                                void* O, int32_t o_dtype, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    int32_t max_kv = 0;
    jfa_status s = check_batch(cache, B, T, q_offsets, kv_lens, page_table, max_pages, &max_kv);
    if (s == JFA_OK) s = check_blocks(cache);
    if (s != JFA_OK) return s;
    if (H < 1 || H > 65535 || H % cache->Hkv != 0 || T * H > INT32_MAX - 256) return JFA_ERR_INVALID_ARG;
    if (H / cache->Hkv > kDecodeRows) return JFA_ERR_UNSUPPORTED;  // a token's rows are one row tile
    if (bias_kind != JFA_BIAS_NONE && bias_kind != JFA_BIAS_RELPOS32)
        return bias_kind == JFA_BIAS_DENSE ? JFA_ERR_UNSUPPORTED : JFA_ERR_INVALID_ARG;
    if (bias_kind == JFA_BIAS_RELPOS32 && (!bias_table || !aligned(bias_table, 4))) return JFA_ERR_INVALID_ARG;
    if (!(scale > 0.f && scale < INFINITY) ||
        (cache->ops && !(scale * cache->k_factor >= 1e-37f && scale * cache->k_factor <= 1e37f)))
        return JFA_ERR_INVALID_ARG;
    if (o_dtype != JFA_BF16 && o_dtype != JFA_F32) return JFA_ERR_INVALID_ARG;
    if (n_blocks < 1 || (int64_t(n_blocks) << cache->page_log2) > (1 << 30)) return JFA_ERR_INVALID_ARG;
    if (T > 0 && (!row_ok(cache, Q, q_stride, H) || !O || O == Q || !aligned(O, 16) || !aligned(lse, 4) || !blocks || !aligned(blocks, 4)))
        return JFA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < jfa_cache_workspace_size(cache, H)) return JFA_ERR_INVALID_ARG;
    // the kernels count units in 31 bits
    const double keys = std::min<double>(double(n_blocks) * (1 << cache->page_log2), max_kv + 1024.0);
    if (double(T) * cache->Hkv * (keys / 64 + 16.0) >= double(INT32_MAX) - 65536.0) return JFA_ERR_UNSUPPORTED;
    if (!on_device(cache)) return JFA_ERR_PLAN_MISMATCH;
    if (B == 0 || T == 0) return JFA_OK;
    CacheFwdParams p{};
    fwd_params(p, cache, B, T, q_offsets, kv_lens, page_table, max_pages, max_kv, Q, q_stride, H, 1, -1,
               bias_kind == JFA_BIAS_RELPOS32 ? bias_table : nullptr, scale, O, o_dtype, lse, workspace);
    p.lists = blocks;
    p.n_list = n_blocks;
    p.bm = p.g;
    p.min_units = 1;
    p.item_cost = cache->ops ? kDecode4ItemUnits : kDecodeItemUnits;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = cache->ops ? launch_cache_decode4(cache->D, cache->mk, cache->mv, p, false, cache->num_sms, st)
                                     : launch_cache_decode_lists(cache->D, cache->mk, cache->mv, p, cache->num_sms, st);
    return e == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

}  // extern "C"
