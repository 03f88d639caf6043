// Attention over selected blocks of a paged cache: the blocks' bounds, the selection, and the
// attention call.  A block is a page.  Semantics are documented in include/jfa.h.
//
// The score of a block for a token and key head is the sum over the group's heads h of an upper
// bound of <q_h, k> over the block's keys,
//   sum_h sum_d max(q_hd lo_d, q_hd hi_d) = <u, hi> + <w, lo>,  u = sum_h max(q_h, 0), w = sum_h min(q_h, 0),
// with lo and hi the block's least and largest elements, so the group costs what one head does.
//
// The selection is that of exact arithmetic.  Scores are taken in fp32: u and w are sums of g values of
// one sign, and a dot product adds at most 128 products (the even or odd ones, or a lane's 32) and
// joins the sums in up to 3 steps, so a score is off by less than
//   slack = (g + 132) 2^-24 max|lo, hi| sum_d (u_d - w_d).
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
constexpr int kSumThreads = 512, kScoreThreads = 256, kTileThreads = 128;
constexpr int kTileTokens = 32;     // tokens that a CTA scores, where a sequence has many
constexpr int kWarpItems = 4, kWarpRegs = 16, kWarpHeld = 32 * kWarpRegs;    // choosing by warps: up to 512 scores
constexpr int kSelThreads = 512, kSelRegs = 16, kHeld = kSelThreads * kSelRegs;  // and by CTAs: so many in registers
constexpr int kExact = 1024;        // candidates whose 64-bit scores a CTA keeps

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
    int tile;                       // summarize: tokens that a CTA looks over
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
#pragma unroll 4
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

// What an fp32 score may be off by: m the largest magnitude among the bounds, norm the sums' norm
// (which is itself a sum of 2 D values, hence the 1.01).
__device__ __forceinline__ float slack_of(const BlockParams& z, float m, float norm) {
    return float(z.g + 132) * (1.01f * 0x1p-24f) * m * norm;
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
        z.slack[(size_t(t) * p.Hkv + hk) * size_t(z.chunks) + blockIdx.y] = slack_of(z, m, norm);
    }
}

// Scores of kChunk blocks for kTileTokens tokens and one key head: a matrix product in fp32 on the CUDA
// cores, bounds and sums in shared memory, four tokens by four blocks a thread, even and odd
// products in the halves of paired sums.  (A tensor core would need the sums in three parts.)  The
// tile's sequences come one after the other: it is taken where they are long.
template <int D>
__global__ void __launch_bounds__(kTileThreads) jfa_cache_score_tile_kernel(const BlockParams z) {
    const CacheAppendParams& p = z.a;
    constexpr int kRow = 2 * D, kPitch = kRow + 4, kBPitch = kRow + 8;  // floats; bf16 (rows of both end 16 bytes apart in the banks)
    extern __shared__ __align__(16) uint8_t tile_smem[];
    float* sums = reinterpret_cast<float*>(tile_smem);                  // [kTileTokens][kPitch]
    __nv_bfloat16* bounds = reinterpret_cast<__nv_bfloat16*>(sums + kTileTokens * kPitch);  // [kChunk][kBPitch]
    __shared__ float norms[kTileTokens];
    __shared__ uint32_t top;
    const int lane = threadIdx.x & 31, hk = blockIdx.z, t0 = blockIdx.x * kTileTokens, t1 = min(t0 + kTileTokens, p.T), k0 = blockIdx.y * kChunk;
    // tokens 4 tg .. and blocks bg + 16 i of a thread: a warp has two token groups
    const int tg = threadIdx.x >> 4, bg = threadIdx.x & 15;
    int b = find_sequence(p.q_off, p.B, t0, lane);
    if (b < 0) b = 0;
    bool have_sums = false;
    for (; b < p.B; ++b) {
        const int q0 = p.q_off[b], q1 = p.q_off[b + 1], kv = p.kv_lens[b];
        if (q0 >= t1) break;
        const int ta = max(q0, t0), tb = min(q1, t1);
        if (ta >= tb) continue;
        if (q0 < 0 || q1 > p.T || kv < 0 || kv > p.max_kv) {
            if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
            continue;
        }
        const int last = kv - q1 + tb - 1;                              // the last token's position
        const int most = last >= 0 ? (last >> p.page_log2) + 1 : 0;
        if (most <= z.n_blocks || k0 >= most - z.n_last) continue;
        const bool fresh = !have_sums;
        if (fresh) {
            have_sums = true;
            for (int e = threadIdx.x; e < kTileTokens * D; e += kTileThreads) {
                const int i = e / D, d = e % D;
                float u = 0.f, w = 0.f;
                if (t0 + i < t1) {
                    const __nv_bfloat16* q = z.Q + (t0 + i) * z.q_stride + hk * z.g * D + d;
                    for (int h = 0; h < z.g; ++h) {
                        const float x = __bfloat162float(q[h * D]);
                        u += fmaxf(x, 0.f);
                        w += fminf(x, 0.f);
                    }
                }
                sums[i * kPitch + d] = w;
                sums[i * kPitch + D + d] = u;
            }
        }
        if (threadIdx.x == 0) top = 0u;
        __syncthreads();
        if (fresh && threadIdx.x < kTileTokens) {
            float n = 0.f;
            for (int d = 0; d < kRow; ++d) n += fabsf(sums[threadIdx.x * kPitch + d]);
            norms[threadIdx.x] = n;
        }
        uint32_t m = 0u;
        for (int e = threadIdx.x; e < kChunk * (kRow / 8); e += kTileThreads) {
            const int i = e / (kRow / 8), v = e % (kRow / 8), k = k0 + i;
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (k >= z.n_first && k < most - z.n_last) {
                const int page = block_page(p, b, k);
                if (page >= 0)
                    x = *reinterpret_cast<const uint4*>(z.bounds + (size_t(page) * p.Hkv + hk) * kRow + 8 * v);
                else
                    atomicOr(p.status, kStatusBounds);
            }
            m = max_bf16x2(max_bf16x2(m, x.x & 0x7fff7fffu), x.y & 0x7fff7fffu);
            m = max_bf16x2(max_bf16x2(m, x.z & 0x7fff7fffu), x.w & 0x7fff7fffu);
            *reinterpret_cast<uint4*>(bounds + i * kBPitch + 8 * v) = x;
        }
        m = max(m & 0xffffu, m >> 16);  // (magnitudes compare like whole numbers)
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) atomicMax(&top, m);
        __syncthreads();
        float2 acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int d = 0; d < kRow; d += 4) {
            float4 u[4];
            uint2 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const float4*>(sums + (4 * tg + i) * kPitch + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const uint2*>(bounds + (bg + 16 * j) * kBPitch + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 lo = make_float2(__uint_as_float(x[j].x << 16), __uint_as_float(x[j].x & 0xffff0000u));
                const float2 hi = make_float2(__uint_as_float(x[j].y << 16), __uint_as_float(x[j].y & 0xffff0000u));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[i][j] = fma2(make_float2(u[i].x, u[i].y), lo, acc[i][j]);
                    acc[i][j] = fma2(make_float2(u[i].z, u[i].w), hi, acc[i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + 4 * tg + i, pos = kv - q1 + t;
            if (t < ta || t >= tb || pos < 0) continue;
            const int n = (pos >> p.page_log2) + 1;
            if (n <= z.n_blocks) continue;
            float* out = z.scores + (size_t(t) * p.Hkv + hk) * size_t(p.max_pages);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = k0 + bg + 16 * j;
                if (k >= z.n_first && k < n - z.n_last) out[k] = acc[i][j].x + acc[i][j].y;
            }
            if (bg == 0)
                z.slack[(size_t(t) * p.Hkv + hk) * size_t(z.chunks) + blockIdx.y] = slack_of(z, __uint_as_float(top << 16), norms[4 * tg + i]);
        }
        __syncthreads();
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

// The k-th largest (k >= 1) of the scores that a group of threads holds, NR a thread (-inf where there
// is none; at least k are finite): the border between `count(c) >= k` and `< k`, count(c) the
// number of scores of at least c, which is the same in all threads.  Halves the values between
// the smallest and the largest, and after that their bit patterns, until a border has k scores above.
template <int NR, typename Count, typename Least>
__device__ __forceinline__ float kth_largest(const float (&v)[NR], float smallest, float largest, int k, Count&& count, Least&& least) {
    uint32_t lo = ordered(smallest), hi = ordered(largest) + 1u;  // count(lo) >= k > count(hi)
    for (int step = 0; hi - lo > 1u; ++step) {
        uint32_t mid = lo + (hi - lo) / 2u;
        if (step < 16) {
            const uint32_t c = ordered(0.5f * unordered(lo) + 0.5f * unordered(hi - 1u));
            if (c > lo && c < hi) mid = c;
        }
        const float c = unordered(mid);
        const int n = count(c);
        if (n == k) return least(c);  // the smallest of those k
        if (n > k)
            lo = mid;
        else
            hi = mid;
    }
    return unordered(lo);
}

// The chosen blocks of one token and key head by one warp, its scores in registers: up to 512 blocks
// that compete.  Bound by latency: the sequence, the scores, about 12 steps of a search.
__global__ void __launch_bounds__(32 * kWarpItems) jfa_cache_choose_warp_kernel(const BlockParams z) {
    const CacheAppendParams& p = z.a;
    __shared__ unsigned long long keys[kWarpItems][kWarpHeld];
    __shared__ uint16_t cand[kWarpItems][kWarpHeld];
    __shared__ double sums[kWarpItems][2 * 128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, item = blockIdx.x * kWarpItems + warp;
    const int t = item / p.Hkv, hk = item - t * p.Hkv;
    if (t >= p.T) return;
    const Chooser c = chooser(p, t, lane, lane == 0);
    if (c.b < 0) return;
    int32_t* out = z.blocks + (size_t(t) * p.Hkv + hk) * size_t(z.n_blocks);
    const int n = c.own + 1;
    if (n <= z.n_blocks) {  // all that there are
        for (int i = lane; i < z.n_blocks; i += 32) out[i] = i < n ? i : -1;
        return;
    }
    const int first = z.n_first, end = n - z.n_last, m = end - first, k = z.n_blocks - z.n_first - z.n_last;  // m > k
    for (int i = lane; i < z.n_first; i += 32) out[i] = i;
    for (int i = lane; i < z.n_last; i += 32) out[z.n_first + k + i] = end + i;
    if (k == 0) return;
    const float* sc = z.scores + (size_t(t) * p.Hkv + hk) * size_t(p.max_pages) + first;
    const float* sl = z.slack + (size_t(t) * p.Hkv + hk) * size_t(z.chunks);
    float v[kWarpRegs], small = INFINITY, large = -INFINITY, slack = 0.f;
#pragma unroll
    for (int r = 0; r < kWarpRegs; ++r) {
        const int i = 32 * r + lane;
        v[r] = -INFINITY;
        if (i < m) {
            v[r] = sc[i] + 0.f;  // (-0 is 0)
            small = fminf(small, v[r]);
            large = fmaxf(large, v[r]);
        }
    }
    for (int i = first / kChunk + lane; i <= (end - 1) / kChunk; i += 32) slack = fmaxf(slack, sl[i]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        small = fminf(small, __shfl_xor_sync(0xffffffffu, small, d));
        large = fmaxf(large, __shfl_xor_sync(0xffffffffu, large, d));
        slack = fmaxf(slack, __shfl_xor_sync(0xffffffffu, slack, d));
    }
    auto count = [&](float c) {
        int a = 0;
#pragma unroll
        for (int r = 0; r < kWarpRegs; ++r) a += v[r] >= c;
        return __reduce_add_sync(0xffffffffu, a);
    };
    auto least = [&](float c) {
        float a = INFINITY;
#pragma unroll
        for (int r = 0; r < kWarpRegs; ++r)
            if (v[r] >= c) a = fminf(a, v[r]);
        return unordered(__reduce_min_sync(0xffffffffu, ordered(a)));
    };
    const float kth = kth_largest(v, small, large, k, count, least);
    // (rounding the limits outwards only moves a block to the candidates)
    const float above = __fadd_ru(kth, 2.f * slack), low = __fadd_rd(kth, -2.f * slack);
    uint32_t is_in = 0u, is_cand = 0u;  // a bit for each register
#pragma unroll
    for (int r = 0; r < kWarpRegs; ++r) {
        if (v[r] > above)
            is_in |= 1u << r;
        else if (v[r] >= low && 32 * r + lane < m)
            is_cand |= 1u << r;
    }
    const int need = k - __reduce_add_sync(0xffffffffu, __popc(is_in)), nc = __reduce_add_sync(0xffffffffu, __popc(is_cand));
    if (nc == need) {
        is_in |= is_cand;
    } else if (slack == 0.f) {
        // bounds or queries of zeros: the scores are exact, and the candidates' equal: by index
        int before = 0;
#pragma unroll
        for (int r = 0; r < kWarpRegs; ++r) {
            const uint32_t votes = __ballot_sync(0xffffffffu, (is_cand >> r) & 1u);
            if (((is_cand >> r) & 1u) && before + __popc(votes & ((1u << lane) - 1u)) < need) is_in |= 1u << r;
            before += __popc(votes);
        }
    } else {
        query_sums<double>(z, t, hk, sums[warp], lane, 32);
        int at = 0;
#pragma unroll
        for (int r = 0; r < kWarpRegs; ++r) {  // the candidates, by index
            const uint32_t votes = __ballot_sync(0xffffffffu, (is_cand >> r) & 1u);
            if ((is_cand >> r) & 1u) cand[warp][at + __popc(votes & ((1u << lane) - 1u))] = uint16_t(32 * r + lane);
            at += __popc(votes);
        }
        __syncwarp();
        for (int i = 0; i < nc; ++i) {
            const double s = exact_score(z, c.b, hk, first + cand[warp][i], sums[warp], lane);
            if (lane == 0) keys[warp][i] = ordered64(s);
        }
        __syncwarp();
        // a candidate's rank among them, noted in the place of its number
        for (int i = lane; i < nc; i += 32) {
            const unsigned long long mine = keys[warp][i];
            int rank = 0;
            for (int j = 0; j < nc; ++j) {
                const unsigned long long other = keys[warp][j];
                rank += other > mine || (other == mine && j < i);
            }
            if (rank >= need) cand[warp][i] = 0xffffu;
        }
        __syncwarp();
        at = 0;
#pragma unroll
        for (int r = 0; r < kWarpRegs; ++r) {
            const uint32_t votes = __ballot_sync(0xffffffffu, (is_cand >> r) & 1u);
            if (((is_cand >> r) & 1u) && cand[warp][at + __popc(votes & ((1u << lane) - 1u))] != 0xffffu) is_in |= 1u << r;
            at += __popc(votes);
        }
    }
    int done = z.n_first;  // the chosen ones, ascending
#pragma unroll
    for (int r = 0; r < kWarpRegs; ++r) {
        const bool in = (is_in >> r) & 1u;
        const uint32_t votes = __ballot_sync(0xffffffffu, in);
        const int to = done + __popc(votes & ((1u << lane) - 1u));
        if (in && to < z.n_first + k) out[to] = first + 32 * r + lane;
        done += __popc(votes);
    }
}

// The same by a CTA: scores in registers up to 8192 blocks, from memory beyond.
__global__ void __launch_bounds__(kSelThreads) jfa_cache_choose_kernel(const BlockParams z) {
    const CacheAppendParams& p = z.a;
    constexpr int kWarps = kSelThreads / 32;
    __shared__ int hist[256];
    __shared__ int cand[kExact];
    __shared__ unsigned long long keys[kExact];
    __shared__ double sums[2 * 128];
    __shared__ float ends[3][kWarps];
    __shared__ int parts[2][kWarps];
    __shared__ int found, left;
    __shared__ unsigned long long prefix;
    const int t = blockIdx.x, hk = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Chooser c = chooser(p, t, lane, threadIdx.x == 0);
    if (c.b < 0) return;
    int32_t* out = z.blocks + (size_t(t) * p.Hkv + hk) * size_t(z.n_blocks);
    const int n = c.own + 1;
    if (n <= z.n_blocks) {  // all that there are
        for (int i = threadIdx.x; i < z.n_blocks; i += kSelThreads) out[i] = i < n ? i : -1;
        return;
    }
    const int first = z.n_first, end = n - z.n_last, m = end - first, k = z.n_blocks - z.n_first - z.n_last;  // m > k
    for (int i = threadIdx.x; i < z.n_first; i += kSelThreads) out[i] = i;
    for (int i = threadIdx.x; i < z.n_last; i += kSelThreads) out[z.n_first + k + i] = end + i;
    if (k == 0) return;
    float* sc = z.scores + (size_t(t) * p.Hkv + hk) * size_t(p.max_pages) + first;
    const float* sl = z.slack + (size_t(t) * p.Hkv + hk) * size_t(z.chunks);
    // Warps hold neighbouring scores: warp w those from w * per on, `per` a multiple of 32.
    const bool held = m <= kHeld;
    const int per = (m + kSelThreads - 1) / kSelThreads * 32, from = warp * per, to = min(m, from + per);
    float v[kSelRegs], small = INFINITY, large = -INFINITY, slack = 0.f;
#pragma unroll
    for (int r = 0; r < kSelRegs; ++r) {
        const int i = from + 32 * r + lane;
        v[r] = -INFINITY;
        if (held && i < to) v[r] = sc[i] + 0.f;
    }
    // f(score, its number) for this thread's scores, in whole warps
    auto each = [&](auto&& f) {
        if (held) {
#pragma unroll
            for (int r = 0; r < kSelRegs; ++r)
                if (32 * r < per) f(v[r], from + 32 * r + lane);
        } else {
            for (int i0 = from; i0 < from + per; i0 += 32) f(i0 + lane < to ? sc[i0 + lane] + 0.f : -INFINITY, i0 + lane);
        }
    };
    each([&](float x, int i) {
        if (i < to) {
            small = fminf(small, x);
            large = fmaxf(large, x);
        }
    });
    for (int i = first / kChunk + threadIdx.x; i <= (end - 1) / kChunk; i += kSelThreads) slack = fmaxf(slack, sl[i]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        small = fminf(small, __shfl_xor_sync(0xffffffffu, small, d));
        large = fmaxf(large, __shfl_xor_sync(0xffffffffu, large, d));
        slack = fmaxf(slack, __shfl_xor_sync(0xffffffffu, slack, d));
    }
    if (lane == 0) {
        ends[0][warp] = small;
        ends[1][warp] = large;
        ends[2][warp] = slack;
    }
    if (threadIdx.x == 0) found = 0;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
        small = fminf(small, ends[0][w]);
        large = fmaxf(large, ends[1][w]);
        slack = fmaxf(slack, ends[2][w]);
    }
    int turn = 0;
    auto total = [&](int a) {  // over the CTA (two buffers: one synchronisation a sum)
        a = __reduce_add_sync(0xffffffffu, a);
        turn ^= 1;
        if (lane == 0) parts[turn][warp] = a;
        __syncthreads();
        return __reduce_add_sync(0xffffffffu, lane < kWarps ? parts[turn][lane] : 0);
    };
    auto count = [&](float x0) {
        int a = 0;
        each([&](float x, int) { a += x >= x0; });
        return total(a);
    };
    auto least = [&](float x0) {
        float a = INFINITY;
        each([&](float x, int) {
            if (x >= x0) a = fminf(a, x);
        });
        const uint32_t o = __reduce_min_sync(0xffffffffu, ordered(a));
        __syncthreads();
        if (lane == 0) ends[0][warp] = unordered(o);
        __syncthreads();
        a = ends[0][0];
        for (int w = 1; w < kWarps; ++w) a = fminf(a, ends[0][w]);
        return a;
    };
    const float kth = kth_largest(v, small, large, k, count, least);
    const float above = __fadd_ru(kth, 2.f * slack), low = __fadd_rd(kth, -2.f * slack);
    int sure = 0, maybe = 0;
    each([&](float x, int i) {
        if (x > above)
            ++sure;
        else if (x >= low && i < to)
            ++maybe;
    });
    const int need = k - total(sure), nc = total(maybe);
    // border: exact keys above it are in, and of equal ones those of lower numbers
    unsigned long long border = 0ull;
    int equal = 0;
    const bool all = nc == need, exact = !all && slack != 0.f, keep = exact && nc <= kExact;
    if (exact) {
        query_sums<double>(z, t, hk, sums, threadIdx.x, kSelThreads);
        __syncthreads();
    }
    auto is_cand = [&](float x, int i) { return i < to && x <= above && x >= low; };
    if (keep) {
        each([&](float x, int i) {
            if (is_cand(x, i)) cand[atomicAdd(&found, 1)] = i;
        });
        __syncthreads();
        for (int i = warp; i < nc; i += kWarps) {
            const double s = exact_score(z, c.b, hk, first + cand[i], sums, lane);
            if (lane == 0) keys[i] = ordered64(s);
        }
        __syncthreads();
        // the need-th of them: its key and number
        for (int i = threadIdx.x; i < nc; i += kSelThreads) {
            int rank = 0;
            for (int j = 0; j < nc; ++j) rank += keys[j] > keys[i] || (keys[j] == keys[i] && cand[j] < cand[i]);
            if (rank == need - 1) {
                prefix = keys[i];
                left = cand[i];
            }
        }
        __syncthreads();
        border = prefix;
        equal = left;
        for (int i = threadIdx.x; i < nc; i += kSelThreads)  // the chosen ones' numbers stay
            if (keys[i] < border || (keys[i] == border && cand[i] > equal)) cand[i] = -1;
        __syncthreads();
    } else if (exact) {
        // Very many nearly equal scores: the need-th largest exact score, eight bits at a time, each
        // pass scoring all candidates again.
        if (threadIdx.x == 0) {
            prefix = 0ull;
            left = need;
        }
        for (int shift = 56; shift >= 0; shift -= 8) {
            if (threadIdx.x < 256) hist[threadIdx.x] = 0;
            __syncthreads();
            const unsigned long long mask = shift == 56 ? 0ull : ~0ull << (shift + 8), want = prefix;
            each([&](float x, int i) {
                for (uint32_t todo = __ballot_sync(0xffffffffu, is_cand(x, i)); todo; todo &= todo - 1) {
                    const unsigned long long key = ordered64(exact_score(z, c.b, hk, first + i - lane + __ffs(todo) - 1, sums, lane));
                    if (lane == 0 && (key & mask) == want) atomicAdd(&hist[int((key >> shift) & 255u)], 1);
                }
            });
            __syncthreads();
            if (threadIdx.x == 0) {
                int higher = 0, d = 255;
                while (d > 0 && higher + hist[d] < left) higher += hist[d--];
                left -= higher;
                prefix |= (unsigned long long)(d) << shift;
            }
            __syncthreads();
        }
        border = prefix;
        equal = left;
    } else if (!all) {
        equal = need;  // (exact and equal: the first so many)
    }
    // The chosen ones, ascending: a warp's numbers come after those of the warps before it.
    // pass 0 counts, pass 1 writes; of candidates at the border (or equal ones) the first come first.
    const bool by_count = !all && !keep;  // `equal` counts candidates, over the warps in order
    int eq_before = 0, base = z.n_first;
    for (int pass = 0; pass < 3; ++pass) {
        // pass 0 (by_count only): candidates at the border before this warp
        if (pass == 0 && !by_count) continue;
        int mine = 0, eq = eq_before, at = base;
        each([&](float x, int i) {
            bool in = x > above, tie = false;
            const bool cd = is_cand(x, i);
            if (all) {
                in = in || cd;
            } else if (keep) {
                if (cd)
                    for (int j = 0; j < nc; ++j) in = in || cand[j] == i;
            } else if (exact) {
                for (uint32_t todo = __ballot_sync(0xffffffffu, cd); todo; todo &= todo - 1) {
                    const int l = __ffs(todo) - 1;
                    const unsigned long long key = ordered64(exact_score(z, c.b, hk, first + i - lane + l, sums, lane));
                    if (l == lane) {
                        in = key > border;
                        tie = key == border;
                    }
                }
            } else {
                tie = cd;
            }
            const uint32_t ties = __ballot_sync(0xffffffffu, tie);
            if (tie && pass > 0) in = eq + __popc(ties & ((1u << lane) - 1u)) < equal;
            eq += __popc(ties);
            if (pass == 0) return;
            const uint32_t votes = __ballot_sync(0xffffffffu, in);
            const int to_at = at + __popc(votes & ((1u << lane) - 1u));
            if (pass == 2 && in && to_at < z.n_first + k) out[to_at] = first + i;
            at += __popc(votes);
            mine += __popc(votes);
        });
        __syncthreads();
        turn ^= 1;
        if (lane == 0) parts[turn][warp] = pass == 0 ? eq : mine;
        __syncthreads();
        const int before = __reduce_add_sync(0xffffffffu, lane < warp ? parts[turn][lane] : 0);
        if (pass == 0) eq_before = before;
        if (pass == 1) base = z.n_first + before;
    }
}

int chunks_of(int32_t max_pages) { return std::max(1, (max_pages + kChunk - 1) / kChunk); }

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
    // a CTA for each token, or where there are many for a page's worth of them
    z.tile = T > 2048 || T >= 8 * int64_t(B) ? 1 << cache->page_log2 : 1;
    const int grid = int((T + z.tile - 1) / z.tile);
    if (cache->ops)
        jfa_cache_summarize_kernel<true><<<grid, kSumThreads, 0, st>>>(z);
    else
        jfa_cache_summarize_kernel<false><<<grid, kSumThreads, 0, st>>>(z);
    return cudaGetLastError() == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

size_t jfa_cache_select_workspace_size(jfa_cache cache, int64_t T, int32_t max_pages) {
    if (!cache || T < 0 || T > (1 << 30) || max_pages < 0) return 0;
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
    if (H / cache->Hkv > 128) return JFA_ERR_UNSUPPORTED;
    if (n_first < 0 || n_last < 1 || n_blocks < 1 || n_first > n_blocks - n_last ||
        (int64_t(n_blocks) << cache->page_log2) > (1 << 30))
        return JFA_ERR_INVALID_ARG;
    if (!bounds || !aligned(bounds, 16) || (T > 0 && (!row_ok(cache, Q, q_stride, H) || !blocks || !aligned(blocks, 4))))
        return JFA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < jfa_cache_select_workspace_size(cache, T, max_pages))
        return JFA_ERR_INVALID_ARG;
    if (chunks_of(max_pages) > 65535) return JFA_ERR_UNSUPPORTED;
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
        // many tokens a sequence (as far as the host knows): 32 of them share the bounds' reads
        const bool tiles = (max_q_len == 0 || max_q_len > 4) && T >= 8 * int64_t(B);
        cudaError_t e = cudaSuccess;
        if (tiles) {
            const dim3 grid((z.a.T + kTileTokens - 1) / kTileTokens, z.chunks, cache->Hkv);
            const int D = cache->D, bytes = kTileTokens * (2 * D + 4) * 4 + kChunk * (2 * D + 8) * 2;
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
    if (max_pages <= kWarpHeld)
        jfa_cache_choose_warp_kernel<<<int((T * cache->Hkv + kWarpItems - 1) / kWarpItems), 32 * kWarpItems, 0, st>>>(z);
    else
        jfa_cache_choose_kernel<<<dim3(z.a.T, cache->Hkv), kSelThreads, 0, st>>>(z);
    return cudaGetLastError() == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
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
    p.item_cost = kDecodeItemUnits;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = cache->ops ? launch_cache_decode4(cache->D, cache->mk, cache->mv, p, false, cache->num_sms, st)
                                     : launch_cache_decode_lists(cache->D, cache->mk, cache->mv, p, cache->num_sms, st);
    return e == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

}  // extern "C"
