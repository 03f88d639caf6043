// Attention over selected blocks of a paged cache: the blocks' bounds, the selection, and the
// attention call.  A block is a page.  Semantics are documented in include/jfa.h.
//
// The score of a block for a token and key head is the sum over the group's heads h of an upper
// bound of <q_h, k> over the block's keys,
//   sum_h sum_d max(q_hd lo_d, q_hd hi_d) = <u, hi> + <w, lo>,  u = sum_h max(q_h, 0), w = sum_h min(q_h, 0),
// with lo and hi the block's least and largest elements, so the group costs what one head does.
//
// The selection is that of exact arithmetic.  Scores are taken in fp32: u and w are sums of g values of
// one sign, and the dot product adds at most 64 products in a lane and joins four lanes, so a
// score is off by less than
//   slack = (g + 68) 2^-24 max|lo, hi| sum_d (u_d - w_d).
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

constexpr int kThreads = 128;
constexpr int kChunk = 64;          // blocks that a CTA scores
constexpr int kSelThreads = 256;
constexpr int kHeld = 8192;         // scores that the selection keeps in shared memory
constexpr int kExact = 256;         // candidates whose 64-bit scores it keeps

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

// The bounds of every page that got new tokens, over all its positions below kv_len.  The CTA of
// a page's first new token takes it; a thread takes eight elements of a head.
template <bool FOUR>
__global__ void __launch_bounds__(kThreads) jfa_cache_summarize_kernel(const BlockParams z) {
    const CacheAppendParams& p = z.a;
    const int t = blockIdx.x, lane = threadIdx.x & 31;
    const CachePlace at = cache_place(p, t, lane);
    if (at.b < 0) return;
    const int size = 1 << p.page_log2, slot = at.pos & (size - 1);
    if (at.page < 0) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
        return;
    }
    if (slot != 0 && t != p.q_off[at.b]) return;  // another token's page
    const int n = min(size, p.kv_lens[at.b] - (at.pos - slot));
    const int vecs = p.D / 8;
    for (int i = threadIdx.x; i < p.Hkv * vecs; i += kThreads) {
        const int h = i / vecs, v = i - h * vecs;
        uint4 lo = make_uint4(0x7f807f80u, 0x7f807f80u, 0x7f807f80u, 0x7f807f80u), hi = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
        auto take = [&](const uint4 x) {
            lo = make_uint4(min_bf16x2(lo.x, x.x), min_bf16x2(lo.y, x.y), min_bf16x2(lo.z, x.z), min_bf16x2(lo.w, x.w));
            hi = make_uint4(max_bf16x2(hi.x, x.x), max_bf16x2(hi.y, x.y), max_bf16x2(hi.z, x.z), max_bf16x2(hi.w, x.w));
        };
        if constexpr (FOUR) {
            const uint8_t* codes = static_cast<const uint8_t*>(p.Kc) + at.page * p.ks[0] + h * p.ks[2] + 4 * v;
            const uint8_t* scales = z.k_scales + at.page * z.kss[0] + h * z.kss[1] + (v >> 1);
#pragma unroll 8
            for (int j = 0; j < n; ++j) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + j * p.ks[1]);
                const float s = f16_to_float(e4m3_to_f16(scales[j * (p.D / 16)])).x;
                uint32_t e[4], o[4];
                e2m1_to_f16(w, e);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 x = f16_to_float(e[k]);
                    o[k] = pack_bf16x2(x.x * s, x.y * s);
                }
                take(make_uint4(o[0], o[1], o[2], o[3]));
            }
        } else {
            const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.Kc) + at.page * p.ks[0] + h * p.ks[2] + 8 * v;
#pragma unroll 8
            for (int j = 0; j < n; ++j) take(*reinterpret_cast<const uint4*>(k + j * p.ks[1]));
        }
        __nv_bfloat16* dst = z.bounds + (size_t(at.page) * p.Hkv + h) * 2 * p.D + 8 * v;
        *reinterpret_cast<uint4*>(dst) = lo;
        *reinterpret_cast<uint4*>(dst + p.D) = hi;
    }
}

// A token of a selection: its sequence and own block, or b < 0.  A row before its sequence's first
// position sees nothing (own = -1).
struct Chooser {
    int b, own;
};
__device__ __forceinline__ Chooser chooser(const CacheAppendParams& p, int t, int lane) {
    Chooser c{find_sequence(p.q_off, p.B, t, lane), -1};
    if (c.b >= p.B) c.b = -1;
    if (c.b < 0) return c;
    const int q0 = p.q_off[c.b], q1 = p.q_off[c.b + 1], kv = p.kv_lens[c.b];
    if (q0 < 0 || q1 > p.T || t < q0 || t >= q1 || kv < 0 || kv > p.max_kv) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
        c.b = -1;
        return c;
    }
    const int pos = kv - q1 + t;
    if (pos >= 0) c.own = pos >> p.page_log2;
    return c;
}

// u and w of a token and key head into sums [2 D] (lo's factors w, then hi's u), by the whole CTA.
template <typename F>
__device__ __forceinline__ void query_sums(const BlockParams& z, int t, int hk, F* sums) {
    const int D = z.a.D;
    for (int d = threadIdx.x; d < D; d += blockDim.x) {
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

// Page of block k of sequence b, or -1.
__device__ __forceinline__ int block_page(const CacheAppendParams& p, int b, int k) {
    const int page = p.table[size_t(b) * size_t(p.max_pages) + size_t(k)];
    return page >= 0 && page < p.n_pages ? page : -1;
}

// Scores of kChunk blocks for one token and key head: four lanes a block.
template <int D>
__global__ void __launch_bounds__(kThreads) jfa_cache_score_kernel(const BlockParams z) {
    const CacheAppendParams& p = z.a;
    const int t = blockIdx.x, hk = blockIdx.z, lane = threadIdx.x & 31;
    const Chooser c = chooser(p, t, lane);
    const int first = z.n_first, end = c.own + 1 - z.n_last, k0 = blockIdx.y * kChunk;  // the blocks that compete
    if (c.b < 0 || c.own + 1 <= z.n_blocks || k0 >= end) return;
    __shared__ __align__(16) float sums[2 * D];
    __shared__ float red[kThreads / 32];
    query_sums<float>(z, t, hk, sums);
    __syncthreads();
    const int part = threadIdx.x & 3;
    float norm = 0.f;
    float f[D / 2];
#pragma unroll
    for (int v = 0; v < D / 16; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[8 * v + i] = sums[8 * (4 * v + part) + i];
            norm += fabsf(f[8 * v + i]);
        }
    norm += __shfl_xor_sync(0xffffffffu, norm, 1);
    norm += __shfl_xor_sync(0xffffffffu, norm, 2);
    uint32_t top = 0u;  // the largest magnitudes
    float* out = z.scores + (size_t(t) * p.Hkv + hk) * size_t(p.max_pages);
#pragma unroll 1
    for (int i = threadIdx.x >> 2; i < kChunk; i += kThreads / 4) {
        const int k = k0 + i;
        const bool in = k >= first && k < end;
        float s = 0.f;
        if (in) {
            const int page = block_page(p, c.b, k);
            if (page < 0) {
                atomicOr(p.status, kStatusBounds);
            } else {
                const uint4* src = reinterpret_cast<const uint4*>(z.bounds + (size_t(page) * p.Hkv + hk) * 2 * D) + part;
#pragma unroll
                for (int v = 0; v < D / 16; ++v) {
                    const uint4 x = src[4 * v];
                    const uint32_t r[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        top = max_bf16x2(top, r[j] & 0x7fff7fffu);
                        s = fmaf(__uint_as_float(r[j] << 16), f[8 * v + 2 * j], s);
                        s = fmaf(__uint_as_float(r[j] & 0xffff0000u), f[8 * v + 2 * j + 1], s);
                    }
                }
            }
        }
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        if (in && part == 0) out[k] = s;
    }
    float m = fmaxf(__uint_as_float(top << 16), __uint_as_float(top & 0xffff0000u));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) m = fmaxf(m, red[w]);
        z.slack[(size_t(t) * p.Hkv + hk) * size_t(z.chunks) + blockIdx.y] = float(z.g + 68) * (1.01f * 0x1p-24f) * m * norm;
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

// The chosen blocks of one token and key head, from its scores.
__global__ void __launch_bounds__(kSelThreads) jfa_cache_choose_kernel(const BlockParams z) {
    const CacheAppendParams& p = z.a;
    const int t = blockIdx.x, hk = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kWarps = kSelThreads / 32;
    const Chooser c = chooser(p, t, lane);
    if (c.b < 0) return;
    int32_t* out = z.blocks + (size_t(t) * p.Hkv + hk) * size_t(z.n_blocks);
    const int n = c.own + 1;
    if (n <= z.n_blocks) {  // all that there are
        for (int i = threadIdx.x; i < z.n_blocks; i += kSelThreads) out[i] = i < n ? i : -1;
        return;
    }
    extern __shared__ float held[];
    __shared__ int hist[256];
    __shared__ uint32_t prefix;
    __shared__ int left, count, found;
    __shared__ float slack;
    __shared__ int cand[kExact];
    __shared__ double cand_s[kExact];
    __shared__ double sums[2 * 128];
    __shared__ int warp_n[kWarps];
    const int first = z.n_first, end = n - z.n_last, m = end - first, k = z.n_blocks - z.n_first - z.n_last;  // m > k
    float* sc = z.scores + (size_t(t) * p.Hkv + hk) * size_t(p.max_pages) + first;
    if (m <= kHeld) {
        for (int i = threadIdx.x; i < m; i += kSelThreads) held[i] = sc[i];
        sc = held;
    }
    float cut = INFINITY;  // blocks scored above it are chosen,
    bool at_cut = false;   // and those at it
    if (k > 0) {
        // the k-th largest fp32 score, eight bits at a time
        if (threadIdx.x == 0) {
            prefix = 0u;
            left = k;
        }
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (threadIdx.x < 256) hist[threadIdx.x] = 0;
            __syncthreads();
            const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8), want = prefix;
            for (int i = threadIdx.x; i < m; i += kSelThreads) {
                const uint32_t key = ordered(sc[i]);
                if ((key & mask) == want) atomicAdd(&hist[(key >> shift) & 255u], 1);
            }
            __syncthreads();
            if (warp == 0) {  // the digit in which the k-th lies, from the top
                int mine[8], sum = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum += mine[j] = hist[255 - (8 * lane + j)];
                int above = warp_scan(sum, lane) - sum;
                const int need = left;
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (above < need && above + mine[j] >= need) {
                        prefix = want | (uint32_t(255 - (8 * lane + j)) << shift);
                        left = need - above;
                    }
                    above += mine[j];
                }
            }
            __syncthreads();
        }
        const float kth = unordered(prefix);
        if (warp == 0) {
            const float* sl = z.slack + (size_t(t) * p.Hkv + hk) * size_t(z.chunks);
            float x = 0.f;
            for (int i = first / kChunk + lane; i <= (end - 1) / kChunk; i += 32) x = fmaxf(x, sl[i]);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            if (lane == 0) {
                slack = 2.f * x;
                count = found = 0;
            }
        }
        __syncthreads();
        // (rounding the limits outwards only moves a block to the candidates)
        const float top = __fadd_ru(kth, slack), low = __fadd_rd(kth, -slack);
        int sure = 0;
        for (int i = threadIdx.x; i < m; i += kSelThreads) {
            const float s = sc[i];
            if (s > top) {
                ++sure;
            } else if (s >= low) {
                const int at = atomicAdd(&found, 1);
                if (at < kExact) cand[at] = i;
            }
        }
        sure = __reduce_add_sync(0xffffffffu, sure);
        if (lane == 0) atomicAdd(&count, sure);
        query_sums<double>(z, t, hk, sums);
        __syncthreads();
        const int need = k - count, nc = found;
        cut = top;
        if (nc == need) {
            cut = low;  // all of them
            at_cut = true;
        } else if (nc <= kExact) {
            for (int i = warp; i < nc; i += kWarps) {
                const double s = exact_score(z, c.b, hk, first + cand[i], sums, lane);
                if (lane == 0) cand_s[i] = s;
            }
            __syncthreads();
            for (int i = threadIdx.x; i < nc; i += kSelThreads) {
                int rank = 0;
                for (int j = 0; j < nc; ++j) rank += cand_s[j] > cand_s[i] || (cand_s[j] == cand_s[i] && cand[j] < cand[i]);
                sc[cand[i]] = rank < need ? INFINITY : -INFINITY;
            }
            __syncthreads();
        } else {
            // Very many nearly equal scores: the need-th largest exact score, eight bits at a
            // time, each pass scoring all candidates again; then equal ones by their index.
            __shared__ unsigned long long prefix64;
            if (threadIdx.x == 0) {
                prefix64 = 0ull;
                left = need;
            }
            auto key64 = [&](int i) {
                const unsigned long long b = __double_as_longlong(exact_score(z, c.b, hk, first + i, sums, lane) + 0.0);
                return b >> 63 ? ~b : b | (1ull << 63);
            };
            for (int shift = 56; shift >= 0; shift -= 8) {
                hist[threadIdx.x] = 0;
                __syncthreads();
                const unsigned long long mask = shift == 56 ? 0ull : ~0ull << (shift + 8), want = prefix64;
                for (int i = warp; i < m; i += kWarps) {
                    if (!(sc[i] <= top && sc[i] >= low)) continue;
                    const unsigned long long key = key64(i);
                    if (lane == 0 && (key & mask) == want) atomicAdd(&hist[int((key >> shift) & 255u)], 1);
                }
                __syncthreads();
                if (threadIdx.x == 0) {
                    int above = 0, d = 255;
                    while (d > 0 && above + hist[d] < left) above += hist[d--];
                    left -= above;
                    prefix64 |= (unsigned long long)(d) << shift;
                }
                __syncthreads();
            }
            const unsigned long long border = prefix64;
            int equal = left;  // of those at the border, the first so many
            for (int base = 0; base < m; base += kWarps) {
                const int i = base + warp;
                const bool is = i < m && sc[i] <= top && sc[i] >= low;
                const unsigned long long key = is ? key64(i) : 0ull;
                __syncthreads();
                if (lane == 0) warp_n[warp] = is && key == border;
                __syncthreads();
                int before = 0, all = 0;
                for (int w = 0; w < kWarps; ++w) {
                    before += w < warp ? warp_n[w] : 0;
                    all += warp_n[w];
                }
                if (is && lane == 0) sc[i] = key > border || (key == border && before < equal) ? INFINITY : -INFINITY;
                equal -= all;
            }
            __syncthreads();
        }
    }
    // the chosen ones, ascending
    for (int i = threadIdx.x; i < z.n_first; i += kSelThreads) out[i] = i;
    for (int i = threadIdx.x; i < z.n_last; i += kSelThreads) out[z.n_first + k + i] = end + i;
    int done = z.n_first;
    for (int base = 0; base < m && k > 0; base += kSelThreads) {
        const int i = base + threadIdx.x;
        const bool in = i < m && (sc[i] > cut || (at_cut && sc[i] == cut));
        const uint32_t votes = __ballot_sync(0xffffffffu, in);
        __syncthreads();
        if (lane == 0) warp_n[warp] = __popc(votes);
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            before += w < warp ? warp_n[w] : 0;
            all += warp_n[w];
        }
        const int to = done + before + __popc(votes & ((1u << lane) - 1u));
        if (in && to < z.n_first + k) out[to] = first + i;
        done += all;
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
    if (cache->ops)
        jfa_cache_summarize_kernel<true><<<z.a.T, kThreads, 0, st>>>(z);
    else
        jfa_cache_summarize_kernel<false><<<z.a.T, kThreads, 0, st>>>(z);
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
        const dim3 grid(z.a.T, z.chunks, cache->Hkv);
        if (cache->D == 128)
            jfa_cache_score_kernel<128><<<grid, kThreads, 0, st>>>(z);
        else
            jfa_cache_score_kernel<64><<<grid, kThreads, 0, st>>>(z);
        if (cudaGetLastError() != cudaSuccess) return JFA_ERR_CUDA;
    }
    const int bytes = std::min(max_pages, kHeld) * 4;
    jfa_cache_choose_kernel<<<dim3(z.a.T, cache->Hkv), kSelThreads, bytes, st>>>(z);
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
