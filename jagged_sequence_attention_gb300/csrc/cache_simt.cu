// Paged-cache attention for few rows, fp32: plain fp32 arithmetic on the CUDA cores.
//
// Single tokens and short query sets are a stream of K and V.  A CTA of four warps, three to an
// SM, streams an item's keys 64 at a time through two buffers of shared memory, copied there 16
// bytes at a time (cp.async) by pages.  A warp owns its rows from scores to output, so the
// softmax needs no exchange between warps: for scores a lane takes two keys, for P V two
// columns (one at head_dim 32).
// Every warp reads the whole tile from shared memory, so the arithmetic grows with the rows and
// the reads do not: with at most four grouped heads an item holds four rows, one a warp, with
// more sixteen (a single token of two heads over 64 histories of 1k-8k keys: 170 us with
// sixteen rows, 111 us with four).
#include "cache_common.cuh"
#include "tilemath.cuh"

namespace jfa {

namespace {

constexpr int kSimtBN = 64, kSimtThreads = 128, kSimtCtasPerSm = 3;

template <int D, int BM>
struct SimtCfg {
    static constexpr int RT = BM / 4;  // rows of a warp
    // floats per staged key row: 16-byte reads of 8 consecutive rows cover all banks
    static constexpr int kStride = D + 4;
    static constexpr int kQ = 0, kK = kQ + BM * kStride, kV = kK + 2 * kSimtBN * kStride;
    static constexpr int kP = kV + 2 * kSimtBN * D, kFloats = kP + BM * kSimtBN;
    static constexpr int kBytes = kFloats * 4;
    static constexpr int kPart = BM * (D + 2);  // floats of a partial result: O, m, l
};

__device__ __forceinline__ void cp16(float* dst, const float* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, int BM, bool BIAS>
__global__ void __launch_bounds__(kSimtThreads, kSimtCtasPerSm) jfa_cache_simt_kernel(const CacheFwdParams p) {
    using C = SimtCfg<D, BM>;
    constexpr int BN = kSimtBN, RT = C::RT, LC = D / 32;  // LC: output columns of a lane
    extern __shared__ __align__(16) float sm[];
    __shared__ int last_flag;
    float* sQ = sm + C::kQ;
    float* sP = sm + C::kP;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const CacheStart start = cache_start<BN>(p, reinterpret_cast<int*>(sm));
    CacheCursor<BN> cur(p, start);
    CacheSeg g;
    const int page_mask = (1 << p.page_log2) - 1;
    while (cur.next(p, g)) {
        const int R = g.s.q_len * p.g, diag = g.s.kv_len - g.s.q_len, r0 = g.tile * BM;
        // 64 rows of K or V from position c0 on, zeros where no row of the item may look
        auto load = [&](float* dst, int stride, const void* base, const int64_t* s, int c0) {
            constexpr int kPieces = D / 4, kStep = kSimtThreads / kPieces;
            const int c = threadIdx.x % kPieces;
#pragma unroll 4
            for (int r = threadIdx.x / kPieces; r < BN; r += kStep) {
                const int j = c0 + r;
                const float* src = static_cast<const float*>(base);
                bool in = j >= g.r.lo && j < g.r.hi;
                if (in) {
                    const int page = p.table[size_t(g.b) * size_t(p.max_pages) + size_t(j >> p.page_log2)];
                    in = page >= 0 && page < p.n_pages;
                    if (in)
                        src += page * s[0] + (j & page_mask) * s[1] + g.hk * s[2] + 4 * c;
                    else if (c == 0)
                        atomicOr(p.status, kStatusBounds);
                }
                cp16(dst + r * stride + 4 * c, src, in);
            }
        };
        auto load_tile = [&](int kt) {
            const int c0 = (g.r.f + kt) * BN;
            load(sm + C::kK + (kt & 1) * BN * C::kStride, C::kStride, p.K, p.ks, c0);
            load(sm + C::kV + (kt & 1) * BN * D, D, p.V, p.vs, c0);
            cp_commit();
        };
        const int k_end = g.r.n > 0 ? g.k1 : g.k0;
        __syncthreads();  // the previous item's last reads
        if (g.k0 < k_end) load_tile(g.k0);
        for (int e = threadIdx.x; e < BM * D / 4; e += kSimtThreads) {
            const int tr = e / (D / 4), c = e % (D / 4), r = r0 + tr;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < R) {
                const int tok = div_g(p, r);
                v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.Q) + (g.s.q0 + tok) * p.q_stride +
                                                     int64_t(g.hk * p.g + r - tok * p.g) * D + 4 * c);
                v = make_float4(v.x * p.scale_log2, v.y * p.scale_log2, v.z * p.scale_log2, v.w * p.scale_log2);
            }
            *reinterpret_cast<float4*>(sQ + tr * C::kStride + 4 * c) = v;
        }
        float m[RT], l[RT];
        float2 o[RT];                // columns LC lane and on
        int rel[RT];                 // position of each row (rows past the end repeat the last one's)
        const float* brow[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int r = min(r0 + warp * RT + i, R - 1), tok = div_g(p, r);
            rel[i] = tok + diag;
            brow[i] = BIAS ? p.bias + (g.hk * p.g + r - tok * p.g) * 32 : nullptr;
            m[i] = -INFINITY;
            l[i] = 0.f;
            o[i] = make_float2(0.f, 0.f);
        }
        const int t_first = div_g(p, r0) + diag, t_last = div_g(p, min(R, r0 + BM) - 1) + diag;
        const int all_hi = p.causal ? min(g.s.kv_len, t_first + 1) : g.s.kv_len;
        const int all_lo = p.window >= 0 ? max(0, t_last - p.window) : 0;
        const bool rows = r0 + warp * RT < R;  // a warp without rows only loads and keeps step
        for (int kt = g.k0; kt < k_end; ++kt) {
            const int c0 = (g.r.f + kt) * BN;
            const float* sK = sm + C::kK + (kt & 1) * BN * C::kStride;
            const float* sV = sm + C::kV + (kt & 1) * BN * D;
            // the next tile's loads go out before this tile is waited for
            if (kt > g.k0) __syncthreads();  // the other buffers have been read
            if (kt + 1 < k_end) {
                load_tile(kt + 1);
                cp_wait<1>();
            } else {
                cp_wait<0>();
            }
            __syncthreads();
            if (!rows) continue;
            float x[RT][2];
#pragma unroll
            for (int i = 0; i < RT; ++i) x[i][0] = x[i][1] = 0.f;
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 kk[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) kk[j] = *reinterpret_cast<const float4*>(sK + (lane + 32 * j) * C::kStride + d);
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const float4 q = *reinterpret_cast<const float4*>(sQ + (warp * RT + i) * C::kStride + d);
#pragma unroll
                    for (int j = 0; j < 2; ++j) x[i][j] = fmaf(q.x, kk[j].x, x[i][j]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) x[i][j] = fmaf(q.y, kk[j].y, x[i][j]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) x[i][j] = fmaf(q.z, kk[j].z, x[i][j]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) x[i][j] = fmaf(q.w, kk[j].w, x[i][j]);
                }
            }
            const bool masked = c0 < all_lo || c0 + BN > all_hi;
            const int bk = BIAS ? relpos_bucket(t_last - c0) : 0;
            const int near = t_first - c0 - (BN - 1);
            const bool one = BIAS && (near >= 0 || t_last <= c0) && bk == relpos_bucket(near);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const float b1 = BIAS && one ? __ldg(brow[i] + bk) * 1.4426950408889634f : 0.f;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int key = c0 + lane + 32 * j;
                    if (BIAS) x[i][j] += one ? b1 : __ldg(brow[i] + relpos_bucket(rel[i] - key)) * 1.4426950408889634f;
                    if (masked) {
                        const bool in = key < g.s.kv_len && (!p.causal || key <= rel[i]) &&
                                        (p.window < 0 || key >= rel[i] - p.window);
                        x[i][j] = in ? x[i][j] : -INFINITY;
                    }
                }
                float mx = fmaxf(x[i][0], x[i][1]);
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
                const float m_new = fmaxf(m[i], mx);
                const float m_use = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = ex2_approx(m[i] - m_use);
                m[i] = m_new;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float e = ex2_approx(x[i][j] - m_use);
                    sP[(warp * RT + i) * BN + lane + 32 * j] = e;
                    sum += e;
                }
                l[i] = fmaf(l[i], alpha, sum);  // this lane's keys; summed over the lanes at the end
                o[i] = mul2(o[i], make_float2(alpha, alpha));
            }
            __syncwarp();
#pragma unroll 4
            for (int j = 0; j < BN; j += 4) {
                float4 e[RT];
#pragma unroll
                for (int i = 0; i < RT; ++i) e[i] = *reinterpret_cast<const float4*>(sP + (warp * RT + i) * BN + j);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float2 v;
                    if constexpr (LC == 2)
                        v = *reinterpret_cast<const float2*>(sV + (j + q) * D + 2 * lane);
                    else
                        v = make_float2(sV[(j + q) * D + lane], 0.f);
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const float w = q == 0 ? e[i].x : q == 1 ? e[i].y : q == 2 ? e[i].z : e[i].w;
                        o[i] = fma2(make_float2(w, w), v, o[i]);
                    }
                }
            }
            __syncwarp();
        }
        // a row's columns, to dst (times mul)
        auto put = [&](float* dst, const float2& v, float mul) {
            if constexpr (LC == 2)
                *reinterpret_cast<float2*>(dst + 2 * lane) = make_float2(v.x * mul, v.y * mul);
            else
                dst[lane] = v.x * mul;
        };
        auto finish = [&](int r, float mm, float ll, const float2& v) {
            const int tok = div_g(p, r);
            const size_t row = size_t(g.s.q0 + tok) * size_t(p.H) + size_t(g.hk * p.g + r - tok * p.g);
            put(static_cast<float*>(p.O) + row * D, v, ll > 0.f ? 1.f / ll : 0.f);
            if (p.lse && lane == 0) p.lse[row] = ll > 0.f ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
        };
        const bool whole = g.whole();
        const int first = whole ? 0 : cache_first_cta(p, start, g), last = whole ? 0 : cache_last_cta(p, start, g);
        float* mine = p.part + size_t(cache_slot(blockIdx.x, first)) * C::kPart;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int tr = warp * RT + i;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], s);
            if (r0 + tr >= R) continue;  // (uniform in the warp)
            if (whole) {
                finish(r0 + tr, m[i], l[i], o[i]);
                continue;
            }
            put(mine + tr * D, o[i], 1.f);
            if (lane == 0) {
                mine[BM * D + tr] = m[i];
                mine[BM * D + BM + tr] = l[i];
            }
        }
        if (whole) continue;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
            last_flag = atomicAdd(p.counters + kCtrSplit + first, 1u) == uint32_t(last - first);
            if (last_flag) p.counters[kCtrSplit + first] = 0u;  // every part has arrived: ready for the next call
            __threadfence();
        }
        __syncthreads();
        if (!last_flag) continue;
        // The last part to arrive adds them up, in the order of the keys: a warp takes a row, its
        // lanes the parts' maxima and sums and then LC columns each.
        const int parts = last - first + 1, nr = min(BM, R - r0);
        auto part_of = [&](int c) { return p.part + size_t(cache_slot(first + c, first)) * C::kPart; };
        for (int tr = warp; tr < nr; tr += 4) {
            float mm = -INFINITY, ll = 0.f;
            float2 v = make_float2(0.f, 0.f);
            for (int c = lane; c < parts; c += 32) mm = fmaxf(mm, __ldcg(part_of(c) + BM * D + tr));
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, s));
            for (int c0 = 0; c0 < parts; c0 += 32) {
                const bool in = c0 + lane < parts;
                const float mc = in ? __ldcg(part_of(c0 + lane) + BM * D + tr) : -INFINITY;
                const float w = mc == -INFINITY ? 0.f : ex2_approx(mc - mm);
                if (in) ll = fmaf(__ldcg(part_of(c0 + lane) + BM * D + BM + tr), w, ll);
#pragma unroll 8
                for (int c = 0; c < min(32, parts - c0); ++c) {
                    const float wc = __shfl_sync(0xffffffffu, w, c);
                    const float* src = part_of(c0 + c) + tr * D + LC * lane;
                    const float2 u = LC == 2 ? __ldcg(reinterpret_cast<const float2*>(src)) : make_float2(__ldcg(src), 0.f);
                    v = fma2(u, make_float2(wc, wc), v);
                }
            }
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, s);
            finish(r0 + tr, mm, ll, v);
        }
    }
    wait_previous();
}

template <int D, int BM, bool BIAS>
cudaError_t launch(const CacheFwdParams& p, bool early, int num_sms, cudaStream_t st) {
    using C = SimtCfg<D, BM>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(jfa_cache_simt_kernel<D, BM, BIAS>, C::kBytes, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms * kSimtCtasPerSm);
    cfg.blockDim = dim3(kSimtThreads);
    cfg.dynamicSmemBytes = C::kBytes;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, jfa_cache_simt_kernel<D, BM, BIAS>, p);
}

template <int D, int BM>
cudaError_t launch_b(const CacheFwdParams& p, bool early, int num_sms, cudaStream_t st) {
    return p.bias ? launch<D, BM, true>(p, early, num_sms, st) : launch<D, BM, false>(p, early, num_sms, st);
}

}  // namespace

size_t cache_simt_part_bytes(int D, int num_sms) { return size_t(num_sms) * kSimtCtasPerSm * 2 * 16 * size_t(D + 2) * 4; }

cudaError_t launch_cache_simt(int D, const CacheFwdParams& p, bool early, int num_sms, cudaStream_t st) {
    if (D == 32) return p.bm == 4 ? launch_b<32, 4>(p, early, num_sms, st) : launch_b<32, 16>(p, early, num_sms, st);
    return p.bm == 4 ? launch_b<64, 4>(p, early, num_sms, st) : launch_b<64, 16>(p, early, num_sms, st);
}

}  // namespace jfa
