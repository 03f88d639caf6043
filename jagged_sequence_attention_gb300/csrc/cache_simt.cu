// Paged-cache attention on the CUDA cores (plain fp32 arithmetic on float inputs).
//
// A CTA of four warps takes 16 packed rows of an item and streams its keys 64 at a time
// through shared memory; warp w owns rows 4w .. 4w+3 from scores to output, so the softmax
// needs no exchange between warps.  Scores: a lane takes two keys and four rows; P V: a lane
// takes D / 32 columns and four rows.
#include "cache_common.cuh"

namespace jfa {

namespace {

constexpr int kSimtBM = 16, kSimtBN = 64, kSimtThreads = 128, kSimtCtasPerSm = 2;

template <int D>
struct SimtCfg {
    static constexpr int kStride = D + 4;  // floats per staged key row: 16-byte reads of 8 rows cover all banks
    static constexpr int kQ = 0, kK = kQ + kSimtBM * D, kV = kK + kSimtBN * kStride, kP = kV + kSimtBN * D;
    static constexpr int kFloats = kP + kSimtBM * kSimtBN;
    static constexpr int kBytes = kFloats * 4;
    static constexpr int kPart = kSimtBM * (D + 2);  // floats of a partial result: O, m, l
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ int rel_bucket(int r) {
    r = abs(r);
    const int rc = min(r, 46339);
    return r >= 46340 ? 31 : 31 - __clz(int(uint32_t(rc + 1) * uint32_t(rc + 1)));
}

template <int D, typename T>
__global__ void __launch_bounds__(kSimtThreads) jfa_cache_simt_kernel(const CacheFwdParams p) {
    using C = SimtCfg<D>;
    constexpr int BM = kSimtBM, BN = kSimtBN, NC = D / 32;
    extern __shared__ __align__(16) float sm[];
    __shared__ CacheStart start;
    __shared__ int last_flag;
    float* sQ = sm + C::kQ;
    float* sK = sm + C::kK;
    float* sV = sm + C::kV;
    float* sP = sm + C::kP;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    cache_start<BM, BN>(p, &start, reinterpret_cast<long long*>(sm));
    CacheCursor<BM, BN> cur(start);
    CacheSeg g;
    const int page_mask = (1 << p.page_log2) - 1;
    while (cur.next(p, g)) {
        const int R = g.s.q_len * p.g, diag = g.s.kv_len - g.s.q_len;
        __syncthreads();
        for (int e = threadIdx.x; e < BM * D; e += kSimtThreads) {
            const int r = g.tile * BM + e / D;
            float v = 0.f;
            if (r < R)
                v = to_f<T>(static_cast<const T*>(p.Q)[(g.s.q0 + r / p.g) * p.q_stride +
                                                       int64_t(g.hk * p.g + r % p.g) * D + e % D]);
            sQ[e] = v;
        }
        // rows 4 warp + i: their limits and heads
        int lim[4], low[4], head[4], tok[4];
        float m[4], l[4], o[4][NC];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = g.tile * BM + 4 * warp + i;
            tok[i] = r / p.g;
            head[i] = r < R ? g.hk * p.g + r % p.g : 0;
            const int at = tok[i] + diag;
            lim[i] = r < R ? (p.causal ? min(g.s.kv_len, at + 1) : g.s.kv_len) : 0;
            low[i] = p.window >= 0 ? at - p.window : 0;
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c) o[i][c] = 0.f;
        }
        const int k_end = g.r.n > 0 ? g.k1 : g.k0;
        for (int kt = g.k0; kt < k_end; ++kt) {
            const int c0 = (g.r.f + kt) * BN;
            __syncthreads();
            for (int e = threadIdx.x; e < BN * D; e += kSimtThreads) {
                const int j = c0 + e / D, d = e % D;
                float kx = 0.f, vx = 0.f;
                if (j >= g.r.lo && j < g.r.hi) {
                    const int page = p.table[size_t(g.b) * size_t(p.max_pages) + size_t(j >> p.page_log2)];
                    if (page >= 0 && page < p.n_pages) {
                        const int slot = j & page_mask;
                        kx = to_f<T>(static_cast<const T*>(p.K)[page * p.ks[0] + slot * p.ks[1] + g.hk * p.ks[2] + d]);
                        vx = to_f<T>(static_cast<const T*>(p.V)[page * p.vs[0] + slot * p.vs[1] + g.hk * p.vs[2] + d]);
                    } else if (d == 0) {
                        atomicOr(p.status, kStatusBounds);
                    }
                }
                sK[(e / D) * C::kStride + d] = kx;
                sV[e] = vx;
            }
            __syncthreads();
            float x[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i][0] = x[i][1] = 0.f;
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 kk[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) kk[c] = *reinterpret_cast<const float4*>(sK + (lane + 32 * c) * C::kStride + d);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 q = *reinterpret_cast<const float4*>(sQ + (4 * warp + i) * D + d);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        x[i][c] = fmaf(q.x, kk[c].x, x[i][c]);
                        x[i][c] = fmaf(q.y, kk[c].y, x[i][c]);
                        x[i][c] = fmaf(q.z, kk[c].z, x[i][c]);
                        x[i][c] = fmaf(q.w, kk[c].w, x[i][c]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int j = c0 + lane + 32 * c;
                    float y = x[i][c] * p.scale_log2;
                    if (p.bias) y += p.bias[head[i] * 32 + rel_bucket(tok[i] + diag - j)] * 1.4426950408889634f;
                    x[i][c] = j < lim[i] && j >= low[i] ? y : -INFINITY;
                    mx = fmaxf(mx, x[i][c]);
                }
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
                const float m_new = fmaxf(m[i], mx);
                const float m_use = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = exp2f(m[i] - m_use);
                m[i] = m_new;
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float e = exp2f(x[i][c] - m_use);
                    sP[(4 * warp + i) * BN + lane + 32 * c] = e;
                    sum += e;
                }
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
                l[i] = l[i] * alpha + sum;
#pragma unroll
                for (int c = 0; c < NC; ++c) o[i][c] *= alpha;
            }
            __syncwarp();
#pragma unroll 2
            for (int j = 0; j < BN; j += 4) {
                float4 e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = *reinterpret_cast<const float4*>(sP + (4 * warp + i) * BN + j);
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const float v = sV[(j + q) * D + lane + 32 * c];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[i][c] = fmaf(q == 0 ? e[i].x : q == 1 ? e[i].y : q == 2 ? e[i].z : e[i].w, v, o[i][c]);
                    }
            }
        }
        // Row i of this warp, written out: O / l and lse.
        auto finish = [&](int i, float mm, float ll, const float (&v)[NC]) {
            const int r = g.tile * BM + 4 * warp + i;
            if (r >= R) return;
            const size_t row = size_t(g.s.q0 + r / p.g) * size_t(p.H) + size_t(g.hk * p.g + r % p.g);
            const float inv = ll > 0.f ? 1.f / ll : 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (p.o_f32)
                    static_cast<float*>(p.O)[row * D + lane + 32 * c] = v[c] * inv;
                else
                    static_cast<__nv_bfloat16*>(p.O)[row * D + lane + 32 * c] = __float2bfloat16(v[c] * inv);
            }
            if (p.lse && lane == 0) p.lse[row] = ll > 0.f ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
        };
        if (g.whole()) {
#pragma unroll
            for (int i = 0; i < 4; ++i) finish(i, m[i], l[i], o[i]);
            continue;
        }
        const int first = cache_cta_of(start, g.first), last = cache_cta_of(start, g.first + g.units - 1);
        float* mine = p.part + size_t(cache_slot(blockIdx.x, first)) * C::kPart;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * warp + i;
#pragma unroll
            for (int c = 0; c < NC; ++c) mine[r * D + lane + 32 * c] = o[i][c];
            if (lane == 0) {
                mine[BM * D + r] = m[i];
                mine[BM * D + BM + r] = l[i];
            }
        }
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
            last_flag = atomicAdd(p.counters + first, 1u) == uint32_t(last - first);
            if (last_flag) p.counters[first] = 0u;  // every part has arrived: ready for the next call
            __threadfence();
        }
        __syncthreads();
        if (!last_flag) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * warp + i;
            float mm = -INFINITY;
            for (int c = first; c <= last; ++c)
                mm = fmaxf(mm, __ldcg(p.part + size_t(cache_slot(c, first)) * C::kPart + BM * D + r));
            const float mu = mm == -INFINITY ? 0.f : mm;
            float ll = 0.f, v[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) v[c] = 0.f;
            for (int c = first; c <= last; ++c) {
                const float* part = p.part + size_t(cache_slot(c, first)) * C::kPart;
                const float w = exp2f(__ldcg(part + BM * D + r) - mu);
                ll = fmaf(__ldcg(part + BM * D + BM + r), w, ll);
#pragma unroll
                for (int k = 0; k < NC; ++k) v[k] = fmaf(__ldcg(part + r * D + lane + 32 * k), w, v[k]);
            }
            finish(i, mm, ll, v);
        }
    }
}

template <int D, typename T>
cudaError_t launch(const CacheFwdParams& p, int num_sms, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(jfa_cache_simt_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         SimtCfg<D>::kBytes);
    if (e != cudaSuccess) return e;
    jfa_cache_simt_kernel<D, T><<<num_sms * kSimtCtasPerSm, kSimtThreads, SimtCfg<D>::kBytes, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t cache_simt_part_bytes(int D, int num_sms) {
    return size_t(num_sms) * kSimtCtasPerSm * 2 * kSimtBM * size_t(D + 2) * 4;
}

cudaError_t launch_cache_simt(int dtype, int D, const CacheFwdParams& p, int num_sms, cudaStream_t st) {
    if (dtype == JFA_F32 && D == 32) return launch<32, float>(p, num_sms, st);
    if (dtype == JFA_F32 && D == 64) return launch<64, float>(p, num_sms, st);
    if (dtype == JFA_BF16 && D == 64) return launch<64, __nv_bfloat16>(p, num_sms, st);
    if (dtype == JFA_BF16 && D == 128) return launch<128, __nv_bfloat16>(p, num_sms, st);
    return cudaErrorInvalidValue;
}

}  // namespace jfa
