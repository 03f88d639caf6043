// Paged-cache attention for fp32: plain fp32 arithmetic on the CUDA cores (the tensor cores'
// fp32-input format would drop 13 mantissa bits), in two row-tile sizes.
//
// A CTA of four warps streams an item's keys 64 at a time through shared memory, copied
// there 16 bytes at a time (cp.async) by pages.  A warp owns its rows from scores to output,
// so the softmax needs no exchange between warps; a thread takes RT rows x KT keys of the
// scores and RT rows x CT columns of P V.
//   128 rows (chunks): bound by the FMA units and, nearly as much, by shared-memory reads --
//     a thread's 8 x 8 tile reads 16 16-byte words per 256 products, as many cycles of the
//     128 B/clk return path as of the FMA units.  K is loaded again during P V and V during
//     the next scores, so one buffer of each is enough and two CTAs fit an SM.
//   16 rows (single tokens, short sets): 4 x 2 scores per thread, two buffers of K and V,
//     three CTAs per SM: bound by the stream of K and V up to a few rows per key head.
#include "cache_common.cuh"
#include "tilemath.cuh"

namespace jfa {

namespace {

constexpr int kSimtBN = 64;

template <int D, int BM>
struct SimtCfg {
    static constexpr bool kBig = BM == 128;
    static constexpr int kWarps = kBig ? 8 : 4, kThreads = 32 * kWarps;
    static constexpr int kRows = BM / kWarps;             // rows of a warp
    static constexpr int LY = 4, LX = 8;                  // big: lanes 4 (rows) x 8 (keys); small: 1 x 32
    static constexpr int RT = kBig ? kRows / LY : kRows;  // rows of a thread
    static constexpr int KT = kBig ? kSimtBN / LX : 2;    // keys of a thread
    static constexpr int kCtasPerSm = kBig ? 2 : 3;
    static constexpr int kBufs = kBig ? 1 : 2;
    // floats per staged row: 16-byte reads of 8 consecutive key rows cover all banks
    static constexpr int kStrideK = D + 4, kStrideQ = D + 4, kStrideP = kBig ? kSimtBN + 8 : kSimtBN;
    static constexpr int kQ = 0, kK = kQ + BM * kStrideQ, kV = kK + kBufs * kSimtBN * kStrideK;
    static constexpr int kP = kV + kBufs * kSimtBN * D, kFloats = kP + BM * kStrideP;
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
__global__ void __launch_bounds__(SimtCfg<D, BM>::kThreads, SimtCfg<D, BM>::kCtasPerSm) jfa_cache_simt_kernel(const CacheFwdParams p) {
    using C = SimtCfg<D, BM>;
    constexpr int BN = kSimtBN, RT = C::RT, KT = C::KT;
    // columns of a thread in P V: big: groups of four at 4 kx + 32 j; small: NC lane and on
    constexpr int NC = C::kBig ? D / C::LX : D / 32;
    extern __shared__ __align__(16) float sm[];
    __shared__ int last_flag;
    float* sQ = sm + C::kQ;
    float* sP = sm + C::kP;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ry = C::kBig ? lane / C::LX : 0, kx = C::kBig ? lane % C::LX : lane;
    // tile row of this thread's row i, tile key of its key j, output column of its column c
    auto row_of = [&](int i) { return warp * C::kRows + (C::kBig ? C::LY * i + ry : i); };
    auto key_of = [&](int j) { return kx + (C::kBig ? C::LX : 32) * j; };
    const CacheStart start = cache_start<BN>(p, reinterpret_cast<int*>(sm));
    CacheCursor<BN> cur(start);
    CacheSeg g;
    const int page_mask = (1 << p.page_log2) - 1;
    while (cur.next(p, g)) {
        const int R = g.s.q_len * p.g, diag = g.s.kv_len - g.s.q_len, r0 = g.tile * BM;
        // 64 rows of K or V from position c0 on, zeros where no row of the item may look
        auto load = [&](float* dst, int stride, const void* base, const int64_t* s, int c0) {
            constexpr int kPieces = D / 4, kStep = C::kThreads / kPieces;
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
            cp_commit();
        };
        auto load_k = [&](int kt) { load(sm + C::kK + (C::kBufs > 1 ? (kt & 1) * BN * C::kStrideK : 0), C::kStrideK, p.K, p.ks, (g.r.f + kt) * BN); };
        auto load_v = [&](int kt) { load(sm + C::kV + (C::kBufs > 1 ? (kt & 1) * BN * D : 0), D, p.V, p.vs, (g.r.f + kt) * BN); };
        const int k_end = g.r.n > 0 ? g.k1 : g.k0;
        __syncthreads();  // the previous item's last reads
        if (g.k0 < k_end) {
            load_k(g.k0);
            load_v(g.k0);
        }
        for (int e = threadIdx.x; e < BM * D / 4; e += C::kThreads) {
            const int tr = e / (D / 4), c = e % (D / 4), r = r0 + tr;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < R) {
                const int tok = div_g(p, r);
                v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.Q) + (g.s.q0 + tok) * p.q_stride +
                                                     int64_t(g.hk * p.g + r - tok * p.g) * D + 4 * c);
                v = make_float4(v.x * p.scale_log2, v.y * p.scale_log2, v.z * p.scale_log2, v.w * p.scale_log2);
            }
            *reinterpret_cast<float4*>(sQ + tr * C::kStrideQ + 4 * c) = v;
        }
        float m[RT], l[RT];
        float2 o[RT][(NC + 1) / 2];  // columns in pairs: two products an instruction
        int rel[RT];                 // position of each row (rows past the end repeat the last one's)
        const float* brow[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int r = min(r0 + row_of(i), R - 1), tok = div_g(p, r);
            rel[i] = tok + diag;
            brow[i] = BIAS ? p.bias + (g.hk * p.g + r - tok * p.g) * 32 : nullptr;
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < (NC + 1) / 2; ++c) o[i][c] = make_float2(0.f, 0.f);
        }
        const int t_first = div_g(p, r0) + diag, t_last = div_g(p, min(R, r0 + BM) - 1) + diag;
        const int all_hi = p.causal ? min(g.s.kv_len, t_first + 1) : g.s.kv_len;
        const int all_lo = p.window >= 0 ? max(0, t_last - p.window) : 0;
        for (int kt = g.k0; kt < k_end; ++kt) {
            const int c0 = (g.r.f + kt) * BN;
            const float* sK = sm + C::kK + (C::kBufs > 1 ? (kt & 1) * BN * C::kStrideK : 0);
            const float* sV = sm + C::kV + (C::kBufs > 1 ? (kt & 1) * BN * D : 0);
            if (C::kBufs > 1) {
                // both of the next tile's loads go out before this tile is waited for
                if (kt > g.k0) __syncthreads();  // the other buffers have been read
                if (kt + 1 < k_end) {
                    load_k(kt + 1);
                    load_v(kt + 1);
                    cp_wait<2>();
                } else {
                    cp_wait<0>();
                }
            } else {
                cp_wait<1>();  // K of this tile (V may still be on its way)
            }
            __syncthreads();
            float x[RT][KT];
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < KT; ++j) x[i][j] = 0.f;
#pragma unroll 1
            for (int d = 0; d < D; d += 4) {
                float4 kk[KT];
#pragma unroll
                for (int j = 0; j < KT; ++j) kk[j] = *reinterpret_cast<const float4*>(sK + key_of(j) * C::kStrideK + d);
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const float4 q = *reinterpret_cast<const float4*>(sQ + row_of(i) * C::kStrideQ + d);
                    // (the keys innermost: consecutive instructions are independent)
#pragma unroll
                    for (int j = 0; j < KT; ++j) x[i][j] = fmaf(q.x, kk[j].x, x[i][j]);
#pragma unroll
                    for (int j = 0; j < KT; ++j) x[i][j] = fmaf(q.y, kk[j].y, x[i][j]);
#pragma unroll
                    for (int j = 0; j < KT; ++j) x[i][j] = fmaf(q.z, kk[j].z, x[i][j]);
#pragma unroll
                    for (int j = 0; j < KT; ++j) x[i][j] = fmaf(q.w, kk[j].w, x[i][j]);
                }
            }
            if (C::kBufs == 1) {
                __syncthreads();  // K has been read: the next tile's loads overlap P V
                if (kt + 1 < k_end) load_k(kt + 1);
            }
            const bool masked = c0 < all_lo || c0 + BN > all_hi;
            const int bk = BIAS ? relpos_bucket(t_last - c0) : 0;
            const int near = t_first - c0 - (BN - 1);
            const bool one = BIAS && (near >= 0 || t_last <= c0) && bk == relpos_bucket(near);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const float b1 = BIAS && one ? __ldg(brow[i] + bk) * 1.4426950408889634f : 0.f;
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < KT; ++j) {
                    const int key = c0 + key_of(j);
                    float add = b1;
                    if (BIAS && !one) add = __ldg(brow[i] + relpos_bucket(rel[i] - key)) * 1.4426950408889634f;
                    float y = BIAS ? x[i][j] + add : x[i][j];
                    if (masked) {
                        const bool in = key < g.s.kv_len && (!p.causal || key <= rel[i]) &&
                                        (p.window < 0 || key >= rel[i] - p.window);
                        y = in ? y : -INFINITY;
                    }
                    x[i][j] = y;
                    mx = fmaxf(mx, y);
                }
#pragma unroll
                for (int s = (C::kBig ? C::LX : 32) / 2; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
                const float m_new = fmaxf(m[i], mx);
                const float m_use = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = ex2_approx(m[i] - m_use);
                m[i] = m_new;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < KT; ++j) {
                    const float e = ex2_approx(x[i][j] - m_use);
                    sP[row_of(i) * C::kStrideP + key_of(j)] = e;
                    sum += e;
                }
                l[i] = fmaf(l[i], alpha, sum);  // this thread's keys; summed over the lanes at the end
#pragma unroll
                for (int c = 0; c < (NC + 1) / 2; ++c) o[i][c] = mul2(o[i][c], make_float2(alpha, alpha));
            }
            __syncwarp();
            if (C::kBufs == 1) {
                if (kt + 1 < k_end)
                    cp_wait<1>();  // V of this tile
                else
                    cp_wait<0>();
                __syncthreads();
            }
            if constexpr (C::kBig) {
#pragma unroll 1
                for (int j = 0; j < BN; j += 4) {
                    float4 e[RT];
#pragma unroll
                    for (int i = 0; i < RT; ++i) e[i] = *reinterpret_cast<const float4*>(sP + row_of(i) * C::kStrideP + j);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int c4 = 0; c4 < NC / 4; ++c4) {
                            const float4 v = *reinterpret_cast<const float4*>(sV + (j + q) * D + 4 * kx + 32 * c4);
#pragma unroll
                            for (int i = 0; i < RT; ++i) {
                                const float w = q == 0 ? e[i].x : q == 1 ? e[i].y : q == 2 ? e[i].z : e[i].w;
                                o[i][2 * c4] = fma2(make_float2(w, w), make_float2(v.x, v.y), o[i][2 * c4]);
                                o[i][2 * c4 + 1] = fma2(make_float2(w, w), make_float2(v.z, v.w), o[i][2 * c4 + 1]);
                            }
                        }
                }
                __syncthreads();  // V has been read: the next tile's loads overlap its scores
                if (kt + 1 < k_end) load_v(kt + 1);
            } else {
#pragma unroll 2
                for (int j = 0; j < BN; j += 4) {
                    float4 e[RT];
#pragma unroll
                    for (int i = 0; i < RT; ++i) e[i] = *reinterpret_cast<const float4*>(sP + row_of(i) * C::kStrideP + j);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float2 v;  // columns NC lane, NC lane + 1
                        if constexpr (NC == 2)
                            v = *reinterpret_cast<const float2*>(sV + (j + q) * D + 2 * lane);
                        else
                            v = make_float2(sV[(j + q) * D + lane], 0.f);
#pragma unroll
                        for (int i = 0; i < RT; ++i) {
                            const float w = q == 0 ? e[i].x : q == 1 ? e[i].y : q == 2 ? e[i].z : e[i].w;
                            o[i][0] = fma2(make_float2(w, w), v, o[i][0]);
                        }
                    }
                }
                __syncwarp();
            }
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int s = (C::kBig ? C::LX : 32) / 2; s > 0; s >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], s);
        // a row's columns as this thread holds them, to dst (times mul)
        auto put = [&](float* dst, const float2 (&v)[(NC + 1) / 2], float mul) {
            if constexpr (C::kBig) {
#pragma unroll
                for (int c = 0; c < NC / 2; c += 2)
                    *reinterpret_cast<float4*>(dst + 4 * kx + 16 * c) =
                        make_float4(v[c].x * mul, v[c].y * mul, v[c + 1].x * mul, v[c + 1].y * mul);
            } else if constexpr (NC == 2) {
                *reinterpret_cast<float2*>(dst + 2 * lane) = make_float2(v[0].x * mul, v[0].y * mul);
            } else {
                dst[lane] = v[0].x * mul;
            }
        };
        auto row_at = [&](int r) {
            const int tok = div_g(p, r);
            return size_t(g.s.q0 + tok) * size_t(p.H) + size_t(g.hk * p.g + r - tok * p.g);
        };
        auto finish = [&](int i, float mm, float ll, const float2 (&v)[(NC + 1) / 2]) {
            const int r = r0 + row_of(i);
            if (r >= R) return;
            const size_t row = row_at(r);
            put(static_cast<float*>(p.O) + row * D, v, ll > 0.f ? 1.f / ll : 0.f);
            if (p.lse && kx == 0) p.lse[row] = ll > 0.f ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
        };
        if (g.whole()) {
#pragma unroll
            for (int i = 0; i < RT; ++i) finish(i, m[i], l[i], o[i]);
            continue;
        }
        const int first = cache_first_cta(p, start, g), last = cache_last_cta(p, start, g);
        float* mine = p.part + size_t(cache_slot(blockIdx.x, first)) * C::kPart;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int tr = row_of(i);
            if (r0 + tr >= R) continue;
            put(mine + tr * D, o[i], 1.f);
            if (kx == 0) {
                mine[BM * D + tr] = m[i];
                mine[BM * D + BM + tr] = l[i];
            }
        }
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
        // lanes the parts' maxima and sums and then D / 32 columns each.
        constexpr int LC = D / 32, kRowsAtOnce = C::kBig ? 4 : 1;
        const int parts = last - first + 1, nr = min(BM, R - r0);
        auto part_of = [&](int c) { return p.part + size_t(cache_slot(first + c, first)) * C::kPart; };
        for (int t0 = warp * kRowsAtOnce; t0 < nr; t0 += C::kWarps * kRowsAtOnce) {
            float mm[kRowsAtOnce], ll[kRowsAtOnce], v[kRowsAtOnce][LC];
#pragma unroll
            for (int k = 0; k < kRowsAtOnce; ++k) {
                const int tr = min(t0 + k, nr - 1);
                mm[k] = -INFINITY;
                ll[k] = 0.f;
                for (int c = lane; c < parts; c += 32) mm[k] = fmaxf(mm[k], __ldcg(part_of(c) + BM * D + tr));
#pragma unroll
                for (int c = 0; c < LC; ++c) v[k][c] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < kRowsAtOnce; ++k)
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) mm[k] = fmaxf(mm[k], __shfl_xor_sync(0xffffffffu, mm[k], s));
            for (int c0 = 0; c0 < parts; c0 += 32) {
                float w[kRowsAtOnce];
#pragma unroll
                for (int k = 0; k < kRowsAtOnce; ++k) {
                    const int tr = min(t0 + k, nr - 1);
                    const float mc = c0 + lane < parts ? __ldcg(part_of(c0 + lane) + BM * D + tr) : -INFINITY;
                    w[k] = mc == -INFINITY ? 0.f : ex2_approx(mc - mm[k]);
                    if (c0 + lane < parts) ll[k] = fmaf(__ldcg(part_of(c0 + lane) + BM * D + BM + tr), w[k], ll[k]);
                }
#pragma unroll 4
                for (int c = 0; c < min(32, parts - c0); ++c)
#pragma unroll
                    for (int k = 0; k < kRowsAtOnce; ++k) {
                        const float wc = __shfl_sync(0xffffffffu, w[k], c);
                        const float* src = part_of(c0 + c) + min(t0 + k, nr - 1) * D + LC * lane;
                        if constexpr (LC == 2) {
                            const float2 u = __ldcg(reinterpret_cast<const float2*>(src));
                            v[k][0] = fmaf(u.x, wc, v[k][0]);
                            v[k][LC - 1] = fmaf(u.y, wc, v[k][LC - 1]);
                        } else {
                            v[k][0] = fmaf(__ldcg(src), wc, v[k][0]);
                        }
                    }
            }
#pragma unroll
            for (int k = 0; k < kRowsAtOnce; ++k) {
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) ll[k] += __shfl_xor_sync(0xffffffffu, ll[k], s);
                if (t0 + k >= nr) continue;
                const size_t row = row_at(r0 + t0 + k);
                const float inv = ll[k] > 0.f ? 1.f / ll[k] : 0.f;
#pragma unroll
                for (int c = 0; c < LC; ++c) static_cast<float*>(p.O)[row * D + LC * lane + c] = v[k][c] * inv;
                if (p.lse && lane == 0) p.lse[row] = ll[k] > 0.f ? (mm[k] + log2f(ll[k])) * 0.6931471805599453f : -INFINITY;
            }
        }
    }
}

template <int D, int BM, bool BIAS>
cudaError_t launch(const CacheFwdParams& p, int num_sms, cudaStream_t st) {
    using C = SimtCfg<D, BM>;
    cudaError_t e = cudaFuncSetAttribute(jfa_cache_simt_kernel<D, BM, BIAS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::kBytes);
    if (e != cudaSuccess) return e;
    jfa_cache_simt_kernel<D, BM, BIAS><<<num_sms * C::kCtasPerSm, C::kThreads, C::kBytes, st>>>(p);
    return cudaGetLastError();
}

template <int D, int BM>
cudaError_t launch_b(const CacheFwdParams& p, int num_sms, cudaStream_t st) {
    return p.bias ? launch<D, BM, true>(p, num_sms, st) : launch<D, BM, false>(p, num_sms, st);
}

}  // namespace

size_t cache_simt_part_bytes(int D, int num_sms) { return size_t(num_sms) * 2 * 2 * 128 * size_t(D + 2) * 4; }

cudaError_t launch_cache_simt(int D, bool chunk, const CacheFwdParams& p, int num_sms, cudaStream_t st) {
    if (D == 32) return chunk ? launch_b<32, 128>(p, num_sms, st) : launch_b<32, 16>(p, num_sms, st);
    return chunk ? launch_b<64, 128>(p, num_sms, st) : launch_b<64, 16>(p, num_sms, st);
}

}  // namespace jfa
