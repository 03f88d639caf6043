// Adds up the parts of items that were cut between CTAs (the few-rows kernels of 4-bit caches and of
// listed blocks).
//
// Every CTA of those kernels leaves a record: the item that starts in it and goes on past it, or
// none.  A CTA here takes a record's row: its four warps deal the parts among them, a lane takes four
// (or two) columns, the loads of 32 parts are in flight at once, and the warps' sums are added
// in order, so the result does not depend on timing.
// Bound by latency: a record, its maxima and its parts, about 2.5 us.  With an item's last CTA adding its parts
// itself, one 4-bit history of 131k keys (57 parts for each of 8 heads) took 43.5 us instead of 37.5, 64
// histories 75 instead of 68.6, 128 listed blocks of 16 keys 14.5 instead of 10.6.  Then with 32 parts in
// flight instead of 64, and twice the CTAs an SM for it: one user 9.6 -> 9.1, 64 histories 67.4 -> 66.0, 64 lists
// of blocks 36.8 -> 35.2 (16 parts: the long history 39.1).
#include <algorithm>

#include "cache_common.cuh"

namespace jfa {

namespace {

constexpr int kJoinWarps = 4, kJoinRows = 4, kAtOnce = 8;
static_assert(kJoinWarps * kAtOnce == 32, "a lane has a part's maximum and sum");

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps, 8) jfa_cache_join_kernel(const CacheFwdParams p) {
    constexpr int V = D / 32, kPart = 16 * (D + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ float sums[kJoinWarps][D];
    wait_previous();
    const CacheCut cut = p.cuts[blockIdx.x];
    const int parts = cut.last - cut.first + 1;
    for (int row = blockIdx.y; row < cut.rows; row += int(gridDim.y)) {
        auto part_of = [&](int c) { return p.part + size_t(cache_slot(cut.first + c, cut.first)) * kPart; };
        float m = -INFINITY, l = 0.f, acc[V];
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.f;
        for (int c0 = 0; c0 < parts; c0 += 32) {
            float x[kAtOnce][V], mc, lc;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int c = c0 + kJoinWarps * k + warp;
                if (c >= parts) continue;
                const float* src = part_of(c) + row * D + V * lane;
                if constexpr (V == 4) {
                    const float4 u = __ldcg(reinterpret_cast<const float4*>(src));
                    x[k][0] = u.x;
                    x[k][1] = u.y;
                    x[k][2] = u.z;
                    x[k][3] = u.w;
                } else {
                    const float2 u = __ldcg(reinterpret_cast<const float2*>(src));
                    x[k][0] = u.x;
                    x[k][1] = u.y;
                }
            }
            const int mine = c0 + lane;  // 32 parts' maxima and sums
            mc = mine < parts ? __ldcg(part_of(mine) + 16 * D + row) : -INFINITY;
            lc = mine < parts ? __ldcg(part_of(mine) + 16 * D + 16 + row) : 0.f;
            float top = fmaxf(m, mc);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            if (top == -INFINITY) continue;  // (no key yet: O is 0 in all of them)
            const float keep = ex2_approx(m - top);
            m = top;
            l *= keep;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] *= keep;
            mc = ex2_approx(mc - top);
            l = fmaf(mc, lc, l);
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int at = kJoinWarps * k + warp;
                const float f = __shfl_sync(0xffffffffu, mc, at);
                if (c0 + at >= parts) continue;
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] = fmaf(x[k][v], f, acc[v]);
            }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
#pragma unroll
        for (int v = 0; v < V; ++v) sums[warp][V * lane + v] = acc[v];
        __syncthreads();
        const int r = cut.row0 + row, tok = div_g(p, r);
        const size_t at = size_t(cut.q0 + tok) * size_t(p.H) + size_t(cut.head0 + r - tok * p.g);
        const float inv = l > 0.f ? p.o_mul / l : 0.f;
        for (int c = threadIdx.x; c < D / 2; c += 32 * kJoinWarps) {
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) {
                a += sums[w][2 * c];
                b += sums[w][2 * c + 1];
            }
            if (p.o_f32)
                *reinterpret_cast<float2*>(static_cast<float*>(p.O) + at * D + 2 * c) = make_float2(a * inv, b * inv);
            else
                *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.O) + at * D + 2 * c) = pack_bf16x2(a * inv, b * inv);
        }
        if (p.lse && threadIdx.x == 0) p.lse[at] = l > 0.f ? (m + __log2f(l)) * 0.6931471805599453f : -INFINITY;
        __syncthreads();
    }
}

template <int D>
cudaError_t launch(const CacheFwdParams& p, int ctas, cudaStream_t st) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, std::min(kJoinRows, p.bm));
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, jfa_cache_join_kernel<D>, p);
}

}  // namespace

cudaError_t launch_cache_join(int D, const CacheFwdParams& p, int ctas, cudaStream_t st) {
    return D == 128 ? launch<128>(p, ctas, st) : launch<64>(p, ctas, st);
}

}  // namespace jfa
