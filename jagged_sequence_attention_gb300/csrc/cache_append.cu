// Appends new tokens' keys and values to a paged cache, rotating keys and queries by their
// position on the way: y_a = x_a cos - x_b sin, y_b = x_b cos + x_a sin on the pairs of each
// head's first rot_dim elements.
//
// Bound by its bytes, each read and written once in 16-byte vectors.  One CTA per token: the
// token's rows are a few KB, and the CTAs of an SM cover each other's chain of offsets, page and
// data.  A thread takes both vectors of a half-split pair, so a query head may be rotated in
// place.  The token's sequence is found by a 32-way search of the offsets (one load deep up to 31
// sequences, two up to 1023).
// Measured: 24 prompts of up to 2048 tokens (32 query and 2 x 8 cached heads of 128, bf16, 710 MB)
// 108 us, 6.5 TB/s, 0.96 of the copy rate; 7 fp32 prompts (60 MB) 13.5 us, 0.65, a few waves
// whose start and end show, and a thread loads its next vectors only after it has stored the
// last; 256 single tokens 3.8 us and one token 3.3 us, the launch and the
// chain of loads.  Loading a token's data before its sequence is found was slower (108 -> 114 us,
// fp32 13.5 -> 15.9 us: more live registers, fewer CTAs an SM).
#include "cache_rows.cuh"

namespace jfa {

namespace {

constexpr int kAppendThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kAppendThreads) jfa_cache_append_kernel(const CacheAppendParams p) {
    constexpr int N = Vec<T>::N;
    const int t = blockIdx.x, lane = threadIdx.x & 31;
    const CachePlace at = cache_place(p, t, lane);
    if (at.b < 0) return;  // rows behind the last sequence
    const int pos = at.pos, page = at.page;
    if (page < 0) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
        return;
    }
    const int slot = pos & ((1 << p.page_log2) - 1);
    T* kdst = static_cast<T*>(p.Kc) + page * p.ks[0] + slot * p.ks[1];
    T* vdst = static_cast<T*>(p.Vc) + page * p.vs[0] + slot * p.vs[1];
    const T* ksrc = static_cast<const T*>(p.K) + t * p.k_stride;
    const T* vsrc = static_cast<const T*>(p.V) + t * p.v_stride;
    const T* qsrc = static_cast<const T*>(p.Q) + t * p.q_stride;
    T* qdst = static_cast<T*>(p.Q_out) + t * p.qo_stride;
    const float* row = p.rot ? p.rot + size_t(pos) * size_t(p.rot_dim) : nullptr;
    const int R = p.rot ? p.rot_dim : 0;
    const int vecs = p.D / N;                                // vectors of a head
    const int units = p.pairs ? vecs : vecs - R / 2 / N;     // units of a rotated head
    const int nq = p.H * units, nk = p.Hkv * units, nv = p.Hkv * vecs;
    for (int i = threadIdx.x; i < nq + nk + nv; i += kAppendThreads) {
        if (i < nq) {
            const int h = i / units, u = i - h * units;
            rotate_unit<T>(qsrc + h * p.D, qdst + h * p.D, u, row, R, p.pairs);
        } else if (i < nq + nk) {
            const int h = (i - nq) / units, u = i - nq - h * units;
            rotate_unit<T>(ksrc + h * p.D, kdst + h * p.ks[2], u, row, R, p.pairs);
        } else {
            const int h = (i - nq - nk) / vecs, u = i - nq - nk - h * vecs;
            *reinterpret_cast<uint4*>(vdst + h * p.vs[2] + u * N) = *reinterpret_cast<const uint4*>(vsrc + h * p.D + u * N);
        }
    }
}

}  // namespace

cudaError_t launch_cache_append(int dtype, const CacheAppendParams& p, cudaStream_t st) {
    if (dtype == JFA_BF16)
        jfa_cache_append_kernel<__nv_bfloat16><<<p.T, kAppendThreads, 0, st>>>(p);
    else
        jfa_cache_append_kernel<float><<<p.T, kAppendThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace jfa
