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
#include "cache_common.cuh"

namespace jfa {

namespace {

constexpr int kAppendThreads = 128;

// The last b with q_off[b] <= t (offsets non-decreasing), by the whole warp; -1 if none.
__device__ __forceinline__ int find_sequence(const int32_t* q_off, int B, int t, int lane) {
    int lo = 0, n = B + 1;  // entries [lo, lo + n) hold the boundary; those before lo are <= t
    while (n > 32) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const uint32_t m = __ballot_sync(0xffffffffu, lane * step < n && q_off[i] <= t);
        const int k = __popc(m);  // the first k probes are <= t
        if (k == 0) return lo - 1;
        const int used = (k - 1) * step;
        lo += used;
        n = min(n - used, step);
    }
    const uint32_t m = __ballot_sync(0xffffffffu, lane < n && q_off[lo + lane] <= t);
    return lo + __popc(m) - 1;
}

template <typename T>
struct Vec {  // 16 bytes of T as floats
    static constexpr int N = 16 / sizeof(T);
    float v[N];
    __device__ __forceinline__ void load(const T* src) {
        const uint4 u = *reinterpret_cast<const uint4*>(src);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                v[i] = __uint_as_float(w[i]);
            } else {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
    __device__ __forceinline__ void store(T* dst) const {
        uint4 u;
        if constexpr (sizeof(T) == 4) {
            u = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        } else {
            u = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                           pack_bf16x2(v[6], v[7]));
        }
        *reinterpret_cast<uint4*>(dst) = u;
    }
};

// Vectors [d, d + N) (and, for a half-split pair, [d + R/2, + N)) of one head, from src to dst.
template <typename T>
__device__ __forceinline__ void rotate_unit(const T* src, T* dst, int unit, const float* row, int R, bool pairs) {
    constexpr int N = Vec<T>::N;
    Vec<T> a;
    if (pairs) {
        const int d = unit * N;
        a.load(src + d);
        if (d < R) {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const float c = row[(d + i) / 2], s = row[R / 2 + (d + i) / 2];
                const float x = a.v[i], y = a.v[i + 1];
                a.v[i] = x * c - y * s;
                a.v[i + 1] = y * c + x * s;
            }
        }
        a.store(dst + d);
        return;
    }
    const int half = R / 2;
    if (unit * N >= half) {  // the elements past R, copied
        const int d = unit * N + half;
        *reinterpret_cast<uint4*>(dst + d) = *reinterpret_cast<const uint4*>(src + d);
        return;
    }
    const int d = unit * N;
    Vec<T> b;
    a.load(src + d);
    b.load(src + d + half);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float c = row[d + i], s = row[half + d + i];
        const float x = a.v[i], y = b.v[i];
        a.v[i] = x * c - y * s;
        b.v[i] = y * c + x * s;
    }
    a.store(dst + d);
    b.store(dst + d + half);
}

template <typename T>
__global__ void __launch_bounds__(kAppendThreads) jfa_cache_append_kernel(const CacheAppendParams p) {
    constexpr int N = Vec<T>::N;
    const int t = blockIdx.x, lane = threadIdx.x & 31;
    const int b = find_sequence(p.q_off, p.B, t, lane);
    if (b < 0 || b >= p.B) return;  // rows behind the last sequence
    const int q0 = p.q_off[b], q1 = p.q_off[b + 1], kv = p.kv_lens[b];
    const int pos = kv - q1 + t;
    // (at least as many positions as new tokens, so that none lies before the first)
    bool ok = q0 >= 0 && q1 <= p.T && t >= q0 && t < q1 && kv >= q1 - q0 && kv <= p.max_kv;
    ok = ok && (!p.rot || pos < p.rot_len);
    int page = -1;
    if (ok) page = p.table[size_t(b) * size_t(p.max_pages) + size_t(pos >> p.page_log2)];
    ok = ok && page >= 0 && page < p.n_pages;
    if (!ok) {
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
