// Paged cache: finding a new token's place, and its rows on the way into the cache.
#pragma once

#include "cache_common.cuh"

namespace jfa {

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
    __device__ __forceinline__ void load(const T* src) { set(*reinterpret_cast<const uint4*>(src)); }
    __device__ __forceinline__ void set(const uint4 u) {
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

// COUNT neighbouring floats (their address a multiple of COUNT floats).
template <int COUNT>
__device__ __forceinline__ void load_floats(const float* src, float (&v)[COUNT]) {
    static_assert(COUNT == 2 || COUNT % 4 == 0, "one or more vectors");
    if constexpr (COUNT == 2) {
        const float2 u = *reinterpret_cast<const float2*>(src);
        v[0] = u.x;
        v[1] = u.y;
    } else {
#pragma unroll
        for (int i = 0; i < COUNT; i += 4) {
            const float4 u = *reinterpret_cast<const float4*>(src + i);
            v[i] = u.x;
            v[i + 1] = u.y;
            v[i + 2] = u.z;
            v[i + 3] = u.w;
        }
    }
}

// rotate_unit of vectors that are loaded, with the angles in vectors as well (the table's rows start on
// 16 bytes, and R is a multiple of 16).  It takes more registers: in the append kernel of 16- and 32-bit
// caches, which lives on many CTAs an SM, 24 prompts took 114 us with it instead of 107.
template <typename T>
__device__ __forceinline__ void rotate_vectors(const uint4 own, const uint4 other, T* dst, int unit, const float* row, int R, bool pairs) {
    constexpr int N = Vec<T>::N;
    Vec<T> a;
    if (pairs) {
        const int d = unit * N;
        a.set(own);
        if (d < R) {
            float cs[N / 2], sn[N / 2];
            load_floats<N / 2>(row + d / 2, cs);
            load_floats<N / 2>(row + R / 2 + d / 2, sn);
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const float c = cs[i / 2], s = sn[i / 2];
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
        *reinterpret_cast<uint4*>(dst + unit * N + half) = own;
        return;
    }
    const int d = unit * N;
    Vec<T> b;
    a.set(own);
    b.set(other);
    float cs[N], sn[N];
    load_floats<N>(row + d, cs);
    load_floats<N>(row + half + d, sn);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float c = cs[i], s = sn[i];
        const float x = a.v[i], y = b.v[i];
        a.v[i] = x * c - y * s;
        b.v[i] = y * c + x * s;
    }
    a.store(dst + d);
    b.store(dst + d + half);
}
// Where new token t lies: its sequence's number, position and page, or b < 0 (it belongs to none)
// or page < 0 (a bad sequence or page).  By a whole warp.
struct CachePlace {
    int b, pos, page;
};
__device__ __forceinline__ CachePlace cache_place(const CacheAppendParams& p, int t, int lane) {
    CachePlace c{find_sequence(p.q_off, p.B, t, lane), -1, -1};
    if (c.b >= p.B) c.b = -1;
    if (c.b < 0) return c;
    const int q0 = p.q_off[c.b], q1 = p.q_off[c.b + 1], kv = p.kv_lens[c.b];
    c.pos = kv - q1 + t;
    // (at least as many positions as new tokens, so that none lies before the first)
    bool ok = q0 >= 0 && q1 <= p.T && t >= q0 && t < q1 && kv >= q1 - q0 && kv <= p.max_kv;
    ok = ok && (!p.rot || c.pos < p.rot_len);
    if (ok) c.page = p.table[size_t(c.b) * size_t(p.max_pages) + size_t(c.pos >> p.page_log2)];
    if (c.page >= p.n_pages) c.page = -1;
    return c;
}

}  // namespace jfa
