// A paged cache held in 4 bits: its handle, appending to it, and reading a cache back.
// Semantics are documented in include/jfa.h, the format in quant.cuh.
//
// Appending: of each 16 elements of a row y (keys rotated first, not rounded)
//   s = e4m3(max|y| / (6 c)),  code_i = e2m1(y_i / (c s)),  c the array's factor,
// each to nearest even, as if in exact arithmetic.  In fp32 the rotated y and the quotients are a
// little off, which matters only next to the middle between two codes (or scales): both ends of
// the interval that y can lie in are rounded, and where they differ (about one group in
// thousands) the 16 elements are done again in 64 bits.  So a cache's contents do not depend on
// how the rotation was computed.  Elements taken as they are, with a factor that is a power
// of two, need no interval: their quotients are rounded correctly in fp32, and a bf16 value that
// is not at a middle is 2^-9 of it away or more.
// A thread takes the 16 elements of a group; a rotated group's partners (the other halves of its
// pairs, eight or sixteen elements on) are read again by it instead of handed over.
#include <cuda_bf16.h>

#include <new>

#include "cache_handle.h"
#include "cache_rows.cuh"
#include "quant.cuh"

using namespace jfa;

namespace jfa {

// bf16 rows, 16 packed rows or fewer in an item; early: as launch_cache_decode's.
cudaError_t launch_cache_decode4(int D, const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p, bool early,
                                 int num_sms, cudaStream_t st);
size_t cache_decode4_part_bytes(int D, int num_sms);
// Items of 256 packed rows.
cudaError_t launch_cache_chunk4(int D, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CacheFwdParams& p,
                                int num_sms, cudaStream_t st);

namespace {

constexpr int kThreads = 128;

struct QuantParams {
    uint8_t *k_scales, *v_scales;
    int64_t kss[2], vss[2];
    float factor[2];
};

// One group of a row: 16 elements from d0 on of src, with its pairs' angles (R: rotated elements).
struct Group {
    const __nv_bfloat16* src;
    const float* row;
    int d0, R;
    bool pairs;
};

// Element i of a rotated group in 64 bits (the products are exact there).
__device__ __forceinline__ double exact_element(const Group& g, int i) {
    const int d = g.d0 + i, half = g.R / 2;
    const double x = double(__bfloat162float(g.src[d]));
    if (d >= g.R) return x;
    const bool first = g.pairs ? (d & 1) == 0 : d < half;
    const int other = g.pairs ? d ^ 1 : first ? d + half : d - half, k = g.pairs ? d / 2 : first ? d : d - half;
    const double y = double(__bfloat162float(g.src[other])), c = double(g.row[k]), s = double(g.row[half + k]);
    return first ? x * c - y * s : x * c + y * s;
}

// A group in 64 bits: its codes, and the nearer one of two neighbouring scales lo <= hi.
__device__ __noinline__ uint2 exact_group(const Group& g, float factor, uint32_t lo, uint32_t hi, uint32_t& scale) {
    double top = 0.0;
    for (int i = 0; i < 16; ++i) top = fmax(top, fabs(exact_element(g, i)));
    auto value = [](uint32_t b) { return double(f16_to_float(e4m3_to_f16(b)).x); };
    const double c = double(factor);
    while (lo < hi) {  // (the middle of two scales has five bits: the comparison is exact)
        const double mid = 0.5 * (value(lo) + value(lo + 1)) * (6.0 * c);
        if (!(top > mid || (top == mid && (lo & 1u)))) break;
        ++lo;
    }
    scale = lo;
    const double step = c * value(lo);
    uint32_t w[2] = {0u, 0u};
    for (int i = 0; i < 16; ++i) {
        const double y = exact_element(g, i), a = fabs(y);
        uint32_t code = 0u;
        const double mids[7] = {0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0};
        if (step > 0.0)
            for (int k = 0; k < 7; ++k) code += (a > mids[k] * step || ((k & 1) && a == mids[k] * step)) ? 1u : 0u;
        if (y < 0.0) code |= 8u;
        w[i >> 3] |= code << (4 * (i & 7));
    }
    return make_uint2(w[0], w[1]);
}

// The group's codes and scale.  exact: a row as it is and a factor that is a power of two.
__device__ __forceinline__ uint2 quantise(const Group& g, float factor, bool exact, uint32_t& scale) {
    float y[16], slack = 0.f;
    const int half = g.R / 2;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const int d = g.d0 + 8 * v;
        Vec<__nv_bfloat16> a;
        a.load(g.src + d);
        if (d < g.R) {
            if (g.pairs) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float c = g.row[(d + i) / 2], s = g.row[half + (d + i) / 2], x = a.v[i], z = a.v[i + 1];
                    a.v[i] = x * c - z * s;
                    a.v[i + 1] = z * c + x * s;
                    slack = fmaxf(slack, (fabsf(x) + fabsf(z)) * fmaxf(fabsf(c), fabsf(s)));
                }
            } else {
                const bool first = d < half;
                const int k = first ? d : d - half;
                Vec<__nv_bfloat16> b;
                b.load(g.src + (first ? d + half : d - half));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float c = g.row[k + i], s = g.row[half + k + i], x = a.v[i], z = first ? -b.v[i] : b.v[i];
                    a.v[i] = x * c + z * s;
                    slack = fmaxf(slack, fabsf(x * c) + fabsf(z * s));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) y[8 * v + i] = a.v[i];
    }
    // a sum of two products is off by less than 2^-22 of their magnitudes
    slack *= 0x1p-22f;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(y[i]));
    const float six = 6.f * factor;
    uint32_t lo, hi;
    if (exact) {
        lo = hi = to_e4m3(__fdiv_rn(top, six), 0.f) & 255u;
    } else {
        const float q = __fdiv_rn(top, six), e = __fdividef(slack, six);
        const uint32_t both = to_e4m3(fmaxf(fmaf(q, -0x1p-22f, q - e), 0.f), fmaf(q, 0x1p-22f, q + e));
        lo = both & 255u;
        hi = both >> 8;
    }
    scale = lo;
    bool sure = lo == hi;
    uint32_t w[2] = {0u, 0u};
    if (sure && lo != 0u) {
        const float step = factor * f16_to_float(e4m3_to_f16(lo)).x;
        if (exact) {
#pragma unroll
            for (int i = 0; i < 16; i += 2)
                w[i >> 3] |= to_e2m1(__fdiv_rn(y[i], step), __fdiv_rn(y[i + 1], step)) << (4 * (i & 7));
        } else {
            const float inv = __fdiv_rn(1.f, step), e = slack * inv * 1.0001f;
            uint32_t above[2] = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float a = fabsf(y[i] * inv), b = fabsf(y[i + 1] * inv);
                w[i >> 3] |= to_e2m1(copysignf(fmaxf(fmaf(a, -0x1p-21f, a - e), 0.f), y[i]),
                                     copysignf(fmaxf(fmaf(b, -0x1p-21f, b - e), 0.f), y[i + 1]))
                             << (4 * (i & 7));
                above[i >> 3] |= to_e2m1(copysignf(fmaf(a, 0x1p-21f, a + e), y[i]), copysignf(fmaf(b, 0x1p-21f, b + e), y[i + 1]))
                                 << (4 * (i & 7));
            }
            sure = w[0] == above[0] && w[1] == above[1];
        }
    }
    if (!sure) return exact_group(g, factor, lo, hi, scale);
    return make_uint2(w[0], w[1]);
}

__global__ void __launch_bounds__(kThreads) jfa_cache_append4_kernel(const CacheAppendParams p, const QuantParams z) {
    using T = __nv_bfloat16;
    const int t = blockIdx.x, lane = threadIdx.x & 31;
    const CachePlace at = cache_place(p, t, lane);
    if (at.b < 0) return;  // rows behind the last sequence
    if (at.page < 0) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
        return;
    }
    const int slot = at.pos & ((1 << p.page_log2) - 1);
    const float* row = p.rot ? p.rot + size_t(at.pos) * size_t(p.rot_dim) : nullptr;
    const int R = p.rot ? p.rot_dim : 0;
    const int ng = p.D / 16, units = p.pairs ? p.D / 8 : p.D / 8 - R / 16;
    const int nk = p.Hkv * ng, nq = p.H * units;
    for (int i = threadIdx.x; i < 2 * nk + nq; i += kThreads) {
        if (i >= 2 * nk) {  // a query head's vectors, as in a 16-bit cache
            const int j = i - 2 * nk, h = j / units, u = j - h * units;
            rotate_unit<T>(static_cast<const T*>(p.Q) + t * p.q_stride + h * p.D, static_cast<T*>(p.Q_out) + t * p.qo_stride + h * p.D,
                           u, row, R, p.pairs);
            continue;
        }
        const bool v = i >= nk;
        const int j = v ? i - nk : i, h = j / ng, gi = j - h * ng;
        Group g;
        g.src = (v ? static_cast<const T*>(p.V) + t * p.v_stride : static_cast<const T*>(p.K) + t * p.k_stride) + h * p.D;
        g.row = row;
        g.d0 = 16 * gi;
        g.R = v ? 0 : R;
        g.pairs = p.pairs;
        const float factor = z.factor[v ? 1 : 0];
        const bool exact = g.d0 >= g.R && (__float_as_uint(factor) & 0x7fffffu) == 0u;
        uint32_t s;
        const uint2 w = quantise(g, factor, exact, s);
        const int64_t* st = v ? p.vs : p.ks;
        const int64_t* ss = v ? z.vss : z.kss;
        uint8_t* codes = static_cast<uint8_t*>(v ? p.Vc : p.Kc) + at.page * st[0] + slot * st[1] + h * st[2] + 8 * gi;
        *reinterpret_cast<uint2*>(codes) = w;
        (v ? z.v_scales : z.k_scales)[at.page * ss[0] + h * ss[1] + slot * ng + gi] = uint8_t(s);
    }
}

// Rows out of a cache of any type: a thread takes 16 elements of a row.  p.K and p.V are the
// outputs (not const here).  Bound by its bytes.
template <int BITS>
__global__ void __launch_bounds__(kThreads) jfa_cache_read_kernel(const CacheAppendParams p, const QuantParams z) {
    const int t = blockIdx.x, lane = threadIdx.x & 31;
    const CachePlace at = cache_place(p, t, lane);
    if (at.b < 0) return;
    if (at.page < 0) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
        return;
    }
    const int slot = at.pos & ((1 << p.page_log2) - 1);
    constexpr int ES = BITS == 32 ? 4 : 2;  // bytes of an output element
    const int ng = p.D / 16, n = p.Hkv * ng;
    for (int i = threadIdx.x; i < 2 * n; i += kThreads) {
        const bool v = i >= n;
        const int j = v ? i - n : i, h = j / ng, gi = j - h * ng;
        const int64_t* st = v ? p.vs : p.ks;
        uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(const_cast<void*>(v ? p.V : p.K)) +
                                              (t * (v ? p.v_stride : p.k_stride) + h * p.D + 16 * gi) * ES);
        const int64_t from = at.page * st[0] + slot * st[1] + h * st[2];
        if constexpr (BITS == 4) {
            const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(v ? p.Vc : p.Kc) + from + 8 * gi);
            const int64_t* ss = v ? z.vss : z.kss;
            const uint32_t s = (v ? z.v_scales : z.k_scales)[at.page * ss[0] + h * ss[1] + slot * ng + gi];
            const float f = z.factor[v ? 1 : 0], sc = f16_to_float(e4m3_to_f16(s)).x;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t e[4], o[4];
                e2m1_to_f16(q ? w.y : w.x, e);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 x = f16_to_float(e[k]);
                    o[k] = pack_bf16x2(x.x * sc * f, x.y * sc * f);
                }
                dst[q] = make_uint4(o[0], o[1], o[2], o[3]);
            }
        } else {
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(v ? p.Vc : p.Kc) + (from + 16 * gi) * ES);
            uint4 x[ES];
#pragma unroll
            for (int k = 0; k < ES; ++k) x[k] = src[k];
#pragma unroll
            for (int k = 0; k < ES; ++k) dst[k] = x[k];
        }
    }
}

QuantParams quant_params(jfa_cache c) {
    QuantParams z{};
    z.k_scales = c->k_scales;
    z.v_scales = c->v_scales;
    for (int i = 0; i < 2; ++i) {
        z.kss[i] = c->kss[i];
        z.vss[i] = c->vss[i];
    }
    z.factor[0] = c->k_factor;
    z.factor[1] = c->v_factor;
    return z;
}

cudaError_t append4(jfa_cache c, CacheAppendParams p, cudaStream_t st) {
    jfa_cache_append4_kernel<<<p.T, kThreads, 0, st>>>(p, quant_params(c));
    return cudaGetLastError();
}

cudaError_t decode4(jfa_cache c, const CacheFwdParams& p, bool early, cudaStream_t st) {
    return launch_cache_decode4(c->D, c->mk, c->mv, p, early, c->num_sms, st);
}

cudaError_t chunk4(jfa_cache c, const CUtensorMap& mq, const CacheFwdParams& p, cudaStream_t st) {
    return launch_cache_chunk4(c->D, mq, c->mk, c->mv, p, c->num_sms, st);
}

const CacheOps kQuantOps = {append4, chunk4, decode4, cache_decode4_part_bytes};

// Pages of codes as bytes (D/2, slot, head, page), boxes of one page's rows (at most 64).
jfa_status make_code_map(CUtensorMap* map, const void* base, const jfa_cache_t* c, const int64_t* s) {
    const auto enc = encode_tiled();
    if (!enc) return JFA_ERR_CUDA;
    const cuuint64_t dims[4] = {cuuint64_t(c->D / 2), cuuint64_t(1) << c->page_log2, cuuint64_t(c->Hkv), cuuint64_t(c->n_pages)};
    const cuuint64_t strides[3] = {cuuint64_t(s[1]), cuuint64_t(s[2]), cuuint64_t(s[0])};
    const cuuint32_t box[4] = {cuuint32_t(c->D / 2), cuuint32_t(std::min(64, 1 << c->page_log2)), 1u, 1u};
    const cuuint32_t one[4] = {1u, 1u, 1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? JFA_OK
               : JFA_ERR_CUDA;
}

}  // namespace

}  // namespace jfa

extern "C" {

jfa_status jfa_cache_create_quantized(int32_t Hkv, int32_t D, int32_t page_size, int64_t n_pages, void* K, void* V,
                                      const int64_t* k_strides, const int64_t* v_strides, void* K_scales, void* V_scales,
                                      const int64_t* ks_strides, const int64_t* vs_strides, float k_factor, float v_factor,
                                      void* stream, jfa_cache* out) {
    if (!out) return JFA_ERR_INVALID_ARG;
    *out = nullptr;
    if (Hkv < 1 || Hkv > 65535 || n_pages < 1 || n_pages > INT32_MAX || !k_strides || !v_strides || !ks_strides || !vs_strides)
        return JFA_ERR_INVALID_ARG;
    const void* arrays[4] = {K, V, K_scales, V_scales};
    for (const void* a : arrays)
        if (!a || !aligned(a, 16)) return JFA_ERR_INVALID_ARG;
    if ((D != 64 && D != 128) || page_size < 8 || page_size > 1024 || (page_size & (page_size - 1))) return JFA_ERR_UNSUPPORTED;
    for (int i = 0; i < 3; ++i)
        for (const int64_t s : {k_strides[i], v_strides[i]})
            if (s < D / 2 || s > (int64_t(1) << 38) || s % 16 != 0) return JFA_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i)
        for (const int64_t s : {ks_strides[i], vs_strides[i]})
            if (s < int64_t(page_size) * (D / 16) || s > (int64_t(1) << 38) || s % 16 != 0) return JFA_ERR_INVALID_ARG;
    // (within these every value that a cache can hold, and its step, is a normal number)
    for (const float f : {k_factor, v_factor})
        if (!(f >= 0x1p-60f && f <= 0x1p60f)) return JFA_ERR_INVALID_ARG;
    jfa_cache_t* c = new (std::nothrow) jfa_cache_t();
    if (!c) return JFA_ERR_CUDA;
    c->dtype = JFA_BF16;
    c->ops = &kQuantOps;
    c->Hkv = Hkv;
    c->D = D;
    while ((1 << c->page_log2) < page_size) ++c->page_log2;
    c->n_pages = int32_t(n_pages);
    c->K = K;
    c->V = V;
    c->k_scales = static_cast<uint8_t*>(K_scales);
    c->v_scales = static_cast<uint8_t*>(V_scales);
    c->k_factor = k_factor;
    c->v_factor = v_factor;
    for (int i = 0; i < 3; ++i) {
        c->ks[i] = k_strides[i];
        c->vs[i] = v_strides[i];
    }
    for (int i = 0; i < 2; ++i) {
        c->kss[i] = ks_strides[i];
        c->vss[i] = vs_strides[i];
    }
    jfa_status s = check_new(c, arrays, 4);
    if (s == JFA_OK) s = make_code_map(&c->mk, K, c, c->ks);
    if (s == JFA_OK) s = make_code_map(&c->mv, V, c, c->vs);
    if (s == JFA_OK) s = make_status(c, stream);
    if (s != JFA_OK) {
        delete c;
        return s;
    }
    *out = c;
    return JFA_OK;
}

jfa_status jfa_cache_read(jfa_cache cache, int32_t B, int64_t T, const int32_t* q_offsets, const int32_t* kv_lens,
                          const int32_t* page_table, int32_t max_pages, void* K, int64_t k_stride, void* V, int64_t v_stride,
                          void* stream) {
    CacheAppendParams p{};
    const jfa_status s = check_batch(cache, B, T, q_offsets, kv_lens, page_table, max_pages, &p.max_kv);
    if (s != JFA_OK) return s;
    if (T > 0 && (!row_ok(cache, K, k_stride, cache->Hkv) || !row_ok(cache, V, v_stride, cache->Hkv))) return JFA_ERR_INVALID_ARG;
    if (!on_device(cache)) return JFA_ERR_PLAN_MISMATCH;
    if (B == 0 || T == 0) return JFA_OK;
    p.q_off = q_offsets;
    p.kv_lens = kv_lens;
    p.table = page_table;
    p.B = B;
    p.max_pages = max_pages;
    p.T = int(T);
    p.Hkv = cache->Hkv;
    p.D = cache->D;
    p.page_log2 = cache->page_log2;
    p.n_pages = cache->n_pages;
    p.K = K;
    p.V = V;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.Kc = cache->K;
    p.Vc = cache->V;
    for (int i = 0; i < 3; ++i) {
        p.ks[i] = cache->ks[i];
        p.vs[i] = cache->vs[i];
    }
    p.status = cache->d_status;
    const QuantParams z = quant_params(cache);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cache->ops)
        jfa_cache_read_kernel<4><<<p.T, kThreads, 0, st>>>(p, z);
    else if (cache->dtype == JFA_BF16)
        jfa_cache_read_kernel<16><<<p.T, kThreads, 0, st>>>(p, z);
    else
        jfa_cache_read_kernel<32><<<p.T, kThreads, 0, st>>>(p, z);
    return cudaGetLastError() == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

}  // extern "C"
