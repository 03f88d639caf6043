// A paged cache held in 4 bits: its handle, appending to it, and reading a cache back.
// Semantics are documented in include/jfa.h, the format in quant.cuh.
//
// Appending: of each 16 elements of a row y (keys rotated first, not rounded)
//   s = e4m3(max|y| / (6 c)),  code_i = e2m1(y_i / (c s)),  c the array's factor,
// each to nearest even, as if in exact arithmetic.  In fp32 the rotated y and the quotients are a
// little off, which matters only next to the middle between two codes (or scales): both ends of
// the interval that a quotient can lie in are rounded, and where they differ (one element in 10^5) the
// element is compared with the middle in 64 bits.  So a cache's contents do not depend on how
// the rotation was computed.  Elements taken as they are, with a factor that is a power of two,
// need no interval: their quotients are rounded correctly in fp32, and a bf16 value that is not
// at a middle is 2^-9 of it away or more.
// A thread takes 8 elements, two threads a group, so that a warp's loads and stores lie side by
// side; a rotated row's other halves are read again (from L1) instead of handed over.
// Bound by its arithmetic beside the stream: 24 prompts of 1-2048 tokens (32 query and 8 key heads of 128, keys
// and queries rotated) append in about 120 us, where their 612 MB take 92 at the copy rate, at 0.72 of the issue
// slots; with their rows read back 152 us, 0.76 of the copy rate.  256 single tokens with
// their reading take 7.6 us: two launches, and the chain offsets -> page -> slot in each.  (16 elements a thread,
// and whole groups compared in 64 bits where one element needed it: 182 us, 27 us.)
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

// Half a group of a row: 8 elements from d on of src (the group's from d & ~15 on), with its pairs'
// angles (R: rotated elements).
struct Half {
    const __nv_bfloat16* src;
    const float* row;
    int d, R;
    bool pairs;
};

// Element d of a rotated row in 64 bits (the products are exact there).
__device__ __forceinline__ double exact_element(const Half& g, int d) {
    const int half = g.R / 2;
    const double x = double(__bfloat162float(g.src[d]));
    if (d >= g.R) return x;
    const bool first = g.pairs ? (d & 1) == 0 : d < half;
    const int other = g.pairs ? d ^ 1 : first ? d + half : d - half, k = g.pairs ? d / 2 : first ? d : d - half;
    const double y = double(__bfloat162float(g.src[other])), c = double(g.row[k]), s = double(g.row[half + k]);
    return first ? x * c - y * s : x * c + y * s;
}

__device__ __forceinline__ float scale_value(uint32_t byte) { return f16_to_float(e4m3_to_f16(byte)).x; }

// The nearer one of neighbouring scales lo <= hi.  (The middle of two has five bits: the comparison
// is exact.)
__device__ __noinline__ uint32_t exact_scale(const Half& g, float factor, uint32_t lo, uint32_t hi) {
    double top = 0.0;
    for (int i = 0; i < 16; ++i) top = fmax(top, fabs(exact_element(g, (g.d & ~15) + i)));
    for (; lo < hi; ++lo) {
        const double mid = 0.5 * (double(scale_value(lo)) + double(scale_value(lo + 1))) * (6.0 * double(factor));
        if (!(top > mid || (top == mid && (lo & 1u)))) break;
    }
    return lo;
}

// The nearer one of codes lo .. hi of element i, for a step of factor * scale, and its sign.
__device__ __noinline__ uint32_t exact_code(const Half& g, double step, int i, uint32_t lo, uint32_t hi) {
    const double x = exact_element(g, g.d + i), y = fabs(x);
    for (; lo < hi; ++lo) {
        const double mid = lo < 4u ? 0.25 + 0.5 * lo : lo == 4u ? 2.5 : lo == 5u ? 3.5 : 5.0;
        if (!(y > mid * step || (y == mid * step && (lo & 1u)))) break;
    }
    return lo | (x < 0.0 ? 8u : 0u);
}

// A half's elements, and those of the other half of its head that a rotation pairs them with.
struct Raw {
    uint4 own, other;
};
__device__ __forceinline__ Raw load_raw(const Half& g) {
    Raw r;
    r.own = *reinterpret_cast<const uint4*>(g.src + g.d);
    const int half = g.R / 2;
    if (g.d < g.R && !g.pairs) r.other = *reinterpret_cast<const uint4*>(g.src + (g.d < half ? g.d + half : g.d - half));
    return r;
}

// Eight codes and the group's scale, by the two lanes (an even one and the next) that have its halves;
// the whole warp comes here.  exact: a row as it is and a factor that is a power of two.
__device__ __forceinline__ uint32_t quantise(const Half& g, const Raw& raw, float factor, bool exact, uint32_t& scale) {
    float y[8], slack = 0.f;
    const int half = g.R / 2;
    Vec<__nv_bfloat16> a;
    a.set(raw.own);
    if (g.d < g.R) {
        if (g.pairs) {
            float cs[4], sn[4];
            load_floats<4>(g.row + g.d / 2, cs);
            load_floats<4>(g.row + half + g.d / 2, sn);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float c = cs[i / 2], s = sn[i / 2], x = a.v[i], z = a.v[i + 1];
                a.v[i] = x * c - z * s;
                a.v[i + 1] = z * c + x * s;
                slack = fmaxf(slack, (fabsf(x) + fabsf(z)) * fmaxf(fabsf(c), fabsf(s)));
            }
        } else {
            const bool first = g.d < half;
            const int k = first ? g.d : g.d - half;
            Vec<__nv_bfloat16> b;
            b.set(raw.other);
            float cs[8], sn[8];
            load_floats<8>(g.row + k, cs);
            load_floats<8>(g.row + half + k, sn);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float u = a.v[i] * cs[i], w = (first ? -b.v[i] : b.v[i]) * sn[i];
                a.v[i] = u + w;
                slack = fmaxf(slack, fabsf(u) + fabsf(w));
            }
        }
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = a.v[i];
        top = fmaxf(top, fabsf(y[i]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    // a sum of two products is off by less than 2^-22 of their magnitudes
    slack = 0x1p-22f * fmaxf(slack, __shfl_xor_sync(0xffffffffu, slack, 1));
    const float six = 6.f * factor, over = __fdiv_rn(top, six);
    uint32_t lo, hi;
    if (exact) {
        lo = hi = to_e4m3(over, 0.f) & 255u;
    } else {
        const float e = __fdividef(slack, six);
        const uint32_t both = to_e4m3(fmaxf(fmaf(over, -0x1p-22f, over - e), 0.f), fmaf(over, 0x1p-22f, over + e));
        lo = both & 255u;
        hi = both >> 8;
    }
    if (lo != hi) lo = exact_scale(g, factor, lo, hi);
    scale = lo;
    if (lo == 0u) return 0u;
    const float step = factor * scale_value(lo), inv = __fdiv_rn(1.f, step);
    if (lo == 0x7eu) {  // the largest scale: what is over 6 steps becomes 6
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fminf(fmaxf(y[i], -8.f * step), 8.f * step);
    }
    if (exact) {
        // Quotients rounded correctly: with the reciprocal so rounded, one step on the remainder makes
        // them so (Markstein, IBM J. Res. Dev. 34, 1990).
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float t = y[i] * inv;
            y[i] = fmaf(fmaf(-t, step, y[i]), inv, t);
        }
        return to_e2m1(y);
    }
    // Quotients are below 9 (the smallest scale stands for up to 1.5 times itself, the others for less), and off
    // by less than 2^-19 besides: the step's and its reciprocal's roundings, 2^-24 of them each, and one of 2^-21.
    const float e = fmaf(slack, inv * 1.0001f, 0x1p-19f);
    float above[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        above[i] = fmaf(y[i], inv, e);
        y[i] = fmaf(y[i], inv, -e);
    }
    uint32_t w = to_e2m1(y);
    const uint32_t x = to_e2m1(above);
    // elements next to a middle: other magnitudes, or other signs of one that is not 0
    const uint32_t other = w ^ x, some = ((w | x) & 0x77777777u) + 0x77777777u;
    for (uint32_t differ = (other & 0x77777777u) | (other & some & 0x88888888u); differ;) {
        const int at = (__ffs(differ) - 1) & 28;
        differ &= ~(15u << at);
        const uint32_t p = (w >> at) & 7u, q = (x >> at) & 7u;
        const bool across = (other >> at) & 8u;
        const uint32_t code = exact_code(g, double(factor) * double(scale_value(lo)), at / 4, across ? 0u : min(p, q), max(p, q));
        w = (w & ~(15u << at)) | (code << at);
    }
    return w;
}

__device__ __forceinline__ bool power_of_two(float f) { return (__float_as_uint(f) & 0x7fffffu) == 0u; }

__global__ void __launch_bounds__(kThreads) jfa_cache_append4_kernel(const CacheAppendParams p, const QuantParams z) {
    using T = __nv_bfloat16;
    const int t = blockIdx.x, lane = threadIdx.x & 31;
    const int vl = p.D == 128 ? 4 : 3, vecs = 1 << vl, nk = p.Hkv << vl;  // vectors of a head, of all key heads
    const int R = p.rot ? p.rot_dim : 0;
    // the vector of a thread in the loops over key heads (past the end: one of the warp's own, again)
    auto vec = [&](int i0) { return i0 + lane < nk ? i0 + lane : i0 + (lane & 1); };
    auto half_of = [&](int i, bool v, const float* row) {
        const T* src = v ? static_cast<const T*>(p.V) + t * p.v_stride : static_cast<const T*>(p.K) + t * p.k_stride;
        return Half{src + (i >> vl) * p.D, row, 8 * (i & (vecs - 1)), v ? 0 : R, p.pairs != 0};
    };
    // rows lie where the token's number says: the first ones are on their way while its place is found
    const int first = threadIdx.x - lane;
    Raw rk{}, rv{};
    if (first < nk) {
        rk = load_raw(half_of(vec(first), false, nullptr));
        rv = load_raw(half_of(vec(first), true, nullptr));
    }
    const CachePlace at = cache_place(p, t, lane);
    if (at.b < 0) return;  // rows behind the last sequence
    if (at.page < 0) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
        return;
    }
    const int slot = at.pos & ((1 << p.page_log2) - 1);
    const float* row = p.rot ? p.rot + size_t(at.pos) * size_t(p.rot_dim) : nullptr;
    // query heads' vectors, as beside a 16-bit cache, two at a time
    const int units = p.pairs ? vecs : vecs - R / 16, nq = p.H * units;
    for (int i = threadIdx.x; i < nq; i += 2 * kThreads) {
        const T* src[2];
        T* dst[2];
        int u[2];
        Raw r[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int j = i + k * kThreads, h = j / units;
            u[k] = j - h * units;
            src[k] = static_cast<const T*>(p.Q) + t * p.q_stride + h * p.D;
            dst[k] = static_cast<T*>(p.Q_out) + t * p.qo_stride + h * p.D;
            if (j < nq) {
                const bool copied = !p.pairs && 16 * u[k] >= R;
                r[k].own = *reinterpret_cast<const uint4*>(src[k] + 8 * u[k] + (copied ? R / 2 : 0));
                if (!p.pairs && !copied) r[k].other = *reinterpret_cast<const uint4*>(src[k] + 8 * u[k] + R / 2);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (i + k * kThreads < nq) rotate_vectors<T>(r[k].own, r[k].other, dst[k], u[k], row, R, p.pairs);
    }
    for (int i0 = first; i0 < nk; i0 += kThreads) {
        const int i = vec(i0), h = i >> vl, u = i & (vecs - 1);
        const Half gk = half_of(i, false, row), gv = half_of(i, true, nullptr);
        if (i0 != first) {
            rk = load_raw(gk);
            rv = load_raw(gv);
        }
        uint32_t sk, sv;
        const uint32_t wk = quantise(gk, rk, z.factor[0], gk.d >= R && power_of_two(z.factor[0]), sk);
        if (i0 + lane < nk) {
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.Kc) + at.page * p.ks[0] + slot * p.ks[1] + h * p.ks[2] + 4 * u) = wk;
            if (!(u & 1)) z.k_scales[at.page * z.kss[0] + h * z.kss[1] + ((slot << vl) + u) / 2] = uint8_t(sk);
        }
        const uint32_t wv = quantise(gv, rv, z.factor[1], power_of_two(z.factor[1]), sv);
        if (i0 + lane < nk) {
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.Vc) + at.page * p.vs[0] + slot * p.vs[1] + h * p.vs[2] + 4 * u) = wv;
            if (!(u & 1)) z.v_scales[at.page * z.vss[0] + h * z.vss[1] + ((slot << vl) + u) / 2] = uint8_t(sv);
        }
    }
}

// a f, cut to 24 bits with the last one set where something was cut off: it rounds to bf16 as the
// product itself would.
__device__ __forceinline__ float odd_product(float a, float f) {
    const float x = __fmul_rz(a, f);
    return __fmaf_rn(a, f, -x) != 0.f ? __uint_as_float(__float_as_uint(x) | 1u) : x;
}

// Rows out of a cache of any type: a thread takes 16 bytes of an output row.  p.K and p.V are the outputs
// (not const here).
template <int BITS>
__global__ void __launch_bounds__(kThreads) jfa_cache_read_kernel(const CacheAppendParams p, const QuantParams z) {
    constexpr int ES = BITS == 32 ? 4 : 2, N = 16 / ES;  // bytes of an output element, elements of a vector
    const int t = blockIdx.x, lane = threadIdx.x & 31;
    const CachePlace at = cache_place(p, t, lane);
    if (at.b < 0) return;
    if (at.page < 0) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
        return;
    }
    const int slot = at.pos & ((1 << p.page_log2) - 1), vl = 31 - __clz(p.D / N), vecs = 1 << vl, n = p.Hkv << vl;
    for (int i = threadIdx.x; i < n; i += kThreads) {  // a vector of K and the same of V
        const int h = i >> vl, u = i & (vecs - 1);
        const int64_t from[2] = {at.page * p.ks[0] + slot * p.ks[1] + h * p.ks[2], at.page * p.vs[0] + slot * p.vs[1] + h * p.vs[2]};
        const int64_t to[2] = {(t * p.k_stride + h * p.D) * ES + 16 * u, (t * p.v_stride + h * p.D) * ES + 16 * u};
        uint4 x[2];
        if constexpr (BITS == 4) {
            uint32_t w[2], s[2];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int64_t* ss = v ? z.vss : z.kss;
                w[v] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(v ? p.Vc : p.Kc) + from[v] + 4 * u);
                s[v] = (v ? z.v_scales : z.k_scales)[at.page * ss[0] + h * ss[1] + ((slot << vl) + u) / 2];
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const float f = z.factor[v], sc = scale_value(s[v]);
                const bool exact = power_of_two(f);
                uint32_t e[4], o[4];
                e2m1_to_f16(w[v], e);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 y = f16_to_float(e[j]);
                    o[j] = exact ? pack_bf16x2(y.x * sc * f, y.y * sc * f) : pack_bf16x2(odd_product(y.x * sc, f), odd_product(y.y * sc, f));
                }
                x[v] = make_uint4(o[0], o[1], o[2], o[3]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < 2; ++v)
                x[v] = *reinterpret_cast<const uint4*>(static_cast<const char*>(v ? p.Vc : p.Kc) + from[v] * ES + 16 * u);
        }
#pragma unroll
        for (int v = 0; v < 2; ++v) *reinterpret_cast<uint4*>(static_cast<char*>(const_cast<void*>(v ? p.V : p.K)) + to[v]) = x[v];
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
