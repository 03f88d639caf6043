// The paged cache's handle and the host code its entry points share.
#pragma once

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "cache_common.cuh"

namespace jfa {

// What a cache held in 4 bits does in place of the 16- and 32-bit kernels.
struct CacheOps {
    cudaError_t (*append)(jfa_cache c, CacheAppendParams p, cudaStream_t st);
    cudaError_t (*chunk)(jfa_cache c, const CUtensorMap& mq, const CacheFwdParams& p, cudaStream_t st);
    cudaError_t (*decode)(jfa_cache c, const CacheFwdParams& p, bool early, cudaStream_t st);
    size_t (*decode_part_bytes)(int D, int num_sms);
};

}  // namespace jfa

struct jfa_cache_t {
    int32_t dtype, Hkv, D, page_log2, n_pages;  // dtype: of the rows appended and attended with
    void* K;
    void* V;
    int64_t ks[3], vs[3];
    int device, num_sms;
    int* d_status;
    CUtensorMap mk, mv;  // the pages as (D, slot, head, page), boxes of one page's keys (at most 64)
    const jfa::CacheOps* ops;  // nullptr: K and V hold elements of dtype
    // 4 bits: K and V hold codes, D/2 bytes a row (strides in bytes), and a scale byte for 16 elements
    uint8_t *k_scales, *v_scales;
    int64_t kss[2], vss[2];  // page, head
    float k_factor, v_factor;
};

namespace jfa {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t elem(int dtype) { return dtype == JFA_F32 ? 4 : 2; }

// The driver's encoder of tensor maps, or nullptr.  (Not inline: a static variable of an inline function is one for all
// libraries of a process, such as this one and a stand-in for its runtime.)
PFN_cuTensorMapEncodeTiled_v12000 encode_tiled();

// Whether the cache's device is the current one.
inline bool on_device(jfa_cache c) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == c->device;
}

// Checks of the arrays that the calls of a step take; max_kv: the longest sequence they can address.
inline jfa_status check_batch(jfa_cache c, int32_t B, int64_t T, const int32_t* q_offsets, const int32_t* kv_lens,
                       const int32_t* page_table, int32_t max_pages, int32_t* max_kv) {
    if (!c || B < 0 || B > kCacheMaxB || T < 0 || T > (1 << 30) || max_pages < 0) return JFA_ERR_INVALID_ARG;
    if (!aligned(q_offsets, 4) || !aligned(kv_lens, 4) || !aligned(page_table, 4)) return JFA_ERR_INVALID_ARG;
    if (B > 0 && (!q_offsets || !kv_lens || (max_pages > 0 && !page_table))) return JFA_ERR_INVALID_ARG;
    *max_kv = int32_t(std::min<int64_t>(int64_t(max_pages) << c->page_log2, INT32_MAX - T - kPositionRoom));
    return JFA_OK;
}

// [T, heads, D] rows `stride` elements apart.
inline bool row_ok(jfa_cache c, const void* p, int64_t stride, int32_t heads) {
    return p && aligned(p, 16) && stride >= int64_t(heads) * c->D && (size_t(stride) * elem(c->dtype)) % 16 == 0;
}

// Checks of a new handle's device and arrays, which it fills in from them.
inline jfa_status check_new(jfa_cache_t* c, const void* const* arrays, int n) {
    cudaDeviceProp prop;
    if (cudaGetDevice(&c->device) != cudaSuccess || cudaGetDeviceProperties(&prop, c->device) != cudaSuccess || prop.major != 10 ||
        prop.multiProcessorCount > kMaxSms)
        return JFA_ERR_NO_DEVICE;
    c->num_sms = prop.multiProcessorCount;
    // (an address that CUDA does not know, or memory of no one device, is the caller's matter)
    for (int i = 0; i < n; ++i) {
        cudaPointerAttributes at;
        if (cudaPointerGetAttributes(&at, arrays[i]) != cudaSuccess)
            (void)cudaGetLastError();
        else if (at.type == cudaMemoryTypeDevice && at.device != c->device)
            return JFA_ERR_INVALID_ARG;
    }
    return JFA_OK;
}

// The handle's status word.
inline jfa_status make_status(jfa_cache_t* c, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaMalloc(reinterpret_cast<void**>(&c->d_status), 256) != cudaSuccess) return JFA_ERR_CUDA;
    if (cudaMemsetAsync(c->d_status, 0, 256, st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess) {
        cudaFree(c->d_status);
        return JFA_ERR_CUDA;
    }
    return JFA_OK;
}

constexpr size_t kCutBytes = size_t(kMaxSms) * kBlocksPerCta * sizeof(CacheCut);
constexpr int kDecodeRows = 16;  // one row tile of the decode kernel
// What an item's start and end cost the decode kernel, in its stages of 32 KB: about 4 us of a
// CTA, at its share of the memory's rate (one history of 131k keys: 100.5 us with 2, 97 with 3, 96
// with 4; 200 sequences of up to 2k keys: 102 with 1, 93 with 2, 95 with 3, 98 with 5).  Beside
// the chunk kernel, on SMs that come free at different times, less (256 ragged query sets: 248.5
// us with 3 and with 5, 244 with 2 and with 1).  And the chunk and split kernels, in their steps
// of 128 keys: 1.8-2.6 us (48 sequences, nine of them prompts: 71 us with 2, 66.5 with 3, 70.5 with
// 5) and 2.5 us (20 ragged sequences: 74.4 with 2, 75.6 with 3, 78.4 with 5); the simt kernel, in
// its steps of 64 keys, the same 2 (64 fp32 single tokens: 109-114 us with 1 to 4, 118 with 6).
// The 4-bit kernel, in its stages of 128 keys (1.7 us): 64 histories 68.6 us with 1, 67.4 with 2, 68.7 with 3, 73.5
// with 6; 64 lists of blocks 36.4, 36.7, 38.7 and 38.8.
constexpr int kDecodeItemUnits = 3, kDecodeItemUnitsBeside = 2, kSimtItemUnits = 2, kDecode4ItemUnits = 2;
constexpr int kChunkItemUnits = 3;
constexpr int kSplitItemUnits = 2;

// The parameters of an attention call that do not depend on its kernels.
inline void fwd_params(CacheFwdParams& p, jfa_cache cache, int32_t B, int64_t T, const int32_t* q_offsets, const int32_t* kv_lens,
                       const int32_t* page_table, int32_t max_pages, int32_t max_kv, const void* Q, int64_t q_stride, int32_t H,
                       int32_t causal, int32_t window, const float* bias, float scale, void* O, int32_t o_dtype, float* lse,
                       void* workspace) {
    p.q_off = q_offsets;
    p.kv_lens = kv_lens;
    p.table = page_table;
    p.B = B;
    p.max_pages = max_pages;
    p.T = int(T);
    p.max_kv = max_kv;
    p.H = H;
    p.Hkv = cache->Hkv;
    p.g = H / cache->Hkv;
    set_div_g(p);
    p.page_log2 = cache->page_log2;
    p.n_pages = cache->n_pages;
    p.causal = causal;
    p.window = window < max_kv ? window : -1;  // a window of every position is none
    // (the factor first: it is the product that the calls check to be a normal number)
    p.scale_log2 = (cache->ops ? scale * cache->k_factor : scale) * 1.4426950408889634f;
    p.bias = bias;
    p.Q = Q;
    p.q_stride = q_stride;
    p.O = O;
    p.o_f32 = o_dtype == JFA_F32;
    p.o_mul = 1.f;
    p.lse = lse;
    p.K = cache->K;
    p.V = cache->V;
    for (int i = 0; i < 3; ++i) {
        p.ks[i] = cache->ks[i];
        p.vs[i] = cache->vs[i];
    }
    if (cache->ops) {
        p.o_mul = cache->v_factor;
        p.k_scales = cache->k_scales;
        p.v_scales = cache->v_scales;
        p.dense = cache->ks[1] == cache->D / 2 && cache->vs[1] == cache->D / 2;
        for (int i = 0; i < 2; ++i) {
            p.kss[i] = cache->kss[i];
            p.vss[i] = cache->vss[i];
        }
    }
    p.counters = static_cast<uint32_t*>(workspace);
    p.cut_flags = p.counters + kCtrCuts;
    p.cuts = reinterpret_cast<CacheCut*>(static_cast<char*>(workspace) + JFA_CACHE_ZERO_BYTES);
    p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + JFA_CACHE_ZERO_BYTES + kCutBytes);
    p.status = cache->d_status;
    p.row_lo = 0;
    p.row_hi = INT32_MAX;
}

}  // namespace jfa
