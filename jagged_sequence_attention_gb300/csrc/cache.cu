// C-ABI of the paged key/value cache: argument checks, the handle, and kernel launches.
// Semantics of every entry point are documented in include/jfa.h.
#include <new>

#include "cache_handle.h"

using namespace jfa;

PFN_cuTensorMapEncodeTiled_v12000 jfa::encode_tiled() {
    static PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(e == cudaSuccess && q == cudaDriverEntryPointSuccess ? f
                                                                                                             : nullptr);
    }();
    return enc;
}

namespace {

// A tensor of `rank` dimensions (the first dense, strides of the others in elements), its boxes
// 128 bytes of the first, with 128-byte swizzle.
jfa_status make_map(CUtensorMap* map, int dtype, const void* base, int rank, const cuuint64_t* dims, const int64_t* strides,
                         const cuuint32_t* box) {
    const auto enc = encode_tiled();
    if (!enc) return JFA_ERR_CUDA;
    cuuint64_t bytes[3];
    for (int i = 0; i + 1 < rank; ++i) bytes[i] = cuuint64_t(strides[i]) * elem(dtype);
    const cuuint32_t one[4] = {1u, 1u, 1u, 1u};
    return enc(map, dtype == JFA_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cuuint32_t(rank), const_cast<void*>(base), dims, bytes, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               dims[0] * elem(dtype) >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? JFA_OK
               : JFA_ERR_CUDA;
}

// The pages by their strides, as (D, slot, head, page), boxes of `rows` slots.
jfa_status make_page_map(CUtensorMap* map, const void* base, const jfa_cache_t* c, const int64_t* s, int rows) {
    const cuuint64_t dims[4] = {cuuint64_t(c->D), cuuint64_t(1) << c->page_log2, cuuint64_t(c->Hkv), cuuint64_t(c->n_pages)};
    const int64_t strides[3] = {s[1], s[2], s[0]};
    const cuuint32_t box[4] = {cuuint32_t(128 / elem(c->dtype)), cuuint32_t(rows), 1u, 1u};
    return make_map(map, c->dtype, base, 4, dims, strides, box);
}

}  // namespace

extern "C" {

jfa_status jfa_cache_create(int32_t dtype, int32_t Hkv, int32_t D, int32_t page_size, int64_t n_pages, void* K, void* V,
                            const int64_t* k_strides, const int64_t* v_strides, void* stream, jfa_cache* out) {
    if (!out) return JFA_ERR_INVALID_ARG;
    *out = nullptr;
    if (dtype != JFA_BF16 && dtype != JFA_F32) return JFA_ERR_INVALID_ARG;
    if (Hkv < 1 || Hkv > 65535 || n_pages < 1 || n_pages > INT32_MAX || !K || !V || !k_strides || !v_strides ||
        !aligned(K, 16) || !aligned(V, 16))
        return JFA_ERR_INVALID_ARG;
    if (!supported(dtype, D) || page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)))
        return JFA_ERR_UNSUPPORTED;
    for (int i = 0; i < 3; ++i)
        for (const int64_t s : {k_strides[i], v_strides[i]})
            if (s < D || s > (int64_t(1) << 38) || (size_t(s) * elem(dtype)) % 16 != 0) return JFA_ERR_INVALID_ARG;
    jfa_cache_t* c = new (std::nothrow) jfa_cache_t();
    if (!c) return JFA_ERR_CUDA;
    c->dtype = dtype;
    c->Hkv = Hkv;
    c->D = D;
    while ((1 << c->page_log2) < page_size) ++c->page_log2;
    c->n_pages = int32_t(n_pages);
    c->K = K;
    c->V = V;
    for (int i = 0; i < 3; ++i) {
        c->ks[i] = k_strides[i];
        c->vs[i] = v_strides[i];
    }
    const void* arrays[2] = {K, V};
    jfa_status s = check_new(c, arrays, 2);
    const int rows = std::min(64, page_size);
    if (s == JFA_OK) s = make_page_map(&c->mk, K, c, c->ks, rows);
    if (s == JFA_OK) s = make_page_map(&c->mv, V, c, c->vs, rows);
    if (s == JFA_OK) s = make_status(c, stream);
    if (s != JFA_OK) {
        delete c;
        return s;
    }
    *out = c;
    return JFA_OK;
}

jfa_status jfa_cache_destroy(jfa_cache cache) {
    if (!cache) return JFA_OK;
    const cudaError_t e = cudaFree(cache->d_status);
    delete cache;
    return e == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

jfa_status jfa_cache_device_status(jfa_cache cache, void* stream) {
    if (!cache) return JFA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int h = 0;
    if (cudaMemcpyAsync(&h, cache->d_status, 4, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaMemsetAsync(cache->d_status, 0, 4, st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
        return JFA_ERR_CUDA;
    if (h & kStatusTimeout) return JFA_ERR_TIMEOUT;
    if (h & kStatusBounds) return JFA_ERR_DEVICE_BOUNDS;
    return JFA_OK;
}

jfa_status jfa_cache_append(jfa_cache cache, int32_t B, int64_t T, const int32_t* q_offsets, const int32_t* kv_lens,
                            const int32_t* page_table, int32_t max_pages, const void* K, int64_t k_stride, const void* V,
                            int64_t v_stride, const void* Q, int64_t q_stride, int32_t H, void* Q_out, int64_t qo_stride,
                            const float* rot, int32_t rot_dim, int64_t rot_len, int32_t rot_kind, void* stream) {
    int32_t max_kv = 0;
    const jfa_status s = check_batch(cache, B, T, q_offsets, kv_lens, page_table, max_pages, &max_kv);
    if (s != JFA_OK) return s;
    if ((Q == nullptr) != (Q_out == nullptr) || (Q && (H < 1 || H > 65535)) || (Q && !rot)) return JFA_ERR_INVALID_ARG;
    if (rot && (rot_dim < 16 || rot_dim > cache->D || rot_dim % 16 != 0 || rot_len < 1 || !aligned(rot, 16) ||
                (rot_kind != JFA_ROT_HALF && rot_kind != JFA_ROT_PAIRS)))
        return JFA_ERR_INVALID_ARG;
    if (T > 0 && (!row_ok(cache, K, k_stride, cache->Hkv) || !row_ok(cache, V, v_stride, cache->Hkv)))
        return JFA_ERR_INVALID_ARG;
    if (T > 0 && Q && (!row_ok(cache, Q, q_stride, H) || !row_ok(cache, Q_out, qo_stride, H)))
        return JFA_ERR_INVALID_ARG;
    if (T > 0 && Q && Q == Q_out && q_stride != qo_stride) return JFA_ERR_INVALID_ARG;
    if (!on_device(cache)) return JFA_ERR_PLAN_MISMATCH;
    if (B == 0 || T == 0) return JFA_OK;
    CacheAppendParams p;
    p.q_off = q_offsets;
    p.kv_lens = kv_lens;
    p.table = page_table;
    p.B = B;
    p.max_pages = max_pages;
    p.T = int(T);
    p.max_kv = max_kv;
    p.H = Q ? H : 0;
    p.Hkv = cache->Hkv;
    p.D = cache->D;
    p.page_log2 = cache->page_log2;
    p.n_pages = cache->n_pages;
    p.K = K;
    p.V = V;
    p.Q = Q;
    p.Q_out = Q_out;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_stride = q_stride;
    p.qo_stride = qo_stride;
    p.Kc = cache->K;
    p.Vc = cache->V;
    for (int i = 0; i < 3; ++i) {
        p.ks[i] = cache->ks[i];
        p.vs[i] = cache->vs[i];
    }
    p.rot = rot;
    p.rot_dim = rot_dim;
    p.rot_len = int(std::min<int64_t>(rot_len, INT32_MAX));
    p.pairs = rot_kind == JFA_ROT_PAIRS;
    p.status = cache->d_status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = cache->ops ? cache->ops->append(cache, p, st) : launch_cache_append(cache->dtype, p, st);
    return e == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

size_t jfa_cache_workspace_size(jfa_cache cache, int32_t H) {
    if (!cache || H < 1 || H > 65535 || H % cache->Hkv != 0) return 0;
    const int D = cache->D, n = cache->num_sms;
    if (cache->dtype == JFA_F32)
        return JFA_CACHE_ZERO_BYTES + kCutBytes + cache_simt_part_bytes(D, n) + cache_split_part_bytes(D, n);
    return JFA_CACHE_ZERO_BYTES + kCutBytes + cache_chunk_part_bytes(D, n) +
           std::max(cache_decode_part_bytes(D, n), cache->ops ? cache->ops->decode_part_bytes(D, n) : 0);
}

jfa_status jfa_cache_fwd(jfa_cache cache, int32_t B, int64_t T, int32_t max_q_len, const int32_t* q_offsets,
                         const int32_t* kv_lens, const int32_t* page_table, int32_t max_pages, const void* Q,
                         int64_t q_stride, int32_t H, int32_t causal, int32_t window, int32_t bias_kind,
                         const float* bias_table, float scale, void* O, int32_t o_dtype, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
    int32_t max_kv = 0;
    const jfa_status s = check_batch(cache, B, T, q_offsets, kv_lens, page_table, max_pages, &max_kv);
    if (s != JFA_OK) return s;
    if (H < 1 || H > 65535 || H % cache->Hkv != 0 || T * H > INT32_MAX - 256 || max_q_len < 0) return JFA_ERR_INVALID_ARG;
    if (cache->dtype == JFA_BF16 && H / cache->Hkv > 128) return JFA_ERR_UNSUPPORTED;  // a token's rows fill one tile
    if ((causal != 0 && causal != 1) || window < -1 || (window >= 0 && causal != 1)) return JFA_ERR_INVALID_ARG;
    if (bias_kind != JFA_BIAS_NONE && bias_kind != JFA_BIAS_RELPOS32)
        return bias_kind == JFA_BIAS_DENSE ? JFA_ERR_UNSUPPORTED : JFA_ERR_INVALID_ARG;
    if (bias_kind == JFA_BIAS_RELPOS32 && (!bias_table || !aligned(bias_table, 4))) return JFA_ERR_INVALID_ARG;
    if (!(scale > 0.f && scale < INFINITY)) return JFA_ERR_INVALID_ARG;
    // (the keys' factor goes into the scores' scale, which has to stay a normal number)
    if (cache->ops && !(scale * cache->k_factor >= 1e-37f && scale * cache->k_factor <= 1e37f)) return JFA_ERR_INVALID_ARG;
    if (o_dtype != JFA_BF16 && o_dtype != JFA_F32) return JFA_ERR_INVALID_ARG;
    if (cache->dtype == JFA_F32 && o_dtype != JFA_F32) return JFA_ERR_UNSUPPORTED;
    if (T > 0 && (!row_ok(cache, Q, q_stride, H) || !O || O == Q || !aligned(O, 16) || !aligned(lse, 4))) return JFA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < jfa_cache_workspace_size(cache, H))
        return JFA_ERR_INVALID_ARG;
    if (!on_device(cache)) return JFA_ERR_PLAN_MISMATCH;
    if (B == 0 || T == 0) return JFA_OK;
    CacheFwdParams p{};
    fwd_params(p, cache, B, T, q_offsets, kv_lens, page_table, max_pages, max_kv, Q, q_stride, H, causal, window,
               bias_kind == JFA_BIAS_RELPOS32 ? bias_table : nullptr, scale, O, o_dtype, lse, workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // Sequences of at most kDecodeRows packed rows run in the decode kernel, the others in the
    // chunk kernel; which there are is known on the device only, beyond max_q_len.
    const int n = cache->num_sms, D = cache->D;
    const bool bf16 = cache->dtype == JFA_BF16;
    const int64_t most_rows = (max_q_len > 0 ? std::min<int64_t>(max_q_len, T) : T) * p.g;
    const bool chunks = most_rows > kDecodeRows;
    // the kernels count units in 31 bits; tiles(): the row tiles of bm rows that `rows` rows have at most
    auto tiles = [&](int64_t rows, int bm) { return rows / bm + B; };
    auto fits = [&](int64_t n_tiles, int bn) {
        return double(n_tiles) * p.Hkv * (double(max_kv) / bn + 16.0) < double(INT32_MAX) - 65536.0;
    };
    // Every check of both kernels comes before the first launch: a refused call does nothing.
    CacheFwdParams pc = p;  // the chunk kernel's parameters, and the merge's
    CUtensorMap mq;
    if (chunks) {
        pc.row_lo = kDecodeRows;
        pc.bm = 128;
        pc.item_cost = kSplitItemUnits;
        pc.min_units = 1;
        if (bf16) {
            pc.tile_tokens = 128 / p.g;
            pc.bm = 2 * pc.tile_tokens * p.g;
            pc.item_cost = kChunkItemUnits;
            pc.min_units = kChunkItemUnits + 1;
        }
        if (!fits(tiles(T * p.g, pc.bm), 128)) return JFA_ERR_UNSUPPORTED;
        p.row_hi = kDecodeRows;
    }
    p.bm = bf16 || p.g > 4 ? 16 : 4;
    if (cache->ops && most_rows <= 8) p.bm = 8;
    p.min_units = 1;
    p.item_cost = !bf16 ? kSimtItemUnits : cache->ops ? kDecode4ItemUnits : chunks ? kDecodeItemUnitsBeside : kDecodeItemUnits;
    if (!fits(chunks ? int64_t(B) * (kDecodeRows / p.bm) : tiles(T * p.g, p.bm), 64)) return JFA_ERR_UNSUPPORTED;
    // (the two kernels may run at once, and the merge comes last)
    p.part += (bf16 ? cache_chunk_part_bytes(D, n) : cache_split_part_bytes(D, n)) / sizeof(float);
    if (chunks && bf16) {  // the queries as (D, head, token), boxes of one tile's rows
        const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(H), cuuint64_t(T)};
        const int64_t strides[2] = {D, q_stride};
        const cuuint32_t box[3] = {64u, cuuint32_t(p.g), cuuint32_t(pc.tile_tokens)};
        const jfa_status ms = make_map(&mq, JFA_BF16, Q, 3, dims, strides, box);
        if (ms != JFA_OK) return ms;
    }
    cudaError_t e = cudaSuccess;
    if (cache->ops) {
        if (chunks) e = cache->ops->chunk(cache, mq, pc, st);
        if (e == cudaSuccess) e = cache->ops->decode(cache, p, chunks, st);
    } else {
        if (chunks)
            e = bf16 ? launch_cache_chunk(D, mq, cache->mk, cache->mv, pc, n, st) : launch_cache_split(D, cache->mk, cache->mv, pc, n, st);
        if (e == cudaSuccess)
            e = bf16 ? launch_cache_decode(D, cache->mk, cache->mv, p, chunks, n, st) : launch_cache_simt(D, p, chunks, n, st);
    }
    if (chunks) {
        // The chunk kernel's flags of cut items are the merge's to clear, so it follows whatever
        // failed before it; where it fails itself they are cleared here.
        const cudaError_t em = launch_cache_merge(D, pc, bf16 ? n * kBlocksPerCta : n, n, st);
        if (em != cudaSuccess) (void)cudaMemsetAsync(workspace, 0, JFA_CACHE_ZERO_BYTES, st);
        if (e == cudaSuccess) e = em;
    }
    return e == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

}  // extern "C"
