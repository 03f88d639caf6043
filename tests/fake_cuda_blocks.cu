// Launches of the 4-bit cache's attention and of attention over blocks, logged with what the host has chosen for
// them (fake_cuda_blocks.cpp).  No kernel of this file's own, and no address is dereferenced.
#include <string>

#include "cache_common.cuh"

extern "C" cudaError_t fake_launched(const char* name, const char* details);

namespace {

float g_scale_log2 = 0.f;

cudaError_t attention(const char* name, const jfa::CacheFwdParams& p, bool early) {
    g_scale_log2 = p.scale_log2;
    return fake_launched(name, (":" + std::to_string(p.bm) + (early ? ":early" : "")).c_str());
}

}  // namespace

namespace jfa {

size_t cache_decode4_part_bytes(int, int) { return 4096; }
cudaError_t launch_cache_decode4(int, const CUtensorMap&, const CUtensorMap&, const CacheFwdParams& p, bool early, int, cudaStream_t) {
    return attention(p.lists ? "lists4" : "decode4", p, early);
}
cudaError_t launch_cache_decode_lists(int, const CUtensorMap&, const CUtensorMap&, const CacheFwdParams& p, int, cudaStream_t) {
    return attention("lists", p, false);
}
cudaError_t launch_cache_chunk4(int, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CacheFwdParams& p, int,
                                cudaStream_t) {
    return attention("chunk4", p, false);
}

}  // namespace jfa

extern "C" {

// The factor of the scores, in log2 units, that the last attention was launched with.
float fake_scale_log2() { return g_scale_log2; }

}  // extern "C"
