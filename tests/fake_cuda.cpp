// A stand-in for the CUDA runtime and for the paged cache's kernel launches, for host tests:
// the library's own cache.cu runs against it on a machine without a GPU.  Every launch and
// memset is logged by name, and any call can be made to fail.  No address is dereferenced.
#include <cuda.h>
#include <cuda_runtime_api.h>

#include <cstring>
#include <string>

namespace {

std::string g_log, g_fail;

bool fails(const char* name) { return g_fail == name; }
cudaError_t result(const char* name) { return fails(name) ? cudaErrorLaunchFailure : cudaSuccess; }
cudaError_t launched(const char* name) {
    g_log += (g_log.empty() ? "" : " ") + std::string(name) + (fails(name) ? "!" : "");
    return result(name);
}

CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    return fails("encode") ? CUDA_ERROR_INVALID_VALUE : CUDA_SUCCESS;
}

}  // namespace

namespace jfa {

struct CacheFwdParams;
struct CacheAppendParams;

bool supported(int, int) { return true; }
size_t cache_simt_part_bytes(int, int) { return 1024; }
size_t cache_split_part_bytes(int, int) { return 1024; }
size_t cache_decode_part_bytes(int, int) { return 1024; }
size_t cache_chunk_part_bytes(int, int) { return 1024; }
cudaError_t launch_cache_append(int, const CacheAppendParams&, cudaStream_t) { return launched("append"); }
cudaError_t launch_cache_split(int, const CUtensorMap&, const CUtensorMap&, const CacheFwdParams&, int, cudaStream_t) {
    return launched("split");
}
cudaError_t launch_cache_simt(int, const CacheFwdParams&, bool, int, cudaStream_t) { return launched("simt"); }
cudaError_t launch_cache_decode(int, const CUtensorMap&, const CUtensorMap&, const CacheFwdParams&, bool, int, cudaStream_t) {
    return launched("decode");
}
cudaError_t launch_cache_chunk(int, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CacheFwdParams&, int,
                               cudaStream_t) {
    return launched("chunk");
}
cudaError_t launch_cache_merge(int, const CacheFwdParams&, int, int, cudaStream_t) { return launched("merge"); }

}  // namespace jfa

extern "C" {

// The log since the last call of this; from here on the call `fail` fails ("": none).
const char* fake_log(const char* fail) {
    static std::string last;
    last = g_log;
    g_log.clear();
    g_fail = fail;
    return last.c_str();
}

cudaError_t cudaGetDevice(int* d) {
    *d = 0;
    return cudaSuccess;
}
cudaError_t cudaGetDeviceProperties(cudaDeviceProp* p, int) {
    std::memset(p, 0, sizeof(*p));
    p->major = 10;
    p->multiProcessorCount = 152;
    return cudaSuccess;
}
// addresses from 2^40 on belong to device 1, those from 2^41 on to no device
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes* a, const void* p) {
    std::memset(a, 0, sizeof(*a));
    const uintptr_t v = reinterpret_cast<uintptr_t>(p);
    a->type = v >> 41 ? cudaMemoryTypeUnregistered : cudaMemoryTypeDevice;
    a->device = v >> 41 ? -2 : int(v >> 40);
    return result("attributes");
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaMalloc(void** p, size_t) {
    *p = reinterpret_cast<void*>(uintptr_t(4096));
    return cudaSuccess;
}
cudaError_t cudaFree(void*) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t) {
    return launched(("memset(" + std::to_string(uintptr_t(p)) + "," + std::to_string(v) + "," + std::to_string(n) + ")").c_str());
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned int, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
    *f = reinterpret_cast<void*>(&encode);
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
// the device code's registration: there is none to load
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}

}  // extern "C"
