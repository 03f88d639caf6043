// fake_cuda.cpp for 4-bit caches and attention over blocks: kernels that their own files launch are logged by name
// as well (jfa_cache_read_kernel<4> as read4).  fake_cuda_blocks.cu has those behind a launch function.
#define cudaGetLastError never_an_error  // (here launches leave one)
#include "fake_cuda.cpp"
#undef cudaGetLastError

#include <cstdio>
#include <map>

#include <vector_types.h>

namespace {

cudaError_t g_last = cudaSuccess;
std::map<const void*, std::string>& kernels() {  // registered before main
    static std::map<const void*, std::string> m;
    return m;
}

}  // namespace

extern "C" {

cudaError_t fake_launched(const char* name, const char* details) {
    const cudaError_t e = launched(name);
    g_log += details;
    return e;
}

cudaError_t cudaGetLastError() {
    const cudaError_t e = g_last;
    g_last = cudaSuccess;
    return e;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return result("attribute"); }

void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, uint3*, uint3*, dim3*, dim3*, int*) {
    // .. jfa_cache_read_kernelILi4EE ..: its name, and its argument if that is a number
    std::string s = name;
    const size_t at = s.find("jfa_cache_"), end = s.find("_kernel");
    if (at == std::string::npos || end == std::string::npos) return;
    std::string base = s.substr(at + 10, end - at - 10);
    int n = 0;
    if (std::sscanf(s.c_str() + end, "_kernelILi%dE", &n) == 1) base += std::to_string(n);
    kernels()[host] = base;
}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* host) {
    *k = reinterpret_cast<cudaKernel_t>(const_cast<void*>(host));
    return cudaSuccess;
}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, CUstream_st*) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* bytes, void* stream) {
    *grid = *block = dim3();
    *bytes = 0;
    *static_cast<void**>(stream) = nullptr;
    return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3, dim3, void**, size_t, cudaStream_t) {
    return g_last = launched(kernels()[reinterpret_cast<const void*>(k)].c_str());
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* host, void**) {
    return fake_launched(kernels()[host].c_str(), c->numAttrs ? ":early" : "");
}

}  // extern "C"
