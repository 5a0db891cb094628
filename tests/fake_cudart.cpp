// A CUDA runtime that runs nothing and writes down what the library asks of it, for the tests of launch
// choices and refusals that need no GPU.  Loaded with global symbols in front of libspkv.so, in a process of
// its own.  Every allocation is host memory; kernels prepared and launched are lines of the log.
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>
#include <vector>

#include "../sparse_paged_kv_score_gb300/csrc/internal.h"

namespace {
std::map<const void*, std::string> names;   // kernels by their host function
std::vector<std::string> events;
int sms = 152;

CUresult encode(CUtensorMap*, ...) { return CUDA_SUCCESS; }
const char* name_of(const void* f) {
  const auto it = names.find(f);
  return it == names.end() ? "?" : it->second.c_str();
}
}  // namespace

extern "C" {

void fake_sms(int n) { sms = n; }
void fake_clear() { events.clear(); }
int fake_events() { return static_cast<int>(events.size()); }
const char* fake_event(int i) { return events[i].c_str(); }

void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* device, int, uint3*, uint3*, dim3*, dim3*, int*) {
  names[host] = device;
}

cudaError_t cudaGetDevice(int* d) {
  *d = 0;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  *v = sms;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute, int) {
  events.push_back(std::string("set ") + name_of(f));
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaMalloc(void** p, size_t n) {
  *p = std::calloc(n, 1);
  return *p ? cudaSuccess : cudaErrorMemoryAllocation;
}
cudaError_t cudaFree(void* p) {
  std::free(p);
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t) {
  std::memset(p, v, n);
  return cudaSuccess;
}
cudaError_t cudaMemset(void* p, int v, size_t n) { return cudaMemsetAsync(p, v, n, nullptr); }
cudaError_t cudaMemcpy(void* to, const void* from, size_t n, cudaMemcpyKind) {
  std::memcpy(to, from, n);
  return cudaSuccess;
}
cudaError_t cudaHostGetDevicePointer(void**, void*, unsigned) { return cudaErrorInvalidValue; }   // not pinned
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *f = reinterpret_cast<void*>(encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
// "launch NAME GRID", and for the 4-bit attention " parts P".
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void* f, void** args) {
  std::string s = std::string("launch ") + name_of(f) + " " + std::to_string(cfg->gridDim.x);
  if (s.find("attn_q4_kernel") != std::string::npos)
    s += " parts " + std::to_string(static_cast<const spkv::AttnQ4Params*>(args[0])->parts);
  events.push_back(s);
  return cudaSuccess;
}

}  // extern "C"
