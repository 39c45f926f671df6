// A stand-in for the CUDA runtime, for tests of the library's host code on a
// machine without a GPU: device memory is host memory, kernels do nothing,
// and a test says which GPUs there are and which launch fails.
#include <cuda_runtime_api.h>
#include <stdlib.h>
#include <string.h>

#include <map>
#include <utility>

namespace {
struct Gpu {
  int sms = 148;
  int clusters_of[17];   // clusters that run at once, by their size
};
Gpu g_gpu[4];
int g_gpus = 1, g_current = 0;
long g_launches = 0, g_fails_at = 0;          // the launch that fails, counted from now (0: none)
int g_launched_on = -1;                       // the current GPU of the last launch
std::map<char*, std::pair<size_t, int>> g_memory;   // address -> bytes, GPU
cudaError_t g_last = cudaSuccess;

cudaError_t done(cudaError_t e) { return e == cudaSuccess ? e : g_last = e; }
cudaError_t launch() {
  ++g_launches;
  g_launched_on = g_current;
  return done(g_fails_at && --g_fails_at == 0 ? cudaErrorLaunchOutOfResources : cudaSuccess);
}
int encode_tensor_map() { return 0; }
}  // namespace

extern "C" {

void fake_gpus(int n) {
  g_gpus = n;
  g_fails_at = 0;
  for (Gpu& g : g_gpu)
    for (int i = 0; i < 17; ++i) g.clusters_of[i] = i ? 132 / i : 0;
}
void fake_clusters(int gpu, int size, int n) { g_gpu[gpu].clusters_of[size] = n; }
void fake_fail_launch(long nth) { g_fails_at = nth; }
long fake_launches() { return g_launches; }
int fake_launched_on() { return g_launched_on; }

cudaError_t cudaGetDeviceCount(int* n) { return *n = g_gpus, cudaSuccess; }
cudaError_t cudaGetDevice(int* d) { return *d = g_current, cudaSuccess; }
cudaError_t cudaSetDevice(int d) { return d < g_gpus ? (g_current = d, cudaSuccess) : done(cudaErrorInvalidDevice); }
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int d) {
  *v = a == cudaDevAttrMultiProcessorCount ? g_gpu[d].sms : a == cudaDevAttrMaxSharedMemoryPerBlockOptin ? 232448 : 1;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() {
  const cudaError_t e = g_last;
  g_last = cudaSuccess;
  return e;
}
const char* cudaGetErrorString(cudaError_t) { return "stand-in error"; }

cudaError_t cudaMalloc(void** p, size_t n) {
  *p = nullptr;
  if (posix_memalign(p, 256, n ? n : 1)) return done(cudaErrorMemoryAllocation);
  memset(*p, 0, n);
  g_memory[(char*)*p] = {n, g_current};
  return cudaSuccess;
}
cudaError_t cudaFree(void* p) {
  g_memory.erase((char*)p);
  free(p);
  return cudaSuccess;
}
cudaError_t cudaMallocAsync(void** p, size_t n, cudaStream_t) { return cudaMalloc(p, n); }
cudaError_t cudaFreeAsync(void* p, cudaStream_t) { return cudaFree(p); }
cudaError_t cudaMemcpy(void* d, const void* s, size_t n, cudaMemcpyKind) { return memmove(d, s, n), cudaSuccess; }
cudaError_t cudaMemcpyAsync(void* d, const void* s, size_t n, cudaMemcpyKind, cudaStream_t) {
  return memmove(d, s, n), cudaSuccess;
}
cudaError_t cudaMemset(void* d, int v, size_t n) { return memset(d, v, n), cudaSuccess; }
cudaError_t cudaMemsetAsync(void* d, int v, size_t n, cudaStream_t) { return memset(d, v, n), cudaSuccess; }
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes* a, const void* p) {
  *a = cudaPointerAttributes{};
  a->type = cudaMemoryTypeUnregistered;
  auto it = g_memory.upper_bound((char*)p);
  if (it != g_memory.begin() && (--it, (char*)p < it->first + it->second.first)) {
    a->type = cudaMemoryTypeDevice;
    a->device = it->second.second;
  }
  return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** p, const void* symbol) { return *p = const_cast<void*>(symbol), cudaSuccess; }

cudaError_t cudaStreamCreateWithFlags(cudaStream_t* s, unsigned) { return *s = (cudaStream_t)&g_current, cudaSuccess; }
cudaError_t cudaStreamDestroy(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamBeginCapture(cudaStream_t, cudaStreamCaptureMode) { return cudaSuccess; }
cudaError_t cudaStreamEndCapture(cudaStream_t, cudaGraph_t* g) { return *g = (cudaGraph_t)&g_current, cudaSuccess; }
cudaError_t cudaGraphGetNodes(cudaGraph_t, cudaGraphNode_t*, size_t* n) { return *n = 0, cudaSuccess; }
cudaError_t cudaGraphNodeGetType(cudaGraphNode_t, cudaGraphNodeType*) { return cudaErrorInvalidValue; }
cudaError_t cudaGraphInstantiate(cudaGraphExec_t* e, cudaGraph_t, unsigned long long) {
  return *e = (cudaGraphExec_t)&g_current, cudaSuccess;
}
cudaError_t cudaGraphUpload(cudaGraphExec_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGraphLaunch(cudaGraphExec_t, cudaStream_t) { return launch(); }
cudaError_t cudaGraphDestroy(cudaGraph_t) { return cudaSuccess; }
cudaError_t cudaGraphExecDestroy(cudaGraphExec_t) { return cudaSuccess; }

cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  *a = cudaFuncAttributes{};
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t, unsigned) {
  return *n = 1, cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
  unsigned size = 1;
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) size = c->attrs[i].val.clusterDim.x;
  return *n = size <= 16 ? g_gpu[g_current].clusters_of[size] : 0, cudaSuccess;
}
cudaError_t cudaGetDriverEntryPoint(const char*, void** p, unsigned long long, cudaDriverEntryPointQueryResult* r) {
  *p = (void*)&encode_tensor_map;
  if (r) *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernel(const void*, dim3, dim3, void**, size_t, cudaStream_t) { return launch(); }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) { return launch(); }

// What compiled device code registers at load, and the <<<>>> form.
void** __cudaRegisterFatBinary(void*) { return (void**)&g_current; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, void*, void*, void*, void*, int*) {}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, void*) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3* g, dim3* b, size_t* m, void*) {
  *g = *b = dim3(1);
  *m = 0;
  return cudaSuccess;
}

}  // extern "C"
