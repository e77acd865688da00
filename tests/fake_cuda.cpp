// fake_cuda.cpp -- a CUDA runtime of no device, for host code under test: a
// device of a stated number of SMs and largest cluster, which refuses the
// launches that such a device would and notes the others.
#include <cuda_runtime_api.h>

extern "C" {

static int device, sms, largest;  // the current device
static int launches, grid, cluster;  // noted: their number, and the last one's

void fake_device(int id, int n, int most) {
  device = id;
  sms = n;
  largest = most;
  launches = 0;
}
void fake_seen(int* n, int* g, int* c) {
  *n = launches;
  *g = grid;
  *c = cluster;
}

static int cluster_of(const cudaLaunchConfig_t* lc) {
  for (unsigned i = 0; i < lc->numAttrs; ++i)
    if (lc->attrs[i].id == cudaLaunchAttributeClusterDimension) return (int)lc->attrs[i].val.clusterDim.x;
  return 1;
}

cudaError_t cudaGetDevice(int* d) {
  *d = device;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrMultiProcessorCount ? sms : 0;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* lc, const void*, void**) {
  const int c = cluster_of(lc);
  if (c > largest || lc->gridDim.x % c) return cudaErrorInvalidClusterSize;
  ++launches;
  grid = (int)lc->gridDim.x;
  cluster = c;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* lc) {
  *n = cluster_of(lc) > largest ? 0 : sms / cluster_of(lc);
  return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  *a = cudaFuncAttributes{};
  a->numRegs = 255;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t cudaMemcpyFromSymbol(void*, const void*, size_t, size_t, cudaMemcpyKind) { return cudaErrorUnknown; }
cudaError_t cudaMemcpyToSymbol(const void*, const void*, size_t, size_t, cudaMemcpyKind) { return cudaErrorUnknown; }

// what nvcc's host code registers its kernels with
int __cudaGetKernel(void*, const void*) { return 0; }
int __cudaLaunchKernel(const void*, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorUnknown; }
int __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaErrorUnknown; }
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, cudaStream_t) { return 1; }
void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}

}  // extern "C"
