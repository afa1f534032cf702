// The CUDA runtime's calls that the 8-bit layer operators' host code makes, without a device: launches
// are recorded, and one of them can be made to fail.
#include <cuda.h>
#include <cuda_runtime.h>
#include <string.h>

#include <map>
#include <string>
#include <vector>

namespace {
std::map<const void *, std::string> names;
std::map<const void *, size_t> sizes;
std::vector<unsigned *> words;                 // symbols of four bytes
int raise_after = -1;                          // the one that grows by one after the next copy from a symbol
std::vector<std::string> launched;
std::vector<std::pair<int, int>> shapes;       // of each launch: blocks along x, and to a cluster
int fail_at = -1, pending = 0;                 // number of the launch that fails; the error not yet collected
struct Config {
  dim3 grid, block;
  size_t smem;
  cudaStream_t st;
} config;

cudaError_t launch(const void *f, unsigned blocks, unsigned cluster = 1) {
  launched.push_back(names[f]);
  shapes.push_back({(int)blocks, (int)cluster});
  if ((int)launched.size() - 1 != fail_at) return cudaSuccess;
  return (cudaError_t)(pending = cudaErrorMemoryAllocation);
}
CUresult encode(...) { return CUDA_SUCCESS; }
}  // namespace

extern "C" {
void fake_reset(int fail) { launched.clear(), shapes.clear(), fail_at = fail, pending = 0; }
int fake_launches() { return (int)launched.size(); }
const char *fake_name(int i) { return launched[i].c_str(); }
int fake_blocks(int i) { return shapes[i].first; }
int fake_cluster(int i) { return shapes[i].second; }
int fake_words() { return (int)words.size(); }
void fake_raise(int i, int after) {
  if (after) raise_after = i;
  else ++*words[i];
}

void **__cudaRegisterFatBinary(void *) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *host, char *, const char *name, int, uint3 *, uint3 *, dim3 *, dim3 *, int *) {
  names[host] = name;
}
void __cudaRegisterVar(void **, char *host, char *, const char *, int, size_t size, int, int) {
  sizes[host] = size;
  if (size == 4) words.push_back((unsigned *)host);
}
unsigned __cudaPushCallConfiguration(dim3 g, dim3 b, size_t smem, cudaStream_t st) {
  config = Config{g, b, smem, st};
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3 *g, dim3 *b, size_t *smem, void *st) {
  *g = config.grid, *b = config.block, *smem = config.smem, *(cudaStream_t *)st = config.st;
  return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t *k, const void *f) {
  *k = (cudaKernel_t)f;
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3 g, dim3, void **, size_t, cudaStream_t) { return launch((const void *)k, g.x); }
cudaError_t cudaLaunchKernel(const void *f, dim3 g, dim3, void **, size_t, cudaStream_t) { return launch(f, g.x); }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **) {
  unsigned cluster = 1;
  for (unsigned i = 0; i < c->numAttrs; i++)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = c->attrs[i].val.clusterDim.x;
  return launch(f, c->gridDim.x, cluster);
}
cudaError_t cudaGetLastError() {
  const int e = pending;
  pending = 0;
  return (cudaError_t)e;
}
cudaError_t cudaGetDevice(int *d) { return *d = 0, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { return *v = 152, cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *r) {
  *f = (void *)encode;
  *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
// A symbol's value on the device is its shadow's on the host here.
cudaError_t cudaMemcpyFromSymbolAsync(void *to, const void *sym, size_t n, size_t off, cudaMemcpyKind, cudaStream_t) {
  if (off + n > sizes[sym]) return cudaErrorInvalidValue;
  memcpy(to, (const char *)sym + off, n);
  if (raise_after >= 0) ++*words[raise_after], raise_after = -1;
  return cudaSuccess;
}
cudaError_t cudaMemcpyToSymbolAsync(const void *sym, const void *from, size_t n, size_t off, cudaMemcpyKind, cudaStream_t) {
  if (off + n > sizes[sym]) return cudaErrorInvalidValue;
  memcpy((char *)sym + off, from, n);
  return cudaSuccess;
}
}
