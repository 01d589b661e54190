// A stand-in for the HIP runtime's entry points that libsvdq uses, for tests
// without a GPU: one gfx950 device of 256 compute units whose launches are
// recorded and run nothing. A launch that the runtime's documented limits
// (fewer than 2^32 threads a dimension, 65535 workgroups in y and z, 1024
// threads a workgroup) exclude is an error, as it is there. Built with g++
// alone; tests/hip_stub.py loads it in front of the runtime.
#include <cstdint>
#include <cstring>
#include <map>
#include <string>
#include <vector>

#define __HIP_PLATFORM_AMD__
#include <hip/hip_runtime_api.h>

namespace {

struct Launch {
  std::string kernel;
  dim3 grid, block;
  size_t lds;
  uint8_t first[256];        // the first argument's bytes (and what follows them)
};
struct Config {
  dim3 grid, block;
  size_t lds;
  hipStream_t stream;
};
std::map<const void*, std::string> g_kernels;
std::vector<Launch> g_launches;
std::vector<Config> g_configs;
std::string g_refused;
hipError_t g_last = hipSuccess;   // what hipGetLastError gives next
alignas(256) char g_symbol[256];

bool fits(dim3 g, dim3 b) {
  const uint64_t gs[3] = {g.x, g.y, g.z}, bs[3] = {b.x, b.y, b.z};
  for (int i = 0; i < 3; ++i)
    if (gs[i] == 0 || bs[i] == 0 || gs[i] * bs[i] >= (uint64_t)1 << 32) return false;
  return gs[1] <= 65535 && gs[2] <= 65535 && bs[0] * bs[1] * bs[2] <= 1024;
}

}  // namespace

extern "C" {

void** __hipRegisterFatBinary(const void*) {
  static void* handle;
  return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
  g_kernels[host] = name;
}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
  g_configs.push_back({grid, block, lds, stream});
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
  const Config c = g_configs.back();
  g_configs.pop_back();
  *grid = c.grid;
  *block = c.block;
  *lds = c.lds;
  *stream = c.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t lds, hipStream_t) {
  Launch l;
  l.kernel = g_kernels[f];
  l.grid = grid;
  l.block = block;
  l.lds = lds;
  std::memcpy(l.first, args[0], sizeof(l.first));   // (on the caller's stack, which goes on past it)
  g_launches.push_back(l);
  if (!fits(grid, block)) g_last = hipErrorInvalidConfiguration;
  return g_last;
}
hipError_t hipGetLastError() {
  const hipError_t e = g_last;
  g_last = hipSuccess;
  return e;
}
hipError_t hipGetDevice(int* d) {
  *d = 0;
  return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int) {
  std::memset(p, 0, sizeof(*p));
  std::strcpy(p->gcnArchName, "gfx950:sramecc+:xnack-");
  p->multiProcessorCount = 256;
  return hipSuccess;
}
hipError_t hipFuncSetAttribute(const void* f, hipFuncAttribute, int) {
  if (g_refused.empty() || g_kernels[f].find(g_refused) == std::string::npos) return hipSuccess;
  return g_last = hipErrorInvalidValue;
}
hipError_t hipGetSymbolAddress(void** p, const void*) {
  *p = g_symbol;
  return hipSuccess;
}
hipError_t hipMemcpyAsync(void*, const void*, size_t, hipMemcpyKind, hipStream_t) { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }

// What the tests ask
void stub_refuse_attributes_of(const char* part_of_name) { g_refused = part_of_name; }
void stub_clear() { g_launches.clear(); }
int stub_launches() { return (int)g_launches.size(); }
const char* stub_kernel(int i) { return g_launches[i].kernel.c_str(); }
void stub_shape(int i, uint32_t* six) {
  const Launch& l = g_launches[i];
  const uint32_t v[6] = {l.grid.x, l.grid.y, l.grid.z, l.block.x, l.block.y, l.block.z};
  std::memcpy(six, v, sizeof(v));
}
const uint8_t* stub_first_argument(int i) { return g_launches[i].first; }

}  // extern "C"
