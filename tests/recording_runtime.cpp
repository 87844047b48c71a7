// A stand-in for the HIP runtime, for host tests: two gfx950 devices that run
// nothing. It notes every kernel launch (name, grid, workgroup, dynamic LDS,
// stream, current device) and hands the notes out as lines of text. Streams
// are numbers: device * 16 + index, NULL the current device's default stream.
#include <cxxabi.h>
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>

namespace {
std::map<const void*, std::string> kernels;
std::string notes;
int current = 0;
struct {
  dim3 grid, block;
  size_t lds;
  hipStream_t stream;
} pushed;

void note(const void* f, dim3 g, dim3 b, size_t lds, hipStream_t s) {
  char line[512];
  snprintf(line, sizeof line, "%u %u %u %u %u %u %zu %zu %d ", g.x, g.y, g.z, b.x, b.y, b.z, lds, (size_t)s, current);
  notes += line + kernels[f] + "\n";
}
}  // namespace

extern "C" {

const char* recorded_launches() { return notes.c_str(); }
void forget_launches() { notes.clear(); }
const char* registered_kernels() {
  static std::string all;
  all.clear();
  for (const auto& k : kernels) all += k.second + "\n";
  return all.c_str();
}

void** __hipRegisterFatBinary(const void*) {
  static void* handle;
  return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, dim3*, dim3*, int*) {
  int status = 0;
  char* plain = abi::__cxa_demangle(name, nullptr, nullptr, &status);
  kernels[host] = plain ? plain : name;
  free(plain);
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
  pushed = {grid, block, lds, stream};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
  *grid = pushed.grid;
  *block = pushed.block;
  *lds = pushed.lds;
  *stream = pushed.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void**, size_t lds, hipStream_t stream) {
  note(f, grid, block, lds, stream);
  return hipSuccess;
}
hipError_t hipExtLaunchKernel(const void* f, dim3 grid, dim3 block, void**, size_t lds, hipStream_t stream, hipEvent_t,
                              hipEvent_t, int) {
  note(f, grid, block, lds, stream);
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) { return hipSuccess; }
hipError_t hipMemset(void*, int, size_t) { return hipSuccess; }
hipError_t hipGetSymbolAddress(void** p, const void*) {
  *p = (void*)0x10000;
  return hipSuccess;
}
hipError_t hipGetDeviceCount(int* n) {
  *n = 2;
  return hipSuccess;
}
hipError_t hipGetDevice(int* d) {
  *d = current;
  return hipSuccess;
}
hipError_t hipSetDevice(int d) {
  current = d;
  return hipSuccess;
}
hipError_t hipStreamGetDevice(hipStream_t s, hipDevice_t* d) {
  *d = s ? (int)((size_t)s / 16) : current;
  return hipSuccess;
}
hipError_t hipGetDeviceProperties(hipDeviceProp_t* p, int) {
  memset(p, 0, sizeof *p);
  strcpy(p->gcnArchName, "gfx950:sramecc+:xnack-");
  return hipSuccess;
}

}  // extern "C"
