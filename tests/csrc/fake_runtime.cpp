// A stand-in for the CUDA runtime under the library's own objects: no GPU, every launch counted and none run, and a
// chosen call made to fail. The thread has no context before cudaSetDevice, as a fresh one. Entry points that the tests' calls only need to return take no parameters here (C linkage;
// what the caller passes is left where it is).
#include <driver_types.h>

#include <cstring>

namespace {
int launches = 0;
char failing[64] = "";
int answer(const char *name) { return std::strcmp(name, failing) ? 0 : (int)cudaErrorInvalidValue; }
bool has_context = false;
int get_current(void **context) {
  static int one;
  *context = has_context ? &one : nullptr;
  return 0;
}
int encode() { return has_context ? answer("cuTensorMapEncodeTiled") : 201; }  // (CUDA_ERROR_INVALID_CONTEXT)
alignas(256) char device_memory[256];
}  // namespace

extern "C" {
void fake_fail(const char *name) { std::strncpy(failing, name, sizeof failing - 1); }
int fake_launches() { return launches; }

void **__cudaRegisterFatBinary() {
  static void *handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd() {}
void __cudaUnregisterFatBinary() {}
void __cudaRegisterFunction() {}
void __cudaRegisterVar() {}
int __cudaGetKernel() { return 0; }
int __cudaPushCallConfiguration() { return 0; }
int __cudaPopCallConfiguration() { return 0; }
int __cudaLaunchKernel() {
  ++launches;
  return 0;
}
int cudaLaunchKernelExC() {
  ++launches;
  return 0;
}
int cudaGetLastError() { return 0; }
int cudaGetDevice(int *device) {
  *device = 0;
  return answer("cudaGetDevice");
}
int cudaSetDevice() {
  has_context = true;
  return answer("cudaSetDevice");
}
int cudaDeviceGetAttribute(int *value) {
  *value = 152;
  return answer("cudaDeviceGetAttribute");
}
int cudaGetSymbolAddress(void **p) {
  *p = device_memory;
  return answer("cudaGetSymbolAddress");
}
int cudaFuncSetAttribute() { return answer("cudaFuncSetAttribute"); }
int cudaFuncGetAttributes(cudaFuncAttributes *a) {
  std::memset(a, 0, sizeof *a);
  a->numRegs = 128;
  return answer("cudaFuncGetAttributes");
}
int cudaGetDriverEntryPointByVersion(const char *name, void **p, unsigned, unsigned long long, int *status) {
  *p = std::strcmp(name, "cuTensorMapEncodeTiled") ? reinterpret_cast<void *>(&get_current) : reinterpret_cast<void *>(&encode);
  *status = 0;
  return 0;
}
int cudaOccupancyMaxActiveClusters() { return cudaErrorNotSupported; }
int cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags() { return cudaErrorNotSupported; }
int cudaMemcpyToSymbol() { return cudaErrorNotSupported; }
int cudaMemcpyFromSymbol() { return cudaErrorNotSupported; }
int cudaStreamSynchronize() { return cudaErrorNotSupported; }
int cudaEventRecord() { return cudaErrorNotSupported; }
}
