// A stand-in for the HIP runtime that runs nothing, for tests of the library's host code without a GPU: one device of
// 256 CUs, device memory that is host memory, streams that are any pointer. It keeps what the tests ask about: kernels
// launched, memory cleared and not waited for, uses of a stream after its end.
//
// Loaded into the global scope before the library, whose HIP calls then bind here.
#include <hip/hip_runtime_api.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <set>
#include <string>

namespace {
std::map<const void *, std::string> kernels;  // host stub -> mangled name
std::set<void *> ended;                       // streams whose handles are dead
bool unwaited = false;                        // memory was set on the null stream and nothing has waited for it
int dead_uses = 0, early_launches = 0, waits = 0;
bool capturing = false;
int next_status = 0;  // what the next four-byte read of device memory returns
std::string log;
dim3 grid_, block_;
size_t shared_;
hipStream_t stream_;
int occupancy_of(const char *name) { return std::strstr(name, "ILi128ELi128E") ? 2 : 1; }
void use(hipStream_t s) {
  if (ended.count(s)) ++dead_uses;
}
}  // namespace

extern "C" {

// ---- for the tests
int stand_in_unwaited() { return unwaited; }
int stand_in_dead_uses() { return dead_uses; }
int stand_in_waits() { return waits; }  // of one stream for another
int stand_in_early_launches() { return early_launches; }
void stand_in_end_stream(void *s) { ended.insert(s); }
void stand_in_capture(int on) { capturing = on; }
void stand_in_device_status(int v) { next_status = v; }
// One line a launch since the last call: mangled name, grid, block and, of the kernels that join split tiles, the first split
// tile and the chunks.
const char *stand_in_launches() {
  static std::string out;
  out.swap(log);
  log.clear();
  return out.c_str();
}
// Every kernel of the library, one a line.
const char *stand_in_kernels() {
  static std::string out;
  out.clear();
  for (const auto &k : kernels) out += k.second + "\n";
  return out.c_str();
}

// ---- registration and launch
void **__hipRegisterFatBinary(const void *) {
  static void *handle;
  return &handle;
}
void __hipUnregisterFatBinary(void **) {}
void __hipRegisterFunction(void **, const void *stub, char *, const char *name, unsigned, void *, void *, void *, void *, int *) {
  kernels[stub] = name;
}
void __hipRegisterVar(void **, void *, char *, char *, int, size_t, int, int) {}
hipError_t __hipPushCallConfiguration(dim3 g, dim3 b, size_t shared, hipStream_t s) {
  grid_ = g;
  block_ = b;
  shared_ = shared;
  stream_ = s;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3 *g, dim3 *b, size_t *shared, hipStream_t *s) {
  *g = grid_;
  *b = block_;
  *shared = shared_;
  *s = stream_;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void *stub, dim3 g, dim3 b, void **args, size_t, hipStream_t s) {
  use(s);
  if (unwaited && s) ++early_launches;
  const std::string &name = kernels[stub];
  char line[512];
  int first = -1, chunks = -1;
  if (name.find("reduce") != std::string::npos) {  // five int32 after the epilogue's arguments and a pointer: m, n, tiles_n, first, chunks
    std::memcpy(&first, (const char *)args[0] + 96 + 12, 4);
    std::memcpy(&chunks, (const char *)args[0] + 96 + 16, 4);
  }
  std::snprintf(line, sizeof(line), "%s %u %u %u %d %d\n", name.c_str(), g.x, g.y, b.x, first, chunks);
  log += line;
  return hipSuccess;
}

// ---- device
hipError_t hipGetDevice(int *d) { return *d = 0, hipSuccess; }
hipError_t hipGetDeviceCount(int *n) { return *n = 1, hipSuccess; }
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600 *p, int) {
  std::memset(p, 0, sizeof(*p));
  std::strcpy(p->gcnArchName, "gfx950:sramecc+:xnack-");
  p->multiProcessorCount = 256;
  p->sharedMemPerBlock = 160 * 1024;
  return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int *v, hipDeviceAttribute_t, int) { return *v = 100000, hipSuccess; }
hipError_t hipOccupancyMaxActiveBlocksPerMultiprocessor(int *n, const void *f, int, size_t) {
  return *n = occupancy_of(kernels[f].c_str()), hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
const char *hipGetErrorString(hipError_t) { return "stand-in error"; }
hipError_t hipGetSymbolAddress(void **p, const void *) { return *p = nullptr, hipErrorInvalidSymbol; }

// ---- memory
hipError_t hipMalloc(void **p, size_t n) { return *p = std::calloc(1, n), *p ? hipSuccess : hipErrorOutOfMemory; }
hipError_t hipFree(void *p) { return std::free(p), hipSuccess; }
hipError_t hipHostMalloc(void **p, size_t n, unsigned) { return *p = std::calloc(1, n), *p ? hipSuccess : hipErrorOutOfMemory; }
hipError_t hipHostFree(void *p) { return std::free(p), hipSuccess; }
hipError_t hipMemset(void *p, int v, size_t n) { return std::memset(p, v, n), unwaited = true, hipSuccess; }
hipError_t hipMemcpy(void *d, const void *s, size_t n, hipMemcpyKind kind) {
  std::memcpy(d, s, n);
  if (kind == hipMemcpyDeviceToHost && n == 4 && next_status) {
    std::memcpy(d, &next_status, 4);
    next_status = 0;
  }
  return hipSuccess;
}
hipError_t hipMemcpyAsync(void *d, const void *s, size_t n, hipMemcpyKind, hipStream_t) { return std::memcpy(d, s, n), hipSuccess; }

// ---- streams and events
hipError_t hipStreamSynchronize(hipStream_t s) {
  use(s);
  if (!s) unwaited = false;
  return ended.count(s) ? hipErrorInvalidHandle : hipSuccess;
}
hipError_t hipDeviceSynchronize() { return unwaited = false, hipSuccess; }
hipError_t hipStreamWaitEvent(hipStream_t s, hipEvent_t, unsigned) { return use(s), ++waits, hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t s, hipStreamCaptureStatus *c) { 
  return use(s), *c = capturing ? hipStreamCaptureStatusActive : hipStreamCaptureStatusNone, hipSuccess;
}
hipError_t hipStreamDestroy(hipStream_t) { return hipSuccess; }
hipError_t hipExtStreamCreateWithCUMask(hipStream_t *s, uint32_t, const uint32_t *) { return *s = nullptr, hipSuccess; }
hipError_t hipEventCreate(hipEvent_t *e) { return *e = (hipEvent_t)std::malloc(1), hipSuccess; }
hipError_t hipEventCreateWithFlags(hipEvent_t *e, unsigned) { return hipEventCreate(e); }
hipError_t hipEventDestroy(hipEvent_t e) { return std::free(e), hipSuccess; }
hipError_t hipEventRecord(hipEvent_t, hipStream_t s) { return use(s), hipSuccess; }
hipError_t hipEventSynchronize(hipEvent_t) { return hipSuccess; }
hipError_t hipEventElapsedTime(float *t, hipEvent_t, hipEvent_t) { return *t = 0.0f, hipSuccess; }

}  // extern "C"
