// A HIP runtime that runs nothing: it hands out addresses that nobody reads and writes down every kernel launch.  Linked
// with the library's own objects it shows on the CPU what the host code would launch, in which order and with which
// grids.  A launch that the device could not hold (2^32 lanes or more in a dimension) is refused, as the runtime does.

#include <hip/hip_runtime_api.h>
#include <time.h>

#include <atomic>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <thread>
#include <vector>

namespace {

struct Launch {
  std::string name;
  uintptr_t stream;
  uint64_t thread;
  uint32_t grid[3], block[3];
  int refused;
};
std::mutex g_mu;
std::vector<Launch> g_launches;
uint64_t g_allocated = 0, g_next = uint64_t{1} << 44;
std::atomic<int> g_hold_ms{0};

std::map<const void*, std::string>& names() {  // filled by constructors of the kernel files
  static std::map<const void*, std::string> m;
  return m;
}

struct Config {
  dim3 grid, block;
  size_t shared;
  hipStream_t stream;
};
thread_local std::vector<Config> t_config;
thread_local hipError_t t_last = hipSuccess;

}  // namespace

extern "C" {

// ---- what the tests ask
void fake_reset(int hold_ms) {  // every later launch keeps its thread for hold_ms
  std::lock_guard<std::mutex> lk(g_mu);
  g_launches.clear();
  g_hold_ms = hold_ms;
}
int fake_launches() {
  std::lock_guard<std::mutex> lk(g_mu);
  return static_cast<int>(g_launches.size());
}
int fake_launch(int i, char* name, int n, uint64_t* v) {  // v: stream, thread, grid, block, refused
  std::lock_guard<std::mutex> lk(g_mu);
  if (i < 0 || i >= static_cast<int>(g_launches.size())) return -1;
  const Launch& l = g_launches[i];
  std::strncpy(name, l.name.c_str(), n - 1);
  name[n - 1] = 0;
  v[0] = l.stream;
  v[1] = l.thread;
  for (int d = 0; d < 3; ++d) v[2 + d] = l.grid[d], v[5 + d] = l.block[d];
  v[8] = l.refused;
  return 0;
}
uint64_t fake_allocated() {
  std::lock_guard<std::mutex> lk(g_mu);
  return g_allocated;
}

// ---- the runtime
void** __hipRegisterFatBinary(const void*) {
  static void* handle = nullptr;
  return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* device, unsigned, void*, void*, dim3*, dim3*, int*) {
  names()[host] = device;
}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}

hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t stream) {
  t_config.push_back({grid, block, shared, stream});
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
  const Config c = t_config.back();
  t_config.pop_back();
  *grid = c.grid;
  *block = c.block;
  *shared = c.shared;
  *stream = c.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void**, size_t, hipStream_t stream) {
  const uint64_t most = uint64_t{1} << 32;
  const bool refused = uint64_t{grid.x} * block.x >= most || uint64_t{grid.y} * block.y >= most || uint64_t{grid.z} * block.z >= most ||
                       !grid.x || !grid.y || !grid.z || !block.x || !block.y || !block.z || block.x * block.y * block.z > 1024;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    g_launches.push_back({names()[f], reinterpret_cast<uintptr_t>(stream), std::hash<std::thread::id>()(std::this_thread::get_id()),
                          {grid.x, grid.y, grid.z}, {block.x, block.y, block.z}, refused});
  }
  const int ms = g_hold_ms;
  if (ms) {
    timespec t{0, ms * 1000000L};
    nanosleep(&t, nullptr);
  }
  t_last = refused ? hipErrorInvalidConfiguration : hipSuccess;
  return t_last;
}
hipError_t hipGetLastError(void) {
  const hipError_t e = t_last;
  t_last = hipSuccess;
  return e;
}
hipError_t hipGetDevice(int* d) {
  *d = 0;
  return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) {
  *v = 256;
  return hipSuccess;
}
hipError_t hipOccupancyMaxActiveBlocksPerMultiprocessor(int* v, const void*, int, size_t) {
  *v = 2;
  return hipSuccess;
}
hipError_t hipStreamGetCaptureInfo(hipStream_t, hipStreamCaptureStatus* s, unsigned long long* id) {
  *s = hipStreamCaptureStatusNone;
  *id = 0;
  return hipSuccess;
}
hipError_t hipThreadExchangeStreamCaptureMode(hipStreamCaptureMode*) { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipMalloc(void** p, size_t bytes) {
  std::lock_guard<std::mutex> lk(g_mu);
  if (bytes > uint64_t{200} << 30) return hipErrorOutOfMemory;
  *p = reinterpret_cast<void*>(g_next);
  g_next += (bytes + 255) / 256 * 256;
  g_allocated += bytes;
  return hipSuccess;
}
hipError_t hipFree(void*) { return hipSuccess; }
hipError_t hipMemcpy(void* dst, const void*, size_t n, hipMemcpyKind) {
  std::memset(dst, 0, n);
  return hipSuccess;
}
hipError_t hipGetSymbolAddress(void** p, const void*) {
  *p = reinterpret_cast<void*>(uint64_t{1} << 43);
  return hipSuccess;
}

// ---- the copy engines: none
int hsa_init(void) { return 1; }
int hsa_iterate_agents(void*, void*) { return 1; }
int hsa_agent_get_info(uint64_t, int, void*) { return 1; }
int hsa_signal_create(int64_t, uint32_t, const void*, void*) { return 1; }
int hsa_amd_signal_create(int64_t, uint32_t, const void*, uint64_t, void*) { return 1; }
int hsa_signal_destroy(uint64_t) { return 1; }
void hsa_signal_subtract_screlease(uint64_t, int64_t) {}
int64_t hsa_signal_wait_scacquire(uint64_t, int, int64_t, uint64_t, int) { return 0; }
int hsa_amd_memory_copy_engine_status(uint64_t, uint64_t, void*) { return 1; }
int hsa_amd_memory_async_copy_on_engine(void*, uint64_t, const void*, uint64_t, size_t, uint32_t, const void*, uint64_t, int, bool) {
  return 1;
}

}  // extern "C"
