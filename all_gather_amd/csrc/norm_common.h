// What the forward and backward layer norm kernels share: where a lane's packs lie in a row, and row sums.
#pragma once

#include "mr_train.h"
#include "packs.h"

namespace mr {

// Elements of a pack, what a lane takes of a row at once: 16 bytes of the row's type, so that neighbouring lanes' accesses
// adjoin (two 16-byte accesses a lane, 32 bytes apart, took an fp32 forward pass of 16384 x 2048 15% longer).
template <class T>
constexpr int kPack = 16 / T::kSize;

// A row lies over B lanes, K packs a lane: B = 8, 16 or 32 (a wave holds several rows), or B = kWaves: whole waves, as many as
// the row takes, a number known at launch.
constexpr int kWaves = 64;

// A lane's packs of V elements of a row of `cols` >= V elements on `lanes` lanes.  The row's last pack, if short, is read as
// the row's last V elements, of which the first `lo` belong to the neighbouring pack: every access is one whole pack, with
// no lane predicated by element, and both lanes store the same bits where they overlap.  A pack past the row's end has
// lo = V: it is read, and stored, as that last pack, and adds nothing to a sum.
template <int V, int K>
struct RowPacks {
  uint32_t at[K];
  int lo[K];
  __device__ RowPacks(uint32_t cols, int lane, int lanes) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t col = (static_cast<uint32_t>(k) * lanes + lane) * V;
      at[k] = col < cols - V ? col : cols - V;
      lo[k] = static_cast<int>(col - at[k] < V ? col - at[k] : V);
    }
  }
};

// Does every lane of the wave own all of its pack?  (Uniform, so the common case runs without selects.)
__device__ __forceinline__ bool wave_full(int lo) { return __builtin_amdgcn_ballot_w64(lo != 0) == 0; }

// A lane's pack of the weights, or `other` in its place.
template <class WT, int V>
__device__ __forceinline__ Raw<WT, V> load_weights(const char* w, uint32_t at, float other) {
  if (w) return load_raw<WT, V, false>(w + static_cast<size_t>(at) * WT::kSize);
  float f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = other;
  return narrow<WT, V>(f);
}

// Elements of a pack of V at `col` that lie in the row (0 .. V).
template <int V>
__device__ __forceinline__ int in_row(size_t col, size_t cols) {
  return col >= cols ? 0 : cols - col < V ? static_cast<int>(cols - col) : V;
}

// Words of the waves' sums, one line of 16 for each row of the workgroup; those no wave writes are zero.
struct alignas(16) WaveWords {
  float w[16];
};
__device__ __forceinline__ float words_sum(const WaveWords& l, int waves) {
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  const f32x4* q = reinterpret_cast<const f32x4*>(l.w);
  f32x4 s = q[0];
  if (waves > 4) s += q[1];
  if (waves > 8) s += q[2] + q[3];
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// Sum over a workgroup of B lanes (several waves), in every one of them.
template <int B>
__device__ __forceinline__ float workgroup_sum(float x, WaveWords& l) {
  x = lanes_sum<64>(x);
  if ((threadIdx.x & 63) == 0) l.w[threadIdx.x >> 6] = x;
  __syncthreads();
  return words_sum(l, B / 64);
}

// A launch holds less than 2^32 lanes; kernels loop over the rows past their grid.
inline uint32_t norm_grid(size_t groups) { return static_cast<uint32_t>(groups < (size_t{1} << 20) ? groups : size_t{1} << 20); }

// Grid of a kernel whose workgroups walk the rows: as many workgroups as the device holds at once, or `groups`.
// (Looked up once per kernel, device and workgroup size.)
template <auto Kernel>
uint32_t resident_grid(int lanes, size_t groups) {
  constexpr int kDevices = 64;
  static std::atomic<long long> cache[kDevices][17];  // by waves of a workgroup; 0: not looked up yet
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kDevices) return norm_grid(groups);
  std::atomic<long long>& slot = cache[dev][lanes / 64];
  long long n = slot.load(std::memory_order_relaxed);
  if (n == 0) {
    int per_cu = 0, cus = 0;
    n = -1;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, Kernel, lanes, 0) == hipSuccess &&
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && per_cu > 0 && cus > 0)
      n = static_cast<long long>(per_cu) * cus;
    slot.store(n, std::memory_order_relaxed);
  }
  if (n <= 0 || groups <= static_cast<size_t>(n)) return norm_grid(groups);
  const size_t rounds = (groups + n - 1) / n;  // the same number of rounds for every workgroup, or one less
  return norm_grid((groups + rounds - 1) / rounds);
}

}  // namespace mr
