// What the forward and backward layer norm kernels share: where a lane's packs lie in a row, and row sums.
#pragma once

#include "mr_train.h"
#include "packs.h"

namespace mr {

constexpr int kV = kNormPack;

// A lane's packs of a row of `cols` >= 8 elements, B lanes with K packs each.  The row's last pack, if short, is read
// as the row's last 8 elements, of which the first `lo` belong to the neighbouring pack: every access is one whole pack,
// and both lanes store the same bits where they overlap (predicated single elements instead took a 200003 x 509
// fp16 backward pass 16% longer).  A pack past the row's end has lo = 8: read as that last pack, never stored.
template <int B, int K>
struct RowPacks {
  uint32_t at[K];
  int lo[K];
  __device__ RowPacks(uint32_t cols, int lane) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t col = (static_cast<uint32_t>(k) * B + lane) * kV;
      at[k] = col < cols - kV ? col : cols - kV;
      lo[k] = static_cast<int>(col - at[k] < kV ? col - at[k] : kV);
    }
  }
};

// Does every lane of the wave own all of its pack?  (Uniform, so the common case runs without selects.)
__device__ __forceinline__ bool wave_full(int lo) { return __builtin_amdgcn_ballot_w64(lo != 0) == 0; }

// A lane's pack of the weights, or `other` in its place.
template <class WT>
__device__ __forceinline__ Raw<WT, kV> load_weights(const char* w, uint32_t at, float other) {
  if (w) return load_raw<WT, kV, false>(w + static_cast<size_t>(at) * WT::kSize);
  float f[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) f[i] = other;
  return narrow<WT, kV>(f);
}

// Elements of a pack at `col` that lie in the row (0 .. 8).
__device__ __forceinline__ int in_row(size_t col, size_t cols) {
  return col >= cols ? 0 : cols - col < kV ? static_cast<int>(cols - col) : kV;
}

// Sum over the B lanes of a row, in every one of them; above a wave through `lds` (a word per wave of the workgroup).
template <int B>
__device__ __forceinline__ float row_sum(float x, float* lds) {
  if constexpr (B <= 64) {
    return lanes_sum<B>(x);
  } else {
    constexpr int kWaves = B / 64;
    const int wave = threadIdx.x >> 6;
    x = lanes_sum<64>(x);
    if ((threadIdx.x & 63) == 0) lds[wave] = x;
    __syncthreads();
    x = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) x += lds[wave / kWaves * kWaves + i];
    return x;
  }
}

// A launch holds less than 2^32 lanes; kernels loop over the rows past their grid.
inline uint32_t norm_grid(size_t groups) { return static_cast<uint32_t>(groups < (size_t{1} << 20) ? groups : size_t{1} << 20); }

// Grid of a kernel whose workgroups walk the rows: as many workgroups as the device holds at once, or `groups`.
// (Looked up once per kernel and device.)
template <auto Kernel>
uint32_t resident_grid(int lanes, size_t groups) {
  constexpr int kDevices = 64;
  static std::atomic<long long> cache[kDevices];  // 0: not looked up yet
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kDevices) return norm_grid(groups);
  long long n = cache[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    int per_cu = 0, cus = 0;
    n = -1;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, Kernel, lanes, 0) == hipSuccess &&
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && per_cu > 0 && cus > 0)
      n = static_cast<long long>(per_cu) * cus;
    cache[dev].store(n, std::memory_order_relaxed);
  }
  if (n <= 0 || groups <= static_cast<size_t>(n)) return norm_grid(groups);
  const size_t rounds = (groups + n - 1) / n;  // the same number of rounds for every workgroup, or one less
  return norm_grid((groups + rounds - 1) / rounds);
}

}  // namespace mr
