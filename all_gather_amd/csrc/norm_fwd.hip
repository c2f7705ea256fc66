// Layer norm's forward pass for gfx950:
//
//   x = in[0] + in[1] + ...                                (rank buffers, then a residual: fp32, in this order)
//   y = (x - mean) * rstd * gamma + beta,  rstd = 1 / sqrt(var + eps),  mean and var over the row
//
// Streaming work: a few operations for each element read.  A row is read once and stays in registers; the
// statistics are two passes over the registers, the second on deviations from the mean, which cancels
// nothing.  Rows too long for that are read again from the caches.  All sums are fp32 in a fixed order.
//
// Bound by the bytes moved: 16384 x 8192 bf16 88.5 us (6.07 TB/s); the sum of 8 rank buffers with a residual, 2048 x 4096
// bf16, 31.3 us (5.89 TB/s over 9 read and 2 written streams); one row of 4096 takes 3.2 us, the launch.

#include <type_traits>

#include "norm_common.h"

namespace mr {
namespace {

constexpr int kFwdLanes = 256;  // lanes of a workgroup whose rows take a wave or less each

// The row set of workgroup b of n: workgroups are dealt to the eight XCDs in turn, and runs of 16 sets that follow one another
// go to one XCD (2048 rows of 4096, W = 8 with a residual: 33.3 us in plain order, 31.8 in runs of 4 to 16).
__device__ __forceinline__ uint32_t group_of(uint32_t b, uint32_t n) {
  constexpr uint32_t kRun = 16, kDeal = 8 * kRun;
  return b < n / kDeal * kDeal ? b / kDeal * kDeal + b % 8 * kRun + b % kDeal / 8 : b;
}

// Row held in registers.  Workgroups walk rows b, b + grid, ...: gamma and beta are loaded once, and with one input the
// next row's packs are loaded before this row's sums.  Loads and stores leave through one counter that a wait can only
// count back on, so every full round issues the same ones on every path: lanes past the row's end store its last pack
// once more, and the row's statistics collect in registers until a wave's lanes are full.  (With predicated stores a
// round waited for the last one's stores to reach memory: 60003 x 1025 bf16 57.8 -> 54.5 us, its backward pass 92.6 -> 81.9.)
// The waits are the compiler's.  As built, rows on whole waves with one pack a lane count past the last round's stores (fp32
// rows, and 16-bit rows with weights of their type); the other single-input builds still wait for all of them at the loop's top.
template <class T, class WT, int B, int K, bool Sum, int Lanes>
__global__ __launch_bounds__(Lanes, K == 1 ? 8 : Lanes == 768 ? 3 : 4) void norm_fwd_row(NormFwdArgs a) {
  constexpr int kV = kPack<T>;
  // gamma and beta stay in registers (their loads would otherwise wait for the next row's, issued before them)
  constexpr bool kHold = K * kV <= 16 && !(Sum && Lanes == 1024 && K > 1);
  constexpr bool kAhead = !Sum && kHold;  // the next row's packs are loaded ahead
  __shared__ WaveWords lds[2][B == kWaves ? 4 : 1];  // rows of 1 wave need none, of more at most 4 fit a workgroup
  const int lanes = B == kWaves ? a.waves * 64 : B;
  const int lane = threadIdx.x % lanes;
  const RowPacks<kV, K> c(static_cast<uint32_t>(a.cols), lane, lanes);
  const uint32_t set = blockDim.x / lanes;  // rows of the workgroup at a time
  const float inv = 1.0f / static_cast<float>(a.cols);
  uint32_t sub = threadIdx.x / lanes;
  if (B == kWaves) sub = __builtin_amdgcn_readfirstlane(sub);
  if (B == kWaves && a.waves > 1) {
    if (threadIdx.x < 128) lds[threadIdx.x >> 6][(threadIdx.x >> 4) & 3].w[threadIdx.x & 15] = 0.0f;
    __syncthreads();
  }
  const int wave = (threadIdx.x >> 6) - static_cast<int>(sub) * a.waves;  // of this row
  // Sum over the lanes of the row, in every one of them.  A round's two sums use words of their own, so a wave may start
  // its next round while others end this one.
  auto row_sum = [&](float x, WaveWords* words) {
    x = lanes_sum<B>(x);
    if (B == kWaves && a.waves > 1) {
      if ((threadIdx.x & 63) == 0) words[sub].w[wave] = x;
      __syncthreads();
      x = words_sum(words[sub], a.waves);
    }
    return x;
  };
  Raw<WT, kV> g[kHold ? K : 1], b[kHold ? K : 1];
  if (kHold) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      g[k] = load_weights<WT, kV>(a.gamma, c.at[k], 1.0f);
      b[k] = load_weights<WT, kV>(a.beta, c.at[k], 0.0f);
    }
  }
  const size_t stride = static_cast<size_t>(gridDim.x) * set;
  size_t base = static_cast<size_t>(group_of(blockIdx.x, gridDim.x)) * set;
  struct Row {
    Raw<T, kV> x[K];
  };
  auto fetch = [&](size_t from) {  // rows past the end: the last row
    Row r;
    const size_t row = from + sub < a.rows ? from + sub : a.rows - 1;
#pragma unroll
    for (int k = 0; k < K; ++k) r.x[k] = load_raw<T, kV, true>(a.in[0] + (row * a.cols + c.at[k]) * T::kSize);
    return r;
  };
  auto sum_inputs = [&](size_t at, float (&x)[K][kV]) {
    constexpr int kTerms = K >= 4 ? 1 : 3 / K;  // inputs loaded before the first is added
    for (int r = 0; r < a.terms; r += kTerms) {
      Raw<T, kV> w[kTerms][K];
#pragma unroll
      for (int j = 0; j < kTerms; ++j)
        if (r + j < a.terms)
#pragma unroll
          for (int k = 0; k < K; ++k) w[j][k] = load_raw<T, kV, true>(a.in[r + j] + (at + c.at[k]) * T::kSize);
#pragma unroll
      for (int j = 0; j < kTerms; ++j)
        if (r + j < a.terms)
#pragma unroll
          for (int k = 0; k < K; ++k) {
            float f[kV];
            widen(w[j][k], f);
            if (j == 0 && r == 0) {
#pragma unroll
              for (int i = 0; i < kV; ++i) x[k][i] = f[i];
            } else {
#pragma unroll
              for (int i = 0; i < kV; ++i) x[k][i] += f[i];
            }
          }
    }
  };
  auto stats = [&](const float (&x)[K][kV], float* mean, float* rstd) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (wave_full(c.lo[k])) {
#pragma unroll
        for (int i = 0; i < kV; ++i) s += x[k][i];
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) s += i >= c.lo[k] ? x[k][i] : 0.0f;
      }
    }
    // With several packs a lane a wave may lie past the row's end with one of them, which it reads and stores as the row's last
    // pack and adds to no sum: it too has x (a pack is one load) before the barrier, after which y may be in its place.
    if (K > 1)
#pragma unroll
      for (int k = 0; k < K; ++k) asm volatile("" ::"v"(x[k][kV - 1]));
    const float m = row_sum(s, lds[0]) * inv;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (wave_full(c.lo[k])) {
#pragma unroll
        for (int i = 0; i < kV; ++i) s = __builtin_fmaf(x[k][i] - m, x[k][i] - m, s);
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const float d = i >= c.lo[k] ? x[k][i] - m : 0.0f;
          s = __builtin_fmaf(d, d, s);
        }
      }
    }
    *mean = m;
    *rstd = 1.0f / __builtin_sqrtf(row_sum(s, lds[1]) * inv + a.eps);
  };
  auto store = [&](size_t at, const float (&x)[K][kV], float mean, float rstd) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (Sum && a.x_out) store_raw<T, kV, true>(a.x_out + (at + c.at[k]) * T::kSize, narrow<T, kV>(x[k]));
      float gf[kV], bf[kV], y[kV];
      widen(kHold ? g[k] : load_weights<WT, kV>(a.gamma, c.at[k], 1.0f), gf);
      widen(kHold ? b[k] : load_weights<WT, kV>(a.beta, c.at[k], 0.0f), bf);
#pragma unroll
      for (int i = 0; i < kV; ++i) y[i] = __builtin_fmaf((x[k][i] - mean) * rstd, gf[i], bf[i]);
      store_raw<T, kV, true>(a.y + (at + c.at[k]) * T::kSize, narrow<T, kV>(y));
    }
  };
  // Lane j keeps the statistics of round first + j until the lanes are full.
  constexpr int kKeep = B == kWaves ? 64 : B;
  float kept_mean = 0.0f, kept_rstd = 0.0f;
  int kept = 0;
  size_t first = base;
  auto flush = [&] {
    const size_t row = first + static_cast<size_t>(lane) * stride + sub;
    if (lane < kept && row < a.rows) {
      if (a.mean) a.mean[row] = kept_mean;
      if (a.rstd) a.rstd[row] = kept_rstd;
    }
    first += kept * stride;
    kept = 0;
  };
  auto keep = [&](float mean, float rstd) {
    if (lane % kKeep == kept) {
      kept_mean = mean;
      kept_rstd = rstd;
    }
    if (++kept == kKeep) flush();
  };
  Row next;
  if (kAhead) next = fetch(base);
  for (; base + set <= a.rows; base += stride) {
    const size_t at = (base + sub) * a.cols;
    float x[K][kV], mean, rstd;
    if constexpr (Sum) {
      sum_inputs(at, x);
    } else {
      const Row r = kAhead ? next : fetch(base);
      if (kAhead) next = fetch(base + stride);
#pragma unroll
      for (int k = 0; k < K; ++k) widen(r.x[k], x[k]);
    }
    stats(x, &mean, &rstd);
    store(at, x, mean, rstd);
    keep(mean, rstd);
  }
  if (base < a.rows) {  // a last set with fewer rows than the workgroup holds
    const bool mine = base + sub < a.rows;
    const size_t at = (mine ? base + sub : a.rows - 1) * a.cols;
    float x[K][kV], mean, rstd;
    if constexpr (Sum) {
      sum_inputs(at, x);
    } else {
      const Row r = fetch(base);
#pragma unroll
      for (int k = 0; k < K; ++k) widen(r.x[k], x[k]);
    }
    stats(x, &mean, &rstd);
    if (mine) store(at, x, mean, rstd);
    keep(mean, rstd);
  }
  flush();
}

// Rows shorter than a pack: a lane to a row.
template <class T, class WT>
__global__ __launch_bounds__(256) void norm_fwd_tiny(NormFwdArgs a) {
  constexpr int kMost = kPack<T> - 1;
  const int cols = static_cast<int>(a.cols);
  const float inv = 1.0f / static_cast<float>(cols);
  for (size_t row = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; row < a.rows; row += static_cast<size_t>(gridDim.x) * 256) {
    float x[kMost];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      if (i >= cols) break;
      const size_t at = (row * cols + i) * T::kSize;
      x[i] = load1<T>(a.in[0] + at);
      for (int r = 1; r < a.terms; ++r) x[i] += load1<T>(a.in[r] + at);
      s += x[i];
    }
    const float mean = s * inv;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kMost; ++i)
      if (i < cols) s = __builtin_fmaf(x[i] - mean, x[i] - mean, s);
    const float rstd = 1.0f / __builtin_sqrtf(s * inv + a.eps);
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      if (i >= cols) break;
      const size_t at = (row * cols + i) * T::kSize;
      if (a.x_out) store1<T>(a.x_out + at, x[i]);
      const float g = a.gamma ? load1<WT>(a.gamma + i * WT::kSize) : 1.0f, b = a.beta ? load1<WT>(a.beta + i * WT::kSize) : 0.0f;
      store1<T>(a.y + at, __builtin_fmaf((x[i] - mean) * rstd, g, b));
    }
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// Rows of any length: three sweeps over the row, the later two from the caches.  A lane reads every input
// of a pack before it writes that pack, so outputs may replace inputs exactly.
template <class T, class WT>
__global__ __launch_bounds__(1024) void norm_fwd_any(NormFwdArgs a) {
  constexpr int B = 1024;
  __shared__ WaveWords lds[2];
  constexpr int kV = kPack<T>;
  const float inv = 1.0f / static_cast<float>(a.cols);
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const size_t at = row * a.cols;
    float x[kV], f[kV];
    auto load = [&](size_t col, int cnt) {
      widen(load_part<T, kV, false>(a.in[0] + (at + col) * T::kSize, cnt), x);  // zeros past the row's end
      for (int r = 1; r < a.terms; ++r) {
        widen(load_part<T, kV, false>(a.in[r] + (at + col) * T::kSize, cnt), f);
#pragma unroll
        for (int i = 0; i < kV; ++i) x[i] += f[i];
      }
    };
    float s = 0.0f;
    for (size_t col = threadIdx.x * kV; col < a.cols; col += B * kV) {
      load(col, in_row<kV>(col, a.cols));
#pragma unroll
      for (int i = 0; i < kV; ++i) s += x[i];
    }
    const float mean = workgroup_sum<B>(s, lds[0]) * inv;
    s = 0.0f;
    for (size_t col = threadIdx.x * kV; col < a.cols; col += B * kV) {
      const int cnt = in_row<kV>(col, a.cols);
      load(col, cnt);
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const float d = i < cnt ? x[i] - mean : 0.0f;
        s = __builtin_fmaf(d, d, s);
      }
    }
    const float rstd = 1.0f / __builtin_sqrtf(workgroup_sum<B>(s, lds[1]) * inv + a.eps);
    for (size_t col = threadIdx.x * kV; col < a.cols; col += B * kV) {
      const int cnt = in_row<kV>(col, a.cols);
      load(col, cnt);
      if (a.x_out) store_part<T, kV, true>(a.x_out + (at + col) * T::kSize, x, cnt);
      float gf[kV], bf[kV], y[kV];
#pragma unroll
      for (int i = 0; i < kV; ++i) gf[i] = 1.0f, bf[i] = 0.0f;
      if (a.gamma) widen(load_part<WT, kV, false>(a.gamma + col * WT::kSize, cnt), gf);
      if (a.beta) widen(load_part<WT, kV, false>(a.beta + col * WT::kSize, cnt), bf);
#pragma unroll
      for (int i = 0; i < kV; ++i) y[i] = __builtin_fmaf((x[i] - mean) * rstd, gf[i], bf[i]);
      store_part<T, kV, true>(a.y + (at + col) * T::kSize, y, cnt);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// With several inputs every row set has a workgroup of its own: a row's loads are many, and a resident grid's last
// round leaves units idle (2048 rows of 4096, W = 8 with a residual: 33.4 us, 34.4 on a resident grid).
template <class T, class WT, int B, int K>
void fwd_row(NormFwdArgs a, int waves, hipStream_t st) {
  a.waves = waves;
  const int lanes = B == kWaves ? waves * 64 : B;
  const int block = lanes < kFwdLanes ? kFwdLanes / lanes * lanes : lanes;  // up to 4 rows of a wave or more
  const size_t groups = (a.rows + block / lanes - 1) / (block / lanes);
  auto launch = [&](auto most) {
    constexpr int kLanes = decltype(most)::value;
    if (a.terms > 1 || a.x_out)
      hipLaunchKernelGGL((norm_fwd_row<T, WT, B, K, true, kLanes>), dim3(norm_grid(groups)), dim3(block), 0, st, a);
    else
      hipLaunchKernelGGL((norm_fwd_row<T, WT, B, K, false, kLanes>),
                         dim3(resident_grid<norm_fwd_row<T, WT, B, K, false, kLanes>>(block, groups)), dim3(block), 0, st, a);
  };
  if constexpr (K > 1)
    if (block <= 768) return launch(std::integral_constant<int, 768>());  // 168 registers a lane, not 128
  launch(std::integral_constant<int, 1024>());
}

template <class T, class WT>
hipError_t fwd(const NormFwdArgs& a, hipStream_t st) {
  constexpr int kV = kPack<T>;
  const size_t packs = (a.cols + kV - 1) / kV;
  const int waves = static_cast<int>((packs + 63) / 64);  // with one pack a lane
  if (a.cols < kV)
    hipLaunchKernelGGL((norm_fwd_tiny<T, WT>), dim3(norm_grid((a.rows + 255) / 256)), dim3(256), 0, st, a);
  else if (kV == 8 && a.terms == 1 && !a.x_out && packs % 128 == 0 && packs <= 1024)
    // two packs a lane where they fill their waves: a row's sums cost each lane some 90 operations whatever it holds
    // (65536 x 1024 bf16 50.8 -> 46.8 us, 16384 x 4096 50.1 -> 48.6; fp32 and part-filled waves measured slower)
    fwd_row<T, WT, kWaves, 2>(a, static_cast<int>(packs / 128), st);
  else if (packs <= 8)
    fwd_row<T, WT, 8, 1>(a, 1, st);
  else if (packs <= 16)
    fwd_row<T, WT, 16, 1>(a, 1, st);
  else if (packs <= 32)
    fwd_row<T, WT, 32, 1>(a, 1, st);
  else if (waves <= 16)
    fwd_row<T, WT, kWaves, 1>(a, waves, st);
  else if (waves <= 32)
    fwd_row<T, WT, kWaves, 2>(a, (waves + 1) / 2, st);
  else if (waves <= 64)
    fwd_row<T, WT, kWaves, 4>(a, (waves + 3) / 4, st);
  else
    hipLaunchKernelGGL((norm_fwd_any<T, WT>), dim3(norm_grid(a.rows)), dim3(1024), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_fwd(const NormFwdArgs& a, mr_dtype dt, mr_dtype wdt, hipStream_t st) {
  if (dt == MR_FP32) return fwd<EFp32, EFp32>(a, st);
  if (dt == MR_BF16) return wdt == MR_FP32 ? fwd<EBf16, EFp32>(a, st) : fwd<EBf16, EBf16>(a, st);
  return wdt == MR_FP32 ? fwd<EFp16, EFp32>(a, st) : fwd<EFp16, EFp16>(a, st);
}

}  // namespace mr
