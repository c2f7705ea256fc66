// Layer norm's forward pass for gfx950:
//
//   x = in[0] + in[1] + ...                                (rank buffers, then a residual: fp32, in this order)
//   y = (x - mean) * rstd * gamma + beta,  rstd = 1 / sqrt(var + eps),  mean and var over the row
//
// Streaming work: a few operations for each element read.  A row is read once and stays in registers; the
// statistics are two passes over the registers, the second on deviations from the mean, which cancels
// nothing.  Rows too long for that are read again from the caches.  All sums are fp32 in a fixed order.

#include "norm_common.h"

namespace mr {
namespace {

#ifndef MR_NF_DEPTH
#define MR_NF_DEPTH 3
#endif
#ifndef MR_NF_LANES
#define MR_NF_LANES 256
#endif
constexpr int kFwdLanes = MR_NF_LANES;  // lanes of a workgroup (more where a row takes more)

// Row held in registers by B lanes, K packs each.  Workgroups walk rows b, b + grid, ...: gamma and beta are
// loaded once, and with one input the next row's packs are loaded before this row's sums.
template <class T, class WT, int B, int K, bool Sum>
__global__ __launch_bounds__(B < kFwdLanes ? kFwdLanes : B) void norm_fwd_row(NormFwdArgs a) {
  constexpr int kLanes = B < kFwdLanes ? kFwdLanes : B;
  constexpr int kRows = kLanes / B;
  __shared__ float lds[2][kLanes / 64];
  const RowPacks<B, K> c(static_cast<uint32_t>(a.cols), threadIdx.x % B);
  const float inv = 1.0f / static_cast<float>(a.cols);
  uint32_t sub = threadIdx.x / B;
  if (B >= 64) sub = __builtin_amdgcn_readfirstlane(sub);
  constexpr bool kHold = K == 1;                // gamma and beta stay in registers
  constexpr bool kAhead = !Sum && K * T::kSize <= 4;
  Raw<WT, kV> g[kHold ? K : 1], b[kHold ? K : 1];
  if (kHold) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      g[k] = load_weights<WT>(a.gamma, c.at[k], 1.0f);
      b[k] = load_weights<WT>(a.beta, c.at[k], 0.0f);
    }
  }
  // Rows of the workgroup's last round may lie past the end: they repeat the last row and store nothing, so that every
  // lane reaches the barriers.
  Raw<T, kV> next[K];
  auto fetch = [&](size_t base) {
    const size_t row = base + sub < a.rows ? base + sub : a.rows - 1;
#pragma unroll
    for (int k = 0; k < K; ++k) next[k] = load_raw<T, kV, true>(a.in[0] + (row * a.cols + c.at[k]) * T::kSize);
  };
  const size_t stride = static_cast<size_t>(gridDim.x) * kRows;
  size_t base = static_cast<size_t>(blockIdx.x) * kRows;
  if (kAhead) fetch(base);
  for (; base < a.rows; base += stride) {
    const bool mine = base + sub < a.rows;
    const size_t row = mine ? base + sub : a.rows - 1;
    const size_t at = row * a.cols;
    float x[K][kV];
    if constexpr (Sum) {
      constexpr int kDepth = K >= 4 ? 1 : MR_NF_DEPTH / K;  // inputs loaded before the first is added
      for (int r = 0; r < a.terms; r += kDepth) {
        Raw<T, kV> w[kDepth][K];
#pragma unroll
        for (int j = 0; j < kDepth; ++j)
          if (r + j < a.terms)
#pragma unroll
            for (int k = 0; k < K; ++k) w[j][k] = load_raw<T, kV, true>(a.in[r + j] + (at + c.at[k]) * T::kSize);
#pragma unroll
        for (int j = 0; j < kDepth; ++j)
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
    } else {
      if (!kAhead) fetch(base);
#pragma unroll
      for (int k = 0; k < K; ++k) widen(next[k], x[k]);
      if (kAhead && base + stride < a.rows) fetch(base + stride);
    }
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
    // the two rounds of row sums use LDS words of their own, so a wave may start its next row while others end this one
    const float mean = row_sum<B>(s, lds[0]) * inv;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (wave_full(c.lo[k])) {
#pragma unroll
        for (int i = 0; i < kV; ++i) s = __builtin_fmaf(x[k][i] - mean, x[k][i] - mean, s);
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const float d = i >= c.lo[k] ? x[k][i] - mean : 0.0f;
          s = __builtin_fmaf(d, d, s);
        }
      }
    }
    const float rstd = 1.0f / __builtin_sqrtf(row_sum<B>(s, lds[1]) * inv + a.eps);
    if (!mine) continue;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (c.lo[k] == kV) continue;
      if (a.x_out) store_raw<T, kV, true>(a.x_out + (at + c.at[k]) * T::kSize, narrow<T, kV>(x[k]));
      float gf[kV], bf[kV], y[kV];
      widen(kHold ? g[k] : load_weights<WT>(a.gamma, c.at[k], 1.0f), gf);
      widen(kHold ? b[k] : load_weights<WT>(a.beta, c.at[k], 0.0f), bf);
#pragma unroll
      for (int i = 0; i < kV; ++i) y[i] = __builtin_fmaf((x[k][i] - mean) * rstd, gf[i], bf[i]);
      store_raw<T, kV, true>(a.y + (at + c.at[k]) * T::kSize, narrow<T, kV>(y));
    }
    if (threadIdx.x % B == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// Rows of any length: three sweeps over the row, the later two from the caches.  A lane reads every input
// of a pack before it writes that pack, so outputs may replace inputs exactly.
template <class T, class WT, int B>
__global__ __launch_bounds__(B) void norm_fwd_any(NormFwdArgs a) {
  __shared__ float lds[2][B / 64];
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
      load(col, in_row(col, a.cols));
#pragma unroll
      for (int i = 0; i < kV; ++i) s += x[i];
    }
    const float mean = row_sum<B>(s, lds[0]) * inv;
    s = 0.0f;
    for (size_t col = threadIdx.x * kV; col < a.cols; col += B * kV) {
      const int cnt = in_row(col, a.cols);
      load(col, cnt);
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const float d = i < cnt ? x[i] - mean : 0.0f;
        s = __builtin_fmaf(d, d, s);
      }
    }
    const float rstd = 1.0f / __builtin_sqrtf(row_sum<B>(s, lds[1]) * inv + a.eps);
    for (size_t col = threadIdx.x * kV; col < a.cols; col += B * kV) {
      const int cnt = in_row(col, a.cols);
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

#ifndef MR_NF_SUMALL
#define MR_NF_SUMALL 1
#endif
template <class T, class WT, int B, int K>
void fwd_row(const NormFwdArgs& a, hipStream_t st) {
  constexpr int kLanes = B < kFwdLanes ? kFwdLanes : B;
  const size_t groups = (a.rows + kLanes / B - 1) / (kLanes / B);
  if (a.terms > 1)
    hipLaunchKernelGGL((norm_fwd_row<T, WT, B, K, true>), dim3(MR_NF_SUMALL ? norm_grid(groups) : resident_grid<norm_fwd_row<T, WT, B, K, true>>(kLanes, groups)),
                       dim3(kLanes), 0, st, a);
  else
    hipLaunchKernelGGL((norm_fwd_row<T, WT, B, K, false>), dim3(resident_grid<norm_fwd_row<T, WT, B, K, false>>(kLanes, groups)),
                       dim3(kLanes), 0, st, a);
}

#ifndef MR_NF_K
#define MR_NF_K 1
#endif
template <class T, class WT>
hipError_t fwd(const NormFwdArgs& a, hipStream_t st) {
  const size_t packs = (a.cols + kV - 1) / kV;
  if (a.cols < kV)
    hipLaunchKernelGGL((norm_fwd_any<T, WT, 64>), dim3(norm_grid(a.rows)), dim3(64), 0, st, a);
  else if (packs <= 1024)
#define MR_LANES(B) fwd_row<T, WT, (B / MR_NF_K < 64 ? B : B / MR_NF_K), (B / MR_NF_K < 64 ? 1 : MR_NF_K)>(a, st)
    switch (norm_lanes(packs)) {
      case 8: MR_LANES(8); break;
      case 32: MR_LANES(32); break;
      case 64: MR_LANES(64); break;
      case 128: MR_LANES(128); break;
      case 256: MR_LANES(256); break;
      case 512: MR_LANES(512); break;
      default: MR_LANES(1024); break;
    }
  else if (packs <= 2048)
    fwd_row<T, WT, 1024, 2>(a, st);
  else if (packs <= 4096)
    fwd_row<T, WT, 1024, 4>(a, st);
  else
    hipLaunchKernelGGL((norm_fwd_any<T, WT, 1024>), dim3(norm_grid(a.rows)), dim3(1024), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_fwd(const NormFwdArgs& a, mr_dtype dt, mr_dtype wdt, hipStream_t st) {
  if (dt == MR_FP32) return fwd<EFp32, EFp32>(a, st);
  if (dt == MR_BF16) return wdt == MR_FP32 ? fwd<EBf16, EFp32>(a, st) : fwd<EBf16, EBf16>(a, st);
  return wdt == MR_FP32 ? fwd<EFp16, EFp32>(a, st) : fwd<EFp16, EFp16>(a, st);
}

}  // namespace mr
