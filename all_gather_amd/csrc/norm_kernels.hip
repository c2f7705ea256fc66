// Layer norm, forward and backward, for gfx950.
//
//   forward   x = in[0] + ... + in[W-1] + residual        (fp32, in this order)
//             y = (x - mean) * rstd * gamma + beta,  rstd = 1 / sqrt(var + eps),  mean and var over the row
//   backward  with xh = (x - mean) * rstd and gd = gamma * dy,
//             dx = rstd * (gd - avg(gd) - xh * avg(gd * xh)) + dres
//             dgamma = sum over rows of dy * xh,  dbeta = sum over rows of dy
//
// Both are streaming work: a few operations for each element read.  A row is read once and stays in
// registers (a wave or a workgroup per row, up to four packs of 8 elements a lane); the statistics are two
// passes over the registers, the second on deviations from the mean, which cancels nothing.  Rows too long
// for that are read again from the caches.  All sums are fp32 in a fixed order.

#include "mr_train.h"
#include "packs.h"

namespace mr {
namespace {

constexpr int kV = 8;  // elements per pack

// Sum of x over the B lanes of a row (B = 64: the wave; else the workgroup, through `lds`, one word per wave).
template <int B>
__device__ __forceinline__ float row_sum(float x, float* lds) {
  x = wave_sum(x);
  if constexpr (B > 64) {
    constexpr int kWaves = B / 64;
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) x += lds[i];
  }
  return x;
}

// The elements of one pack of the row: the sum of the rank buffers and the residual, in fp32.
template <class T, bool Sum>
__device__ __forceinline__ void load_x(const NormFwdArgs& a, size_t at, int cnt, float (&x)[kV]) {
  widen(load_part<T, kV, true>(a.in[0] + at * T::kSize, cnt), x);
  if constexpr (Sum) {
    float f[kV];
    for (int r = 1; r < a.W; ++r) {
      widen(load_part<T, kV, true>(a.in[r] + at * T::kSize, cnt), f);
#pragma unroll
      for (int i = 0; i < kV; ++i) x[i] += f[i];
    }
    if (a.residual) {
      widen(load_part<T, kV, true>(a.residual + at * T::kSize, cnt), f);
#pragma unroll
      for (int i = 0; i < kV; ++i) x[i] += f[i];
    }
  }
}

template <class T, class WT>
__device__ __forceinline__ void write_y(const NormFwdArgs& a, size_t at, size_t col, int cnt, const float (&x)[kV], float mean,
                                        float rstd) {
  float g[kV], b[kV], y[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) g[i] = 1.0f, b[i] = 0.0f;
  if (a.gamma) widen(load_part<WT, kV, false>(a.gamma + col * WT::kSize, cnt), g);
  if (a.beta) widen(load_part<WT, kV, false>(a.beta + col * WT::kSize, cnt), b);
#pragma unroll
  for (int i = 0; i < kV; ++i) y[i] = __builtin_fmaf((x[i] - mean) * rstd, g[i], b[i]);
  store_part<T, kV, true>(a.y + at * T::kSize, y, cnt);
}

// Elements of pack `col` that lie in the row (0 .. 8).
__device__ __forceinline__ int in_row(size_t col, size_t cols) {
  return col >= cols ? 0 : cols - col < kV ? static_cast<int>(cols - col) : kV;
}

// A row per B lanes, K packs a lane.
template <class T, class WT, int B, int K, bool Sum>
__global__ __launch_bounds__(B < 256 ? 256 : B) void norm_fwd_row(NormFwdArgs a) {
  constexpr int kRows = B < 256 ? 256 / B : 1;
  __shared__ float lds[2][16];
  const int lane = threadIdx.x % B;
  const float inv = 1.0f / static_cast<float>(a.cols);
  // the two rounds of row sums use LDS words of their own, so a wave may start the next row while others end this one
  for (size_t row = static_cast<size_t>(blockIdx.x) * kRows + threadIdx.x / B; row < a.rows;
       row += static_cast<size_t>(gridDim.x) * kRows) {
    const size_t at = row * a.cols;
    float x[K][kV];
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const size_t col = (static_cast<size_t>(k) * B + lane) * kV;
      const int cnt = in_row(col, a.cols);
#pragma unroll
      for (int i = 0; i < kV; ++i) x[k][i] = 0.0f;
      if (cnt) load_x<T, Sum>(a, at + col, cnt, x[k]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < kV; ++i) s += x[k][i];
    const float mean = row_sum<B>(s, lds[0]) * inv;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int cnt = in_row((static_cast<size_t>(k) * B + lane) * kV, a.cols);
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const float d = i < cnt ? x[k][i] - mean : 0.0f;
        s = __builtin_fmaf(d, d, s);
      }
    }
    const float rstd = 1.0f / __builtin_sqrtf(row_sum<B>(s, lds[1]) * inv + a.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const size_t col = (static_cast<size_t>(k) * B + lane) * kV;
      const int cnt = in_row(col, a.cols);
      if (!cnt) continue;
      if (a.x_out) store_part<T, kV, true>(a.x_out + (at + col) * T::kSize, x[k], cnt);
      write_y<T, WT>(a, at + col, col, cnt, x[k], mean, rstd);
    }
    if (lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// Rows of any length: three sweeps over the row, the later two from the caches.  A lane reads every input
// of a pack before it writes that pack, so outputs may replace inputs exactly.
template <class T, class WT>
__global__ __launch_bounds__(1024) void norm_fwd_long(NormFwdArgs a) {
  __shared__ float lds[2][16];
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const size_t at = static_cast<size_t>(row) * a.cols;
    const float inv = 1.0f / static_cast<float>(a.cols);
    float x[kV];
    float s = 0.0f;
    for (size_t col = threadIdx.x * kV; col < a.cols; col += 1024 * kV) {
      load_x<T, true>(a, at + col, in_row(col, a.cols), x);  // zeros past the row's end
#pragma unroll
      for (int i = 0; i < kV; ++i) s += x[i];
    }
    const float mean = row_sum<1024>(s, lds[0]) * inv;
    s = 0.0f;
    for (size_t col = threadIdx.x * kV; col < a.cols; col += 1024 * kV) {
      const int cnt = in_row(col, a.cols);
      load_x<T, true>(a, at + col, cnt, x);
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const float d = i < cnt ? x[i] - mean : 0.0f;
        s = __builtin_fmaf(d, d, s);
      }
    }
    const float rstd = 1.0f / __builtin_sqrtf(row_sum<1024>(s, lds[1]) * inv + a.eps);
    for (size_t col = threadIdx.x * kV; col < a.cols; col += 1024 * kV) {
      const int cnt = in_row(col, a.cols);
      load_x<T, true>(a, at + col, cnt, x);
      if (a.x_out) store_part<T, kV, true>(a.x_out + (at + col) * T::kSize, x, cnt);
      write_y<T, WT>(a, at + col, col, cnt, x, mean, rstd);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// ------------------------------------------------------------------------------------------- backward

// Both row sums of the backward pass at once.
template <int B>
__device__ __forceinline__ void row_sum2(float& x, float& y, float (*lds)[16]) {
  x = wave_sum(x);
  y = wave_sum(y);
  if constexpr (B > 64) {
    constexpr int kWaves = B / 64;
    if ((threadIdx.x & 63) == 0) {
      lds[0][threadIdx.x >> 6] = x;
      lds[1][threadIdx.x >> 6] = y;
    }
    __syncthreads();
    x = y = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      x += lds[0][i];
      y += lds[1][i];
    }
    __syncthreads();  // the words are reused for the next row
  }
}

template <class T>
__device__ __forceinline__ void write_dx(const NormBwdArgs& a, size_t at, int cnt, const float (&gd)[kV], const float (&xh)[kV],
                                         float c1, float c2, float rstd) {
  float dx[kV], f[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) dx[i] = rstd * (gd[i] - __builtin_fmaf(xh[i], c2, c1));
  if (a.dres) {
    widen(load_part<T, kV, true>(a.dres + at * T::kSize, cnt), f);
#pragma unroll
    for (int i = 0; i < kV; ++i) dx[i] += f[i];
  }
  store_part<T, kV, true>(a.dx + at * T::kSize, dx, cnt);
}

// Workgroup b of `groups` takes rows b, b + groups, ... (B = 64: each of its four waves a row) and keeps its
// columns' sums of dy * xh and dy in registers; at the end it writes them to row b of `part`.
template <class T, class WT, int B, int K>
__global__ __launch_bounds__(B < 256 ? 256 : B) void norm_bwd_row(NormBwdArgs a) {
  constexpr int kRows = B < 256 ? 256 / B : 1;
  __shared__ float lds[2][16];
  __shared__ float part[kRows > 1 ? kRows * B * kV : 1];
  const int lane = threadIdx.x % B;
  const int sub = threadIdx.x / B;
  float dg[K][kV], db[K][kV];
  Raw<WT, kV> gamma[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const size_t col = (static_cast<size_t>(k) * B + lane) * kV;
#pragma unroll
    for (int i = 0; i < kV; ++i) dg[k][i] = db[k][i] = 0.0f;
    float one[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) one[i] = 1.0f;
    gamma[k] = a.gamma ? load_part<WT, kV, false>(a.gamma + col * WT::kSize, in_row(col, a.cols)) : narrow<WT, kV>(one);
  }
  const float inv = 1.0f / static_cast<float>(a.cols);
  for (size_t row = static_cast<size_t>(blockIdx.x) * kRows + sub; row < a.rows; row += static_cast<size_t>(gridDim.x) * kRows) {
    const size_t at = row * a.cols;
    const float mean = a.mean[row], rstd = a.rstd[row];
    Raw<T, kV> x[K], dy[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const size_t col = (static_cast<size_t>(k) * B + lane) * kV;
      const int cnt = in_row(col, a.cols);
      x[k] = load_part<T, kV, true>(a.x + (at + col) * T::kSize, cnt);
      dy[k] = load_part<T, kV, true>(a.dy + (at + col) * T::kSize, cnt);  // zeros past the row's end
    }
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float xf[kV], df[kV], gf[kV];
      widen(x[k], xf);
      widen(dy[k], df);
      widen(gamma[k], gf);
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const float xh = (xf[i] - mean) * rstd;
        const float gd = gf[i] * df[i];
        c1 += gd;
        c2 = __builtin_fmaf(gd, xh, c2);
        dg[k][i] = __builtin_fmaf(df[i], xh, dg[k][i]);
        db[k][i] += df[i];
      }
    }
    row_sum2<B>(c1, c2, lds);
    c1 *= inv;
    c2 *= inv;
    if (a.dx) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const size_t col = (static_cast<size_t>(k) * B + lane) * kV;
        const int cnt = in_row(col, a.cols);
        if (!cnt) continue;
        float xf[kV], gf[kV], df[kV];
        widen(x[k], xf);
        widen(dy[k], df);
        widen(gamma[k], gf);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          xf[i] = (xf[i] - mean) * rstd;
          gf[i] *= df[i];
        }
        write_dx<T>(a, at + col, cnt, gf, xf, c1, c2, rstd);
      }
    }
  }
  if (!a.part) return;
  float* out = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.cols;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const size_t col = (static_cast<size_t>(k) * B + lane) * kV;
    const int cnt = in_row(col, a.cols);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float f[kV];
#pragma unroll
      for (int i = 0; i < kV; ++i) f[i] = h ? db[k][i] : dg[k][i];
      if constexpr (kRows > 1) {  // add the four waves' sums up
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kV; ++i) part[(sub * kV + i) * B + lane] = f[i];
        __syncthreads();
        if (sub == 0) {
#pragma unroll
          for (int s = 1; s < kRows; ++s)
#pragma unroll
            for (int i = 0; i < kV; ++i) f[i] += part[(s * kV + i) * B + lane];
        }
      }
      if (sub == 0)
        store_part<EFp32, kV, false>(reinterpret_cast<char*>(out + h * a.cols + col), f, cnt);
    }
  }
}

// Rows of any length: dx with two sweeps over the row.
template <class T, class WT>
__global__ __launch_bounds__(1024) void norm_bwd_long_dx(NormBwdArgs a) {
  __shared__ float lds[2][16];
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const size_t at = static_cast<size_t>(row) * a.cols;
    const float mean = a.mean[row], rstd = a.rstd[row];
    const float inv = 1.0f / static_cast<float>(a.cols);
    float xh[kV], gd[kV], g[kV];
    auto load = [&](size_t col, int cnt) {
      widen(load_part<T, kV, false>(a.x + (at + col) * T::kSize, cnt), xh);
      widen(load_part<T, kV, false>(a.dy + (at + col) * T::kSize, cnt), gd);
#pragma unroll
      for (int i = 0; i < kV; ++i) g[i] = 1.0f;
      if (a.gamma) widen(load_part<WT, kV, false>(a.gamma + col * WT::kSize, cnt), g);
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        xh[i] = (xh[i] - mean) * rstd;
        gd[i] *= g[i];
      }
    };
    float c1 = 0.0f, c2 = 0.0f;
    for (size_t col = threadIdx.x * kV; col < a.cols; col += 1024 * kV) {
      load(col, in_row(col, a.cols));
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        c1 += gd[i];
        c2 = __builtin_fmaf(gd[i], xh[i], c2);
      }
    }
    row_sum2<1024>(c1, c2, lds);
    c1 *= inv;
    c2 *= inv;
    for (size_t col = threadIdx.x * kV; col < a.cols; col += 1024 * kV) {
      const int cnt = in_row(col, a.cols);
      load(col, cnt);
      write_dx<T>(a, at + col, cnt, gd, xh, c1, c2, rstd);
    }
  }
}

// Rows of any length: a wave's 512 columns over the rows blockIdx.y, blockIdx.y + gridDim.y, ...
template <class T>
__global__ __launch_bounds__(64) void norm_bwd_long_weights(NormBwdArgs a) {
  const size_t col = (static_cast<size_t>(blockIdx.x) * 64 + threadIdx.x) * kV;
  const int cnt = in_row(col, a.cols);
  if (!cnt) return;
  float dg[kV], db[kV], x[kV], dy[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) dg[i] = db[i] = 0.0f;
  for (size_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    widen(load_part<T, kV, false>(a.x + (row * a.cols + col) * T::kSize, cnt), x);
    widen(load_part<T, kV, false>(a.dy + (row * a.cols + col) * T::kSize, cnt), dy);
    const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      dg[i] = __builtin_fmaf(dy[i], (x[i] - mean) * rstd, dg[i]);
      db[i] += dy[i];
    }
  }
  float* out = a.part + static_cast<size_t>(blockIdx.y) * 2 * a.cols + col;
  store_part<EFp32, kV, false>(reinterpret_cast<char*>(out), dg, cnt);
  store_part<EFp32, kV, false>(reinterpret_cast<char*>(out + a.cols), db, cnt);
}

// dgamma and dbeta: the sum of the groups' rows of `part`.  A workgroup takes 64 of the 2*cols columns; its
// 16 waves each add up every 16th group, and the first wave adds the 16 sums.
template <class WT>
__global__ __launch_bounds__(1024) void norm_bwd_finish(NormBwdArgs a) {
  __shared__ float lds[16][64];
  const size_t c = static_cast<size_t>(blockIdx.x) * 64 + (threadIdx.x & 63);
  const int w = threadIdx.x >> 6;
  float s = 0.0f;
  if (c < 2 * a.cols)
    for (uint32_t g = w; g < a.groups; g += 16) s += a.part[static_cast<size_t>(g) * 2 * a.cols + c];
  lds[w][threadIdx.x & 63] = s;
  __syncthreads();
  if (w || c >= 2 * a.cols) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += lds[i][threadIdx.x];
  char* out = c < a.cols ? a.dgamma : a.dbeta;
  if (out) store1<WT>(out + (c < a.cols ? c : c - a.cols) * WT::kSize, s);
}

// ---------------------------------------------------------------------------------------------- launch

// Lanes per row and packs per lane: the narrowest that holds the row with up to four packs a lane.
constexpr size_t kFwdHeld = size_t{1024} * 4 * kV;  // longest row held in registers
constexpr size_t kBwdHeld = size_t{1024} * 2 * kV;  // the backward holds two rows and two sums a column

// A launch holds less than 2^32 lanes; kernels loop over the rows past their grid.
uint32_t grid_for(size_t groups) { return static_cast<uint32_t>(groups < (size_t{1} << 20) ? groups : size_t{1} << 20); }

template <class T, class WT, int B, int K>
void fwd_row(const NormFwdArgs& a, hipStream_t st) {
  constexpr int kRows = B < 256 ? 256 / B : 1;
  const dim3 grid(grid_for((a.rows + kRows - 1) / kRows)), block(B < 256 ? 256 : B);
  if (a.W > 1 || a.residual)
    hipLaunchKernelGGL((norm_fwd_row<T, WT, B, K, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((norm_fwd_row<T, WT, B, K, false>), grid, block, 0, st, a);
}

template <class T, class WT>
hipError_t fwd(const NormFwdArgs& a, hipStream_t st) {
  const size_t packs = (a.cols + kV - 1) / kV;
  if (packs <= 64) fwd_row<T, WT, 64, 1>(a, st);
  else if (packs <= 128) fwd_row<T, WT, 64, 2>(a, st);
  else if (packs <= 256) fwd_row<T, WT, 256, 1>(a, st);
  else if (packs <= 512) fwd_row<T, WT, 256, 2>(a, st);
  else if (packs <= 1024) fwd_row<T, WT, 256, 4>(a, st);
  else if (packs <= 2048) fwd_row<T, WT, 1024, 2>(a, st);
  else if (packs <= 4096) fwd_row<T, WT, 1024, 4>(a, st);
  else hipLaunchKernelGGL((norm_fwd_long<T, WT>), dim3(grid_for(a.rows)), dim3(1024), 0, st, a);
  return hipGetLastError();
}

template <class T, class WT, int B, int K>
void bwd_row(const NormBwdArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((norm_bwd_row<T, WT, B, K>), dim3(a.groups), dim3(B < 256 ? 256 : B), 0, st, a);
}

template <class T, class WT>
hipError_t bwd(const NormBwdArgs& a, hipStream_t st) {
  const size_t packs = (a.cols + kV - 1) / kV;
  if (a.rows) {
    if (packs <= 64) bwd_row<T, WT, 64, 1>(a, st);
    else if (packs <= 128) bwd_row<T, WT, 64, 2>(a, st);
    else if (packs <= 256) bwd_row<T, WT, 256, 1>(a, st);
    else if (packs <= 512) bwd_row<T, WT, 256, 2>(a, st);
    else if (packs <= 1024) bwd_row<T, WT, 512, 2>(a, st);
    else if (packs <= 2048) bwd_row<T, WT, 1024, 2>(a, st);
    else {
      if (a.part)  // first: dx may take the place of x or dy
        hipLaunchKernelGGL((norm_bwd_long_weights<T>), dim3(static_cast<uint32_t>((packs + 63) / 64), a.groups), dim3(64), 0, st, a);
      if (a.dx) hipLaunchKernelGGL((norm_bwd_long_dx<T, WT>), dim3(grid_for(a.rows)), dim3(1024), 0, st, a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.dgamma || a.dbeta)
    hipLaunchKernelGGL((norm_bwd_finish<WT>), dim3(static_cast<uint32_t>((2 * a.cols + 63) / 64)), dim3(1024), 0, st, a);
  return hipGetLastError();
}

}  // namespace

uint32_t norm_bwd_groups(size_t rows, size_t cols) {
  const size_t packs = (cols + kV - 1) / kV;
  const size_t per = packs <= 128 ? 4 : 1;                             // rows of one workgroup at a time
  const size_t most = packs <= 256 ? 1024 : packs <= 512 ? 512 : packs <= 2048 ? 256 : 64;
  const size_t want = (rows + per - 1) / per;
  return static_cast<uint32_t>(want < most ? want : most);
}

hipError_t launch_norm_fwd(const NormFwdArgs& a, mr_dtype dt, mr_dtype wdt, hipStream_t st) {
  if (dt == MR_FP32) return fwd<EFp32, EFp32>(a, st);
  if (dt == MR_BF16) return wdt == MR_FP32 ? fwd<EBf16, EFp32>(a, st) : fwd<EBf16, EBf16>(a, st);
  return wdt == MR_FP32 ? fwd<EFp16, EFp32>(a, st) : fwd<EFp16, EFp16>(a, st);
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, mr_dtype dt, mr_dtype wdt, hipStream_t st) {
  if (dt == MR_FP32) return bwd<EFp32, EFp32>(a, st);
  if (dt == MR_BF16) return wdt == MR_FP32 ? bwd<EBf16, EFp32>(a, st) : bwd<EBf16, EBf16>(a, st);
  return wdt == MR_FP32 ? bwd<EFp16, EFp32>(a, st) : bwd<EFp16, EFp16>(a, st);
}

}  // namespace mr
