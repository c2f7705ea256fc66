// Layer norm's backward pass for gfx950.  With xh = (x - mean) * rstd and gd = gamma * dy,
//
//   dx     = rstd * (gd - avg(gd) - xh * avg(gd * xh)) + dres
//   dgamma = sum over rows of dy * xh,  dbeta = sum over rows of dy
//
// Streaming work, read once: a workgroup holds its current rows of x and dy in registers and its columns' two
// weight sums beside them, and walks the rows; at the end it writes one row of partial sums, and a second
// launch adds those rows up.  Few, wide workgroups keep the partial sums a small part of the traffic.  All sums are
// fp32 in an order set by the shape alone.

#include "norm_common.h"

namespace mr {
namespace {

constexpr int kBwdLanes = 1024;
#ifndef MR_NB_AHEAD
#define MR_NB_AHEAD 1
#endif
constexpr int kDepth = MR_NB_AHEAD;

// Workgroup b of `groups` takes row sets b, b + groups, ...; a set is one row for each B lanes.  The next set's x and
// dy are loaded before this set's sums where registers allow.
template <class T, class WT, int B, int K>
__global__ __launch_bounds__(kBwdLanes) void norm_bwd_row(NormBwdArgs a) {
  constexpr int kRows = kBwdLanes / B;
  constexpr bool kAhead = K == 1;  // and gamma stays in registers
  __shared__ float lds[2][2][kBwdLanes / 64];
  __shared__ float part[kRows > 1 ? kBwdLanes * kV : 1];
  const int lane = threadIdx.x % B;
  const RowPacks<B, K> c(static_cast<uint32_t>(a.cols), lane);
  uint32_t sub = threadIdx.x / B;
  if (B >= 64) sub = __builtin_amdgcn_readfirstlane(sub);
  const float inv = 1.0f / static_cast<float>(a.cols);
  float dg[K][kV], db[K][kV];
  Raw<WT, kV> gamma;
  if (kAhead) gamma = load_weights<WT>(a.gamma, c.at[0], 1.0f);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < kV; ++i) dg[k][i] = db[k][i] = 0.0f;
  struct Row {
    Raw<T, kV> x[K], dy[K];
    float mean, rstd;
  };
  // A set may hold rows past the end: they repeat the last row, add nothing and store nothing, so that every lane
  // reaches the barriers.
  auto fetch = [&](size_t base) {
    Row r;
    const size_t row = base + sub < a.rows ? base + sub : a.rows - 1;
    const size_t at = row * a.cols;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      r.x[k] = load_raw<T, kV, true>(a.x + (at + c.at[k]) * T::kSize);
      r.dy[k] = load_raw<T, kV, true>(a.dy + (at + c.at[k]) * T::kSize);
    }
    r.mean = a.mean[row];
    r.rstd = a.rstd[row];
    return r;
  };
  const size_t stride = static_cast<size_t>(gridDim.x) * kRows;
  size_t base = static_cast<size_t>(blockIdx.x) * kRows;
  Row next[kDepth];
  if (kAhead)
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
      if (base + d * stride < a.rows) next[d] = fetch(base + d * stride);
  int flip = 0;
  for (; base < a.rows; base += stride) {
    const bool mine = base + sub < a.rows;
    const size_t at = (mine ? base + sub : a.rows - 1) * a.cols;
    const Row r = kAhead ? next[0] : fetch(base);
    Raw<T, kV> dres[K];
    if (kAhead && a.dres)
#pragma unroll
      for (int k = 0; k < K; ++k) dres[k] = load_raw<T, kV, true>(a.dres + (at + c.at[k]) * T::kSize);
    if (kAhead) {
#pragma unroll
      for (int d = 1; d < kDepth; ++d) next[d - 1] = next[d];
      if (base + kDepth * stride < a.rows) next[kDepth - 1] = fetch(base + kDepth * stride);
    }
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int lo = mine ? c.lo[k] : kV;
      float xf[kV], df[kV], gf[kV];
      widen(r.x[k], xf);
      widen(r.dy[k], df);
      widen(kAhead ? gamma : load_weights<WT>(a.gamma, c.at[k], 1.0f), gf);
      auto add = [&](int i) {
        const float xh = (xf[i] - r.mean) * r.rstd;
        const float gd = gf[i] * df[i];
        c1 += gd;
        c2 = __builtin_fmaf(gd, xh, c2);
        dg[k][i] = __builtin_fmaf(df[i], xh, dg[k][i]);
        db[k][i] += df[i];
      };
      if (wave_full(lo)) {
#pragma unroll
        for (int i = 0; i < kV; ++i) add(i);
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
          if (i >= lo) add(i);
      }
    }
    if constexpr (B <= 64) {
      c1 = lanes_sum<B>(c1);
      c2 = lanes_sum<B>(c2);
    } else {  // two sets of words in turn: one barrier a round
      constexpr int kWaves = B / 64;
      const int wave = threadIdx.x >> 6;
      c1 = lanes_sum<64>(c1);
      c2 = lanes_sum<64>(c2);
      if ((threadIdx.x & 63) == 0) {
        lds[flip][0][wave] = c1;
        lds[flip][1][wave] = c2;
      }
      __syncthreads();
      c1 = c2 = 0.0f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) {
        c1 += lds[flip][0][sub * kWaves + i];
        c2 += lds[flip][1][sub * kWaves + i];
      }
      flip ^= 1;
    }
    c1 *= inv;
    c2 *= inv;
    if (!a.dx || !mine) continue;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (c.lo[k] == kV) continue;
      float xf[kV], gf[kV], df[kV], dx[kV];
      widen(r.x[k], xf);
      widen(r.dy[k], df);
      widen(kAhead ? gamma : load_weights<WT>(a.gamma, c.at[k], 1.0f), gf);
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const float xh = (xf[i] - r.mean) * r.rstd;
        dx[i] = r.rstd * (gf[i] * df[i] - __builtin_fmaf(xh, c2, c1));
      }
      if (a.dres) {
        widen(kAhead ? dres[k] : load_raw<T, kV, true>(a.dres + (at + c.at[k]) * T::kSize), df);
#pragma unroll
        for (int i = 0; i < kV; ++i) dx[i] += df[i];
      }
      store_raw<T, kV, true>(a.dx + (at + c.at[k]) * T::kSize, narrow<T, kV>(dx));
    }
  }
  if (!a.part) return;
  float* out = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.cols;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float f[kV];
#pragma unroll
      for (int i = 0; i < kV; ++i) f[i] = h ? db[k][i] : dg[k][i];
      if constexpr (kRows > 1) {  // add the set's rows up
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kV; ++i) part[(sub * kV + i) * B + lane] = f[i];
        __syncthreads();
        if (sub == 0)
#pragma unroll 1
          for (int s = 1; s < kRows; ++s)
#pragma unroll
            for (int i = 0; i < kV; ++i) f[i] += part[(s * kV + i) * B + lane];
      }
      if (sub == 0) {
        float* o = out + h * a.cols + c.at[k];
        if (c.lo[k] == 0) {
          store_raw<EFp32, kV, false>(reinterpret_cast<char*>(o), narrow<EFp32, kV>(f));
        } else {
#pragma unroll
          for (int i = 0; i < kV; ++i)
            if (i >= c.lo[k]) o[i] = f[i];
        }
      }
    }
}

// Rows of any length: dx with two sweeps over the row, the second from the caches.  A lane reads a pack's inputs
// before it writes that pack, so dx may take the place of one of them.
template <class T, class WT, int B>
__global__ __launch_bounds__(B) void norm_bwd_any_dx(NormBwdArgs a) {
  __shared__ float lds[2][B / 64];
  const float inv = 1.0f / static_cast<float>(a.cols);
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const size_t at = row * a.cols;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float xh[kV], gd[kV], g[kV];
    auto load = [&](size_t col, int cnt) {
      widen(load_part<T, kV, false>(a.x + (at + col) * T::kSize, cnt), xh);
      widen(load_part<T, kV, false>(a.dy + (at + col) * T::kSize, cnt), gd);  // zeros past the row's end
#pragma unroll
      for (int i = 0; i < kV; ++i) g[i] = 1.0f;
      if (a.gamma) widen(load_part<WT, kV, false>(a.gamma + col * WT::kSize, cnt), g);
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        xh[i] = i < cnt ? (xh[i] - mean) * rstd : 0.0f;
        gd[i] *= g[i];
      }
    };
    float c1 = 0.0f, c2 = 0.0f;
    for (size_t col = threadIdx.x * kV; col < a.cols; col += B * kV) {
      load(col, in_row(col, a.cols));
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        c1 += gd[i];
        c2 = __builtin_fmaf(gd[i], xh[i], c2);
      }
    }
    // a set of words for each sum: a wave may start its next row while others read this one's second sum
    c1 = row_sum<B>(c1, lds[0]) * inv;
    c2 = row_sum<B>(c2, lds[1]) * inv;
    for (size_t col = threadIdx.x * kV; col < a.cols; col += B * kV) {
      const int cnt = in_row(col, a.cols);
      load(col, cnt);
      float dx[kV], f[kV];
#pragma unroll
      for (int i = 0; i < kV; ++i) dx[i] = rstd * (gd[i] - __builtin_fmaf(xh[i], c2, c1));
      if (a.dres) {
        widen(load_part<T, kV, true>(a.dres + (at + col) * T::kSize, cnt), f);
#pragma unroll
        for (int i = 0; i < kV; ++i) dx[i] += f[i];
      }
      store_part<T, kV, true>(a.dx + (at + col) * T::kSize, dx, cnt);
    }
  }
}

// Rows of any length: a wave's 512 columns over the rows blockIdx.y, blockIdx.y + gridDim.y, ...
template <class T>
__global__ __launch_bounds__(64) void norm_bwd_any_weights(NormBwdArgs a) {
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

// dgamma and dbeta: the sum of the groups' rows of `part`.  A workgroup takes 32 of the 2*cols columns; its 32
// half waves each add up every 32nd group (8 loads of 256 groups, all in flight), and the first adds the 32 sums.
template <class WT>
__global__ __launch_bounds__(1024) void norm_bwd_finish(NormBwdArgs a) {
  constexpr int kCols = 32, kParts = 1024 / kCols;
  __shared__ float lds[kParts][kCols];
  const size_t c = static_cast<size_t>(blockIdx.x) * kCols + threadIdx.x % kCols;
  const uint32_t w = threadIdx.x / kCols;
  float s = 0.0f;
  if (c < 2 * a.cols) {
#pragma unroll 8
    for (uint32_t g = w; g < a.groups; g += kParts) s += a.part[static_cast<size_t>(g) * 2 * a.cols + c];
  }
  lds[w][threadIdx.x % kCols] = s;
  __syncthreads();
  if (w || c >= 2 * a.cols) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < kParts; ++i) s += lds[i][threadIdx.x];
  char* out = c < a.cols ? a.dgamma : a.dbeta;
  if (out) store1<WT>(out + (c < a.cols ? c : c - a.cols) * WT::kSize, s);
}

constexpr size_t kHeldPacks = 2048;  // longest row held in registers (two packs a lane)
bool held(size_t cols) { return cols >= kV && (cols + kV - 1) / kV <= kHeldPacks; }

template <class T, class WT, int B, int K>
void bwd_row(const NormBwdArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((norm_bwd_row<T, WT, B, K>), dim3(a.groups), dim3(kBwdLanes), 0, st, a);
}

template <class T, class WT, int B>
void bwd_any(const NormBwdArgs& a, size_t packs, hipStream_t st) {
  if (a.part)  // first: dx may take the place of x or dy
    hipLaunchKernelGGL((norm_bwd_any_weights<T>), dim3(static_cast<uint32_t>((packs + 63) / 64), a.groups), dim3(64), 0, st, a);
  if (a.dx) hipLaunchKernelGGL((norm_bwd_any_dx<T, WT, B>), dim3(norm_grid(a.rows)), dim3(B), 0, st, a);
}

template <class T, class WT>
hipError_t bwd(const NormBwdArgs& a, hipStream_t st) {
  const size_t packs = (a.cols + kV - 1) / kV;
  if (a.rows) {
    if (a.cols < kV)
      bwd_any<T, WT, 64>(a, packs, st);
    else if (!held(a.cols))
      bwd_any<T, WT, 1024>(a, packs, st);
    else if (packs > 1024)
      bwd_row<T, WT, 1024, 2>(a, st);
    else
      switch (norm_lanes(packs)) {
        case 8: bwd_row<T, WT, 8, 1>(a, st); break;
        case 32: bwd_row<T, WT, 32, 1>(a, st); break;
        case 64: bwd_row<T, WT, 64, 1>(a, st); break;
        case 128: bwd_row<T, WT, 128, 1>(a, st); break;
        case 256: bwd_row<T, WT, 256, 1>(a, st); break;
        case 512: bwd_row<T, WT, 512, 1>(a, st); break;
        default: bwd_row<T, WT, 1024, 1>(a, st); break;
      }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.dgamma || a.dbeta)
    hipLaunchKernelGGL((norm_bwd_finish<WT>), dim3(static_cast<uint32_t>((2 * a.cols + 31) / 32)), dim3(1024), 0, st, a);
  return hipGetLastError();
}

}  // namespace

#ifndef MR_NB_GROUPS
#define MR_NB_GROUPS 256
#endif
uint32_t norm_bwd_groups(size_t rows, size_t cols) {
  const size_t packs = (cols + kV - 1) / kV;
  const size_t set = !held(cols) ? 1 : packs > 1024 ? 1 : kBwdLanes / norm_lanes(packs);  // rows of a workgroup at a time
  const size_t most = held(cols) ? MR_NB_GROUPS : 64;
  const size_t want = (rows + set - 1) / set;
  return static_cast<uint32_t>(want < most ? want : most);
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, mr_dtype dt, mr_dtype wdt, hipStream_t st) {
  if (dt == MR_FP32) return bwd<EFp32, EFp32>(a, st);
  if (dt == MR_BF16) return wdt == MR_FP32 ? bwd<EBf16, EFp32>(a, st) : bwd<EBf16, EBf16>(a, st);
  return wdt == MR_FP32 ? bwd<EFp16, EFp32>(a, st) : bwd<EFp16, EFp16>(a, st);
}

}  // namespace mr
