// Layer norm's backward pass for gfx950.  With xh = (x - mean) * rstd and gd = gamma * dy,
//
//   dx     = rstd * (gd - avg(gd) - xh * avg(gd * xh)) + dres
//   dgamma = sum over rows of dy * xh,  dbeta = sum over rows of dy
//
// Streaming work, read once: a workgroup holds its current rows of x and dy in registers and its columns' two
// weight sums beside them, and walks the rows; at the end it writes one row of partial sums, and a second
// launch adds those rows up.  Few, wide workgroups keep the partial sums a small part of the traffic (512 groups instead
// of 256: 8192 x 4096 bf16 53.9 -> 61.2 us).  All sums are fp32 in an order set by the shape alone.
//
// Bound by the bytes moved, and below them by the wait of a row's waves for one another: 65536 x 1024 bf16 with dres 90 us
// (5.96 TB/s); 8192 x 4096 51.4 us, of which the second launch is 4.7; 200003 x 509 fp16 122 to 124 us (5.0 TB/s), whose rows
// start off the 16-byte grid and share their first and last lines with neighbours (x 512: 105 us).

#include "norm_common.h"

namespace mr {
namespace {

constexpr int kBwdLanes = 1024;  // most lanes of a workgroup; with 768 a lane has 168 registers, not 128

// Column c of dgamma and then dbeta.
template <class WT>
__device__ __forceinline__ void write_weight(const NormBwdArgs& a, size_t c, float s) {
  char* out = c < a.cols ? a.dgamma : a.dbeta;
  if (out) store1<WT>(out + (c < a.cols ? c : c - a.cols) * WT::kSize, s);
}

// Workgroup b of `groups` takes row sets b, b + groups, ...; a set is as many rows as the workgroup holds (one with more
// than a pack a lane).  The next set's x and dy are loaded before this set's sums where registers allow; as in the
// forward pass every full round issues the same loads and stores on every path, and as built the waits count past the last
// round's stores, but for fp16 rows without dres on one pack a lane, which wait for all of them at the loop's top.
template <class T, class WT, int B, int K, bool Dres, int Lanes>
__global__ __launch_bounds__(Lanes) void norm_bwd_row(NormBwdArgs a) {
  constexpr int kV = kPack<T>;
  constexpr bool kAhead = K * kV <= 8 || (Lanes < 1024 && (T::kSize == 2 || !Dres));
  // gamma stays in registers (its loads would otherwise wait for the next set's, issued before them)
  constexpr bool kHold = kAhead;
  __shared__ WaveWords lds[2][2][B == kWaves ? 8 : 1];  // rows of several waves: at most 8 fit a workgroup
  __shared__ float part[K == 1 ? Lanes / 2 * kV : 1];
  const int lanes = B == kWaves ? a.waves * 64 : B;
  const int lane = threadIdx.x % lanes;
  const RowPacks<kV, K> c(static_cast<uint32_t>(a.cols), lane, lanes);
  const uint32_t set = blockDim.x / lanes;
  uint32_t sub = threadIdx.x / lanes;
  if (B == kWaves) sub = __builtin_amdgcn_readfirstlane(sub);
  const int wave = (threadIdx.x >> 6) - static_cast<int>(sub) * a.waves;  // of this row
  if (B == kWaves && a.waves > 1) {
    if (threadIdx.x < 512) reinterpret_cast<float*>(lds)[threadIdx.x] = 0.0f;
    __syncthreads();
  }
  const float inv = 1.0f / static_cast<float>(a.cols);
  float dg[K][kV], db[K][kV];
  Raw<WT, kV> gamma[kHold ? K : 1];
  if (kHold)
#pragma unroll
    for (int k = 0; k < K; ++k) gamma[k] = load_weights<WT, kV>(a.gamma, c.at[k], 1.0f);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < kV; ++i) dg[k][i] = db[k][i] = 0.0f;
  struct Row {
    Raw<T, kV> dres[Dres ? K : 1], x[K], dy[K];
    float mean, rstd;
  };
  auto fetch = [&](size_t from) {  // rows past the end: the last row
    Row r;
    const size_t row = from + sub < a.rows ? from + sub : a.rows - 1;
    const size_t at = row * a.cols;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (Dres) r.dres[k] = load_raw<T, kV, true>(a.dres + (at + c.at[k]) * T::kSize);
      r.x[k] = load_raw<T, kV, true>(a.x + (at + c.at[k]) * T::kSize);
      r.dy[k] = load_raw<T, kV, true>(a.dy + (at + c.at[k]) * T::kSize);
    }
    r.mean = a.mean[row];
    r.rstd = a.rstd[row];
    return r;
  };
  // The row's two sums, and its part of the weight sums; elements before lo belong to another lane.
  auto sums = [&](const Row& r, int k, int lo, float* c1, float* c2) {
    float xf[kV], df[kV], gf[kV];
    widen(r.x[k], xf);
    widen(r.dy[k], df);
    widen(kHold ? gamma[kHold ? k : 0] : load_weights<WT, kV>(a.gamma, c.at[k], 1.0f), gf);
    auto add = [&](int i) {
      const float xh = (xf[i] - r.mean) * r.rstd;
      const float gd = gf[i] * df[i];
      *c1 += gd;
      *c2 = __builtin_fmaf(gd, xh, *c2);
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
  };
  int flip = 0;
  auto row_sums = [&](const Row& r, float* c1, float* c2) {
    const bool alone = K == 1 && (B != kWaves || a.waves == 1);  // no wave waits for another
    float x = alone ? wave_sum<B>(*c1) : lanes_sum<B>(*c1), y = alone ? wave_sum<B>(*c2) : lanes_sum<B>(*c2);
    if (Dres)  // has arrived before the barrier: dx may take its place, and a short last pack reads a neighbour's elements
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < Raw<T, kV>::kWords; ++i) asm volatile("" ::"v"(r.dres[k].w[i]));
    // With several packs a lane a wave may lie past the row's end with one of them, which it reads and stores as the row's last
    // pack and adds to no sum: it too has x and dy (a pack is one load) before the barrier, after which dx may be in their place.
    if (K > 1)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        constexpr int kLast = Raw<T, kV>::kWords - 1;
        asm volatile("" ::"v"(r.x[k].w[kLast]), "v"(r.dy[k].w[kLast]));
      }
    if (B == kWaves && a.waves > 1) {  // two sets of words in turn: one barrier a round
      if ((threadIdx.x & 63) == 0) {
        lds[flip][0][sub].w[wave] = x;
        lds[flip][1][sub].w[wave] = y;
      }
      __syncthreads();
      x = words_sum(lds[flip][0][sub], a.waves);
      y = words_sum(lds[flip][1][sub], a.waves);
      flip ^= 1;
    }
    *c1 = x * inv;
    *c2 = y * inv;
  };
  auto store = [&](const Row& r, int k, size_t at, float c1, float c2) {
    float xf[kV], gf[kV], df[kV], dx[kV];
    widen(r.x[k], xf);
    widen(r.dy[k], df);
    widen(kHold ? gamma[kHold ? k : 0] : load_weights<WT, kV>(a.gamma, c.at[k], 1.0f), gf);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const float xh = (xf[i] - r.mean) * r.rstd;
      dx[i] = r.rstd * (gf[i] * df[i] - __builtin_fmaf(xh, c2, c1));
    }
    if (Dres) {
      widen(r.dres[Dres ? k : 0], df);
#pragma unroll
      for (int i = 0; i < kV; ++i) dx[i] += df[i];
    }
    store_raw<T, kV, true>(a.dx + (at + c.at[k]) * T::kSize, narrow<T, kV>(dx));
  };
  const size_t stride = static_cast<size_t>(gridDim.x) * set;
  size_t base = static_cast<size_t>(blockIdx.x) * set;
  Row next;
  if (kAhead) next = fetch(base);
  for (; base + set <= a.rows; base += stride) {
    const size_t at = (base + sub) * a.cols;
    const Row r = kAhead ? next : fetch(base);
    if (kAhead) next = fetch(base + stride);
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) sums(r, k, c.lo[k], &c1, &c2);
    row_sums(r, &c1, &c2);
#pragma unroll
    for (int k = 0; k < K; ++k) store(r, k, at, c1, c2);
  }
  if (base < a.rows) {  // a last set with fewer rows than the workgroup holds: the others add and store nothing
    const bool mine = base + sub < a.rows;
    const size_t at = (mine ? base + sub : a.rows - 1) * a.cols;
    const Row r = fetch(base);
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) sums(r, k, mine ? c.lo[k] : kV, &c1, &c2);
    row_sums(r, &c1, &c2);
    if (mine)
#pragma unroll
      for (int k = 0; k < K; ++k) store(r, k, at, c1, c2);
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
      if (K == 1)  // add the set's rows up, the upper half's to the lower half's
        for (uint32_t n = set; n > 1; n = (n + 1) / 2) {
          const uint32_t half = (n + 1) / 2;
          if (sub >= half && sub < n)
#pragma unroll
            for (int i = 0; i < kV; ++i) part[((sub - half) * kV + i) * lanes + lane] = f[i];
          __syncthreads();
          if (sub < n - half)
#pragma unroll
            for (int i = 0; i < kV; ++i) f[i] += part[(sub * kV + i) * lanes + lane];
          __syncthreads();
        }
      if (sub == 0) {
        float* o = out + h * a.cols + c.at[k];
        if (a.groups == 1) {
#pragma unroll
          for (int i = 0; i < kV; ++i)
            if (i >= c.lo[k]) write_weight<WT>(a, h * a.cols + c.at[k] + i, f[i]);
        } else if (a.one_launch) {  // write-through, for a reader in this launch
#pragma unroll
          for (int i = 0; i < kV; ++i)
            if (i >= c.lo[k]) __hip_atomic_store(o + i, f[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        } else if (c.lo[k] == 0) {
          store_raw<EFp32, kV, false>(reinterpret_cast<char*>(o), narrow<EFp32, kV>(f));
        } else {
#pragma unroll
          for (int i = 0; i < kV; ++i)
            if (i >= c.lo[k]) o[i] = f[i];
        }
      }
    }
  if (!a.one_launch || a.groups == 1) return;
  // Every lane's stores are acknowledged before the workgroup's arrival is counted; the last one's loads follow the count.
  __shared__ bool last;
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  __syncthreads();
  if (threadIdx.x == 0) {
    last = __hip_atomic_fetch_add(a.arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    if (last) __hip_atomic_store(a.arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!last) return;
  // `slices` lanes share a column where there are few; device-scope loads are slow, so eight of a lane's are in flight.
  const uint32_t n = 2 * static_cast<uint32_t>(a.cols);
  const uint32_t slices = n < blockDim.x ? blockDim.x / n : 1;
  const uint32_t slice = threadIdx.x / n;
  for (uint32_t j = slices > 1 ? threadIdx.x % n : threadIdx.x; j < n; j += blockDim.x) {
    float s = 0.0f;
    if (slices == 1 || slice < slices) {
#pragma unroll 8
      for (uint32_t g = slices > 1 ? slice : 0; g < a.groups; g += slices)
        s += __hip_atomic_load(a.part + static_cast<size_t>(g) * n + j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (slices == 1) {
      write_weight<WT>(a, j, s);
      continue;
    }
    if (slice < slices) part[slice * n + j] = s;
    __syncthreads();
    if (threadIdx.x < n) {
      s = 0.0f;
      for (uint32_t i = 0; i < slices; ++i) s += part[i * n + threadIdx.x];
      write_weight<WT>(a, threadIdx.x, s);
    }
    break;
  }
}

// Rows shorter than a pack: a lane to a row, `groups` waves; each writes its rows' part of the weight gradients.
template <class T, class WT>
__global__ __launch_bounds__(64) void norm_bwd_tiny(NormBwdArgs a) {
  constexpr int kMost = kPack<T> - 1;
  const int cols = static_cast<int>(a.cols);
  const float inv = 1.0f / static_cast<float>(cols);
  float dg[kMost], db[kMost];
#pragma unroll
  for (int i = 0; i < kMost; ++i) dg[i] = db[i] = 0.0f;
  for (size_t row = static_cast<size_t>(blockIdx.x) * 64 + threadIdx.x; row < a.rows; row += static_cast<size_t>(gridDim.x) * 64) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    float xh[kMost], gd[kMost], c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      if (i >= cols) break;
      const size_t at = (row * cols + i) * T::kSize;
      xh[i] = (load1<T>(a.x + at) - mean) * rstd;
      const float dy = load1<T>(a.dy + at);
      gd[i] = a.gamma ? load1<WT>(a.gamma + i * WT::kSize) * dy : dy;
      c1 += gd[i];
      c2 = __builtin_fmaf(gd[i], xh[i], c2);
      dg[i] = __builtin_fmaf(dy, xh[i], dg[i]);
      db[i] += dy;
    }
    c1 *= inv;
    c2 *= inv;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      if (i >= cols || !a.dx) break;
      const size_t at = (row * cols + i) * T::kSize;
      float dx = rstd * (gd[i] - __builtin_fmaf(xh[i], c2, c1));
      if (a.dres) dx += load1<T>(a.dres + at);
      store1<T>(a.dx + at, dx);
    }
  }
  if (!a.part) return;
  float* out = a.part + static_cast<size_t>(blockIdx.x) * 2 * cols;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    if (i >= cols) break;
    const float g = wave_sum(dg[i]), b = wave_sum(db[i]);
    if (threadIdx.x == 0) {
      out[i] = g;
      out[cols + i] = b;
    }
  }
}

// Rows of any length: dx with two sweeps over the row, the second from the caches.  A lane reads a pack's inputs
// before it writes that pack, so dx may take the place of one of them.
template <class T, class WT>
__global__ __launch_bounds__(1024) void norm_bwd_any_dx(NormBwdArgs a) {
  constexpr int B = 1024;
  __shared__ WaveWords lds[2];
  constexpr int kV = kPack<T>;
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
      load(col, in_row<kV>(col, a.cols));
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        c1 += gd[i];
        c2 = __builtin_fmaf(gd[i], xh[i], c2);
      }
    }
    // a set of words for each sum: a wave may start its next row while others read this one's second sum
    c1 = workgroup_sum<B>(c1, lds[0]) * inv;
    c2 = workgroup_sum<B>(c2, lds[1]) * inv;
    for (size_t col = threadIdx.x * kV; col < a.cols; col += B * kV) {
      const int cnt = in_row<kV>(col, a.cols);
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

// Rows of any length: a wave's 64 packs of columns over the rows blockIdx.y, blockIdx.y + gridDim.y, ...
template <class T>
__global__ __launch_bounds__(64) void norm_bwd_any_weights(NormBwdArgs a) {
  constexpr int kV = kPack<T>;
  const size_t col = (static_cast<size_t>(blockIdx.x) * 64 + threadIdx.x) * kV;
  const int cnt = in_row<kV>(col, a.cols);
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

// dgamma and dbeta: the sum of the groups' rows of `part`.  A workgroup takes 32 of the 2*cols columns at a time; its 32
// half waves each add up every 32nd group (8 loads of 256 groups, all in flight), and the first adds the 32 sums.
template <class WT>
__global__ __launch_bounds__(1024) void norm_bwd_finish(NormBwdArgs a) {
  constexpr int kCols = 32, kParts = 1024 / kCols;
  __shared__ float lds[kParts][kCols];
  const uint32_t w = threadIdx.x / kCols;
  const size_t first = static_cast<size_t>(blockIdx.x) * kCols, n = 2 * a.cols;
  for (size_t block = first; block < n; block += static_cast<size_t>(gridDim.x) * kCols) {
    if (block != first) __syncthreads();  // the last columns' sums have been read
    const size_t c = block + threadIdx.x % kCols;
    float s = 0.0f;
    if (c < n) {
#pragma unroll 8
      for (uint32_t g = w; g < a.groups; g += kParts) s += a.part[g * n + c];
    }
    lds[w][threadIdx.x % kCols] = s;
    __syncthreads();
    if (w || c >= n) continue;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) s += lds[i][threadIdx.x];
    write_weight<WT>(a, c, s);
  }
}

// The shape of a row that is held in registers: lanes (B, waves) and packs a lane; K = 0 if it is not.
struct Held {
  int B, waves, K;
};
Held held(size_t cols, int kV) {
  const size_t packs = (cols + kV - 1) / kV;
  if (cols < static_cast<size_t>(kV) || cols > 16384) return {0, 0, 0};
  if (packs <= 32) return {packs <= 8 ? 8 : packs <= 16 ? 16 : 32, 1, 1};
  const int waves = static_cast<int>((packs + 63) / 64);
  return waves <= 16 ? Held{kWaves, waves, 1} : waves <= 32 ? Held{kWaves, (waves + 1) / 2, 2} : Held{kWaves, (waves + 3) / 4, 4};
}
// Rows of a set.  (Two packs a lane for rows of up to 8192 16-bit elements, on sets of 768 lanes, measured slower: 65536 x
// 1024 bf16 with dres 90 -> 103 us, 8192 x 4096 51.4 -> 54.0.)
int set_of(const Held& h) { return h.K > 1 ? 1 : kBwdLanes / (h.B == kWaves ? h.waves * 64 : h.B); }

template <class T, class WT, int B, int K>
void bwd_row(NormBwdArgs a, const Held& h, hipStream_t st) {
  a.waves = h.waves;
  const dim3 grid(a.groups), block(set_of(h) * (B == kWaves ? h.waves * 64 : B));
  if (K > 1 && block.x <= 768) {
    if constexpr (K > 1) {
      if (a.dres)
        hipLaunchKernelGGL((norm_bwd_row<T, WT, B, K, true, 768>), grid, block, 0, st, a);
      else
        hipLaunchKernelGGL((norm_bwd_row<T, WT, B, K, false, 768>), grid, block, 0, st, a);
    }
  } else if (a.dres) {
    hipLaunchKernelGGL((norm_bwd_row<T, WT, B, K, true, 1024>), grid, block, 0, st, a);
  } else {
    hipLaunchKernelGGL((norm_bwd_row<T, WT, B, K, false, 1024>), grid, block, 0, st, a);
  }
}

template <class T, class WT>
void bwd_any(const NormBwdArgs& a, size_t packs, hipStream_t st) {
  if (a.part)  // first: dx may take the place of x or dy
    hipLaunchKernelGGL((norm_bwd_any_weights<T>), dim3(static_cast<uint32_t>((packs + 63) / 64), a.groups), dim3(64), 0, st, a);
  if (a.dx) hipLaunchKernelGGL((norm_bwd_any_dx<T, WT>), dim3(norm_grid(a.rows)), dim3(1024), 0, st, a);
}

// Does the launch's last workgroup add the partial sums up by itself, sparing the second launch?  Where its lanes need at
// most two rounds of loads: a pass of 1000 x 100 fp32, 64 x 512 or 16 x 1024 bf16 takes 8.2 us from the host with it and 11.3
// without.  Device-scope loads make a round 2 to 3 us: 256 x 1024 bf16 (8 rounds) took 25 us with and 11.3 without.
bool one_launch(const NormBwdArgs& a, const Held& h) {
  if (!h.K || !a.dx || !a.part) return false;
  if (a.groups == 1) return true;  // no partial sums at all
  const size_t n = 2 * a.cols, lanes = set_of(h) * (h.B == kWaves ? h.waves * 64 : h.B);
  const size_t loads = n < lanes ? (a.groups + lanes / n - 1) / (lanes / n) : a.groups;  // of a lane, for one column
  return (n + lanes - 1) / lanes * ((loads + 7) / 8) <= 2;
}

template <class T, class WT>
hipError_t bwd(NormBwdArgs a, hipStream_t st) {
  constexpr int kV = kPack<T>;
  const size_t packs = (a.cols + kV - 1) / kV;
  if (a.rows) {
    const Held h = held(a.cols, kV);
    a.one_launch = one_launch(a, h);
    if (a.cols < kV)
      hipLaunchKernelGGL((norm_bwd_tiny<T, WT>), dim3(a.groups), dim3(64), 0, st, a);
    else if (h.K == 0 || !a.dx)
      bwd_any<T, WT>(a, packs, st);
    else if (h.B == 8)
      bwd_row<T, WT, 8, 1>(a, h, st);
    else if (h.B == 16)
      bwd_row<T, WT, 16, 1>(a, h, st);
    else if (h.B == 32)
      bwd_row<T, WT, 32, 1>(a, h, st);
    else if (h.K == 1)
      bwd_row<T, WT, kWaves, 1>(a, h, st);
    else if (h.K == 2)
      bwd_row<T, WT, kWaves, 2>(a, h, st);
    else if constexpr (kV == 4)
      bwd_row<T, WT, kWaves, 4>(a, h, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.part && !a.one_launch)
    hipLaunchKernelGGL((norm_bwd_finish<WT>), dim3(norm_grid((2 * a.cols + 31) / 32)), dim3(1024), 0, st, a);
  return hipGetLastError();
}

}  // namespace

uint32_t norm_bwd_groups(size_t rows, size_t cols, mr_dtype dt) {
  const Held h = held(cols, 16 / elem_size(dt));
  const bool tiny = cols < static_cast<size_t>(16 / elem_size(dt));
  const size_t set = h.K ? set_of(h) : tiny ? 64 : 1, most = h.K ? 256 : tiny ? 1024 : 64;
  const size_t want = (rows + set - 1) / set;
  return static_cast<uint32_t>(want < most ? want : most);
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, mr_dtype dt, mr_dtype wdt, hipStream_t st) {
  if (dt == MR_FP32) return bwd<EFp32, EFp32>(a, st);
  if (dt == MR_BF16) return wdt == MR_FP32 ? bwd<EBf16, EFp32>(a, st) : bwd<EBf16, EBf16>(a, st);
  return wdt == MR_FP32 ? bwd<EFp16, EFp32>(a, st) : bwd<EFp16, EFp16>(a, st);
}

}  // namespace mr
