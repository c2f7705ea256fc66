// Losses on logits for gfx950: log-probabilities of target tokens, their backward pass, the clipped policy loss with a
// KL term, and the preference loss over pairs of sequences.
//
//   m = max z,  S = sum exp((z - m) / T),  logp = (z_t - m) / T - ln S,   d logp / d z_j = ([j = t] - exp((z_j - m) / T) / S) / T
//
// Row statistics are taken online, in one pass: a lane keeps the maximum and the sum of what it has seen, and scales the sum
// down where the maximum rises.  Exponents are (z - m) * log2(e)/T, not z * log2(e)/T - m * log2(e)/T: the difference is
// exact near the maximum, and a row whose every element is the type's lowest value stays a uniform distribution.
//
// The policy loss's gradient needs nothing but its own row, so a row that fits the registers of a workgroup is read once
// and its gradient written straight from them (policy_held).  Longer rows, and calls of too few rows to fill the device, go over
// the logits twice: row_stats, whose workgroups may share a row, and logit_grad.

#include <hip/hip_runtime.h>
#include <math.h>

#include "mr_train.h"
#include "packs.h"

namespace mr {
namespace {

constexpr float kNone = -__builtin_huge_valf();

// Running maximum and sum of exp2((z - maximum) * c).
struct Stat {
  float m, s;
};
// What exponents are taken against: a row of -inf alone has sum 0, not NaN.
__device__ __forceinline__ float base_of(float m) { return m == kNone ? 0.0f : m; }
__device__ __forceinline__ float power(float z, float base, float c) { return __builtin_amdgcn_exp2f((z - base) * c); }

template <int N>
__device__ __forceinline__ void add_values(Stat& a, const float (&f)[N], float c) {
  float m = a.m;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, f[i]);
  const float base = base_of(m);
  float s0 = a.s * power(a.m, base, c), s1 = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    s0 += power(f[i], base, c);
    s1 += power(f[i + 1], base, c);
  }
  a.m = m;
  a.s = s0 + s1;
}
__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, dpp<0xB1>(x));   // quad lanes 1 0 3 2
  x = fmaxf(x, dpp<0x4E>(x));   // quad lanes 2 3 0 1
  x = fmaxf(x, dpp<0x141>(x));  // half row mirrored
  x = fmaxf(x, dpp<0x140>(x));  // row mirrored
  const int b = __float_as_int(x);
  return fmaxf(fmaxf(__int_as_float(__builtin_amdgcn_readlane(b, 0)), __int_as_float(__builtin_amdgcn_readlane(b, 16))),
               fmaxf(__int_as_float(__builtin_amdgcn_readlane(b, 32)), __int_as_float(__builtin_amdgcn_readlane(b, 48))));
}
__device__ __forceinline__ Stat wave_join(Stat a, float c) {
  const float m = wave_max(a.m);
  a.s = lanes_sum<64>(a.s * power(a.m, base_of(m), c));
  a.m = m;
  return a;
}

// The sum of a workgroup's waves, in every lane: one join over the lanes, not one after another.
constexpr int kMostWaves = 16;
__device__ __forceinline__ Stat all_waves(const Stat* words, uint32_t waves, float c) {
  const uint32_t lane = threadIdx.x & 63;
  Stat st{kNone, 0.0f};
  if (lane < waves) st = words[lane];
  return waves > 1 ? wave_join(st, c) : Stat{__shfl(st.m, 0), __shfl(st.s, 0)};
}

// ln S without the rounding of a large logarithm: S = f * 2^e with f around 1, so that ln 1 is 0.
__device__ __forceinline__ double ln(float S) {
  int e;
  float f = frexpf(S, &e);
  if (f < 0.70710678f) f *= 2.0f, e -= 1;
  return static_cast<double>(e) * 0.6931471805599453 + static_cast<double>(logf(f));
}
__device__ __forceinline__ double logp_of(const LogitArgs& a, float m, float S, float zt) {
  return (static_cast<double>(zt) - static_cast<double>(m)) * a.inv_temp - ln(S);
}

// A value of a row, at an address that is the same for every lane and that this launch does not write: by way of the scalar
// cache, whose loads do not wait in line behind the vector loads of a row.
template <class X>
__device__ __forceinline__ X row_value(const X* p) {
  return *reinterpret_cast<const __attribute__((address_space(4))) X*>(reinterpret_cast<uintptr_t>(p));
}

// A row that carries a loss: its target is one of the columns, and its weight is not zero.
// (The same for every lane: read into scalar registers, so that rows' addresses are too.)
__device__ __forceinline__ bool row_live(const LogitArgs& a, size_t row, uint32_t* t) {
  const uint64_t x = static_cast<uint64_t>(row_value(a.targets + row));
  *t = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x));
  const uint32_t high = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x >> 32));
  uint32_t weight = 1;
  if (a.weights) weight = __builtin_amdgcn_readfirstlane(__float_as_uint(row_value(a.weights + row))) << 1;
  return high == 0 && *t < static_cast<uint32_t>(a.cols) && weight != 0;
}

// exp(d), past fp32's range as an eighth power, finite as far as fp64 goes (expf's error 8 times over: 2^-20): what a coefficient of 0 or a
// small weight multiplies stays a number.
constexpr float kExpRange = 88.0f;
__device__ __forceinline__ double exp_of(float d) {
  const bool past = d > kExpRange;
  double e = static_cast<double>(expf(past ? 0.125f * d : d));
  if (!past) return e;
  e *= e;
  e *= e;
  return e * e;
}

// exp(d) - d - 1 (`e` is expm1f(d)), without the cancellation of its leading terms where d is small: there its power series,
// whose first term left out, d^11 / 11!, is below 2^-23 of the sum for |d| <= 1 (2^-24 down to d = -0.98).
__device__ __forceinline__ float excess(float d, float e) {
  if (fabsf(d) > 1.0f) return e - d;
  float p = 1.0f + d * (1.0f / 10.0f);
#pragma unroll
  for (int n = 9; n >= 3; --n) p = 1.0f + d * p * (1.0f / static_cast<float>(n));
  return 0.5f * d * d * p;
}

// The policy loss of one row: the gradient of its log-probability (grad_scale in it), and its terms of the record.
struct PolicyRow {
  float g;
  double loss, kl, held, w;
};
struct PolicyIn {
  float w, adv, old, ref;
  __device__ PolicyIn(const LogitArgs& a, size_t row)
      : w(a.weights ? row_value(a.weights + row) : 1.0f), adv(row_value(a.adv + row)), old(a.old_logp ? row_value(a.old_logp + row) : 0.0f),
        ref(a.ref_logp ? row_value(a.ref_logp + row) : 0.0f) {}
};
__device__ __forceinline__ PolicyRow policy_row(const LogitArgs& a, const PolicyIn& in, double logp) {
  const double w = static_cast<double>(in.w), adv = static_cast<double>(in.adv);
  // (without old_logp: NaN stays, and a target that is ruled out has r = 1 too)
  const double r = a.old_logp ? exp_of(static_cast<float>(logp - static_cast<double>(in.old))) : logp != logp ? logp : 1.0;
  double near = r < 1.0 - a.clip_lo ? 1.0 - a.clip_lo : r;
  near = near > 1.0 + a.clip_hi ? 1.0 + a.clip_hi : near;
  const double free = -adv * r, held = -adv * near;
  const bool cut = held > free;
  PolicyRow p;
  double g = cut ? 0.0 : free, k = 0.0, term = 0.0;
  if (a.ref_logp) {
    const float d = static_cast<float>(static_cast<double>(in.ref) - logp);
    const float e = expm1f(d);
    double more = static_cast<double>(e);
    k = static_cast<double>(excess(d, e));
    if (d > kExpRange) more = k = exp_of(d);
    if (a.kl != 0.0) {  // a coefficient of 0 leaves the term out, whatever it is
      g -= a.kl * more;
      term = a.kl * k;
    }
  }
  p.g = static_cast<float>(a.grad_scale * w * g);
  p.loss = w * ((cut ? held : free) + term);
  p.kl = w * k;
  p.held = cut ? w : 0.0;
  p.w = w;
  return p;
}

// Workgroups' sums to the record, in up to 8 sets of workgroups.  Each leaves four through write-through stores, acknowledged
// before its arrival is counted; the one that arrives last of its set adds the set's up, and the last of those the sets', all
// in their order.  (One set of 1024: 46 us of a preference loss, most of it one wave's loads after another.)
__device__ __forceinline__ void leave4(double* p, double v0, double v1, double v2, double v3) {
  __hip_atomic_store(p, v0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(p + 1, v1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(p + 2, v2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(p + 3, v3, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Counts an arrival after this lane's stores; is it the last of `members`?
__device__ __forceinline__ bool arrive(uint32_t* count, uint32_t members) {
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  const bool last = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == members - 1;
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  return last;
}
// A wave's sum of n entries of four values, `stride` entries apart; lane j has value j % 4.  8 loads of a lane are on their way at once.
__device__ __forceinline__ double sum4(const double* p, uint32_t n, uint32_t stride) {
  const uint32_t lane = threadIdx.x & 63;
  double s = 0.0;
  for (uint32_t i0 = lane >> 2; i0 < n; i0 += 128) {
    double v[8];
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
      const uint32_t i = i0 + 16 * k < n ? i0 + 16 * k : i0;
      v[k] = __hip_atomic_load(p + size_t{i} * stride * 4 + (lane & 3), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) s += i0 + 16 * k < n ? v[k] : 0.0;
  }
#pragma unroll
  for (int m = 32; m >= 4; m >>= 1) s += __shfl_xor(s, m);
  return s;
}
// By the first wave of every workgroup, with the sums in its first lane.
__device__ __forceinline__ void finish_record(double v0, double v1, double v2, double v3, double* sums, uint32_t (*arrived)[64],
                                              float* record, uint32_t words) {
  const uint32_t groups = gridDim.x, lane = threadIdx.x;
  if (lane >= 64) return;
  const uint32_t sets = groups < 4 * kNormSets ? 1 : kNormSets, set = blockIdx.x % sets, members = (groups - set + sets - 1) / sets;
  int last = 0;
  if (lane == 0) {
    leave4(sums + size_t{blockIdx.x} * 4, v0, v1, v2, v3);
    last = arrive(&arrived[set][0], members);
  }
  if (!__shfl(last, 0)) return;
  double s = sum4(sums + size_t{set} * 4, members, sets);
  if (sets > 1) {
    double* of_sets = sums + size_t{groups} * 4;
    if (lane < 4) __hip_atomic_store(of_sets + set * 4 + lane, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (lane == 0) last = arrive(&arrived[kNormSets][0], sets);  // (waits for the stores of the whole wave)
    if (!__shfl(last, 0)) return;
    s = sum4(of_sets, sets, 1);
  }
  if (lane <= kNormSets) __hip_atomic_store(&arrived[lane][0], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (lane < words) record[lane] = static_cast<float>(s);
}

// Rows are read in packs on z's 16-byte grid, so the first pack of a row that starts off it holds `off` elements less.
template <class T>
__device__ __forceinline__ uint32_t row_off(const char* z) {
  return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(z) & 15u)) / T::kSize;
}
// The columns of pack p of a row: `n` (0 or less: none) from `col` on.
template <int V>
struct PackAt {
  size_t col;
  int n;
  __device__ PackAt(size_t p, uint32_t off, size_t cols) {
    const int64_t c = static_cast<int64_t>(p * V) - off, end = c + V < static_cast<int64_t>(cols) ? c + V : static_cast<int64_t>(cols);
    col = c < 0 ? 0 : static_cast<size_t>(c);
    n = end - static_cast<int64_t>(col) < 0 ? 0 : static_cast<int>(end - static_cast<int64_t>(col));
  }
};

// --------------------------------------------------------------------------------- statistics of rows
//
// A workgroup takes one of `splits` parts of a row.  The parts' maxima and sums are joined, in their order, by the workgroup
// that finishes its row last.  Bound by the reads: 16384 rows of 50001 fp16 columns, a tenth of them without a loss, in 225 us (6.5 TB/s
// of 1.475 GB); 8192 of 32768 fp32 in 154 (6.97 TB/s).  Rows of a wave or less are bound by the 600 instructions a row: 65536 of 512
// bf16 in 39 us.
// Packs a lane has in flight: 4 take 62 us there, 2 take 39; 16384 rows of 50001 271 and 262 at the same lanes; 8 take 410.
constexpr int kStatPacks = 2;

template <class T, bool Policy>
__global__ __launch_bounds__(1024) void row_stats(LogitArgs a) {
  constexpr int V = 16 / T::kSize;
  __shared__ Stat waves[kMostWaves];
  __shared__ bool last;
  const uint32_t lanes = blockDim.x, lane = threadIdx.x;
  const size_t parts = a.rows * a.splits;
  const size_t packs = a.packs, per = (packs + a.splits - 1) / a.splits;
  double loss = 0.0, kl = 0.0, cut = 0.0, weight = 0.0;
  uint32_t t = 0, t_next = 0;
  bool live = blockIdx.x < parts && row_live(a, blockIdx.x / a.splits, &t), live_next = false;
  for (size_t part = blockIdx.x; part < parts; part += gridDim.x, t = t_next, live = live_next) {
    const size_t row = part / a.splits, next = part + gridDim.x;
    const uint32_t split = static_cast<uint32_t>(part % a.splits);
    if (!live) {  // the same for every lane, and for every part of the row
      if (lane == 0 && split == 0) {
        if (a.logp) a.logp[row] = 0.0f;
        if (a.stats) a.stats[2 * row] = a.stats[2 * row + 1] = 0.0f;
        if (Policy && a.dz) const_cast<float*>(a.dlogp)[row] = 0.0f;
      }
      live_next = next < parts && row_live(a, next / a.splits, &t_next);
      continue;
    }
    const char* z = a.z + row * a.stride * T::kSize;
    const uint32_t off = row_off<T>(z);
    const char* grid = z - off * T::kSize;  // where pack 0 would start
    const float zt = load1<T>(z + static_cast<size_t>(t) * T::kSize);
    const size_t first = split * per, end = first + per < packs ? first + per : packs;
    Stat st{kNone, 0.0f};
    for (size_t p = first + lane; p < end; p += static_cast<size_t>(lanes) * kStatPacks) {
      float f[kStatPacks * V];
      Raw<T, V> raw[kStatPacks];
      const size_t p0 = p - lane, top = p0 + static_cast<size_t>(lanes) * kStatPacks;
      if (top <= end && top * V <= a.cols + off && (p0 > 0 || off == 0)) {  // the same for every lane
#pragma unroll
        for (int k = 0; k < kStatPacks; ++k) raw[k] = load_raw<T, V, true>(grid + (p + static_cast<size_t>(lanes) * k) * 16);
#pragma unroll
        for (int k = 0; k < kStatPacks; ++k) widen(raw[k], reinterpret_cast<float(&)[V]>(f[k * V]));
      } else if (a.cols >= V) {
        // packs that pass an end of the row are read as V elements from that end on; those that are another pack's are left out
        int from[kStatPacks];
#pragma unroll
        for (int k = 0; k < kStatPacks; ++k) {
          const size_t q = p + static_cast<size_t>(lanes) * k;
          const int64_t c = static_cast<int64_t>(q * V) - off, last = static_cast<int64_t>(a.cols) - V, at = c < 0 ? 0 : c < last ? c : last;
          from[k] = q < end && c - at < V ? static_cast<int>(c - at) : V;
          raw[k] = load_raw<T, V, true>(z + at * T::kSize);
        }
#pragma unroll
        for (int k = 0; k < kStatPacks; ++k) {
          float (&g)[V] = reinterpret_cast<float(&)[V]>(f[k * V]);
          widen(raw[k], g);
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (i < from[k] || i >= from[k] + V) g[i] = kNone;
        }
      } else {
#pragma unroll
        for (int k = 0; k < kStatPacks; ++k) {
          const size_t q = p + static_cast<size_t>(lanes) * k;
          const PackAt<V> at(q, off, a.cols);
          const int n = q < end ? at.n : 0;
          float (&g)[V] = reinterpret_cast<float(&)[V]>(f[k * V]);
          widen(load_part<T, V, true>(z + at.col * T::kSize, n), g);
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (i >= n) g[i] = kNone;
        }
      }
      add_values(st, f, a.c);
    }
    live_next = next < parts && row_live(a, next / a.splits, &t_next);
    st = wave_join(st, a.c);
    if (lanes > 64) {
      __syncthreads();  // the last row's words have been read
      if ((lane & 63) == 0) waves[lane >> 6] = st;
      __syncthreads();
      if (lane < 64) st = all_waves(waves, lanes / 64, a.c);
    }
    if (lane >= 64 && a.splits == 1) continue;
    if (a.splits > 1) {
      if (lane == 0) {
        float* at = a.part + part * 2;
        __hip_atomic_store(at, st.m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(at + 1, st.s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        last = __hip_atomic_fetch_add(a.row_arrived + row, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.splits - 1;
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        if (last) __hip_atomic_store(a.row_arrived + row, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __syncthreads();
      if (!last || lane >= 64) continue;
      Stat mine{kNone, 0.0f};
      if (lane < a.splits) {
        const float* at = a.part + (row * a.splits + lane) * 2;
        mine.m = __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        mine.s = __hip_atomic_load(at + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      st = wave_join(mine, a.c);
    }
    const double lp = logp_of(a, st.m, st.s, zt);
    if (lane == 0) {
      if (a.logp) a.logp[row] = static_cast<float>(lp);
      if (a.stats) {
        a.stats[2 * row] = st.m;
        a.stats[2 * row + 1] = st.s;
      }
      if constexpr (Policy) {
        const PolicyRow p = policy_row(a, PolicyIn(a, row), lp);
        if (a.dz) const_cast<float*>(a.dlogp)[row] = p.g;
        loss += p.loss, kl += p.kl, cut += p.held, weight += p.w;
      }
    }
  }
  if constexpr (Policy) finish_record(loss, kl, cut, weight, a.sums, a.arrived, a.record, 4);
}

// ------------------------------------------------------------------------------ gradient of the logits
//
// dz_j = g/T ([j = t] - exp((z_j - m) / T) / S), element by element; a wave takes a run of packs of one row.  Bound by the bytes: 8192
// rows of 32768 fp32 columns in 339 us (6.33 TB/s, what a copy reaches); 16384 of 50001 bf16, off the 16-byte grid, in 565 (5.8).
// A wave's packs a lane, 2, 4 and 8: 4096 rows of 131072 bf16 344, 352 and 362 us; 65536 of 512 27, 36 and 56.
constexpr int kGradPacks = 2;

template <class T>
__global__ __launch_bounds__(256) void logit_grad(LogitArgs a) {
  constexpr int V = 16 / T::kSize;
  constexpr uint32_t lanes = 64;
  const uint32_t lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const size_t packs = a.packs, run = size_t{lanes} * kGradPacks;
  const size_t runs = (packs + run - 1) / run;
  for (size_t item = size_t{blockIdx.x} * 4 + wave; item < a.rows * runs; item += size_t{gridDim.x} * 4) {
    const size_t row = item / runs, p0 = item % runs * run + lane;
    uint32_t t;
    const bool live = row_live(a, row, &t);  // (the backward pass has no weights)
    const char* z = a.z + row * a.stride * T::kSize;
    char* dz = a.dz + row * a.dstride * T::kSize;
    const uint32_t off = row_off<T>(z);
    const bool whole = (p0 - lane + run) * V <= a.cols + off && (p0 > lane || off == 0);
    if (!live) {
      const float none[V] = {};
#pragma unroll
      for (int k = 0; k < kGradPacks; ++k) {
        const PackAt<V> at(p0 + static_cast<size_t>(lanes) * k, off, a.cols);
        if (at.n > 0) store_part<T, V, true>(dz + at.col * T::kSize, none, at.n);
      }
      continue;
    }
    Raw<T, V> raw[kGradPacks];
#pragma unroll
    for (int k = 0; k < kGradPacks; ++k) {
      const size_t q = p0 + static_cast<size_t>(lanes) * k;
      if (whole) {
        raw[k] = load_raw<T, V, true>(z + q * 16 - off * T::kSize);
      } else {
        const PackAt<V> at(q, off, a.cols);
        raw[k] = load_part<T, V, true>(z + at.col * T::kSize, at.n);
      }
    }
    const float base = base_of(a.stats[2 * row]), g = static_cast<float>(static_cast<double>(a.dlogp[row]) * a.inv_temp);
    const float share = -g / a.stats[2 * row + 1];
#pragma unroll
    for (int k = 0; k < kGradPacks; ++k) {
      const PackAt<V> p(p0 + static_cast<size_t>(lanes) * k, off, a.cols);
      if (!whole && p.n <= 0) continue;
      float f[V];
      widen(raw[k], f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = share * power(f[i], base, a.c);
      const uint64_t at = static_cast<uint64_t>(t) - p.col;
      if (at < V) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (at == static_cast<uint64_t>(i)) f[i] += g;
      }
      if (whole)
        store_raw<T, V, true>(dz + p.col * T::kSize, narrow<T, V>(f));
      else
        store_part<T, V, true>(dz + p.col * T::kSize, f, p.n);
    }
  }
}

// ------------------------------------------------------------------------- the policy loss in one pass
//
// A workgroup holds a row in registers, K packs a lane, and walks the rows.  As each pack's gradient leaves, the next row's
// pack is loaded into its place, so that reads and writes flow together.  One barrier a row: its words are of alternating
// sets; the next row's target is read a row ahead.  Packs lie on z's 16-byte grid; only the first strip's first pack and
// the last two of the K strips can pass the row's ends (held_row).  Such a pack is read, and stored, as V whole elements from the
// nearest end on; those that are another pack's add nothing to the sums, and both store the same bits.
//
// Bound by the bytes, and by what a workgroup waits between a row's last load and its first store: 8192 rows of 131072 bf16 in
// 802 to 822 us (5.3 TB/s; no less with the exponentials left out), 8192 of 32768 fp32 in 379 (5.7), 16384 of 50001 bf16 in 685 (4.8;
// of 50048, whose rows start on 128-byte lines, 616 to 626).  Rows are dealt out by a stride, so the workgroups that meet no ignored row set
// the time: 4096 of 50001 take 169 to 179 all live, and 173 with a quarter ignored.  K = 16 keeps 4 registers in scratch (20 bytes a lane), which
// its row loop loads again; no other K does.  (Statistics and gradient as two passes over the same rows: 160 + 344 us for 4096 of 131072,
// here 402; at most 8, 10 or 12 packs a lane instead of 16 are no faster, nor are loads and stores that stay in the caches.)
template <class T, int K>
__global__ __launch_bounds__(1024) void policy_held(LogitArgs a) {
  constexpr int V = 16 / T::kSize, kEnd = K < 2 ? K : 2;
  __shared__ Stat words[2][kMostWaves];
  __shared__ double sums[4];  // the first lane's
  const uint32_t lanes = blockDim.x, lane = threadIdx.x, nw = lanes / 64;
  const int last = static_cast<int>(a.cols) - V;  // the last column where a pack can start
  auto at_end = [](int k) { return k == 0 || k >= K - kEnd; };
  // Bytes from the row's start to a lane's pack of strip k, as a part of all lanes (scalar) and its own.
  struct Place {
    int64_t all;
    uint32_t own;
  };
  auto column = [&](uint32_t off, int k) { return static_cast<int>((k * lanes + lane) * V) - static_cast<int>(off); };
  auto place = [&](uint32_t off, int k) {
    if (!at_end(k)) return Place{(static_cast<int64_t>(k * lanes * V) - off) * T::kSize, lane * 16};
    int c = column(off, k);
    c = c < last ? c : last;
    return Place{0, static_cast<uint32_t>(c < 0 ? 0 : c) * T::kSize};
  };
  if (lane == 0) sums[0] = sums[1] = sums[2] = sums[3] = 0.0;
  Raw<T, V> raw[K];
  // A row's packs; where there is no row to load, every lane reads the first pack of this one.  Loads behind a branch would keep
  // the packs that leave and those that come in registers of their own.
  auto load = [&](const char* z, uint32_t off, uint32_t some, int k) {
    const Place p = place(off, k);
    raw[k] = load_raw<T, V, true>(z + (p.all & static_cast<int32_t>(some)) + (p.own & some));
  };
  const size_t step = gridDim.x;
  uint32_t t_next = 0;
  // The first row at or after r that carries a loss; those before it get their zeros.
  auto advance = [&](size_t r) {
    for (; r < a.rows && !row_live(a, r, &t_next); r += step) {
      char* dz = a.dz + r * a.dstride * T::kSize;
      const uint32_t off = row_off<T>(a.z + r * a.stride * T::kSize);
      if (lane == 0 && a.logp) a.logp[r] = 0.0f;
      const float none[V] = {};
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const Place p = place(off, k);
        store_raw<T, V, true>(dz + p.all + p.own, narrow<T, V>(none));
      }
    }
    return r;
  };
  size_t row = advance(blockIdx.x), next = row;
  uint32_t t = t_next, off = 0;
  const char* z = a.z;
  if (row < a.rows) {
    z += row * a.stride * T::kSize;
    off = row_off<T>(z);
  }
#pragma unroll
  for (int k = 0; k < K; ++k) load(z, off, row < a.rows ? ~0u : 0u, k);
  for (uint32_t turn = 0; row < a.rows; row = next, ++turn) {
    const float zt = load1<T>(z + size_t{t} * T::kSize);
    const PolicyIn in(a, row);
    next = advance(row + step);
    const uint32_t some = next < a.rows ? ~0u : 0u;
    const char* z_next = a.z + (some ? next : row) * a.stride * T::kSize;
    const uint32_t off_next = row_off<T>(z_next);
    char* dz = a.dz + row * a.dstride * T::kSize;
    Stat st{kNone, 0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      // packs in turn: their values are not held beside one another
#pragma unroll
      for (int i = 0; i < Raw<T, V>::kWords; ++i) asm volatile("" : "+v"(raw[k].w[i]), "+v"(st.m), "+v"(st.s));
      float f[V];
      widen(raw[k], f);
      if (at_end(k)) {
        // columns of the pack that are its own: from its place on the grid on, V of them
        const int c = column(off, k), at = c < last ? c < 0 ? 0 : c : last;
        int from = c - at;
        asm volatile("" : "+v"(from));  // compared anew in every row: kept, the comparisons' masks would take 16 scalar registers a strip
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (k == 0 ? i < from || i >= from + V : i < from) f[i] = kNone;
      }
      add_values(st, f, a.c);
    }
    st = wave_join(st, a.c);
    if ((lane & 63) == 0) words[turn & 1][lane >> 6] = st;
    __syncthreads();
    st = all_waves(words[turn & 1], nw, a.c);
    const double lp = logp_of(a, st.m, st.s, zt);
    const PolicyRow p = policy_row(a, in, lp);
    if (lane == 0) {
      if (a.logp) a.logp[row] = static_cast<float>(lp);
      sums[0] += p.loss, sums[1] += p.kl, sums[2] += p.held, sums[3] += p.w;
    }
    const float base = base_of(st.m), g = static_cast<float>(static_cast<double>(p.g) * a.inv_temp), share = -g / st.s;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      // widened anew: kept from the sums, the values would take twice the registers that hold the row
#pragma unroll
      for (int i = 0; i < Raw<T, V>::kWords; ++i) asm volatile("" : "+v"(raw[k].w[i]));
      float f[V];
      widen(raw[k], f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = share * power(f[i], base, a.c);
      const Place to = place(off, k);
      store_raw<T, V, true>(dz + to.all + to.own, narrow<T, V>(f));
      load(z_next, off_next, some, k);
      __builtin_amdgcn_sched_barrier(0);
    }
    // The target's own element, by every lane that stored a pack with it, after that pack: one of them writes it last.
    const uint32_t q = (t + off) / V;
    bool mine = q % lanes == lane;  // it is on the grid
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (at_end(k)) mine = mine || t - place(off, k).own / T::kSize < V;
    if (mine) store1<T>(dz + size_t{t} * T::kSize, share * power(zt, base, a.c) + g);
    t = t_next;
    off = off_next;
    z = z_next;
  }
  finish_record(sums[0], sums[1], sums[2], sums[3], a.sums, a.arrived, a.record, 4);
}

// ------------------------------------------------------------------------------------- preference loss

__device__ __forceinline__ double group_sum(double x, double* lds) {
  x = wave_sum(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0.0;
  for (uint32_t i = 0; i < blockDim.x / 64; ++i) x += lds[i];
  return x;
}

constexpr int kPrefPacks = 2;  // of 4 floats that a lane has in flight, of each input

// A workgroup takes a pair: the sums of both sequences' log ratios in fp64, then the gradient of each of their tokens.  1024 pairs of
// 4.4M tokens in 20.4 us: 52.8 MB, 2.6 TB/s.  The longest pairs set it: a workgroup's share is two trips through a few rounds of loads
// (8 pairs of 2 x 16384 20.5 us, one of 2 x 100000 96).
__global__ __launch_bounds__(256, 4) void preference(PreferenceArgs a) {
  __shared__ double lds[kMostWaves];
  const uint32_t lanes = blockDim.x, lane = threadIdx.x;
  const int64_t rows = static_cast<int64_t>(a.rows);
  auto bound = [&](size_t i) {
    const int64_t o = a.offsets[i];
    return o < 0 ? 0 : o > rows ? rows : o;
  };
  double loss = 0.0, right = 0.0, margin = 0.0;
  for (size_t pair = blockIdx.x; pair < a.pairs; pair += gridDim.x) {
    const int64_t from = bound(2 * pair), mid = bound(2 * pair + 1), to = bound(2 * pair + 2);
    double s = 0.0;  // the chosen sequence's sum less the rejected one's
    for (int64_t i0 = from + lane * 4; i0 < to; i0 += int64_t{lanes} * 4 * kPrefPacks) {
      Raw<EFp32, 4> x[kPrefPacks], y[kPrefPacks];
#pragma unroll
      for (int k = 0; k < kPrefPacks; ++k) {
        const int64_t i = i0 + int64_t{lanes} * 4 * k;
        const int n = i >= to ? 0 : to - i < 4 ? static_cast<int>(to - i) : 4;
        x[k] = load_part<EFp32, 4, false>(reinterpret_cast<const char*>(a.logp + i), n);
        y[k] = load_part<EFp32, 4, false>(reinterpret_cast<const char*>(a.ref + i), a.ref ? n : 0);
      }
#pragma unroll
      for (int k = 0; k < kPrefPacks; ++k) {
        const int64_t i = i0 + int64_t{lanes} * 4 * k;
        float u[4], v[4];
        widen(x[k], u);
        widen(y[k], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const double d = static_cast<double>(u[j]) - static_cast<double>(v[j]);
          s += i + j < mid ? d : -d;
        }
      }
    }
    const double h = a.beta * group_sum(s, lds);
    const double e = exp(-fabs(h)), small = log1p(e);  // -ln sigmoid(x) = log1p(exp(-|x|)) + max(-x, 0)
    const double below = e / (1.0 + e), sig_minus = h >= 0.0 ? below : 1.0 - below;  // sigmoid(-h)
    if (lane == 0) {
      loss += (1.0 - a.smoothing) * (small + fmax(-h, 0.0));
      if (a.smoothing > 0.0) loss += a.smoothing * (small + fmax(h, 0.0));
      right += h > 0.0 ? 1.0 : 0.0;
      margin += h;
      if (a.margins) a.margins[pair] = static_cast<float>(h);
    }
    if (a.dlogp) {
      const float g = static_cast<float>(a.grad_scale * a.loss_scale * a.beta * (a.smoothing - sig_minus));
      for (int64_t i = from + lane * 4; i < to; i += int64_t{lanes} * 4) {
        const float v[4] = {i < mid ? g : -g, i + 1 < mid ? g : -g, i + 2 < mid ? g : -g, i + 3 < mid ? g : -g};
        store_part<EFp32, 4, false>(reinterpret_cast<char*>(a.dlogp + i), v, to - i < 4 ? static_cast<int>(to - i) : 4);
      }
    }
  }
  if (a.dlogp) {  // rows of no sequence
    const int64_t first = bound(0), end = bound(2 * a.pairs), step = static_cast<int64_t>(gridDim.x) * lanes;
    const int64_t me = static_cast<int64_t>(blockIdx.x) * lanes + lane;
    for (int64_t i = me; i < first; i += step) a.dlogp[i] = 0.0f;
    for (int64_t i = (end > first ? end : first) + me; i < rows; i += step) a.dlogp[i] = 0.0f;
  }
  const double n = a.pairs ? 1.0 / static_cast<double>(a.pairs) : 0.0;
  finish_record(loss * a.loss_scale, right * n, margin * n, 0.0, a.sums, a.arrived, a.record, 3);
}

// ---------------------------------------------------------------------------------------------- launches

constexpr size_t kMostGrid = size_t{1} << 20;  // below 2^32 lanes; kernels loop over what lies past their grid
inline uint32_t grid_of(size_t n) { return static_cast<uint32_t>(n < kMostGrid ? n : kMostGrid); }


bool rows_on_grid(const char* z, size_t rows, size_t stride, size_t es) {
  return (reinterpret_cast<uintptr_t>(z) | (rows > 1 ? stride * es : 0)) % 16 == 0;
}

constexpr uint32_t kCus = 256;

// Lanes of a workgroup of row_stats.  (Forward pass, us.  Waves alone where a row feeds no more: 65536 rows of 2048 16-bit columns 52,
// by 256 lanes 212.  A workgroup a compute unit, 1024 lanes and 512: 24 of 32768 5.7 and 6.4, 256 of 131072 14.3 and 18.2; 256 lanes
// 28.0.  Many rows, 256 and 512: 16384 of 50001 248 and 254, 1001 of 32003 14.0 and 15.7, but 4096 of 131072 163 and 160,
// 8192 of 32768 fp32 161 and 155; 1024 lanes 14 to 340% more.)
inline uint32_t stat_lanes(size_t parts, size_t packs_of_part) {
  if (packs_of_part <= 256) return 64;
  if (parts <= kCus) return packs_of_part <= 2048 ? 256 : 1024;
  return packs_of_part < 8192 ? 256 : 512;
}

// Rows in registers: lanes and packs a lane.  Up to a row for each compute unit as many waves as a row feeds (24 rows of 32768 bf16 7.9 us,
// by as few as hold it 10.2; 100 9.3 and 11.5); else as few as hold it, so that several rows are on their way at once (8192 of 16384 bf16 102 us, by as
// many as it feeds 121; 65536 of 2048 101 and 154).
struct Held {
  uint32_t waves;
  int K;
};
constexpr int kHeldMost = 16;
Held held_row(size_t rows, size_t cols, int V, bool on_grid) {
  const size_t packs = (cols + (on_grid ? V - 1 : 2 * V - 2)) / V, whole = cols / V;  // packs of any row; those that no row's end cuts
  if (whole == 0) return {0, 0};
  const auto shape = [&](uint32_t waves) {
    const int need = static_cast<int>((packs + 64 * waves - 1) / (64 * waves)), K = need <= 2 ? need : (need + 1) / 2 * 2;
    const bool fits = K <= kHeldMost && (K <= 2 || static_cast<size_t>(K - 2) * 64 * waves <= whole);  // only the last two strips pass an end
    return fits ? Held{waves, K} : Held{0, 0};
  };
  if (rows <= kCus) {  // a compute unit each: as many waves as a row feeds
    const size_t wide = (packs + 63) / 64;
    for (uint32_t waves = wide < kMostWaves ? static_cast<uint32_t>(wide) : kMostWaves; waves >= 1; --waves)
      if (const Held h = shape(waves); h.K) return h;
  } else {
    for (uint32_t waves = 1; waves <= kMostWaves; ++waves)
      if (const Held h = shape(waves); h.K) return h;
  }
  return {0, 0};
}

template <class T, int K>
void held(const LogitArgs& a, uint32_t waves, uint32_t groups, hipStream_t st) {
  hipLaunchKernelGGL((policy_held<T, K>), dim3(groups), dim3(waves * 64), 0, st, a);
}
template <class T>
void launch_held(const LogitArgs& a, uint32_t groups, hipStream_t st) {
  const Held h = held_row(a.rows, a.cols, 16 / T::kSize, rows_on_grid(a.z, a.rows, a.stride, T::kSize));
  switch (h.K) {
    case 1: held<T, 1>(a, h.waves, groups, st); break;
    case 2: held<T, 2>(a, h.waves, groups, st); break;
    case 4: held<T, 4>(a, h.waves, groups, st); break;
    case 6: held<T, 6>(a, h.waves, groups, st); break;
    case 8: held<T, 8>(a, h.waves, groups, st); break;
    case 10: held<T, 10>(a, h.waves, groups, st); break;
    case 12: held<T, 12>(a, h.waves, groups, st); break;
    case 14: held<T, 14>(a, h.waves, groups, st); break;
    default: held<T, 16>(a, h.waves, groups, st); break;
  }
}

template <class T, bool Policy>
void stats(const LogitArgs& a, uint32_t groups, hipStream_t st) {
  const size_t packs = a.packs;
  hipLaunchKernelGGL((row_stats<T, Policy>), dim3(groups), dim3(stat_lanes(a.rows * a.splits, (packs + a.splits - 1) / a.splits)), 0, st, a);
}
template <class T>
void grad(const LogitArgs& a, hipStream_t st) {
  const size_t run = size_t{64} * kGradPacks, items = a.rows * ((a.packs + run - 1) / run);
  hipLaunchKernelGGL((logit_grad<T>), dim3(grid_of((items + 3) / 4)), dim3(256), 0, st, a);
}

// Packs that cover every row: one more where rows start off the grid.
uint32_t packs_of(const LogitArgs& a, mr_dtype dt) {
  const size_t es = elem_size(dt), V = 16 / es;
  return static_cast<uint32_t>((a.cols + (rows_on_grid(a.z, a.rows, a.stride, es) ? V - 1 : 2 * V - 2)) / V);
}

template <class F>
void by_type(mr_dtype dt, F f) {
  if (dt == MR_BF16)
    f(EBf16{});
  else if (dt == MR_FP16)
    f(EFp16{});
  else
    f(EFp32{});
}

}  // namespace

LogitPlan plan_logits(const char* z, size_t rows, size_t cols, size_t stride, mr_dtype dt, bool gradient) {
  const int V = 16 / elem_size(dt);
  const size_t packs = (cols + V - 1) / V;
  LogitPlan pl{};
  const Held h = held_row(rows, cols, V, rows_on_grid(z, rows, stride, elem_size(dt)));
  // A few rows of many packs a lane take longer in one launch than in two of all compute units (us, one and two): 8 rows of 131072
  // 16-bit columns 17.2 and 14.0, 48 17.9 and 18.1; 8 of 100000 15.2 and 14.1, 32 16.0 and 16.5; one of 65536 10.5 and 11.5; 24 of 32768
  // 7.9 and 14.4.
  if (gradient && rows && h.K && (rows >= kCus / 8 || h.K <= 12)) {
    pl.held = 1;
    pl.splits = 1;
    const size_t per_cu = (h.K <= 4 ? 24 : 16) / h.waves;  // waves that a compute unit's registers hold
    const size_t most = kCus * (per_cu > 16 ? 16 : per_cu), rounds = (rows + most - 1) / most;
    pl.groups = static_cast<uint32_t>((rows + rounds - 1) / rounds);
    return pl;
  }
  // A few long rows: each over several workgroups, one on every compute unit.  (Forward pass, us, in parts and whole: 1 row of
  // 131072 16-bit columns 6.0 and 10.5, 63 8.2 and 12.3, 2 of 262144 6.0 and 19.4, 8 of 32768 5.8 and 5.4.  Up to 1024 parts, whose
  // arrivals wait for one another: 16 of 131072 16.4 against 8.1.  Whole rows leave compute units idle below 256 of them: 64 take 11.8,
  // 128 12.7; two to four parts for those were not measured.)
  size_t splits = 1;
  if (rows && rows < kCus / 4 && packs > 4096) {
    splits = kCus / rows;
    splits = splits > 64 ? 64 : splits;
  }
  pl.splits = static_cast<uint32_t>(splits);
  const size_t parts = rows * splits, most = size_t{kCus} * 16;
  pl.groups = static_cast<uint32_t>(parts < 1 ? 1 : parts < most ? parts : most);
  return pl;
}

hipError_t launch_logprob(const LogitArgs& args, mr_dtype dt, hipStream_t st) {
  LogitArgs a = args;
  a.packs = packs_of(a, dt);
  // rows of one wave: as many as the device holds, each walking its rows (a launch starts about one workgroup a nanosecond)
  const size_t parts = a.rows * a.splits, most = (a.packs + a.splits - 1) / a.splits <= 256 ? size_t{kCus} * 24 : parts;
  by_type(dt, [&](auto t) { stats<decltype(t), false>(a, grid_of(parts < most ? parts : most), st); });
  return hipGetLastError();
}

hipError_t launch_logprob_bwd(const LogitArgs& args, mr_dtype dt, hipStream_t st) {
  LogitArgs a = args;
  a.packs = packs_of(a, dt);
  by_type(dt, [&](auto t) { grad<decltype(t)>(a, st); });
  return hipGetLastError();
}

hipError_t launch_policy(const LogitArgs& args, const LogitPlan& pl, mr_dtype dt, hipStream_t st) {
  LogitArgs a = args;
  a.packs = packs_of(a, dt);
  if (pl.held) {
    by_type(dt, [&](auto t) { launch_held<decltype(t)>(a, pl.groups, st); });
    return hipGetLastError();
  }
  by_type(dt, [&](auto t) { stats<decltype(t), true>(a, pl.groups, st); });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.dz) return e;
  by_type(dt, [&](auto t) { grad<decltype(t)>(a, st); });
  return hipGetLastError();
}

uint32_t preference_groups(size_t pairs) { return static_cast<uint32_t>(pairs < 1 ? 1 : pairs < 4 * kCus ? pairs : 4 * kCus); }

hipError_t launch_preference(const PreferenceArgs& a, hipStream_t st) {
  const uint32_t groups = preference_groups(a.pairs);
  const uint32_t lanes = 256;  // (4.4M tokens of 1024 pairs: 21.3 us; 512 lanes 23.2)
  hipLaunchKernelGGL(preference, dim3(groups), dim3(lanes), 0, st, a);
  return hipGetLastError();
}

}  // namespace mr
