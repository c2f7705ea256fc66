// The norm of a list of gradients with its clip factor, and the AdamW step over a list of tensors, for gfx950.
//
// Both walk the tensors of one launch as one list of tiles: the kernel arguments hold the tensors' pointers
// and a prefix of their tile counts, and a workgroup finds its tile's tensor by comparing its number with the whole prefix.
//
//   norm    N = scale * sqrt(sum of all g^2), factor = scale * min(1, max_norm / (N + 1e-6))
//   AdamW   g' = factor * g,  m' = b1*m + (1-b1)*g',  v' = b2*v + (1-b2)*g'^2,
//           p' = (1 - lr*wd)*p - lr/(1-b1^t) * m' / (sqrt(v') / sqrt(1-b2^t) + eps)
//
// Moments in 8 bits: blocks of 32 elements of the flat state share a power-of-two scale and each element is
// an E4M3 number times it (the OCP microscaling format MXFP8, an element and a shared-scale byte each).  The
// first moment is stored as it is, the second as its square root, which halves the exponents it spans.  Both
// are rounded stochastically: with b2 = 0.999 a step changes v by 0.1%, far below E4M3's spacing, so rounding to
// nearest would never move it, while a rounding up with probability (distance to the lower neighbour) /
// (spacing) keeps the average.  A second moment that is not zero is never stored as zero, so that no later
// step divides by eps alone.
//
// The norm and the 32-bit step are bound by the bytes they move: 537M bf16 gradients 155 us (6.9 TB/s, reads only), 134M
// fp32 elements 617 to 654 us (5.7 to 6.1 TB/s over 4 read and 3 written streams, by where the buffers lie).  The 8-bit
// step is near both bounds: 42 vector operations an element at 10.1 bytes, 28M bf16 elements 49.9 us (5.7 TB/s), 130M
// 205 to 209 us (6.3 to 6.4 TB/s).

#include <type_traits>

#include "mr_train.h"
#include "packs.h"

namespace mr {
namespace {

// The tensor whose tiles hold tile t: tile_prefix[s] <= t < tile_prefix[s + 1].  Every lane holds entries of the table
// and compares them at once: a search would wait for a load of the launch's arguments at each of its steps.
template <int N>
struct TensorTable {
  static constexpr int kWords = (N + 63) / 64;
  uint32_t first[kWords];
  __device__ TensorTable(const uint32_t* tile_prefix, uint32_t P) {
    const uint32_t lane = threadIdx.x & 63;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const uint32_t i = w * 64 + lane;
      first[w] = i < P ? tile_prefix[i] : 0xffffffffu;
    }
  }
  __device__ uint32_t find(uint32_t t) const {
    uint32_t n = 0;
#pragma unroll
    for (int w = 0; w < kWords; ++w) n += __builtin_popcountll(__builtin_amdgcn_ballot_w64(first[w] <= t));
    return n - 1;
  }
};

// --------------------------------------------------------------------------------------- gradient norm

constexpr int kNormLanes = 512;

// Sum of x over the workgroup, in every lane.
__device__ __forceinline__ double group_sum(double x) {
  __shared__ double lds[kNormLanes / 64];
  x = wave_sum(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0.0;
#pragma unroll
  for (int i = 0; i < kNormLanes / 64; ++i) x += lds[i];
  return x;
}

// Squares are added in fp64: fp32's rate on this part's vector units, and a sum of fp32 squares that no finite
// gradient overflows, so the sum is finite exactly where every gradient is.  Workgroups walk the tiles, the next one's
// loads issued before this one's sums.  The workgroup that arrives last adds the workgroups' sums in their order: the
// result does not depend on which one that is.
template <class T>
__global__ __launch_bounds__(kNormLanes) void grad_norm(GradNormArgs a) {
  constexpr int kN = 16 / T::kSize;  // elements per 16-byte pack
  constexpr uint32_t kTile = kNormTileBytes / T::kSize;
  constexpr int kU = kTile / (kNormLanes * kN);
  const TensorTable<kNormTensors> table(a.tile_prefix, a.P);
  const uint32_t tiles = a.tile_prefix[a.P];
  struct Tile {
    Raw<T, kN> r[kU];
  };
  auto fetch = [&](uint32_t t) {
    Tile x;
    const uint32_t i = table.find(t);
    const uint64_t e0 = static_cast<uint64_t>(t - a.tile_prefix[i]) * kTile;
    const uint64_t left = a.n[i] - e0;
    const char* p = a.g[i] + e0 * T::kSize;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t e = (u * kNormLanes + threadIdx.x) * kN;
      if (left >= kTile)
        x.r[u] = load_raw<T, kN, true>(p + e * T::kSize);
      else
        x.r[u] = load_part<T, kN, true>(p + e * T::kSize, e >= left ? 0 : left - e < kN ? static_cast<int>(left - e) : kN);
    }
    return x;
  };
  double s = 0.0;
  uint32_t t = blockIdx.x;
  Tile next;
  if (t < tiles) next = fetch(t);
  for (; t < tiles; t += gridDim.x) {
    const Tile now = next;
    if (t + gridDim.x < tiles) next = fetch(t + gridDim.x);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float f[kN];
      widen(now.r[u], f);
#pragma unroll
      for (int j = 0; j < kN; ++j) s = __builtin_fma(static_cast<double>(f[j]), static_cast<double>(f[j]), s);
    }
  }
  s = group_sum(s);
  // Hand-off without the compiler's agent-scope release and acquire, whose cache write-back costs a workgroup about
  // 40 ns in line with the others: the sum leaves through a device-scope (write-through) store, is acknowledged before the
  // arrival is counted, and the last workgroup reads the sums with device-scope loads after the counts told it to.
  __shared__ bool last;
  if (threadIdx.x == 0) {
    __hip_atomic_store(a.part + a.part_base + blockIdx.x, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    last = false;
    if (a.finish) {
      const uint32_t sets = gridDim.x < 4 * kNormSets ? 1 : kNormSets, set = blockIdx.x % sets;
      const uint32_t members = (gridDim.x - set + sets - 1) / sets;
      last = __hip_atomic_fetch_add(&a.arrived[set][0], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == members - 1;
      if (last && sets > 1)
        last = __hip_atomic_fetch_add(&a.arrived[kNormSets][0], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == sets - 1;
    }
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
  }
  __syncthreads();
  if (!last) return;
  s = 0.0;
  for (uint32_t i = threadIdx.x; i < a.part_base + gridDim.x; i += kNormLanes)
    s += __hip_atomic_load(a.part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  s = group_sum(s);
  if (threadIdx.x <= kNormSets) __hip_atomic_store(&a.arrived[threadIdx.x][0], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (threadIdx.x == 0) {
    const double norm = a.scale * __builtin_sqrt(s);
    const bool finite = norm <= 1.7976931348623157e308;  // false for NaN too
    double f = a.max_norm > 0.0 ? a.max_norm / (norm + 1e-6) : 1.0;
    f = f < 1.0 ? f : 1.0;
    a.out[0] = static_cast<float>(norm);
    a.out[1] = finite ? static_cast<float>(a.scale * f) : 0.0f;
    a.out[2] = finite ? 1.0f : 0.0f;
  }
}

// ------------------------------------------------------------------------------------------- MXFP8 blocks

// 2^(byte - 127): 2^-127 for 0, NaN for 255.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  const uint32_t b = byte == 0 ? 0x00400000u : byte << 23;
  return __uint_as_float(byte == 255 ? 0x7fc00000u : b);
}

// Scale byte of a block whose largest magnitude, times 2^Up, has the fp32 bits `top`: the smallest power of two that
// brings it to 448, E4M3's largest, or less; 255 if it is infinite or NaN (as an integer NaN is the largest of all).
template <int Up>
__device__ __forceinline__ uint32_t mx_byte(uint32_t top) {
  const int b = static_cast<int>((top + 0x1fffffu) >> 23) - 8 - Up;  // mantissas above 1.75 carry into the exponent
  return top >= 0x7f800000u ? 255u : static_cast<uint32_t>(b < 0 ? 0 : b);
}

// Largest of the lanes that hold a block, E elements each, in every one of them.
template <int E>
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
  const auto with = [&](int y) { x = x > static_cast<uint32_t>(y) ? x : static_cast<uint32_t>(y); };
  with(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0xB1, 0xf, 0xf, true));   // quad lanes 1 0 3 2
  with(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x4E, 0xf, 0xf, true));   // quad lanes 2 3 0 1
  if (E == 4) with(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x141, 0xf, 0xf, true));  // half row mirrored
  return x;
}

// 32 random bits for each of the elements idx .. idx + E - 1 of the flat state (idx a multiple of E): a Weyl step on the
// key of (seed, step) and one multiply-xorshift round.  The step is the prime next to 2^32 over the golden ratio (Knuth's
// multiplicative hashing); the round's multiplier and shifts come from Wellons' published search for 32-bit mixers of low
// bias, and the odd multiplier of the index's upper half from Collet's published hash constants.
template <int E>
__device__ __forceinline__ void random_bits(uint32_t key, uint64_t idx, uint32_t (&r)[E]) {
  const uint32_t first = key + static_cast<uint32_t>(idx) * 0x9E3779B1u + static_cast<uint32_t>(idx >> 32) * 0x85EBCA77u;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    uint32_t x = first + static_cast<uint32_t>(j) * 0x9E3779B1u;
    x ^= x >> 16;
    x *= 0x7FEB352Du;
    r[j] = x ^ (x >> 15);
  }
}

// The codes of E neighbouring elements (aligned).
template <int E>
struct Codes {
  uint32_t w[E / 4];
};
template <int E>
__device__ __forceinline__ Codes<E> load_codes(const char* p) {
  Codes<E> c;
  if constexpr (E == 8) {
    const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
    c.w[0] = v[0];
    c.w[1] = v[1];
  } else {
    c.w[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
  }
  return c;
}
template <int E>
__device__ __forceinline__ void store_codes(char* p, const Codes<E>& c) {
  if constexpr (E == 8)
    __builtin_nontemporal_store(u32x2{c.w[0], c.w[1]}, reinterpret_cast<u32x2*>(p));
  else
    __builtin_nontemporal_store(c.w[0], reinterpret_cast<uint32_t*>(p));
}
// The codes' values times s.
template <int E>
__device__ __forceinline__ void mx_decode(const Codes<E>& c, float s, float (&f)[E]) {
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c.w[i]), false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c.w[i]), true);
    f[4 * i] = lo[0] * s;
    f[4 * i + 1] = lo[1] * s;
    f[4 * i + 2] = hi[0] * s;
    f[4 * i + 3] = hi[1] * s;
  }
}

// This lane's E of the block's 32 values (neighbouring lanes hold a block) as codes; the block's byte.
// v_cvt_sr_fp8_f32 adds the random word's upper 20 bits below the third mantissa bit (below 2^-6, the smallest
// normal number, below the 2^-9 place) and drops what lies there: up with probability (distance to the lower
// neighbour) / (spacing).  It takes 16 of them here, from the lower half of r, or for `Second` from the upper half.  Second
// moments are raised to the smallest code, 2^-9, unless they are zero.
// f holds the values times 2^Up.
template <bool Second, int Up, int E>
__device__ __forceinline__ Codes<E> mx_encode(const float (&f)[E], const uint32_t (&r)[E], uint32_t* byte) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const uint32_t b = Second ? __float_as_uint(f[i]) : __float_as_uint(f[i]) & 0x7fffffffu;  // roots have no sign
    top = top > b ? top : b;
  }
  const uint32_t e = mx_byte<Up>(block_max<E>(top));
  *byte = e;
  const float inv = __uint_as_float((254u - Up - (e < 253u - Up ? e : 253u - Up)) << 23);
  Codes<E> c;
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    int x = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float y = f[4 * i + j] * inv;
      if (Second) y = __builtin_amdgcn_fmed3f(y, 0.001953125f, y * 1.2676506002282294e30f);  // 2^-9; y * 2^100
      const uint32_t bits = Second ? r[4 * i + j] & 0xffff0000u : r[4 * i + j] << 16;
      x = j == 0   ? __builtin_amdgcn_cvt_sr_fp8_f32(y, bits, x, 0)
          : j == 1 ? __builtin_amdgcn_cvt_sr_fp8_f32(y, bits, x, 1)
          : j == 2 ? __builtin_amdgcn_cvt_sr_fp8_f32(y, bits, x, 2)
                   : __builtin_amdgcn_cvt_sr_fp8_f32(y, bits, x, 3);
    }
    c.w[i] = e == 255u ? 0u : static_cast<uint32_t>(x);
  }
  return c;
}

// ------------------------------------------------------------------------------------------------- AdamW

constexpr int kLanes = 256;

// sqrt and quotient from the hardware's square root and reciprocal, each within 1 ulp: the correctly rounded ones take three
// times the operations, and the 8-bit step is bound by its operations.  The 32-bit step, bound by its bytes, takes the same
// ones; its error against 64 bits is no larger for it (4.5e-8 of the result over 134M elements, as with the correctly rounded
// ones).  Both flush subnormal arguments, so squares below 2^-100 are taken at a larger scale.
//
// The 8-bit step never holds v itself.  It carries the root times 2^kAdamUp all through, the divisor and lr with it: v is finite
// for gradients below 2^47, and the divisor is normal for every root that the format holds.  The 32-bit step's divisor is the
// root of an fp32 number or at least eps, which is 0 or normal.
constexpr uint32_t kSmallSquare = 0x0d800000u;  // 2^-100
__device__ __forceinline__ float root(float v) {
  const bool small = v < 7.8886090522101181e-31f;  // 2^-100
  const float r = __builtin_amdgcn_sqrtf(v * (small ? 18446744073709551616.0f : 1.0f));
  return r * (small ? 2.3283064365386963e-10f : 1.0f);
}
// sqrt(x^2 + y^2), where the squares may leave fp32's range below.
__device__ __forceinline__ float small_hypot(float x, float y) {
  const bool small = __float_as_uint(__builtin_fmaf(y, y, x * x)) < kSmallSquare;
  const float up = small ? 1.2676506002282294e30f : 1.0f;  // 2^100
  x *= up;
  y *= up;
  return __builtin_amdgcn_sqrtf(__builtin_fmaf(y, y, x * x)) * (small ? 7.8886090522101181e-31f : 1.0f);
}

// Elements a lane takes at once: 4 where some stream is fp32 (one 16-byte access each), 8 where the moments are bytes and
// the rest 16-bit.
template <class T, class G, bool Mx, bool Master>
constexpr int kLaneElems = Mx && !Master && T::kSize == 2 && G::kSize == 2 ? 8 : 4;

// The step is not taken (clip says that a gradient is not finite): outputs that are not the inputs get copies.
template <class T, bool Mx, bool Master, int E>
__device__ __forceinline__ void keep_tile(const AdamArgs& a, uint32_t i, uint64_t e, uint64_t idx, int cnt, bool live) {
  float f[E];
  if (Master) {
    if (live && a.out.master != a.in.master)
      store_raw<EFp32, E, true>(reinterpret_cast<char*>(a.out.master + idx),
                                load_raw<EFp32, E, true>(reinterpret_cast<const char*>(a.in.master + idx)));
    if (cnt && a.po[i] != a.p[i]) {
      widen(load_raw<EFp32, E, true>(reinterpret_cast<const char*>(a.in.master + idx)), f);
      store_part<T, E, true>(a.po[i] + e * T::kSize, f, cnt);
    }
  } else if (cnt && a.po[i] != a.p[i]) {
    widen(load_part<T, E, true>(a.p[i] + e * T::kSize, cnt), f);
    store_part<T, E, true>(a.po[i] + e * T::kSize, f, cnt);
  }
  if (!live) return;
  if constexpr (Mx) {
    const uint64_t blk = idx / kMxBlock;
    if (a.out.m != a.in.m) store_codes<E>(a.out.m + idx, load_codes<E>(a.in.m + idx));
    if (a.out.v != a.in.v) store_codes<E>(a.out.v + idx, load_codes<E>(a.in.v + idx));
    if (a.out.ms != a.in.ms) a.out.ms[blk] = a.in.ms[blk];
    if (a.out.vs != a.in.vs) a.out.vs[blk] = a.in.vs[blk];
  } else {
    if (a.out.m != a.in.m) store_raw<EFp32, E, true>(a.out.m + 4 * idx, load_raw<EFp32, E, true>(a.in.m + 4 * idx));
    if (a.out.v != a.in.v) store_raw<EFp32, E, true>(a.out.v + 4 * idx, load_raw<EFp32, E, true>(a.in.v + 4 * idx));
  }
}

// The tile of workgroup b of n.  Workgroups are dealt to the eight XCDs in turn; runs of 32 tiles that follow one
// another go to one XCD, so each streams long stretches of every buffer (28M elements, 8-bit moments: 52.5 us in plain
// order, 50.1 in runs of 16 to 128; 130M fp32: 640, 596 to 622; runs of 160 or 250 are 2% slower again).
__device__ __forceinline__ uint32_t tile_of(uint32_t b, uint32_t n) {
  constexpr uint32_t kRun = 32, kDeal = 8 * kRun;
  return b < n / kDeal * kDeal ? b / kDeal * kDeal + b % 8 * kRun + b % kDeal / 8 : b;
}

// One tile per workgroup, a pack of E elements a lane, all of its loads first; a whole tile runs without a lane's checks.
// Every byte is touched once, and loads and stores are non-temporal.  (Two or four packs a lane, 256 lanes apart: 28M
// elements with 8-bit moments 49.3 -> 53.7 us, 134M fp32 634 -> 633 and 685.)
template <class T, class G, bool Mx, bool Master>
__global__ __launch_bounds__(kLanes) void adamw(AdamArgs a) {
  constexpr int E = kLaneElems<T, G, Mx, Master>;
  constexpr uint32_t kTile = kLanes * E;
  using P = std::conditional_t<Master, EFp32, T>;  // what p is read as
  const uint32_t tile = tile_of(blockIdx.x, gridDim.x);
  const uint32_t i = TensorTable<kAdamTensors>(a.tile_prefix, a.P).find(tile);
  const uint64_t start = static_cast<uint64_t>(tile - a.tile_prefix[i]) * kTile;
  const uint64_t n = a.n[i];
  const uint64_t first = static_cast<uint64_t>(a.block0[i]) * kMxBlock;  // of the tensor in the flat state
  const uint64_t state_end = (n + (kMxBlock - 1)) & ~uint64_t{kMxBlock - 1};
  const uint64_t e = start + threadIdx.x * E, idx = first + e;  // this lane's pack
  const int cnt = e >= n ? 0 : n - e < E ? static_cast<int>(n - e) : E;
  const bool live = e < state_end;
  float factor = 1.0f;
  if (a.clip) {
    factor = a.clip[1];
    if (a.clip[2] == 0.0f) {
      keep_tile<T, Mx, Master, E>(a, i, e, idx, cnt, live);
      return;
    }
  }
  const char* const pin = Master ? reinterpret_cast<const char*>(a.in.master + first) : a.p[i];
  struct In {
    Raw<P, E> p;
    Raw<G, E> g;
    Raw<EFp32, E> m, v;
    Codes<E> mc, vc;
    uint8_t ms, vs;
  };
  auto run = [&](auto full) {
    constexpr bool kFull = decltype(full)::value;
    In x = {};
    if (kFull || live) {
      if (kFull || Master)
        x.p = load_raw<P, E, true>(pin + e * P::kSize);
      else
        x.p = load_part<P, E, true>(pin + e * P::kSize, cnt);
      if constexpr (Mx) {
        x.mc = load_codes<E>(a.in.m + idx);
        x.vc = load_codes<E>(a.in.v + idx);
        x.ms = a.in.ms[idx / kMxBlock];
        x.vs = a.in.vs[idx / kMxBlock];
      } else {
        x.m = load_raw<EFp32, E, true>(a.in.m + 4 * idx);
        x.v = load_raw<EFp32, E, true>(a.in.v + 4 * idx);
      }
    }
    if (kFull)
      x.g = load_raw<G, E, true>(a.g[i] + e * G::kSize);
    else
      x.g = load_part<G, E, true>(a.g[i] + e * G::kSize, cnt);
    float p[E], g[E], m[E], v[E];
    widen(x.p, p);
    widen(x.g, g);
    if constexpr (Mx) {
      // The decays ride on the blocks' scales: m holds b1*m, v holds sqrt(b2) times the stored root times 2^kAdamUp.
      mx_decode(x.mc, mx_scale(x.ms) * a.b1, m);
      mx_decode(x.vc, mx_scale(x.vs) * a.root_b2, v);
      const float gm = factor * a.c1, gv = factor * a.root_c2;
      float y[E];
      uint32_t least = 0xffffffffu;  // of the squares' bits: they have no sign
#pragma unroll
      for (int j = 0; j < E; ++j) {
        m[j] = __builtin_fmaf(g[j], gm, m[j]);
        y[j] = g[j] * gv;
        const uint32_t b = __float_as_uint(__builtin_fmaf(y[j], y[j], v[j] * v[j]));
        least = b < least ? b : least;
      }
      if (__builtin_amdgcn_ballot_w64(least < kSmallSquare) == 0) {
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] = __builtin_amdgcn_sqrtf(__builtin_fmaf(y[j], y[j], v[j] * v[j]));
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] = small_hypot(v[j], y[j]);
      }
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float u = m[j] * __builtin_amdgcn_rcpf(__builtin_fmaf(v[j], a.inv_sqrt_bc2, a.eps));
        p[j] = __builtin_fmaf(-u, a.lr_t, p[j] * a.keep);
      }
    } else {
      widen(x.m, m);
      widen(x.v, v);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float gj = g[j] * factor;
        m[j] = m[j] * a.b1 + gj * a.c1;
        v[j] = v[j] * a.b2 + gj * gj * a.c2;
        const float u = m[j] * __builtin_amdgcn_rcpf(__builtin_fmaf(root(v[j]), a.inv_sqrt_bc2, a.eps));
        p[j] = p[j] * a.keep - u * a.lr_t;
      }
    }
    if (!kFull && cnt < E) {  // elements between tensors are kept at zero
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (j >= cnt) p[j] = m[j] = v[j] = 0.0f;
    }
    if constexpr (Master) {
      // the parameter is the master copy as it is stored, rounded: keeps the last operation and the conversion to
      // fp16 from becoming one mixed-precision instruction, which rounds once
#pragma unroll
      for (int j = 0; j < E; ++j) asm("" : "+v"(p[j]));
    }
    if (kFull)
      store_raw<T, E, true>(a.po[i] + e * T::kSize, narrow<T, E>(p));
    else if (cnt)
      store_part<T, E, true>(a.po[i] + e * T::kSize, p, cnt);
    if constexpr (Mx) {  // all lanes: the block's scale is the largest of neighbouring lanes' values
      uint32_t bits[E], mb, vb;
      random_bits(a.key, idx, bits);
      const Codes<E> mw = mx_encode<false, 0>(m, bits, &mb);
      const Codes<E> vw = mx_encode<true, kAdamUp>(v, bits, &vb);
      if (kFull || live) {
        store_codes<E>(a.out.m + idx, mw);
        store_codes<E>(a.out.v + idx, vw);
        if (threadIdx.x % (kMxBlock / E) == 0) {
          a.out.ms[idx / kMxBlock] = static_cast<uint8_t>(mb);
          a.out.vs[idx / kMxBlock] = static_cast<uint8_t>(vb);
        }
      }
    } else if (kFull || live) {
      store_raw<EFp32, E, true>(a.out.m + 4 * idx, narrow<EFp32>(m));
      store_raw<EFp32, E, true>(a.out.v + 4 * idx, narrow<EFp32>(v));
    }
    if constexpr (Master)
      if (kFull || live) store_raw<EFp32, E, true>(reinterpret_cast<char*>(a.out.master + idx), narrow<EFp32>(p));
  };
  if (n - start >= kTile)
    run(std::true_type());
  else
    run(std::false_type());
}

template <class T, class G, bool Mx>
void adam_master(const AdamArgs& a, bool master, hipStream_t st) {
  const dim3 grid(a.tile_prefix[a.P]), block(kLanes);
  if constexpr (T::kSize == 2) {
    if (master) {
      hipLaunchKernelGGL((adamw<T, G, Mx, true>), grid, block, 0, st, a);
      return;
    }
  }
  hipLaunchKernelGGL((adamw<T, G, Mx, false>), grid, block, 0, st, a);
}
template <class T, class G>
void adam_format(const AdamArgs& a, mr_state_format fmt, hipStream_t st) {
  if (fmt == MR_STATE_MXFP8)
    adam_master<T, G, true>(a, a.in.master != nullptr, st);
  else
    adam_master<T, G, false>(a, a.in.master != nullptr, st);
}

}  // namespace

hipError_t launch_grad_norm(const GradNormArgs& a, mr_dtype dt, hipStream_t st) {
  const dim3 grid(grad_norm_groups(a.tile_prefix[a.P])), block(kNormLanes);
  if (dt == MR_FP32)
    hipLaunchKernelGGL((grad_norm<EFp32>), grid, block, 0, st, a);
  else if (dt == MR_BF16)
    hipLaunchKernelGGL((grad_norm<EBf16>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((grad_norm<EFp16>), grid, block, 0, st, a);
  return hipGetLastError();
}

uint32_t adam_tile_elems(mr_dtype dt, mr_dtype gdt, mr_state_format fmt, bool master) {
  return kLanes * (fmt == MR_STATE_MXFP8 && !master && dt != MR_FP32 && gdt != MR_FP32 ? kLaneElems<EBf16, EBf16, true, false>
                                                                                       : kLaneElems<EFp32, EFp32, false, false>);
}

hipError_t launch_adam(const AdamArgs& a, mr_dtype dt, mr_dtype gdt, mr_state_format fmt, hipStream_t st) {
  if (dt == MR_FP32)
    adam_format<EFp32, EFp32>(a, fmt, st);
  else if (dt == MR_BF16 && gdt == MR_FP32)
    adam_format<EBf16, EFp32>(a, fmt, st);
  else if (dt == MR_BF16)
    adam_format<EBf16, EBf16>(a, fmt, st);
  else if (gdt == MR_FP32)
    adam_format<EFp16, EFp32>(a, fmt, st);
  else
    adam_format<EFp16, EFp16>(a, fmt, st);
  return hipGetLastError();
}

}  // namespace mr
