// The norm of a list of gradients with its clip factor, and the AdamW step over a list of tensors, for gfx950.
//
// Both walk the tensors of one launch as one list of tiles: the kernel arguments hold the tensors' pointers
// and a prefix of their tile counts, and a workgroup finds its tile's tensor with a scalar binary search.
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

#include "mr_train.h"
#include "packs.h"

namespace mr {
namespace {

constexpr int kLanes = 256;

// The tensor whose tiles hold tile t: tile_prefix[s] <= t < tile_prefix[s + 1].
__device__ __forceinline__ uint32_t tensor_of(const uint32_t* tile_prefix, uint32_t P, uint32_t t) {
  uint32_t lo = 0, hi = P;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) >> 1;
    if (tile_prefix[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// --------------------------------------------------------------------------------------- gradient norm

// Sum of x over the workgroup, in every lane.
__device__ __forceinline__ double group_sum(double x) {
  __shared__ double lds[kLanes / 64];
  x = wave_sum(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0.0;
#pragma unroll
  for (int i = 0; i < kLanes / 64; ++i) x += lds[i];
  return x;
}

// Squares are added in fp64: fp32's rate on this part's vector units, and a sum of fp32 squares that no finite
// gradient overflows, so the sum is finite exactly where every gradient is.  The workgroup that arrives last
// adds the workgroups' sums in their order: the result does not depend on which one that is.
template <class T>
__global__ __launch_bounds__(kLanes) void grad_norm(GradNormArgs a) {
  constexpr int kN = 16 / T::kSize;  // elements per 16-byte pack
  constexpr int kU = kNormTile / (kLanes * kN);
  double s = 0.0;
  for (uint32_t t = blockIdx.x; t < a.tile_prefix[a.P]; t += gridDim.x) {
    const uint32_t i = tensor_of(a.tile_prefix, a.P, t);
    const uint64_t e0 = static_cast<uint64_t>(t - a.tile_prefix[i]) * kNormTile;
    const uint64_t left = a.n[i] - e0;
    const char* p = a.g[i] + e0 * T::kSize;
    Raw<T, kN> r[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t e = (u * kLanes + threadIdx.x) * kN;
      const int cnt = e >= left ? 0 : left - e < kN ? static_cast<int>(left - e) : kN;
      r[u] = load_part<T, kN, true>(p + e * T::kSize, cnt);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float f[kN];
      widen(r[u], f);
#pragma unroll
      for (int j = 0; j < kN; ++j) s = __builtin_fma(static_cast<double>(f[j]), static_cast<double>(f[j]), s);
    }
  }
  s = group_sum(s);
  const uint32_t mine = a.part_base + blockIdx.x;
  __shared__ uint32_t last;
  if (threadIdx.x == 0) {
    __hip_atomic_store(a.part + mine, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = 0;
    if (a.finish)
      last = __hip_atomic_fetch_add(a.arrived, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  s = 0.0;
  for (uint32_t i = threadIdx.x; i < a.part_base + gridDim.x; i += kLanes)
    s += __hip_atomic_load(a.part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  s = group_sum(s);
  if (threadIdx.x == 0) {
    __hip_atomic_store(a.arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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

// Scale byte of a block whose largest magnitude has the fp32 bits `top`: the smallest power of two that brings
// it to 448, E4M3's largest, or less; 255 if it is infinite or NaN (as an integer NaN is the largest of all).
__device__ __forceinline__ uint32_t mx_byte(uint32_t top) {
  const int b = static_cast<int>((top + 0x1fffffu) >> 23) - 8;  // mantissas above 1.75 carry into the exponent
  return top >= 0x7f800000u ? 255u : static_cast<uint32_t>(b < 0 ? 0 : b);
}

// Largest of the four lanes of a quad, in each of them.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  const uint32_t y = __builtin_amdgcn_mov_dpp(static_cast<int>(x), 0xB1, 0xf, 0xf, true);  // lanes 1 0 3 2
  x = x > y ? x : y;
  const uint32_t z = __builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x4E, 0xf, 0xf, true);  // lanes 2 3 0 1
  return x > z ? x : z;
}

// |y| (0 .. 448) on the E4M3 grid, up with probability (distance to the lower neighbour) / (spacing): r16 / 2^16
// of a spacing is added and the bits below the third mantissa bit are dropped.  Below 2^-6, the smallest normal
// number, the spacing stays 2^-9: adding 2^-6 first puts it there.
__device__ __forceinline__ float round_e4m3(float y, uint32_t r16) {
  const float small = y < 0.015625f ? 0.015625f : 0.0f;
  const uint32_t b = (__float_as_uint(y + small) + (r16 << 4)) & 0xfff00000u;
  return __uint_as_float(b) - small;
}

__device__ __forceinline__ uint32_t e4m3x2(float a, float b, uint32_t old, bool high) {
  return high ? __builtin_amdgcn_cvt_pk_fp8_f32(a, b, static_cast<int>(old), true)
              : __builtin_amdgcn_cvt_pk_fp8_f32(a, b, static_cast<int>(old), false);
}

// 32 random bits of element idx of the flat state: a Weyl step on the key of (seed, step) and one
// multiply-xorshift round.
__device__ __forceinline__ uint32_t random_bits(uint32_t key, uint64_t idx) {
  uint32_t x = key + static_cast<uint32_t>(idx) * 0x9E3779B1u + static_cast<uint32_t>(idx >> 32) * 0x85EBCA77u;
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  return x ^ (x >> 15);
}

// Eight codes at c (8 bytes, aligned) times the block's scale.
__device__ __forceinline__ void mx_load(const char* c, uint32_t byte, float (&f)[8]) {
  const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(c));
  const float s = mx_scale(byte);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), true);
    f[4 * i] = lo[0] * s;
    f[4 * i + 1] = lo[1] * s;
    f[4 * i + 2] = hi[0] * s;
    f[4 * i + 3] = hi[1] * s;
  }
}

// This lane's eight of the block's 32 values (four neighbouring lanes hold a block) as codes; the block's byte.
template <bool Floor, int Shift>
__device__ __forceinline__ u32x2 mx_encode(const float (&f)[8], const uint32_t (&r)[8], uint32_t* byte) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(f[i]) & 0x7fffffffu;
    top = top > b ? top : b;
  }
  const uint32_t e = mx_byte(quad_max(top));
  *byte = e;
  const float inv = __uint_as_float((254u - (e < 253u ? e : 253u)) << 23);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = __builtin_fabsf(f[i]) * inv;
    q[i] = round_e4m3(y, (r[i] >> Shift) & 0xffffu);
    if (Floor) q[i] = y > 0.0f && q[i] == 0.0f ? 0.001953125f : q[i];
    q[i] = e == 255u ? 0.0f : __builtin_copysignf(q[i], f[i]);
  }
  u32x2 w = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = e4m3x2(q[4 * i], q[4 * i + 1], 0, false);
    w[i] = e4m3x2(q[4 * i + 2], q[4 * i + 3], w[i], true);
  }
  return w;
}

// ------------------------------------------------------------------------------------------------- AdamW

// Elements a lane takes at once: 8 where the moments are bytes (8 codes are 8 bytes, four lanes a block), 4
// where they are fp32 (one 16-byte access each).
template <bool Mx>
constexpr int kLaneElems = Mx ? 8 : 4;
template <bool Mx>
constexpr uint32_t kTileElems = kLanes * kLaneElems<Mx>;

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
    if (a.out.m != a.in.m) *reinterpret_cast<u32x2*>(a.out.m + idx) = *reinterpret_cast<const u32x2*>(a.in.m + idx);
    if (a.out.v != a.in.v) *reinterpret_cast<u32x2*>(a.out.v + idx) = *reinterpret_cast<const u32x2*>(a.in.v + idx);
    if (a.out.ms != a.in.ms) a.out.ms[blk] = a.in.ms[blk];
    if (a.out.vs != a.in.vs) a.out.vs[blk] = a.in.vs[blk];
  } else {
    if (a.out.m != a.in.m) store_raw<EFp32, E, true>(a.out.m + 4 * idx, load_raw<EFp32, E, true>(a.in.m + 4 * idx));
    if (a.out.v != a.in.v) store_raw<EFp32, E, true>(a.out.v + 4 * idx, load_raw<EFp32, E, true>(a.in.v + 4 * idx));
  }
}

// One tile per workgroup.  Every byte is touched once; loads and stores are non-temporal.
template <class T, class G, bool Mx, bool Master>
__global__ __launch_bounds__(kLanes) void adamw(AdamArgs a) {
  constexpr int E = kLaneElems<Mx>;
  const uint32_t i = tensor_of(a.tile_prefix, a.P, blockIdx.x);
  const uint64_t e = static_cast<uint64_t>(blockIdx.x - a.tile_prefix[i]) * kTileElems<Mx> + threadIdx.x * E;
  const uint64_t n = a.n[i];
  const int cnt = e >= n ? 0 : n - e < E ? static_cast<int>(n - e) : E;
  const bool live = e < ((n + (kMxBlock - 1)) & ~uint64_t{kMxBlock - 1});  // in a block of the tensor's state
  const uint64_t idx = static_cast<uint64_t>(a.block0[i]) * kMxBlock + e;
  float factor = 1.0f;
  if (a.clip) {
    factor = a.clip[1];
    if (a.clip[2] == 0.0f) {
      keep_tile<T, Mx, Master, E>(a, i, e, idx, cnt, live);
      return;
    }
  }
  float p[E], g[E], m[E], v[E], r[E];
#pragma unroll
  for (int j = 0; j < E; ++j) p[j] = m[j] = v[j] = 0.0f;
  if (live) {
    if constexpr (Master)
      widen(load_raw<EFp32, E, true>(reinterpret_cast<const char*>(a.in.master + idx)), p);
    else
      widen(load_part<T, E, true>(a.p[i] + e * T::kSize, cnt), p);
    if constexpr (Mx) {
      mx_load(a.in.m + idx, a.in.ms[idx / kMxBlock], m);
      mx_load(a.in.v + idx, a.in.vs[idx / kMxBlock], v);
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] *= v[j];
    } else {
      widen(load_raw<EFp32, E, true>(a.in.m + 4 * idx), m);
      widen(load_raw<EFp32, E, true>(a.in.v + 4 * idx), v);
    }
  }
  widen(load_part<G, E, true>(a.g[i] + e * G::kSize, cnt), g);
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const float gj = g[j] * factor;
    m[j] = j < cnt ? m[j] * a.b1 + gj * a.c1 : 0.0f;
    v[j] = j < cnt ? v[j] * a.b2 + gj * gj * a.c2 : 0.0f;
    r[j] = __builtin_sqrtf(v[j]);
    const float u = m[j] / __builtin_fmaf(r[j], a.inv_sqrt_bc2, a.eps);
    p[j] = j < cnt ? p[j] * a.keep - u * a.lr_t : 0.0f;
  }
  if (cnt) store_part<T, E, true>(a.po[i] + e * T::kSize, p, cnt);
  if constexpr (Mx) {  // all lanes: the block's scale is the largest of four lanes' values
    uint32_t bits[E], mb, vb;
#pragma unroll
    for (int j = 0; j < E; ++j) bits[j] = random_bits(a.key, idx + j);
    const u32x2 mw = mx_encode<false, 0>(m, bits, &mb);
    const u32x2 vw = mx_encode<true, 16>(r, bits, &vb);
    if (live) {
      __builtin_nontemporal_store(mw, reinterpret_cast<u32x2*>(a.out.m + idx));
      __builtin_nontemporal_store(vw, reinterpret_cast<u32x2*>(a.out.v + idx));
      if ((threadIdx.x & 3) == 0) {
        a.out.ms[idx / kMxBlock] = static_cast<uint8_t>(mb);
        a.out.vs[idx / kMxBlock] = static_cast<uint8_t>(vb);
      }
    }
  } else if (live) {
    store_raw<EFp32, E, true>(a.out.m + 4 * idx, narrow<EFp32>(m));
    store_raw<EFp32, E, true>(a.out.v + 4 * idx, narrow<EFp32>(v));
  }
  if constexpr (Master)
    if (live) store_raw<EFp32, E, true>(reinterpret_cast<char*>(a.out.master + idx), narrow<EFp32>(p));
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
  const dim3 grid(grad_norm_groups(a.tile_prefix[a.P])), block(kLanes);
  if (dt == MR_FP32)
    hipLaunchKernelGGL((grad_norm<EFp32>), grid, block, 0, st, a);
  else if (dt == MR_BF16)
    hipLaunchKernelGGL((grad_norm<EBf16>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((grad_norm<EFp16>), grid, block, 0, st, a);
  return hipGetLastError();
}

uint32_t adam_tile_elems(mr_dtype, mr_dtype, mr_state_format fmt, bool) {
  return fmt == MR_STATE_MXFP8 ? kTileElems<true> : kTileElems<false>;
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
