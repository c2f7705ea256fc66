// Packs of consecutive elements between memory and fp32 registers, and wave64 reductions, for the
// training-step kernels (norm_fwd.hip, norm_bwd.hip, optim_kernels.hip).
//
// Rows and tensors of odd sizes start anywhere on the element grid, so a pack may start off its own
// 16-byte grid.  Global memory on gfx950 takes multi-dword accesses at any byte address (the compiler's
// unaligned access mode for this target); a type of reduced alignment tells the compiler so, and one
// wide access serves every phase.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mr {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// A dtype's element in memory: widening to fp32 is exact, narrowing rounds to nearest even.  pair() and
// unpair() convert two elements held in one dword (16-bit types).
struct EBf16 {
  static constexpr int kSize = 2;
  __device__ static void unpair(uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
  }
  __device__ static uint32_t pair(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  }
};
struct EFp16 {
  static constexpr int kSize = 2;
  __device__ static void unpair(uint32_t w, float& a, float& b) {
    const f16x2 h = __builtin_bit_cast(f16x2, w);
    a = static_cast<float>(h[0]);
    b = static_cast<float>(h[1]);
  }
  __device__ static uint32_t pair(float a, float b) {
    const f16x2 h = {static_cast<_Float16>(a), static_cast<_Float16>(b)};
    return __builtin_bit_cast(uint32_t, h);
  }
};
struct EFp32 {
  static constexpr int kSize = 4;
};

// One element.
template <class T>
__device__ __forceinline__ float load1(const char* p) {
  if constexpr (T::kSize == 4) {
    return *reinterpret_cast<const float*>(p);
  } else {
    float a, b;
    T::unpair(*reinterpret_cast<const uint16_t*>(p), a, b);
    return a;
  }
}
template <class T>
__device__ __forceinline__ void store1(char* p, float f) {
  if constexpr (T::kSize == 4)
    *reinterpret_cast<float*>(p) = f;
  else
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(T::pair(f, 0.0f));
}

// The memory words of N consecutive elements (N = 4 or 8; any element alignment), kept as loaded: a 16-bit
// pack costs half the registers of its fp32 values.
template <class T, int N>
struct Raw {
  static constexpr int kWords = N * T::kSize / 4;
  uint32_t w[kWords];
};

// Accesses of 8 and 16 bytes at addresses that are multiples of A (2 or 4).  The vector type of reduced alignment is named
// where memory is touched: as a template argument it would lose that attribute.  Nt: non-temporal, for bytes that
// this launch touches once.
template <int A, bool Nt>
__device__ __forceinline__ u32x4 load16(const char* p) {
  if constexpr (A == 2) {
    const u32x4_a2* q = reinterpret_cast<const u32x4_a2*>(p);
    if constexpr (Nt) return __builtin_nontemporal_load(q); else return *q;
  } else {
    const u32x4_a4* q = reinterpret_cast<const u32x4_a4*>(p);
    if constexpr (Nt) return __builtin_nontemporal_load(q); else return *q;
  }
}
template <int A, bool Nt>
__device__ __forceinline__ void store16(char* p, u32x4 v) {
  if constexpr (A == 2) {
    u32x4_a2* q = reinterpret_cast<u32x4_a2*>(p);
    if constexpr (Nt) __builtin_nontemporal_store(v, q); else *q = v;
  } else {
    u32x4_a4* q = reinterpret_cast<u32x4_a4*>(p);
    if constexpr (Nt) __builtin_nontemporal_store(v, q); else *q = v;
  }
}
template <bool Nt>
__device__ __forceinline__ u32x2 load8(const char* p) {
  const u32x2_a2* q = reinterpret_cast<const u32x2_a2*>(p);
  if constexpr (Nt) return __builtin_nontemporal_load(q); else return *q;
}
template <bool Nt>
__device__ __forceinline__ void store8(char* p, u32x2 v) {
  u32x2_a2* q = reinterpret_cast<u32x2_a2*>(p);
  if constexpr (Nt) __builtin_nontemporal_store(v, q); else *q = v;
}

template <class T, int N, bool Nt>
__device__ __forceinline__ Raw<T, N> load_raw(const char* p) {
  Raw<T, N> r;
  if constexpr (Raw<T, N>::kWords == 2) {
    const u32x2 v = load8<Nt>(p);
    r.w[0] = v[0];
    r.w[1] = v[1];
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T, N>::kWords; i += 4) {
      const u32x4 v = load16<T::kSize, Nt>(p + 4 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) r.w[i + j] = v[j];
    }
  }
  return r;
}
template <class T, int N, bool Nt>
__device__ __forceinline__ void store_raw(char* p, const Raw<T, N>& r) {
  if constexpr (Raw<T, N>::kWords == 2) {
    store8<Nt>(p, u32x2{r.w[0], r.w[1]});
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T, N>::kWords; i += 4)
      store16<T::kSize, Nt>(p + 4 * i, u32x4{r.w[i], r.w[i + 1], r.w[i + 2], r.w[i + 3]});
  }
}

template <class T, int N>
__device__ __forceinline__ void widen(const Raw<T, N>& r, float (&f)[N]) {
  if constexpr (T::kSize == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __uint_as_float(r.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) T::unpair(r.w[i / 2], f[i], f[i + 1]);
  }
}
template <class T, int N>
__device__ __forceinline__ Raw<T, N> narrow(const float (&f)[N]) {
  Raw<T, N> r;
  if constexpr (T::kSize == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) r.w[i / 2] = T::pair(f[i], f[i + 1]);
  }
  return r;
}

// The first `cnt` (0 .. N) elements at p as a pack, zeros after them.
template <class T, int N, bool Nt>
__device__ __forceinline__ Raw<T, N> load_part(const char* p, int cnt) {
  if (cnt >= N) return load_raw<T, N, Nt>(p);
  float f[N];
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = i < cnt ? load1<T>(p + i * T::kSize) : 0.0f;
  return narrow<T, N>(f);  // exact: every value came from the type
}
template <class T, int N, bool Nt>
__device__ __forceinline__ void store_part(char* p, const float (&f)[N], int cnt) {
  if (cnt >= N) {
    store_raw<T, N, Nt>(p, narrow<T, N>(f));
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < cnt) store1<T>(p + i * T::kSize, f[i]);
}

// Sum over the B neighbouring lanes (8, 16, 32 or 64) that hold a row, in every one of them, in a fixed order.  Moves within 16
// lanes ride on the adds as DPP operands (quads by 1 and 2, then the mirrored half row and row); the four rows of a
// wave are read into scalar registers.  A butterfly of LDS-routed shuffles (wave_sum) measured slower where the waves of
// a workgroup wait for one another: forward 16384 x 8192 89.1 -> 90.4 us, backward 60003 x 1025 84 -> 87.  Where they do
// not it leaves the vector units free: backward 200003 x 512 109.7 -> 103.4 us.
template <int Ctrl>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), Ctrl, 0xf, 0xf, true));
}
template <int B>
__device__ __forceinline__ float lanes_sum(float x) {
  static_assert(B == 8 || B == 16 || B == 32 || B == 64, "lanes of a row");
  x += dpp<0xB1>(x);   // quad lanes 1 0 3 2
  x += dpp<0x4E>(x);   // quad lanes 2 3 0 1
  x += dpp<0x141>(x);  // half row mirrored
  if constexpr (B > 8) x += dpp<0x140>(x);  // row mirrored
  if constexpr (B == 32) x += __shfl_xor(x, 16);
  if constexpr (B == 64) {
    const int b = __float_as_int(x);
    x = (__int_as_float(__builtin_amdgcn_readlane(b, 0)) + __int_as_float(__builtin_amdgcn_readlane(b, 16))) +
        (__int_as_float(__builtin_amdgcn_readlane(b, 32)) + __int_as_float(__builtin_amdgcn_readlane(b, 48)));
  }
  return x;
}

// The same sum as a butterfly of shuffles (B lanes), in every lane.
template <int B = 64, class F>
__device__ __forceinline__ F wave_sum(F x) {
#pragma unroll
  for (int m = B / 2; m; m >>= 1) x += __shfl_xor(x, m);
  return x;
}

}  // namespace mr
