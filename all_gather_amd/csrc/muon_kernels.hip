// Muon's step over a list of matrices, for gfx950: momentum, Newton-Schulz orthogonalisation, update.
//
//   m' = mu m + (1 - mu) f g,   u = mu m' + (1 - mu) f g (Nesterov) or m',   X = u / max(|u|, eps)
//   steps times:  A = X X^T,  P = a I + b A + c A^2,  X = P X
//   p' = (1 - lr wd) p - lr s X
//
// The products are the work: per step 2 m^2 n (A, half of it by symmetry), 2 m^3 (A^2, likewise) and 2 m^2 n operations.
// They run on the matrix cores with fp16 operands and fp32 sums.  fp16, not bf16: X, A and P are bounded by their spectral norms (the
// host checks that the polynomials keep them below 16), so held times 2^12 they use fp16's range and have 8 times bf16's
// precision at the same rate.  The polynomial raises what is left of a small singular value 485-fold in five steps, and the
// rounding of X with it: after them X is off by 1e-3 to 2e-2 of its norm (bf16: 1e-2 to 2e-1), which an update of 16-bit parameters does
// not resolve.  For fp32 results every matrix is held in two fp16 pieces, hi + lo, and a product is three: off by 1e-5, as in fp32.
//
// Every product is C = A B^T with both operands' rows along the sum, so one kernel serves all three: X's transpose is kept
// beside it, and A and P are symmetric.

#include <hip/hip_runtime.h>

#include <type_traits>

#include "mr_train.h"
#include "packs.h"

namespace mr {
namespace {

typedef _Float16 f16;
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kUp = 1 << kNsShift, kDown = 1.0f / (1 << kNsShift);

// A matrix of `rows` rows lies in panels of 32 columns, each panel's rows after one another (64 bytes a row): what a product
// fetches at a time is one run of memory, and no stride of a power of two.  In two pieces a panel is 16 columns, their first
// pieces and then their second: a stage holds both, and every operand that it brings in is used twice.
constexpr uint32_t kPieceAt = kNsK / 2;  // from a value's first piece to its second
__device__ __forceinline__ size_t in_panels(size_t rows, uint32_t r, uint32_t c, int pieces) {
  const uint32_t w = kNsK / pieces;
  return (c / w * rows + r) * kNsK + c % w;
}

// The matrix whose tiles hold tile t.
__device__ __forceinline__ uint32_t entry_of(const uint32_t* prefix, uint32_t P, uint32_t t) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t first = lane < P ? prefix[lane] : 0xffffffffu;
  return static_cast<uint32_t>(__builtin_popcountll(__builtin_amdgcn_ballot_w64(first <= t))) - 1;
}
static_assert(kMuonMats <= 64, "one prefix entry a lane");

struct Clip {
  float f;
  bool take;
};
__device__ __forceinline__ Clip clip_of(const float* clip) { return clip ? Clip{clip[1], clip[2] != 0.0f} : Clip{1.0f, true}; }

// The new momentum and the update before it is normalised, from the old momentum and from the new: the same bits.
__device__ __forceinline__ float new_momentum(float m, float g, float mu, float c) { return mu * m + c * g; }
__device__ __forceinline__ float update_of(float m_new, float g, float mu, float c, int nesterov) { return nesterov ? mu * m_new + c * g : m_new; }

__device__ __forceinline__ double group_sum(double x) {
  __shared__ double lds[4];
  x = wave_sum(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// m' of a tile of one matrix, and its part of |u|^2 in fp64; the workgroup that finishes its matrix last adds the parts up in order.
// Bound by the bytes (m, g, m'), so every load of 4096 elements is on its way before the first is used: 201M elements with bf16
// gradients in 360 us (5.6 TB/s).  A matrix's own size sets its tiles, so that its norm is summed in the same order alone and in any
// list.  Large tiles for large matrices: a workgroup counts its arrival at its matrix's counter, which takes 11.6 ns (2000 x 2000 16.5 us,
// by tiles of 4096 21.2; 1500 x 1500 14.3 by both).  Counters lie a line apart: neighbours' arrivals wait for one another (48 of 2048 x 2048
// by tiles of 4096 took 240 us longer).
template <class G>
__global__ __launch_bounds__(256) void momentum(MomentumArgs a) {
  const Clip clip = clip_of(a.clip);
  const uint32_t i = entry_of(a.tile_prefix, a.P, blockIdx.x), tile = blockIdx.x - a.tile_prefix[i];
  const uint32_t tile_elems = a.tile[i];
  const uint64_t n = a.n[i], padded = (n + kMxBlock - 1) / kMxBlock * kMxBlock;
  const uint64_t end = uint64_t{tile + 1} * tile_elems < padded ? uint64_t{tile + 1} * tile_elems : padded;
  const char* g = a.g[i];
  const float* m = a.m + a.at[i];
  float* mo = a.m_out + a.at[i];
  constexpr int kU = 4;
  double s = 0.0;
  for (uint64_t e0 = uint64_t{tile} * tile_elems + threadIdx.x * 4; e0 < end; e0 += kU * 1024) {
    Raw<G, 4> gr[kU];
    Raw<EFp32, 4> mr[kU];
    const bool whole = e0 - threadIdx.x * 4 + kU * 1024 <= n;
    if (whole) {
#pragma unroll
      for (int k = 0; k < kU; ++k) {
        gr[k] = load_raw<G, 4, false>(g + (e0 + k * 1024) * G::kSize);
        mr[k] = load_raw<EFp32, 4, true>(reinterpret_cast<const char*>(m + e0 + k * 1024));
      }
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const uint64_t e = e0 + k * 1024;
      int live = 4;
      if (!whole) {
        if (e >= end) break;  // whole packs of the state
        live = e >= n ? 0 : n - e < 4 ? static_cast<int>(n - e) : 4;
        gr[k] = load_part<G, 4, false>(g + e * G::kSize, live);
        mr[k] = load_raw<EFp32, 4, true>(reinterpret_cast<const char*>(m + e));
      }
      float gf[4], mf[4], out[4];
      widen(gr[k], gf);
      widen(mr[k], mf);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float gj = clip.f * gf[j];
        out[j] = j < live ? clip.take ? new_momentum(mf[j], gj, a.mu, a.c) : mf[j] : 0.0f;
        const double u = j < live ? static_cast<double>(update_of(out[j], gj, a.mu, a.c, a.nesterov)) : 0.0;
        s = __builtin_fma(u, u, s);
      }
      store_raw<EFp32, 4, false>(reinterpret_cast<char*>(mo + e), narrow<EFp32, 4>(out));
      if (a.master_out)
        for (int j = live; j < 4; ++j) a.master_out[a.at[i] + e + j] = 0.0f;
    }
  }
  s = group_sum(s);
  __shared__ bool last;
  const uint32_t tiles = a.tile_prefix[i + 1] - a.tile_prefix[i];
  if (threadIdx.x == 0) {
    __hip_atomic_store(a.sums + blockIdx.x, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    last = __hip_atomic_fetch_add(a.arrived + i * kMuonCount, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == tiles - 1;
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
  }
  __syncthreads();
  if (!last) return;
  s = 0.0;
  for (uint32_t t = threadIdx.x; t < tiles; t += 256)
    s += __hip_atomic_load(a.sums + a.tile_prefix[i] + t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  s = group_sum(s);
  if (threadIdx.x == 0) {
    a.norms[i] = __builtin_sqrt(s);
    __hip_atomic_store(a.arrived + i * kMuonCount, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

// N values in fp16 (the rest of them in a second piece) to `at`.
template <int N>
__device__ __forceinline__ void store_pieces(f16* at, int pieces, const float (&v)[N]) {
  typedef f16 Pack __attribute__((ext_vector_type(N)));
  Pack hi, lo;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    hi[q] = static_cast<f16>(v[q]);
    lo[q] = static_cast<f16>(v[q] - static_cast<float>(hi[q]));
  }
  *reinterpret_cast<Pack*>(at) = hi;
  if (pieces == 2) *reinterpret_cast<Pack*>(at + kPieceAt) = lo;
}

// u / |u| of a 64 x 64 tile, times 2^12, in fp16: as it lies, and transposed.  Columns past the matrix become zeros.  Bound by the bytes:
// m', g and two results of 201M elements in 376 us (5.3 TB/s).  A tile is turned through LDS, so both results are stored in runs of 16 bytes a lane.
template <class G>
__global__ __launch_bounds__(256) void orient(OrientArgs a) {
  __shared__ float tile[64][65];
  const Clip clip = clip_of(a.clip);
  const uint32_t i = entry_of(a.tile_prefix, a.P, blockIdx.x), t = blockIdx.x - a.tile_prefix[i];
  const uint32_t rows = a.rows[i], cols = a.cols[i], ld_direct = ns_padded(cols), ld_turned = ns_padded(rows), across = (ld_direct + 63) / 64;
  const uint32_t r0 = t / across * 64, c0 = t % across * 64;
  const double norm = a.norms[i];
  const double by = norm > a.eps ? norm : norm == norm ? a.eps : norm;  // NaN stays
  const float inv = static_cast<float>(static_cast<double>(kUp) / by);
  {
    const uint32_t x = threadIdx.x % 16 * 4, y = threadIdx.x / 16, c = c0 + x;
    const int live = c >= cols ? 0 : cols - c < 4 ? static_cast<int>(cols - c) : 4;
    Raw<G, 4> gr[4];
    Raw<EFp32, 4> mr[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t r = r0 + k * 16 + y;
      const size_t e = static_cast<size_t>(r) * cols + c;
      const int n = r < rows ? live : 0;
      gr[k] = load_part<G, 4, true>(a.g[i] + e * G::kSize, n);
      mr[k] = load_part<EFp32, 4, false>(reinterpret_cast<const char*>(a.m + a.at[i] + e), n);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t r = r0 + k * 16 + y;
      float gf[4], mf[4], u[4];
      widen(gr[k], gf);
      widen(mr[k], mf);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u[j] = r < rows && j < live ? update_of(mf[j], clip.f * gf[j], a.mu, a.c, a.nesterov) * inv : 0.0f;
        tile[k * 16 + y][x + j] = u[j];
      }
      if (r < rows && c < ld_direct) store_pieces(a.direct[i] + in_panels(rows, r, c, a.pieces), a.pieces, u);
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t y = threadIdx.x % 8 * 8, x = k * 32 + threadIdx.x / 8, c = c0 + x, r = r0 + y;
    if (c >= cols || r >= ld_turned) continue;
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = tile[y + j][x];
    store_pieces(a.turned[i] + in_panels(cols, c, r, a.pieces), a.pieces, u);
  }
}

// ------------------------------------------------------------------------------------------- products
//
// A workgroup of WR x WC waves makes a BM x BN tile; a wave holds its part of it as 32 x 32 blocks in accumulators.  The operands
// go from memory straight to LDS, in stages of 32 columns on a ring of 3: one stage is multiplied while the next is there or
// on its way and the one after it is asked for, so that a wait finds loads that were issued a stage's products ago (a ring of 4: the same
// time).  In LDS a row of a stage is 4 chunks of 16 bytes;
// chunk c of row r lies at place c ^ swizzle(r), so that the 16 rows that are read at once fall on all 64 banks.  (The hardware
// writes a wave's 64 chunks one after another: the lane that fills a place fetches the chunk that belongs there.)
//
// The matrix cores are busy for 69% of the cycles at the 1.6 to 1.7 GHz (of 2.4) that such products run at, the epilogue takes 7%; what the
// rest waits for was not found.  (The library's plain 4096^3 fp16 product reaches 1.30 PFLOP/s on this card, 8192^3 1.43, so the power limit
// alone is not it.)  For four matrices of 4096 x 4096 and two of 4096 x 16384 P X takes 1.46 to 1.51 ms a launch (1.10 to 1.13 PFLOP/s),
// X X^T 0.82 (1.01) and A^2 0.43 to 0.44 (0.95 to 0.97).  In two pieces a step of those matrices takes 36.6 to 37.5 ms, 1.16 to 1.18 PFLOP/s.
// Measured and no faster: tiles of 256 x 256 on 8 waves, of 128 x 128 a wave on 4 (15.1 against 14.6 ms a step), results stored past the
// caches, panels of 4 tile rows instead of 8.
constexpr int kStages = 3, kRow = kNsK;  // halves of an LDS row
__device__ __forceinline__ uint32_t swizzle(uint32_t r) { return r >> 2 & 3; }

// Rows [0, R) of an operand's tile, one stage, by all waves of the workgroup.  The buffer ends with the matrix's rows: past them
// the hardware fills in zeros.
template <int R, int Waves>
struct Fetch {
  static constexpr int kLoads = R / 16 / Waves;
  static_assert(R % (16 * Waves) == 0, "whole loads");
  int off;    // bytes, of the first load; a further one lies 16 * Waves rows on
  int bytes;  // of the tile's rows in a panel
  __device__ explicit Fetch(uint32_t rows_left) {
    const uint32_t lane = threadIdx.x & 63, r = (threadIdx.x >> 6) * 16 + lane / 4;
    off = static_cast<int>((r * kNsK + ((lane % 4) ^ swizzle(r)) * 8) * 2);
    bytes = static_cast<int>((rows_left < R ? rows_left : R) * kNsK * 2);
  }
  // One of the loads.  `wave` is in a scalar register.
  __device__ __forceinline__ void issue(const f16* base, f16* lds, uint32_t wave, int i) const {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<f16*>(base), 0, bytes, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)(lds + (i * Waves + wave) * 16 * kRow), 16,
                                             off + i * Waves * 16 * kRow * 2, 0, 0, 0);
  }
};

struct Where {  // a workgroup's tile
  uint32_t i, ti, tj;
};
template <int BM, int BN>
__device__ __forceinline__ Where tile_of(const NsArgs& a, bool symmetric) {
  Where w;
  w.i = __builtin_amdgcn_readfirstlane(entry_of(a.tile_prefix, a.P, blockIdx.x));
  // neighbouring tiles of a matrix on one XCD, whose L2 then holds their operands; every matrix over all XCDs
  const uint32_t first = a.tile_prefix[w.i], total = a.tile_prefix[w.i + 1] - first, b = blockIdx.x - first;
  const uint32_t per = total / kXcds, rest = total % kXcds, x = b % kXcds;
  const uint32_t q = x * per + (x < rest ? x : rest) + b / kXcds;
  const uint32_t tm = (a.p[w.i].ldct + BM - 1) / BM, tn = (a.p[w.i].ldc + BN - 1) / BN;
  if (symmetric) {  // tiles that meet the lower triangle, by blocks of BN rows
    constexpr uint32_t kRatio = BN / BM;
    uint32_t r = static_cast<uint32_t>((__builtin_sqrtf(8.0f / kRatio * q + 1.0f) - 1.0f) * 0.5f);  // kRatio r (r + 1) / 2 tiles lie before block r
    while (kRatio * r * (r + 1) / 2 > q) --r;
    while (kRatio * (r + 1) * (r + 2) / 2 <= q) ++r;
    const uint32_t in = q - kRatio * r * (r + 1) / 2;
    w.ti = kRatio * r + in / (r + 1);
    w.tj = in % (r + 1);
  } else {  // panels of 8 tile rows, column by column
    const uint32_t panel = q / (8 * tn), rows = tm - panel * 8 < 8 ? tm - panel * 8 : 8, in = q - panel * 8 * tn;
    w.ti = panel * 8 + in % rows;
    w.tj = in / rows;
  }
  w.ti = __builtin_amdgcn_readfirstlane(w.ti);
  w.tj = __builtin_amdgcn_readfirstlane(w.tj);
  return w;
}

template <int BM, int BN, int WR, int WC>
struct Tile {
  static constexpr int kWaves = WR * WC, kMi = BM / WR / 32, kNj = BN / WC / 32;
  static constexpr int kHalves = (BM + BN) * kRow;  // of a stage
  f32x16 acc[kMi][kNj];  // block (i, j), transposed: lane l has row l % 32, columns 8 (e / 4) + 4 (l / 32) + e % 4

  // Arrays of their own: so the compiler knows that a stage's reads need not wait for what is on its way to another.
  template <int S>
  static __device__ __forceinline__ f16* stage() {
    __shared__ __attribute__((aligned(16))) f16 s[kHalves];
    return s;
  }

  // A wave's operands of 16 columns.
  struct Part {
    f16x8 x[kMi], y[kNj];
  };
  static constexpr int kReads = kMi + kNj, kProducts = kMi * kNj;
  // The n-th of them from LDS: x0 y0 x1 y1 ..., as the products take them.
  __device__ __forceinline__ void read(Part& p, const f16* lds, int k, int n) const {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t ra = wave / WC * (BM / WR) + lane % 32, rb = wave % WC * (BN / WC) + lane % 32;
    const int most = kMi < kNj ? kMi : kNj;
    const bool is_x = n < 2 * most ? n % 2 == 0 : kMi > kNj;
    const int i = n < 2 * most ? n / 2 : n - most;
    if (is_x)
      p.x[i] = *reinterpret_cast<const f16x8*>(lds + (ra + i * 32) * kRow + ((2 * k + lane / 32) ^ swizzle(ra)) * 8);
    else
      p.y[i] = *reinterpret_cast<const f16x8*>(lds + (BM + rb + i * 32) * kRow + ((2 * k + lane / 32) ^ swizzle(rb)) * 8);
  }
  // The n-th block's product of px's x and py's y.
  __device__ __forceinline__ void product(const Part& px, const Part& py, int n) {
    const int i = n / kNj, j = n % kNj;
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(py.y[j], px.x[i], acc[i][j], 0, 0, 0);
  }
  static __device__ __forceinline__ void clear(Part& p) {
#pragma unroll
    for (int i = 0; i < kMi; ++i) p.x[i] = f16x8{};
#pragma unroll
    for (int j = 0; j < kNj; ++j) p.y[j] = f16x8{};
  }

  // The sum over K columns (a whole number of turns of the ring, an even one for two pieces).
  template <int Pieces>
  __device__ __forceinline__ void run(const NsProduct& p, uint32_t ti, uint32_t tj) {
#pragma unroll
    for (int i = 0; i < kMi; ++i)
#pragma unroll
      for (int j = 0; j < kNj; ++j) acc[i][j] = f32x16{};
    if (ti * BM >= p.M || tj * BN >= p.N) return;  // columns past the matrix alone
    const Fetch<BM, kWaves> fa(p.M - ti * BM);
    const Fetch<BN, kWaves> fb(p.N - tj * BN);
    const f16* a = p.a + size_t{ti} * BM * kNsK;
    const f16* b = p.b + size_t{tj} * BN * kNsK;
    const size_t a_panel = size_t{p.M} * kNsK, b_panel = size_t{p.N} * kNsK;
    const uint32_t steps = p.K / kNsK * Pieces;
    uint32_t ahead = 0;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int kLoads = Fetch<BM, kWaves>::kLoads + Fetch<BN, kWaves>::kLoads;  // of a stage
    auto fetch = [&](f16* s, int i) {
      if (i < Fetch<BM, kWaves>::kLoads)
        fa.issue(a, s, wave, i);
      else
        fb.issue(b, s + BM * kRow, wave, i - Fetch<BM, kWaves>::kLoads);
    };
    auto advance = [&] {
      // past the end the last stage is fetched again, which nobody reads: so that every wait counts the same loads
      const bool more = ++ahead < steps;
      a += more ? a_panel : 0;
      b += more ? b_panel : 0;
    };
    for (f16* s : {stage<0>(), stage<1>()}) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) fetch(s, i);
      advance();
    }
    auto enter = [&] {
      __builtin_amdgcn_s_waitcnt(0x0070 | kLoads);  // vmcnt: all but the next stage's loads are here; lgkmcnt(0): the last one is read
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    // Beside one of a stage's Pieces + 1 groups of products: reads from LDS, and the fetches evenly over the stage (one that finds the
    // memory pipeline full holds its wave up).
    auto beside = [&](f16* last, int slot) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        if (i * (Pieces + 1) * kProducts / kLoads == slot) fetch(last, i);
      __builtin_amdgcn_sched_barrier(0);
    };
    // One stage.  Its last group of products is made after the next barrier, while that stage's first operands are read: the
    // matrix cores have work on both sides of it.
    if constexpr (Pieces == 1) {
      Part even, odd;  // the stage's first 16 columns, and its others
      clear(odd);
      auto turn = [&](const f16* now, f16* last) {
        constexpr int kEach = (kReads + kProducts - 1) / kProducts;  // reads beside a product
        enter();
#pragma unroll
        for (int n = 0; n < kProducts; ++n) {
          product(odd, odd, n);
#pragma unroll
          for (int o = n * kEach; o < (n + 1) * kEach; ++o)
            if (o < kReads) read(even, now, 0, o);
          beside(last, n);
        }
#pragma unroll
        for (int n = 0; n < kProducts; ++n) {
          product(even, even, n);
#pragma unroll
          for (int o = n * kEach; o < (n + 1) * kEach; ++o)
            if (o < kReads) read(odd, now, 1, o);
          beside(last, kProducts + n);
        }
        advance();
      };
      for (uint32_t k = 0; k < steps; k += kStages) {
        turn(stage<0>(), stage<2>());
        turn(stage<1>(), stage<0>());
        turn(stage<2>(), stage<1>());
      }
#pragma unroll
      for (int n = 0; n < kProducts; ++n) product(odd, odd, n);
    } else {
      Part hi0, hi1, lo;  // first pieces of this stage and the last one, by turns; second pieces
      clear(hi1);
      auto turn = [&](const f16* now, f16* last, Part& hi, Part& before) {
        constexpr int kEach = (2 * kReads + kProducts - 1) / kProducts;
        enter();
#pragma unroll
        for (int n = 0; n < kProducts; ++n) {
          product(before, before, n);
#pragma unroll
          for (int o = n * kEach; o < (n + 1) * kEach; ++o) {
            if (o < kReads)
              read(hi, now, 0, o);
            else if (o < 2 * kReads)
              read(lo, now, 1, o - kReads);
          }
          beside(last, n);
        }
#pragma unroll
        for (int n = 0; n < kProducts; ++n) {
          product(hi, lo, n);
          beside(last, kProducts + n);
        }
#pragma unroll
        for (int n = 0; n < kProducts; ++n) {
          product(lo, hi, n);
          beside(last, 2 * kProducts + n);
        }
        advance();
      };
      for (uint32_t k = 0; k < steps; k += 2 * kStages) {
        turn(stage<0>(), stage<2>(), hi0, hi1);
        turn(stage<1>(), stage<0>(), hi1, hi0);
        turn(stage<2>(), stage<1>(), hi0, hi1);
        turn(stage<0>(), stage<2>(), hi1, hi0);
        turn(stage<1>(), stage<0>(), hi0, hi1);
        turn(stage<2>(), stage<1>(), hi1, hi0);
      }
#pragma unroll
      for (int n = 0; n < kProducts; ++n) product(hi1, hi1, n);
    }
  }

  // Results leave through LDS, where each wave turns 32 rows of its part at a time in a place of its own, so that a lane has 8
  // values that lie together in memory.  A row is kCc / 4 places of 16 bytes; place c of row r lies at c ^ spread(r): a wave's
  // writes (32 rows, one place each), its reads along the rows and those down the columns each meet all banks.
  static constexpr int kCr = 32, kCc = BN / WC;
  static __device__ __forceinline__ uint32_t place(uint32_t r, uint32_t c) {
    return r * kCc + (((c / 4) ^ ((r ^ (r >> 3) << 2) & (kCc / 4 - 1))) * 4) + c % 4;
  }

  // row(r, c, v): 8 values of row r from column c on, which it may change; column(r, c, v): 8 values of column c from row r on.
  template <bool Rows, bool Columns, class R, class C>
  __device__ __forceinline__ void leave(uint32_t ti, uint32_t tj, R row, C column) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    constexpr uint32_t kPer = (kWaves + kStages - 1) / kStages;  // waves whose places share a stage
    static_assert(kPer * kCr * kCc * 4 <= 2 * kHalves, "room in a stage");
    const uint32_t in = wave / kPer;
    float* lds = reinterpret_cast<float*>(in == 0 ? stage<0>() : in == 1 ? stage<1>() : stage<2>()) + wave % kPer * (kCr * kCc);
    const uint32_t r0 = ti * BM + wave / WC * (BM / WR), c0 = tj * BN + wave % WC * (BN / WC);
    // What was fetched past the end is on its way to the stages that are written next, and a barrier does not wait for it.
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    asm volatile("" ::: "memory");
    __syncthreads();  // the stages have been read
#pragma unroll
    for (int h = 0; h < kMi * 32 / kCr; ++h) {
#pragma unroll
      for (int i = 0; i < kCr / 32; ++i)
#pragma unroll
        for (int j = 0; j < kNj; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            typedef float f32x4 __attribute__((ext_vector_type(4)));
            const f32x16& x = acc[h * (kCr / 32) + i][j];
            *reinterpret_cast<f32x4*>(lds + place(i * 32 + lane % 32, j * 32 + 8 * e + 4 * (lane / 32))) =
                f32x4{x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]};
          }
      if constexpr (Rows) {
#pragma unroll
        for (int k = 0; k < kCr * kCc / 512; ++k) {
          const uint32_t r = k * (512 / kCc) + lane / (kCc / 8), c = lane % (kCc / 8) * 8;
          float v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = lds[place(r, c + q / 4 * 4) + q % 4];
          row(r0 + h * kCr + r, c0 + c, v);
          if constexpr (Columns)
#pragma unroll
            for (int q = 0; q < 8; ++q) lds[place(r, c + q / 4 * 4) + q % 4] = v[q];
        }
      }
      if constexpr (Columns) {
#pragma unroll
        for (int k = 0; k < kCr * kCc / 512; ++k) {
          const uint32_t c = k * (512 / kCr) + lane / (kCr / 8), r = lane % (kCr / 8) * 8;
          float v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = lds[place(r + q, c)];
          column(r0 + h * kCr + r, c0 + c, v);
        }
      }
    }
  }
};

template <NsKind Kind, int Pieces, int BM, int BN, int WR, int WC>
__global__ __launch_bounds__(WR* WC * 64) void ns_product(NsArgs a) {
  constexpr bool kSym = Kind != kNsStep;
  const Where w = tile_of<BM, BN>(a, kSym);
  const NsProduct p = a.p[w.i];
  Tile<BM, BN, WR, WC> t;
  t.template run<Pieces>(p, w.ti, w.tj);
  const bool both = !kSym || w.tj < w.ti / (BN / BM);  // else the transpose's places are another tile's, or this one's
  t.template leave<true, true>(
      w.ti, w.tj,
      [&](uint32_t r, uint32_t c, float (&v)[8]) {
        const bool in = r < p.M && c < p.ldc;
        if constexpr (Kind == kNsPoly) {
          float add[8] = {};
          if (in) {  // P's columns are A's
            for (int s = 0; s < Pieces; ++s) {
              const f16x8 x = *reinterpret_cast<const f16x8*>(p.a + s * kPieceAt + in_panels(p.M, r, c, Pieces));
#pragma unroll
              for (int q = 0; q < 8; ++q) add[q] += static_cast<float>(x[q]);
            }
          }
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = a.cb * add[q] + a.cc * (v[q] * kDown) + (r == c + q ? a.ca * kUp : 0.0f);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] *= kDown;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (c + q >= p.N || r >= p.M) v[q] = 0.0f;  // what lies past the matrix, in C and in its transpose
        if (in) store_pieces(p.c + in_panels(p.M, r, c, Pieces), Pieces, v);
      },
      [&](uint32_t r, uint32_t c, float (&v)[8]) {
        if (both && r < p.ldct && c < p.N) store_pieces((kSym ? p.c : p.ct) + in_panels(p.N, c, r, Pieces), Pieces, v);
      });
}

// The last product of the last step, which updates the parameters instead of being stored: as long as a step's other product (201M
// bf16 parameters 1.47 ms; a launch of its own for them would move 1.2 GB in 0.2).
template <class T, int Pieces, int BM, int BN, int WR, int WC>
__global__ __launch_bounds__(WR* WC * 64) void ns_last(NsLastArgs a) {
  const Where w = tile_of<BM, BN>(a.s, false);
  const NsProduct p = a.s.p[w.i];
  const NsUpdate u = a.u[w.i];
  const Clip clip = clip_of(a.clip);
  Tile<BM, BN, WR, WC> t;
  t.template run<Pieces>(p, w.ti, w.tj);
  const float by = u.scale * kDown * kDown;
  // n (1 to 8) of the values v belong to the matrix, from its element e on
  auto update = [&](size_t e, int n, const float (&v)[8]) {
    float x[8];
    if (a.master)
      widen(load_part<EFp32, 8, true>(reinterpret_cast<const char*>(a.master + u.at + e), n), x);
    else
      widen(load_part<T, 8, true>(u.p + e * T::kSize, n), x);
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = clip.take ? a.keep * x[q] - by * v[q] : x[q];
    if (a.master) store_part<EFp32, 8, true>(reinterpret_cast<char*>(a.master_out + u.at + e), x, n);
    store_part<T, 8, true>(u.po + e * T::kSize, x, n);
  };
  auto left = [](uint32_t at, uint32_t end) { return end - at < 8 ? static_cast<int>(end - at) : 8; };
  if (u.turned)
    t.template leave<false, true>(w.ti, w.tj, [](uint32_t, uint32_t, float (&)[8]) {}, [&](uint32_t r, uint32_t c, float (&v)[8]) {
      if (r < p.M && c < p.N) update(static_cast<size_t>(c) * p.M + r, left(r, p.M), v);
    });
  else
    t.template leave<true, false>(w.ti, w.tj, [&](uint32_t r, uint32_t c, float (&v)[8]) {
      if (r < p.M && c < p.N) update(static_cast<size_t>(r) * p.N + c, left(c, p.N), v);
    }, [](uint32_t, uint32_t, float (&)[8]) {});
}

template <NsKind Kind, int Pieces>
void product(const NsArgs& a, uint32_t tile, hipStream_t st) {
  const dim3 grid(a.tile_prefix[a.P]);
  if (tile == 256)
    hipLaunchKernelGGL((ns_product<Kind, Pieces, 128, 256, 1, 4>), grid, dim3(256), 0, st, a);
  else if (tile == 128)
    hipLaunchKernelGGL((ns_product<Kind, Pieces, 128, 128, 2, 2>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((ns_product<Kind, Pieces, 64, 64, 2, 2>), grid, dim3(256), 0, st, a);
}
template <class T, int Pieces>
void last(const NsLastArgs& a, uint32_t tile, hipStream_t st) {
  const dim3 grid(a.s.tile_prefix[a.s.P]);
  if (tile == 256)
    hipLaunchKernelGGL((ns_last<T, Pieces, 128, 256, 1, 4>), grid, dim3(256), 0, st, a);
  else if (tile == 128)
    hipLaunchKernelGGL((ns_last<T, Pieces, 128, 128, 2, 2>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((ns_last<T, Pieces, 64, 64, 2, 2>), grid, dim3(256), 0, st, a);
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

// Tiles of 128 x 256 ask least of LDS and L2, tiles of 128 x 128 and of 64 x 64 leave fewer compute units idle where a launch has few.
// A step with wide tiles and square ones (ms): eight of 4096 x 4096 11.2 and 12.7; 32 of 768 x 8192 4.45 and 4.64; one of 4096 x 4096
// (512 wide tiles a product) 1.98 and 1.91; one of 2048 x 2048 0.56 and 0.47 (0.39 to 0.42 by 64 x 64); one of 4096 x 8192 (1024) 3.08 and 3.04, of
// 4096 x 16384 (2048) 5.33 and 5.41.
// With tiles of 128 x 128 and of 64 x 64 (us): one of 512 x 512 171 and 124, eight (128 square tiles a product) 200 and 160, 32 (512) 372
// and 393; one of 1024 x 1024 (64) 237 and 177, one of 1536 x 4096 (384) 452 and 424, eight of 1000 x 1000 (648) 455 and 470; 32 of
// 384 x 1536 (1152) 439 and 476.
// In two pieces the order of an element's sums differs between tile sizes (A and P are mirrored), so there a matrix's rows alone choose
// between the smaller two: in a list without wide tiles it gets the bits that it gets alone.  (One of 512 x 512 255 us by 128 x 128, 172 by 64 x 64.)
constexpr uint64_t kNsMany = 1024, kNsSome = 400;
uint32_t ns_tile(uint32_t m, const NsTiles& list, int pieces) {
  if (m >= kNsWideFrom && list.wide > kNsMany) return 256;
  if (pieces == 2) return m >= kNsWideFrom ? 128 : 64;
  return m >= kNsSquareFrom && list.square > kNsSome ? 128 : 64;
}

uint32_t ns_tiles(uint32_t tile, uint32_t rows, uint32_t cols, bool symmetric) {
  const uint32_t bm = tile == 256 ? 128 : tile, bn = tile, ratio = bn / bm;
  const uint32_t tm = (rows + bm - 1) / bm, tn = (cols + bn - 1) / bn;
  if (!symmetric) return tm * tn;
  const uint32_t h = tm / ratio;  // whole blocks of bn rows
  return ratio * h * (h + 1) / 2 + tm % ratio * (h + 1);
}

hipError_t launch_momentum(const MomentumArgs& a, mr_dtype gdt, hipStream_t st) {
  by_type(gdt, [&](auto g) { hipLaunchKernelGGL((momentum<decltype(g)>), dim3(a.tile_prefix[a.P]), dim3(256), 0, st, a); });
  return hipGetLastError();
}
hipError_t launch_orient(const OrientArgs& a, mr_dtype gdt, hipStream_t st) {
  by_type(gdt, [&](auto g) { hipLaunchKernelGGL((orient<decltype(g)>), dim3(a.tile_prefix[a.P]), dim3(256), 0, st, a); });
  return hipGetLastError();
}
hipError_t launch_ns(const NsArgs& a, NsKind kind, uint32_t tile, hipStream_t st) {
  auto go = [&](auto pieces) {
    constexpr int kPieces = decltype(pieces)::value;
    if (kind == kNsGram)
      product<kNsGram, kPieces>(a, tile, st);
    else if (kind == kNsPoly)
      product<kNsPoly, kPieces>(a, tile, st);
    else
      product<kNsStep, kPieces>(a, tile, st);
  };
  if (a.pieces == 2)
    go(std::integral_constant<int, 2>{});
  else
    go(std::integral_constant<int, 1>{});
  return hipGetLastError();
}
hipError_t launch_ns_last(const NsLastArgs& a, mr_dtype dt, uint32_t tile, hipStream_t st) {
  by_type(dt, [&](auto t) {
    if (a.s.pieces == 2)
      last<decltype(t), 2>(a, tile, st);
    else
      last<decltype(t), 1>(a, tile, st);
  });
  return hipGetLastError();
}

}  // namespace mr
