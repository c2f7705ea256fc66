// Launch interface of the training-step operators, shared by train_api.hip and the kernel files.
#pragma once

#include <mutex>

#include "mr_internal.h"

namespace mr {

// ---------------------------------------------------------------------------------------- layer norm
struct NormFwdArgs {
  const char* in[MR_MAX_W + 1];  // the rank buffers and then the residual, added in this order
  const char* gamma;         // null: ones
  const char* beta;          // null: zeros
  char* x_out;               // may be null
  char* y;
  float* mean;               // may be null
  float* rstd;               // may be null
  size_t rows, cols;
  float eps;
  int terms;                 // entries of `in`
  int waves;                 // waves to a row (set by the launch)
};
hipError_t launch_norm_fwd(const NormFwdArgs& a, mr_dtype dt, mr_dtype wdt, hipStream_t st);

struct NormBwdArgs {
  const char* dy;
  const char* x;
  const char* gamma;  // null: ones
  const float* mean;
  const float* rstd;
  const char* dres;   // may be null
  char* dx;           // may be null
  char* dgamma;       // may be null
  char* dbeta;        // may be null
  float* part;        // [groups][2][cols] partial weight gradients (null: none wanted)
  size_t rows, cols;
  uint32_t groups;
  int waves;          // waves to a row (set by the launch)
  uint32_t* arrived;  // zero between launches
  int one_launch;     // 1: the workgroup that arrives last adds `part` up (set by the launch)
};
// Row groups of the backward pass of this shape: each sums its rows' part of the weight gradients in
// registers and writes one row of `part`.  A function of the shape alone, so results do not depend on the device.
uint32_t norm_bwd_groups(size_t rows, size_t cols, mr_dtype dt);
hipError_t launch_norm_bwd(const NormBwdArgs& a, mr_dtype dt, mr_dtype wdt, hipStream_t st);

// --------------------------------------------------------------------------------- gradient norm, AdamW
constexpr int kNormTensors = 128;           // tensors per launch (their table rides in the kernel arguments)
constexpr uint32_t kNormTileBytes = 16384;  // of one tensor
constexpr uint32_t kNormMaxGroups = 512;    // workgroups, and so partial sums, per launch: two to a compute unit
constexpr uint32_t kNormSets = 8;           // arrivals are counted in sets, then sets: one address takes 11.6 ns an arrival
struct GradNormArgs {
  const char* g[kNormTensors];
  uint64_t n[kNormTensors];
  uint32_t tile_prefix[kNormTensors + 1];
  uint32_t P;
  double* part;             // partial sums of squares, one per workgroup of every launch of the call
  uint32_t part_base;       // this launch's first one
  uint32_t finish;          // 1: the last launch; its last workgroup adds all of them up
  uint32_t (*arrived)[64];  // zero between launches
  double scale, max_norm;
  float* out;
};
inline uint32_t grad_norm_groups(uint32_t tiles) { return tiles == 0 ? 1 : tiles < kNormMaxGroups ? tiles : kNormMaxGroups; }
hipError_t launch_grad_norm(const GradNormArgs& a, mr_dtype dt, hipStream_t st);

constexpr int kAdamTensors = 80;   // tensors per launch
constexpr uint32_t kMxBlock = 32;  // elements that share a scale; a tensor's state starts on a block
struct AdamState {
  char* m;
  char* v;
  uint8_t* ms;
  uint8_t* vs;
  float* master;
};
struct AdamArgs {
  const char* p[kAdamTensors];
  const char* g[kAdamTensors];
  char* po[kAdamTensors];
  uint64_t n[kAdamTensors];
  uint32_t block0[kAdamTensors];            // first block of the tensor in the flat state
  uint32_t tile_prefix[kAdamTensors + 1];
  uint32_t P;
  uint32_t key;                             // of (seed, step)
  AdamState in, out;
  const float* clip;                        // {norm, factor, all finite} or null
  float b1, c1, b2, c2, eps, keep, lr_t, inv_sqrt_bc2;  // keep = 1 - lr*wd, lr_t = lr / (1 - b1^t)
  float root_b2, root_c2;  // 8-bit moments: sqrt(b2), sqrt(c2) times 2^kAdamUp, with eps and lr_t times it too
};
constexpr int kAdamUp = 16;
uint32_t adam_tile_elems(mr_dtype dt, mr_dtype gdt, mr_state_format fmt, bool master);
hipError_t launch_adam(const AdamArgs& a, mr_dtype dt, mr_dtype gdt, mr_state_format fmt, hipStream_t st);

// ------------------------------------------------------------------------------------ losses on logits
struct LogitArgs {
  const char* z;        // logits, rows of `stride` elements
  char* dz;             // their gradient, rows of `dstride` elements; may be null, may be z
  size_t rows, cols, stride, dstride;
  const int64_t* targets;
  float c;              // log2(e) / temperature
  double inv_temp;
  float* logp;          // may be null
  float* stats;         // [rows][2]: the row's maximum and the sum of exp((z - maximum) / temperature); may be null
  const float* dlogp;   // backward pass: gradient of each row's log-probability
  // policy loss
  const float* old_logp;  // null: the log-probabilities themselves
  const float* ref_logp;  // null: no KL term
  const float* adv;
  const float* weights;   // null: ones
  double clip_lo, clip_hi, kl, grad_scale;
  float* record;
  // workspace
  float* part;            // [rows][splits][2]: maximum and sum of a part of a row
  uint32_t* row_arrived;  // [rows] parts that are done; zero between launches
  double* sums;           // [workgroups + kNormSets][4] parts of the policy loss's record
  uint32_t (*arrived)[64];
  uint32_t splits;        // parts of a row (set by the plan)
  uint32_t packs;         // 16-byte packs that cover a row wherever it starts (set by the launch)
};
// How a call over logits is launched: a function of its shape and alignment alone.
struct LogitPlan {
  int held;          // policy loss: rows in registers, one launch
  uint32_t splits;   // else: parts of a row in the statistics pass
  uint32_t groups;   // workgroups that add up the policy loss's record
};
LogitPlan plan_logits(const char* z, size_t rows, size_t cols, size_t stride, mr_dtype dt, bool gradient);
inline size_t record_bytes(uint32_t groups) { return (size_t{groups} + kNormSets) * 32; }
hipError_t launch_logprob(const LogitArgs& a, mr_dtype dt, hipStream_t st);
hipError_t launch_logprob_bwd(const LogitArgs& a, mr_dtype dt, hipStream_t st);
hipError_t launch_policy(const LogitArgs& a, const LogitPlan& pl, mr_dtype dt, hipStream_t st);

struct PreferenceArgs {
  const float* logp;
  const float* ref;        // may be null
  const int64_t* offsets;  // [2 * pairs + 1]
  size_t rows, pairs;
  double beta, smoothing, loss_scale, grad_scale;
  float* margins;  // may be null
  float* dlogp;    // may be null
  float* record;
  double* sums;    // [workgroups + kNormSets][4]
  uint32_t (*arrived)[64];
};
uint32_t preference_groups(size_t pairs);
hipError_t launch_preference(const PreferenceArgs& a, hipStream_t st);

// ------------------------------------------------------------------------------------------------ Muon
//
// A matrix of rows x cols is orthogonalised as X, m x n with m <= n: itself, or its transpose where rows > cols.  The
// stream's workspace holds, in fp16, in one or two pieces and in panels of kNsK of them, X [m][ldn], its transpose [n][ldm] twice (a
// product reads one and writes the other), A = X X^T and P = a I + b A + c A^2 [m][ldm]; ldm and ldn are m and n rounded up to
// three of a product's stages (ns_padded), and columns past m and n are zero.
constexpr int kMuonMats = 32;       // matrices of one launch
constexpr uint32_t kMuonCount = 32; // words from a matrix's arrival counter to the next one's
constexpr uint32_t kNsK = 32;       // columns that a product takes at a time: a stage
constexpr uint32_t kNsPad = 3 * kNsK;
__host__ __device__ inline uint32_t ns_padded(uint32_t n) { return (n + kNsPad - 1) / kNsPad * kNsPad; }
constexpr int kNsShift = 12;        // matrices are held times 2^12
inline uint32_t momentum_tile(uint64_t n) { return n < uint64_t{1} << 21 ? 4096 : 16384; }  // elements, of a matrix of n
inline uint32_t momentum_tiles(uint64_t n) { return static_cast<uint32_t>((n + momentum_tile(n) - 1) / momentum_tile(n)); }
struct MomentumArgs {
  const char* g[kMuonMats];
  uint64_t n[kMuonMats];
  uint64_t at[kMuonMats];  // first element in the flat state
  uint32_t tile[kMuonMats];  // elements of its tiles
  uint32_t tile_prefix[kMuonMats + 1];
  uint32_t P;
  const float* m;
  float* m_out;
  float* master_out;      // null: none (its elements between matrices become zeros)
  const float* clip;      // {norm, factor, all finite} or null
  double* sums;           // [tiles] sums of squares
  double* norms;          // [P] their sums
  uint32_t* arrived;      // [P][kMuonCount] zero between launches: a matrix's arrivals in a line of its own
  float mu, c;            // c = 1 - mu
  int nesterov;
};
struct OrientArgs {
  const char* g[kMuonMats];
  _Float16* direct[kMuonMats];  // rows x ld_direct: the matrix itself
  _Float16* turned[kMuonMats];  // cols x ld_turned: its transpose
  uint64_t at[kMuonMats];
  uint32_t rows[kMuonMats], cols[kMuonMats];
  uint32_t tile_prefix[kMuonMats + 1];
  uint32_t P;
  const float* m;  // the new momentum
  const float* clip;
  const double* norms;
  double eps;
  float mu, c;
  int nesterov, pieces;
};
// C = A B^T with A [M][K], B [N][K], and what becomes of it:
enum NsKind { kNsGram, kNsPoly, kNsStep };
struct NsProduct {
  const _Float16* a;
  const _Float16* b;
  _Float16* c;       // [M][ldc]; the last product: unused
  _Float16* ct;      // [N][ldct], the transpose (kNsStep)
  uint32_t M, N, K;    // K: padded
  uint32_t ldc, ldct;  // N and M padded: the tiles cover them
};
struct NsArgs {
  NsProduct p[kMuonMats];
  uint32_t tile_prefix[kMuonMats + 1];
  uint32_t P;
  int pieces;
  float ca, cb, cc;  // kNsPoly
};
struct NsUpdate {
  const char* p;   // parameters: null where a master copy is read
  char* po;
  uint64_t at;     // first element in the flat state
  float scale;     // lr times the matrix's factor
  uint32_t turned; // the product is the matrix's transpose
};
struct NsLastArgs {
  NsArgs s;
  NsUpdate u[kMuonMats];
  const float* master;
  float* master_out;
  const float* clip;
  float keep;
};
// Columns of a product's tiles for a matrix of m rows, in a list of so many tiles of 256 columns and of 128 if all that can take them do.
struct NsTiles {
  uint64_t wide, square;
};
constexpr uint32_t kNsWideFrom = 512, kNsSquareFrom = 256;  // rows
uint32_t ns_tile(uint32_t m, const NsTiles& list, int pieces);
uint32_t ns_tiles(uint32_t tile, uint32_t rows, uint32_t cols, bool symmetric);
hipError_t launch_momentum(const MomentumArgs& a, mr_dtype gdt, hipStream_t st);
hipError_t launch_orient(const OrientArgs& a, mr_dtype gdt, hipStream_t st);
hipError_t launch_ns(const NsArgs& a, NsKind kind, uint32_t tile, hipStream_t st);
hipError_t launch_ns_last(const NsLastArgs& a, mr_dtype dt, uint32_t tile, hipStream_t st);

// Helpers of api.hip.  stream_workspace: the stream's library workspace (or the one of the capture under way), with room
// for `bytes`: its Ctrl words and its data area.  Earlier work on the stream has finished with both when a later launch
// runs, and no other thread's call uses them between this call's launches while `use` is held.
bool trace_on();  // MR_TRACE=1
mr_status stream_workspace(hipStream_t st, size_t bytes, Ctrl** ctrl, char** data, std::unique_lock<std::mutex>* use);

}  // namespace mr
