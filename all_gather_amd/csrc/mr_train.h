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

// Helpers of api.hip.  stream_workspace: the stream's library workspace (or the one of the capture under way), with room
// for `bytes`: its Ctrl words and its data area.  Earlier work on the stream has finished with both when a later launch
// runs, and no other thread's call uses them between this call's launches while `use` is held.
bool trace_on();  // MR_TRACE=1
mr_status stream_workspace(hipStream_t st, size_t bytes, Ctrl** ctrl, char** data, std::unique_lock<std::mutex>* use);

}  // namespace mr
