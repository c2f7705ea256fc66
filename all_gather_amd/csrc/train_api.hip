// C ABI of the training-step operators (include/mr.h): argument checks, launch tables, launches.

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <new>
#include <vector>

#include "mr_train.h"

namespace {

mr_status hip_fail(hipError_t e) {
  mr::set_last_hip_error(static_cast<int>(e));
  return MR_ERR_HIP;
}

bool is_float(mr_dtype d) { return d == MR_BF16 || d == MR_FP16 || d == MR_FP32; }
bool valid_dtype(mr_dtype d) { return d >= MR_BF16 && d <= MR_INT32; }

// dtype and a second type that is the same or fp32 (weights, gradients).
mr_status check_types(mr_dtype dt, mr_dtype second) {
  if (!valid_dtype(dt) || !valid_dtype(second)) return MR_ERR_INVALID_ARG;
  if (!is_float(dt) || (second != dt && second != MR_FP32)) return MR_ERR_DTYPE;
  return MR_OK;
}

bool on_grid(const void* p, size_t es) { return reinterpret_cast<uintptr_t>(p) % es == 0; }

// A buffer of a call.  Outputs may share memory with nothing but the inputs they are allowed to replace, and
// those exactly.
struct Span {
  uintptr_t lo, hi;
  int id;
};
Span span(const void* p, size_t bytes, int id) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{a, a + bytes, id};
}

// Outputs, sorted by address; ok() is false once two of them overlap.
class Outputs {
 public:
  explicit Outputs(std::vector<Span>* v) : v_(v) { v_->clear(); }
  void add(const void* p, size_t bytes, int id) {
    if (p && bytes) v_->push_back(span(p, bytes, id));
  }
  bool ok() {
    auto less = [](const Span& a, const Span& b) { return a.lo < b.lo; };
    if (!std::is_sorted(v_->begin(), v_->end(), less)) std::sort(v_->begin(), v_->end(), less);
    for (size_t i = 1; i < v_->size(); ++i)
      if ((*v_)[i].lo < (*v_)[i - 1].hi) return false;
    return true;
  }
  // May an input lie at [p, p + bytes)?  Only clear of every output, or exactly at an output that `same` allows.
  template <class Same>
  bool admits(const void* p, size_t bytes, Same same) const {
    if (!p || !bytes) return true;
    const Span s = span(p, bytes, 0);
    auto it = std::upper_bound(v_->begin(), v_->end(), s.lo, [](uintptr_t x, const Span& o) { return x < o.hi; });
    for (; it != v_->end() && it->lo < s.hi; ++it)
      if (it->lo != s.lo || it->hi != s.hi || !same(it->id)) return false;
    return true;
  }
  bool admits(const void* p, size_t bytes) const {
    return admits(p, bytes, [](int) { return false; });
  }

 private:
  std::vector<Span>* v_;
};

thread_local std::vector<Span> t_spans;

// An allocation failure inside the library is reported, never thrown through the C boundary.
template <class F>
mr_status guarded(F f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return hip_fail(hipErrorOutOfMemory);
  } catch (...) {
    return hip_fail(hipErrorUnknown);
  }
}

mr_status check_norm(size_t rows, size_t cols, mr_dtype dtype, mr_dtype wdtype) {
  const mr_status s = check_types(dtype, wdtype);
  if (s != MR_OK) return s;
  if (cols > 0x7fffffffu || rows > (size_t{1} << 56)) return MR_ERR_INVALID_ARG;
  if (cols && rows > (size_t{1} << 56) / cols) return MR_ERR_INVALID_ARG;
  return MR_OK;
}

mr_status layer_norm_forward(const void* const* bufs, int W, const void* residual, const void* gamma, const void* beta,
                             size_t rows, size_t cols, mr_dtype dtype, mr_dtype wdtype, double eps, void* x_out, void* y,
                             float* mean, float* rstd, hipStream_t st) {
  const float eps32 = static_cast<float>(eps);
  if (W < 1 || W > MR_MAX_W || !(eps >= 0.0) || !std::isfinite(eps32) || (eps > 0.0 && eps32 == 0.0f)) return MR_ERR_INVALID_ARG;
  const mr_status s = check_norm(rows, cols, dtype, wdtype);
  if (s != MR_OK) return s;
  if (rows == 0 || cols == 0) return MR_OK;
  if (!bufs || !y) return MR_ERR_INVALID_ARG;
  const size_t es = mr::elem_size(dtype), ws = mr::elem_size(wdtype), bytes = rows * cols * es;
  if (!on_grid(residual, es) || !on_grid(x_out, es) || !on_grid(y, es) || !on_grid(gamma, ws) || !on_grid(beta, ws) ||
      !on_grid(mean, 4) || !on_grid(rstd, 4))
    return MR_ERR_INVALID_ARG;
  mr::NormFwdArgs a{};
  for (int r = 0; r < W; ++r) {
    if (!bufs[r] || !on_grid(bufs[r], es)) return MR_ERR_INVALID_ARG;
    a.in[r] = static_cast<const char*>(bufs[r]);
  }
  Outputs outs(&t_spans);
  outs.add(y, bytes, 1);
  outs.add(x_out, bytes, 1);
  outs.add(mean, rows * 4, 0);
  outs.add(rstd, rows * 4, 0);
  auto in_place = [](int id) { return id == 1; };
  if (!outs.ok() || !outs.admits(residual, bytes, in_place) || !outs.admits(gamma, cols * ws) || !outs.admits(beta, cols * ws))
    return MR_ERR_ALIAS;
  for (int r = 0; r < W; ++r)
    if (!outs.admits(bufs[r], bytes, in_place)) return MR_ERR_ALIAS;
  a.terms = W;
  if (residual) a.in[a.terms++] = static_cast<const char*>(residual);
  a.gamma = static_cast<const char*>(gamma);
  a.beta = static_cast<const char*>(beta);
  a.x_out = static_cast<char*>(x_out);
  a.y = static_cast<char*>(y);
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.cols = cols;
  a.eps = eps32;
  if (mr::trace_on())
    std::fprintf(stderr, "[mr] layer_norm forward W=%d rows=%zu cols=%zu dtype=%d\n", W, rows, cols, static_cast<int>(dtype));
  const hipError_t e = mr::launch_norm_fwd(a, dtype, wdtype, st);
  return e == hipSuccess ? MR_OK : hip_fail(e);
}

mr_status layer_norm_backward(const void* dy, const void* x, const void* gamma, const float* mean, const float* rstd,
                              const void* dres, size_t rows, size_t cols, mr_dtype dtype, mr_dtype wdtype, void* dx,
                              void* dgamma, void* dbeta, hipStream_t st) {
  mr_status s = check_norm(rows, cols, dtype, wdtype);
  if (s != MR_OK) return s;
  if (cols == 0 || (!dx && !dgamma && !dbeta) || (rows == 0 && !dgamma && !dbeta)) return MR_OK;
  if (rows && (!dy || !x || !mean || !rstd)) return MR_ERR_INVALID_ARG;
  const size_t es = mr::elem_size(dtype), ws = mr::elem_size(wdtype), bytes = rows * cols * es;
  if (!on_grid(dy, es) || !on_grid(x, es) || !on_grid(dres, es) || !on_grid(dx, es) || !on_grid(gamma, ws) ||
      !on_grid(dgamma, ws) || !on_grid(dbeta, ws) || !on_grid(mean, 4) || !on_grid(rstd, 4))
    return MR_ERR_INVALID_ARG;
  Outputs outs(&t_spans);
  outs.add(dx, bytes, 1);
  outs.add(dgamma, cols * ws, 0);
  outs.add(dbeta, cols * ws, 0);
  auto in_place = [](int id) { return id == 1; };
  if (!outs.ok() || !outs.admits(dy, bytes, in_place) || !outs.admits(x, bytes, in_place) ||
      !outs.admits(dres, bytes, in_place) || !outs.admits(gamma, cols * ws) || !outs.admits(mean, rows * 4) ||
      !outs.admits(rstd, rows * 4))
    return MR_ERR_ALIAS;
  mr::NormBwdArgs a{};
  a.dy = static_cast<const char*>(dy);
  a.x = static_cast<const char*>(x);
  a.gamma = static_cast<const char*>(gamma);
  a.mean = mean;
  a.rstd = rstd;
  a.dres = static_cast<const char*>(dres);
  a.dx = static_cast<char*>(dx);
  a.dgamma = static_cast<char*>(dgamma);
  a.dbeta = static_cast<char*>(dbeta);
  a.rows = rows;
  a.cols = cols;
  a.groups = mr::norm_bwd_groups(rows, cols, dtype);
  std::unique_lock<std::mutex> use;  // to the last launch
  if (dgamma || dbeta) {
    mr::Ctrl* ctrl = nullptr;
    char* data = nullptr;
    s = mr::stream_workspace(st, size_t{a.groups} * 2 * cols * 4, &ctrl, &data, &use);
    if (s != MR_OK) return s;
    a.part = reinterpret_cast<float*>(data);
    a.arrived = &ctrl->arrived[0][0];
  }
  if (mr::trace_on())
    std::fprintf(stderr, "[mr] layer_norm backward rows=%zu cols=%zu dtype=%d groups=%u\n", rows, cols,
                 static_cast<int>(dtype), a.groups);
  const hipError_t e = mr::launch_norm_bwd(a, dtype, wdtype, st);
  return e == hipSuccess ? MR_OK : hip_fail(e);
}

constexpr double kLog2E = 1.4426950408889634;
constexpr uint64_t kMaxCount = uint64_t{1} << 33;  // elements of one tensor
constexpr double kLeastEps = 0x1p-126;             // fp32's smallest normal number: the reciprocal takes smaller ones as zero
constexpr uint32_t kMaxTiles = 1u << 23;           // tiles of one launch (256 lanes each, below 2^32 lanes)

mr_status grad_norm(const void* const* grads, const uint64_t* counts, int P, mr_dtype dtype, double scale, double max_norm,
                    float* out, hipStream_t st) {
  if (P < 0 || !valid_dtype(dtype) || !(scale > 0.0) || !std::isfinite(scale) || !std::isfinite(max_norm))
    return MR_ERR_INVALID_ARG;
  if (!is_float(dtype)) return MR_ERR_DTYPE;
  if ((P && (!grads || !counts)) || !out || !on_grid(out, 4)) return MR_ERR_INVALID_ARG;
  const size_t es = mr::elem_size(dtype);
  for (int i = 0; i < P; ++i) {
    if (counts[i] == 0) continue;
    if (counts[i] > kMaxCount || !grads[i] || !on_grid(grads[i], es)) return MR_ERR_INVALID_ARG;
    const Span g = span(grads[i], counts[i] * es, 0), o = span(out, 12, 0);
    if (g.lo < o.hi && o.lo < g.hi) return MR_ERR_ALIAS;
  }
  // the launches' tables: tensors in order, none empty
  std::vector<mr::GradNormArgs> launches;
  uint64_t groups = 0;
  mr::GradNormArgs a;
  auto reset = [&] {
    std::memset(&a, 0, sizeof(a));
    a.scale = scale;
    a.max_norm = max_norm;
    a.out = out;
  };
  auto emit = [&] {
    a.part_base = static_cast<uint32_t>(groups);
    groups += mr::grad_norm_groups(a.tile_prefix[a.P]);
    launches.push_back(a);
    reset();
  };
  reset();
  for (int i = 0; i < P; ++i) {
    if (counts[i] == 0) continue;
    const uint32_t tiles = static_cast<uint32_t>((counts[i] * es + mr::kNormTileBytes - 1) / mr::kNormTileBytes);
    a.g[a.P] = static_cast<const char*>(grads[i]);
    a.n[a.P] = counts[i];
    a.tile_prefix[a.P + 1] = a.tile_prefix[a.P] + tiles;
    if (++a.P == mr::kNormTensors || a.tile_prefix[a.P] >= kMaxTiles) emit();
  }
  if (a.P || launches.empty()) emit();
  mr::Ctrl* ctrl = nullptr;
  char* data = nullptr;
  std::unique_lock<std::mutex> use;  // to the last launch
  const mr_status s = mr::stream_workspace(st, groups * sizeof(double), &ctrl, &data, &use);
  if (s != MR_OK) return s;
  for (size_t k = 0; k < launches.size(); ++k) {
    mr::GradNormArgs& l = launches[k];
    l.part = reinterpret_cast<double*>(data);
    l.arrived = ctrl->arrived;
    l.finish = k + 1 == launches.size();
    if (mr::trace_on())
      std::fprintf(stderr, "[mr] grad_norm tensors=%u tiles=%u dtype=%d\n", l.P, l.tile_prefix[l.P], static_cast<int>(dtype));
    const hipError_t e = mr::launch_grad_norm(l, dtype, st);
    if (e != hipSuccess) return hip_fail(e);
  }
  return MR_OK;
}

mr_status state_elems(const uint64_t* counts, int P, uint64_t* elems) {
  if (P < 0 || (P && !counts) || !elems) return MR_ERR_INVALID_ARG;
  uint64_t n = 0;
  for (int i = 0; i < P; ++i) {
    if (counts[i] > kMaxCount) return MR_ERR_INVALID_ARG;
    n += (counts[i] + mr::kMxBlock - 1) / mr::kMxBlock * mr::kMxBlock;
    if (n >= uint64_t{mr::kMxBlock} << 32) return MR_ERR_INVALID_ARG;
  }
  *elems = n;
  return MR_OK;
}

// 32 bits that stand for (seed, step): the 64-bit finaliser of a Weyl sequence generator (Steele, Lea and Flood,
// "Fast splittable pseudorandom number generators", 2014).
uint32_t random_key(uint64_t seed, uint64_t step) {
  uint64_t z = seed + 0x9E3779B97F4A7C15ull * step;
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return static_cast<uint32_t>(z ^ (z >> 31));
}

mr_status adamw_step(const void* const* params, const void* const* grads, const uint64_t* counts, int P, mr_dtype dtype,
                     mr_dtype gdtype, mr_state_format fmt, const mr_adamw_state* in, void* const* params_out,
                     const mr_adamw_state* out, const mr_adamw_hyper* h, const float* clip, hipStream_t st) {
  mr_status s = check_types(dtype, gdtype);
  if (s != MR_OK) return s;
  if (P < 0 || (fmt != MR_STATE_FP32 && fmt != MR_STATE_MXFP8) || !h) return MR_ERR_INVALID_ARG;
  if (!std::isfinite(h->lr) || !std::isfinite(h->weight_decay) || !(h->beta1 >= 0.0 && h->beta1 < 1.0) ||
      !(h->beta2 >= 0.0 && h->beta2 < 1.0) || !(h->eps == 0.0 || h->eps >= kLeastEps) || !std::isfinite(h->eps) || h->step < 1)
    return MR_ERR_INVALID_ARG;
  uint64_t total = 0;
  s = state_elems(counts, P, &total);
  if (s != MR_OK) return s;
  if (total == 0) return MR_OK;
  if (!in || !grads) return MR_ERR_INVALID_ARG;
  const bool mx = fmt == MR_STATE_MXFP8, master = in->master != nullptr;
  if (master && dtype == MR_FP32) return MR_ERR_DTYPE;
  if (!out) out = in;
  if ((!params && !(master && params_out)) || (master != (out->master != nullptr))) return MR_ERR_INVALID_ARG;
  const size_t es = mr::elem_size(dtype), gs = mr::elem_size(gdtype), ms = mx ? 1 : 4;
  for (const mr_adamw_state* q : {in, out}) {
    if (!q->m || !q->v || !on_grid(q->m, 256) || !on_grid(q->v, 256) || !on_grid(q->master, 256)) return MR_ERR_INVALID_ARG;
    if (mx != (q->m_scale != nullptr) || mx != (q->v_scale != nullptr)) return MR_ERR_INVALID_ARG;
  }
  if (!on_grid(clip, 4)) return MR_ERR_INVALID_ARG;
  auto param_in = [&](int i) { return params ? params[i] : nullptr; };
  auto param_out = [&](int i) { return params_out ? params_out[i] : const_cast<void*>(params[i]); };
  for (int i = 0; i < P; ++i) {
    if (counts[i] == 0) continue;
    if (!grads[i] || !on_grid(grads[i], gs) || !param_out(i) || !on_grid(param_out(i), es)) return MR_ERR_INVALID_ARG;
    if (!master && (!param_in(i) || !on_grid(param_in(i), es))) return MR_ERR_INVALID_ARG;
  }
  const size_t blocks = total / mr::kMxBlock;
  Outputs outs(&t_spans);
  for (int i = 0; i < P; ++i) outs.add(param_out(i), counts[i] * es, i);
  outs.add(out->m, total * ms, -1);
  outs.add(out->v, total * ms, -2);
  outs.add(out->m_scale, blocks, -3);
  outs.add(out->v_scale, blocks, -4);
  outs.add(out->master, total * 4, -5);
  if (!outs.ok()) return MR_ERR_ALIAS;
  auto only = [](int id) { return [id](int o) { return o == id; }; };
  bool fine = outs.admits(in->m, total * ms, only(-1)) && outs.admits(in->v, total * ms, only(-2)) &&
              outs.admits(in->m_scale, blocks, only(-3)) && outs.admits(in->v_scale, blocks, only(-4)) &&
              outs.admits(in->master, total * 4, only(-5)) && outs.admits(clip, 12);
  for (int i = 0; fine && i < P; ++i)
    fine = outs.admits(grads[i], counts[i] * gs) && (master || outs.admits(param_in(i), counts[i] * es, only(i)));
  if (!fine) return MR_ERR_ALIAS;

  mr::AdamArgs a;
  std::memset(&a, 0, sizeof(a));
  auto state = [](const mr_adamw_state& q) {
    return mr::AdamState{static_cast<char*>(q.m), static_cast<char*>(q.v), q.m_scale, q.v_scale, q.master};
  };
  a.in = state(*in);
  a.out = state(*out);
  a.clip = clip;
  a.key = random_key(h->seed, h->step);
  a.b1 = static_cast<float>(h->beta1);
  a.c1 = static_cast<float>(1.0 - h->beta1);
  a.b2 = static_cast<float>(h->beta2);
  a.c2 = static_cast<float>(1.0 - h->beta2);
  const double up = mx ? std::ldexp(1.0, mr::kAdamUp) : 1.0;
  a.eps = static_cast<float>(h->eps * up);
  a.keep = static_cast<float>(1.0 - h->lr * h->weight_decay);
  a.lr_t = static_cast<float>(h->lr / (1.0 - std::pow(h->beta1, static_cast<double>(h->step))) * up);
  a.inv_sqrt_bc2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(h->beta2, static_cast<double>(h->step))));
  a.root_b2 = static_cast<float>(std::sqrt(h->beta2) * up);
  a.root_c2 = static_cast<float>(std::sqrt(1.0 - h->beta2) * up);
  const uint32_t tile = mr::adam_tile_elems(dtype, gdtype, fmt, master);
  uint64_t block = 0;
  hipError_t e = hipSuccess;
  for (int i = 0; i < P && e == hipSuccess; ++i) {
    if (counts[i]) {
      const uint32_t k = a.P++;
      a.p[k] = static_cast<const char*>(master ? param_in(i) : params[i]);
      a.g[k] = static_cast<const char*>(grads[i]);
      a.po[k] = static_cast<char*>(param_out(i));
      a.n[k] = counts[i];
      a.block0[k] = static_cast<uint32_t>(block);
      const uint64_t padded = (counts[i] + mr::kMxBlock - 1) / mr::kMxBlock * mr::kMxBlock;
      a.tile_prefix[k + 1] = a.tile_prefix[k] + static_cast<uint32_t>((padded + tile - 1) / tile);
      block += padded / mr::kMxBlock;
    }
    if (a.P && (a.P == mr::kAdamTensors || a.tile_prefix[a.P] >= kMaxTiles || i + 1 == P)) {
      if (mr::trace_on())
        std::fprintf(stderr, "[mr] adamw tensors=%u tiles=%u dtype=%d grad=%d format=%d master=%d\n", a.P, a.tile_prefix[a.P],
                     static_cast<int>(dtype), static_cast<int>(gdtype), static_cast<int>(fmt), master ? 1 : 0);
      e = mr::launch_adam(a, dtype, gdtype, fmt, st);
      a.P = 0;
    }
  }
  return e == hipSuccess ? MR_OK : hip_fail(e);
}

// Rows of a call over logits: `stride` elements apart, `cols` of them used.
mr_status check_logits(size_t rows, size_t cols, size_t stride, mr_dtype dtype, double temperature) {
  if (!valid_dtype(dtype)) return MR_ERR_INVALID_ARG;
  if (!is_float(dtype)) return MR_ERR_DTYPE;
  if (cols > 0x7fffffffu || rows > (size_t{1} << 40) || stride > (size_t{1} << 40) || (rows > 1 && stride < cols)) return MR_ERR_INVALID_ARG;
  if (rows && stride > (size_t{1} << 56) / rows) return MR_ERR_INVALID_ARG;
  const float c = static_cast<float>(kLog2E / temperature);
  if (!(temperature > 0.0) || !std::isfinite(temperature) || !std::isfinite(c) || c < 0x1p-126f) return MR_ERR_INVALID_ARG;
  return MR_OK;
}
// Bytes that a call touches from the first element of the first row to the last of the last.
size_t extent(size_t rows, size_t cols, size_t stride, size_t es) { return rows && cols ? ((rows - 1) * stride + cols) * es : 0; }

mr::LogitArgs logit_args(const void* logits, size_t rows, size_t cols, size_t stride, const int64_t* targets, double temperature) {
  mr::LogitArgs a{};
  a.z = static_cast<const char*>(logits);
  a.rows = rows;
  a.cols = cols;
  a.stride = stride;
  a.targets = targets;
  a.c = static_cast<float>(kLog2E / temperature);
  a.inv_temp = 1.0 / temperature;
  a.splits = 1;
  return a;
}

// Arrival counters of `n` rows in the stream's workspace: the words after its control words, zero between calls.
size_t row_words_bytes(size_t n) { return n << 8; }
uint32_t* row_words(mr::Ctrl* ctrl) { return reinterpret_cast<uint32_t*>(reinterpret_cast<char*>(ctrl) + mr::kCtrlBytes); }

mr_status token_logprob_forward(const void* logits, size_t rows, size_t cols, size_t stride, mr_dtype dtype, const int64_t* targets,
                                double temperature, float* logp, float* stats, hipStream_t st) {
  mr_status s = check_logits(rows, cols, stride, dtype, temperature);
  if (s != MR_OK) return s;
  if (rows == 0 || (!logp && !stats)) return MR_OK;
  if ((!logits && cols) || !targets) return MR_ERR_INVALID_ARG;
  const size_t es = mr::elem_size(dtype), in = extent(rows, cols, stride, es);
  if (!on_grid(logits, es) || !on_grid(targets, 8) || !on_grid(logp, 4) || !on_grid(stats, 4)) return MR_ERR_INVALID_ARG;
  Outputs outs(&t_spans);
  outs.add(logp, rows * 4, 0);
  outs.add(stats, rows * 8, 0);
  if (!outs.ok() || !outs.admits(logits, in) || !outs.admits(targets, rows * 8)) return MR_ERR_ALIAS;
  mr::LogitArgs a = logit_args(logits, rows, cols, stride, targets, temperature);
  a.logp = logp;
  a.stats = stats;
  a.splits = mr::plan_logits(a.z, rows, cols, stride, dtype, false).splits;
  std::unique_lock<std::mutex> use;  // to the last launch
  if (a.splits > 1) {
    mr::Ctrl* ctrl = nullptr;
    char* data = nullptr;
    s = mr::stream_workspace(st, std::max(rows * a.splits * 8, row_words_bytes(rows)), &ctrl, &data, &use);
    if (s != MR_OK) return s;
    a.part = reinterpret_cast<float*>(data);
    a.row_arrived = row_words(ctrl);
  }
  if (mr::trace_on())
    std::fprintf(stderr, "[mr] token_logprob forward rows=%zu cols=%zu dtype=%d splits=%u\n", rows, cols, static_cast<int>(dtype), a.splits);
  const hipError_t e = mr::launch_logprob(a, dtype, st);
  return e == hipSuccess ? MR_OK : hip_fail(e);
}

mr_status token_logprob_backward(const void* logits, size_t rows, size_t cols, size_t stride, mr_dtype dtype, const int64_t* targets,
                                 double temperature, const float* stats, const float* dlogp, void* dlogits, size_t dstride,
                                 hipStream_t st) {
  mr_status s = check_logits(rows, cols, stride, dtype, temperature);
  if (s == MR_OK) s = check_logits(rows, cols, dstride, dtype, temperature);
  if (s != MR_OK) return s;
  if (rows == 0 || cols == 0) return MR_OK;
  if (!logits || !targets || !stats || !dlogp || !dlogits) return MR_ERR_INVALID_ARG;
  const size_t es = mr::elem_size(dtype), in = extent(rows, cols, stride, es), out = extent(rows, cols, dstride, es);
  if (!on_grid(logits, es) || !on_grid(dlogits, es) || !on_grid(targets, 8) || !on_grid(stats, 4) || !on_grid(dlogp, 4))
    return MR_ERR_INVALID_ARG;
  Outputs outs(&t_spans);
  outs.add(dlogits, out, 1);
  if (!outs.admits(logits, in, [](int id) { return id == 1; }) || !outs.admits(targets, rows * 8) || !outs.admits(stats, rows * 8) ||
      !outs.admits(dlogp, rows * 4))
    return MR_ERR_ALIAS;
  mr::LogitArgs a = logit_args(logits, rows, cols, stride, targets, temperature);
  a.stats = const_cast<float*>(stats);
  a.dlogp = dlogp;
  a.dz = static_cast<char*>(dlogits);
  a.dstride = dstride;
  if (mr::trace_on())
    std::fprintf(stderr, "[mr] token_logprob backward rows=%zu cols=%zu dtype=%d\n", rows, cols, static_cast<int>(dtype));
  const hipError_t e = mr::launch_logprob_bwd(a, dtype, st);
  return e == hipSuccess ? MR_OK : hip_fail(e);
}

mr_status policy_loss(const void* logits, size_t rows, size_t cols, size_t stride, mr_dtype dtype, const int64_t* targets,
                      const float* old_logp, const float* ref_logp, const float* advantages, const float* weights,
                      const mr_policy_hyper* h, float* record, float* logp, void* dlogits, size_t dstride, hipStream_t st) {
  if (!h) return MR_ERR_INVALID_ARG;
  mr_status s = check_logits(rows, cols, stride, dtype, h->temperature);
  if (s == MR_OK && dlogits) s = check_logits(rows, cols, dstride, dtype, h->temperature);
  if (s != MR_OK) return s;
  if (!(h->clip_low >= 0.0 && h->clip_low <= 1.0) || !(h->clip_high >= 0.0) || !std::isfinite(h->clip_high) || !std::isfinite(h->kl_coef) ||
      !(h->grad_scale > 0.0) || !std::isfinite(h->grad_scale) || (h->kl_coef != 0.0 && !ref_logp))
    return MR_ERR_INVALID_ARG;
  if (!record || !on_grid(record, 4) || (rows && ((!logits && cols) || !targets || !advantages))) return MR_ERR_INVALID_ARG;
  const size_t es = mr::elem_size(dtype), in = extent(rows, cols, stride, es), out = extent(rows, cols, dstride, es);
  if (!on_grid(logits, es) || !on_grid(dlogits, es) || !on_grid(targets, 8) || !on_grid(old_logp, 4) || !on_grid(ref_logp, 4) ||
      !on_grid(advantages, 4) || !on_grid(weights, 4) || !on_grid(logp, 4))
    return MR_ERR_INVALID_ARG;
  Outputs outs(&t_spans);
  outs.add(dlogits, out, 1);
  outs.add(record, 16, 0);
  outs.add(logp, rows * 4, 0);
  if (!outs.ok() || !outs.admits(logits, in, [](int id) { return id == 1; }) || !outs.admits(targets, rows * 8)) return MR_ERR_ALIAS;
  for (const float* p : {old_logp, ref_logp, advantages, weights})
    if (!outs.admits(p, rows * 4)) return MR_ERR_ALIAS;
  mr::LogitArgs a = logit_args(logits, rows, cols, stride, targets, h->temperature);
  a.old_logp = old_logp;
  a.ref_logp = ref_logp;
  a.adv = advantages;
  a.weights = weights;
  a.clip_lo = h->clip_low;
  a.clip_hi = h->clip_high;
  a.kl = h->kl_coef;
  a.grad_scale = h->grad_scale;
  a.record = record;
  a.logp = logp;
  a.dz = rows && cols ? static_cast<char*>(dlogits) : nullptr;
  a.dstride = dstride;
  const mr::LogitPlan pl = mr::plan_logits(a.z, rows, cols, stride, dtype, a.dz != nullptr);
  a.splits = pl.splits;
  // the workspace: workgroups' sums, then (on the path of two passes) rows' statistics, gradients and parts
  const size_t sums = mr::record_bytes(pl.groups), two = pl.held ? 0 : rows * 12 + rows * (pl.splits > 1 ? pl.splits * 8 : 0);
  mr::Ctrl* ctrl = nullptr;
  char* data = nullptr;
  std::unique_lock<std::mutex> use;  // to the last launch
  s = mr::stream_workspace(st, std::max(sums + two, pl.splits > 1 ? row_words_bytes(rows) : 0), &ctrl, &data, &use);
  if (s != MR_OK) return s;
  a.sums = reinterpret_cast<double*>(data);
  a.arrived = ctrl->arrived;
  if (!pl.held) {
    a.stats = reinterpret_cast<float*>(data + sums);
    a.dlogp = a.stats + 2 * rows;
    a.part = a.stats + 3 * rows;
    a.row_arrived = row_words(ctrl);
  }
  if (mr::trace_on())
    std::fprintf(stderr, "[mr] policy_loss rows=%zu cols=%zu dtype=%d held=%d splits=%u groups=%u\n", rows, cols, static_cast<int>(dtype),
                 pl.held, pl.splits, pl.groups);
  const hipError_t e = mr::launch_policy(a, pl, dtype, st);
  return e == hipSuccess ? MR_OK : hip_fail(e);
}

mr_status preference_loss(const float* logp, const float* ref_logp, size_t rows, const int64_t* offsets, size_t pairs,
                          const mr_preference_hyper* h, float* record, float* margins, float* dlogp, hipStream_t st) {
  if (!h || !std::isfinite(h->beta) || !(h->smoothing >= 0.0 && h->smoothing <= 0.5) || !std::isfinite(h->loss_scale) ||
      !(h->grad_scale > 0.0) || !std::isfinite(h->grad_scale))
    return MR_ERR_INVALID_ARG;
  if (rows > (size_t{1} << 40) || pairs > (size_t{1} << 40) || !record || !offsets || (rows && !logp)) return MR_ERR_INVALID_ARG;
  if (!on_grid(logp, 4) || !on_grid(ref_logp, 4) || !on_grid(offsets, 8) || !on_grid(record, 4) || !on_grid(margins, 4) || !on_grid(dlogp, 4))
    return MR_ERR_INVALID_ARG;
  Outputs outs(&t_spans);
  outs.add(record, 12, 0);
  outs.add(margins, pairs * 4, 0);
  outs.add(dlogp, rows * 4, 1);
  if (!outs.ok() || !outs.admits(logp, rows * 4, [](int id) { return id == 1; }) || !outs.admits(ref_logp, rows * 4) ||
      !outs.admits(offsets, (2 * pairs + 1) * 8))
    return MR_ERR_ALIAS;
  mr::PreferenceArgs a{logp, ref_logp, offsets, rows, pairs, h->beta, h->smoothing, h->loss_scale, h->grad_scale, margins, dlogp, record, nullptr, nullptr};
  mr::Ctrl* ctrl = nullptr;
  char* data = nullptr;
  std::unique_lock<std::mutex> use;  // to the last launch
  const mr_status s = mr::stream_workspace(st, mr::record_bytes(mr::preference_groups(pairs)), &ctrl, &data, &use);
  if (s != MR_OK) return s;
  a.sums = reinterpret_cast<double*>(data);
  a.arrived = ctrl->arrived;
  if (mr::trace_on()) std::fprintf(stderr, "[mr] preference_loss rows=%zu pairs=%zu\n", rows, pairs);
  const hipError_t e = mr::launch_preference(a, st);
  return e == hipSuccess ? MR_OK : hip_fail(e);
}

// Do the polynomials keep X, A = X X^T and P = a I + b A + c A^2 where fp16 times 2^12 holds them?  R bounds X's singular values:
// 1 at the start, where the Frobenius norm is; with some room for the roundings.
bool polynomials_fit(const double* coef, int steps) {
  double R = 1.0;
  const auto at = [](const double* k, double l) { return k[0] + l * (k[1] + l * k[2]); };
  for (int i = 0; i < steps; ++i, coef += 3) {
    for (int j = 0; j < 3; ++j)
      if (!std::isfinite(coef[j])) return false;
    R *= 1.01;
    const double L = R * R;
    // P's eigenvalues are largest at an end of [0, L] or where the derivative in l = s^2 is zero, X's singular values s P(s^2) likewise
    double p = std::max(std::fabs(at(coef, 0.0)), std::fabs(at(coef, L)));
    if (coef[2] != 0.0) {
      const double l = -coef[1] / (2.0 * coef[2]);
      if (l > 0.0 && l < L) p = std::max(p, std::fabs(at(coef, l)));
    }
    double x = R * std::fabs(at(coef, L));
    const double qa = 5.0 * coef[2], qb = 3.0 * coef[1], qc = coef[0], d = qb * qb - 4.0 * qa * qc;
    const double roots[3] = {qa != 0.0 && d >= 0.0 ? (-qb + std::sqrt(d)) / (2.0 * qa) : -1.0,
                             qa != 0.0 && d >= 0.0 ? (-qb - std::sqrt(d)) / (2.0 * qa) : -1.0, qa == 0.0 && qb != 0.0 ? -qc / qb : -1.0};
    for (double l : roots)
      if (l > 0.0 && l < L) x = std::max(x, std::sqrt(l) * std::fabs(at(coef, l)));
    if (L > 15.0 || p > 15.0 || x > 3.8) return false;
    R = x;
  }
  return true;
}

constexpr double kLeastNorm = 0x1p-114;           // 2^12 over it is an fp32 number
constexpr double kNsCoef[3] = {3.4445, -4.775, 2.0315};
constexpr int kNsMostSteps = 16;
constexpr uint64_t kMostSide = 1 << 16;           // rows or columns of a matrix
constexpr uint64_t kMuonGroupBytes = uint64_t{2} << 30;  // workspace from which a list is worked off in parts

// A matrix's part of the workspace: elements of fp16.
struct MuonShape {
  uint32_t m, n, ldm, ldn;
  bool turned;
  uint64_t halves;  // of X, X^T twice, A and P
};
MuonShape muon_shape(uint64_t rows, uint64_t cols, int pieces) {
  MuonShape s;
  s.turned = rows > cols;
  s.m = static_cast<uint32_t>(s.turned ? cols : rows);
  s.n = static_cast<uint32_t>(s.turned ? rows : cols);
  s.ldm = mr::ns_padded(s.m);
  s.ldn = mr::ns_padded(s.n);
  s.halves = pieces * (uint64_t{s.m} * s.ldn + 2 * (uint64_t{s.n} * s.ldm) + 2 * (uint64_t{s.m} * s.ldm));
  return s;
}

// Matrices of one workspace: those from `first` on that fit together, and the bytes they take.
struct MuonGroup {
  int first, end, count;  // count: those that are not empty
  uint64_t bytes;         // of halves, then sums, then norms
  uint64_t sums;
};
MuonGroup muon_group(const uint64_t* rows, const uint64_t* cols, int P, int first, int pieces) {
  MuonGroup g{first, first, 0, 0, 0};
  uint64_t halves = 0;
  for (; g.end < P && g.count < mr::kMuonMats; ++g.end) {
    if (rows[g.end] * cols[g.end] == 0) continue;
    const uint64_t more = muon_shape(rows[g.end], cols[g.end], pieces).halves;
    if (g.count && (halves + more) * 2 > kMuonGroupBytes) break;
    halves += more;
    g.sums += mr::momentum_tiles(rows[g.end] * cols[g.end]);
    ++g.count;
  }
  g.bytes = halves * 2 + g.sums * 8 + mr::kMuonMats * 8;
  return g;
}

mr_status check_matrices(const uint64_t* rows, const uint64_t* cols, int P) {
  if (P < 0 || (P && (!rows || !cols))) return MR_ERR_INVALID_ARG;
  for (int i = 0; i < P; ++i)
    if (rows[i] > kMostSide || cols[i] > kMostSide) return MR_ERR_INVALID_ARG;
  return MR_OK;
}

size_t muon_workspace(const uint64_t* rows, const uint64_t* cols, int P, int products) {
  if ((products != 16 && products != 32) || check_matrices(rows, cols, P) != MR_OK) return 0;
  uint64_t most = 0;
  for (int i = 0; i < P;) {
    const MuonGroup g = muon_group(rows, cols, P, i, products / 16);
    most = std::max(most, g.bytes);
    i = g.end;
  }
  return mr::workspace_bytes_for(std::max<uint64_t>(most, row_words_bytes(mr::kMuonMats * mr::kMuonCount)), 1);
}

mr_status muon_step(const void* const* params, const void* const* grads, const uint64_t* rows, const uint64_t* cols, int P, mr_dtype dtype,
                    mr_dtype gdtype, const mr_muon_state* in, void* const* params_out, const mr_muon_state* out, const mr_muon_hyper* h,
                    const float* clip, hipStream_t st) {
  mr_status s = check_types(dtype, gdtype);
  if (s != MR_OK) return s;
  if (!h || (h->products != 16 && h->products != 32) || (h->adjust != MR_MUON_RATIO && h->adjust != MR_MUON_RMS) || h->steps < 1 ||
      h->steps > kNsMostSteps)
    return MR_ERR_INVALID_ARG;
  const float eps32 = static_cast<float>(h->eps);
  if (!std::isfinite(h->lr) || !std::isfinite(h->weight_decay) || !(h->momentum >= 0.0 && h->momentum < 1.0) || !(h->eps >= kLeastNorm) ||
      !std::isfinite(eps32))
    return MR_ERR_INVALID_ARG;
  double coef[3 * kNsMostSteps];
  for (int i = 0; i < 3 * h->steps; ++i) coef[i] = h->coefficients ? h->coefficients[i] : kNsCoef[i % 3];
  if (!polynomials_fit(coef, h->steps)) return MR_ERR_INVALID_ARG;
  s = check_matrices(rows, cols, P);
  if (s != MR_OK) return s;
  uint64_t total = 0;
  for (int i = 0; i < P; ++i) {
    total += (rows[i] * cols[i] + mr::kMxBlock - 1) / mr::kMxBlock * mr::kMxBlock;
    if (total >= uint64_t{mr::kMxBlock} << 32) return MR_ERR_INVALID_ARG;
  }
  if (total == 0) return MR_OK;
  if (!in || !grads) return MR_ERR_INVALID_ARG;
  const bool master = in->master != nullptr;
  if (master && dtype == MR_FP32) return MR_ERR_DTYPE;
  if (!out) out = in;
  if ((!params && !(master && params_out)) || master != (out->master != nullptr)) return MR_ERR_INVALID_ARG;
  for (const mr_muon_state* q : {in, out})
    if (!q->momentum || !on_grid(q->momentum, 256) || !on_grid(q->master, 256)) return MR_ERR_INVALID_ARG;
  if (!on_grid(clip, 4)) return MR_ERR_INVALID_ARG;
  const size_t es = mr::elem_size(dtype), gs = mr::elem_size(gdtype);
  auto count = [&](int i) { return rows[i] * cols[i]; };
  auto param_in = [&](int i) { return params ? params[i] : nullptr; };
  auto param_out = [&](int i) { return params_out ? params_out[i] : const_cast<void*>(params[i]); };
  for (int i = 0; i < P; ++i) {
    if (count(i) == 0) continue;
    if (!grads[i] || !on_grid(grads[i], gs) || !param_out(i) || !on_grid(param_out(i), es)) return MR_ERR_INVALID_ARG;
    if (!master && (!param_in(i) || !on_grid(param_in(i), es))) return MR_ERR_INVALID_ARG;
  }
  Outputs outs(&t_spans);
  for (int i = 0; i < P; ++i) outs.add(param_out(i), count(i) * es, i);
  outs.add(out->momentum, total * 4, -1);
  outs.add(out->master, total * 4, -2);
  if (!outs.ok()) return MR_ERR_ALIAS;
  auto only = [](int id) { return [id](int o) { return o == id; }; };
  bool fine = outs.admits(in->momentum, total * 4, only(-1)) && outs.admits(in->master, total * 4, only(-2)) && outs.admits(clip, 12);
  for (int i = 0; fine && i < P; ++i)
    fine = outs.admits(grads[i], count(i) * gs) && (master || outs.admits(param_in(i), count(i) * es, only(i)));
  if (!fine) return MR_ERR_ALIAS;

  const int pieces = h->products / 16;
  const float mu = static_cast<float>(h->momentum), c = static_cast<float>(1.0 - h->momentum);
  mr::Ctrl* ctrl = nullptr;
  char* data = nullptr;
  std::unique_lock<std::mutex> use;  // to the last launch
  uint64_t most = row_words_bytes(mr::kMuonMats * mr::kMuonCount);
  for (int i = 0; i < P;) {
    const MuonGroup g = muon_group(rows, cols, P, i, pieces);
    most = std::max(most, g.bytes);
    i = g.end;
  }
  s = mr::stream_workspace(st, most, &ctrl, &data, &use);
  if (s != MR_OK) return s;
  uint64_t at = 0;
  for (int first = 0; first < P;) {
    const MuonGroup g = muon_group(rows, cols, P, first, pieces);
    struct Mat {
      MuonShape s;
      int i;
      uint64_t at;
      _Float16 *x, *xt[2], *a, *p;
    } mats[mr::kMuonMats];
    mr::MomentumArgs mo{};
    mr::OrientArgs od{};
    _Float16* next = reinterpret_cast<_Float16*>(data);
    for (int i = first; i < g.end; ++i) {
      if (count(i) == 0) continue;
      const uint32_t k = mo.P++;
      Mat& q = mats[k];
      q.s = muon_shape(rows[i], cols[i], pieces);
      q.i = i;
      q.at = at;
      auto take = [&](uint64_t halves) {
        _Float16* r = next;
        next += halves * pieces;
        return r;
      };
      const MuonShape& z = q.s;
      q.x = take(uint64_t{z.m} * z.ldn);
      q.xt[0] = take(uint64_t{z.n} * z.ldm);
      q.xt[1] = take(uint64_t{z.n} * z.ldm);
      q.a = take(uint64_t{z.m} * z.ldm);
      q.p = take(uint64_t{z.m} * z.ldm);
      mo.g[k] = static_cast<const char*>(grads[i]);
      mo.n[k] = count(i);
      mo.at[k] = at;
      mo.tile[k] = mr::momentum_tile(count(i));
      mo.tile_prefix[k + 1] = mo.tile_prefix[k] + mr::momentum_tiles(count(i));
      od.g[k] = mo.g[k];
      od.direct[k] = z.turned ? q.xt[0] : q.x;
      od.turned[k] = z.turned ? q.x : q.xt[0];
      od.at[k] = at;
      od.rows[k] = static_cast<uint32_t>(rows[i]);
      od.cols[k] = static_cast<uint32_t>(cols[i]);
      od.tile_prefix[k + 1] = od.tile_prefix[k] + ((z.ldm + 63) / 64) * ((z.ldn + 63) / 64);
      at += (count(i) + mr::kMxBlock - 1) / mr::kMxBlock * mr::kMxBlock;
    }
    first = g.end;
    if (mo.P == 0) continue;
    mo.m = in->momentum;
    mo.m_out = out->momentum;
    mo.master_out = out->master;
    mo.clip = od.clip = clip;
    mo.sums = reinterpret_cast<double*>(next);
    mo.norms = mo.sums + g.sums;
    mo.arrived = row_words(ctrl);
    mo.mu = od.mu = mu;
    mo.c = od.c = c;
    mo.nesterov = od.nesterov = h->nesterov != 0;
    od.P = mo.P;
    od.m = out->momentum;
    od.norms = mo.norms;
    od.eps = h->eps;
    od.pieces = pieces;
    if (mr::trace_on())
      std::fprintf(stderr, "[mr] muon matrices=%u dtype=%d grad=%d products=%d master=%d workspace=%llu\n", mo.P, static_cast<int>(dtype),
                   static_cast<int>(gdtype), h->products, master ? 1 : 0, static_cast<unsigned long long>(g.bytes));
    hipError_t e = mr::launch_momentum(mo, gdtype, st);
    if (e == hipSuccess) e = mr::launch_orient(od, gdtype, st);
    mr::NsTiles list{0, 0};
    for (uint32_t k = 0; k < mo.P; ++k) {
      const MuonShape& z = mats[k].s;
      if (z.m >= mr::kNsWideFrom) list.wide += mr::ns_tiles(256, z.ldm, z.ldn, false);
      if (z.m >= mr::kNsSquareFrom) list.square += mr::ns_tiles(128, z.ldm, z.ldn, false);
    }
    // one launch for the matrices of each tile size; those of the longest sums first, so that the short tiles fill the end
    uint32_t order[mr::kMuonMats];
    for (uint32_t k = 0; k < mo.P; ++k) order[k] = k;
    std::stable_sort(order, order + mo.P, [&](uint32_t x, uint32_t y) { return mats[x].s.n > mats[y].s.n; });
    for (int step = 0; step < h->steps && e == hipSuccess; ++step) {
      const double* k3 = coef + 3 * step;
      for (int kind = mr::kNsGram; kind <= mr::kNsStep && e == hipSuccess; ++kind)
        for (uint32_t tile : {256u, 128u, 64u}) {
          mr::NsLastArgs la{};
          mr::NsArgs& a = la.s;
          const bool final = kind == mr::kNsStep && step + 1 == h->steps;
          for (uint32_t o = 0; o < mo.P; ++o) {
            const Mat& q = mats[order[o]];
            const MuonShape& z = q.s;
            if (mr::ns_tile(z.m, list, pieces) != tile) continue;
            mr::NsProduct& p = a.p[a.P];
            p.M = z.m;
            p.ldct = z.ldm;
            if (kind == mr::kNsStep) {
              p.a = q.p, p.b = q.xt[step & 1], p.c = q.x, p.ct = q.xt[(step + 1) & 1];
              p.N = z.n, p.K = z.ldm, p.ldc = z.ldn;
            } else {
              p.a = p.b = kind == mr::kNsGram ? q.x : q.a;
              p.c = kind == mr::kNsGram ? q.a : q.p;
              p.N = z.m, p.K = kind == mr::kNsGram ? z.ldn : z.ldm, p.ldc = z.ldm;
            }
            a.tile_prefix[a.P + 1] = a.tile_prefix[a.P] + mr::ns_tiles(tile, z.ldm, kind == mr::kNsStep ? z.ldn : z.ldm, kind != mr::kNsStep);
            if (final) {
              mr::NsUpdate& u = la.u[a.P];
              u.p = static_cast<const char*>(param_in(q.i));
              u.po = static_cast<char*>(param_out(q.i));
              u.at = q.at;
              const double r = static_cast<double>(rows[q.i]), cc = static_cast<double>(cols[q.i]);
              u.scale = static_cast<float>(h->lr * (h->adjust == MR_MUON_RATIO ? std::sqrt(std::max(1.0, r / cc)) : 0.2 * std::sqrt(std::max(r, cc))));
              u.turned = z.turned;
            }
            ++a.P;
          }
          if (a.P == 0) continue;
          a.pieces = pieces;
          a.ca = static_cast<float>(k3[0]);
          a.cb = static_cast<float>(k3[1]);
          a.cc = static_cast<float>(k3[2]);
          if (final) {
            la.master = in->master;
            la.master_out = out->master;
            la.clip = clip;
            la.keep = static_cast<float>(1.0 - h->lr * h->weight_decay);
            e = mr::launch_ns_last(la, dtype, tile, st);
          } else {
            e = mr::launch_ns(a, static_cast<mr::NsKind>(kind), tile, st);
          }
          if (e != hipSuccess) break;
        }
    }
    if (e != hipSuccess) return hip_fail(e);
  }
  return MR_OK;
}

}  // namespace

extern "C" {

mr_status mr_layer_norm_forward(const void* const* bufs, int W, const void* residual, const void* gamma, const void* beta,
                                size_t rows, size_t cols, mr_dtype dtype, mr_dtype wdtype, double eps, void* x_out, void* y,
                                float* mean, float* rstd, mr_stream stream) {
  return guarded([&] {
    return layer_norm_forward(bufs, W, residual, gamma, beta, rows, cols, dtype, wdtype, eps, x_out, y, mean, rstd,
                              reinterpret_cast<hipStream_t>(stream));
  });
}

mr_status mr_layer_norm_backward(const void* dy, const void* x, const void* gamma, const float* mean, const float* rstd,
                                 const void* dres, size_t rows, size_t cols, mr_dtype dtype, mr_dtype wdtype, void* dx,
                                 void* dgamma, void* dbeta, mr_stream stream) {
  return guarded([&] {
    return layer_norm_backward(dy, x, gamma, mean, rstd, dres, rows, cols, dtype, wdtype, dx, dgamma, dbeta,
                               reinterpret_cast<hipStream_t>(stream));
  });
}

mr_status mr_grad_norm(const void* const* grads, const uint64_t* counts, int P, mr_dtype dtype, double scale, double max_norm,
                       float* out, mr_stream stream) {
  return guarded([&] { return grad_norm(grads, counts, P, dtype, scale, max_norm, out, reinterpret_cast<hipStream_t>(stream)); });
}

mr_status mr_adamw_state_elems(const uint64_t* counts, int P, uint64_t* elems) { return state_elems(counts, P, elems); }

mr_status mr_adamw_step(const void* const* params, const void* const* grads, const uint64_t* counts, int P, mr_dtype dtype,
                        mr_dtype grad_dtype, mr_state_format format, const mr_adamw_state* state, void* const* params_out,
                        const mr_adamw_state* state_out, const mr_adamw_hyper* hyper, const float* clip, mr_stream stream) {
  return guarded([&] {
    return adamw_step(params, grads, counts, P, dtype, grad_dtype, format, state, params_out, state_out, hyper, clip,
                      reinterpret_cast<hipStream_t>(stream));
  });
}

mr_status mr_token_logprob_forward(const void* logits, size_t rows, size_t cols, size_t stride, mr_dtype dtype, const int64_t* targets,
                                   double temperature, float* logp, float* stats, mr_stream stream) {
  return guarded([&] {
    return token_logprob_forward(logits, rows, cols, stride, dtype, targets, temperature, logp, stats, reinterpret_cast<hipStream_t>(stream));
  });
}

mr_status mr_token_logprob_backward(const void* logits, size_t rows, size_t cols, size_t stride, mr_dtype dtype, const int64_t* targets,
                                    double temperature, const float* stats, const float* dlogp, void* dlogits, size_t dstride,
                                    mr_stream stream) {
  return guarded([&] {
    return token_logprob_backward(logits, rows, cols, stride, dtype, targets, temperature, stats, dlogp, dlogits, dstride,
                                  reinterpret_cast<hipStream_t>(stream));
  });
}

mr_status mr_policy_loss(const void* logits, size_t rows, size_t cols, size_t stride, mr_dtype dtype, const int64_t* targets,
                         const float* old_logp, const float* ref_logp, const float* advantages, const float* weights,
                         const mr_policy_hyper* hyper, float* record, float* logp, void* dlogits, size_t dstride, mr_stream stream) {
  return guarded([&] {
    return policy_loss(logits, rows, cols, stride, dtype, targets, old_logp, ref_logp, advantages, weights, hyper, record, logp, dlogits,
                       dstride, reinterpret_cast<hipStream_t>(stream));
  });
}

mr_status mr_preference_loss(const float* logp, const float* ref_logp, size_t rows, const int64_t* offsets, size_t pairs,
                             const mr_preference_hyper* hyper, float* record, float* margins, float* dlogp, mr_stream stream) {
  return guarded([&] {
    return preference_loss(logp, ref_logp, rows, offsets, pairs, hyper, record, margins, dlogp, reinterpret_cast<hipStream_t>(stream));
  });
}

size_t mr_muon_workspace_bytes(const uint64_t* rows, const uint64_t* cols, int P, int products) { return muon_workspace(rows, cols, P, products); }

mr_status mr_muon_step(const void* const* params, const void* const* grads, const uint64_t* rows, const uint64_t* cols, int P,
                       mr_dtype dtype, mr_dtype grad_dtype, const mr_muon_state* state, void* const* params_out,
                       const mr_muon_state* state_out, const mr_muon_hyper* hyper, const float* clip, mr_stream stream) {
  return guarded([&] {
    return muon_step(params, grads, rows, cols, P, dtype, grad_dtype, state, params_out, state_out, hyper, clip,
                     reinterpret_cast<hipStream_t>(stream));
  });
}

}  // extern "C"
