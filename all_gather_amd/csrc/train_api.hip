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

}  // extern "C"
