// gm_marshal.cpp -- what the Python binding of the layers and of the draw does for each call: checks tensors, makes the
// results, fills the descriptors of the C interface and calls it on the current stream. Compiled because a call of one row
// takes the GPU a few microseconds, and the same in Python took 20 (a product 5 so, a norm 8).
//
// The functions of the C interface are handed in by address (init): which build of the library they
// come from is the binding's choice. Arguments that do not fit raise ValueError; statuses are returned.
#include <algorithm>
#include <cstdint>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>
#include <tuple>
#include <type_traits>
#include <vector>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include "gm_layers.h"
#include "gm_sampling.h"

namespace {

using at::Tensor;
using Opt = std::optional<Tensor>;

struct Functions {
  decltype(&gm_linear_forward) linear_forward;
  decltype(&gm_linear_backward) linear_backward;
  decltype(&gm_linear_workspace) linear_workspace;
  decltype(&gm_norm_forward) norm_forward;
  decltype(&gm_norm_backward) norm_backward;
  decltype(&gm_norm_workspace) norm_workspace;
  decltype(&gm_draw) draw;
} fn = {};

template <class... A>
[[noreturn]] void refuse(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw std::invalid_argument(s.str());
}

int type_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return GM_LOSS_F32;
    case at::kBFloat16: return GM_LOSS_BF16;
    case at::kHalf: return GM_LOSS_F16;
    default: return -1;
  }
}

struct Matrix {
  void* p = nullptr;
  int64_t ld = 0;
};
void* address(const Tensor& t) { return t.numel() ? t.data_ptr() : nullptr; }

// A CUDA matrix whose rows are consecutive elements; as `like`, and of the given size.
Matrix matrix(const char* name, const Tensor& t, const Tensor* like = nullptr, int64_t rows = -1, int64_t cols = -1) {
  if (!t.defined() || !t.is_cuda() || t.dim() != 2 || type_of(t) < 0)
    refuse(name, " must be a 2-d CUDA tensor of float32, bfloat16 or float16");
  if (like && (t.scalar_type() != like->scalar_type() || t.device() != like->device()))
    refuse(name, " must be ", like->scalar_type(), " on ", like->device(), ", not ", t.scalar_type(), " on ", t.device());
  const int64_t n = t.size(0), m = t.size(1), ld = t.stride(0), step = t.stride(1);
  if (rows >= 0 && (n != rows || m != cols)) refuse(name, " must be ", rows, " x ", cols, ", not ", n, " x ", m);
  if ((step != 1 && m > 1) || (ld < m && n > 1))
    refuse(name, "'s rows must be consecutive elements that do not overlap (strides ", ld, ", ", step, ")");
  return Matrix{address(t), n > 1 ? ld : std::max<int64_t>(m, 1)};
}
Matrix matrix(const char* name, const Opt& t, const Tensor* like, int64_t rows, int64_t cols) {
  return t ? matrix(name, *t, like, rows, cols) : Matrix{};
}
void* vector(const char* name, const Tensor& t, int64_t n, at::ScalarType type, const at::Device& device) {
  if (!t.defined() || t.dim() != 1 || t.size(0) != n || t.scalar_type() != type || t.device() != device || !t.is_contiguous())
    refuse(name, " must be a contiguous tensor of ", n, " elements of ", type, " on ", device);
  return address(t);
}
void* vector(const char* name, const Opt& t, int64_t n, const Tensor& like) {
  return t ? vector(name, *t, n, like.scalar_type(), like.device()) : nullptr;
}
// From torch's allocator, on x's device. Straight from its CUDA function: by way of the dispatcher three results take 2.4 us longer.
Tensor made(const Tensor& x, at::IntArrayRef size, at::ScalarType type) {
  return Tensor(at::detail::empty_cuda(size, type, x.device(), std::nullopt));
}
Tensor rows_like(const Tensor& x, int64_t rows, int64_t cols) { return made(x, {rows, cols}, x.scalar_type()); }

struct Here {  // the tensors' device, and its current stream
  c10::cuda::CUDAGuard guard;
  void* stream;
  explicit Here(const Tensor& x) : guard(x.device()), stream(c10::cuda::getCurrentCUDAStream(x.device().index()).stream()) {}
};
// Workspace from torch's allocator, on the current stream, for the time of a call.
struct Work {
  Tensor t;
  gm_layer_config cfg = {};
  Work(const Tensor& x, int64_t bytes) {
    if (!bytes) return;
    t = made(x, {bytes}, at::kByte);
    cfg.workspace = t.data_ptr();
    cfg.workspace_bytes = bytes;
  }
};

// ---- product ------------------------------------------------------------------------------
gm_linear linear_of(const Tensor& x, const Tensor& w, int act) {
  const Matrix mx = matrix("x", x), mw = matrix("w", w, &x);
  if (w.size(1) != x.size(1) || x.size(1) < 1 || w.size(0) < 1)
    refuse("x has rows of ", x.size(1), " elements, w is ", w.size(0), " x ", w.size(1));
  return gm_linear{x.size(0), x.size(1), w.size(0), mx.p, mx.ld, mw.p, mw.ld, type_of(x), act};
}

// y and z: the caller's, or made (z with keep and an activation).
std::tuple<int, Opt, Opt> linear_forward(const Tensor& x, const Tensor& w, const Opt& bias, int act, const Opt& residual, bool keep,
                                         Opt y, Opt z, bool make) {
  const gm_linear p = linear_of(x, w, act);
  const void* b = vector("bias", bias, p.n_outs, x);
  const Matrix r = matrix("residual", residual, &x, p.n_rows, p.n_outs);
  const Here here(x);
  if (make) {
    y = rows_like(x, p.n_rows, p.n_outs);
    if (keep && act != GM_ACT_NONE) z = rows_like(x, p.n_rows, p.n_outs);
  }
  const Matrix my = matrix("y", y, &x, p.n_rows, p.n_outs), mz = matrix("z", z, &x, p.n_rows, p.n_outs);
  int64_t bytes = 0;
  int rc = fn.linear_workspace(&p, 0, &bytes);
  if (rc == GM_OK) {
    const Work work(x, bytes);
    rc = fn.linear_forward(&p, &work.cfg, here.stream, b, r.p, r.ld, my.p, my.ld, mz.p, mz.ld);
  }
  return {rc, y, z};
}

std::tuple<int, Opt, Opt, Opt> linear_backward(const Tensor& x, const Tensor& w, const Tensor& grad, int act, const Opt& z, Opt dx, Opt dw,
                                               Opt db, bool make_x, bool make_w, bool make_b) {
  const gm_linear p = linear_of(x, w, act);
  const Matrix g = matrix("grad", grad, &x, p.n_rows, p.n_outs), mz = matrix("z", z, &x, p.n_rows, p.n_outs);
  const Here here(x);
  if (make_x) dx = rows_like(x, p.n_rows, p.dim);
  if (make_w) dw = rows_like(x, p.n_outs, p.dim);
  if (make_b) db = made(x, {p.n_outs}, x.scalar_type());
  const Matrix mx = matrix("dx", dx, &x, p.n_rows, p.dim), mw = matrix("dw", dw, &x, p.n_outs, p.dim);
  void* b = vector("dbias", db, p.n_outs, x);
  int64_t bytes = 0;
  int rc = fn.linear_workspace(&p, 1, &bytes);
  if (rc == GM_OK) {
    const Work work(x, bytes);
    rc = fn.linear_backward(&p, &work.cfg, here.stream, g.p, g.ld, mz.p, mz.ld, mx.p, mx.ld, mw.p, mw.ld, b);
  }
  return {rc, dx, dw, db};
}

// A number that 32 bits would take to 0 means something else than 0 does.
void still_a_number(const char* name, double v) {
  if (v != 0 && static_cast<float>(v) == 0) refuse(name, " is ", v, ": 0 in 32 bits");
}

// ---- norms around a residual -----------------------------------------------------------------
struct Rule {
  int norm;
  const Opt &after, &after_bias, &gate;
  double scale;
  const Opt &before, &before_bias;
  double eps;
};
gm_norm norm_of(const Tensor& x, const Opt& f, const Rule& r) {
  const Matrix mx = matrix("x", x);
  const int64_t n = x.size(0), dim = x.size(1);
  if (dim < 1) refuse("x must have rows of an element at least");
  if (!f && (r.after || r.after_bias || r.gate)) refuse("after, after_bias and gate belong to f, which is None");
  if ((!r.after && r.after_bias) || (!r.before && r.before_bias)) refuse("a bias needs its norm's weight");
  still_a_number("eps", r.eps);
  const Matrix mf = matrix("f", f, &x, n, dim);
  int kind = GM_GATE_NONE;
  Matrix g;
  if (r.gate) {
    kind = r.gate->dim() == 1 ? GM_GATE_VECTOR : GM_GATE_MATRIX;
    if (kind == GM_GATE_VECTOR) g.p = vector("gate", r.gate, dim, x);
    else g = matrix("gate", *r.gate, &x, n, dim);
  }
  return gm_norm{n, dim, type_of(x), r.norm, kind, static_cast<float>(r.scale), static_cast<float>(r.eps), mx.p, mx.ld, mf.p, mf.ld,
                 vector("after", r.after, dim, x), vector("after_bias", r.after_bias, dim, x), g.p, g.ld,
                 vector("before", r.before, dim, x), vector("before_bias", r.before_bias, dim, x)};
}
float* stats_of(const Opt& t, const Tensor& x) {
  if (!t) return nullptr;
  if (t->dim() != 2 || t->size(0) != x.size(0) || t->size(1) != 4 || t->scalar_type() != at::kFloat || t->device() != x.device() ||
      !t->is_contiguous())
    refuse("stats must be a contiguous float32 tensor of ", x.size(0), " x 4 on ", x.device());
  return static_cast<float*>(address(*t));
}

std::tuple<int, Opt, Opt, Opt> norm_forward(const Tensor& x, const Opt& f, int norm, const Opt& after, const Opt& after_bias, const Opt& gate,
                                            double scale, const Opt& before, const Opt& before_bias, double eps, Opt x_out, Opt y, Opt stats,
                                            bool make) {
  const gm_norm n = norm_of(x, f, Rule{norm, after, after_bias, gate, scale, before, before_bias, eps});
  const Here here(x);
  if (make) {
    if (!f && !before) refuse("there is nothing to compute without f and before");
    if (f) x_out = rows_like(x, n.n_rows, n.dim);
    if (before) y = rows_like(x, n.n_rows, n.dim);
    stats = made(x, {n.n_rows, 4}, at::kFloat);
  }
  const Matrix o = matrix("x_out", x_out, &x, n.n_rows, n.dim), my = matrix("y", y, &x, n.n_rows, n.dim);
  const int rc = fn.norm_forward(&n, here.stream, o.p, o.ld, my.p, my.ld, stats_of(stats, x));
  return {rc, x_out, y, stats};
}

// grads: the caller's seven, or with make those of `need` (bits in the order of gm_norm_grads).
std::tuple<int, std::vector<Opt>> norm_backward(const Tensor& x, const Opt& f, const Opt& stats, const Opt& gx, const Opt& gy, int norm,
                                                const Opt& after, const Opt& after_bias, const Opt& gate, double scale, const Opt& before,
                                                const Opt& before_bias, double eps, std::vector<Opt> grads, bool make, int need) {
  const gm_norm n = norm_of(x, f, Rule{norm, after, after_bias, gate, scale, before, before_bias, eps});
  const Matrix mgx = matrix("grad_x", gx, &x, n.n_rows, n.dim), mgy = matrix("grad_y", gy, &x, n.n_rows, n.dim);
  const float* st = stats_of(stats, x);
  const Here here(x);
  if (make) {
    const Opt all[7] = {x, f, gate, after, after_bias, before, before_bias};
    grads.assign(7, Opt());
    bool any = false;
    for (int i = 0; i < 7; ++i)
      if (all[i] && (need >> i & 1)) grads[i] = made(x, all[i]->sizes(), x.scalar_type()), any = true;
    if (!any) return {GM_OK, std::move(grads)};
  } else if (grads.size() != 7) {
    refuse("grads must be seven");
  }
  gm_norm_grads o = {};
  const Matrix ox = matrix("grads.x", grads[0], &x, n.n_rows, n.dim), of = matrix("grads.f", grads[1], &x, n.n_rows, n.dim);
  o.x = ox.p, o.x_ld = ox.ld, o.f = of.p, o.f_ld = of.ld;
  if (n.gate_kind == GM_GATE_MATRIX) {
    const Matrix og = matrix("grads.gate", grads[2], &x, n.n_rows, n.dim);
    o.gate = og.p, o.gate_ld = og.ld;
  } else {
    o.gate = vector("grads.gate", grads[2], n.dim, x);
  }
  o.after = vector("grads.after", grads[3], n.dim, x);
  o.after_bias = vector("grads.after_bias", grads[4], n.dim, x);
  o.before = vector("grads.before", grads[5], n.dim, x);
  o.before_bias = vector("grads.before_bias", grads[6], n.dim, x);
  int64_t bytes = 0;
  int rc = fn.norm_workspace(&n, &bytes);
  if (rc == GM_OK && (n.n_rows > 0 || o.after || o.after_bias || o.before || o.before_bias || o.gate)) {
    const Work work(x, bytes);
    rc = fn.norm_backward(&n, &work.cfg, here.stream, st, mgx.p, mgx.ld, mgy.p, mgy.ld, &o);
  }
  return {rc, std::move(grads)};
}

// ---- draw ------------------------------------------------------------------------------------
// A value of the rule: a number, or a tensor of one a row.
template <class T>
void value_of(const char* name, const pybind11::object& v, int64_t n, const Tensor& z, at::ScalarType type, const T** rows, T* all) {
  if (THPVariable_Check(v.ptr())) {
    *rows = static_cast<const T*>(vector(name, THPVariable_Unpack(v.ptr()), n, type, z.device()));
    return;
  }
  try {
    *all = v.cast<T>();
    if (std::is_floating_point_v<T>) still_a_number(name, v.cast<double>());
  } catch (const pybind11::cast_error&) {
    refuse(name, type == at::kInt ? " must be a whole number of 32 bits" : " must be a number", ", or a tensor of one a row");
  }
}

// index, logprob and kept: the caller's, or with make made.
std::tuple<int, Tensor, Tensor, Tensor> draw(const Tensor& z, const Tensor& u, const pybind11::object& temperature, const pybind11::object& top_k,
                                             const pybind11::object& top_p, const pybind11::object& min_p, Opt index, Opt logprob, Opt kept,
                                             bool make) {
  if (!make && (!index || !logprob || !kept)) refuse("index, logprob and kept must be tensors");
  const Matrix m = matrix("logits", z);
  const int64_t n = z.size(0);
  if (z.size(1) < 1) refuse("logits must have a class at least");
  gm_draw_rule r = {};
  value_of("temperature", temperature, n, z, at::kFloat, &r.temperature, &r.all_temperature);
  value_of("top_k", top_k, n, z, at::kInt, &r.top_k, &r.all_top_k);
  value_of("top_p", top_p, n, z, at::kFloat, &r.top_p, &r.all_top_p);
  value_of("min_p", min_p, n, z, at::kFloat, &r.min_p, &r.all_min_p);
  const float* pu = static_cast<const float*>(vector("u", u, n, at::kFloat, z.device()));
  const Here here(z);
  if (make) {
    index = made(z, {n}, at::kLong);
    logprob = made(z, {n}, at::kFloat);
    kept = made(z, {n}, at::kInt);
  }
  const int rc = fn.draw(m.p, n, z.size(1), m.ld, type_of(z), &r, pu, here.stream,
                         static_cast<int64_t*>(vector("index", *index, n, at::kLong, z.device())),
                         static_cast<float*>(vector("logprob", *logprob, n, at::kFloat, z.device())),
                         static_cast<int32_t*>(vector("kept", *kept, n, at::kInt, z.device())));
  return {rc, *index, *logprob, *kept};
}

}  // namespace

PYBIND11_MODULE(gm_marshal, m) {
  m.def("init", [](const std::vector<uintptr_t>& a) {
    if (a.size() != 7) refuse("seven functions");
    fn = {reinterpret_cast<decltype(fn.linear_forward)>(a[0]),   reinterpret_cast<decltype(fn.linear_backward)>(a[1]),
          reinterpret_cast<decltype(fn.linear_workspace)>(a[2]), reinterpret_cast<decltype(fn.norm_forward)>(a[3]),
          reinterpret_cast<decltype(fn.norm_backward)>(a[4]),    reinterpret_cast<decltype(fn.norm_workspace)>(a[5]),
          reinterpret_cast<decltype(fn.draw)>(a[6])};
  });
  m.def("linear_forward", &linear_forward);
  m.def("linear_backward", &linear_backward);
  m.def("norm_forward", &norm_forward);
  m.def("norm_backward", &norm_backward);
  m.def("draw", &draw);
}
