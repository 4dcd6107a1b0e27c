// torch_ops.cpp -- the torch-facing calls of the norm + rotation, the FP8 cache and decoding: checks of
// the arguments, outputs and workspaces, the current device and stream, and autograd, around the C ABI.
// Every step of the computation runs in the library.
//
// These calls are made once per layer and decoding step, on a few microseconds of GPU work, so what the
// host spends on them is what they cost; in Python it was two to three times as much (a decode call on one
// sequence 28 us, a training pass of the norm + rotation through autograd 300).
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/graph_task.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/variable.h>
#include <torch/csrc/utils/pybind.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <array>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <initializer_list>
#include <optional>
#include <tuple>
#include <unordered_set>
#include <vector>

#include "qat_attn.h"

namespace py = pybind11;
using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
using OptTensor = std::optional<Tensor>;

namespace {

// The Python exception of a C status.
[[noreturn]] void raise_status(qat_status_t st, const char* what) {
  py::gil_scoped_acquire gil;
  const py::object cls = py::module_::import("quantization_aware_attention_gb300.capi").attr("QatError");
  const py::object e = cls(static_cast<int>(st), what);
  PyErr_SetObject(cls.ptr(), e.ptr());
  throw py::error_already_set();
}

inline void ok(qat_status_t st, const char* what) {
  if (st != QAT_OK) raise_status(st, what);
}

inline void* stream_of(const at::Device& dev) {
  return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
}

inline bool aligned16(const Tensor& t) { return (reinterpret_cast<uintptr_t>(t.const_data_ptr()) & 15) == 0; }

// check=True, or None with QAT_CHECK_STATUS=1 in the environment: reads the device error word.
void check_status(std::optional<bool> check, const at::Device& dev, const char* what) {
  if (!check.has_value()) {
    const char* env = std::getenv("QAT_CHECK_STATUS");
    check = env != nullptr && env[0] == '1' && env[1] == 0;
  }
  if (*check) ok(qat_attn_device_status(stream_of(dev)), what);
}

// A wrapper (a fake or distributed tensor, a subclass around other tensors) has sizes and a device but no
// memory of its own; its null pointer would read as an argument that was left out.
void with_memory(const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.numel() == 0 || t.const_data_ptr() != nullptr, name, " has no memory of its own");
}

void on_cuda(const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor (this library has no CPU path)");
}

// A tensor that the kernels read or write in place: bf16 [B, H, N, D], D innermost, rows on 16-byte
// boundaries.
struct Rows {
  void* ptr;
  long long s[3];
  bool dense;
  const long long* strides() const { return dense ? nullptr : s; }
};

bool readable(const Tensor& t, Rows* out) {
  out->ptr = const_cast<void*>(t.const_data_ptr());
  out->dense = t.is_contiguous();
  if (!aligned16(t)) return false;
  if (out->dense) return true;
  const auto st = t.strides(), sz = t.sizes();
  if (st[3] != 1) return false;
  for (int i = 0; i < 3; ++i) {
    out->s[i] = st[i];
    if (sz[i] > 1 && st[i] % 8 != 0) return false;
  }
  return true;
}

// `shape`: what it has to be, or -1.
Rows rows(const Tensor& t, const char* name, const at::Device& dev, std::array<int64_t, 4> shape) {
  TORCH_CHECK_VALUE(t.is_cuda() && t.device() == dev, name, " must be a CUDA tensor on ", dev, ", got ",
                    t.device());
  TORCH_CHECK_VALUE(t.scalar_type() == at::kBFloat16, name, " must be torch.bfloat16, got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.dim() == 4, name, " must be [B, H, N, D], got shape ", t.sizes());
  for (int i = 0; i < 4; ++i) {
    TORCH_CHECK_VALUE(shape[i] < 0 || t.size(i) == shape[i], name, " has shape ", t.sizes(), ", expected ",
                      at::IntArrayRef(shape.data(), 4), " (-1: any)");
    TORCH_CHECK_VALUE(t.size(i) <= INT32_MAX, name, " is too large: ", t.sizes());
  }
  with_memory(t, name);
  Rows r;
  TORCH_CHECK_VALUE(readable(t, &r), name, " must have D innermost and rows on 16-byte boundaries, got strides ",
                    t.strides());
  return r;
}

const int* index_ptr(const Tensor& t, const char* name, const at::Device& dev, int64_t n, int64_t m) {
  TORCH_CHECK_VALUE(t.device() == dev, name, " must be a tensor on ", dev, ", got ", t.device());
  TORCH_CHECK_VALUE(t.scalar_type() == at::kInt, name, " must be torch.int32, got ", t.scalar_type());
  const int64_t dims = m == -2 ? 1 : 2;
  TORCH_CHECK_VALUE(t.dim() == dims && t.is_contiguous() && (n < 0 || t.size(0) == n), name,
                    " must be contiguous with ", dims, " dimension(s)", n < 0 ? "" : ", one row a sequence",
                    ", got shape ", t.sizes());
  with_memory(t, name);
  return t.const_data_ptr<int>();
}

// An uninitialized tensor from the caching allocator, not by way of the dispatcher (0.6 us more for each).
Tensor new_tensor(at::IntArrayRef sizes, at::ScalarType type, const at::Device& dev) {
  return at::detail::empty_cuda(sizes, type, dev, std::nullopt);
}

void no_gradient(const char* what, const Tensor& t) {
  TORCH_CHECK_VALUE(!(at::GradMode::is_enabled() && t.requires_grad()), what,
                    " has no backward: call it under torch.no_grad(), or with tensors that do not require "
                    "gradients");
}

// Forward-mode derivatives would be dropped: the direct calls look at requires_grad alone.
void no_tangent(const char* what, std::initializer_list<const Tensor*> in) {
  for (const Tensor* t : in)
    TORCH_CHECK_VALUE(!t->defined() || !t->_fw_grad(0).defined(), what, " has no forward-mode derivative");
}

Tensor workspace_or_new(const OptTensor& ws, int64_t bytes, const at::Device& dev) {
  if (!ws.has_value()) return new_tensor({bytes}, at::kByte, dev);
  TORCH_CHECK_VALUE(ws->device() == dev && ws->scalar_type() == at::kByte && ws->is_contiguous(),
                    "workspace must be a contiguous uint8 tensor on ", dev);
  with_memory(*ws, "workspace");
  return *ws;
}

const void* ptr_or_null(const Tensor& t) { return t.defined() ? t.const_data_ptr() : nullptr; }

// ------------------------------------------------------------------------------- norm + rotation

struct RopeArgs {
  int rotary_dim;
  bool interleaved;
  double amplitude, eps;
};

struct NormRopeShape {
  at::Device dev;
  int64_t B, Hq, Hk, N, D, pos_stride;
  bool w_bf16, has_k;
  Rows q, k;
};

// Undefined tensors are absent ones.
NormRopeShape check_norm_rope(const Tensor& q, const Tensor& k, const Tensor& positions, const Tensor& phases,
                              const Tensor& wq, const Tensor& wk, const RopeArgs& a) {
  on_cuda(q, "q");
  NormRopeShape s{q.device(), 0, 0, 0, 0, 0, 0, false, k.defined(), {}, {nullptr, {0, 0, 0}, true}};
  s.q = rows(q, "q", s.dev, {-1, -1, -1, -1});
  s.B = q.size(0);
  s.Hq = q.size(1);
  s.N = q.size(2);
  s.D = q.size(3);
  TORCH_CHECK_VALUE(s.D == 64 || s.D == 128, "the head dimension must be 64 or 128, got ", s.D);
  if (k.defined()) {
    s.k = rows(k, "k", s.dev, {s.B, -1, s.N, s.D});
    s.Hk = k.size(1);
    TORCH_CHECK_VALUE(wq.defined() == wk.defined(), "q_weight and k_weight go together");
  } else {
    TORCH_CHECK_VALUE(!wk.defined(), "k_weight without k");
  }
  for (const Tensor* w : {&wq, &wk}) {
    if (!w->defined()) continue;
    TORCH_CHECK_VALUE(w->device() == s.dev, "the weights must lie on ", s.dev, ", got ", w->device());
    TORCH_CHECK_VALUE((w->scalar_type() == at::kFloat || w->scalar_type() == at::kBFloat16) &&
                          w->scalar_type() == wq.scalar_type(),
                      "the weights must both be torch.float32 or torch.bfloat16");
    TORCH_CHECK_VALUE(w->dim() == 1 && w->size(0) == s.D && w->is_contiguous() && aligned16(*w),
                      "a weight must be contiguous [", s.D, "] on a 16-byte boundary, got shape ", w->sizes());
    with_memory(*w, "a weight");
  }
  s.w_bf16 = wq.defined() && wq.scalar_type() == at::kBFloat16;
  if (!phases.defined()) {
    TORCH_CHECK_VALUE(!positions.defined(), "positions without a RopePlan");
    return s;
  }
  TORCH_CHECK_VALUE(phases.device() == s.dev, "the RopePlan lies on ", phases.device(), ", q on ", s.dev);
  TORCH_CHECK_VALUE(phases.scalar_type() == at::kLong && phases.is_contiguous() &&
                        phases.numel() == a.rotary_dim / 2,
                    "the RopePlan's phases must be contiguous int64 [rotary_dim / 2]");
  with_memory(phases, "the RopePlan");
  TORCH_CHECK_VALUE(a.rotary_dim <= s.D, "rotary_dim ", a.rotary_dim, " exceeds the head dimension ", s.D);
  TORCH_CHECK_VALUE(positions.defined() && positions.device() == s.dev, "positions must be a tensor on ", s.dev);
  with_memory(positions, "positions");
  TORCH_CHECK_VALUE(positions.scalar_type() == at::kInt, "positions must be torch.int32, got ",
                    positions.scalar_type());
  const auto ps = positions.sizes();
  TORCH_CHECK_VALUE((ps.size() == 1 && ps[0] == s.N) || (ps.size() == 2 && ps[0] == s.B && ps[1] == s.N),
                    "positions has shape ", ps, ", expected [", s.N, "] or [", s.B, ", ", s.N, "]");
  TORCH_CHECK_VALUE(s.N <= 1 || positions.stride(-1) == 1, "positions must be contiguous along the tokens");
  if (ps.size() == 2 && s.B > 1) s.pos_stride = positions.stride(0);
  return s;
}

variable_list norm_rope_forward(const NormRopeShape& s, const Tensor& positions, const Tensor& phases,
                                const Tensor& wq, const Tensor& wk, const RopeArgs& a) {
  const c10::cuda::CUDAGuard guard(s.dev);
  variable_list out;
  out.reserve(2);
  out.push_back(new_tensor({s.B, s.Hq, s.N, s.D}, at::kBFloat16, s.dev));
  if (s.has_k) out.push_back(new_tensor({s.B, s.Hk, s.N, s.D}, at::kBFloat16, s.dev));
  ok(qat_qk_norm_rope(s.q.ptr, s.q.strides(), s.k.ptr, s.k.strides(), out[0].mutable_data_ptr(),
                      out.size() > 1 ? out[1].mutable_data_ptr() : nullptr,
                      static_cast<const int*>(ptr_or_null(positions)), s.pos_stride,
                      static_cast<const unsigned long long*>(ptr_or_null(phases)), ptr_or_null(wq),
                      ptr_or_null(wk), s.w_bf16, static_cast<int>(s.B), static_cast<int>(s.Hq),
                      static_cast<int>(s.Hk), static_cast<int>(s.N), static_cast<int>(s.D), a.rotary_dim,
                      a.interleaved, static_cast<float>(a.amplitude), static_cast<float>(a.eps),
                      stream_of(s.dev)),
     "qat_qk_norm_rope");
  return out;
}

// dx in the input's order in memory: heads inner where a projection wrote them so.
Tensor grad_like(const Rows& x, const NormRopeShape& s, int64_t H, Rows* out) {
  out->dense = true;
  Tensor g;
  if (!x.dense && x.s[2] > x.s[1]) {
    g = new_tensor({s.B, s.N, H, s.D}, at::kBFloat16, s.dev).transpose(1, 2);
    out->dense = false;
    out->s[0] = s.N * H * s.D;
    out->s[1] = s.D;
    out->s[2] = H * s.D;
  } else {
    g = new_tensor({s.B, H, s.N, s.D}, at::kBFloat16, s.dev);
  }
  out->ptr = g.mutable_data_ptr();
  return g;
}

// {dq, dk, dwq, dwk}, undefined where the input is absent.
std::array<Tensor, 4> norm_rope_backward(const NormRopeShape& s, const Tensor& positions,
                                         const Tensor& phases, const Tensor& wq, const Tensor& wk,
                                         const Tensor& dq_out, const Tensor& dk_out, const RopeArgs& a,
                                         const OptTensor& workspace) {
  const c10::cuda::CUDAGuard guard(s.dev);
  const Rows gq = rows(dq_out, "dq_out", s.dev, {s.B, s.Hq, s.N, s.D});
  Rows gk{nullptr, {0, 0, 0}, true}, dq, dk = gk;
  std::array<Tensor, 4> out;
  out[0] = grad_like(s.q, s, s.Hq, &dq);
  if (s.has_k) {
    gk = rows(dk_out, "dk_out", s.dev, {s.B, s.Hk, s.N, s.D});
    out[1] = grad_like(s.k, s, s.Hk, &dk);
  }
  Tensor ws;
  void *dwq = nullptr, *dwk = nullptr;
  if (wq.defined()) {
    // of a tensor without heads the weight's gradient is zero (the entry takes none for it)
    const auto weight_grad = [&](const Tensor& w, int64_t H, void** dw) {
      Tensor g = new_tensor({s.D}, w.scalar_type(), s.dev);
      if (H > 0)
        *dw = g.mutable_data_ptr();
      else
        g.zero_();
      return g;
    };
    out[2] = weight_grad(wq, s.Hq, &dwq);
    if (s.has_k) out[3] = weight_grad(wk, s.Hk, &dwk);
    ws = workspace_or_new(workspace, static_cast<int64_t>(qat_qk_norm_rope_bwd_workspace_bytes(static_cast<int>(s.D))),
                          s.dev);
  }
  ok(qat_qk_norm_rope_bwd(
         s.q.ptr, s.q.strides(), s.k.ptr, s.k.strides(), gq.ptr, gq.strides(), gk.ptr, gk.strides(),
         static_cast<const int*>(ptr_or_null(positions)), s.pos_stride,
         static_cast<const unsigned long long*>(ptr_or_null(phases)), ptr_or_null(wq), ptr_or_null(wk), s.w_bf16,
         dq.ptr, dq.strides(), dk.ptr, dk.strides(), dwq, dwk, static_cast<int>(s.B), static_cast<int>(s.Hq),
         static_cast<int>(s.Hk), static_cast<int>(s.N), static_cast<int>(s.D), a.rotary_dim, a.interleaved,
         static_cast<float>(a.amplitude), static_cast<float>(a.eps), ws.defined() ? ws.mutable_data_ptr() : nullptr,
         ws.defined() ? static_cast<size_t>(ws.numel()) : 0, stream_of(s.dev)),
     "qat_qk_norm_rope_bwd");
  return out;
}

Tensor or_undefined(const OptTensor& t) { return t.has_value() ? *t : Tensor(); }

// A backward step under capture must not pass gradients to a node of the default stream: torch would have that
// stream wait for the capturing one, which ends the capture and may end the process.  A node's stream is the one
// that was current when it was made, and a leaf keeps one accumulation node as long as any graph that ends in it
// lives.
bool on_default_stream(torch::autograd::Node& node, const c10::Stream& none) {
  const auto on = node.stream();
  return on.has_value() && *on == none;
}

constexpr const char* kOnDefault =
    " was made on the default stream and is still alive: drop its outputs before capturing a backward, or make it "
    "on another stream";

// Whether the current stream is being captured, and the device's default stream (never captured itself).
std::optional<c10::Stream> default_beside_capture(const at::Device& dev) {
  const c10::cuda::CUDAStream now = c10::cuda::getCurrentCUDAStream(dev.index());
  const c10::cuda::CUDAStream none = c10::cuda::getDefaultCUDAStream(dev.index());
  if (now == none) return std::nullopt;
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(now.stream(), &status) != cudaSuccess || status == cudaStreamCaptureStatusNone)
    return std::nullopt;
  return none.unwrap();
}

// The forward looks at the leaves that it is given itself.
void check_capture(std::initializer_list<const Tensor*> leaves, const at::Device& dev) {
  const auto none = default_beside_capture(dev);
  if (!none.has_value()) return;
  for (const Tensor* t : leaves) {
    if (!t->defined() || !t->requires_grad() || !t->is_leaf()) continue;
    const auto node = torch::autograd::impl::try_get_grad_accumulator(*t);
    TORCH_CHECK_VALUE(node == nullptr || !on_default_stream(*node, *none), "a graph that ends in one of these leaves",
                      kOnDefault);
  }
}

// The backward at all that lies before it -- a projection and its leaves -- as far as this pass will run it.
void check_capture_before(const at::Device& dev) {
  const auto none = default_beside_capture(dev);
  const auto self = torch::autograd::get_current_node();
  if (!none.has_value() || self == nullptr) return;
  const auto* plan = torch::autograd::get_current_graph_task_exec_info();  // empty: everything runs
  std::vector<torch::autograd::Node*> todo{self.get()};
  std::unordered_set<torch::autograd::Node*> seen;
  while (!todo.empty()) {
    torch::autograd::Node* at = todo.back();
    todo.pop_back();
    for (const auto& edge : at->next_edges()) {
      torch::autograd::Node* node = edge.function.get();
      if (node == nullptr || !seen.insert(node).second) continue;
      if (plan != nullptr && !plan->empty()) {
        const auto it = plan->find(node);
        if (it == plan->end() || !it->second.should_execute()) continue;
      }
      TORCH_CHECK_VALUE(!on_default_stream(*node, *none), "a graph that this backward passes through", kOnDefault);
      todo.push_back(node);
    }
  }
}

// Forward returns the normed and rotated q (and k); nothing but the inputs is saved, the backward
// recomputes the norm.
struct NormRope : torch::autograd::Function<NormRope> {
  static variable_list forward(AutogradContext* ctx, const Tensor& q, const OptTensor& k_,
                               const OptTensor& positions_, const OptTensor& phases_, const OptTensor& wq_,
                               const OptTensor& wk_, int64_t rotary_dim, bool interleaved, double amplitude,
                               double eps) {
    const Tensor k = or_undefined(k_), positions = or_undefined(positions_), phases = or_undefined(phases_);
    const Tensor wq = or_undefined(wq_), wk = or_undefined(wk_);
    const RopeArgs a{static_cast<int>(rotary_dim), interleaved, amplitude, eps};
    const NormRopeShape s = check_norm_rope(q, k, positions, phases, wq, wk, a);
    ctx->save_for_backward({q, k, positions, phases, wq, wk});
    ctx->saved_data["rotary_dim"] = rotary_dim;
    ctx->saved_data["interleaved"] = interleaved;
    ctx->saved_data["amplitude"] = amplitude;
    ctx->saved_data["eps"] = eps;
    return norm_rope_forward(s, positions, phases, wq, wk, a);
  }

  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    TORCH_CHECK(!at::GradMode::is_enabled(), "qat_qk_norm_rope has no second derivative");
    const variable_list v = ctx->get_saved_variables();
    const RopeArgs a{static_cast<int>(ctx->saved_data["rotary_dim"].toInt()),
                     ctx->saved_data["interleaved"].toBool(), ctx->saved_data["amplitude"].toDouble(),
                     ctx->saved_data["eps"].toDouble()};
    const NormRopeShape s = check_norm_rope(v[0], v[1], v[2], v[3], v[4], v[5], a);
    check_capture_before(s.dev);
    for (Tensor& g : grads) {
      no_tangent("qat_qk_norm_rope_backward", {&g});
      Rows r;
      if (!readable(g, &r)) g = g.contiguous();
    }
    auto d = norm_rope_backward(s, v[2], v[3], v[4], v[5], grads[0], s.has_k ? grads[1] : Tensor(), a,
                                std::nullopt);
    return {d[0], d[1], Tensor(), Tensor(), d[2], d[3], Tensor(), Tensor(), Tensor(), Tensor()};
  }
};

py::object norm_rope(const Tensor& q, const OptTensor& k_, const OptTensor& positions_, const OptTensor& phases_,
                     const OptTensor& wq_, const OptTensor& wk_, int64_t rotary_dim, bool interleaved,
                     double amplitude, double eps) {
  const Tensor k = or_undefined(k_), positions = or_undefined(positions_), phases = or_undefined(phases_);
  const Tensor wq = or_undefined(wq_), wk = or_undefined(wk_);
  no_tangent("qat_qk_norm_rope", {&q, &k, &wq, &wk});
  const auto needs = [](const Tensor& t) { return t.defined() && t.requires_grad(); };
  variable_list out;
  if (at::GradMode::is_enabled() && (needs(q) || needs(k) || needs(wq) || needs(wk))) {
    on_cuda(q, "q");
    check_capture({&q, &k, &wq, &wk}, q.device());
    out = NormRope::apply(q, k_, positions_, phases_, wq_, wk_, rotary_dim, interleaved, amplitude, eps);
  } else {
    const RopeArgs a{static_cast<int>(rotary_dim), interleaved, amplitude, eps};
    out = norm_rope_forward(check_norm_rope(q, k, positions, phases, wq, wk, a), positions, phases, wq, wk, a);
  }
  if (!k.defined()) return py::cast(out[0]);
  return py::make_tuple(out[0], out[1]);
}

std::tuple<OptTensor, OptTensor, OptTensor, OptTensor> norm_rope_bwd(
    const Tensor& q, const OptTensor& k_, const OptTensor& positions_, const OptTensor& phases_,
    const OptTensor& wq_, const OptTensor& wk_, int64_t rotary_dim, bool interleaved, double amplitude, double eps,
    const Tensor& dq_out, const OptTensor& dk_out, const OptTensor& workspace) {
  const Tensor k = or_undefined(k_), positions = or_undefined(positions_), phases = or_undefined(phases_);
  const Tensor wq = or_undefined(wq_), wk = or_undefined(wk_);
  TORCH_CHECK_VALUE(k.defined() == dk_out.has_value(), "dk_out goes together with k");
  const Tensor dk = or_undefined(dk_out);
  no_tangent("qat_qk_norm_rope_backward", {&q, &k, &wq, &wk, &dq_out, &dk});
  const RopeArgs a{static_cast<int>(rotary_dim), interleaved, amplitude, eps};
  auto d = norm_rope_backward(check_norm_rope(q, k, positions, phases, wq, wk, a), positions, phases, wq, wk, dq_out,
                              dk, a, workspace);
  const auto opt = [](const Tensor& t) { return t.defined() ? OptTensor(t) : std::nullopt; };
  return {d[0], opt(d[1]), opt(d[2]), opt(d[3])};
}

// ------------------------------------------------------------------------------- windowed attention

// What the attention is called with beside its tensors.
struct WindowArgs {
  double sm_scale;
  int quant_mode, window, sinks;
  bool check;
};

// What the forward runs on, and the backward (both q, k, v by default), each q, k, v; smooth_k's mean or undefined.
struct WindowTensors {
  std::array<Tensor, 3> by, back;
  Tensor k_mean;
};

void dense(const Tensor& t, const char* name, const at::Device& dev, at::IntArrayRef shape) {
  TORCH_CHECK_VALUE(t.is_cuda() && t.device() == dev, name, " must be a CUDA tensor on ", dev, ", got ", t.device());
  TORCH_CHECK_VALUE(t.scalar_type() == at::kBFloat16, name, " must be torch.bfloat16, got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", t.sizes(), ", expected ", shape);
  TORCH_CHECK_VALUE(t.is_contiguous() && aligned16(t), name, " must be contiguous on a 16-byte boundary");
  with_memory(t, name);
}

// {o_q, o_hp, lse}; without `hp` o_hp is undefined.
std::array<Tensor, 3> window_forward(const Tensor& q, const Tensor& k, const Tensor& v, const WindowArgs& a, bool hp) {
  on_cuda(q, "q");
  const at::Device dev = q.device();
  TORCH_CHECK_VALUE(q.dim() == 4, "q must be [B, H, N, D], got shape ", q.sizes());
  for (int i = 0; i < 4; ++i) TORCH_CHECK_VALUE(q.size(i) <= INT32_MAX, "q is too large: ", q.sizes());
  dense(q, "q", dev, q.sizes());
  dense(k, "k", dev, q.sizes());
  dense(v, "v", dev, q.sizes());
  const int64_t B = q.size(0), H = q.size(1), N = q.size(2), D = q.size(3);
  const c10::cuda::CUDAGuard guard(dev);
  std::array<Tensor, 3> out{new_tensor(q.sizes(), at::kBFloat16, dev), Tensor(), new_tensor({B, H, N}, at::kFloat, dev)};
  if (hp) out[1] = new_tensor(q.sizes(), at::kFloat, dev);
  ok(qat_attn_fwd_window(q.const_data_ptr(), k.const_data_ptr(), v.const_data_ptr(), out[0].mutable_data_ptr(),
                         hp ? out[1].mutable_data_ptr<float>() : nullptr, out[2].mutable_data_ptr<float>(), static_cast<int>(B),
                         static_cast<int>(H), static_cast<int>(N), static_cast<int>(D), static_cast<float>(a.sm_scale),
                         a.window, a.sinks, a.quant_mode, stream_of(dev)),
     "qat_attn_fwd_window");
  check_status(a.check, dev, "qat_attn_fwd_window");
  return out;
}

// The forward ran on the leaves or on what was made of them (fake-quantized copies); the backward goes through the
// tensors it is given as if they were the leaves.
struct WindowAttention : torch::autograd::Function<WindowAttention> {
  static variable_list forward(AutogradContext* ctx, const Tensor& q, const Tensor& k, const Tensor& v,
                               const WindowTensors& x, const WindowArgs& a) {
    // the page's backward variant forms Delta from O_q, the straight-through one from O_hp
    const bool page = a.quant_mode == QAT_QUANT_P_FP8E4M3_ROW_TILE64_PAGE_BWD;
    const auto out = window_forward(x.by[0], x.by[1], x.by[2], a, !page);
    const Tensor& o = page ? out[0] : out[1];
    ctx->save_for_backward({x.back[0], x.back[1], x.back[2], o, out[2], x.k_mean});
    ctx->saved_data["sm_scale"] = a.sm_scale;
    ctx->saved_data["quant_mode"] = static_cast<int64_t>(a.quant_mode);
    ctx->saved_data["window"] = static_cast<int64_t>(a.window);
    ctx->saved_data["sinks"] = static_cast<int64_t>(a.sinks);
    ctx->saved_data["check"] = a.check;
    return {out[0]};
  }

  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    TORCH_CHECK(!at::GradMode::is_enabled(), "windowed attention has no second derivative");
    const variable_list t = ctx->get_saved_variables();
    const at::Device dev = t[0].device();
    check_capture_before(dev);
    no_tangent("windowed attention's backward", {&grads[0]});
    Tensor g = grads[0].contiguous();
    if (!aligned16(g)) g = g.clone();
    dense(g, "the gradient", dev, t[0].sizes());
    const int B = static_cast<int>(t[0].size(0)), H = static_cast<int>(t[0].size(1)), N = static_cast<int>(t[0].size(2)),
              D = static_cast<int>(t[0].size(3));
    const int window = static_cast<int>(ctx->saved_data["window"].toInt()),
              sinks = static_cast<int>(ctx->saved_data["sinks"].toInt());
    const c10::cuda::CUDAGuard guard(dev);
    const size_t bytes = qat_attn_bwd_window_workspace_bytes(B, H, N, D, window, sinks);
    Tensor ws = new_tensor({std::max<int64_t>(static_cast<int64_t>(bytes), 256)}, at::kByte, dev);
    variable_list d(3);
    for (Tensor& x : d) x = new_tensor(t[0].sizes(), at::kBFloat16, dev);
    ok(qat_attn_bwd_window(t[0].const_data_ptr(), t[1].const_data_ptr(), t[2].const_data_ptr(), t[3].const_data_ptr(),
                           t[4].const_data_ptr<float>(), g.const_data_ptr(), d[0].mutable_data_ptr(),
                           d[1].mutable_data_ptr(), d[2].mutable_data_ptr(),
                           static_cast<const float*>(ptr_or_null(t[5])), B, H, N, D,
                           static_cast<float>(ctx->saved_data["sm_scale"].toDouble()), window, sinks,
                           static_cast<int>(ctx->saved_data["quant_mode"].toInt()), ws.mutable_data_ptr(),
                           static_cast<size_t>(ws.numel()), stream_of(dev)),
       "qat_attn_bwd_window");
    check_status(ctx->saved_data["check"].toBool(), dev, "qat_attn_bwd_window");
    return {d[0], d[1], d[2], Tensor(), Tensor()};
  }
};

Tensor window_attention(const Tensor& q, const Tensor& k, const Tensor& v, const WindowTensors& x,
                        std::optional<double> sm_scale, int64_t quant_mode, int64_t window, int64_t sinks,
                        std::optional<bool> check) {
  no_tangent("windowed attention", {&q, &k, &v});
  TORCH_CHECK_VALUE(quant_mode >= 0 && quant_mode <= 2, "quant_mode ", quant_mode);
  TORCH_CHECK_VALUE(window >= 1 && sinks >= 0, "window must be at least 1 and sinks at least 0, got ", window, " and ",
                    sinks);
  if (!check.has_value()) {
    const char* env = std::getenv("QAT_CHECK_STATUS");
    check = env != nullptr && env[0] == '1' && env[1] == 0;
  }
  const double scale = sm_scale.has_value() ? *sm_scale
                       : q.dim() == 4       ? 1.0 / std::sqrt(static_cast<double>(std::max<int64_t>(q.size(3), 1)))
                                            : 1.0;
  window = std::min<int64_t>(window, 1 << 30);
  sinks = std::min<int64_t>(sinks, 1 << 30);
  const WindowArgs a{scale, static_cast<int>(quant_mode), static_cast<int>(window), static_cast<int>(sinks), *check};
  if (!at::GradMode::is_enabled() || !(q.requires_grad() || k.requires_grad() || v.requires_grad()))
    return window_forward(x.by[0], x.by[1], x.by[2], a, false)[0];
  on_cuda(q, "q");
  check_capture({&q, &k, &v}, q.device());
  return WindowAttention::apply(q, k, v, x, a)[0];
}

// ------------------------------------------------------------------------------- cache

struct Cache {
  at::Device dev;
  int64_t pages, H, page, D, B, max_pages;
  void *k, *v;
  float *ks, *vs;
  const int *table, *lens;
};

Cache cache_of(const Tensor& k, const Tensor& v, const Tensor& ks, const Tensor& vs, const Tensor& table,
               const Tensor& lens) {
  on_cuda(k, "the cache");
  const at::Device dev = k.device();
  TORCH_CHECK_VALUE(k.dim() == 4, "the cache must be [pages, H, page_size, D]");
  for (const Tensor* t : {&k, &v})
    TORCH_CHECK_VALUE(t->device() == dev && t->scalar_type() == at::kFloat8_e4m3fn && t->is_contiguous() &&
                          t->sizes() == k.sizes() && aligned16(*t),
                      "the cache's codes must be alike, contiguous torch.float8_e4m3fn");
  for (const Tensor* t : {&ks, &vs})
    TORCH_CHECK_VALUE(t->device() == dev && t->scalar_type() == at::kFloat && t->is_contiguous() &&
                          t->sizes() == k.sizes().slice(0, 3) && aligned16(*t),
                      "the cache's scales must be contiguous torch.float32 [pages, H, page_size]");
  no_tangent("the cache", {&ks, &vs});
  for (const Tensor* t : {&k, &v, &ks, &vs}) with_memory(*t, "the cache");
  Cache c{dev, k.size(0), k.size(1), k.size(2), k.size(3), 0, 0, k.mutable_data_ptr(), v.mutable_data_ptr(),
          ks.mutable_data_ptr<float>(), vs.mutable_data_ptr<float>(), nullptr, nullptr};
  c.lens = index_ptr(lens, "seq_lens", dev, -1, -2);
  c.B = lens.size(0);
  c.table = index_ptr(table, "block_table", dev, c.B, -1);
  c.max_pages = table.size(1);
  TORCH_CHECK_VALUE(c.max_pages > 0, "block_table has no pages");
  for (int64_t n : {c.pages, c.H, c.page, c.B, c.max_pages})
    TORCH_CHECK_VALUE(n <= INT32_MAX, "the cache or its table is too large");
  return c;
}

void kv_append(const Tensor& ck, const Tensor& cv, const Tensor& cks, const Tensor& cvs, const Tensor& k,
               const Tensor& v, const Tensor& table, const Tensor& lens, const OptTensor& new_lens,
               std::optional<bool> check) {
  const Cache c = cache_of(ck, cv, cks, cvs, table, lens);
  const Rows rk = rows(k, "k", c.dev, {c.B, c.H, -1, c.D});
  const int64_t N = k.size(2);
  const Rows rv = rows(v, "v", c.dev, {c.B, c.H, N, c.D});
  no_gradient("append", k);
  no_gradient("append", v);
  no_tangent("append", {&k, &v});
  const int* nl = new_lens.has_value() ? index_ptr(*new_lens, "new_lens", c.dev, c.B, -2) : nullptr;
  const c10::cuda::CUDAGuard guard(c.dev);
  ok(qat_kv_cache_append(rk.ptr, rk.strides(), rv.ptr, rv.strides(), c.k, c.v, c.ks, c.vs, c.table, c.lens, nl,
                         static_cast<int>(c.B), static_cast<int>(c.H), static_cast<int>(N), static_cast<int>(c.D),
                         static_cast<int>(c.pages), static_cast<int>(c.page), static_cast<int>(c.max_pages),
                         stream_of(c.dev)),
     "qat_kv_cache_append");
  check_status(check, c.dev, "qat_kv_cache_append");
}

std::tuple<Tensor, Tensor> kv_read(const Tensor& ck, const Tensor& cv, const Tensor& cks, const Tensor& cvs,
                                   const Tensor& table, const Tensor& lens, int64_t begin,
                                   std::optional<int64_t> length, std::optional<bool> check) {
  const Cache c = cache_of(ck, cv, cks, cvs, table, lens);
  TORCH_CHECK_VALUE(begin >= 0 && begin <= INT32_MAX && (!length.has_value() || *length >= 0),
                    "begin and length must not be negative");
  const int64_t N = length.has_value() ? *length : std::max<int64_t>(c.max_pages * c.page - begin, 0);
  TORCH_CHECK_VALUE(N <= INT32_MAX, "length is too large");
  const c10::cuda::CUDAGuard guard(c.dev);
  Tensor k = new_tensor({c.B, c.H, N, c.D}, at::kBFloat16, c.dev), v = new_tensor(k.sizes(), at::kBFloat16, c.dev);
  ok(qat_kv_cache_read(c.k, c.v, c.ks, c.vs, c.table, c.lens, k.mutable_data_ptr(), v.mutable_data_ptr(),
                       static_cast<int>(c.B), static_cast<int>(c.H), static_cast<int>(begin), static_cast<int>(N),
                       static_cast<int>(c.D), static_cast<int>(c.pages), static_cast<int>(c.page),
                       static_cast<int>(c.max_pages), stream_of(c.dev)),
     "qat_kv_cache_read");
  check_status(check, c.dev, "qat_kv_cache_read");
  return {k, v};
}

// Masks (parents) of a batch's trees: [B, T], or [T] for all sequences; the step from one to the next.
int64_t tree_stride(const Tensor& t, const char* name, at::ScalarType type, const at::Device& dev, int64_t B,
                    int64_t T) {
  TORCH_CHECK_VALUE(t.device() == dev, name, " must be a tensor on ", dev, ", got ", t.device());
  TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be torch.", type == at::kLong ? "int64" : "int32", ", got ",
                    t.scalar_type());
  const auto sz = t.sizes();
  TORCH_CHECK_VALUE((sz.size() == 1 && sz[0] == T) || (sz.size() == 2 && sz[0] == B && sz[1] == T), name,
                    " has shape ", sz, ", expected [", B, ", ", T, "] or [", T, "]");
  TORCH_CHECK_VALUE(T <= 1 || t.numel() == 0 || t.stride(-1) == 1, name, " must be contiguous along the tokens");
  with_memory(t, name);
  return sz.size() == 2 && B > 1 ? t.stride(0) : 0;
}

// With a tree: the last T tokens are drafted ones.
py::object decode(const Tensor& ck, const Tensor& cv, const Tensor& cks, const Tensor& cvs, const Tensor& q,
                  const Tensor& table, const Tensor& lens, const OptTensor& tree, std::optional<double> sm_scale,
                  int quant_mode, bool return_lse, const OptTensor& workspace, std::optional<bool> check,
                  std::optional<int64_t> window, int64_t sinks) {
  const char* what = tree.has_value() ? "qat_attention_tree" : "qat_attention_decode";
  const Cache c = cache_of(ck, cv, cks, cvs, table, lens);
  const Rows rq = rows(q, "q", c.dev, {c.B, -1, -1, c.D});
  TORCH_CHECK_VALUE(rq.dense, "q must be contiguous");
  no_gradient(what, q);
  no_tangent(what, {&q});
  TORCH_CHECK_VALUE(window.has_value() || sinks == 0, "sinks go together with a window");
  TORCH_CHECK_VALUE((!window.has_value() || *window >= 1) && sinks >= 0, "window must be at least 1 and sinks at "
                    "least 0, got ", window.value_or(1), " and ", sinks);
  const int64_t Hq = q.size(1), T = q.size(2);
  TORCH_CHECK_VALUE(Hq >= 1 && Hq % c.H == 0, Hq, " query heads do not share the cache's ", c.H, " evenly");
  const int64_t tree_sb = tree.has_value() ? tree_stride(*tree, "tree", at::kLong, c.dev, c.B, T) : 0;
  const auto limited = [](int64_t x) { return static_cast<int>(std::min<int64_t>(x, INT32_MAX)); };
  const c10::cuda::CUDAGuard guard(c.dev);
  const auto workspace_bytes = tree.has_value() ? qat_attn_tree_workspace_bytes : qat_attn_decode_workspace_bytes;
  const size_t bytes = workspace_bytes(static_cast<int>(Hq), static_cast<int>(c.H),
                                       static_cast<int>(std::min<int64_t>(T, 1 << 20)), static_cast<int>(c.D));
  const Tensor ws = workspace_or_new(workspace, std::max<int64_t>(static_cast<int64_t>(bytes), 256), c.dev);
  Tensor o = new_tensor(q.sizes(), at::kBFloat16, c.dev), lse;
  if (return_lse) lse = new_tensor({c.B, Hq, T}, at::kFloat, c.dev);
  float* lse_ptr = return_lse ? lse.mutable_data_ptr<float>() : nullptr;
  const int B = static_cast<int>(c.B), Hkv = static_cast<int>(c.H), D = static_cast<int>(c.D);
  const int pages = static_cast<int>(c.pages), page = static_cast<int>(c.page);
  const int max_pages = static_cast<int>(c.max_pages);
  const float scale = static_cast<float>(sm_scale.has_value() ? *sm_scale : 1.0 / std::sqrt(static_cast<double>(c.D)));
  const size_t ws_bytes = static_cast<size_t>(ws.numel());
  if (tree.has_value()) {
    what = "qat_attn_tree";
    ok(qat_attn_tree(q.const_data_ptr(), c.k, c.v, c.ks, c.vs, c.table, c.lens,
                     static_cast<const unsigned long long*>(tree->const_data_ptr()), tree_sb, o.mutable_data_ptr(),
                     lse_ptr, B, static_cast<int>(Hq), Hkv, static_cast<int>(T), D, pages, page, max_pages, scale,
                     limited(window.value_or(0)), limited(sinks), quant_mode, ws.mutable_data_ptr(), ws_bytes,
                     stream_of(c.dev)),
       what);
  } else if (window.has_value()) {
    what = "qat_attn_decode_window";
    ok(qat_attn_decode_window(q.const_data_ptr(), c.k, c.v, c.ks, c.vs, c.table, c.lens, o.mutable_data_ptr(),
                              lse_ptr, B, static_cast<int>(Hq), Hkv, static_cast<int>(T), D, pages, page, max_pages,
                              scale, limited(*window), limited(sinks), quant_mode, ws.mutable_data_ptr(), ws_bytes,
                              stream_of(c.dev)),
       what);
  } else {
    what = "qat_attn_decode";
    ok(qat_attn_decode(q.const_data_ptr(), c.k, c.v, c.ks, c.vs, c.table, c.lens, o.mutable_data_ptr(), lse_ptr, B,
                       static_cast<int>(Hq), Hkv, static_cast<int>(T), D, pages, page, max_pages, scale, quant_mode,
                       ws.mutable_data_ptr(), ws_bytes, stream_of(c.dev)),
       what);
  }
  check_status(check, c.dev, what);
  if (return_lse) return py::make_tuple(o, lse);
  return py::cast(o);
}

std::tuple<Tensor, Tensor> draft_tree(const Tensor& parents, const Tensor& lens) {
  on_cuda(parents, "parents");
  const at::Device dev = parents.device();
  const int* seq_lens = index_ptr(lens, "seq_lens", dev, -1, -2);
  const int64_t B = lens.size(0), T = parents.dim() > 0 ? parents.size(-1) : 0;
  const int64_t sb = tree_stride(parents, "parents", at::kInt, dev, B, T);
  TORCH_CHECK_VALUE(T <= 64, "a tree has at most 64 tokens, got ", T);
  TORCH_CHECK_VALUE(B <= INT32_MAX, "seq_lens is too large");
  const c10::cuda::CUDAGuard guard(dev);
  Tensor tree = new_tensor({B, T}, at::kLong, dev), positions = new_tensor({B, T}, at::kInt, dev);
  ok(qat_draft_tree(parents.const_data_ptr<int>(), sb, seq_lens,
                    static_cast<unsigned long long*>(tree.mutable_data_ptr()), positions.mutable_data_ptr<int>(),
                    static_cast<int>(B), static_cast<int>(T), stream_of(dev)),
     "qat_draft_tree");
  return {tree, positions};
}

Tensor kv_keep(const Tensor& ck, const Tensor& cv, const Tensor& cks, const Tensor& cvs, const Tensor& table,
               const Tensor& lens, int64_t T, const Tensor& path, const Tensor& path_lens,
               std::optional<bool> check) {
  const Cache c = cache_of(ck, cv, cks, cvs, table, lens);
  const int* rows_of = index_ptr(path, "path", c.dev, c.B, -1);
  const int64_t L = path.size(1);
  const int* kept = index_ptr(path_lens, "path_lens", c.dev, c.B, -2);
  TORCH_CHECK_VALUE(T >= 0 && T <= 64, "drafted must lie in 0 .. 64, got ", T);
  TORCH_CHECK_VALUE(L <= T, "path has ", L, " places for ", T, " drafted tokens");
  const c10::cuda::CUDAGuard guard(c.dev);
  Tensor out = new_tensor({c.B}, at::kInt, c.dev);
  ok(qat_kv_cache_keep(c.k, c.v, c.ks, c.vs, c.table, c.lens, rows_of, kept, out.mutable_data_ptr<int>(),
                       static_cast<int>(c.B), static_cast<int>(c.H), static_cast<int>(T), static_cast<int>(L),
                       static_cast<int>(c.D), static_cast<int>(c.pages), static_cast<int>(c.page),
                       static_cast<int>(c.max_pages), stream_of(c.dev)),
     "qat_kv_cache_keep");
  check_status(check, c.dev, "qat_kv_cache_keep");
  return out;
}

// ------------------------------------------------------------------------------- Python

// The arguments of a call, in order.  (Read here and not by generated casters: an append takes 3.0 us on the
// host, 3.35 with them.)
class Args {
 public:
  Args(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : a_(a) {
    TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n);
  }
  const Tensor& tensor() {
    PyObject* o = *a_++;
    TORCH_CHECK_TYPE(THPVariable_Check(o), "expected a tensor, got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
  }
  OptTensor optional_tensor() {
    if (none()) return std::nullopt;
    return tensor();
  }
  int64_t integer() {
    const long long x = PyLong_AsLongLong(*a_++);
    if (x == -1 && PyErr_Occurred()) throw py::error_already_set();
    return x;
  }
  std::optional<int64_t> optional_integer() {
    if (none()) return std::nullopt;
    return integer();
  }
  double real() {
    const double x = PyFloat_AsDouble(*a_++);
    if (x == -1.0 && PyErr_Occurred()) throw py::error_already_set();
    return x;
  }
  std::optional<double> optional_real() {
    if (none()) return std::nullopt;
    return real();
  }
  bool boolean() {
    const int x = PyObject_IsTrue(*a_++);
    if (x < 0) throw py::error_already_set();
    return x != 0;
  }
  std::optional<bool> optional_boolean() {
    if (none()) return std::nullopt;
    return boolean();
  }

 private:
  bool none() {
    if (*a_ != Py_None) return false;
    ++a_;
    return true;
  }
  PyObject* const* a_;
};

PyObject* py_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 10);
  const Tensor& q = a.tensor();
  const OptTensor k = a.optional_tensor(), positions = a.optional_tensor(), phases = a.optional_tensor(),
                  wq = a.optional_tensor(), wk = a.optional_tensor();
  const int64_t rotary_dim = a.integer();
  const bool interleaved = a.boolean();
  const double amplitude = a.real(), eps = a.real();
  return norm_rope(q, k, positions, phases, wq, wk, rotary_dim, interleaved, amplitude, eps).release().ptr();
  END_HANDLE_TH_ERRORS
}

PyObject* py_window_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 15);
  const Tensor &q = a.tensor(), &k = a.tensor(), &v = a.tensor();
  WindowTensors x;
  for (auto* list : {&x.by, &x.back})
    for (int i = 0; i < 3; ++i) {
      const OptTensor t = a.optional_tensor();
      (*list)[i] = t.has_value() ? *t : i == 0 ? q : i == 1 ? k : v;
    }
  x.k_mean = or_undefined(a.optional_tensor());
  const std::optional<double> sm_scale = a.optional_real();
  const int64_t quant_mode = a.integer(), window = a.integer(), sinks = a.integer();
  return py::cast(window_attention(q, k, v, x, sm_scale, quant_mode, window, sinks, a.optional_boolean()))
      .release()
      .ptr();
  END_HANDLE_TH_ERRORS
}

PyObject* py_kv_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 10);
  const Tensor &ck = a.tensor(), &cv = a.tensor(), &cks = a.tensor(), &cvs = a.tensor(), &k = a.tensor(),
               &v = a.tensor(), &table = a.tensor(), &lens = a.tensor();
  const OptTensor new_lens = a.optional_tensor();
  kv_append(ck, cv, cks, cvs, k, v, table, lens, new_lens, a.optional_boolean());
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

PyObject* py_kv_read(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 9);
  const Tensor &ck = a.tensor(), &cv = a.tensor(), &cks = a.tensor(), &cvs = a.tensor(), &table = a.tensor(),
               &lens = a.tensor();
  const int64_t begin = a.integer();
  const std::optional<int64_t> length = a.optional_integer();
  const auto out = kv_read(ck, cv, cks, cvs, table, lens, begin, length, a.optional_boolean());
  return py::make_tuple(std::get<0>(out), std::get<1>(out)).release().ptr();
  END_HANDLE_TH_ERRORS
}

PyObject* py_decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 15);
  const Tensor &ck = a.tensor(), &cv = a.tensor(), &cks = a.tensor(), &cvs = a.tensor(), &q = a.tensor(),
               &table = a.tensor(), &lens = a.tensor();
  const OptTensor tree = a.optional_tensor();
  const std::optional<double> sm_scale = a.optional_real();
  const int64_t quant_mode = a.integer();
  TORCH_CHECK_VALUE(quant_mode >= INT32_MIN && quant_mode <= INT32_MAX, "quant_mode ", quant_mode);
  const bool return_lse = a.boolean();
  const OptTensor workspace = a.optional_tensor();
  const std::optional<bool> check = a.optional_boolean();
  const std::optional<int64_t> window = a.optional_integer();
  return decode(ck, cv, cks, cvs, q, table, lens, tree, sm_scale, static_cast<int>(quant_mode), return_lse, workspace,
                check, window, a.integer())
      .release()
      .ptr();
  END_HANDLE_TH_ERRORS
}

PyObject* py_draft_tree(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 2);
  const Tensor &parents = a.tensor(), &lens = a.tensor();
  const auto out = draft_tree(parents, lens);
  return py::make_tuple(std::get<0>(out), std::get<1>(out)).release().ptr();
  END_HANDLE_TH_ERRORS
}

PyObject* py_kv_keep(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 10);
  const Tensor &ck = a.tensor(), &cv = a.tensor(), &cks = a.tensor(), &cvs = a.tensor(), &table = a.tensor(),
               &lens = a.tensor();
  const int64_t drafted = a.integer();
  const Tensor &path = a.tensor(), &path_lens = a.tensor();
  return py::cast(kv_keep(ck, cv, cks, cvs, table, lens, drafted, path, path_lens, a.optional_boolean()))
      .release()
      .ptr();
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

}  // namespace

PYBIND11_MODULE(_qat_torch, m) {
  m.def("norm_rope_bwd", &norm_rope_bwd);
  static PyMethodDef methods[] = {method<py_norm_rope>("norm_rope"), method<py_window_attention>("window_attention"),
                                  method<py_kv_append>("kv_append"), method<py_kv_read>("kv_read"),
                                  method<py_decode>("decode"), method<py_draft_tree>("draft_tree"),
                                  method<py_kv_keep>("kv_keep"),
                                  {nullptr, nullptr, 0, nullptr}};
  if (PyModule_AddFunctions(m.ptr(), methods) != 0) throw py::error_already_set();
}
