// calls.cpp -- the calls around the routed experts for Python: checks of torch tensors, their
// outputs and scratch, and the C ABI (include/moe.h) on the current stream, in one step each.
// Those calls take a few microseconds on the device, less than marshalling them through ctypes.
#define PY_SSIZE_T_CLEAN
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <Python.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <map>
#include <string>
#include <utility>

#include "../../include/moe.h"

namespace {

PyObject* g_error = nullptr;  // binding.MoeError(code, what)

// Raised as ValueError / TypeError by the entry points.
struct Refusal {
  PyObject* type;
  std::string what;
};
[[noreturn]] void refuse(const std::string& what) { throw Refusal{PyExc_ValueError, what}; }

#define CALL_BEGIN \
  HANDLE_TH_ERRORS \
  try {
#define CALL_END                                   \
  }                                                \
  catch (const Refusal& r) {                       \
    PyErr_SetString(r.type, r.what.c_str());       \
    return nullptr;                                \
  }                                                \
  END_HANDLE_TH_ERRORS

std::string shape_text(c10::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i)
    t += std::to_string(s[i]) + (s.size() == 1 ? "," : (i + 1 < s.size() ? ", " : ""));
  return t + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o))
    throw Refusal{PyExc_TypeError, std::string(name) + " must be a torch.Tensor"};
  return THPVariable_Unpack(o);
}
at::Tensor optional(PyObject* o, const char* name) {
  return o == Py_None ? at::Tensor() : tensor(o, name);
}
void need(const at::Tensor& t, const char* name, at::ScalarType dtype, c10::IntArrayRef shape) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t.scalar_type() != dtype)
    refuse(std::string(name) + " must have dtype " + c10::toString(dtype) + ", got " +
           c10::toString(t.scalar_type()));
  if (t.sizes() != shape)
    refuse(std::string(name) + " must have shape " + shape_text(shape) + ", got " +
           shape_text(t.sizes()));
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
}
void need_if(const at::Tensor& t, const char* name, at::ScalarType dtype,
             c10::IntArrayRef shape, const at::Tensor& like) {
  if (!t.defined()) return;
  need(t, name, dtype, shape);
  if (t.device() != like.device()) refuse(std::string(name) + " is on another device");
}
void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

int dtype_code(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return MOE_BF16;
  if (t.scalar_type() == at::kHalf) return MOE_F16;
  refuse(std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
}
int as_int(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return (int)v;
}
float as_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)v;
}
bool as_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
int length(int64_t n) {
  if (n > INT32_MAX) refuse("a dimension is over 2^31 - 1");
  return (int)n;
}

bool failed(moe_status_t rc, const char* what) {
  if (rc == MOE_OK) return false;
  PyObject* e = PyObject_CallFunction(g_error, "is", (int)rc, what);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return true;
}

// An output on `like`'s device (current).
at::Tensor fresh(const at::Tensor& like, c10::IntArrayRef shape, at::ScalarType dtype) {
  return at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt);
}
at::Tensor fresh(const at::Tensor& like) { return fresh(like, like.sizes(), like.scalar_type()); }

// Small outputs share one allocation: contiguous tensors of `base`'s storage, `offset` in elements.
at::Tensor part_of(const at::Tensor& base, int64_t offset, c10::IntArrayRef shape,
                   at::ScalarType dtype) {
  auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(),
                                                   c10::scalarTypeToTypeMeta(dtype));
  impl->set_storage_offset(offset);
  impl->set_sizes_contiguous(shape);
  return at::Tensor(std::move(impl));
}

at::Tensor zeros(int64_t bytes, c10::Device dev) {
  return at::zeros({bytes}, at::TensorOptions().dtype(at::kByte).device(dev));
}

constexpr int64_t kHeader = 256;  // of every workspace: the status word first

// Scratch of the current stream: one per stream, since calls on other streams may run at the same
// time, and never freed while a call may still use it (a larger one replaces it, with what was
// reported so far; torch's allocator reuses the memory in the stream's order).  Host threads share it: a call holds the interpreter's
// lock from here to its last launch, so the launches of two calls do not mix.  A captured call gets
// its own, which lives in the graph's memory.
at::Tensor scratch(int64_t bytes, const c10::cuda::CUDAStream& s) {
  if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None)
    return zeros(bytes, s.device());
  using Key = std::pair<int, int64_t>;
  // leaked on purpose: a destructor at the process' end may find no CUDA context
  static auto* cache = new std::map<Key, at::Tensor>();
  at::Tensor& t = (*cache)[Key(s.device_index(), (int64_t)(intptr_t)s.stream())];
  if (!t.defined() || t.numel() < bytes) {
    at::Tensor larger = zeros(std::max(bytes, kHeader), s.device());
    if (t.defined()) larger.narrow(0, 0, kHeader).copy_(t.narrow(0, 0, kHeader));
    t = std::move(larger);
  }
  return t;
}
// The caller's workspace, or scratch of at least `bytes` bytes.
at::Tensor workspace(PyObject* o, int64_t bytes, const c10::cuda::CUDAStream& s) {
  if (o == Py_None) return scratch(bytes, s);
  const at::Tensor& t = tensor(o, "workspace");
  if (!t.is_cuda() || t.scalar_type() != at::kByte || !t.is_contiguous())
    refuse("workspace must be a contiguous uint8 CUDA tensor");
  if (t.device() != s.device()) refuse("workspace is on another device");
  return t;
}

c10::cuda::CUDAStream stream_of(const at::Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(t.device().index());
}

void arguments(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) throw Refusal{PyExc_TypeError, "wrong number of arguments"};
}

// scratch(nbytes, device index): the current stream's scratch.
PyObject* call_scratch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  CALL_BEGIN
  arguments(n, 2);
  const c10::DeviceIndex dev = (c10::DeviceIndex)as_int(a[1]);
  c10::cuda::CUDAGuard guard(dev);
  return THPVariable_Wrap(scratch(as_int(a[0]), c10::cuda::getCurrentCUDAStream(dev)));
  CALL_END
}

// linear(x, w, bias, act, residual, out_f32, out, workspace)
PyObject* call_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  CALL_BEGIN
  arguments(n, 8);
  const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w");
  const at::Tensor bias = optional(a[2], "bias"), res = optional(a[4], "residual");
  at::Tensor out = optional(a[6], "out");
  if (x.dim() != 2 || w.dim() != 2) refuse("x and w must have two dimensions");
  moe_linear_t g;
  g.dtype = dtype_code(x);
  g.T = length(x.size(0));
  g.K = length(x.size(1));
  g.N = length(w.size(0));
  g.activation = as_int(a[3]);
  g.out_f32 = as_bool(a[5]);
  const at::ScalarType dt = x.scalar_type(), odt = g.out_f32 ? at::kFloat : dt;
  need(x, "x", dt, {g.T, g.K});
  need_if(w, "w", dt, {g.N, g.K}, x);
  need_if(bias, "bias", dt, {g.N}, x);
  need_if(res, "residual", odt, {g.T, g.N}, x);
  need_if(out, "out", odt, {g.T, g.N}, x);
  c10::cuda::CUDAGuard guard(x.device());
  const auto s = stream_of(x);
  if (!out.defined()) out = fresh(x, {g.T, g.N}, odt);
  const at::Tensor ws = workspace(a[7], (int64_t)moe_linear_workspace_size(&g), s);
  if (failed(moe_linear(&g, ptr(x), ptr(w), ptr(bias), ptr(res), ptr(out), ptr(ws),
                        (size_t)ws.numel(), s.stream()),
             "moe_linear"))
    return nullptr;
  return THPVariable_Wrap(std::move(out));
  CALL_END
}

// The options and inputs of the norm: branch, residual, gate, post_weight, pre_weight, post, pre,
// residual_scale, weight_offset, eps, gate kind (moe_gate_t, or -1: by the gate's shape).
struct Norm {
  at::Tensor y, x, g, wq, wp;
  moe_block_norm_t p;
  explicit Norm(PyObject* const* a) {
    y = tensor(a[0], "branch");
    x = optional(a[1], "residual");
    g = optional(a[2], "gate");
    wq = optional(a[3], "post_weight");
    wp = optional(a[4], "pre_weight");
    if (y.dim() != 2) refuse("branch must have two dimensions");
    p.dtype = dtype_code(y);
    p.T = length(y.size(0));
    p.H = length(y.size(1));
    p.post_norm = as_bool(a[5]);
    p.pre_norm = as_bool(a[6]);
    p.residual_scale = as_float(a[7]);
    p.weight_offset = as_float(a[8]);
    p.eps = as_float(a[9]);
    const at::ScalarType dt = y.scalar_type();
    need(y, "branch", dt, {p.T, p.H});
    need_if(x, "residual", dt, {p.T, p.H}, y);
    need_if(wq, "post_weight", dt, {p.H}, y);
    need_if(wp, "pre_weight", dt, {p.H}, y);
    p.gate = as_int(a[10]);
    if (!g.defined()) {
      if (p.gate >= 0) refuse("gate_kind is given without a gate");
      p.gate = MOE_GATE_NONE;
    } else {
      if (p.gate < 0) p.gate = by_shape();
      if (p.gate == MOE_GATE_CHANNEL)
        need_if(g, "gate", dt, {p.H}, y);
      else if (p.gate == MOE_GATE_ELEMENT)
        need_if(g, "gate", dt, {p.T, p.H}, y);
      else if (g.dim() == 1)
        need_if(g, "gate", dt, {p.T}, y);
      else
        need_if(g, "gate", dt, {p.T, 1}, y);
    }
  }

 private:
  // One dimension: its length tells, unless there are as many rows as channels.
  int by_shape() const {
    if (g.dim() == 1 && g.size(0) == p.H && p.T == p.H)
      refuse("a gate of T = H values may be one per channel or per token: give gate_kind");
    if (g.dim() == 1) return g.size(0) == p.H ? MOE_GATE_CHANNEL : MOE_GATE_TOKEN;
    return g.dim() == 2 && g.size(1) == 1 ? MOE_GATE_TOKEN : MOE_GATE_ELEMENT;
  }
};

// block_norm(<Norm>, stream_out, want_stream) -> (stream, normed)
PyObject* call_block_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  CALL_BEGIN
  arguments(n, 13);
  const Norm m(a);
  at::Tensor r = optional(a[11], "stream_out"), h;
  need_if(r, "stream_out", m.y.scalar_type(), m.y.sizes(), m.y);
  c10::cuda::CUDAGuard guard(m.y.device());
  if (!r.defined() && as_bool(a[12])) r = fresh(m.y);
  if (m.p.pre_norm) h = fresh(m.y);
  if (failed(moe_block_norm_fwd(&m.p, ptr(m.y), ptr(m.x), ptr(m.g), ptr(m.wq), ptr(m.wp), ptr(r),
                                ptr(h), stream_of(m.y).stream()),
             "moe_block_norm_fwd"))
    return nullptr;
  PyObject* out = PyTuple_New(2);
  if (!out) return nullptr;
  PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(r));  // None where it is undefined
  PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(h));
  return out;
  CALL_END
}

bool put(PyObject* dict, const char* key, const at::Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  if (!o) return false;
  const int rc = PyDict_SetItemString(dict, key, o);
  Py_DECREF(o);
  return rc == 0;
}

// block_norm_bwd(<Norm>, d_stream, d_normed, workspace) -> dict
PyObject* call_block_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  CALL_BEGIN
  arguments(n, 14);
  const Norm m(a);
  const at::Tensor dr = optional(a[11], "d_stream"), dh = optional(a[12], "d_normed");
  if (dh.defined() != (m.p.pre_norm != 0)) refuse("d_normed goes with pre_norm");
  need_if(dr, "d_stream", m.y.scalar_type(), m.y.sizes(), m.y);
  need_if(dh, "d_normed", m.y.scalar_type(), m.y.sizes(), m.y);
  c10::cuda::CUDAGuard guard(m.y.device());
  const auto s = stream_of(m.y);
  const at::Tensor ws = workspace(a[13], (int64_t)moe_block_norm_bwd_workspace_size(&m.p), s);
  auto like = [](const at::Tensor& t) { return t.defined() ? fresh(t) : at::Tensor(); };
  const at::Tensor dy = like(m.y), dx = like(m.x);
  at::Tensor dg, dq, dp;  // the per-channel ones lie in one allocation
  const bool gc = m.p.gate == MOE_GATE_CHANNEL;
  const int chans = gc + m.wq.defined() + m.wp.defined();
  if (chans > 0) {
    const at::ScalarType dt = m.y.scalar_type();
    const at::Tensor all = fresh(m.y, {(int64_t)chans * m.p.H}, dt);
    int64_t at = 0;
    for (auto [have, d] : {std::pair<bool, at::Tensor*>(gc, &dg), {m.wq.defined(), &dq},
                           {m.wp.defined(), &dp}})
      if (have) {
        *d = part_of(all, at, {m.p.H}, dt);
        at += m.p.H;
      }
  }
  if (!gc) dg = like(m.g);
  if (failed(moe_block_norm_bwd(&m.p, ptr(dr), ptr(dh), ptr(m.y), ptr(m.x), ptr(m.g), ptr(m.wq),
                                ptr(m.wp), ptr(dy), ptr(dx), ptr(dg), ptr(dq), ptr(dp), ptr(ws),
                                (size_t)ws.numel(), s.stream()),
             "moe_block_norm_bwd"))
    return nullptr;
  PyObject* out = PyDict_New();
  if (!out) return nullptr;
  if (put(out, "d_branch", dy) && (!dx.defined() || put(out, "d_residual", dx)) &&
      (!dg.defined() || put(out, "d_gate", dg)) &&
      (!dq.defined() || put(out, "d_post_weight", dq)) &&
      (!dp.defined() || put(out, "d_pre_weight", dp)))
    return out;
  Py_DECREF(out);
  return nullptr;
  CALL_END
}

// gating_output, topk_ids, seq_offsets, scoring, renormalize, routed_scaling_factor
struct Router {
  at::Tensor x, ids, off;
  moe_problem_t p = {};
  int n_seq = 1;
  explicit Router(PyObject* const* a) {
    x = tensor(a[0], "gating_output");
    ids = tensor(a[1], "topk_ids");
    off = optional(a[2], "seq_offsets");
    if (x.dim() != 2 || ids.dim() != 2)
      refuse("gating_output and topk_ids must have two dimensions");
    p.T = length(x.size(0));
    p.E = length(x.size(1));
    p.top_k = length(ids.size(1));
    p.H = p.F = 8;  // not used here
    p.dtype = MOE_BF16;
    p.scoring = as_int(a[3]);
    p.renormalize = as_bool(a[4]);
    p.routed_scaling_factor = as_float(a[5]);
    need(x, "gating_output", at::kFloat, {p.T, p.E});
    need_if(ids, "topk_ids", at::kInt, {p.T, p.top_k}, x);
    if (off.defined()) {
      if (off.dim() != 1 || off.size(0) < 2) refuse("seq_offsets must hold n_seq + 1 offsets");
      n_seq = length(off.size(0) - 1);
      need_if(off, "seq_offsets", at::kInt, {n_seq + 1}, x);
    }
  }
  const float* logits() const { return static_cast<const float*>(ptr(x)); }
  const int32_t* routes() const { return static_cast<const int32_t*>(ptr(ids)); }
  const int32_t* offsets() const { return static_cast<const int32_t*>(ptr(off)); }
};

// balance_loss(<Router>, coeff, workspace) -> dict
PyObject* call_balance_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  CALL_BEGIN
  arguments(n, 8);
  const Router r(a);
  c10::cuda::CUDAGuard guard(r.x.device());
  const auto s = stream_of(r.x);
  const at::Tensor ws =
      workspace(a[7], (int64_t)moe_balance_loss_workspace_size(&r.p, r.n_seq), s);
  // prob_sum, coef, counts, live_tokens, loss: 32-bit values, each on a 16-byte boundary
  const int64_t table = ((int64_t)r.n_seq * r.p.E + 3) / 4 * 4, few = (r.n_seq + 3) / 4 * 4;
  const at::Tensor all = fresh(r.x, {3 * table + few + 1}, at::kFloat);
  const at::Tensor sums = part_of(all, 0, {r.n_seq, r.p.E}, at::kFloat),
                   coef = part_of(all, table, {r.n_seq, r.p.E}, at::kFloat),
                   counts = part_of(all, 2 * table, {r.n_seq, r.p.E}, at::kInt),
                   live = part_of(all, 3 * table, {r.n_seq}, at::kInt),
                   loss = part_of(all, 3 * table + few, {1}, at::kFloat);
  if (failed(moe_balance_loss_fwd(&r.p, r.n_seq, as_float(a[6]), r.logits(), r.routes(),
                                  r.offsets(), static_cast<float*>(ptr(loss)),
                                  static_cast<int32_t*>(ptr(counts)),
                                  static_cast<int32_t*>(ptr(live)),
                                  static_cast<float*>(ptr(sums)),
                                  static_cast<float*>(ptr(coef)), ptr(ws), (size_t)ws.numel(),
                                  s.stream()),
             "moe_balance_loss_fwd"))
    return nullptr;
  PyObject* out = PyDict_New();
  if (!out) return nullptr;
  if (put(out, "loss", loss) && put(out, "counts", counts) && put(out, "live_tokens", live) &&
      put(out, "prob_sum", sums) && put(out, "coef", coef))
    return out;
  Py_DECREF(out);
  return nullptr;
  CALL_END
}

// router_bwd(<Router>, d_topk_weights, coef, d_loss, out) -> d_gating_output
PyObject* call_router_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  CALL_BEGIN
  arguments(n, 10);
  const Router r(a);
  const at::Tensor dw = optional(a[6], "d_topk_weights"), coef = optional(a[7], "coef"),
                   dl = optional(a[8], "d_loss");
  at::Tensor out = optional(a[9], "out");
  need_if(dw, "d_topk_weights", at::kFloat, {r.p.T, r.p.top_k}, r.x);
  need_if(coef, "coef", at::kFloat, {r.n_seq, r.p.E}, r.x);
  need_if(out, "out", at::kFloat, {r.p.T, r.p.E}, r.x);
  if (dl.defined()) {
    if (dl.numel() != 1) refuse("d_loss must hold one value");
    need_if(dl, "d_loss", at::kFloat, dl.sizes(), r.x);
  }
  c10::cuda::CUDAGuard guard(r.x.device());
  if (!out.defined()) out = fresh(r.x);
  if (failed(moe_router_bwd(&r.p, r.n_seq, r.logits(), r.routes(),
                            static_cast<const float*>(ptr(dw)),
                            static_cast<const float*>(ptr(coef)), r.offsets(),
                            static_cast<const float*>(ptr(dl)), static_cast<float*>(ptr(out)),
                            stream_of(r.x).stream()),
             "moe_router_bwd"))
    return nullptr;
  return THPVariable_Wrap(std::move(out));
  CALL_END
}

// set_error(class): what a status other than MOE_OK raises.
PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL,
          nullptr};
}
PyMethodDef g_methods[] = {
    method<call_scratch>("scratch"),
    method<call_linear>("linear"),
    method<call_block_norm>("block_norm"),
    method<call_block_norm_bwd>("block_norm_bwd"),
    method<call_balance_loss>("balance_loss"),
    method<call_router_bwd>("router_bwd"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "gb300moe_calls", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gb300moe_calls() { return PyModule_Create(&g_module); }
