// Python side of the serving steps, the norms with rotation and residual, linear attention and a step's maps: checks the tensors, allocates
// the outputs and calls the C ABI (include/gdn.h). These calls are short (a decoding step takes a few
// microseconds on the GPU), so their argument marshalling is native: a step's host time is 4 to 6 us
// instead of 10 to 16 us with the same checks written in Python.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/Storage.h>
#include <c10/core/TensorImpl.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <exception>
#include <optional>

#include "gdn.h"

namespace {

using at::Tensor;

// The library's entry points, by the addresses that the package hands over (no link to the library).
struct Entries {
  decltype(&gdn_recurrent) recurrent;
  decltype(&gdn_conv_step) conv_step;
  decltype(&gdn_qk_rope_fwd) rope_fwd;
  decltype(&gdn_qk_rope_bwd) rope_bwd;
  decltype(&gdn_qk_rope_workspace_bytes) rope_workspace;
  decltype(&gdn_last_error) last_error;
  decltype(&gdn_linear_fwd) linear_fwd;
  decltype(&gdn_linear_bwd) linear_bwd;
  decltype(&gdn_linear_workspace_bytes) linear_workspace;
  decltype(&gdn_linear_step) linear_step;
  decltype(&gdn_rms_norm_fwd) norm_fwd;
  decltype(&gdn_rms_norm_bwd) norm_bwd;
  decltype(&gdn_rms_norm_workspace_bytes) norm_workspace;
  decltype(&gdn_step_maps) step_maps;
} g_lib;
constexpr int ENTRIES = sizeof(Entries) / sizeof(void*);
PyObject* g_error = nullptr; // the package's GdnError

struct Raised {}; // a Python exception is set

[[noreturn]] void raise(int code, const char* msg) {
  PyObject* e = PyObject_CallFunction(g_error, "is", code, msg);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

[[noreturn]] void refuse(const char* fmt, ...) {
  char buf[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  raise(GDN_EINVAL, buf);
}

void check(int rc) {
  if (rc != GDN_OK) raise(rc, g_lib.last_error());
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s is not a tensor", name);
  return THPVariable_Unpack(o);
}

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

// The tensor's address. Refuses it unless it has this shape, type and device and is contiguous or,
// where `stride` is given, contiguous but for the distance between its first dimension's entries,
// which goes there (0: contiguous).
void* expect(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Device& dev,
             int64_t* stride = nullptr) {
  if (t.sizes() != shape)
    refuse("%s has shape %s, expected %s", name, text(t.sizes()).c_str(), text(shape).c_str());
  if (t.scalar_type() != type)
    refuse("%s has type %s, expected %s", name, c10::toString(t.scalar_type()), c10::toString(type));
  if (t.device() != dev) refuse("%s is on %s, expected %s", name, t.device().str().c_str(), dev.str().c_str());
  if (stride) *stride = 0;
  if (!t.is_contiguous()) {
    bool rows = stride != nullptr;
    int64_t below = 1;
    for (int64_t d = t.dim() - 1; d >= 1 && rows; --d) {
      rows = t.size(d) == 1 || t.stride(d) == below;
      below *= t.size(d);
    }
    if (!rows || t.stride(0) < below) refuse("%s is not contiguous%s", name, stride ? " within a token" : "");
    *stride = t.stride(0);
  }
  return t.data_ptr();
}

template <typename T>
T* optional(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Device& dev) {
  return o == Py_None ? nullptr : (T*)expect(tensor(o, name), name, shape, type, dev);
}

Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Device& dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

// A call's tensors that the caller did not give. An allocation and its release take 0.8 us of the
// host; a decoding step with three outputs took 5.9 us, and 3.3 with the outputs given. So those of a
// short call are parts of one allocation, a workspace that the caller did not give among them. One part keeps
// all of it alive: up to SHARED bytes, which is nothing beside what the allocator rounds up, or up to what the call
// names instead (step_maps: more, since a step's maps are used and dropped together).
class Buffers {
 public:
  explicit Buffers(const at::Device& dev, int64_t shared = SHARED) : dev_(dev), shared_(shared) {}
  // t becomes o, or is made by allocate()
  void want(Tensor& t, PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type) {
    if (o != Py_None) t = tensor(o, name);
    else want(t, shape, type);
  }
  void want(Tensor& t, at::IntArrayRef shape, at::ScalarType type) {
    int64_t bytes = (int64_t)c10::elementSize(type);
    for (const int64_t x : shape) bytes *= x;
    wants_[n_++] = {&t, at::DimVector(shape.begin(), shape.end()), type, total_};
    total_ += (bytes + ALIGN - 1) / ALIGN * ALIGN;
  }
  void allocate() {
    Tensor all;
    if (n_ > 1 && total_ > 0 && total_ <= shared_) all = empty({total_}, at::kByte, dev_);
    for (int i = 0; i < n_; ++i) {
      const Want& w = wants_[i];
      if (!all.defined()) {
        *w.to = empty(w.shape, w.type, dev_);
        continue;
      }
      *w.to = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), c10::scalarTypeToTypeMeta(w.type));
      c10::TensorImpl* t = w.to->unsafeGetTensorImpl();
      t->set_storage_offset(w.from / (int64_t)c10::elementSize(w.type));
      t->set_sizes_contiguous(w.shape);
    }
  }

 private:
  static constexpr int64_t ALIGN = 512, SHARED = 1 << 20;
  struct Want {
    Tensor* to;
    at::DimVector shape;
    at::ScalarType type;
    int64_t from; // bytes
  };
  at::Device dev_;
  int64_t shared_; // bytes up to which the outputs share one allocation
  Want wants_[10];
  int n_ = 0;
  int64_t total_ = 0;
};

const at::Device gpu_of(const Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse("%s is on %s, expected a GPU", name, t.device().str().c_str());
  return t.device();
}
void* stream_of(const at::Device& dev) { return c10::hip::getCurrentHIPStream(dev.index()).stream(); }
at::ScalarType io_type(int dtype) { return dtype == GDN_DTYPE_BF16 ? at::kBFloat16 : at::kFloat; }

template <typename P>
P problem(PyObject* address) {
  void* at = PyLong_AsVoidPtr(address);
  if (!at) throw Raised{};
  return *(const P*)at;
}

// Runs f with C++ exceptions turned into the Python ones that torch makes of them (an allocation that
// fails is a torch.OutOfMemoryError, as where the package allocates in Python).
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Raised&) {
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse("%zd arguments, expected %zd", n, want);
}

// recurrent(problem, q, k, v, g, beta, states, slot_in, slot_out, slot_tok, cu_seqlens, o) -> o
PyObject* recurrent(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 12);
    gdn_recurrent_problem p = problem<gdn_recurrent_problem>(a[0]);
    const Tensor& v = tensor(a[3], "v");
    const at::Device dev = gpu_of(v, "v");
    const c10::DeviceGuard guard(dev);
    const at::ScalarType io = io_type(p.dtype);
    const int64_t T = p.n_tokens, N = p.n_seqs;
    const int64_t qs[] = {T, p.h_qk, p.d}, vs[] = {T, p.h_v, p.d}, gs[] = {T, p.h_v}, ss[] = {p.n_slots, p.h_v, p.d, p.d};
    void* vp = expect(v, "v", vs, io, dev, &p.v_stride);
    void* qp = expect(tensor(a[1], "q"), "q", qs, io, dev, &p.q_stride);
    void* kp = expect(tensor(a[2], "k"), "k", qs, io, dev, &p.k_stride);
    void* gp = expect(tensor(a[4], "g"), "g", gs, at::kFloat, dev);
    void* bp = expect(tensor(a[5], "beta"), "beta", gs, at::kFloat, dev);
    void* sp = expect(tensor(a[6], "states"), "states", ss, at::kFloat, dev);
    void* in = expect(tensor(a[7], "slot_in"), "slot_in", {N}, at::kInt, dev);
    void* out = expect(tensor(a[8], "slot_out"), "slot_out", {N}, at::kInt, dev);
    const int32_t* tok = optional<int32_t>(a[9], "slot_tok", {T}, at::kInt, dev);
    const int32_t* cu = optional<int32_t>(a[10], "cu_seqlens", {N + 1}, at::kInt, dev);
    const Tensor o = a[11] == Py_None ? empty(vs, io, dev) : tensor(a[11], "o");
    void* op = expect(o, "o", vs, io, dev);
    check(g_lib.recurrent(&p, qp, kp, vp, (float*)gp, (float*)bp, cu, (int32_t*)in, (int32_t*)out, tok, (float*)sp, op,
                          stream_of(dev)));
    return THPVariable_Wrap(o);
  });
}

// conv_step(problem, x, weight, bias, windows, slot_in, slot_out, slot_tok, cu_seqlens, outs) -> outs
PyObject* conv_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 10);
    gdn_conv_step_problem p = problem<gdn_conv_step_problem>(a[0]);
    const Tensor& x = tensor(a[1], "x");
    const at::Device dev = gpu_of(x, "x");
    const c10::DeviceGuard guard(dev);
    const at::ScalarType io = io_type(p.dtype);
    const int64_t T = p.n_tokens, N = p.n_seqs, C = p.channels, W = p.width;
    void* xp = expect(x, "x", {T, C}, io, dev, &p.x_stride);
    void* wp = expect(tensor(a[2], "weight"), "weight", {C, W}, at::kFloat, dev);
    const float* bp = optional<float>(a[3], "bias", {C}, at::kFloat, dev);
    void* win = optional<void>(a[4], "windows", {p.n_slots, W - 1, C}, io, dev);
    void* in = expect(tensor(a[5], "slot_in"), "slot_in", {N}, at::kInt, dev);
    void* out = expect(tensor(a[6], "slot_out"), "slot_out", {N}, at::kInt, dev);
    const int32_t* tok = optional<int32_t>(a[7], "slot_tok", {T}, at::kInt, dev);
    const int32_t* cu = optional<int32_t>(a[8], "cu_seqlens", {N + 1}, at::kInt, dev);
    for (int i = 0; i < p.n_groups && i < 4; ++i)
      if (p.group_channels[i] < 0) refuse("group %d has %d channels", i, (int)p.group_channels[i]);
    const bool given = a[9] != Py_None;
    if (given && (!PyList_Check(a[9]) || PyList_GET_SIZE(a[9]) != p.n_groups))
      refuse("outs has to be a list of %d tensors", p.n_groups);
    Tensor ys[4];
    void* yp[4] = {};
    Buffers made(dev);
    for (int i = 0; i < p.n_groups && i < 4; ++i)
      made.want(ys[i], given ? PyList_GET_ITEM(a[9], i) : Py_None, "outs", {T, p.group_channels[i]}, io);
    made.allocate();
    for (int i = 0; i < p.n_groups && i < 4; ++i) yp[i] = expect(ys[i], "outs", {T, p.group_channels[i]}, io, dev);
    check(g_lib.conv_step(&p, xp, (float*)wp, bp, cu, (int32_t*)in, (int32_t*)out, tok, win, yp, stream_of(dev)));
    if (given) {
      Py_INCREF(a[9]);
      return a[9];
    }
    PyObject* list = PyList_New(p.n_groups);
    for (int i = 0; list && i < p.n_groups; ++i) PyList_SET_ITEM(list, i, THPVariable_Wrap(ys[i]));
    return list;
  });
}

// What both directions of the rotation read.
struct RopeInputs {
  const int32_t* pos;
  const uint64_t* freqs;
  const float *wq, *wk;
  RopeInputs(const gdn_qk_rope_problem& p, PyObject* const* a, const at::Device& dev) {
    pos = optional<int32_t>(a[0], "positions", {p.n_tokens}, at::kInt, dev);
    freqs = optional<uint64_t>(a[1], "freqs", {p.rotary_dim / 2}, at::kLong, dev);
    wq = optional<float>(a[2], "q_weight", {p.d}, at::kFloat, dev);
    wk = optional<float>(a[3], "k_weight", {p.d}, at::kFloat, dev);
  }
};

PyObject* wrap_or_none(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

// rope_fwd(problem, q, k, positions, freqs, q_weight, k_weight, q_out, k_out) -> (q_out, k_out)
PyObject* rope_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 9);
    gdn_qk_rope_problem p = problem<gdn_qk_rope_problem>(a[0]);
    const Tensor& q = tensor(a[1], "q");
    const at::Device dev = gpu_of(q, "q");
    const c10::DeviceGuard guard(dev);
    const at::ScalarType io = io_type(p.dtype);
    const int64_t qs[] = {p.n_tokens, p.h_q, p.d}, ks[] = {p.n_tokens, p.h_k, p.d};
    void* qp = expect(q, "q", qs, io, dev, &p.q_stride);
    void* kp = a[2] == Py_None ? nullptr : expect(tensor(a[2], "k"), "k", ks, io, dev, &p.k_stride);
    const RopeInputs r(p, a + 3, dev);
    Tensor qo, ko;
    Buffers made(dev);
    made.want(qo, a[7], "q_out", qs, io);
    if (a[2] != Py_None) made.want(ko, a[8], "k_out", ks, io);
    made.allocate();
    void* qop = expect(qo, "q_out", qs, io, dev, &p.qo_stride);
    void* kop = ko.defined() ? expect(ko, "k_out", ks, io, dev, &p.ko_stride) : nullptr;
    check(g_lib.rope_fwd(&p, qp, kp, r.pos, r.freqs, r.wq, r.wk, qop, kop, stream_of(dev)));
    return Py_BuildValue("NN", THPVariable_Wrap(qo), wrap_or_none(ko));
  });
}

// rope_bwd(problem, q, k, positions, freqs, q_weight, k_weight, dq_out, dk_out, dq, dk, dq_weight, dk_weight,
//          workspace) -> (dq, dk, dq_weight, dk_weight)
PyObject* rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 14);
    gdn_qk_rope_problem p = problem<gdn_qk_rope_problem>(a[0]);
    const Tensor& dqo = tensor(a[7], "dq_out");
    const at::Device dev = gpu_of(dqo, "dq_out");
    const c10::DeviceGuard guard(dev);
    const at::ScalarType io = io_type(p.dtype);
    const int64_t qs[] = {p.n_tokens, p.h_q, p.d}, ks[] = {p.n_tokens, p.h_k, p.d};
    const auto rows = [&](PyObject* o, const char* name, at::IntArrayRef shape, int64_t* stride) -> void* {
      return o == Py_None ? nullptr : expect(tensor(o, name), name, shape, io, dev, stride);
    };
    void* qp = rows(a[1], "q", qs, &p.q_stride);
    void* kp = rows(a[2], "k", ks, &p.k_stride);
    void* dqop = rows(a[7], "dq_out", qs, &p.qo_stride);
    void* dkop = rows(a[8], "dk_out", ks, &p.ko_stride);
    const RopeInputs r(p, a + 3, dev);
    Tensor dq, dk, dwq, dwk, ws;
    Buffers made(dev);
    made.want(dq, a[9], "dq", qs, io);
    const bool with_k = a[8] != Py_None; // (of no tokens the addresses are NULL)
    if (with_k) made.want(dk, a[10], "dk", ks, io);
    if (r.wq) made.want(dwq, a[11], "dq_weight", {p.d}, at::kFloat);
    if (r.wk) made.want(dwk, a[12], "dk_weight", {p.d}, at::kFloat);
    size_t bytes = 0;
    if (a[13] != Py_None) {
      ws = tensor(a[13], "workspace");
      bytes = (size_t)ws.numel();
      expect(ws, "workspace", {ws.numel()}, at::kByte, dev);
    } else if (r.wq || r.wk) {
      bytes = g_lib.rope_workspace(&p);
      if (!bytes) raise(GDN_EINVAL, g_lib.last_error());
      made.want(ws, {(int64_t)bytes}, at::kByte);
    }
    made.allocate();
    void* dqp = expect(dq, "dq", qs, io, dev, &p.dq_stride);
    void* dkp = with_k ? expect(dk, "dk", ks, io, dev, &p.dk_stride) : nullptr;
    float* dwqp = r.wq ? (float*)expect(dwq, "dq_weight", {p.d}, at::kFloat, dev) : nullptr;
    float* dwkp = r.wk ? (float*)expect(dwk, "dk_weight", {p.d}, at::kFloat, dev) : nullptr;
    check(g_lib.rope_bwd(&p, qp, kp, r.pos, r.freqs, r.wq, r.wk, dqop, dkop, dqp, dkp, dwqp, dwkp,
                         ws.defined() ? ws.data_ptr() : nullptr, bytes, stream_of(dev)));
    return Py_BuildValue("NNNN", THPVariable_Wrap(dq), wrap_or_none(dk), wrap_or_none(dwq), wrap_or_none(dwk));
  });
}

// The problem's workspace: `given`, or one of the size that `bytes` names, among the call's buffers.
struct Workspace {
  Tensor t;
  size_t bytes = 0;
  template <typename F>
  Workspace(PyObject* given, const at::Device& dev, Buffers& made, F needed) {
    if (given != Py_None) {
      t = tensor(given, "workspace");
      bytes = (size_t)t.numel();
      expect(t, "workspace", {t.numel()}, at::kByte, dev);
      return;
    }
    bytes = needed();
    if (!bytes) raise(GDN_EINVAL, g_lib.last_error());
    made.want(t, {(int64_t)bytes}, at::kByte);
  }
};

// What both directions of linear attention read, with the strides put into the problem.
struct LinearInputs {
  void *q, *k, *v;
  const float *g, *h0;
  const int32_t* cu;
  LinearInputs(gdn_linear_problem& p, PyObject* const* a, const at::Device& dev) {
    const at::ScalarType io = io_type(p.dtype);
    const int64_t T = p.n_tokens, N = p.n_seqs;
    const int64_t qs[] = {T, p.h_qk, p.d}, vs[] = {T, p.h_v, p.d}, ss[] = {N, p.h_v, p.d, p.d}, gs[] = {T, p.h_v};
    q = expect(tensor(a[0], "q"), "q", qs, io, dev, &p.q_stride);
    k = expect(tensor(a[1], "k"), "k", qs, io, dev, &p.k_stride);
    v = expect(tensor(a[2], "v"), "v", vs, io, dev, &p.v_stride);
    const at::IntArrayRef shape = p.decay == GDN_DECAY_HEAD ? at::IntArrayRef(gs + 1, 1) : at::IntArrayRef(gs);
    g = (float*)expect(tensor(a[3], "g"), "g", shape, at::kFloat, dev);
    cu = (int32_t*)expect(tensor(a[4], "cu_seqlens"), "cu_seqlens", {N + 1}, at::kInt, dev);
    h0 = optional<float>(a[5], "h0", ss, at::kFloat, dev);
    if ((h0 != nullptr) != (p.has_h0 != 0)) refuse("h0 must be given iff has_h0");
  }
};

// linear_fwd(problem, q, k, v, g, cu_seqlens, h0, o, ht, workspace) -> (o, ht)
PyObject* linear_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 10);
    gdn_linear_problem p = problem<gdn_linear_problem>(a[0]);
    const at::Device dev = gpu_of(tensor(a[3], "v"), "v");
    const c10::DeviceGuard guard(dev);
    const LinearInputs in(p, a + 1, dev);
    const int64_t vs[] = {p.n_tokens, p.h_v, p.d}, ss[] = {p.n_seqs, p.h_v, p.d, p.d};
    Tensor o, ht;
    Buffers made(dev);
    made.want(o, a[7], "o", vs, io_type(p.dtype));
    if (p.want_ht) made.want(ht, a[8], "ht", ss, at::kFloat);
    else if (a[8] != Py_None) refuse("ht is given but want_ht is not set");
    Workspace ws(a[9], dev, made, [&] { return g_lib.linear_workspace(&p, GDN_OP_FWD); });
    made.allocate();
    void* op = expect(o, "o", vs, io_type(p.dtype), dev);
    float* htp = p.want_ht ? (float*)expect(ht, "ht", ss, at::kFloat, dev) : nullptr;
    check(g_lib.linear_fwd(&p, in.q, in.k, in.v, in.g, in.cu, in.h0, op, htp, ws.t.data_ptr(), ws.bytes, stream_of(dev)));
    return Py_BuildValue("NN", THPVariable_Wrap(o), wrap_or_none(ht));
  });
}

// linear_bwd(problem, q, k, v, g, cu_seqlens, h0, dO, dht, want_dg, dq, dk, dv, dg, dh0, workspace) -> (dq, dk, dv, dg, dh0)
PyObject* linear_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 16);
    gdn_linear_problem p = problem<gdn_linear_problem>(a[0]);
    const at::Device dev = gpu_of(tensor(a[3], "v"), "v");
    const c10::DeviceGuard guard(dev);
    const LinearInputs in(p, a + 1, dev);
    const at::ScalarType io = io_type(p.dtype);
    const int64_t qs[] = {p.n_tokens, p.h_qk, p.d}, vs[] = {p.n_tokens, p.h_v, p.d}, ss[] = {p.n_seqs, p.h_v, p.d, p.d};
    const int64_t gs[] = {p.n_tokens, p.h_v};
    const at::IntArrayRef gshape = p.decay == GDN_DECAY_HEAD ? at::IntArrayRef(gs + 1, 1) : at::IntArrayRef(gs);
    void* dop = expect(tensor(a[7], "dO"), "dO", vs, io, dev);
    const float* dht = optional<float>(a[8], "dht", ss, at::kFloat, dev);
    const bool with_g = a[9] == Py_True;
    if (!with_g && a[13] != Py_None) refuse("dg is given but not wanted");
    if (!p.has_h0 && a[14] != Py_None) refuse("dh0 is given but has_h0 is not set");
    Tensor dq, dk, dv, dg, dh0;
    Buffers made(dev);
    made.want(dq, a[10], "dq", qs, io);
    made.want(dk, a[11], "dk", qs, io);
    made.want(dv, a[12], "dv", vs, io);
    if (with_g) made.want(dg, a[13], "dg", gshape, at::kFloat);
    if (p.has_h0) made.want(dh0, a[14], "dh0", ss, at::kFloat);
    Workspace ws(a[15], dev, made, [&] { return g_lib.linear_workspace(&p, GDN_OP_BWD); });
    made.allocate();
    void* dqp = expect(dq, "dq", qs, io, dev);
    void* dkp = expect(dk, "dk", qs, io, dev);
    void* dvp = expect(dv, "dv", vs, io, dev);
    float* dgp = with_g ? (float*)expect(dg, "dg", gshape, at::kFloat, dev) : nullptr;
    float* dh0p = p.has_h0 ? (float*)expect(dh0, "dh0", ss, at::kFloat, dev) : nullptr;
    check(g_lib.linear_bwd(&p, in.q, in.k, in.v, in.g, in.cu, in.h0, dop, dht, dqp, dkp, dvp, dgp, dh0p, ws.t.data_ptr(),
                           ws.bytes, stream_of(dev)));
    return Py_BuildValue("NNNNN", THPVariable_Wrap(dq), THPVariable_Wrap(dk), THPVariable_Wrap(dv), wrap_or_none(dg),
                         wrap_or_none(dh0));
  });
}

// linear_step(problem, q, k, v, g, states, slot_in, slot_out, slot_tok, cu_seqlens, o) -> o
PyObject* linear_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 11);
    gdn_linear_step_problem p = problem<gdn_linear_step_problem>(a[0]);
    const Tensor& v = tensor(a[3], "v");
    const at::Device dev = gpu_of(v, "v");
    const c10::DeviceGuard guard(dev);
    const at::ScalarType io = io_type(p.dtype);
    const int64_t T = p.n_tokens, N = p.n_seqs;
    const int64_t qs[] = {T, p.h_qk, p.d}, vs[] = {T, p.h_v, p.d}, gs[] = {T, p.h_v}, ss[] = {p.n_slots, p.h_v, p.d, p.d};
    const at::IntArrayRef gshape = p.decay == GDN_DECAY_HEAD ? at::IntArrayRef(gs + 1, 1) : at::IntArrayRef(gs);
    void* vp = expect(v, "v", vs, io, dev, &p.v_stride);
    void* qp = expect(tensor(a[1], "q"), "q", qs, io, dev, &p.q_stride);
    void* kp = expect(tensor(a[2], "k"), "k", qs, io, dev, &p.k_stride);
    void* gp = expect(tensor(a[4], "g"), "g", gshape, at::kFloat, dev);
    void* sp = expect(tensor(a[5], "states"), "states", ss, at::kFloat, dev);
    void* in = expect(tensor(a[6], "slot_in"), "slot_in", {N}, at::kInt, dev);
    void* out = expect(tensor(a[7], "slot_out"), "slot_out", {N}, at::kInt, dev);
    const int32_t* tok = optional<int32_t>(a[8], "slot_tok", {T}, at::kInt, dev);
    const int32_t* cu = optional<int32_t>(a[9], "cu_seqlens", {N + 1}, at::kInt, dev);
    const Tensor o = a[10] == Py_None ? empty(vs, io, dev) : tensor(a[10], "o");
    void* op = expect(o, "o", vs, io, dev);
    check(g_lib.linear_step(&p, qp, kp, vp, (float*)gp, cu, (int32_t*)in, (int32_t*)out, tok, (float*)sp, op, stream_of(dev)));
    return THPVariable_Wrap(o);
  });
}

// norm_fwd(problem, x, weight, residual, y, scales, residual_out) -> (y, scales, residual_out)
PyObject* norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 7);
    gdn_rms_norm_problem p = problem<gdn_rms_norm_problem>(a[0]);
    const Tensor& x = tensor(a[1], "x");
    const at::Device dev = gpu_of(x, "x");
    const c10::DeviceGuard guard(dev);
    const at::ScalarType io = io_type(p.dtype), yt = p.out == GDN_OUT_E4M3 ? at::kFloat8_e4m3fn : io;
    if (p.d < 1 || p.group < 0 || p.n_rows < 0) refuse("d must be >= 1, group and n_rows >= 0");
    const int64_t xs[] = {p.n_rows, p.d}, ss[] = {p.n_rows, p.group ? p.d / p.group : 1};
    void* xp = expect(x, "x", xs, io, dev, &p.x_stride);
    const float* w = optional<float>(a[2], "weight", {p.d}, at::kFloat, dev);
    void* res = a[3] == Py_None ? nullptr : expect(tensor(a[3], "residual"), "residual", xs, io, dev, &p.residual_stride);
    const bool with_res = a[3] != Py_None, scaled = p.out == GDN_OUT_E4M3;
    if (!scaled && a[5] != Py_None) refuse("scales are given but out is not e4m3");
    if (!with_res && a[6] != Py_None) refuse("residual_out is given without residual");
    Tensor y, scales, out;
    Buffers made(dev);
    made.want(y, a[4], "y", xs, yt);
    if (scaled) made.want(scales, a[5], "scales", ss, at::kFloat);
    if (with_res) made.want(out, a[6], "residual_out", xs, io);
    made.allocate();
    void* yp = expect(y, "y", xs, yt, dev);
    float* sp = scaled ? (float*)expect(scales, "scales", ss, at::kFloat, dev) : nullptr;
    void* op = with_res ? expect(out, "residual_out", xs, io, dev) : nullptr;
    check(g_lib.norm_fwd(&p, xp, w, res, yp, sp, op, stream_of(dev)));
    return Py_BuildValue("NNN", THPVariable_Wrap(y), wrap_or_none(scales), wrap_or_none(out));
  });
}

// norm_bwd(problem, x, dy, weight, d_residual, dx, dweight, workspace) -> (dx, dweight)
PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 8);
    gdn_rms_norm_problem p = problem<gdn_rms_norm_problem>(a[0]);
    const Tensor& x = tensor(a[1], "x");
    const at::Device dev = gpu_of(x, "x");
    const c10::DeviceGuard guard(dev);
    const at::ScalarType io = io_type(p.dtype);
    if (p.d < 1 || p.n_rows < 0) refuse("d must be >= 1 and n_rows >= 0");
    const int64_t xs[] = {p.n_rows, p.d};
    void* xp = expect(x, "x", xs, io, dev, &p.x_stride);
    void* dyp = expect(tensor(a[2], "dy"), "dy", xs, io, dev);
    const float* w = optional<float>(a[3], "weight", {p.d}, at::kFloat, dev);
    void* res = a[4] == Py_None ? nullptr : expect(tensor(a[4], "d_residual"), "d_residual", xs, io, dev, &p.residual_stride);
    if (!w && a[6] != Py_None) refuse("dweight is given without weight");
    Tensor dx, dw;
    Buffers made(dev);
    made.want(dx, a[5], "dx", xs, io);
    if (w) made.want(dw, a[6], "dweight", {p.d}, at::kFloat);
    std::optional<Workspace> ws; // the weight's
    if (w) ws.emplace(a[7], dev, made, [&] { return g_lib.norm_workspace(&p); });
    made.allocate();
    void* dxp = expect(dx, "dx", xs, io, dev);
    float* dwp = w ? (float*)expect(dw, "dweight", {p.d}, at::kFloat, dev) : nullptr;
    check(g_lib.norm_bwd(&p, xp, w, dyp, res, dxp, dwp, ws ? ws->t.data_ptr() : nullptr, ws ? ws->bytes : 0, stream_of(dev)));
    return Py_BuildValue("NN", THPVariable_Wrap(dx), wrap_or_none(dw));
  });
}

// step_maps(problem, lengths, contexts, block_table, free_list, free_count, cu_seqlens, positions, token_slots, granted,
//           slot_in, slot_out, slot_tok, contexts_out, free_count_out) -> the nine outputs
PyObject* step_maps(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 15);
    const gdn_step_maps_problem p = problem<gdn_step_maps_problem>(a[0]);
    const Tensor& lengths = tensor(a[1], "lengths");
    const at::Device dev = gpu_of(lengths, "lengths");
    const c10::DeviceGuard guard(dev);
    if (p.n_seqs < 0 || p.n_tokens < 0 || p.max_blocks < 0 || p.n_free < 0) refuse("sizes must be >= 0");
    const int64_t N = p.n_seqs, T = p.n_tokens;
    void* lp = expect(lengths, "lengths", {N}, at::kInt, dev);
    void* cp = expect(tensor(a[2], "contexts"), "contexts", {N}, at::kInt, dev);
    void* tp = expect(tensor(a[3], "block_table"), "block_table", {N, p.max_blocks}, at::kInt, dev);
    void* fp = expect(tensor(a[4], "free_list"), "free_list", {p.n_free}, at::kInt, dev);
    void* np = expect(tensor(a[5], "free_count"), "free_count", {1}, at::kInt, dev);
    const char* names[] = {"cu_seqlens", "positions", "token_slots", "granted", "slot_in", "slot_out", "slot_tok", "contexts_out", "free_count_out"};
    const int64_t sizes[] = {N + 1, T, T, N, N, N, T, N, 1};
    Tensor out[9];
    void* at[9];
    Buffers made(dev, 64 << 20); // a step's maps go together, up to 4 million tokens (65,536: 6.7 us, apart 10.3)
    for (int i = 0; i < 9; ++i) made.want(out[i], a[6 + i], names[i], {sizes[i]}, i == 2 ? at::kLong : at::kInt);
    made.allocate();
    for (int i = 0; i < 9; ++i) at[i] = expect(out[i], names[i], {sizes[i]}, i == 2 ? at::kLong : at::kInt, dev);
    const gdn_step_maps_out o = {(int32_t*)at[0], (int32_t*)at[1], (int64_t*)at[2], (int32_t*)at[3], (int32_t*)at[4],
                                 (int32_t*)at[5], (int32_t*)at[6], (int32_t*)at[7], (int32_t*)at[8]};
    check(g_lib.step_maps(&p, (int32_t*)lp, (int32_t*)cp, (int32_t*)tp, (int32_t*)fp, (int32_t*)np, &o, stream_of(dev)));
    PyObject* r = PyTuple_New(9);
    for (int i = 0; r && i < 9; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(out[i]));
    return r;
  });
}

// init(GdnError, addresses of the entry points in the order of Entries)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 1 + ENTRIES) {
    PyErr_Format(PyExc_TypeError, "init takes %d arguments", 1 + ENTRIES);
    return nullptr;
  }
  void* f[ENTRIES];
  for (int i = 0; i < ENTRIES; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "NULL entry point");
      return nullptr;
    }
  }
  Py_INCREF(a[0]);
  Py_XDECREF(g_error);
  g_error = a[0];
  static_assert(sizeof f == sizeof g_lib, "one address an entry");
  std::memcpy(&g_lib, f, sizeof g_lib);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))init, METH_FASTCALL, nullptr},
    {"recurrent", (PyCFunction)(void (*)(void))recurrent, METH_FASTCALL, nullptr},
    {"conv_step", (PyCFunction)(void (*)(void))conv_step, METH_FASTCALL, nullptr},
    {"rope_fwd", (PyCFunction)(void (*)(void))rope_fwd, METH_FASTCALL, nullptr},
    {"rope_bwd", (PyCFunction)(void (*)(void))rope_bwd, METH_FASTCALL, nullptr},
    {"linear_fwd", (PyCFunction)(void (*)(void))linear_fwd, METH_FASTCALL, nullptr},
    {"linear_bwd", (PyCFunction)(void (*)(void))linear_bwd, METH_FASTCALL, nullptr},
    {"linear_step", (PyCFunction)(void (*)(void))linear_step, METH_FASTCALL, nullptr},
    {"norm_fwd", (PyCFunction)(void (*)(void))norm_fwd, METH_FASTCALL, nullptr},
    {"norm_bwd", (PyCFunction)(void (*)(void))norm_bwd, METH_FASTCALL, nullptr},
    {"step_maps", (PyCFunction)(void (*)(void))step_maps, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
