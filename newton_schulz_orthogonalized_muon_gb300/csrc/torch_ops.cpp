// The training operators' calls on torch tensors: an extension module that
// checks the tensors, has torch allocate outputs and scratch, and calls the C
// ABI on torch's current stream.  ops.py holds the functions that users call,
// with their documentation; each passes on its positional arguments behind the
// handle's address and its device.
//
// A function returns its results, or an int, the status of a C call that was
// not MUON_OK.  Arguments that do not go together raise ValueError.
//
// The smallest kernels take 7 us and a call by way of ctypes took 17 (layer
// norm) to 29 us (attention backward), most of it checks and conversions one
// Python operation at a time; here 7 to 10 and 12 to 15.
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <new>
#include <optional>
#include <string>
#include <vector>

#include "muon.h"

namespace {

constexpr int64_t kBlock = 128;                 // columns that share one scale

struct Refusal {
  std::string what;
};
[[noreturn]] void refuse(std::string what) { throw Refusal{std::move(what)}; }

// An exception that Python has already been told of.
struct Raised {};

// Other Python threads run while torch allocates and the call queues its work
// (which waits when the launch queue is full).  Between the arguments and the
// results nothing is Python's.
class NoGil {
 public:
  NoGil() : state_(PyEval_SaveThread()) {}
  ~NoGil() { PyEval_RestoreThread(state_); }
  NoGil(const NoGil&) = delete;
  NoGil& operator=(const NoGil&) = delete;

 private:
  PyThreadState* state_;
};

// ---------------------------------------------------------------- arguments
// The calls' first two arguments.
struct Target {
  muon_handle_t h;
  int dev;
  void* stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }
};

struct Args {
  PyObject* const* a;
  Py_ssize_t n, i = 0;

  PyObject* next() {
    if (i >= n) refuse("too few arguments");
    return a[i++];
  }
  int64_t integer() {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
  }
  double number() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
  }
  bool truth() {
    const int v = PyObject_IsTrue(next());
    if (v < 0) throw Raised{};
    return v != 0;
  }
  Target target() {
    void* h = PyLong_AsVoidPtr(next());
    if (h == nullptr && PyErr_Occurred()) throw Raised{};
    return Target{static_cast<muon_handle_t>(h), static_cast<int>(integer())};
  }
  // a CUDA tensor on the target's device; None: nullptr where that is allowed
  const at::Tensor* tensor(const Target& t, const char* what, bool optional = false) {
    PyObject* o = next();
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(std::string(what) + " must be a CUDA tensor");
    const at::Tensor& v = THPVariable_Unpack(o);
    if (!v.is_cuda() || v.get_device() != t.dev)
      refuse(std::string(what) + " must be a CUDA tensor on device " + std::to_string(t.dev));
    return &v;
  }
  // torch.dtype or None
  std::optional<at::ScalarType> dtype() {
    PyObject* o = next();
    if (o == Py_None) return std::nullopt;
    if (!THPDtype_Check(o)) refuse("dtype must be a torch.dtype");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
  }
};

int code_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return MUON_F32;
    case at::kBFloat16: return MUON_BF16;
    case at::kHalf: return MUON_F16;
    default: return -1;
  }
}

int code(const at::Tensor& t, const char* what) {
  const int c = code_of(t.scalar_type());
  if (c < 0) refuse(std::string(what) + " must be float32, bfloat16 or float16");
  return c;
}

std::string shape(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

at::Tensor empty(at::IntArrayRef sizes, const at::Tensor& like, at::ScalarType type) {
  return at::empty(sizes, like.options().dtype(type));
}

// The tensors, or the status where it is not MUON_OK.
PyObject* result(muon_status_t st, at::Tensor a) {
  return st != MUON_OK ? PyLong_FromLong(st) : THPVariable_Wrap(std::move(a));
}
PyObject* results(muon_status_t st, at::Tensor a, at::Tensor b, at::Tensor c) {
  if (st != MUON_OK) return PyLong_FromLong(st);
  const int n = c.defined() ? 3 : 2;
  PyObject* t = PyTuple_New(n);
  if (t == nullptr) throw Raised{};
  at::Tensor* all[3] = {&a, &b, &c};
  for (int i = 0; i < n; ++i) {
    PyObject* o = THPVariable_Wrap(std::move(*all[i]));
    if (o == nullptr) {
      Py_DECREF(t);
      throw Raised{};
    }
    PyTuple_SET_ITEM(t, i, o);
  }
  return t;
}

// [.., cols] seen as rows: the last dimension contiguous, the others with one
// stride between rows.  Anything else is copied once.
struct Rows {
  at::Tensor t;
  int64_t rows, ld;
};

Rows rows_of(const at::Tensor& t, const char* what) {
  const int64_t d = t.dim();
  if (d == 0) refuse(std::string(what) + " must have at least one dimension");
  const int64_t cols = t.size(d - 1), rows = cols ? t.numel() / cols : 0;
  int64_t ld = cols, step = -1;                  // step: what the next dimension's stride has to be
  bool one = t.stride(d - 1) == 1 || cols <= 1;
  for (int64_t i = d - 2; one && i >= 0; --i) {
    const int64_t n = t.size(i), s = t.stride(i);
    if (n == 1) continue;
    if (step < 0)
      ld = s;
    else
      one = s == step;
    step = s * n;
  }
  if (one && ld >= cols) return Rows{t, rows, ld};
  return Rows{t.contiguous(), rows, cols};
}

// --------------------------------------------------------------- layer norm
// Pointer and type code of a weight or bias vector.
struct Affine {
  const void* p;
  int code;
};

Affine affine(const at::Tensor* t, const char* what, at::ScalarType type, int64_t cols) {
  if (t == nullptr) return Affine{nullptr, MUON_F32};
  if (t->dim() != 1 || t->size(0) != cols || !t->is_contiguous())
    refuse(std::string(what) + " must be a contiguous vector of " + std::to_string(cols) + " elements");
  if (t->scalar_type() != at::kFloat && t->scalar_type() != type)
    refuse(std::string(what) + " must be float32 or of x's type");
  return Affine{t->data_ptr(), code_of(t->scalar_type())};
}

PyObject* layer_norm(Args a) {
  const Target t = a.target();
  const at::Tensor& x = *a.tensor(t, "x");
  const at::Tensor *weight = a.tensor(t, "weight", true), *bias = a.tensor(t, "bias", true);
  const double eps = a.number();
  at::Tensor y, mean, rstd;
  muon_status_t st;
  {
    NoGil free;
    const int type = code(x, "x");
    const Rows xr = rows_of(x, "x");
    const int64_t cols = x.size(-1);
    const Affine w = affine(weight, "weight", x.scalar_type(), cols), b = affine(bias, "bias", x.scalar_type(), cols);
    if (w.p != nullptr && b.p != nullptr && w.code != b.code) refuse("weight and bias must have one type");
    const at::IntArrayRef sizes = x.sizes(), outer = sizes.slice(0, sizes.size() - 1);
    y = empty(sizes, x, x.scalar_type());
    mean = empty(outer, x, at::kFloat);
    rstd = empty(outer, x, at::kFloat);
    st = muon_layer_norm_forward(
        t.h, xr.t.data_ptr(), xr.ld, w.p, b.p, y.data_ptr(), cols, mean.data_ptr<float>(), rstd.data_ptr<float>(),
        xr.rows, cols, type, w.p == nullptr ? b.code : w.code, static_cast<float>(eps), t.stream());
  }
  return results(st, std::move(y), std::move(mean), std::move(rstd));
}

PyObject* layer_norm_backward(Args a) {
  const Target t = a.target();
  const at::Tensor &dy = *a.tensor(t, "dy"), &x = *a.tensor(t, "x"), &mean = *a.tensor(t, "mean"),
                   &rstd = *a.tensor(t, "rstd");
  const at::Tensor* weight = a.tensor(t, "weight", true);
  at::Tensor dx, dw, db;
  muon_status_t st;
  {
    NoGil free;
    const int type = code(x, "x");
    if (dy.sizes() != x.sizes() || dy.scalar_type() != x.scalar_type()) refuse("dy must have x's shape and type");
    const Rows xr = rows_of(x, "x"), gr = rows_of(dy, "dy");
    const int64_t cols = x.size(-1);
    const at::IntArrayRef sizes = x.sizes(), outer = sizes.slice(0, sizes.size() - 1);
    for (const at::Tensor* s : {&mean, &rstd})
      if (s->scalar_type() != at::kFloat || s->sizes() != outer || !s->is_contiguous())
        refuse("mean and rstd must be contiguous float32 of x's shape without the last dimension");
    const Affine w = affine(weight, "weight", x.scalar_type(), cols);
    uint64_t need = 0;
    st = muon_layer_norm_workspace(t.h, xr.rows, cols, &need);
    if (st == MUON_OK) {
      at::Tensor ws = empty({static_cast<int64_t>(need)}, x, at::kByte);
      dx = empty(sizes, x, x.scalar_type());
      dw = empty({cols}, x, at::kFloat);
      db = empty({cols}, x, at::kFloat);
      st = muon_layer_norm_backward(t.h, gr.t.data_ptr(), gr.ld, xr.t.data_ptr(), xr.ld, mean.data_ptr<float>(),
                                    rstd.data_ptr<float>(), w.p, dx.data_ptr(), cols, dw.data_ptr<float>(),
                                    db.data_ptr<float>(), xr.rows, cols, type, w.code, ws.data_ptr(), need, t.stream());
    }
  }
  return results(st, std::move(dx), std::move(dw), std::move(db));
}

// ---------------------------------------------------------------- attention
// Strides (batch, token, head) of [batch, token, head, dim], or of [token,
// head, dim] when packed.
void set_strides(int64_t* to, const at::Tensor& t, const char* what, bool packed) {
  const int64_t d = packed ? 3 : 4;
  if (t.dim() != d) refuse(std::string(what) + " must have " + std::to_string(d) + " dimensions");
  if (t.stride(d - 1) != 1 && t.size(d - 1) != 1) refuse(std::string(what) + " must be contiguous in its last dimension");
  to[0] = packed ? 0 : t.stride(0);
  to[1] = t.stride(d - 3);
  to[2] = t.stride(d - 2);
}

// Checks and packs what both directions share; reads causal, window, scale
// and the offsets from the arguments.
muon_attention_t attention_args(const Target& t, Args& a, const at::Tensor& q, const at::Tensor& k, const at::Tensor& v) {
  muon_attention_t p{};
  p.causal = a.truth() ? 1 : 0;
  const int64_t window = a.integer();
  PyObject* scale = a.next();
  const at::Tensor *cu_q = a.tensor(t, "cu_seqlens_q", true), *cu_k = a.tensor(t, "cu_seqlens_k", true);
  if (q.scalar_type() != at::kBFloat16 && q.scalar_type() != at::kHalf) refuse("q must be bfloat16 or float16");
  if (k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type()) refuse("q, k and v must have one type");
  const bool packed = cu_q != nullptr || cu_k != nullptr;
  set_strides(p.q_stride, q, "q", packed);
  set_strides(p.k_stride, k, "k", packed);
  set_strides(p.v_stride, v, "v", packed);
  const int64_t d = q.dim();
  if (k.sizes() != v.sizes() || q.size(d - 1) != k.size(d - 1) || (!packed && q.size(0) != k.size(0)))
    refuse("shapes do not go together: q " + shape(q) + ", k " + shape(k) + ", v " + shape(v));
  int64_t batch;
  if (packed) {
    if (cu_q == nullptr || cu_k == nullptr) refuse("cu_seqlens_q and cu_seqlens_k go together");
    for (const at::Tensor* c : {cu_q, cu_k})
      if (c->scalar_type() != at::kInt || c->dim() != 1 || c->size(0) < 1 || !c->is_contiguous())
        refuse("cu_seqlens_q and cu_seqlens_k must be contiguous int32 vectors of at least one element");
    if (cu_q->size(0) != cu_k->size(0)) refuse("cu_seqlens_q and cu_seqlens_k must have one length");
    batch = cu_q->size(0) - 1;
    p.cu_seqlens_q = cu_q->data_ptr<int32_t>();
    p.cu_seqlens_k = cu_k->data_ptr<int32_t>();
  } else {
    batch = q.size(0);
  }
  const int64_t ints[7] = {batch,         q.size(d - 3), k.size(d - 3), q.size(d - 2),
                           k.size(d - 2), q.size(d - 1), window};
  for (const int64_t i : ints)
    if (i < 0 || i > INT32_MAX) refuse("negative or oversized shape or window");
  p.batch = static_cast<int32_t>(batch);
  p.sq = static_cast<int32_t>(ints[1]);
  p.sk = static_cast<int32_t>(ints[2]);
  p.heads = static_cast<int32_t>(ints[3]);
  p.kv_heads = static_cast<int32_t>(ints[4]);
  p.dim = static_cast<int32_t>(ints[5]);
  p.window = static_cast<int32_t>(window);
  p.dtype = code_of(q.scalar_type());
  if (scale == Py_None) {
    p.scale = p.dim ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(p.dim))) : 0.f;
  } else {
    const double s = PyFloat_AsDouble(scale);
    if (s == -1.0 && PyErr_Occurred()) throw Raised{};
    p.scale = static_cast<float>(s);
  }
  p.q = q.data_ptr();
  p.k = k.data_ptr();
  p.v = v.data_ptr();
  return p;
}

// [heads, sq] or [batch, heads, sq]
struct LseShape {
  int64_t n[3];
  size_t dims;
  explicit LseShape(const muon_attention_t& p) {
    dims = 0;
    if (p.cu_seqlens_q == nullptr) n[dims++] = p.batch;
    n[dims++] = p.heads;
    n[dims++] = p.sq;
  }
  at::IntArrayRef ref() const { return at::IntArrayRef(n, dims); }
};

PyObject* attention(Args a) {
  const Target t = a.target();
  const at::Tensor &q = *a.tensor(t, "q"), &k = *a.tensor(t, "k"), &v = *a.tensor(t, "v");
  muon_attention_t p = attention_args(t, a, q, k, v);
  at::Tensor o, lse;
  muon_status_t st;
  {
    NoGil free;
    o = empty(q.sizes(), q, q.scalar_type());
    lse = empty(LseShape(p).ref(), q, at::kFloat);
    p.o = o.data_ptr();
    p.lse = lse.data_ptr<float>();
    set_strides(p.o_stride, o, "o", p.cu_seqlens_q != nullptr);
    uint64_t need = 0;
    st = muon_attention_forward_workspace(t.h, &p, &need);
    if (st == MUON_OK) {
      at::Tensor ws;
      if (need > 0) ws = empty({static_cast<int64_t>(need)}, q, at::kByte);
      st = muon_attention_forward_ex(t.h, &p, need > 0 ? ws.data_ptr() : nullptr, need, t.stream());
    }
  }
  return results(st, std::move(o), std::move(lse), at::Tensor());
}

PyObject* attention_backward(Args a) {
  const Target t = a.target();
  const at::Tensor &given = *a.tensor(t, "do"), &q = *a.tensor(t, "q"), &k = *a.tensor(t, "k"), &v = *a.tensor(t, "v"),
                   &o = *a.tensor(t, "o"), &lse = *a.tensor(t, "lse");
  muon_attention_t p = attention_args(t, a, q, k, v);
  at::Tensor dq, dk, dv;
  muon_status_t st;
  {
    NoGil free;
    const bool packed = p.cu_seqlens_q != nullptr;
    if (given.sizes() != q.sizes() || o.sizes() != q.sizes() || given.scalar_type() != q.scalar_type() ||
        o.scalar_type() != q.scalar_type())
      refuse("do and o must have q's shape and type");
    if (lse.scalar_type() != at::kFloat || lse.sizes() != LseShape(p).ref() || !lse.is_contiguous())
      refuse("lse must be the contiguous float32 tensor that attention returned");
    // autograd hands over expanded gradients, and parts of larger ones that start anywhere
    at::Tensor dout = given;
    bool copy = reinterpret_cast<uintptr_t>(dout.data_ptr()) % 16 != 0;
    if (!dout.is_contiguous()) {
      copy = copy || dout.stride(-1) != 1;
      for (int64_t i = 0; i + 1 < dout.dim(); ++i) copy = copy || dout.stride(i) == 0 || dout.stride(i) % 8 != 0;
    }
    if (copy) dout = dout.clone(at::MemoryFormat::Contiguous);
    dq = empty(q.sizes(), q, q.scalar_type());
    dk = empty(k.sizes(), k, k.scalar_type());
    dv = empty(v.sizes(), v, v.scalar_type());
    p.o = o.data_ptr();
    p.lse = lse.data_ptr<float>();
    p.dout = dout.data_ptr();
    p.dq = dq.data_ptr();
    p.dk = dk.data_ptr();
    p.dv = dv.data_ptr();
    set_strides(p.o_stride, o, "o", packed);
    set_strides(p.dout_stride, dout, "do", packed);
    set_strides(p.dq_stride, dq, "dq", packed);
    set_strides(p.dk_stride, dk, "dk", packed);
    set_strides(p.dv_stride, dv, "dv", packed);
    uint64_t need = 0;
    st = muon_attention_workspace(t.h, &p, &need);
    if (st == MUON_OK) {
      at::Tensor ws = empty({static_cast<int64_t>(need)}, q, at::kByte);
      st = muon_attention_backward(t.h, &p, ws.data_ptr(), need, t.stream());
    }
  }
  return results(st, std::move(dq), std::move(dk), std::move(dv));
}

// --------------------------------------------------- activations in 8 bits
int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// [rows][cols] bytes with row stride ld, on storage of whole rows: the kernels
// read codes in groups of 8 and scales in groups of 16, the last ones too.
at::Tensor padded(int64_t rows, int64_t cols, int64_t ld, const at::Tensor& like, at::ScalarType type) {
  at::Tensor t = empty({rows, ld}, like, type);
  t.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef({rows, cols}), at::IntArrayRef({ld, 1}));
  return t;
}

PyObject* act8_store(Args a) {
  const Target t = a.target();
  const at::Tensor& x = *a.tensor(t, "x");
  at::Tensor codes, scales;
  muon_status_t st;
  {
    NoGil free;
    const int type = code(x, "x");
    if (x.dim() != 2) refuse("x must be 2-D");
    const Rows xr = rows_of(x, "x");
    const int64_t rows = x.size(0), cols = x.size(1), blocks = round_up(cols, kBlock) / kBlock;
    const int64_t ldc = blocks * kBlock, lds = round_up(rows, 16);
    codes = padded(rows, cols, ldc, x, at::kFloat8_e4m3fn);
    scales = padded(blocks, rows, lds, x, at::kByte);
    st = muon_act8_store(t.h, xr.t.data_ptr(), xr.ld, static_cast<uint8_t*>(codes.data_ptr()), ldc,
                        static_cast<uint8_t*>(scales.data_ptr()), lds, rows, cols, type, t.stream());
  }
  return results(st, std::move(codes), std::move(scales), at::Tensor());
}

// codes and scales as the kernels read them (padded row strides), copied if
// they come in another layout.
struct Act8 {
  at::Tensor codes, scales;
  int64_t rows, cols, ldc, lds;
  const uint8_t* code() const { return static_cast<const uint8_t*>(codes.data_ptr()); }
  const uint8_t* scale() const { return static_cast<const uint8_t*>(scales.data_ptr()); }
};

Act8 act8_of(const at::Tensor& codes, const at::Tensor& scales) {
  if (codes.dim() != 2 || (codes.scalar_type() != at::kFloat8_e4m3fn && codes.scalar_type() != at::kByte))
    refuse("codes must be 2-D float8_e4m3fn");
  const int64_t rows = codes.size(0), cols = codes.size(1), blocks = round_up(cols, kBlock) / kBlock;
  if (scales.scalar_type() != at::kByte || scales.dim() != 2 || scales.size(0) != blocks || scales.size(1) != rows)
    refuse("scales must be uint8 of shape (" + std::to_string(blocks) + ", " + std::to_string(rows) + ")");
  Act8 r{codes, scales, rows, cols, codes.stride(0), scales.stride(0)};
  if (rows == 0 || cols == 0) return r;
  auto usable = [](const at::Tensor& t, int64_t ld, int64_t unit, int64_t group) {
    if ((t.stride(1) != 1 && t.size(1) != 1) || ld % unit != 0 || ld < t.size(1)) return false;
    const int64_t end = t.storage_offset() + (t.size(0) - 1) * ld + round_up(t.size(1), group);
    return end <= static_cast<int64_t>(t.storage().nbytes()) && reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0;
  };
  if (!usable(r.codes, r.ldc, kBlock, 8)) {
    r.ldc = blocks * kBlock;
    r.codes = padded(rows, cols, r.ldc, codes, at::kByte);
    r.codes.copy_(codes.scalar_type() == at::kByte ? codes : codes.view(at::kByte));
  }
  if (!usable(r.scales, r.lds, 16, 16)) {
    r.lds = round_up(rows, 16);
    r.scales = padded(blocks, rows, r.lds, scales, at::kByte);
    r.scales.copy_(scales);
  }
  return r;
}

PyObject* act8_restore(Args a) {
  const Target t = a.target();
  const at::Tensor &codes = *a.tensor(t, "codes"), &scales = *a.tensor(t, "scales");
  const std::optional<at::ScalarType> type = a.dtype();
  if (!type || code_of(*type) < 0) refuse("dtype must be float32, bfloat16 or float16");
  at::Tensor out;
  muon_status_t st;
  {
    NoGil free;
    const Act8 c = act8_of(codes, scales);
    out = empty({c.rows, c.cols}, codes, *type);
    st = muon_act8_restore(t.h, c.code(), c.ldc, c.scale(), c.lds, out.data_ptr(), c.cols, c.rows,
                                               c.cols, code_of(*type), t.stream());
  }
  return result(st, std::move(out));
}

PyObject* act8_weight_grad(Args a) {
  const Target t = a.target();
  const at::Tensor &dy = *a.tensor(t, "dy"), &codes = *a.tensor(t, "codes"), &scales = *a.tensor(t, "scales");
  const at::Tensor *add = a.tensor(t, "add", true), *given = a.tensor(t, "out", true);
  std::optional<at::ScalarType> type = a.dtype();
  at::Tensor out;
  muon_status_t st;
  {
    NoGil free;
    if (dy.scalar_type() != at::kBFloat16) refuse("dy must be bfloat16");
    if (dy.dim() != 2 || codes.dim() != 2 || dy.size(0) != codes.size(0))
      refuse("dy must be [rows, out] and codes [rows, cols]");
    const int64_t outs = dy.size(1), cols = codes.size(1);
    int64_t ld[2] = {cols, cols};
    const at::Tensor* both[2] = {add, given};
    for (int i = 0; i < 2; ++i) {
      const at::Tensor* m = both[i];
      const std::string what = i == 0 ? "add" : "out";
      if (m == nullptr) continue;
      if (m->dim() != 2 || m->size(0) != outs || m->size(1) != cols)
        refuse(what + " must have shape (" + std::to_string(outs) + ", " + std::to_string(cols) + ")");
      if (type && m->scalar_type() != *type) refuse(what + " does not have the result's type");
      type = m->scalar_type();
      if ((m->stride(1) != 1 && cols > 1) || (m->stride(0) < cols && outs > 1)) refuse(what + " must have contiguous rows");
      ld[i] = std::max(m->stride(0), cols);
    }
    if (!type) type = at::kFloat;
    if (*type != at::kFloat && *type != at::kBFloat16) refuse("dtype must be float32 or bfloat16");
    const Rows g = rows_of(dy, "dy");
    const Act8 c = act8_of(codes, scales);
    out = given != nullptr ? *given : empty({outs, cols}, dy, *type);
    if (given != nullptr) out.unsafeGetTensorImpl()->bump_version();     // autograd sees the write
    uint64_t need = 0;
    st = muon_act8_weight_grad_workspace(t.h, g.t.data_ptr(), g.ld, c.rows, cols, outs, &need);
    if (st == MUON_OK) {
      at::Tensor ws;
      if (need > 0) ws = empty({static_cast<int64_t>(need)}, dy, at::kByte);
      st = muon_act8_weight_grad(t.h, g.t.data_ptr(), g.ld, c.code(), c.ldc, c.scale(), c.lds,
                                 add != nullptr ? add->data_ptr() : nullptr, ld[0], out.data_ptr(), ld[1], c.rows, cols, outs,
                                 code_of(*type), need > 0 ? ws.data_ptr() : nullptr, need, t.stream());
    }
  }
  return result(st, std::move(out));
}

// ------------------------------------------------------ products by expert
// [.., rows, cols] of 16-bit elements as the kernels read it: the last dimension
// contiguous, the other strides multiples of 8 that do not overlap, on a 16-byte
// boundary.  Anything else is copied once.
at::Tensor by_rows(const at::Tensor& t) {
  const int64_t d = t.dim();
  bool fine = reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0 && (t.stride(d - 1) == 1 || t.size(d - 1) == 1);
  int64_t span = t.size(d - 1);
  for (int64_t i = d - 2; i >= 0; --i) {
    if (t.size(i) <= 1) continue;
    fine = fine && t.stride(i) % 8 == 0 && t.stride(i) >= span;
    span += (t.size(i) - 1) * t.stride(i);
  }
  return fine ? t : t.clone(at::MemoryFormat::Contiguous);
}

const int32_t* expert_offsets(const at::Tensor& t, int64_t experts) {
  if (t.scalar_type() != at::kInt || t.dim() != 1 || !t.is_contiguous()) refuse("offsets must be a contiguous int32 vector");
  if (experts >= 0 && t.size(0) != experts + 1)
    refuse("offsets must have " + std::to_string(experts + 1) + " elements, one more than there are experts");
  if (t.size(0) < 2) refuse("offsets must have at least two elements");
  return t.data_ptr<int32_t>();
}

void need_16_bit(const at::Tensor& t, const char* what) {
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kHalf) refuse(std::string(what) + " must be bfloat16 or float16");
}

PyObject* expert_matmul(Args a) {
  const Target t = a.target();
  const at::Tensor &x = *a.tensor(t, "x"), &weight = *a.tensor(t, "weight"), &offsets = *a.tensor(t, "offsets");
  const bool transpose = a.truth();
  at::Tensor y;
  muon_status_t st;
  {
    NoGil free;
    need_16_bit(x, "x");
    if (weight.scalar_type() != x.scalar_type()) refuse("weight must have x's type");
    if (x.dim() != 2 || weight.dim() != 3 || x.size(1) != weight.size(transpose ? 1 : 2))
      refuse("shapes do not go together: x " + shape(x) + ", weight " + shape(weight));
    const int64_t experts = weight.size(0), out = weight.size(1), cols = weight.size(2), tokens = x.size(0);
    const int32_t* at = expert_offsets(offsets, experts);
    const at::Tensor xr = by_rows(x), w = by_rows(weight);
    const int64_t to = transpose ? cols : out;
    y = empty({tokens, to}, x, x.scalar_type());
    st = muon_expert_matmul(t.h, xr.data_ptr(), xr.stride(0), w.data_ptr(), w.stride(1), w.stride(0), at, y.data_ptr(), to,
                            tokens, cols, out, experts, transpose ? 1 : 0, code_of(x.scalar_type()), t.stream());
  }
  return result(st, std::move(y));
}

PyObject* expert_weight_grad(Args a) {
  const Target t = a.target();
  const at::Tensor &dy = *a.tensor(t, "dy"), &x = *a.tensor(t, "x"), &offsets = *a.tensor(t, "offsets");
  const at::Tensor *add = a.tensor(t, "add", true), *given = a.tensor(t, "out", true);
  std::optional<at::ScalarType> type = a.dtype();
  at::Tensor out;
  muon_status_t st;
  {
    NoGil free;
    need_16_bit(dy, "dy");
    if (x.scalar_type() != dy.scalar_type()) refuse("x must have dy's type");
    if (dy.dim() != 2 || x.dim() != 2 || dy.size(0) != x.size(0)) refuse("dy must be [tokens, out] and x [tokens, cols]");
    const int32_t* at = expert_offsets(offsets, -1);
    const int64_t experts = offsets.size(0) - 1, outs = dy.size(1), cols = x.size(1);
    int64_t ld[2] = {cols, cols}, group[2] = {outs * cols, outs * cols};
    const at::Tensor* both[2] = {add, given};
    for (int i = 0; i < 2; ++i) {
      const at::Tensor* m = both[i];
      const std::string what = i == 0 ? "add" : "out";
      if (m == nullptr) continue;
      if (m->dim() != 3 || m->size(0) != experts || m->size(1) != outs || m->size(2) != cols)
        refuse(what + " must have shape (" + std::to_string(experts) + ", " + std::to_string(outs) + ", " + std::to_string(cols) + ")");
      if (type && m->scalar_type() != *type) refuse(what + " does not have the result's type");
      type = m->scalar_type();
      const bool rows = m->stride(2) == 1 && (m->stride(1) >= cols || outs == 1);
      if (!rows || (experts > 1 && m->stride(0) < (outs - 1) * m->stride(1) + cols)) refuse(what + " must have contiguous rows that do not overlap");
      ld[i] = std::max(m->stride(1), cols);
      group[i] = m->stride(0);
    }
    if (!type) type = at::kFloat;
    if (*type != at::kFloat && *type != dy.scalar_type()) refuse("dtype must be float32 or dy's type");
    const at::Tensor g = by_rows(dy), xr = by_rows(x);
    out = given != nullptr ? *given : empty({experts, outs, cols}, dy, *type);
    if (given != nullptr) out.unsafeGetTensorImpl()->bump_version();     // autograd sees the write
    uint64_t need = 0;
    st = muon_expert_weight_grad_workspace(t.h, dy.size(0), cols, outs, experts, &need);
    if (st == MUON_OK) {
      at::Tensor ws;
      if (need > 0) ws = empty({static_cast<int64_t>(need)}, dy, at::kByte);
      st = muon_expert_weight_grad(t.h, g.data_ptr(), g.stride(0), xr.data_ptr(), xr.stride(0), at,
                                   add != nullptr ? add->data_ptr() : nullptr, ld[0], group[0], out.data_ptr(), ld[1], group[1],
                                   dy.size(0), cols, outs, experts, code_of(dy.scalar_type()), code_of(*type),
                                   need > 0 ? ws.data_ptr() : nullptr, need, t.stream());
    }
  }
  return result(st, std::move(out));
}

// --------------------------------------------------------- weights in 8 bits
// Bytes of scales [column blocks][row blocks] for a weight [out][cols]; the
// strides are any.
void check_weight_scales(const at::Tensor& s, int64_t out, int64_t cols) {
  const int64_t kb = round_up(cols, kBlock) / kBlock, ob = round_up(out, kBlock) / kBlock;
  if (s.scalar_type() != at::kByte || s.dim() != 2 || s.size(0) != kb || s.size(1) != ob)
    refuse("the weight's scales must be uint8 of shape (" + std::to_string(kb) + ", " + std::to_string(ob) + ")");
}

// Codes [rows][cols] as the kernels read them: rows a multiple of 128 bytes apart
// on a 16-byte boundary.  Anything else is copied once.
struct Codes {
  at::Tensor t;
  int64_t ld;
  const uint8_t* p() const { return static_cast<const uint8_t*>(t.data_ptr()); }
};

Codes codes_of(const at::Tensor& t, const char* what) {
  if (t.dim() != 2 || (t.scalar_type() != at::kFloat8_e4m3fn && t.scalar_type() != at::kByte))
    refuse(std::string(what) + " must be 2-D float8_e4m3fn");
  const int64_t rows = t.size(0), cols = t.size(1), ld = t.stride(0);
  if ((t.stride(1) == 1 || cols == 1) && ld % kBlock == 0 && ld >= cols && reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0)
    return Codes{t, ld};
  Codes c{padded(rows, cols, round_up(cols, kBlock), t, at::kByte), round_up(cols, kBlock)};
  c.t.copy_(t.scalar_type() == at::kByte ? t : t.view(at::kByte));
  return c;
}

PyObject* act8_store_weight(Args a) {
  const Target t = a.target();
  const at::Tensor& w = *a.tensor(t, "w");
  const bool transposed = a.truth();
  at::Tensor codes, scales, codes_t;
  muon_status_t st;
  {
    NoGil free;
    const int type = code(w, "w");
    if (w.dim() != 2) refuse("w must be 2-D");
    const Rows wr = rows_of(w, "w");
    const int64_t out = w.size(0), cols = w.size(1), kb = round_up(cols, kBlock) / kBlock, ob = round_up(out, kBlock) / kBlock;
    codes = padded(out, cols, kb * kBlock, w, at::kFloat8_e4m3fn);
    scales = empty({kb, ob}, w, at::kByte);
    if (transposed) codes_t = padded(cols, out, ob * kBlock, w, at::kFloat8_e4m3fn);
    st = muon_act8_store_weight(t.h, wr.t.data_ptr(), wr.ld, static_cast<uint8_t*>(codes.data_ptr()), kb * kBlock,
                                transposed ? static_cast<uint8_t*>(codes_t.data_ptr()) : nullptr, ob * kBlock,
                                static_cast<uint8_t*>(scales.data_ptr()), ob, out, cols, type, t.stream());
  }
  return results(st, std::move(codes), std::move(scales), std::move(codes_t));
}

PyObject* act8_restore_weight(Args a) {
  const Target t = a.target();
  const at::Tensor &codes = *a.tensor(t, "codes"), &scales = *a.tensor(t, "scales");
  const std::optional<at::ScalarType> type = a.dtype();
  if (!type || code_of(*type) < 0) refuse("dtype must be float32, bfloat16 or float16");
  at::Tensor w;
  muon_status_t st;
  {
    NoGil free;
    const Codes c = codes_of(codes, "codes");
    const int64_t out = codes.size(0), cols = codes.size(1);
    check_weight_scales(scales, out, cols);
    w = empty({out, cols}, codes, *type);
    st = muon_act8_restore_weight(t.h, c.p(), c.ld, static_cast<const uint8_t*>(scales.data_ptr()), scales.stride(0),
                                  scales.stride(1), w.data_ptr(), cols, out, cols, code_of(*type), t.stream());
  }
  return result(st, std::move(w));
}

PyObject* act8_matmul(Args a) {
  const Target t = a.target();
  const at::Tensor &codes = *a.tensor(t, "codes"), &scales = *a.tensor(t, "scales"), &wcodes = *a.tensor(t, "wcodes"),
                   &wscales = *a.tensor(t, "wscales");
  const std::optional<at::ScalarType> type = a.dtype();
  if (!type || code_of(*type) < 0) refuse("dtype must be float32, bfloat16 or float16");
  at::Tensor y;
  muon_status_t st;
  {
    NoGil free;
    const Act8 x = act8_of(codes, scales);
    const Codes w = codes_of(wcodes, "wcodes");
    const int64_t out = wcodes.size(0), cols = wcodes.size(1);
    if (cols != x.cols) refuse("shapes do not go together: codes " + shape(codes) + ", wcodes " + shape(wcodes));
    check_weight_scales(wscales, out, cols);
    y = empty({x.rows, out}, codes, *type);
    st = muon_act8_matmul(t.h, x.code(), x.ldc, x.scale(), x.lds, w.p(), w.ld, static_cast<const uint8_t*>(wscales.data_ptr()),
                          wscales.stride(0), wscales.stride(1), y.data_ptr(), out, x.rows, cols, out, code_of(*type), t.stream());
  }
  return result(st, std::move(y));
}

// ------------------------------------------------- AdamW with states in 8 bits
// Where a refused item stands, put into words only then.
struct Place {
  const char* list;
  Py_ssize_t i;
  const char* part = "";
  std::string text() const { return std::string(list) + "[" + std::to_string(i) + "]" + part; }
};

// A list or tuple, held while its items are read.
struct Items {
  PyObject* seq;
  // (no other sequence: reading one runs its code, which may change the lists)
  Items(PyObject* o, const Place& what) : seq(o) {
    if (!PyTuple_Check(o) && !PyList_Check(o)) refuse(what.text() + " must be an Adamw8State");
    Py_INCREF(o);
  }
  Items(PyObject* o, const char* what) : seq(PySequence_Fast(o, "")) {
    if (seq == nullptr) {
      PyErr_Clear();
      refuse(std::string(what) + " must be a list");
    }
  }
  ~Items() { Py_DECREF(seq); }
  Items(const Items&) = delete;
  Items& operator=(const Items&) = delete;
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
  PyObject* at(Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
  // item i, a contiguous tensor on the target's device of one of two types
  const at::Tensor& tensor(Py_ssize_t i, const Target& t, const Place& what, at::ScalarType one, at::ScalarType other) const {
    if (!THPVariable_Check(at(i))) refuse(what.text() + " must be a CUDA tensor");
    const at::Tensor& v = THPVariable_Unpack(at(i));
    if (!v.is_cuda() || v.get_device() != t.dev) refuse(what.text() + " must be a CUDA tensor on device " + std::to_string(t.dev));
    if (!v.is_contiguous()) refuse(what.text() + " must be contiguous");
    if (v.scalar_type() != one && v.scalar_type() != other) refuse(what.text() + " has a type that is not supported");
    return v;
  }
};

// The states' part of a tensor's entry.  Whatever a call reads is kept by it: the
// lists may change while other Python threads run.
muon_adamw8_t state_of(const Target& t, PyObject* state, Py_ssize_t i, std::vector<at::Tensor>& keep) {
  const Items s(state, Place{"states", i});
  if (s.size() != 4) refuse(Place{"states", i}.text() + " must be an Adamw8State");
  const at::Tensor &avg = s.tensor(0, t, Place{"states", i, ".avg"}, at::kFloat8_e4m3fn, at::kByte),
                   &root = s.tensor(1, t, Place{"states", i, ".root"}, at::kByte, at::kByte),
                   &as = s.tensor(2, t, Place{"states", i, ".avg_scale"}, at::kByte, at::kByte),
                   &rs = s.tensor(3, t, Place{"states", i, ".root_scale"}, at::kByte, at::kByte);
  const int64_t n = avg.numel(), blocks = round_up(n, kBlock) / kBlock;
  if (root.numel() != n || as.numel() != blocks || rs.numel() != blocks)
    refuse(Place{"states", i}.text() + " needs as many roots as averages, and a scale of each for 128 of them");
  for (const at::Tensor* k : {&avg, &root, &as, &rs}) keep.push_back(*k);
  muon_adamw8_t e{};
  e.avg = static_cast<uint8_t*>(avg.data_ptr());
  e.root = static_cast<uint8_t*>(root.data_ptr());
  e.avg_scale = static_cast<uint8_t*>(as.data_ptr());
  e.root_scale = static_cast<uint8_t*>(rs.data_ptr());
  e.numel = n;
  return e;
}

PyObject* adamw8_step(Args a) {
  const Target t = a.target();
  const Items params(a.next(), "params"), grads(a.next(), "grads"), states(a.next(), "states");
  const int64_t step = a.integer(), seed = a.integer();
  double hyper[5];
  for (double& h : hyper) h = a.number();
  const Py_ssize_t n = params.size();
  if (grads.size() != n || states.size() != n) refuse("params, grads and states must have the same length");
  std::vector<muon_adamw8_t> all;
  std::vector<at::Tensor> written, keep;
  all.reserve(n);
  written.reserve(n);
  keep.reserve(5 * n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    const at::Tensor &p = params.tensor(i, t, Place{"params", i}, at::kFloat, at::kBFloat16),
                     &g = grads.tensor(i, t, Place{"grads", i}, at::kFloat, at::kBFloat16);
    muon_adamw8_t e = state_of(t, states.at(i), i, keep);
    if (g.numel() != p.numel() || e.numel != p.numel())
      refuse(Place{"grads", i}.text() + " or " + Place{"states", i}.text() + " has the wrong size");
    e.param = p.data_ptr();
    e.grad = g.data_ptr();
    e.param_dtype = code_of(p.scalar_type());
    e.grad_dtype = code_of(g.scalar_type());
    all.push_back(e);
    written.push_back(p);
    keep.push_back(g);
  }
  muon_status_t st;
  {
    NoGil free;
    st = muon_adamw8_step(t.h, all.data(), static_cast<int32_t>(n), step, static_cast<uint32_t>(seed), hyper[0], hyper[1],
                          hyper[2], hyper[3], hyper[4], t.stream());
  }
  if (st == MUON_OK)
    for (at::Tensor& p : written) p.unsafeGetTensorImpl()->bump_version();     // autograd sees the write
  return PyLong_FromLong(st);
}

PyObject* adamw8_restore(Args a) {
  const Target t = a.target();
  const Items states(a.next(), "states");
  const std::optional<at::ScalarType> type = a.dtype();
  if (!type || (*type != at::kFloat && *type != at::kBFloat16)) refuse("dtype must be float32 or bfloat16");
  const Py_ssize_t n = states.size();
  std::vector<muon_adamw8_t> all;
  std::vector<at::Tensor> values, keep;                 // four of each state
  std::vector<void*> avg, root;
  std::vector<int64_t> bytes;
  int64_t total = 0;
  for (Py_ssize_t i = 0; i < n; ++i) {
    all.push_back(state_of(t, states.at(i), i, keep));
    // each on a boundary of 256 bytes
    bytes.push_back(total);
    total += round_up(all.back().numel * static_cast<int64_t>(c10::elementSize(*type)), 256) * 2;
  }
  // one storage for all: an allocation for each took 1 us, most of a small call
  const at::Tensor whole = n > 0 ? empty({total}, keep[0], at::kByte) : at::Tensor();
  for (Py_ssize_t i = 0; i < n; ++i) {
    for (int k = 0; k < 2; ++k) {
      const int64_t from = bytes[i] + k * round_up(all[i].numel * static_cast<int64_t>(c10::elementSize(*type)), 256);
      at::Tensor v = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(),
                                                              c10::scalarTypeToTypeMeta(*type));
      v.unsafeGetTensorImpl()->set_storage_offset(from / static_cast<int64_t>(c10::elementSize(*type)));
      v.unsafeGetTensorImpl()->set_sizes_contiguous(keep[4 * i].sizes());
      (k == 0 ? avg : root).push_back(v.data_ptr());
      values.push_back(std::move(v));
    }
  }
  muon_status_t st;
  {
    NoGil free;
    st = muon_adamw8_restore(t.h, all.data(), avg.data(), root.data(), static_cast<int32_t>(n), code_of(*type), t.stream());
  }
  if (st != MUON_OK) return PyLong_FromLong(st);
  PyObject* list = PyList_New(n);
  if (list == nullptr) throw Raised{};
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* pair = nullptr;
    try {
      pair = results(st, std::move(values[2 * i]), std::move(values[2 * i + 1]), at::Tensor());
    } catch (...) {
      Py_DECREF(list);
      throw;
    }
    PyList_SET_ITEM(list, i, pair);
  }
  return list;
}

// ------------------------------------------------------------------- module
template <PyObject* (*F)(Args)>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(Args{args, n});
  } catch (const Raised&) {
  } catch (const Refusal& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch != nullptr ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type != nullptr) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::bad_alloc&) {
    PyErr_NoMemory();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define ENTRY(f) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&call<f>)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {ENTRY(layer_norm), ENTRY(layer_norm_backward), ENTRY(attention), ENTRY(attention_backward),
                         ENTRY(act8_store), ENTRY(act8_restore), ENTRY(act8_weight_grad),
                         ENTRY(expert_matmul), ENTRY(expert_weight_grad), ENTRY(act8_store_weight),
                         ENTRY(act8_restore_weight), ENTRY(act8_matmul), ENTRY(adamw8_step), ENTRY(adamw8_restore),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_ops() { return PyModule_Create(&module); }
