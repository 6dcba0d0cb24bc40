// paged_binding.cpp -- the compiled half of the Python binding of the operators
// around a paged cache (paged.py has the signatures and their documentation):
// checks of tensor metadata, outputs from PyTorch's allocator, and the call of
// the C ABI of include/gbattn.h.  A token's worth of these operators is a few
// microseconds on the device; the same checks in Python took 12 to 20 of them.
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cmath>
#include <cstring>
#include <optional>
#include <sstream>
#include <string>

#include "gbattn.h"

namespace {

using at::Tensor;
using Shape = at::IntArrayRef;

PyObject* g_error = nullptr;  // GbattnError

// A refusal of an argument: the Python exception's type and message.
struct Refused {
  PyObject* type;
  std::string message;
};

template <typename... T>
std::string text(const T&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  return s.str();
}
template <typename... T>
[[noreturn]] void refuse_type(const T&... parts) {
  throw Refused{PyExc_TypeError, text(parts...)};
}
template <typename... T>
[[noreturn]] void refuse_value(const T&... parts) {
  throw Refused{PyExc_ValueError, text(parts...)};
}

bool none(PyObject* o) { return o == Py_None; }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse_type(name, " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

const Tensor& tensor_of_dims(PyObject* o, const char* name, int64_t dims) {
  if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != dims)
    refuse_value(name, " must be a tensor of ", dims, " dims");
  return THPVariable_Unpack(o);
}

int size(int64_t v, const char* name) {
  if (v > INT_MAX) refuse_value(name, " has more than ", INT_MAX, " elements in a dimension");
  return static_cast<int>(v);
}

// The type and device that every tensor of a call has to agree with.
struct First {
  at::ScalarType type;
  c10::Device device;
  int code;  // GBATTN_F16 or GBATTN_BF16
};

int dtype_code(at::ScalarType t, const char* name) {
  if (t == at::kHalf) return GBATTN_F16;
  if (t == at::kBFloat16) return GBATTN_BF16;
  refuse_type("unsupported dtype ", t, " of ", name, "; expected float16 or bfloat16");
}

First first(PyObject* o, const char* name) {
  const Tensor& t = tensor(o, name);
  if (!t.is_cuda()) refuse_value(name, " must be a CUDA tensor (there is no CPU path)");
  const int code = dtype_code(t.scalar_type(), name);
  if (t.dim() != 4) refuse_value(name, " must have 4 dims, got shape ", t.sizes());
  return {t.scalar_type(), t.device(), code};
}

void check(const Tensor& t, const char* name, Shape shape, at::ScalarType type, const c10::Device& device) {
  if (t.scalar_type() != type) refuse_type(name, " must be ", type, ", got ", t.scalar_type());
  if (t.sizes() != shape) refuse_value(name, " must have shape ", shape, ", got ", t.sizes());
  if (t.device() != device) refuse_value(name, " must be on ", device, ", got ", t.device(), " (there is no CPU path)");
}

// Address of a contiguous tensor.
void* ptr(PyObject* o, const char* name, Shape shape, at::ScalarType type, const c10::Device& device) {
  const Tensor& t = tensor(o, name);
  check(t, name, shape, type, device);
  if (!t.is_contiguous()) refuse_value(name, " must be contiguous");
  return t.data_ptr();
}

void* opt(PyObject* o, const char* name, Shape shape, at::ScalarType type, const c10::Device& device) {
  return none(o) ? nullptr : ptr(o, name, shape, type, device);
}

// A [B, heads, S, d] tensor whose rows of d elements are contiguous.
struct Rows {
  void* data = nullptr;
  long long strides[3] = {0, 0, 0};
  bool plain = true;
  const long long* stride() const { return plain ? nullptr : strides; }
};

// Whether rows of shape[3] elements at these strides (0: a dimension of one) lie
// apart because each dimension steps over all of the next smaller one, as in any
// view of a tensor with more heads.
bool nested(Shape shape, const long long (&strides)[3]) {
  bool used[3] = {};
  long long extent = shape[3];
  for (int dims = 0; dims < 3; ++dims) {
    int next = -1;
    for (int i = 0; i < 3; ++i)
      if (!used[i] && (next < 0 || shape[next] == 1 || (shape[i] > 1 && strides[i] < strides[next]))) next = i;
    used[next] = true;
    if (shape[next] == 1) continue;
    if (strides[next] < extent) return false;
    extent = strides[next] * shape[next];
  }
  return true;
}

Rows rows(PyObject* o, const char* name, Shape shape, const First& f, bool output = false) {
  const Tensor& t = tensor(o, name);
  check(t, name, shape, f.type, f.device);
  Rows r;
  r.data = t.data_ptr();
  if (t.is_contiguous()) return r;
  r.plain = false;
  for (int i = 0; i < 3; ++i) r.strides[i] = shape[i] > 1 ? t.stride(i) : 0;  // no step, whatever the stride says
  if (t.stride(3) != 1 || ((r.strides[0] | r.strides[1] | r.strides[2]) & 7))
    refuse_value(name, " needs contiguous rows of d elements that start on 16-byte boundaries, got strides ", t.strides());
  if (output && !nested(shape, r.strides))
    refuse_value(name, " is written: its rows must not share memory, got strides ", t.strides());
  return r;
}

// An output: the caller's tensor, checked, or a new one.
struct Output {
  PyObject* object = nullptr;  // owned
  void* data = nullptr;
  Output() = default;
  Output(const Output&) = delete;
  Output& operator=(const Output&) = delete;
  ~Output() { Py_XDECREF(object); }
  void make(Shape shape, at::ScalarType type, const c10::Device& device) {
    Tensor t = at::detail::empty_cuda(shape, type, device, std::nullopt);
    data = t.data_ptr();
    object = THPVariable_Wrap(std::move(t));
    if (object == nullptr) throw python_error();
  }
  void take(PyObject* o, const char* name, Shape shape, at::ScalarType type, const c10::Device& device) {
    if (none(o)) return make(shape, type, device);
    data = ptr(o, name, shape, type, device);
    object = Py_NewRef(o);
  }
  PyObject* release() {
    PyObject* o = object != nullptr ? object : Py_NewRef(Py_None);
    object = nullptr;
    return o;
  }
};

PyObject* tuple(std::initializer_list<Output*> outs) {
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(outs.size()));
  if (t == nullptr) throw python_error();
  Py_ssize_t i = 0;
  for (Output* o : outs) PyTuple_SET_ITEM(t, i++, o->release());
  return t;
}

// A workspace: the caller's tensor, or a new one of `need` bytes.
struct Workspace {
  Tensor own;
  void* data = nullptr;
  size_t bytes = 0;
  void take(PyObject* o, size_t need, const c10::Device& device) {
    if (none(o)) {
      own = at::detail::empty_cuda({static_cast<int64_t>(need > 16 ? need : 16)}, at::kByte, device, std::nullopt);
      data = own.data_ptr();
      bytes = need;
      return;
    }
    const Tensor& t = tensor(o, "workspace");
    if (t.device() != device || !t.is_contiguous()) refuse_value("workspace must be a contiguous tensor on ", device);
    data = t.data_ptr();
    bytes = t.nbytes();
  }
};

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}

// Makes the call's device current, and the caller's stream (a torch stream or a
// raw handle) where one is given: what is allocated for the call then belongs to
// the stream that it runs on, so a workspace that is released on return is not
// handed out again before the kernels are through with it.
struct Target {
  c10::cuda::CUDAGuard device;
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  void* stream;

  Target(PyObject* o, const c10::Device& d) : device(d) {
    if (none(o)) {
      stream = c10::cuda::getCurrentCUDAStream(d.index()).stream();
      return;
    }
    PyObject* handle = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : Py_NewRef(o);
    if (handle == nullptr) throw python_error();
    stream = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (stream == nullptr && PyErr_Occurred()) throw python_error();
    guard.emplace(stream == nullptr
                      ? c10::cuda::getDefaultCUDAStream(d.index())
                      : c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), d.index()));
  }
};

void done(int rc, const char* name) {
  if (rc == GBATTN_OK) return;
  PyObject* e = g_error != nullptr ? PyObject_CallFunction(g_error, "is", rc, name) : nullptr;
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_Format(PyExc_RuntimeError, "%s: %s", name, gbattn_error_string(rc));
  }
  throw python_error();
}

// The position rotation's table.
struct Rope {
  const float* table = nullptr;
  int rows = 0, rot = 0;
  Rope(PyObject* o, const c10::Device& device) {
    if (none(o)) return;
    const Tensor& t = tensor_of_dims(o, "rope", 2);
    table = static_cast<const float*>(ptr(o, "rope", t.sizes(), at::kFloat, device));
    rows = size(t.size(0), "rope");
    rot = size(t.size(1), "rope");
  }
};

// Positions of several axes: the axis of each pair of the rotation.
struct PairAxes {
  unsigned char of[256];
  int n = 0;  // axes; 0: one position
  PairAxes(PyObject* o, PyObject* positions, const Rope& rope) {
    if (none(o)) return;
    if (rope.table == nullptr) refuse_value("axes without rope");
    const int64_t axes = tensor_of_dims(positions, "positions (with axes)", 3).size(0);
    if (axes < 1 || axes > 4) refuse_value("positions must be of 1 to 4 axes, got ", axes);
    // A tuple of this call's own: what turns an entry into a number may be Python code,
    // which could change a list meanwhile.
    PyObject* seq = PySequence_Tuple(o);
    if (seq == nullptr) throw python_error();
    const Py_ssize_t pairs = PyTuple_GET_SIZE(seq);
    bool fits = pairs == rope.rot / 2 && pairs <= static_cast<Py_ssize_t>(sizeof(of));
    for (Py_ssize_t i = 0; fits && i < pairs; ++i) {
      const long v = PyLong_AsLong(PyTuple_GET_ITEM(seq, i));
      if (v == -1 && PyErr_Occurred()) {
        Py_DECREF(seq);
        throw python_error();
      }
      fits = v >= 0 && v < axes;
      of[i] = static_cast<unsigned char>(v);
    }
    Py_DECREF(seq);
    if (!fits)
      refuse_value("axes must be one of the ", axes, " axes for each of the rotation's ", rope.rot / 2, " pairs");
    n = static_cast<int>(axes);
  }
};

// What both directions of the norm take.
struct NormRope {
  First f;
  int B, H, S, d, Hkv;
  Rows q, k;
  const float *q_weight = nullptr, *k_weight = nullptr;
  Rope rope;
  PairAxes axes;
  const int* positions;
  int64_t q_shape[4], k_shape[4];

  NormRope(PyObject* qo, PyObject* ko, PyObject* qw, PyObject* kw, PyObject* ro, PyObject* po, PyObject* ao)
      : f(first(qo, "q")), rope(ro, f.device), axes(ao, po, rope) {
    const Tensor& qt = THPVariable_Unpack(qo);
    const int64_t heads = tensor_of_dims(ko, "k", 4).size(1);
    for (int i = 0; i < 4; ++i) q_shape[i] = k_shape[i] = qt.size(i);
    k_shape[1] = heads;
    q = rows(qo, "q", q_shape, f);
    k = rows(ko, "k", k_shape, f);
    B = size(q_shape[0], "q");
    H = size(q_shape[1], "q");
    S = size(q_shape[2], "q");
    d = size(q_shape[3], "q");
    Hkv = size(heads, "k");
    if (none(qw) != none(kw))
      refuse_value("q_weight and k_weight go together: both, or neither (rotation alone)");
    if (none(qw) && none(ro)) refuse_value("nothing to do: neither norm weights nor a rotation table");
    q_weight = static_cast<const float*>(opt(qw, "q_weight", {q_shape[3]}, at::kFloat, f.device));
    k_weight = static_cast<const float*>(opt(kw, "k_weight", {q_shape[3]}, at::kFloat, f.device));
    positions = static_cast<const int*>(
        axes.n > 0 ? ptr(po, "positions", {axes.n, q_shape[0], q_shape[2]}, at::kInt, f.device)
                   : opt(po, "positions", {q_shape[0], q_shape[2]}, at::kInt, f.device));
    if (none(po) && !none(ro) && rope.rows < S) refuse_value("rope has ", rope.rows, " rows for ", S, " tokens");
  }
};

PyObject* norm_rope(PyObject* const* a) {
  NormRope n(a[0], a[1], a[2], a[3], a[4], a[5], a[11]);
  const Target target(a[10], n.f.device);
  Output q_out, k_out;
  q_out.take(a[8], "q_out", n.q_shape, n.f.type, n.f.device);
  k_out.take(a[9], "k_out", n.k_shape, n.f.type, n.f.device);
  if (n.axes.n > 0)
    done(attn_qk_norm_rope_axes(n.q.data, n.k.data, n.q_weight, n.k_weight, n.rope.table, n.positions, n.axes.of,
                                q_out.data, k_out.data, n.B, n.H, n.Hkv, n.S, n.d, n.axes.n, n.q.stride(),
                                n.k.stride(), static_cast<float>(number(a[6])), n.rope.rows, n.rope.rot, truth(a[7]),
                                n.f.code, target.stream),
         "attn_qk_norm_rope_axes");
  else
    done(attn_qk_norm_rope(n.q.data, n.k.data, n.q_weight, n.k_weight, n.rope.table, n.positions, q_out.data, k_out.data,
                           n.B, n.H, n.Hkv, n.S, n.d, n.q.stride(), n.k.stride(), static_cast<float>(number(a[6])),
                           n.rope.rows, n.rope.rot, truth(a[7]), n.f.code, target.stream),
         "attn_qk_norm_rope");
  return tuple({&q_out, &k_out});
}

PyObject* norm_rope_bwd(PyObject* const* a) {
  NormRope n(a[2], a[3], a[4], a[5], a[6], a[7], a[16]);
  const Target target(a[15], n.f.device);
  const void* dqo = ptr(a[0], "dq_out", n.q_shape, n.f.type, n.f.device);
  const void* dko = ptr(a[1], "dk_out", n.k_shape, n.f.type, n.f.device);
  Output dq, dk, dqw, dkw;
  Rows dq_rows, dk_rows;
  if (none(a[11])) {
    dq.make(n.q_shape, n.f.type, n.f.device);
    dq_rows.data = dq.data;
  } else {
    dq_rows = rows(a[11], "dq", n.q_shape, n.f, true);
    dq.object = Py_NewRef(a[11]);
  }
  if (none(a[12])) {
    dk.make(n.k_shape, n.f.type, n.f.device);
    dk_rows.data = dk.data;
  } else {
    dk_rows = rows(a[12], "dk", n.k_shape, n.f, true);
    dk.object = Py_NewRef(a[12]);
  }
  Workspace ws;
  if (n.q_weight != nullptr) {
    dqw.take(a[13], "dq_weight", {n.d}, at::kFloat, n.f.device);
    dkw.take(a[14], "dk_weight", {n.d}, at::kFloat, n.f.device);
    ws.take(a[10], attn_qk_norm_rope_bwd_workspace_bytes(n.d), n.f.device);
  }
  float *dqwp = static_cast<float*>(dqw.data), *dkwp = static_cast<float*>(dkw.data);
  const float eps = static_cast<float>(number(a[8]));
  const int il = truth(a[9]);
  if (n.axes.n > 0)
    done(attn_qk_norm_rope_axes_bwd(dqo, dko, n.q.data, n.k.data, n.q_weight, n.k_weight, n.rope.table, n.positions,
                                    n.axes.of, dq_rows.data, dk_rows.data, dqwp, dkwp, n.B, n.H, n.Hkv, n.S, n.d,
                                    n.axes.n, n.q.stride(), n.k.stride(), dq_rows.stride(), dk_rows.stride(), eps,
                                    n.rope.rows, n.rope.rot, il, ws.data, ws.bytes, n.f.code, target.stream),
         "attn_qk_norm_rope_axes_bwd");
  else
    done(attn_qk_norm_rope_bwd(dqo, dko, n.q.data, n.k.data, n.q_weight, n.k_weight, n.rope.table, n.positions,
                               dq_rows.data, dk_rows.data, dqwp, dkwp, n.B, n.H, n.Hkv, n.S, n.d, n.q.stride(),
                               n.k.stride(), dq_rows.stride(), dk_rows.stride(), eps, n.rope.rows, n.rope.rot, il,
                               ws.data, ws.bytes, n.f.code, target.stream),
         "attn_qk_norm_rope_bwd");
  return tuple({&dq, &dk, &dqw, &dkw});
}

// A paged cache's tensors, checked against its first one.
struct Cache {
  void *k = nullptr, *v = nullptr, *k_factors = nullptr, *v_factors = nullptr;
  const float *k_descale = nullptr, *v_descale = nullptr;
  const int *table, *lens;
  int page, n_pages, max_pages;

  void tables(PyObject* to, PyObject* lo, int64_t B, const c10::Device& device) {
    const int64_t width = tensor_of_dims(to, "page_table", 2).size(1);
    table = static_cast<const int*>(ptr(to, "page_table", {B, width}, at::kInt, device));
    lens = static_cast<const int*>(ptr(lo, "seqlens", {B}, at::kInt, device));
    max_pages = size(width, "page_table");
  }
  // 16 bits
  Cache(PyObject* ko, PyObject* vo, PyObject* to, PyObject* lo, int64_t B, int64_t Hkv, int64_t d, const First& f) {
    const Tensor& kt = tensor_of_dims(ko, "k_cache", 4);
    if (kt.size(1) != Hkv || kt.size(3) != d)
      refuse_value("k_cache must be a tensor [n_pages, ", Hkv, ", page_size, ", d, "], got ", kt.sizes());
    k = ptr(ko, "k_cache", kt.sizes(), f.type, f.device);
    v = ptr(vo, "v_cache", kt.sizes(), f.type, f.device);
    n_pages = size(kt.size(0), "k_cache");
    page = size(kt.size(2), "k_cache");
    tables(to, lo, B, f.device);
  }
  // 4 bits: c = k_codes, k_factors, v_codes, v_factors, page_table, seqlens
  Cache(PyObject* const* c, PyObject* kd, PyObject* vd, int64_t B, int64_t Hkv, int64_t d, const c10::Device& device) {
    const Tensor& kt = tensor_of_dims(c[0], "k_codes", 4);
    if (kt.size(1) != Hkv || kt.size(3) * 2 != d)
      refuse_value("k_codes must be a tensor [n_pages, ", Hkv, ", page_size, ", d / 2, "], got ", kt.sizes());
    const int64_t factors[4] = {kt.size(0), Hkv, kt.size(2), d / 16};
    // E4M3 values, or their bytes; both factors alike
    const auto type = tensor(c[1], "k_factors").scalar_type() == at::kByte ? at::kByte : at::kFloat8_e4m3fn;
    k = ptr(c[0], "k_codes", kt.sizes(), at::kByte, device);
    k_factors = ptr(c[1], "k_factors", factors, type, device);
    v = ptr(c[2], "v_codes", kt.sizes(), at::kByte, device);
    v_factors = ptr(c[3], "v_factors", factors, type, device);
    k_descale = static_cast<const float*>(opt(kd, "k_descale", {Hkv}, at::kFloat, device));
    v_descale = static_cast<const float*>(opt(vd, "v_descale", {Hkv}, at::kFloat, device));
    n_pages = size(kt.size(0), "k_codes");
    page = size(kt.size(2), "k_codes");
    tables(c[4], c[5], B, device);
  }
};

PyObject* append(const First& f, const Tensor& kt, PyObject* ko, PyObject* vo, const Cache& c, PyObject* new_lens,
                 PyObject* rope_o, PyObject* interleaved, PyObject* qo, PyObject* q_out, PyObject* stream,
                 PyObject* positions_o, PyObject* axes_o, bool fp4) {
  const Rows k = rows(ko, "k", kt.sizes(), f), v = rows(vo, "v", kt.sizes(), f);
  const int B = size(kt.size(0), "k"), Hkv = size(kt.size(1), "k"), S = size(kt.size(2), "k");
  const int d = size(kt.size(3), "k");
  const Target target(stream, f.device);
  int H = Hkv;
  Rows q;
  Output out;
  if (!none(qo)) {
    const int64_t heads = tensor_of_dims(qo, "q", 4).size(1);
    const int64_t shape[4] = {B, heads, S, d};
    q = rows(qo, "q", shape, f);
    H = size(heads, "q");
    out.take(q_out, "q_out", shape, f.type, f.device);
  } else if (!none(q_out)) {
    refuse_value("q_out without q");
  }
  const int* n = static_cast<const int*>(opt(new_lens, "new_lens", {B}, at::kInt, f.device));
  const Rope rope(rope_o, f.device);
  PairAxes axes(axes_o, positions_o, rope);
  const int* positions = nullptr;
  if (axes.n > 0) {
    positions = static_cast<const int*>(ptr(positions_o, "positions", {axes.n, B, S}, at::kInt, f.device));
  } else if (!none(positions_o)) {  // one axis for all pairs
    if (rope.table == nullptr) refuse_value("positions without rope");
    positions = static_cast<const int*>(ptr(positions_o, "positions", {B, S}, at::kInt, f.device));
    axes.n = 1;
    std::memset(axes.of, 0, sizeof(axes.of));
  }
  void* s = target.stream;
  const int il = truth(interleaved);
  if (axes.n > 0) {
    // The C library reads rot_dim / 2 of them, after it has bounded rot_dim by d.
    if (fp4)
      done(attn_cache_append_axes_fp4(k.data, v.data, c.k, c.k_factors, c.v, c.v_factors, c.k_descale, c.v_descale,
                                      c.table, c.lens, n, rope.table, positions, axes.of, q.data, out.data, B, H, Hkv,
                                      S, d, axes.n, c.page, c.n_pages, c.max_pages, q.stride(), k.stride(),
                                      v.stride(), rope.rows, rope.rot, il, f.code, s),
           "attn_cache_append_axes_fp4");
    else
      done(attn_cache_append_axes(k.data, v.data, c.k, c.v, c.table, c.lens, n, rope.table, positions, axes.of, q.data,
                                  out.data, B, H, Hkv, S, d, axes.n, c.page, c.n_pages, c.max_pages, q.stride(),
                                  k.stride(), v.stride(), rope.rows, rope.rot, il, f.code, s),
           "attn_cache_append_axes");
    return out.release();
  }
  if (fp4)
    done(attn_cache_append_fp4(k.data, v.data, c.k, c.k_factors, c.v, c.v_factors, c.k_descale, c.v_descale, c.table,
                               c.lens, n, rope.table, q.data, out.data, B, H, Hkv, S, d, c.page, c.n_pages,
                               c.max_pages, q.stride(), k.stride(), v.stride(), rope.rows, rope.rot, il, f.code, s),
         "attn_cache_append_fp4");
  else
    done(attn_cache_append(k.data, v.data, c.k, c.v, c.table, c.lens, n, rope.table, q.data, out.data, B, H, Hkv, S, d,
                           c.page, c.n_pages, c.max_pages, q.stride(), k.stride(), v.stride(), rope.rows, rope.rot, il,
                           f.code, s),
         "attn_cache_append");
  return out.release();
}

PyObject* cache_append(PyObject* const* a) {
  const First f = first(a[0], "k");
  const Tensor& k = THPVariable_Unpack(a[0]);
  const Cache c(a[2], a[3], a[4], a[5], k.size(0), k.size(1), k.size(3), f);
  return append(f, k, a[0], a[1], c, a[6], a[7], a[8], a[9], a[10], a[11], a[12], a[13], false);
}

PyObject* cache_append_fp4(PyObject* const* a) {
  const First f = first(a[0], "k");
  const Tensor& k = THPVariable_Unpack(a[0]);
  const Cache c(a + 2, a[9], a[10], k.size(0), k.size(1), k.size(3), f.device);
  return append(f, k, a[0], a[1], c, a[8], a[11], a[12], a[13], a[14], a[15], a[16], a[17], true);
}

int tokens(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v < 1 || v > INT_MAX) refuse_value("S must be in 1 .. ", INT_MAX, ", got ", v);
  return static_cast<int>(v);
}

PyObject* cache_gather(PyObject* const* a) {
  const First f = first(a[0], "k_cache");
  const Tensor& kt = THPVariable_Unpack(a[0]);
  const int64_t B = tensor_of_dims(a[3], "seqlens", 1).size(0);
  const Cache c(a[0], a[1], a[2], a[3], B, kt.size(1), kt.size(3), f);
  const int S = tokens(a[4]);
  const int64_t shape[4] = {B, kt.size(1), S, kt.size(3)};
  const Target target(a[7], f.device);
  Output k, v;
  k.take(a[5], "k_out", shape, f.type, f.device);
  v.take(a[6], "v_out", shape, f.type, f.device);
  done(attn_cache_gather(c.k, c.v, c.table, c.lens, k.data, v.data, size(B, "seqlens"), size(shape[1], "k_cache"), S,
                         size(shape[3], "k_cache"), c.page, c.n_pages, c.max_pages, f.code, target.stream),
       "attn_cache_gather");
  return tuple({&k, &v});
}

PyObject* cache_gather_fp4(PyObject* const* a) {
  const Tensor& kt = tensor_of_dims(a[0], "k_codes", 4);
  if (!kt.is_cuda()) refuse_value("k_codes must be a CUDA tensor (there is no CPU path)");
  if (!THPDtype_Check(a[9])) refuse_type("dtype must be a torch.dtype");
  const at::ScalarType type = reinterpret_cast<THPDtype*>(a[9])->scalar_type;
  const First f{type, kt.device(), dtype_code(type, "the outputs")};
  const int64_t B = tensor_of_dims(a[5], "seqlens", 1).size(0);
  const Cache c(a, a[7], a[8], B, kt.size(1), kt.size(3) * 2, f.device);
  const int S = tokens(a[6]);
  const int64_t shape[4] = {B, kt.size(1), S, kt.size(3) * 2};
  const Target target(a[12], f.device);
  Output k, v;
  k.take(a[10], "k_out", shape, f.type, f.device);
  v.take(a[11], "v_out", shape, f.type, f.device);
  done(attn_cache_gather_fp4(c.k, c.k_factors, c.v, c.v_factors, c.k_descale, c.v_descale, c.table, c.lens, k.data,
                             v.data, size(B, "seqlens"), size(shape[1], "k_codes"), S, size(shape[3], "k_codes"), c.page,
                             c.n_pages, c.max_pages, f.code, target.stream),
       "attn_cache_gather_fp4");
  return tuple({&k, &v});
}

PyObject* decode(const First& f, PyObject* qo, int64_t Hkv, const Cache& c, PyObject* scale_o, PyObject* workspace,
                 PyObject* out_o, PyObject* lse_o, PyObject* return_lse, PyObject* stream, bool fp4) {
  const Tensor& q = THPVariable_Unpack(qo);
  if (q.size(2) != 1) refuse_value("decode takes exactly one query per sequence: q [B,Hq,1,d]");
  const void* q_ptr = ptr(qo, "q", q.sizes(), f.type, f.device);
  const int B = size(q.size(0), "q"), H = size(q.size(1), "q"), d = size(q.size(3), "q"), hkv = size(Hkv, "the cache");
  const int64_t cap = static_cast<int64_t>(c.page) * c.max_pages;
  const Target target(stream, f.device);
  Workspace ws;
  ws.take(workspace, attn_decode_paged_workspace_bytes(B, H, hkv, d, static_cast<int>(cap < INT_MAX ? cap : INT_MAX)),
          f.device);
  Output out, lse;
  out.take(out_o, "out", q.sizes(), f.type, f.device);
  if (!none(lse_o) || truth(return_lse)) lse.take(lse_o, "lse", {B, H}, at::kFloat, f.device);
  const float scale = static_cast<float>(none(scale_o) ? 1.0 / std::sqrt(static_cast<double>(d)) : number(scale_o));
  void* s = target.stream;
  if (fp4)
    done(attn_decode_paged_fp4(q_ptr, c.k, c.k_factors, c.v, c.v_factors, c.k_descale, c.v_descale, c.table, c.lens,
                               out.data, static_cast<float*>(lse.data), B, H, hkv, d, c.page, c.n_pages, c.max_pages,
                               scale, ws.data, ws.bytes, f.code, s),
         "attn_decode_paged_fp4");
  else
    done(attn_decode_paged(q_ptr, c.k, c.v, c.table, c.lens, out.data, static_cast<float*>(lse.data), B, H, hkv, d,
                           c.page, c.n_pages, c.max_pages, scale, ws.data, ws.bytes, f.code, s),
         "attn_decode_paged");
  return tuple({&out, &lse});
}

PyObject* decode_paged(PyObject* const* a) {
  const First f = first(a[0], "q");
  const Tensor& q = THPVariable_Unpack(a[0]);
  const int64_t Hkv = tensor_of_dims(a[1], "k_cache", 4).size(1);
  const Cache c(a[1], a[2], a[3], a[4], q.size(0), Hkv, q.size(3), f);
  return decode(f, a[0], Hkv, c, a[5], a[6], a[7], a[8], a[9], a[10], false);
}

PyObject* decode_paged_fp4(PyObject* const* a) {
  const First f = first(a[0], "q");
  const Tensor& q = THPVariable_Unpack(a[0]);
  const int64_t Hkv = tensor_of_dims(a[1], "k_codes", 4).size(1);
  const Cache c(a + 1, a[7], a[8], q.size(0), Hkv, q.size(3), f.device);
  return decode(f, a[0], Hkv, c, a[9], a[10], a[11], a[12], a[13], a[14], true);
}

// Device memory that a call reads or writes.
struct Range {
  const char* name;
  const void* data;
  int64_t bytes;
};

// Refuses an output that the caller gave and that shares memory with one of `others`
// (contiguous tensors; those of no bytes or that are not given do not count).
void check_apart(const Range& out, std::initializer_list<Range> others) {
  const char* const begin = static_cast<const char*>(out.data);
  for (const Range& r : others) {
    const char* const b = static_cast<const char*>(r.data);
    if (b != nullptr && begin < b + r.bytes && b < begin + out.bytes)
      refuse_value(out.name, " is written: it must not share memory with ", r.name);
  }
}

// c, the cache, is checked against q [B, H, S, d]; o = out, lse, return_lse, stream.
PyObject* fwd_paged(const First& f, PyObject* qo, int64_t Hkv, const Cache& c, PyObject* new_lens, PyObject* scale_o,
                    PyObject* causal_o, PyObject* workspace, PyObject* const* o, bool fp4) {
  const Tensor& q = THPVariable_Unpack(qo);
  const void* q_ptr = ptr(qo, "q", q.sizes(), f.type, f.device);
  const int B = size(q.size(0), "q"), H = size(q.size(1), "q"), S = size(q.size(2), "q"), d = size(q.size(3), "q");
  const int hkv = size(Hkv, "the cache");
  const int* n = static_cast<const int*>(opt(new_lens, "new_lens", {B}, at::kInt, f.device));
  const int causal = truth(causal_o);
  const float scale = static_cast<float>(none(scale_o) ? 1.0 / std::sqrt(static_cast<double>(d)) : number(scale_o));
  const int64_t cap = static_cast<int64_t>(c.page) * c.max_pages;
  const Target target(o[3], f.device);
  Workspace ws;
  ws.take(workspace, attn_fwd_paged_workspace_bytes(B, H, hkv, S, d, static_cast<int>(cap < INT_MAX ? cap : INT_MAX)),
          f.device);
  Output out, lse;
  out.take(o[0], "out", q.sizes(), f.type, f.device);
  if (!none(o[1]) || truth(o[2])) lse.take(o[1], "lse", {B, H, S}, at::kFloat, f.device);
  const int64_t slots = static_cast<int64_t>(c.n_pages) * hkv * c.page;
  const int64_t queries = static_cast<int64_t>(B) * H * S, row = fp4 ? d / 2 : 2 * d;
  const Range out_range{"out", out.data, queries * d * 2}, lse_range{"lse", lse.data, queries * 4};
  auto apart = [&](const Range& own, const Range& other) {
    check_apart(own, {{"q", q_ptr, queries * d * 2},
                      {"the keys' pool", c.k, slots * row},
                      {"the values' pool", c.v, slots * row},
                      {"k_factors", c.k_factors, slots * (d / 16)},
                      {"v_factors", c.v_factors, slots * (d / 16)},
                      {"k_descale", c.k_descale, 4LL * hkv},
                      {"v_descale", c.v_descale, 4LL * hkv},
                      {"page_table", c.table, 4LL * B * c.max_pages},
                      {"seqlens", c.lens, 4LL * B},
                      {"new_lens", n, 4LL * B},
                      {"workspace", ws.data, static_cast<int64_t>(ws.bytes)},
                      other});
  };
  if (!none(o[0])) apart(out_range, lse_range);
  if (!none(o[1])) apart(lse_range, out_range);
  if (fp4)
    done(attn_fwd_paged_fp4(q_ptr, c.k, c.k_factors, c.v, c.v_factors, c.k_descale, c.v_descale, c.table, c.lens, n,
                            out.data, static_cast<float*>(lse.data), B, H, hkv, S, d, c.page, c.n_pages, c.max_pages,
                            scale, causal, ws.data, ws.bytes, f.code, target.stream),
         "attn_fwd_paged_fp4");
  else
    done(attn_fwd_paged(q_ptr, c.k, c.v, c.table, c.lens, n, out.data, static_cast<float*>(lse.data), B, H, hkv, S, d,
                        c.page, c.n_pages, c.max_pages, scale, causal, ws.data, ws.bytes, f.code, target.stream),
         "attn_fwd_paged");
  return tuple({&out, &lse});
}

PyObject* forward_paged(PyObject* const* a) {
  const First f = first(a[0], "q");
  const Tensor& q = THPVariable_Unpack(a[0]);
  const int64_t Hkv = tensor_of_dims(a[1], "k_cache", 4).size(1);
  const Cache c(a[1], a[2], a[3], a[4], q.size(0), Hkv, q.size(3), f);
  return fwd_paged(f, a[0], Hkv, c, a[5], a[6], a[7], a[8], a + 9, false);
}

PyObject* forward_paged_fp4(PyObject* const* a) {
  const First f = first(a[0], "q");
  const Tensor& q = THPVariable_Unpack(a[0]);
  const int64_t Hkv = tensor_of_dims(a[1], "k_codes", 4).size(1);
  const Cache c(a + 1, a[8], a[9], q.size(0), Hkv, q.size(3), f.device);
  return fwd_paged(f, a[0], Hkv, c, a[7], a[10], a[11], a[12], a + 13, true);
}

// A function of N positional arguments; no C++ exception leaves it.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.message.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XDECREF(g_error);
  g_error = Py_NewRef(cls);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"set_error", set_error, METH_O, nullptr},
    method<norm_rope, 12>("attn_qk_norm_rope"),
    method<norm_rope_bwd, 17>("attn_qk_norm_rope_bwd"),
    method<cache_append, 14>("attn_cache_append"),
    method<cache_append_fp4, 18>("attn_cache_append_fp4"),
    method<cache_gather, 8>("attn_cache_gather"),
    method<cache_gather_fp4, 13>("attn_cache_gather_fp4"),
    method<forward_paged, 13>("attn_fwd_paged"),
    method<forward_paged_fp4, 17>("attn_fwd_paged_fp4"),
    method<decode_paged, 11>("attn_decode_paged"),
    method<decode_paged_fp4, 15>("attn_decode_paged_fp4"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }
