// The quick way from a Python call to the library for the calls that a serving step
// makes between its products (moe_gate, moe_route, moe_kv_pages, moe_verify_drafts).
// In Python the checks of a call's tensors can take longer than its launch or its kernel (12
// tensors: a call among others took 7.8 us, here 3.8).  A call that is not as
// it should be is not refused here but left to the Python binding, which makes the
// same checks and says what is wrong.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "../../include/moe_fp8.h"

namespace {

constexpr int kLeftToPython = 1;      // library calls return 0 or less

int (*g_gate)(const moe_gate_desc*, void*) = nullptr;
int (*g_route)(const moe_route_desc*, void*) = nullptr;
int (*g_pages)(const moe_kv_pages_desc*, void*) = nullptr;
int (*g_verify)(const moe_verify_desc*, void*) = nullptr;

struct NotQuick {};                   // thrown where Python has to look

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw NotQuick{};
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda()) throw NotQuick{};
  return t;
}

// What a call's tensors have in common: the GPU, which has to be the current one.
struct Call {
  int device;
  explicit Call(const at::Tensor& t) : device(t.get_device()) {
    if (c10::cuda::current_device() != device) throw NotQuick{};
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }

  // a [rows, cols] tensor of contiguous rows; the stride of a single row is never used, and may be anything
  template <class T>
  T* rows(const at::Tensor& t, int64_t n, int64_t cols, at::ScalarType type, int64_t& ld) const {
    if (t.dim() != 2 || t.size(0) != n || t.size(1) != cols || t.scalar_type() != type || t.get_device() != device ||
        (cols != 1 && t.stride(1) != 1))
      throw NotQuick{};
    ld = n > 1 ? t.stride(0) : cols;
    return static_cast<T*>(t.data_ptr());
  }
  // n contiguous elements; NULL for None
  template <class T>
  T* flat(PyObject* o, int64_t n, at::ScalarType type) const {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    if (t.numel() != n || t.scalar_type() != type || t.get_device() != device || !t.is_contiguous()) throw NotQuick{};
    return static_cast<T*>(t.data_ptr());
  }
  template <class T>
  T* some(PyObject* o, int64_t n, at::ScalarType type) const {
    if (o == Py_None) throw NotQuick{};
    return flat<T>(o, n, type);
  }
};

int32_t number(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if ((v == -1 && PyErr_Occurred()) || v != static_cast<int32_t>(v)) throw NotQuick{};
  return static_cast<int32_t>(v);
}

int32_t dtype_of(const at::Tensor& t, bool wide) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MOE_DTYPE_BF16;
    case at::kHalf: return MOE_DTYPE_F16;
    case at::kFloat:
      if (wide) return MOE_DTYPE_F32;
      [[fallthrough]];
    default: throw NotQuick{};
  }
}

// Runs `call` and hands its status back; whatever C++ throws is left to Python.
template <class F>
PyObject* quick(Py_ssize_t n, Py_ssize_t wanted, F call) {
  int rc = kLeftToPython;
  try {
    if (n == wanted) rc = call();
  } catch (...) {
    PyErr_Clear();
  }
  return PyLong_FromLong(rc);
}

// The call itself, in which other Python threads run: a launch waits where the stream's queue is full,
// maybe behind a function of the host that needs the interpreter.
template <class Desc>
int launch(int (*f)(const Desc*, void*), const Desc& d, void* stream) {
  PyThreadState* state = PyEval_SaveThread();
  const int rc = f(&d, stream);
  PyEval_RestoreThread(state);
  return rc;
}

// gate(x, w, logits, err)
PyObject* gate(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return quick(n, 4, [&] {
    const at::Tensor &x = tensor(a[0]), &w = tensor(a[1]), &logits = tensor(a[2]);
    if (x.dim() != 2 || w.dim() != 2) throw NotQuick{};
    const Call c(x);
    moe_gate_desc d{};
    const int64_t T = x.size(0), H = x.size(1), E = w.size(0);
    if (H > INT32_MAX || E > INT32_MAX) throw NotQuick{};
    d.dtype = dtype_of(x, false);
    d.x = c.rows<void>(x, T, H, x.scalar_type(), d.x_ld);
    d.w = c.rows<void>(w, E, H, x.scalar_type(), d.w_ld);
    d.logits = c.rows<float>(logits, T, E, at::kFloat, d.logits_ld);
    d.err = c.flat<int32_t>(a[3], 1, at::kInt);
    d.T = T;
    d.E = static_cast<int32_t>(E);
    d.H = static_cast<int32_t>(H);
    return launch(g_gate, d, c.stream());
  });
}

// route(logits, topk_ids, topk_w, bias, n_tokens, n_group, topk_group, scale, flags)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return quick(n, 9, [&] {
    const at::Tensor &z = tensor(a[0]), &ids = tensor(a[1]), &w = tensor(a[2]);
    if (z.dim() != 2 || ids.dim() != 2) throw NotQuick{};
    const Call c(z);
    moe_route_desc d{};
    const int64_t T = z.size(0), E = z.size(1), k = ids.size(1);
    if (E > INT32_MAX || k > INT32_MAX) throw NotQuick{};
    d.dtype = dtype_of(z, true);
    d.logits = c.rows<void>(z, T, E, z.scalar_type(), d.logits_ld);
    d.topk_ids = c.rows<int32_t>(ids, T, k, at::kInt, d.ids_ld);
    d.topk_w = c.rows<float>(w, T, k, at::kFloat, d.w_ld);
    d.bias = c.flat<float>(a[3], E, at::kFloat);
    d.n_tokens = c.flat<int32_t>(a[4], 1, at::kInt);
    d.T = T;
    d.E = static_cast<int32_t>(E);
    d.k = static_cast<int32_t>(k);
    d.n_group = number(a[5]);
    d.topk_group = number(a[6]);
    const double scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) throw NotQuick{};
    d.scale = static_cast<float>(scale);
    d.flags = number(a[8]);
    return launch(g_route, d, c.stream());
  });
}

// kv_pages(kv_old, n_new, page_table, free_list, free_count, page_size, kv_len, cu_new, free_count_out, kv_keep, seqs,
//          positions, slots, err)
PyObject* kv_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return quick(n, 14, [&] {
    const at::Tensor &table = tensor(a[2]), &list = tensor(a[3]);
    if (table.dim() != 2) throw NotQuick{};
    const Call c(tensor(a[0]));
    moe_kv_pages_desc d{};
    const int64_t batch = table.size(0), max_pages = table.size(1);
    if (batch > INT32_MAX || max_pages > INT32_MAX) throw NotQuick{};
    d.kv_old = c.some<int32_t>(a[0], batch, at::kInt);
    d.n_new = c.some<int32_t>(a[1], batch, at::kInt);
    d.page_table = c.rows<int32_t>(table, batch, max_pages, at::kInt, d.table_ld);
    d.free_capacity = list.numel();
    d.free_list = c.some<int32_t>(a[3], d.free_capacity, at::kInt);
    d.free_count = c.some<int32_t>(a[4], 1, at::kInt);
    d.page_size = number(a[5]);
    d.kv_len = c.some<int32_t>(a[6], batch, at::kInt);
    d.cu_new = c.some<int32_t>(a[7], batch + 1, at::kInt);
    d.free_count_out = c.some<int32_t>(a[8], 1, at::kInt);
    d.kv_keep = c.flat<int32_t>(a[9], batch, at::kInt);
    d.rows = 1 << 30;                      // no row tensors: nothing limits the rows
    for (int i = 12; i >= 10; --i)
      if (a[i] != Py_None) d.rows = tensor(a[i]).numel();
    d.seqs = c.flat<int32_t>(a[10], d.rows, at::kInt);
    d.positions = c.flat<int32_t>(a[11], d.rows, at::kInt);
    d.slots = c.flat<int64_t>(a[12], d.rows, at::kLong);
    d.err = c.flat<int32_t>(a[13], 1, at::kInt);
    d.batch = static_cast<int32_t>(batch);
    d.max_pages = static_cast<int32_t>(max_pages);
    return launch(g_pages, d, c.stream());
  });
}

// verify(probs, tokens, cu_new, u_accept, u_sample, accepted, out_tokens, draft_probs, n_draft, kv_len, kv_keep, err)
PyObject* verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return quick(n, 12, [&] {
    const at::Tensor &p = tensor(a[0]), &out = tensor(a[6]);
    if (p.dim() != 2 || out.dim() != 2) throw NotQuick{};
    const Call c(p);
    moe_verify_desc d{};
    const int64_t T = p.size(0), batch = out.size(0), max_out = out.size(1);
    if (batch > INT32_MAX || max_out > INT32_MAX) throw NotQuick{};
    d.T = T;
    d.vocab = p.size(1);
    d.dtype = dtype_of(p, true);
    d.probs = c.rows<void>(p, T, d.vocab, p.scalar_type(), d.p_ld);
    if (a[7] != Py_None) d.draft_probs = c.rows<void>(tensor(a[7]), T, d.vocab, p.scalar_type(), d.q_ld);
    d.tokens = c.some<int32_t>(a[1], T, at::kInt);
    d.cu_new = c.some<int32_t>(a[2], batch + 1, at::kInt);
    d.u_accept = c.some<float>(a[3], T, at::kFloat);
    d.u_sample = c.some<float>(a[4], batch, at::kFloat);
    d.accepted = c.some<int32_t>(a[5], batch, at::kInt);
    d.out_tokens = c.rows<int32_t>(out, batch, max_out, at::kInt, d.out_ld);
    d.n_draft = c.flat<int32_t>(a[8], batch, at::kInt);
    d.kv_len = c.flat<int32_t>(a[9], batch, at::kInt);
    d.kv_keep = c.flat<int32_t>(a[10], batch, at::kInt);
    d.err = c.flat<int32_t>(a[11], 1, at::kInt);
    d.batch = static_cast<int32_t>(batch);
    d.max_out = static_cast<int32_t>(max_out);
    return launch(g_verify, d, c.stream());
  });
}

// connect(gate, route, kv_pages, verify): addresses of the library's entry points
PyObject* connect(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "connect: four addresses");
    return nullptr;
  }
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "connect: a null address");
      return nullptr;
    }
  }
  g_gate = reinterpret_cast<decltype(g_gate)>(p[0]);
  g_route = reinterpret_cast<decltype(g_route)>(p[1]);
  g_pages = reinterpret_cast<decltype(g_pages)>(p[2]);
  g_verify = reinterpret_cast<decltype(g_verify)>(p[3]);
  Py_RETURN_NONE;
}

// made_for(): the releases of torch and Python whose layouts this holds, and the descriptors' sizes
PyObject* made_for(PyObject*, PyObject* const*, Py_ssize_t) {
  return Py_BuildValue("(iiiiinnnn)", TORCH_VERSION_MAJOR, TORCH_VERSION_MINOR, TORCH_VERSION_PATCH, PY_MAJOR_VERSION, PY_MINOR_VERSION,
                       static_cast<Py_ssize_t>(sizeof(moe_gate_desc)), static_cast<Py_ssize_t>(sizeof(moe_route_desc)),
                       static_cast<Py_ssize_t>(sizeof(moe_kv_pages_desc)), static_cast<Py_ssize_t>(sizeof(moe_verify_desc)));
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"connect", FAST(connect)}, {"gate", FAST(gate)},     {"route", FAST(route)},
                         {"kv_pages", FAST(kv_pages)}, {"verify", FAST(verify)}, {"made_for", FAST(made_for)}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
