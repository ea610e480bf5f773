// binding.cpp -- native argument marshalling for the calls whose launch costs
// less than their checks do in Python (module _marshal).
//
// A step over the adapters of a model names hundreds of small tensors, seven
// per parameter: in Python their checks take longer than the step does on the
// GPU (32 parameters: about 70 us against 24 us), here a few us.  One decoded
// token through a layer of many adapters is 10 us of GPU time; its nine
// tensors, descriptors and stream take 6 us in Python, under one here.
// Only well-formed arguments are packed: for anything else (memory that two of
// the tensors written share too) the caller gets None and finds the fault and its message.
#define PY_SSIZE_T_CLEAN
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/qlora_nf4.h"

#include <algorithm>
#include <cstdint>
#include <exception>
#include <utility>
#include <vector>

namespace {

constexpr int64_t kBlock = 256;   // elements per 8-bit state block

const at::Tensor* tensor(PyObject* o) { return o && THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// (a subclass that dispatches to Python, such as a tracer's, has no memory of its own)
bool plain(const at::Tensor* t) {
  return t && t->defined() && !t->key_set().has(c10::DispatchKey::Python) && t->layout() == at::kStrided;
}

bool fits(const at::Tensor* t, at::ScalarType type, int64_t numel, int64_t device) {
  return plain(t) && t->scalar_type() == type && t->is_cuda() && t->get_device() == device && t->numel() == numel &&
         t->is_contiguous();
}

// An attribute, held while this lives; empty where there is none.
struct Attr {
  PyObject* o;
  Attr(PyObject* owner, PyObject* name) : o(PyObject_GetAttr(owner, name)) {
    if (!o) PyErr_Clear();
  }
  ~Attr() { Py_XDECREF(o); }
  Attr(const Attr&) = delete;
  Attr& operator=(const Attr&) = delete;

  // the tensor, if it has this type, device and (contiguous) shape
  const at::Tensor* of(at::ScalarType type, at::IntArrayRef shape, int64_t device) const {
    const at::Tensor* t = tensor(o);
    return t && t->defined() && t->sizes() == shape && fits(t, type, t->numel(), device) ? t : nullptr;
  }
  int64_t integer() const {
    const int64_t v = o ? PyLong_AsLongLong(o) : -1;
    if (PyErr_Occurred()) PyErr_Clear();
    return v;
  }
  // which of two words it is, or -1
  int word(const char* a, const char* b) const {
    if (!o || !PyUnicode_Check(o)) return -1;
    return PyUnicode_CompareWithASCIIString(o, a) == 0 ? 0 : PyUnicode_CompareWithASCIIString(o, b) == 0 ? 1 : -1;
  }
};

// adamw8(params, grads, states, masters, device) -> bytes of qlora_adamw8_tensor[n], or None.
// The first four are lists of one length; a state has the attributes of AdamW8State.
PyObject* adamw8(PyObject*, PyObject* const* a, Py_ssize_t na) {
  if (na != 5) {
    PyErr_SetString(PyExc_TypeError, "adamw8(params, grads, states, masters, device)");
    return nullptr;
  }
  for (int i = 0; i < 4; ++i)
    if (!PyList_CheckExact(a[i])) Py_RETURN_NONE;
  const Py_ssize_t n = PyList_GET_SIZE(a[0]);
  for (int i = 1; i < 4; ++i)
    if (PyList_GET_SIZE(a[i]) != n) Py_RETURN_NONE;
  const int64_t device = PyLong_AsLongLong(a[4]);
  if (device == -1 && PyErr_Occurred()) return nullptr;
  static PyObject* const names[4] = {PyUnicode_InternFromString("exp_avg"), PyUnicode_InternFromString("exp_root"),
                                     PyUnicode_InternFromString("exp_avg_scale"),
                                     PyUnicode_InternFromString("exp_root_scale")};
  std::vector<uint64_t> table((size_t)n * 8);   // (freed if a tensor throws)
  std::vector<std::pair<uint64_t, uint64_t>> written;   // first byte and end of what the step writes
  uint64_t* w = table.data();
  written.reserve((size_t)n * 6);
  bool ok = true;
  for (Py_ssize_t i = 0; ok && i < n; ++i, w += 8) {
    const at::Tensor* p = tensor(PyList_GET_ITEM(a[0], i));
    const at::Tensor* g = tensor(PyList_GET_ITEM(a[1], i));
    PyObject *state = PyList_GET_ITEM(a[2], i), *master = PyList_GET_ITEM(a[3], i);
    const int64_t numel = p ? p->numel() : 0, blocks = (numel + kBlock - 1) / kBlock;
    ok = fits(p, at::kBFloat16, numel, device) && fits(g, at::kBFloat16, numel, device) && p->sizes() == g->sizes();
    for (int k = 0; ok && k < 4; ++k) {
      const Attr attr(state, names[k]);   // (the state keeps the tensor)
      const at::Tensor* t = tensor(attr.o);
      ok = fits(t, k < 2 ? at::kByte : at::kFloat, k < 2 ? numel : blocks, device) && t->dim() == 1;
      if (ok) w[2 + k] = reinterpret_cast<uint64_t>(t->data_ptr());
    }
    w[6] = 0;
    if (ok && master != Py_None) {
      const at::Tensor* m = tensor(master);
      ok = fits(m, at::kFloat, numel, device) && m->sizes() == p->sizes();
      if (ok) w[6] = reinterpret_cast<uint64_t>(m->data_ptr());
    }
    if (!ok) break;
    w[0] = reinterpret_cast<uint64_t>(p->data_ptr());
    w[1] = reinterpret_cast<uint64_t>(g->data_ptr());
    w[7] = static_cast<uint64_t>(numel);
    if (numel == 0) continue;
    const uint64_t bytes[7] = {2 * w[7], 0, w[7], w[7], 4 * (uint64_t)blocks, 4 * (uint64_t)blocks, 4 * w[7]};
    for (int k : {0, 2, 3, 4, 5, 6})
      if (w[k]) written.emplace_back(w[k], w[k] + bytes[k]);
  }
  std::sort(written.begin(), written.end());
  const auto shared = [](const auto& x, const auto& y) { return y.first < x.second; };
  if (!ok || std::adjacent_find(written.begin(), written.end(), shared) != written.end()) Py_RETURN_NONE;
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(table.data()), n * 8 * (Py_ssize_t)sizeof(uint64_t));
}

// has_memory(tensor) -> whether it is a tensor with an address to ask for.
PyObject* has_memory(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return PyBool_FromLong(na == 1 && plain(tensor(a[0])));
}

// layer(w, adapters, X, ids) -> (qlora_nf4_weight and qlora_adapter_set as bytes, M, N, K, r, count, the device's
// current stream, whether the device is the current one), or None.  w, adapters: NF4Weight and AdapterSet.
PyObject* layer(PyObject*, PyObject* const* a, Py_ssize_t na) {
  if (na != 4) {
    PyErr_SetString(PyExc_TypeError, "layer(w, adapters, X, ids)");
    return nullptr;
  }
  enum { CODES, QSCALE, DSCALE, ROWS, COLS, CODEBOOK, DQ_FORMAT, A, B, SCALE, COUNT };
  static PyObject* const name[COUNT] = {
      PyUnicode_InternFromString("codes"),     PyUnicode_InternFromString("qscale"),
      PyUnicode_InternFromString("dscale"),    PyUnicode_InternFromString("rows"),
      PyUnicode_InternFromString("cols"),      PyUnicode_InternFromString("codebook"),
      PyUnicode_InternFromString("dq_format"), PyUnicode_InternFromString("A"),
      PyUnicode_InternFromString("B"),         PyUnicode_InternFromString("scale")};
  const Attr codes_(a[0], name[CODES]), qscale_(a[0], name[QSCALE]), dscale_(a[0], name[DSCALE]), A_(a[1], name[A]),
      B_(a[1], name[B]), scale_(a[1], name[SCALE]);
  const int64_t N = Attr(a[0], name[ROWS]).integer(), K = Attr(a[0], name[COLS]).integer();
  const int book = Attr(a[0], name[CODEBOOK]).word("nf4", "int4"), fmt = Attr(a[0], name[DQ_FORMAT]).word("e4m3", "uint8");
  const at::Tensor *X = tensor(a[2]), *ids = tensor(a[3]), *any_A = tensor(A_.o);
  if (!X || !X->defined() || !X->is_cuda() || X->dim() != 2 || !any_A || !any_A->defined() || any_A->dim() != 3 ||
      N <= 0 || K <= 0 || N > ((int64_t)1 << 31) || K > ((int64_t)1 << 31) || K % 64 || book < 0 || fmt < 0 || !qscale_.o)
    Py_RETURN_NONE;
  const bool dq = qscale_.o != Py_None;
  const int64_t dev = X->get_device(), M = X->size(0), nb = N * K / 64, n = any_A->size(0), r = any_A->size(1);
  const at::Tensor* codes = codes_.of(at::kByte, {N * K / 2}, dev);
  const at::Tensor* qs = dq ? qscale_.of(at::kByte, {nb}, dev) : nullptr;
  const at::Tensor* ds = dscale_.of(at::kFloat, {dq ? (nb + 255) / 256 : nb}, dev);
  const at::Tensor* At = A_.of(at::kBFloat16, {n, r, K}, dev);
  const at::Tensor* Bt = B_.of(at::kBFloat16, {n, N, r}, dev);
  const at::Tensor* sc = scale_.of(at::kFloat, {n}, dev);
  if (!codes || (dq && !qs) || !ds || !At || !Bt || !sc || n > INT32_MAX || r > INT32_MAX || X->size(1) != K ||
      !fits(X, at::kBFloat16, M * K, dev) || !fits(ids, at::kInt, M, dev) || ids->dim() != 1)
    Py_RETURN_NONE;
  const qlora_nf4_weight wd = {static_cast<const uint8_t*>(codes->data_ptr()),
                               qs ? static_cast<const uint8_t*>(qs->data_ptr()) : nullptr,
                               static_cast<const float*>(ds->data_ptr()),
                               N,
                               K,
                               64,
                               dq ? 256 : 0,
                               book ? QL_CODEBOOK_INT4 : QL_CODEBOOK_NF4,
                               fmt ? QL_DQ_UINT8 : QL_DQ_E4M3};
  const qlora_adapter_set as = {static_cast<const uint16_t*>(At->data_ptr()), static_cast<const uint16_t*>(Bt->data_ptr()),
                                static_cast<const float*>(sc->data_ptr()), (int32_t)n, (int32_t)r};
  const auto stream = c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev);
  return Py_BuildValue("y#y#LLLLLKO", reinterpret_cast<const char*>(&wd), (Py_ssize_t)sizeof(wd),
                       reinterpret_cast<const char*>(&as), (Py_ssize_t)sizeof(as), (long long)M, (long long)N,
                       (long long)K, (long long)r, (long long)n,
                       (unsigned long long)reinterpret_cast<uintptr_t>(stream.stream()),
                       c10::hip::current_device() == dev ? Py_True : Py_False);
}

// A tensor whose sizes are symbols throws where it is asked for them, a stream
// where there is no device: no exception leaves, the caller gets None.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  try {
    return F(self, a, na);
  } catch (const std::exception&) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

PyMethodDef methods[] = {{"layer", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<layer>)), METH_FASTCALL,
                          "describe a layer of many adapters"},
                         {"adamw8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<adamw8>)), METH_FASTCALL,
                          "pack the tensors of an 8-bit AdamW step"},
                         {"has_memory", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<has_memory>)),
                          METH_FASTCALL, "whether a tensor has an address"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
