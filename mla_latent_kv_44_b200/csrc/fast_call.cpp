// _fast_call: argument checks and calls of the tree functions for the Python binding.
//
// A step's smaller calls run for 2 to 7 microseconds on the GPU. Checking a dozen tensors and
// converting as many arguments one by one in Python took longer than that; here a call costs its
// launch and a few hundred nanoseconds. The module holds no computation and no state but the
// library's function addresses, which the binding gives it (bind), so that both always use the
// same library.
//
// Every function takes (config address or None, tensors and numbers in the C call's order, stream
// or None) and returns the C call's status; kRefused when a tensor is not what the call needs (the
// binding then says which), kOtherDevice when the tensors' device is not the current one.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>

#include "mla.h"

namespace {

constexpr long kRefused = -1, kOtherDevice = -2;

decltype(&mla_build_tables) g_build_tables;
decltype(&mla_tree_masks) g_tree_masks;
decltype(&mla_append_slots) g_append_slots;
decltype(&mla_decode_tree) g_decode_tree;
decltype(&mla_commit_tree) g_commit_tree;

// The arguments of one call.
struct Args {
  PyObject* const* a;
  int dev = -1;
  bool ok = true;

  const at::Tensor* tensor(int i) {
    if (!THPVariable_Check(a[i])) {
      ok = false;
      return nullptr;
    }
    return &THPVariable_Unpack(a[i]);
  }
  // the tensor whose device and some of whose sizes the call takes over, as 32-bit numbers
  const at::Tensor* lead(int i, int dims, int64_t most = INT32_MAX) {
    const at::Tensor* t = tensor(i);
    if (!t || !t->is_cuda() || t->dim() != dims) {
      ok = false;
      return nullptr;
    }
    for (const int64_t n : t->sizes()) ok = ok && n <= most;
    if (dev < 0) dev = t->get_device();
    return t;
  }
  // data of a contiguous tensor of this type and shape on the device
  template <typename T>
  T* data(int i, at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor* t = tensor(i);
    if (!t || t->scalar_type() != type || !t->is_cuda() || t->get_device() != dev ||
        t->sizes() != shape || !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    return static_cast<T*>(t->data_ptr());
  }
  const mla_config* config(int i) { return static_cast<const mla_config*>(PyLong_AsVoidPtr(a[i])); }
  int number(int i) {
    const long v = PyLong_AsLong(a[i]);
    if (v != static_cast<int>(v)) ok = false;
    return static_cast<int>(v);
  }
  // the stream's handle; what is none (not a number, or no pointer holds it) leaves Python's error
  void* stream(int i) {
    if (a[i] == Py_None) return c10::cuda::getCurrentCUDAStream(dev).stream();
    void* const handle = PyLong_AsVoidPtr(a[i]);
    if (!handle && PyErr_Occurred()) ok = false;
    return handle;
  }
  // checks done: the call may go out
  bool elsewhere() const { return c10::cuda::current_device() != dev; }
};

PyObject* status(long s) { return PyErr_Occurred() ? nullptr : PyLong_FromLong(s); }

bool counted(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

constexpr auto kI32 = at::kInt, kI64 = at::kLong, kF32 = at::kFloat;
at::ScalarType dtype_of(const mla_config* c) { return c->dtype == MLA_BF16 ? at::kBFloat16 : kF32; }

// cfg, seq_lens, new_lens, block_table, blocks_held, free_blocks, free_count, blocks_held_out,
// free_count_out, cu_new, seq_idx, pos, slots, dev_err, stream
PyObject* build_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted(n, 15)) return nullptr;
  Args g{a};
  const mla_config* c = g.config(0);
  const at::Tensor *lens = g.lead(1, 1), *table = g.lead(3, 2), *free_ = g.lead(5, 1),
                   *slots = g.lead(12, 1);
  if (!g.ok) return status(kRefused);
  const int64_t b = lens->size(0), width = table->size(1), blocks = free_->size(0),
                tokens = slots->size(0);
  auto* p1 = g.data<int32_t>(1, kI32, {b});
  auto* p2 = g.data<int32_t>(2, kI32, {b});
  auto* p3 = g.data<int32_t>(3, kI32, {b, width});
  auto* p4 = g.data<int32_t>(4, kI32, {b});
  auto* p5 = g.data<int32_t>(5, kI32, {blocks});
  auto* p6 = g.data<int32_t>(6, kI32, {1});
  auto* p7 = g.data<int32_t>(7, kI32, {b});
  auto* p8 = g.data<int32_t>(8, kI32, {1});
  auto* p9 = g.data<int32_t>(9, kI32, {b + 1});
  auto* p10 = g.data<int32_t>(10, kI32, {tokens});
  auto* p11 = g.data<int32_t>(11, kI32, {tokens});
  auto* p12 = g.data<int64_t>(12, kI64, {tokens});
  auto* p13 = g.data<int32_t>(13, kI32, {1});
  if (!g.ok) return status(kRefused);
  if (g.elsewhere()) return status(kOtherDevice);
  void* const stream = g.stream(14);
  if (!g.ok) return status(kRefused);
  return status(g_build_tables(c, p1, p2, b, p3, width, p4, p5, p6, blocks, p7, p8, p9, p10, p11,
                               p12, tokens, (uint32_t*)p13, stream));
}

// parents, seq_lens, mask, pos, dev_err, stream
PyObject* tree_masks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted(n, 6)) return nullptr;
  Args g{a};
  const at::Tensor *parents = g.lead(0, 2), *lens = g.lead(1, 1);
  if (!g.ok) return status(kRefused);
  const int64_t rows = parents->size(0), T = parents->size(1), b = lens->size(0);
  auto* p0 = g.data<int32_t>(0, kI32, {rows, T});
  auto* p1 = g.data<int32_t>(1, kI32, {b});
  auto* p2 = g.data<int32_t>(2, kI32, {b * T, (T + 31) / 32});
  auto* p3 = g.data<int32_t>(3, kI32, {b * T});
  auto* p4 = g.data<int32_t>(4, kI32, {1});
  if (!g.ok) return status(kRefused);
  if (g.elsewhere()) return status(kOtherDevice);
  void* const stream = g.stream(5);
  if (!g.ok) return status(kRefused);
  return status(g_tree_masks(p0, rows, p1, b, T, (uint32_t*)p2, p3, (uint32_t*)p4, stream));
}

// cfg, ckv_raw, krope_raw, gamma, pos, slots, pool, dev_err, stream
PyObject* append_slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted(n, 9)) return nullptr;
  Args g{a};
  const mla_config* c = g.config(0);
  const at::Tensor *pool = g.lead(6, 3), *slots = g.lead(5, 1);
  if (!g.ok) return status(kRefused);
  const auto dt = dtype_of(c);
  const int64_t r = c->kv_rank, dr = c->rope_dim, blocks = pool->size(0), m = slots->size(0);
  auto* p1 = g.data<void>(1, dt, {m, r});
  auto* p2 = dr ? g.data<void>(2, dt, {m, dr}) : nullptr;
  auto* p3 = g.data<float>(3, kF32, {r});
  auto* p4 = g.data<int32_t>(4, kI32, {m});
  auto* p5 = g.data<int64_t>(5, kI64, {m});
  auto* p6 = g.data<void>(6, dt, {blocks, c->block_size, r + dr});
  auto* p7 = g.data<int32_t>(7, kI32, {1});
  if (!g.ok) return status(kRefused);
  if (g.elsewhere()) return status(kOtherDevice);
  void* const stream = g.stream(8);
  if (!g.ok) return status(kRefused);
  return status(g_append_slots(c, p1, p2, p3, p4, p5, p6, blocks, m, (uint32_t*)p7, stream));
}

// cfg, q, pool, block_table, seq_lens, q_per_seq, tree_mask, w_uv, workspace, o, lse, dev_err,
// stream
PyObject* decode_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted(n, 13)) return nullptr;
  Args g{a};
  const mla_config* c = g.config(0);
  const at::Tensor *pool = g.lead(2, 3), *table = g.lead(3, 2), *lens = g.lead(4, 1),
                   *ws = g.lead(8, 1, INT64_MAX);
  const int64_t T = g.number(5);
  if (!g.ok || T < 0) return status(kRefused);
  const auto dt = dtype_of(c);
  const int64_t b = lens->size(0), width = table->size(1), blocks = pool->size(0), H = c->num_heads,
                r = c->kv_rank, D = r + c->rope_dim, dv = c->head_dim_v, m = b * T;
  auto* p1 = g.data<void>(1, dt, {m, H, D});
  auto* p2 = g.data<void>(2, dt, {blocks, c->block_size, D});
  auto* p3 = g.data<int32_t>(3, kI32, {b, width});
  auto* p4 = g.data<int32_t>(4, kI32, {b});
  auto* p6 = a[6] == Py_None ? nullptr : g.data<int32_t>(6, kI32, {m, (T + 31) / 32});
  auto* p7 = g.data<void>(7, dt, {H, dv, r});
  auto* p8 = g.data<void>(8, at::kByte, {ws->size(0)});
  auto* p9 = g.data<void>(9, dt, {m, H, dv});
  auto* p10 = a[10] == Py_None ? nullptr : g.data<float>(10, kF32, {m, H});
  auto* p11 = g.data<int32_t>(11, kI32, {1});
  if (!g.ok) return status(kRefused);
  if (g.elsewhere()) return status(kOtherDevice);
  void* const stream = g.stream(12);
  if (!g.ok) return status(kRefused);
  return status(g_decode_tree(c, p1, p2, p3, width, blocks, p4, b, T, (const uint32_t*)p6, p7, p8,
                              ws->size(0), p9, p10, (uint32_t*)p11, stream));
}

// cfg, path, path_len, q_per_seq, block_table, pool, seq_lens, seq_lens_out, dev_err, stream
PyObject* commit_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted(n, 10)) return nullptr;
  Args g{a};
  const mla_config* c = g.config(0);
  const at::Tensor *pool = g.lead(5, 3), *path = g.lead(1, 2), *table = g.lead(4, 2),
                   *lens = g.lead(6, 1);
  const int T = g.number(3);
  if (!g.ok) return status(kRefused);
  const int64_t b = lens->size(0), steps = path->size(1), width = table->size(1),
                blocks = pool->size(0);
  auto* p1 = g.data<int32_t>(1, kI32, {b, steps});
  auto* p2 = g.data<int32_t>(2, kI32, {b});
  auto* p4 = g.data<int32_t>(4, kI32, {b, width});
  auto* p5 = g.data<void>(5, dtype_of(c), {blocks, c->block_size, c->kv_rank + c->rope_dim});
  auto* p6 = g.data<int32_t>(6, kI32, {b});
  auto* p7 = g.data<int32_t>(7, kI32, {b});
  auto* p8 = g.data<int32_t>(8, kI32, {1});
  if (!g.ok) return status(kRefused);
  if (g.elsewhere()) return status(kOtherDevice);
  void* const stream = g.stream(9);
  if (!g.ok) return status(kRefused);
  return status(g_commit_tree(c, p1, p2, steps, T, p4, width, p5, blocks, p6, p7, b, (uint32_t*)p8,
                              stream));
}

// name, address of the library's function
PyObject* bind(PyObject*, PyObject* args) {
  const char* name;
  unsigned long long at;
  if (!PyArg_ParseTuple(args, "sK", &name, &at)) return nullptr;
  void* p = reinterpret_cast<void*>(at);
  if (!std::strcmp(name, "mla_build_tables")) g_build_tables = (decltype(g_build_tables))p;
  else if (!std::strcmp(name, "mla_tree_masks")) g_tree_masks = (decltype(g_tree_masks))p;
  else if (!std::strcmp(name, "mla_append_slots")) g_append_slots = (decltype(g_append_slots))p;
  else if (!std::strcmp(name, "mla_decode_tree")) g_decode_tree = (decltype(g_decode_tree))p;
  else if (!std::strcmp(name, "mla_commit_tree")) g_commit_tree = (decltype(g_commit_tree))p;
  else return PyErr_Format(PyExc_KeyError, "%s", name);
  Py_RETURN_NONE;
}

// C++ exceptions of torch end here as Python errors.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef kMethods[] = {
    {"build_tables", (PyCFunction)(void*)guarded<build_tables>, METH_FASTCALL, nullptr},
    {"tree_masks", (PyCFunction)(void*)guarded<tree_masks>, METH_FASTCALL, nullptr},
    {"append_slots", (PyCFunction)(void*)guarded<append_slots>, METH_FASTCALL, nullptr},
    {"decode_tree", (PyCFunction)(void*)guarded<decode_tree>, METH_FASTCALL, nullptr},
    {"commit_tree", (PyCFunction)(void*)guarded<commit_tree>, METH_FASTCALL, nullptr},
    {"bind", bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fast_call", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast_call(void) { return PyModule_Create(&kModule); }
