// cache_torch.cpp - torch tensors to the C ABI of cmd_cache.h: a CPython module
// that describes tensors to the library, allocates outputs and workspaces on
// the current stream and raises CmdError. In native code because describing
// the eight or nine tensors of a call from Python took 30 us on the GB300's
// host, several times what a decode step's kernels take; this takes 2 to 3.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <string>

#include "../../include/cmd_cache.h"

namespace {

PyObject* g_error = nullptr;  // CmdError(status, function, message)

// A Python exception that is set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& msg) {
  PyErr_SetString(type, msg.c_str());
  throw Raised{};
}

// Runs f, turning what it throws into a Python exception.
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

void check(cmd_status s, const char* function) {
  if (s == CMD_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "iss", (int)s, function, cmd_last_error());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " is no tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) raise(PyExc_ValueError, std::string(name) + " is not on a GPU");
  return t;
}

cmd_operand describe(const at::Tensor& t, const char* name) {
  cmd_operand x = {};
  switch (t.scalar_type()) {
    case at::kFloat: x.dtype = CMD_F32; break;
    case at::kHalf: x.dtype = CMD_F16; break;
    case at::kBFloat16: x.dtype = CMD_BF16; break;
    case at::kInt: x.dtype = CMD_I32; break;
    default: raise(PyExc_TypeError, std::string(name) + " is not float32, float16, bfloat16 or int32");
  }
  if (t.is_neg()) raise(PyExc_ValueError, std::string(name) + " is a view of negated numbers (resolve_neg() makes them so)");
  const int64_t rank = t.dim();
  if (rank > CMD_MAX_RANK) raise(PyExc_ValueError, std::string(name) + " has more than 4 dims");
  x.rank = (int32_t)rank;
  x.ptr = const_cast<void*>(t.const_data_ptr());
  for (int64_t d = 0; d < rank; ++d) {
    x.sizes[d] = t.size(d);
    x.strides[d] = t.stride(d);
  }
  return x;
}
cmd_operand operand(PyObject* o, const char* name) { return describe(tensor(o, name), name); }
cmd_operand optional(PyObject* o, const char* name) { return o == Py_None ? cmd_operand{} : operand(o, name); }

int32_t* status_word(PyObject* o) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "status");
  if (t.scalar_type() != at::kInt || t.numel() != 1) raise(PyExc_ValueError, "status is one int32 on a GPU");
  return static_cast<int32_t*>(t.data_ptr());
}

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised{};
  return x;
}
int32_t integer(PyObject* o, const char* name) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised{};
  if (x < INT32_MIN || x > INT32_MAX) raise(PyExc_ValueError, std::string(name) + " is out of range");
  return (int32_t)x;
}

// The device of a call's tensors, made current, and its current stream.
struct Where {
  c10::cuda::CUDAGuard guard;
  void* stream;
  explicit Where(const at::Tensor& t)
      : guard(t.device()), stream(c10::cuda::getCurrentCUDAStream(t.device().index()).stream()) {}
  at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type) const {
    return at::detail::empty_cuda(sizes, type, guard.current_device(), std::nullopt);
  }
  // memory for the current stream, given back (for work after the call's on that stream) when the result goes
  c10::DataPtr scratch(int64_t bytes) const { return c10::cuda::CUDACachingAllocator::get()->allocate((size_t)bytes); }
};

void same_device(const Where& w, PyObject* o, const char* name) {
  if (o != Py_None && tensor(o, name).device() != w.guard.current_device())
    raise(PyExc_ValueError, std::string(name) + " is on another GPU");
}

// A tensor that a call is to write, where one is given: autograd keeps no record
// of it, so none may be asked for.
void writable(PyObject* o, const char* name) {
  if (o != Py_None && at::GradMode::is_enabled() && tensor(o, name).requires_grad())
    raise(PyExc_ValueError, std::string(name) + " is written and requires a gradient: none would be recorded");
}
// Tells autograd that a tensor was written: gradients that need what it held are
// refused.
void written(PyObject* o) {
  if (o == Py_None) return;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

PyObject* wrap(const at::Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  if (!o) throw Raised{};
  return o;
}
// A new reference to a given output, or to an allocated one.
PyObject* result(PyObject* given, const at::Tensor& made) {
  if (given == Py_None) return wrap(made);
  Py_INCREF(given);
  return given;
}
PyObject* none() { Py_RETURN_NONE; }
PyObject* pack(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) PyTuple_SET_ITEM(t, i++, o);
  return t;
}

void expect(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) raise(PyExc_TypeError, "wrong number of arguments");
}

cmd_rope_spec rope_spec(PyObject* turns, PyObject* layout, PyObject* scale, int backward) {
  cmd_rope_spec r = {};
  r.layout = integer(layout, "layout");
  r.scale = (float)number(scale);
  r.backward = backward;
  if (turns != Py_None) {
    const at::Tensor& t = tensor(turns, "turns");
    if (t.scalar_type() != at::kLong || t.dim() != 1 || !t.is_contiguous())
      raise(PyExc_ValueError, "turns is a contiguous int64 vector on a GPU (see rope_turns)");
    if (t.size(0) > INT32_MAX) raise(PyExc_ValueError, "turns is too long");
    r.turns = static_cast<const uint64_t*>(t.const_data_ptr());
    r.n_pairs = (int32_t)t.size(0);
  }
  return r;
}

// rope(q, k, positions, turns, layout, scale, q_out, k_out, backward) -> (q_out, k_out)
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 9);
    if (a[0] == Py_None && a[1] == Py_None) raise(PyExc_ValueError, "q and k are both absent");
    const Where w(tensor(a[0] != Py_None ? a[0] : a[1], "q or k"));
    const char* names[2] = {"q", "k"};
    cmd_operand in[2], out[2];
    at::Tensor made[2];
    for (int i = 0; i < 2; ++i) {
      if (a[i] == Py_None) continue;
      const at::Tensor& t = tensor(a[i], names[i]);
      same_device(w, a[i], names[i]);
      in[i] = describe(t, names[i]);
      if (a[6 + i] == Py_None) out[i] = describe(made[i] = w.empty(t.sizes(), t.scalar_type()), names[i]);
      else out[i] = operand(a[6 + i], "out"), same_device(w, a[6 + i], "out");
    }
    const cmd_operand positions = operand(a[2], "positions");
    same_device(w, a[2], "positions");
    const cmd_rope_spec r = rope_spec(a[3], a[4], a[5], PyObject_IsTrue(a[8]));
    same_device(w, a[3], "turns");
    const bool q = a[0] != Py_None, k = a[1] != Py_None;
    if (q) writable(a[6], "out");
    if (k) writable(a[7], "out");
    check(cmd_rope(q ? &in[0] : nullptr, q ? &out[0] : nullptr, k ? &in[1] : nullptr, k ? &out[1] : nullptr, &positions, &r,
                   w.stream),
          "cmd_rope");
    if (q) written(a[6]);
    if (k) written(a[7]);
    return pack({q ? result(a[6], made[0]) : none(), k ? result(a[7], made[1]) : none()});
  });
}

// cache_append(k, v, k_cache, v_cache, tables, positions, rows, q, q_out, turns, layout, scale, status) -> q_out
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 13);
    const Where w(tensor(a[0], "k"));
    cmd_append_args x = {};
    x.k = operand(a[0], "k");
    x.v = operand(a[1], "v");
    x.k_cache = operand(a[2], "k_cache");
    x.v_cache = operand(a[3], "v_cache");
    x.tables = operand(a[4], "tables");
    x.positions = operand(a[5], "positions");
    x.rows = optional(a[6], "rows");
    x.q = optional(a[7], "q");
    at::Tensor made;
    if (a[7] != Py_None) {
      const at::Tensor& q = THPVariable_Unpack(a[7]);
      x.q_out = a[8] == Py_None ? describe(made = w.empty(q.sizes(), q.scalar_type()), "q_out") : operand(a[8], "q_out");
    }
    x.rope = rope_spec(a[9], a[10], a[11], 0);
    x.status = status_word(a[12]);
    same_device(w, a[12], "status");
    const char* names[] = {"k", "v", "k_cache", "v_cache", "tables", "positions", "rows", "q", "q_out", "turns"};
    for (int i = 0; i < 10; ++i) same_device(w, a[i], names[i]);
    const int outs[] = {2, 3, 8};
    for (int i : outs)
      if (i != 8 || a[7] != Py_None) writable(a[i], names[i]);
    check(cmd_cache_append(&x, w.stream), "cmd_cache_append");
    for (int i : outs)
      if (i != 8 || a[7] != Py_None) written(a[i]);
    return a[7] == Py_None ? none() : result(a[8], made);
  });
}

// attention_decode(q, k_cache, v_cache, tables, lengths, scale, softcap, window, out, lse, return_lse, workspace,
// status) -> out or (out, lse)
PyObject* py_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 13);
    const at::Tensor& q = tensor(a[0], "q");
    const Where w(q);
    cmd_attention_args x = {};
    x.q = operand(a[0], "q");
    x.k_cache = operand(a[1], "k_cache");
    x.v_cache = operand(a[2], "v_cache");
    x.tables = operand(a[3], "tables");
    x.lengths = operand(a[4], "lengths");
    if (x.q.rank != 3 || x.k_cache.rank != 4) raise(PyExc_ValueError, "q has rank 3 and the caches have rank 4");
    const int64_t dim = x.q.sizes[2];
    x.scale = (float)(a[5] != Py_None ? number(a[5]) : dim > 0 ? 1.0 / std::sqrt((double)dim) : 1.0);
    x.softcap = (float)number(a[6]);
    x.window = integer(a[7], "window");
    at::Tensor out, lse;
    c10::DataPtr workspace;
    x.out = a[8] == Py_None ? describe(out = w.empty(q.sizes(), q.scalar_type()), "out") : operand(a[8], "out");
    const bool with_lse = PyObject_IsTrue(a[10]);
    if (a[9] != Py_None) x.lse = operand(a[9], "lse");
    else if (with_lse) x.lse = describe(lse = w.empty({q.size(0), q.size(1)}, at::kFloat), "lse");
    const int64_t heads = x.q.sizes[1], kv = x.k_cache.sizes[2];
    if (a[11] != Py_None) {
      const at::Tensor& t = tensor(a[11], "workspace");
      if (!t.is_contiguous()) raise(PyExc_ValueError, "workspace is not contiguous");
      x.workspace = t.data_ptr();
      x.workspace_bytes = (int64_t)t.nbytes();
    } else if (heads > 0 && kv > 0 && heads % kv == 0 && heads <= INT32_MAX && dim <= CMD_CACHE_MAX_DIM) {
      check(cmd_attention_workspace((int32_t)heads, (int32_t)kv, (int32_t)dim, &x.workspace_bytes), "cmd_attention_workspace");
      workspace = w.scratch(x.workspace_bytes);
      x.workspace = workspace.get();
    }
    x.status = status_word(a[12]);
    same_device(w, a[12], "status");
    const char* names[] = {"q", "k_cache", "v_cache", "tables", "lengths"};
    for (int i = 0; i < 5; ++i) same_device(w, a[i], names[i]);
    same_device(w, a[8], "out");
    same_device(w, a[9], "lse");
    same_device(w, a[11], "workspace");
    writable(a[8], "out");
    writable(a[9], "lse");
    check(cmd_attention_decode(&x, w.stream), "cmd_attention_decode");
    written(a[8]);
    written(a[9]);
    PyObject* o = result(a[8], out);
    return with_lse ? pack({o, result(a[9], lse)}) : o;
  });
}

// The pools of a list or tuple of tensors, each [pages, ...] with the elements
// of a page dense, in any order.
int pools(PyObject* list, int64_t pages, const Where& w, cmd_pool* out) {
  const bool tuple = PyTuple_Check(list);
  if (!tuple && !PyList_Check(list)) raise(PyExc_TypeError, "pools is a list or tuple of tensors");
  const Py_ssize_t n = tuple ? PyTuple_GET_SIZE(list) : PyList_GET_SIZE(list);
  if (n > CMD_CACHE_MAX_POOLS) raise(PyExc_ValueError, "more than 64 pools");
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = tuple ? PyTuple_GET_ITEM(list, i) : PyList_GET_ITEM(list, i);
    const at::Tensor& t = tensor(o, "a pool");
    same_device(w, o, "a pool");
    writable(o, "a pool");
    const int64_t rank = t.dim();
    if (rank < 1 || t.size(0) != pages)
      raise(PyExc_ValueError,
            "pool " + std::to_string(i) + " does not have " + std::to_string(pages) + " pages in its first dim");
    int64_t block = 1, dims = 0;
    for (int64_t d = 1; d < rank; ++d) {
      block *= t.size(d);
      dims += t.size(d) != 1;
    }
    int64_t reach = 1;  // the dims of a page, smallest stride first, must follow one another
    for (int64_t k = 0; k < dims && block > 0; ++k) {
      int64_t d = 1;
      while (d < rank && (t.size(d) == 1 || t.stride(d) != reach)) ++d;
      if (d == rank) raise(PyExc_ValueError, "a page of pool " + std::to_string(i) + " is not dense");
      reach *= t.size(d);
    }
    const int64_t es = (int64_t)t.element_size();
    out[i].ptr = t.data_ptr();
    out[i].page_bytes = block * es;
    out[i].page_stride = (pages > 1 ? t.stride(0) : block) * es;
  }
  return (int)n;
}

void pools_written(PyObject* list) {
  const bool tuple = PyTuple_Check(list);
  const Py_ssize_t n = tuple ? PyTuple_GET_SIZE(list) : PyList_GET_SIZE(list);
  for (Py_ssize_t i = 0; i < n; ++i) written(tuple ? PyTuple_GET_ITEM(list, i) : PyList_GET_ITEM(list, i));
}

// Item i of a given tuple of outputs (None where none was given).
PyObject* item(PyObject* out, int i, int n) {
  if (out == Py_None) return Py_None;
  if (!PyTuple_Check(out) || PyTuple_GET_SIZE(out) != n)
    raise(PyExc_TypeError, "out is a tuple of " + std::to_string(n) + " tensors");
  return PyTuple_GET_ITEM(out, i);
}
cmd_operand output(PyObject* given, const Where& w, at::IntArrayRef sizes, at::Tensor* made, const char* name) {
  if (given == Py_None) return describe(*made = w.empty(sizes, at::kInt), name);
  const cmd_operand x = operand(given, name);
  same_device(w, given, name);
  return x;
}

// cache_select(tables, lengths, refs, parents, pools, page_size, grow, out, status) -> (tables, lengths, refs)
PyObject* py_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 9);
    const Where w(tensor(a[0], "tables"));
    cmd_select_args x = {};
    x.tables = operand(a[0], "tables");
    x.lengths = operand(a[1], "lengths");
    x.refs = operand(a[2], "refs");
    x.parents = operand(a[3], "parents");
    x.grow = optional(a[6], "grow");
    if (x.tables.rank != 2 || x.refs.rank != 1 || x.parents.rank != 1)
      raise(PyExc_ValueError, "tables has rank 2, refs and parents have rank 1");
    const int64_t rows = x.parents.sizes[0], pages = x.refs.sizes[0];
    at::Tensor made[3];
    c10::DataPtr workspace;
    PyObject* out[3] = {item(a[7], 0, 3), item(a[7], 1, 3), item(a[7], 2, 3)};
    x.tables_out = output(out[0], w, {rows, x.tables.sizes[1]}, &made[0], "tables_out");
    x.lengths_out = output(out[1], w, {rows}, &made[1], "lengths_out");
    x.refs_out = output(out[2], w, {pages}, &made[2], "refs_out");
    cmd_pool list[CMD_CACHE_MAX_POOLS];
    x.pools = list;
    x.n_pools = pools(a[4], pages, w, list);
    x.page_size = integer(a[5], "page_size");
    check(cmd_select_workspace(x.tables.sizes[0], rows, pages, &x.workspace_bytes), "cmd_select_workspace");
    workspace = w.scratch(x.workspace_bytes);
    x.workspace = workspace.get();
    x.status = status_word(a[8]);
    same_device(w, a[8], "status");
    const char* names[] = {"tables", "lengths", "refs", "parents"};
    for (int i = 0; i < 4; ++i) same_device(w, a[i], names[i]);
    same_device(w, a[6], "grow");
    check(cmd_cache_select(&x, w.stream), "cmd_cache_select");
    for (PyObject* o : out) written(o);
    pools_written(a[4]);
    return pack({result(out[0], made[0]), result(out[1], made[1]), result(out[2], made[2])});
  });
}

// cache_compact(tables, lengths, refs, pools, page_size, out, status) -> (tables, refs, page_map)
PyObject* py_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 7);
    const Where w(tensor(a[0], "tables"));
    cmd_compact_args x = {};
    x.tables = operand(a[0], "tables");
    x.lengths = operand(a[1], "lengths");
    x.refs = operand(a[2], "refs");
    if (x.tables.rank != 2 || x.refs.rank != 1) raise(PyExc_ValueError, "tables has rank 2 and refs has rank 1");
    const int64_t pages = x.refs.sizes[0];
    at::Tensor made[3];
    c10::DataPtr workspace;
    PyObject* out[3] = {item(a[5], 0, 3), item(a[5], 1, 3), item(a[5], 2, 3)};
    x.tables_out = output(out[0], w, {x.tables.sizes[0], x.tables.sizes[1]}, &made[0], "tables_out");
    x.refs_out = output(out[1], w, {pages}, &made[1], "refs_out");
    x.page_map_out = output(out[2], w, {pages}, &made[2], "page_map_out");
    cmd_pool list[CMD_CACHE_MAX_POOLS];
    x.pools = list;
    x.n_pools = pools(a[3], pages, w, list);
    x.page_size = integer(a[4], "page_size");
    check(cmd_compact_workspace(pages, &x.workspace_bytes), "cmd_compact_workspace");
    workspace = w.scratch(x.workspace_bytes);
    x.workspace = workspace.get();
    x.status = status_word(a[6]);
    same_device(w, a[6], "status");
    const char* names[] = {"tables", "lengths", "refs"};
    for (int i = 0; i < 3; ++i) same_device(w, a[i], names[i]);
    check(cmd_cache_compact(&x, w.stream), "cmd_cache_compact");
    for (PyObject* o : out) written(o);
    pools_written(a[3]);
    return pack({result(out[0], made[0]), result(out[1], made[1]), result(out[2], made[2])});
  });
}

// cache_status(status)
PyObject* py_status(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 1);
    const Where w(tensor(a[0], "status"));
    int32_t* word = status_word(a[0]);
    cmd_status s;
    Py_BEGIN_ALLOW_THREADS;
    s = cmd_cache_status(word, nullptr, w.stream);
    Py_END_ALLOW_THREADS;
    check(s, "cmd_cache_status");
    return none();
  });
}

// set_error(CmdError)
PyObject* py_set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XSETREF(g_error, type);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<py_rope>("rope"),
                           method<py_append>("cache_append"),
                           method<py_attend>("attention_decode"),
                           method<py_select>("cache_select"),
                           method<py_compact>("cache_compact"),
                           method<py_status>("cache_status"),
                           {"set_error", py_set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_cache_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__cache_torch() { return PyModule_Create(&g_module); }
