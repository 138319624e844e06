// Python calls of the operators that take a few microseconds on the GPU: the
// checks of their tensors in C++ instead of one Python attribute after another
// (gqa_kv_keep: 9.3 us of host time became 4.3). Nothing is refused here: a
// function returns None when anything is not as the library needs it, and the
// Python binding then goes through its own checks, which say what it is; else it
// returns the library's status.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <memory>
#include <new>
#include <vector>

#include "gqa_kv.h"
#include "gqa_prompt.h"

namespace {

// The library's functions, from the binding that loaded it.
decltype(&gqa_prompt_attn) prompt_fn;
decltype(&gqa_tree_attn) tree_fn;
decltype(&gqa_kv_fork) fork_fn;
decltype(&gqa_kv_keep) keep_fn;
decltype(&gqa_kv_release) release_fn;

const at::Tensor* tensor(PyObject* x) {
  return THPVariable_Check(x) ? &THPVariable_Unpack(x) : nullptr;
}

// The checks of one call: `ok` falls when one fails.
struct Call {
  int64_t dev = -1;
  bool ok = true;

  // The first tensor's device, which has to be the current one.
  void on(const at::Tensor* t) {
    ok = t && t->is_cuda();
    if (!ok) return;
    dev = t->get_device();
    ok = dev == c10::cuda::current_device();
  }
  bool here(const at::Tensor* t) {
    ok = ok && t && t->is_cuda() && t->get_device() == dev;
    return ok;
  }
  int32_t* ints(PyObject* x, std::initializer_list<int64_t> sizes) {
    const at::Tensor* t = tensor(x);
    if (!here(t)) return nullptr;
    ok = t->scalar_type() == at::kInt && t->sizes() == at::IntArrayRef(sizes) && t->is_contiguous();
    return ok ? static_cast<int32_t*>(t->data_ptr()) : nullptr;
  }
  int32_t* ints_or_none(PyObject* x, std::initializer_list<int64_t> sizes) {
    return x == Py_None ? nullptr : ints(x, sizes);
  }
  // Sizes that a call takes from its tensors fit the library's ints.
  int size(int64_t n) {
    ok = ok && n <= 0x7fffffff;
    return static_cast<int>(n);
  }
  // The stream's handle: an int, or None for the current one.
  void* stream(PyObject* x) {
    if (!ok) return nullptr;
    if (x == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    void* s = PyLong_AsVoidPtr(x);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return s;
  }
  // A whole number that fits an int.
  int number(PyObject* x) {
    const long n = PyLong_AsLong(x);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return size(n);
  }
};

PyObject* status(int rc) { return PyLong_FromLong(rc); }

struct Released {   // the interpreter's lock, while the library works
  PyThreadState* state = PyEval_SaveThread();
  ~Released() { PyEval_RestoreThread(state); }
};

// q, k_pool, v_pool, token_start, cached_lens, tree_mask or None, block_table,
// seq_lens, out, scale or None, stream
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 11) Py_RETURN_NONE;
  const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *table = tensor(a[6]),
                   *out = tensor(a[8]);
  const bool tree = a[5] != Py_None;
  Call c;
  c.on(k);
  if (!c.ok || !c.here(q) || !c.here(v) || !c.here(table) || !c.here(out) || k->dim() != 4 ||
      q->dim() != 3 || table->dim() != 2 || (tree && a[4] == Py_None))
    Py_RETURN_NONE;
  const auto type = k->scalar_type();
  const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2), B = table->size(0);
  if ((type != at::kBFloat16 && type != at::kHalf) || v->scalar_type() != type ||
      q->scalar_type() != type || out->scalar_type() != type || k->size(3) != D ||
      v->sizes() != k->sizes() || out->sizes() != q->sizes() || !k->is_contiguous() ||
      !v->is_contiguous() || !out->is_contiguous() ||
      (T && (q->stride(2) != 1 || (Hq > 1 && q->stride(1) != D))))
    Py_RETURN_NONE;
  const int32_t* start = c.ints(a[3], {B + 1});
  const int32_t* cached = c.ints_or_none(a[4], {B});
  const int32_t* lens = c.ints_or_none(a[7], {B});
  const int32_t* blocks = c.ints(a[6], {B, table->size(1)});
  const int32_t* mask = nullptr;
  int64_t words = 0;
  if (tree) {
    const at::Tensor* m = tensor(a[5]);
    if (!m || m->dim() != 2) Py_RETURN_NONE;
    words = m->size(1);
    mask = c.ints(a[5], {T, words});
  }
  double scale = 0.0;
  if (a[9] == Py_None) {
    scale = 1.0 / std::sqrt(static_cast<double>(D));
  } else {
    scale = PyFloat_AsDouble(a[9]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
  }
  void* stream = c.stream(a[10]);
  const int code = type == at::kBFloat16 ? GQA_AV_BF16 : GQA_AV_FP16;
  const int iB = c.size(B), iT = c.size(T), iHq = c.size(Hq), iHkv = c.size(k->size(2)), iD = c.size(D),
            bs = c.size(k->size(1)), nb = c.size(k->size(0)), mb = c.size(table->size(1)), iw = c.size(words);
  if (!c.ok) Py_RETURN_NONE;
  const void *qp = q->data_ptr(), *kp = k->data_ptr(), *vp = v->data_ptr();
  void* op = out->data_ptr();
  const int64_t stride = q->stride(0);
  int rc;
  {
    Released lock;
    rc = tree ? tree_fn(qp, stride, kp, vp, start, cached, mask, iw, blocks, lens, op, iB, iT, iHq, iHkv,
                        iD, code, bs, nb, mb, static_cast<float>(scale), stream)
              : prompt_fn(qp, stride, kp, vp, start, cached, blocks, lens, op, iB, iT, iHq, iHkv, iD,
                          code, bs, nb, mb, static_cast<float>(scale), stream);
  }
  return status(rc);
} catch (...) {
  Py_RETURN_NONE;
}

// The pools of a KvPools, as a capsule.
struct Pools {
  std::vector<void*> at;
  int64_t dev, row_bytes;
  int num_blocks, block_size;
};
const char* const kPoolsName = "gqa_pools";
void free_pools(PyObject* x) { delete static_cast<Pools*>(PyCapsule_GetPointer(x, kPoolsName)); }

// addresses (a tuple of ints), device, bytes of a row, num_blocks, block_size
PyObject* make_pools(PyObject*, PyObject* args) try {
  PyObject* list;
  long long dev, row, nb, bs;
  if (!PyArg_ParseTuple(args, "O!LLLL", &PyTuple_Type, &list, &dev, &row, &nb, &bs)) return nullptr;
  if (nb > 0x7fffffff || bs > 0x7fffffff) Py_RETURN_NONE;
  std::unique_ptr<Pools> p(new Pools{{}, dev, row, static_cast<int>(nb), static_cast<int>(bs)});
  p->at.reserve(static_cast<size_t>(PyTuple_GET_SIZE(list)));
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(list); ++i)
    p->at.push_back(PyLong_AsVoidPtr(PyTuple_GET_ITEM(list, i)));
  if (PyErr_Occurred()) return nullptr;
  PyObject* capsule = PyCapsule_New(p.get(), kPoolsName, free_pools);
  if (capsule) p.release();   // the capsule's from here on
  return capsule;
} catch (const std::bad_alloc&) {
  return PyErr_NoMemory();
}
const Pools* pools_of(PyObject* x, Call* c) {
  if (!PyCapsule_IsValid(x, kPoolsName)) {
    c->ok = false;
    return nullptr;
  }
  const auto* p = static_cast<const Pools*>(PyCapsule_GetPointer(x, kPoolsName));
  c->dev = p->dev;
  c->ok = p->dev == c10::cuda::current_device();
  return p;
}

// pools, parent, child, block_table, seq_lens, shares, free_list, free_count,
// fork_block, free_left, stream
PyObject* fork(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 11) Py_RETURN_NONE;
  const at::Tensor *table = tensor(a[3]), *parent = tensor(a[1]), *list = tensor(a[6]);
  Call c;
  const Pools* p = pools_of(a[0], &c);
  if (!c.ok || !table || !parent || !list || table->dim() != 2 || parent->dim() != 1 || list->dim() != 1)
    Py_RETURN_NONE;
  const int64_t B = table->size(0), mb = table->size(1), N = parent->size(0), nf = list->size(0);
  const int32_t *pa = c.ints(a[1], {N}), *ch = c.ints(a[2], {N});
  int32_t *tab = c.ints(a[3], {B, mb}), *lens = c.ints(a[4], {B});
  int32_t* shares = c.ok ? c.ints(a[5], {p->num_blocks}) : nullptr;
  const int32_t *fl = c.ints(a[6], {nf}), *fc = c.ints(a[7], {1});
  int32_t *fb = c.ints(a[8], {N}), *left = c.ints(a[9], {1});
  void* stream = c.stream(a[10]);
  const int iN = c.size(N), iB = c.size(B), imb = c.size(mb), inf = c.size(nf);
  if (!c.ok) Py_RETURN_NONE;
  int rc;
  {
    Released lock;
    rc = fork_fn(p->at.data(), static_cast<int>(p->at.size()), p->row_bytes, pa, ch, tab, lens, shares,
                 fl, fc, fb, left, iN, iB, imb, inf, p->block_size, p->num_blocks, stream);
  }
  return status(rc);
} catch (...) {
  Py_RETURN_NONE;
}

// pools, cached_lens, accepted, accepted_count, block_table, seq_lens, kept_lens, stream
PyObject* keep(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 8) Py_RETURN_NONE;
  const at::Tensor *table = tensor(a[4]), *accepted = tensor(a[2]);
  Call c;
  const Pools* p = pools_of(a[0], &c);
  if (!c.ok || !table || !accepted || table->dim() != 2 || accepted->dim() != 2) Py_RETURN_NONE;
  const int64_t B = table->size(0), mb = table->size(1), W = accepted->size(1);
  const int32_t *cached = c.ints(a[1], {B}), *acc = c.ints(a[2], {B, W}), *count = c.ints(a[3], {B}),
                *tab = c.ints(a[4], {B, mb}), *lens = c.ints(a[5], {B});
  int32_t* kept = c.ints(a[6], {B});
  void* stream = c.stream(a[7]);
  const int iB = c.size(B), iW = c.size(W), imb = c.size(mb);
  if (!c.ok) Py_RETURN_NONE;
  int rc;
  {
    Released lock;
    rc = keep_fn(p->at.data(), static_cast<int>(p->at.size()), p->row_bytes, cached, acc, count, tab,
                 lens, kept, iB, iW, imb, p->block_size, p->num_blocks, stream);
  }
  return status(rc);
} catch (...) {
  Py_RETURN_NONE;
}

// block_table, old_lens, new_lens, shares or None, free_list, free_count, free_left,
// block_size, num_blocks or None, stream
PyObject* release(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n != 10) Py_RETURN_NONE;
  const at::Tensor *table = tensor(a[0]), *list = tensor(a[4]), *shares = tensor(a[3]);
  Call c;
  c.on(table);
  if (!c.ok || !list || table->dim() != 2 || list->dim() != 1 || (a[3] != Py_None && !shares) ||
      (shares && shares->dim() != 1) || (!shares && a[8] == Py_None))
    Py_RETURN_NONE;
  const int64_t B = table->size(0), mb = table->size(1), nf = list->size(0);
  const int64_t nb = a[8] == Py_None ? shares->size(0) : c.number(a[8]);
  const int32_t *tab = c.ints(a[0], {B, mb}), *old = c.ints(a[1], {B}), *now = c.ints(a[2], {B});
  int32_t *sh = c.ints_or_none(a[3], {nb}), *fl = c.ints(a[4], {nf});
  const int32_t* fc = c.ints(a[5], {1});
  int32_t* left = c.ints(a[6], {1});
  const int bs = c.number(a[7]);
  void* stream = c.stream(a[9]);
  const int iB = c.size(B), imb = c.size(mb), inf = c.size(nf), inb = c.size(nb);
  if (!c.ok) Py_RETURN_NONE;
  int rc;
  {
    Released lock;
    rc = release_fn(tab, old, now, sh, fl, fc, left, iB, imb, inf, bs, inb, stream);
  }
  return status(rc);
} catch (...) {
  Py_RETURN_NONE;
}

// The addresses of gqa_prompt_attn, gqa_tree_attn, gqa_kv_fork, gqa_kv_keep and
// gqa_kv_release in the library that the binding has loaded.
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long f[5];
  if (!PyArg_ParseTuple(args, "KKKKK", f, f + 1, f + 2, f + 3, f + 4)) return nullptr;
  prompt_fn = reinterpret_cast<decltype(prompt_fn)>(static_cast<uintptr_t>(f[0]));
  tree_fn = reinterpret_cast<decltype(tree_fn)>(static_cast<uintptr_t>(f[1]));
  fork_fn = reinterpret_cast<decltype(fork_fn)>(static_cast<uintptr_t>(f[2]));
  keep_fn = reinterpret_cast<decltype(keep_fn)>(static_cast<uintptr_t>(f[3]));
  release_fn = reinterpret_cast<decltype(release_fn)>(static_cast<uintptr_t>(f[4]));
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction as_method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"pools", make_pools, METH_VARARGS, nullptr},
    {"attend", as_method(attend), METH_FASTCALL, nullptr},
    {"fork", as_method(fork), METH_FASTCALL, nullptr},
    {"keep", as_method(keep), METH_FASTCALL, nullptr},
    {"release", as_method(release), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall(void) { return PyModule_Create(&module); }
