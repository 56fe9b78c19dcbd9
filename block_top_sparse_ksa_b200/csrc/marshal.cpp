// marshal.cpp -- the Python binding's short way for the serving calls.
//
// A serving step makes these calls for a few microseconds of GPU work, and reading ten tensors'
// types, shapes, devices and addresses in Python takes longer than that (page assignment: 6 of
// 10.5 us a call).  Each function here makes the binding's checks on complete arguments (every
// output and the workspace given, tensors on the current device) and calls the library on the
// current stream.  It returns the library's status, or None if something does not match: the
// binding then goes its long way, which fills in what is left out and names what is wrong.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "ksa.h"

namespace {

// The arguments of one call; `ok` falls when one does not match.
struct Call {
  PyObject *const *args;
  int dev = -1;
  bool ok = true;

  const at::Tensor *tensor(int i, c10::ScalarType type) {
    if (!ok || !THPVariable_Check(args[i])) return fail();
    const at::Tensor &t = THPVariable_Unpack(args[i]);
    if (t.scalar_type() != type || !t.is_cuda()) return fail();
    if (dev < 0) dev = t.get_device();
    return t.get_device() == dev ? &t : fail();
  }
  const at::Tensor *fail() {
    ok = false;
    return nullptr;
  }
  // The address of a contiguous vector of n elements.
  void *vec(int i, c10::ScalarType type, int64_t n) {
    const at::Tensor *t = tensor(i, type);
    if (t == nullptr || t->numel() != n || !t->is_contiguous()) return fail(), nullptr;
    return t->data_ptr();
  }
  // ... of a contiguous tensor of these sizes.
  void *dense(int i, c10::ScalarType type, at::IntArrayRef sizes) {
    const at::Tensor *t = tensor(i, type);
    if (t == nullptr || t->sizes() != sizes || !t->is_contiguous()) return fail(), nullptr;
    return t->data_ptr();
  }
  // ... of [tokens, heads, dims] bf16 whose heads and dims are dense, and its token stride.
  uint16_t *rows(int i, int64_t n, int64_t h, int64_t d, int32_t *stride) {
    const at::Tensor *t = tensor(i, at::kBFloat16);
    if (t == nullptr || t->dim() != 3 || t->size(0) != n || t->size(1) != h || t->size(2) != d ||
        t->stride(2) != 1 || (h > 1 && t->stride(1) != d) || t->stride(0) >= (1LL << 31))
      return fail(), nullptr;
    *stride = static_cast<int32_t>(n > 1 ? t->stride(0) : h * d);
    return static_cast<uint16_t *>(t->data_ptr());
  }
  // ... of the workspace, and its bytes.
  void *workspace(int i, size_t *bytes) {
    if (!ok || !THPVariable_Check(args[i])) return fail(), nullptr;
    const at::Tensor &t = THPVariable_Unpack(args[i]);
    if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous()) return fail(), nullptr;
    *bytes = t.nbytes();
    return t.data_ptr();
  }
  // ... of the status word, or null for None.
  uint32_t *status(int i) {
    if (!ok || args[i] == Py_None) return nullptr;
    if (!THPVariable_Check(args[i])) return fail(), nullptr;
    const at::Tensor &t = THPVariable_Unpack(args[i]);
    if (!t.is_cuda() || t.get_device() != dev || t.nbytes() < 4) return fail(), nullptr;
    return static_cast<uint32_t *>(t.data_ptr());
  }
  int32_t integer(int i) {
    if (!ok || !PyLong_Check(args[i])) return fail(), 0;
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(args[i], &over);
    if (over != 0 || v < INT32_MIN || v > INT32_MAX) return fail(), 0;
    return static_cast<int32_t>(v);
  }
  // A size that the library takes as 32 bits.
  int32_t narrow(int64_t v) {
    if (v < 0 || v > INT32_MAX) fail();
    return static_cast<int32_t>(v);
  }
  template <typename T>
  T address(int i) {
    void *p = ok && PyLong_Check(args[i]) ? PyLong_AsVoidPtr(args[i]) : nullptr;
    if (p == nullptr) fail();
    return reinterpret_cast<T>(p);
  }
  // The stream of the call; no call on another device than the current one.
  void *stream() {
    if (!ok || c10::cuda::current_device() != dev) return fail(), nullptr;
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  }
};

// Runs `body`, which returns a status or leaves call.ok false, without the interpreter's lock
// around the library call alone.
template <typename Body>
PyObject *answer(Py_ssize_t given, Py_ssize_t wanted, Body &&body) {
  if (given != wanted) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  int status = -1;
  try {
    status = body();
  } catch (...) {  // a tensor without storage, say: the long way reports it
    status = -1;
  }
  if (PyErr_Occurred()) PyErr_Clear();
  if (status < 0) Py_RETURN_NONE;
  return PyLong_FromLong(status);
}

template <typename F>
int unlocked(F &&f) {
  PyThreadState *state = PyEval_SaveThread();
  const int status = f();
  PyEval_RestoreThread(state);
  return status;
}

// (entry, ctx_lens, new_lens, block_table, free_pages, num_free, block_size, num_tokens,
//  num_free_out or None, seq_lens, cu_new, slots, positions, workspace, dev_status)
PyObject *assign_pages(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return answer(n, 15, [&]() -> int {
    Call c{args};
    const auto entry = c.address<decltype(&ksa_assign_pages)>(0);
    const at::Tensor *table = c.tensor(3, at::kInt), *free = c.tensor(4, at::kInt);
    if (!c.ok || table->dim() != 2 || !table->is_contiguous() || !free->is_contiguous()) return -1;
    const int64_t B = table->size(0), mb = table->size(1);
    const int32_t bs = c.integer(6), N = c.integer(7);
    const int32_t blocks = c.narrow(mb);
    const ksa_shape sh = {c.narrow(B), 1, 1, 64, c.narrow(mb * bs), bs};
    const int32_t pages = c.narrow(free->numel());
    const auto ctx = static_cast<const int32_t *>(c.vec(1, at::kInt, B));
    const auto add = static_cast<const int32_t *>(c.vec(2, at::kInt, B));
    const auto num = static_cast<int32_t *>(c.vec(5, at::kInt, 1));
    const auto left = args[8] == Py_None ? num : static_cast<int32_t *>(c.vec(8, at::kInt, 1));
    const auto seq = static_cast<int32_t *>(c.vec(9, at::kInt, B));
    const auto cu = static_cast<int32_t *>(c.vec(10, at::kInt, B + 1));
    const auto slots = static_cast<int64_t *>(c.vec(11, at::kLong, N));
    const auto positions = static_cast<int32_t *>(c.vec(12, at::kInt, N));
    size_t bytes = 0;
    void *ws = c.workspace(13, &bytes);
    uint32_t *status = c.status(14);
    void *stream = c.stream();
    if (!c.ok) return -1;
    return unlocked([&] {
      return entry(&sh, ctx, add, static_cast<int32_t *>(table->data_ptr()), blocks, pages,
                   static_cast<const int32_t *>(free->data_ptr()), num, left, N, seq, cu, slots,
                   positions, ws, bytes, status, stream);
    });
  });
}

// (entry, seq_lens, done, block_table, free_pages, num_free, block_size, workspace, dev_status)
PyObject *release_pages(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return answer(n, 9, [&]() -> int {
    Call c{args};
    const auto entry = c.address<decltype(&ksa_release_pages)>(0);
    const at::Tensor *table = c.tensor(3, at::kInt), *free = c.tensor(4, at::kInt);
    if (!c.ok || table->dim() != 2 || !table->is_contiguous() || !free->is_contiguous()) return -1;
    const int64_t B = table->size(0), mb = table->size(1);
    const int32_t bs = c.integer(6);
    const int32_t blocks = c.narrow(mb);
    const ksa_shape sh = {c.narrow(B), 1, 1, 64, c.narrow(mb * bs), bs};
    const int32_t pages = c.narrow(free->numel());
    const auto seq = static_cast<int32_t *>(c.vec(1, at::kInt, B));
    const auto done = static_cast<const int32_t *>(c.vec(2, at::kInt, B));
    const auto num = static_cast<int32_t *>(c.vec(5, at::kInt, 1));
    size_t bytes = 0;
    void *ws = c.workspace(7, &bytes);
    uint32_t *status = c.status(8);
    void *stream = c.stream();
    if (!c.ok) return -1;
    return unlocked([&] {
      return entry(&sh, done, seq, static_cast<int32_t *>(table->data_ptr()), blocks, pages,
                   static_cast<int32_t *>(free->data_ptr()), num, ws, bytes, status, stream);
    });
  });
}

// (entry, paged, q, k, v, positions, slots, K, V, rotary, q_out, dev_status): all of them given
PyObject *rotary_append(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return answer(n, 12, [&]() -> int {
    Call c{args};
    void *entry = c.address<void *>(0);
    const bool paged = args[1] == Py_True;
    const at::Tensor *q = c.tensor(2, at::kBFloat16), *K = c.tensor(7, at::kBFloat16);
    const auto rotary = c.address<const ksa_rotary *>(9);
    if (!c.ok || q->dim() != 3 || K->dim() != 4 || K->size(3) != q->size(2)) return -1;
    const int64_t N = q->size(0), Hq = q->size(1), D = q->size(2), Hkv = K->size(1);
    int32_t qs = 0, ks = 0, vs = 0, os = 0;
    const uint16_t *qp = c.rows(2, N, Hq, D, &qs), *kp = c.rows(3, N, Hkv, D, &ks),
                   *vp = c.rows(4, N, Hkv, D, &vs);
    uint16_t *op = c.rows(10, N, Hq, D, &os);
    const at::Tensor *pos = c.tensor(5, at::kInt);
    const int64_t axes = rotary->num_axes;
    if (!c.ok || !pos->is_contiguous() ||
        !((axes == 1 && pos->dim() == 1 && pos->size(0) == N) ||
          (pos->dim() == 2 && pos->size(0) == axes && pos->size(1) == N)))
      return -1;
    const auto slots = static_cast<const int64_t *>(c.vec(6, at::kLong, N));
    const auto Kp = static_cast<uint16_t *>(c.dense(7, at::kBFloat16, K->sizes()));
    const auto Vp = static_cast<uint16_t *>(c.dense(8, at::kBFloat16, K->sizes()));
    const int32_t lead = c.narrow(K->size(0)), T = c.narrow(K->size(2));
    const ksa_shape sh = {paged ? 1 : lead, c.narrow(Hq), c.narrow(Hkv), c.narrow(D),
                          T, paged ? T : 16};
    const int32_t tokens = c.narrow(N);
    uint32_t *status = c.status(11);
    void *stream = c.stream();
    if (!c.ok) return -1;
    const auto positions = static_cast<const int32_t *>(pos->data_ptr());
    return unlocked([&] {
      return paged ? reinterpret_cast<decltype(&ksa_rotary_append_kv_paged)>(entry)(
                         &sh, tokens, rotary, qp, qs, kp, ks, vp, vs, positions, slots, op, os,
                         Kp, Vp, lead, status, stream)
                   : reinterpret_cast<decltype(&ksa_rotary_append_kv)>(entry)(
                         &sh, tokens, rotary, qp, qs, kp, ks, vp, vs, positions, slots, op, os,
                         Kp, Vp, status, stream);
    });
  });
}

// (entry, q, K, V, block_table or None, cu_q, seq_lens, mask, scale, out, lse or None, workspace,
//  dev_status)
PyObject *chunk_attn(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return answer(n, 13, [&]() -> int {
    Call c{args};
    void *entry = c.address<void *>(0);
    const at::Tensor *q = c.tensor(1, at::kBFloat16), *K = c.tensor(2, at::kBFloat16);
    if (!c.ok || q->dim() != 3 || K->dim() != 4 || K->size(3) != q->size(2)) return -1;
    const int64_t N = q->size(0), Hq = q->size(1), D = q->size(2);
    int32_t qs = 0;
    const uint16_t *qp = c.rows(1, N, Hq, D, &qs);
    const auto Kp = static_cast<const uint16_t *>(c.dense(2, at::kBFloat16, K->sizes()));
    const auto Vp = static_cast<const uint16_t *>(c.dense(3, at::kBFloat16, K->sizes()));
    const bool paged = args[4] != Py_None;
    int64_t B = K->size(0), T = K->size(2), bs = 16;
    ksa_pages pages = {};
    if (paged) {
      const at::Tensor *table = c.tensor(4, at::kInt);
      if (!c.ok || table->dim() != 2 || !table->is_contiguous()) return -1;
      pages.block_table = static_cast<const int32_t *>(table->data_ptr());
      pages.max_blocks = c.narrow(table->size(1));
      pages.num_pages = c.narrow(B);
      B = table->size(0);
      bs = T;
      T = table->size(1) * bs;
    }
    const ksa_shape sh = {c.narrow(B), c.narrow(Hq), c.narrow(K->size(1)), c.narrow(D),
                          c.narrow(T), c.narrow(bs)};
    const auto cu = static_cast<const int32_t *>(c.vec(5, at::kInt, B + 1));
    const auto seq = static_cast<const int32_t *>(c.vec(6, at::kInt, B));
    const int32_t mask = c.integer(7), tokens = c.narrow(N);
    if (!PyFloat_Check(args[8])) return -1;
    const float scale = static_cast<float>(PyFloat_AS_DOUBLE(args[8]));
    const auto out = static_cast<uint16_t *>(c.dense(9, at::kBFloat16, q->sizes()));
    float *lse = args[10] == Py_None
                     ? nullptr
                     : static_cast<float *>(c.dense(10, at::kFloat, {N, Hq}));
    size_t bytes = 0;
    void *ws = c.workspace(11, &bytes);
    uint32_t *status = c.status(12);
    void *stream = c.stream();
    if (!c.ok) return -1;
    return unlocked([&] {
      return paged ? reinterpret_cast<decltype(&ksa_chunk_attn_paged)>(entry)(
                         &sh, tokens, qp, qs, Kp, Vp, &pages, cu, seq, mask, scale, out, lse, ws,
                         bytes, status, stream)
                   : reinterpret_cast<decltype(&ksa_chunk_attn)>(entry)(
                         &sh, tokens, qp, qs, Kp, Vp, cu, seq, mask, scale, out, lse, ws, bytes,
                         status, stream);
    });
  });
}

#define FAST(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(assign_pages), FAST(release_pages), FAST(rotary_append),
                         FAST(chunk_attn), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
  PyObject *m = PyModule_Create(&module);
  // the torch and Python whose layouts are compiled in: the binding uses no other build
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", KSA_BUILT_FOR) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
