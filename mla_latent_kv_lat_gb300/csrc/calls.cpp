// The paged calls' way from Python to the C ABI, for a step's short calls: a decode
// step makes each of them once a layer, and in Python the checks of ten tensors and the
// conversion of twenty arguments take longer than the kernels (normed append of 64
// tokens: 11.5 us in Python, 3.5 on the GPU).
//
// Each function takes the arguments of the binding's function of that name, in order,
// checks what that function checks, and returns the C call's status; or None for
// anything that is not plainly right (a wrong type, shape or device, another current
// device): the binding then takes its own way, which says what is wrong.  The C call
// itself is made without the interpreter's lock, as ctypes makes it: a launch waits
// where the queue is full, maybe for a host function that needs the lock.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>

#include "mla.h"

namespace {

constexpr int64_t kLatent = 512, kRope = 64, kNope = 128, kRow = 576, kRowE4m3 = 656, kBlock = 64;

struct Lib {
  decltype(&::mla_paged_append) append;
  decltype(&::mla_paged_gather) gather;
  decltype(&::mla_attn_paged) attn;
  decltype(&::mla_paged_norm_append) norm_append;
  decltype(&::mla_paged_block_keys) block_keys;
  decltype(&::mla_paged_block_scores) block_scores;
  decltype(&::mla_paged_select_blocks) select_blocks;
  decltype(&::mla_attn_paged_blocks) attn_blocks;
} lib;

struct NotPlain {};                          // thrown where the arguments are not what a call takes
void need(bool ok) {
  if (!ok) throw NotPlain();
}

const at::Tensor& tensor(PyObject* o) {
  need(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

// A call's device: its first tensor's, which has to be the current one.
int device_of(const at::Tensor& t) {
  need(t.is_cuda() && t.get_device() == c10::cuda::current_device());
  return static_cast<int>(t.get_device());
}

void* contiguous(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, int dev) {
  const at::Tensor& t = tensor(o);
  need(t.scalar_type() == type && t.is_cuda() && t.get_device() == dev && t.sizes() == at::IntArrayRef(shape) &&
       t.is_contiguous());
  return t.data_ptr();
}
const int32_t* i32(PyObject* o, std::initializer_list<int64_t> shape, int dev) {
  return static_cast<const int32_t*>(contiguous(o, at::kInt, shape, dev));
}
int32_t fit(int64_t x) {
  need(x >= INT32_MIN && x <= INT32_MAX);
  return static_cast<int32_t>(x);
}
int32_t integer(PyObject* o) {
  need(PyLong_Check(o));
  int over = 0;
  const long long x = PyLong_AsLongLongAndOverflow(o, &over);
  need(over == 0);
  return fit(x);
}
float number(PyObject* o) {
  need(PyFloat_Check(o) || PyLong_Check(o));
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw NotPlain();
  }
  return static_cast<float>(x);
}
void* stream(PyObject* o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  PyObject* handle = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  if (handle == nullptr) {
    PyErr_Clear();
    throw NotPlain();
  }
  void* s = PyLong_Check(handle) ? PyLong_AsVoidPtr(handle) : nullptr;
  const bool ok = PyLong_Check(handle) && PyErr_Occurred() == nullptr;
  Py_DECREF(handle);
  PyErr_Clear();
  need(ok);
  return s;
}

mla_dims dims(int64_t heads, PyObject* scale) {
  mla_dims d = {fit(heads), kLatent, kRope, kNope, 128, static_cast<float>(1.0 / std::sqrt(192.0))};
  if (scale != nullptr && scale != Py_None) d.scale = number(scale);
  return d;
}

// The block table's part of a cache; rows may be further apart than they are long.
void table(mla_paged_cache& c, PyObject* o, int dev, int32_t& B) {
  const at::Tensor& t = tensor(o);
  need(t.scalar_type() == at::kInt && t.dim() == 2 && t.is_cuda() && t.get_device() == dev && t.size(0) >= 1 &&
       t.size(1) >= 1 && (t.stride(1) == 1 || t.size(1) == 1));
  c.block_table = static_cast<const int32_t*>(t.data_ptr());
  c.table_stride = t.stride(0);
  c.max_pages = fit(t.size(1));
  B = fit(t.size(0));
}
mla_paged_cache paged(PyObject* pages, PyObject* block_table, int dev, int32_t& B) {
  const at::Tensor& t = tensor(pages);
  const bool f16 = t.scalar_type() == at::kHalf;
  need((f16 || t.scalar_type() == at::kByte) && t.dim() == 3 && t.size(2) == (f16 ? kRow : kRowE4m3) && t.is_cuda() &&
       t.get_device() == dev && t.is_contiguous());
  mla_paged_cache c = {};
  c.pages = t.data_ptr();
  c.n_pages = fit(t.size(0));
  c.page_size = fit(t.size(1));
  c.type = f16 ? MLA_PAGE_F16 : MLA_PAGE_E4M3;
  table(c, block_table, dev, B);
  return c;
}

// f(args...) without the interpreter's lock; the arguments are made with it.
template <typename F, typename... Args>
int unlocked(F f, Args... args) {
  PyThreadState* state = PyEval_SaveThread();
  const int status = f(args...);       // (a C entry: it throws nothing)
  PyEval_RestoreThread(state);
  return status;
}

template <typename Call>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, Call call) {
  try {
    if (n == want) return PyLong_FromLong(call());
  } catch (...) {                            // NotPlain, or what a tensor without storage throws
    PyErr_Clear();
  }
  Py_RETURN_NONE;
}

// q, kv, q_weight, kv_weight, pages, block_table, cu_new, seq_len, q_nope, q_pe, eps, freq_base, freq_scale, stream
PyObject* norm_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> int {
    const at::Tensor &q = tensor(a[0]), &kv = tensor(a[1]);
    const int dev = device_of(q);
    need(q.scalar_type() == at::kBFloat16 && q.dim() == 3 && q.size(2) == kNope + kRope && q.stride(2) == 1);
    const int64_t T = q.size(0), H = q.size(1);
    need(kv.scalar_type() == at::kBFloat16 && kv.is_cuda() && kv.get_device() == dev && kv.dim() == 2 && kv.size(0) == T &&
         kv.size(1) == kRow && kv.stride(1) == 1);
    const mla_dims d = dims(H, nullptr);
    int32_t B;
    const mla_paged_cache c = paged(a[4], a[5], dev, B);
    // (the stride of a dimension of one counts for nothing, and may be anything)
    return unlocked(lib.norm_append, &d, q.data_ptr(), T > 1 ? q.stride(0) : 0, H > 1 ? q.stride(1) : 0, kv.data_ptr(),
                           T > 1 ? kv.stride(0) : 0,
                           a[2] == Py_None ? nullptr : contiguous(a[2], at::kBFloat16, {kNope + kRope}, dev),
                           contiguous(a[3], at::kBFloat16, {kLatent}, dev), &c, i32(a[6], {int64_t{B} + 1}, dev),
                           i32(a[7], {B}, dev), B, fit(T), number(a[10]), number(a[11]), number(a[12]),
                           contiguous(a[8], at::kBFloat16, {T, H, kNope}, dev),
                           contiguous(a[9], at::kBFloat16, {T, H, kRope}, dev), stream(a[13], dev));
  });
}

// c_kv, k_pe, pages, block_table, cu_new, seq_len, freq_base, freq_scale, stream
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> int {
    const at::Tensor& kv = tensor(a[0]);
    const int dev = device_of(kv);
    need(kv.dim() == 2);
    const int64_t T = kv.size(0);
    int32_t B;
    const mla_paged_cache c = paged(a[2], a[3], dev, B);
    return unlocked(lib.append, &c, contiguous(a[0], at::kBFloat16, {T, kLatent}, dev), contiguous(a[1], at::kBFloat16, {T, kRope}, dev),
                      i32(a[4], {int64_t{B} + 1}, dev), i32(a[5], {B}, dev), B, fit(T), number(a[6]), number(a[7]),
                      stream(a[8], dev));
  });
}

// pages, block_table, row0, cu_rows, out, stream
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> int {
    const at::Tensor& out = tensor(a[4]);
    const int dev = device_of(out);
    const bool f16 = out.scalar_type() == at::kHalf;
    need(out.dim() == 2);
    const int64_t R = out.size(0);
    int32_t B;
    const mla_paged_cache c = paged(a[0], a[1], dev, B);
    return unlocked(lib.gather, &c, a[2] == Py_None ? nullptr : i32(a[2], {B}, dev), i32(a[3], {int64_t{B} + 1}, dev), B, fit(R),
                      contiguous(a[4], f16 ? at::kHalf : at::kBFloat16, {R, kRow}, dev), f16, stream(a[5], dev));
  });
}

// pages, block_table, cu_new, seq_len, block_keys, T, stream
PyObject* block_keys(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> int {
    const int dev = device_of(tensor(a[0]));
    int32_t B;
    const mla_paged_cache c = paged(a[0], a[1], dev, B);
    return unlocked(lib.block_keys, &c, i32(a[2], {int64_t{B} + 1}, dev), i32(a[3], {B}, dev), B, integer(a[5]),
                          contiguous(a[4], at::kHalf, {c.n_pages, c.page_size / kBlock, kRow}, dev), stream(a[6], dev));
  });
}

struct Rows {
  const at::Tensor& t;
  Rows(PyObject* o, int64_t T, int dev) : t(tensor(o)) {
    need(t.scalar_type() == at::kFloat && t.dim() == 2 && t.size(0) == T && t.size(1) >= 1 && t.is_cuda() &&
         t.get_device() == dev && (t.stride(1) == 1 || t.size(1) == 1));
  }
  float* data() const { return static_cast<float*>(t.data_ptr()); }
};

struct Queries {
  const at::Tensor& t;
  int dev;
  int64_t T, H;
  explicit Queries(PyObject* o) : t(tensor(o)), dev(device_of(t)) {
    need(t.scalar_type() == at::kHalf && t.dim() == 3 && t.size(2) == kLatent && t.is_contiguous());
    T = t.size(0);
    H = t.size(1);
  }
};

// q_lat, q_pe, block_keys, block_table, cu_q, seq_len, scores, scale, stream
PyObject* block_scores(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> int {
    const Queries q(a[0]);
    const mla_dims d = dims(q.H, a[7]);
    const at::Tensor& keys = tensor(a[2]);
    need(keys.dim() == 3);
    void* k = contiguous(a[2], at::kHalf, {keys.size(0), keys.size(1), kRow}, q.dev);
    mla_paged_cache c = {};
    c.n_pages = fit(keys.size(0));
    c.page_size = fit(keys.size(1) * kBlock);
    int32_t B;
    table(c, a[3], q.dev, B);
    const Rows s(a[6], q.T, q.dev);
    return unlocked(lib.block_scores, &d, q.t.data_ptr(), contiguous(a[1], at::kBFloat16, {q.T, q.H, kRope}, q.dev), &c, k,
                            i32(a[4], {int64_t{B} + 1}, q.dev), i32(a[5], {B}, q.dev), B, fit(q.T), s.data(), s.t.stride(0),
                            fit(s.t.size(1)), stream(a[8], q.dev));
  });
}

// scores, cu_q, seq_len, blocks, counts, n_sink, n_local, stream
PyObject* select_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> int {
    const int dev = device_of(tensor(a[0]));
    const at::Tensor &blocks = tensor(a[3]), &len = tensor(a[2]);
    need(blocks.dim() == 2 && len.dim() == 1);
    const int64_t T = blocks.size(0), K = blocks.size(1), B = len.size(0);
    const Rows s(a[0], T, dev);
    return unlocked(lib.select_blocks, s.data(), s.t.stride(0), fit(s.t.size(1)), i32(a[1], {B + 1}, dev), i32(a[2], {B}, dev), fit(B),
                             fit(T), integer(a[5]), integer(a[6]), const_cast<int32_t*>(i32(a[3], {T, K}, dev)),
                             const_cast<int32_t*>(i32(a[4], {T}, dev)), fit(K), stream(a[7], dev));
  });
}

// q_lat, q_pe, pages, block_table, cu_q, seq_len, o_lat, window, n_sink, workspace, scale, stream
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> int {
    const Queries q(a[0]);
    const mla_dims d = dims(q.H, a[10]);
    int32_t B;
    const mla_paged_cache c = paged(a[2], a[3], q.dev, B);
    const at::Tensor& ws = tensor(a[9]);
    need(ws.scalar_type() == at::kByte && ws.is_cuda() && ws.get_device() == q.dev && ws.is_contiguous());
    return unlocked(lib.attn, &d, q.t.data_ptr(), contiguous(a[1], at::kBFloat16, {q.T, q.H, kRope}, q.dev), &c,
                    i32(a[4], {int64_t{B} + 1}, q.dev), i32(a[5], {B}, q.dev), B, fit(q.T), integer(a[7]), integer(a[8]),
                    ws.data_ptr(), static_cast<size_t>(ws.numel()), contiguous(a[6], at::kHalf, {q.T, q.H, kLatent}, q.dev),
                    stream(a[11], q.dev));
  });
}

// q_lat, q_pe, pages, block_table, cu_q, seq_len, blocks, counts, o_lat, workspace, scale, stream
PyObject* attn_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> int {
    const Queries q(a[0]);
    const mla_dims d = dims(q.H, a[10]);
    int32_t B;
    const mla_paged_cache c = paged(a[2], a[3], q.dev, B);
    const at::Tensor &blocks = tensor(a[6]), &ws = tensor(a[9]);
    need(blocks.dim() == 2 && blocks.size(0) == q.T);
    need(ws.scalar_type() == at::kByte && ws.is_cuda() && ws.get_device() == q.dev && ws.is_contiguous());
    const int64_t K = blocks.size(1);
    return unlocked(lib.attn_blocks, &d, q.t.data_ptr(), contiguous(a[1], at::kBFloat16, {q.T, q.H, kRope}, q.dev), &c,
                           i32(a[4], {int64_t{B} + 1}, q.dev), i32(a[5], {B}, q.dev), B, fit(q.T), i32(a[6], {q.T, K}, q.dev),
                           i32(a[7], {q.T}, q.dev), fit(K), ws.data_ptr(), static_cast<size_t>(ws.numel()),
                           contiguous(a[8], at::kHalf, {q.T, q.H, kLatent}, q.dev), stream(a[11], q.dev));
  });
}

// The library whose functions are called.
PyObject* bind(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (p == nullptr) return nullptr;
  void* h = dlopen(p, RTLD_NOW | RTLD_LOCAL);
  if (h == nullptr) return PyErr_Format(PyExc_RuntimeError, "%s", dlerror());
  auto find = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(dlsym(h, name));
    return f != nullptr;
  };
  if (!find(lib.append, "mla_paged_append") || !find(lib.gather, "mla_paged_gather") || !find(lib.attn, "mla_attn_paged") ||
      !find(lib.norm_append, "mla_paged_norm_append") || !find(lib.block_keys, "mla_paged_block_keys") ||
      !find(lib.block_scores, "mla_paged_block_scores") || !find(lib.select_blocks, "mla_paged_select_blocks") ||
      !find(lib.attn_blocks, "mla_attn_paged_blocks"))
    return PyErr_Format(PyExc_RuntimeError, "%s lacks a function", p);
  Py_RETURN_NONE;
}

#define MLA_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         {"append", MLA_FAST(append), METH_FASTCALL, nullptr},
                         {"gather", MLA_FAST(gather), METH_FASTCALL, nullptr},
                         {"attn", MLA_FAST(attn), METH_FASTCALL, nullptr},
                         {"norm_append", MLA_FAST(norm_append), METH_FASTCALL, nullptr},
                         {"block_keys", MLA_FAST(block_keys), METH_FASTCALL, nullptr},
                         {"block_scores", MLA_FAST(block_scores), METH_FASTCALL, nullptr},
                         {"select_blocks", MLA_FAST(select_blocks), METH_FASTCALL, nullptr},
                         {"attn_blocks", MLA_FAST(attn_blocks), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
