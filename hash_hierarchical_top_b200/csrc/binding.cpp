// Python marshalling of the cache and page-attention calls of include/hhr.h.
//
// One token's call takes 4 to 10 us on the GPU; checking and converting a dozen tensors through
// ctypes takes 6 us more of the calling thread, this module under one. It checks every tensor
// (type, device, layout, size), takes the current stream and calls the C function; argument
// errors are Python exceptions, the C function's status is returned. The functions' addresses
// come from the already loaded library (`bind`), so there is one copy of it in the process.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <stdexcept>
#include <string>

#include "../../include/hhr.h"

namespace {

struct ArgError {  // a Python exception that is already set
};
[[noreturn]] void fail(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw ArgError{};
}

using Types = std::initializer_list<at::ScalarType>;
const Types kBf16 = {at::kBFloat16, at::kShort, at::kUInt16};
const Types kE4m3 = {at::kFloat8_e4m3fn, at::kByte};
const Types kU8 = {at::kByte};
const Types kI32 = {at::kInt};
const Types kF32 = {at::kFloat};
const Types kOut = {at::kFloat, at::kBFloat16};

// One call: its dims and device.
struct Call {
  const hhr_dims* d;
  Py_buffer buf;
  int dev = -1;  // of the first tensor that is looked at; it has to be the current one
  explicit Call(PyObject* dims) {
    if (PyObject_GetBuffer(dims, &buf, PyBUF_SIMPLE) != 0) throw ArgError{};
    if (buf.len != (Py_ssize_t)sizeof(hhr_dims)) {
      PyBuffer_Release(&buf);
      fail(PyExc_TypeError, "dims: expected the dims of make_dims");
    }
    d = static_cast<const hhr_dims*>(buf.buf);
  }
  ~Call() { PyBuffer_Release(&buf); }
  Call(const Call&) = delete;

  const at::Tensor& tensor(PyObject* o, const char* name, const Types& types) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + ": expected a torch tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) fail(PyExc_ValueError, std::string(name) + ": expected a CUDA tensor");
    if (dev < 0) dev = c10::cuda::current_device();
    if (t.get_device() != dev)
      fail(PyExc_ValueError, std::string(name) + ": on cuda:" + std::to_string(t.get_device()) +
                                 ", expected cuda:" + std::to_string(dev) + ", the current device");
    for (at::ScalarType s : types)
      if (t.scalar_type() == s) return t;
    fail(PyExc_TypeError, std::string(name) + ": dtype " + c10::toString(t.scalar_type()) +
                              " is not one that this argument takes");
  }
  // Address of a contiguous tensor of at least n elements.
  void* ptr(PyObject* o, const char* name, const Types& types, int64_t n) {
    const at::Tensor& t = tensor(o, name, types);
    if (!t.is_contiguous()) fail(PyExc_ValueError, std::string(name) + ": expected a contiguous tensor");
    if (t.numel() < n)
      fail(PyExc_ValueError, std::string(name) + ": " + std::to_string(t.numel()) +
                                 " elements, expected at least " + std::to_string(n));
    return t.data_ptr();
  }
  void* opt(PyObject* o, const char* name, const Types& types, int64_t n) {
    return o == Py_None ? nullptr : ptr(o, name, types, n);
  }
  template <typename T>
  T* as(PyObject* o, const char* name, const Types& types, int64_t n) {
    return static_cast<T*>(opt(o, name, types, n));
  }

  int64_t rows() const { return (int64_t)d->n_phys_pages * d->n_kv_heads * d->page_size; }
  int64_t sel_rows() const { return d->select_per_head ? d->n_q_heads : d->n_kv_heads; }
  const int32_t* page_table(PyObject* o) {
    return as<const int32_t>(o, "page_table", kI32, (int64_t)d->batch * d->max_pages_per_seq);
  }
  const int32_t* per_sequence(PyObject* o, const char* name) {
    return as<const int32_t>(o, name, kI32, d->batch);
  }
  // The raw handle of a stream argument (None: the current stream of the device).
  void* stream(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    PyObject* v = PyLong_Check(o) ? (Py_INCREF(o), o) : PyObject_GetAttrString(o, "cuda_stream");
    if (v == nullptr) throw ArgError{};
    void* p = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (p == nullptr && PyErr_Occurred()) throw ArgError{};
    return p;
  }
};

// A paged cache: bf16 when both exponents are None.
struct Cache {
  uint8_t *k, *v, *k_exp, *v_exp;
  Cache(Call& c, PyObject* const* a, bool must_be_8bit) {
    const bool bf16 = a[2] == Py_None && a[3] == Py_None;
    if (must_be_8bit && (a[2] == Py_None || a[3] == Py_None))
      fail(PyExc_ValueError, "k_exp, v_exp: an 8-bit cache has exponents");
    const Types& types = bf16 ? kBf16 : kE4m3;
    const int64_t n = c.rows();
    k = c.as<uint8_t>(a[0], "k", types, n * c.d->head_dim);
    v = c.as<uint8_t>(a[1], "v", types, n * c.d->head_dim);
    k_exp = c.as<uint8_t>(a[2], "k_exp", kU8, n);
    v_exp = c.as<uint8_t>(a[3], "v_exp", kU8, n);
  }
};

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw ArgError{};
  return v;
}

// New rows [B][n][G][d] or [B][G][d]: channels and heads side by side, tokens evenly spaced over
// all sequences.
struct NewRows {
  const uint16_t* p;
  int64_t n, stride;
  NewRows(Call& c, PyObject* o, const char* name) {
    const at::Tensor& t = c.tensor(o, name, kBf16);
    const int64_t B = c.d->batch, G = c.d->n_kv_heads, D = c.d->head_dim, m = t.dim();
    if ((m != 3 && m != 4) || t.size(0) != B || t.size(m - 2) != G || t.size(m - 1) != D)
      fail(PyExc_ValueError, std::string(name) + ": expected the shape [" + std::to_string(B) +
                                 "][n][" + std::to_string(G) + "][" + std::to_string(D) + "]");
    n = m == 4 ? t.size(1) : 1;
    // One token a sequence: the tokens' spacing is the sequences'.
    stride = n != 1 ? t.stride(1) : B > 1 ? t.stride(0) : G * D;
    if (t.stride(m - 1) != 1 || (G > 1 && t.stride(m - 2) != D) ||
        (B > 1 && n > 0 && t.stride(0) != n * stride))
      fail(PyExc_ValueError, std::string(name) + ": its strides are not those of evenly spaced tokens");
    p = static_cast<const uint16_t*>(t.data_ptr());
  }
};

decltype(&hhr_append_kv8) f_append;
decltype(&hhr_read_kv8) f_read;
decltype(&hhr_paged_attn) f_paged;
decltype(&hhr_block_select) f_select;
decltype(&hhr_block_attn) f_block;

// Without the interpreter's lock: a launch can wait for room in the stream.
template <typename F, typename... Args>
int unlocked(F f, Args... args) {
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = f(args...);
  Py_END_ALLOW_THREADS
  return st;
}

// Runs `body` with the argument count checked; C++ exceptions become Python's.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F body) {
  try {
    if (n != want) fail(PyExc_TypeError, "expected " + std::to_string(want) + " arguments");
    if (f_append == nullptr) fail(PyExc_RuntimeError, "the library is not bound");
    return PyLong_FromLong(body());
  } catch (const ArgError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (d, k_new, v_new, start, n_new, page_table, k, v, k_exp, v_exp, block_mean, stream)
PyObject* append_kv8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> int {
    Call c(a[0]);
    const NewRows k(c, a[1], "k_new"), v(c, a[2], "v_new");
    if (k.n != v.n || k.stride != v.stride)
      fail(PyExc_ValueError, "k_new and v_new: expected the same shape and strides");
    const Cache w(c, a + 6, true);
    if (k.n > INT32_MAX) fail(PyExc_ValueError, "k_new: too many rows");
    const int32_t *start = c.per_sequence(a[3], "start"), *count = c.per_sequence(a[4], "n_new"),
                  *pt = c.page_table(a[5]);
    float* mean = c.as<float>(a[10], "block_mean", kF32,
                              (int64_t)c.d->n_phys_pages * c.d->n_kv_heads * c.d->head_dim);
    if (k.n == 0) return HHR_OK;  // no element, hence no address to pass
    return unlocked(f_append, c.d, k.p, v.p, k.stride, start, count, (int)k.n, pt, w.k, w.v, w.k_exp, w.v_exp,
                    mean, c.stream(a[11]));
  });
}

// (d, k, v, k_exp, v_exp, page_table, start, n, k_out, v_out, stream)
PyObject* read_kv8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> int {
    Call c(a[0]);
    const at::Tensor &ko = c.tensor(a[8], "k_out", kBf16), &vo = c.tensor(a[9], "v_out", kBf16);
    if (ko.dim() != 4 || ko.sizes() != vo.sizes() || ko.size(0) != c.d->batch ||
        ko.size(2) != c.d->n_kv_heads || ko.size(3) != c.d->head_dim || ko.size(1) > INT32_MAX)
      fail(PyExc_ValueError, "k_out, v_out: expected [B][max_n][G][d], both alike");
    const Cache w(c, a + 1, true);
    const int64_t total = ko.numel();
    const int32_t *pt = c.page_table(a[5]), *start = c.per_sequence(a[6], "start"),
                  *count = c.per_sequence(a[7], "n");
    uint16_t *kp = c.as<uint16_t>(a[8], "k_out", kBf16, total),
             *vp = c.as<uint16_t>(a[9], "v_out", kBf16, total);
    if (total == 0) return HHR_OK;
    return unlocked(f_read, c.d, w.k, w.v, w.k_exp, w.v_exp, pt, start, count, (int)ko.size(1), kp, vp,
                  c.stream(a[10]));
  });
}

// (d, q, k_new, v_new, k, v, k_exp, v_exp, page_table, seq_len, scale, out, workspace, lse, stream)
PyObject* paged_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> int {
    Call c(a[0]);
    const int64_t B = c.d->batch, heads = B * c.d->n_q_heads, D = c.d->head_dim;
    const uint16_t* q = c.as<const uint16_t>(a[1], "q", kBf16, heads * D);
    const uint16_t* kn = c.as<const uint16_t>(a[2], "k_new", kBf16, B * c.d->n_kv_heads * D);
    const uint16_t* vn = c.as<const uint16_t>(a[3], "v_new", kBf16, B * c.d->n_kv_heads * D);
    const Cache w(c, a + 4, false);
    const int32_t *pt = c.page_table(a[8]), *len = c.per_sequence(a[9], "seq_len");
    void* out = c.ptr(a[11], "out", kOut, heads * D);
    void* ws = c.ptr(a[12], "workspace", kU8, 0);
    return unlocked(f_paged, c.d, q, kn, vn, w.k, w.v, w.k_exp, w.v_exp, pt, len, (float)number(a[10]), out,
                   THPVariable_Unpack(a[11]).scalar_type() == at::kBFloat16,
                   c.as<float>(a[13], "lse", kF32, heads), ws,
                   (size_t)THPVariable_Unpack(a[12]).numel(), c.stream(a[14]));
  });
}

// Queries per sequence of q [B][T][Hq][d].
int64_t queries(Call& c, PyObject* o) {
  const at::Tensor& q = c.tensor(o, "q", kBf16);
  if (q.dim() != 4 || q.size(0) != c.d->batch || q.size(2) != c.d->n_q_heads ||
      q.size(3) != c.d->head_dim || q.size(1) > INT32_MAX)
    fail(PyExc_ValueError, "q: expected the shape [B][T][Hq][d]");
  return q.size(1);
}

// (d, q, seq_len, q_pos, page_table, block_mean, m_pages, opts, blocks, count, workspace, stream)
PyObject* block_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> int {
    Call c(a[0]);
    const int64_t T = queries(c, a[1]), B = c.d->batch, rows = B * T * c.sel_rows();
    const long m = PyLong_AsLong(a[6]);
    if (m == -1 && PyErr_Occurred()) throw ArgError{};
    const long m_max = std::max(0L, std::min<long>(m, c.d->max_pages_per_seq));
    hhr_select_opts opts{0, 0};
    if (a[7] != Py_None) {
      Py_buffer b;
      if (PyObject_GetBuffer(a[7], &b, PyBUF_SIMPLE) != 0) throw ArgError{};
      const bool ok = b.len == (Py_ssize_t)sizeof(opts);
      if (ok) opts = *static_cast<const hhr_select_opts*>(b.buf);
      PyBuffer_Release(&b);
      if (!ok) fail(PyExc_TypeError, "opts: expected the options of make_opts");
    }
    const uint16_t* q = c.as<const uint16_t>(a[1], "q", kBf16, 0);
    const int32_t *len = c.per_sequence(a[2], "seq_len"),
                  *pos = c.as<const int32_t>(a[3], "q_pos", kI32, B * T), *pt = c.page_table(a[4]);
    const float* mean = c.as<const float>(a[5], "block_mean", kF32,
                                          (int64_t)c.d->n_phys_pages * c.d->n_kv_heads * c.d->head_dim);
    int32_t *blocks = c.as<int32_t>(a[8], "out_blocks", kI32, rows * m_max),
            *count = c.as<int32_t>(a[9], "out_count", kI32, rows);
    void* ws = c.ptr(a[10], "workspace", kU8, 0);
    return unlocked(f_select, c.d, (int)T, q, len, pos, pt, mean, (int)std::max(-1L, std::min<long>(m, INT32_MAX)),
                    &opts, blocks, count, ws, (size_t)THPVariable_Unpack(a[10]).numel(),
                    c.stream(a[11]));
  });
}

// (d, q, k, v, k_exp, v_exp, page_table, seq_len, q_pos, blocks, count, scale, out, workspace, lse,
//  stream)
PyObject* block_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> int {
    Call c(a[0]);
    const int64_t T = queries(c, a[1]), B = c.d->batch, heads = B * T * c.d->n_q_heads;
    const int64_t rows = B * T * c.sel_rows();
    const uint16_t* q = c.as<const uint16_t>(a[1], "q", kBf16, 0);
    const Cache w(c, a + 2, false);
    const int32_t *pt = c.page_table(a[6]), *len = c.per_sequence(a[7], "seq_len"),
                  *pos = c.as<const int32_t>(a[8], "q_pos", kI32, B * T);
    const at::Tensor& bl = c.tensor(a[9], "blocks", kI32);
    const int64_t m = bl.dim() > 0 ? bl.size(-1) : 0;
    if (m > INT32_MAX) fail(PyExc_ValueError, "blocks: too many columns");
    const int32_t *blocks = c.as<const int32_t>(a[9], "blocks", kI32, rows * m),
                  *count = c.as<const int32_t>(a[10], "block_count", kI32, rows);
    void* out = c.ptr(a[12], "out", kOut, heads * c.d->head_dim);
    void* ws = c.ptr(a[13], "workspace", kU8, 0);
    return unlocked(f_block, c.d, (int)T, q, w.k, w.v, w.k_exp, w.v_exp, pt, len, pos, blocks, count, (int)m,
                   (float)number(a[11]), out, THPVariable_Unpack(a[12]).scalar_type() == at::kBFloat16,
                   c.as<float>(a[14], "lse", kF32, heads), ws,
                   (size_t)THPVariable_Unpack(a[13]).numel(), c.stream(a[15]));
  });
}

// bind(append, read, paged, select, block): the C functions' addresses.
PyObject* bind(PyObject*, PyObject* args) {
  Py_ssize_t p[5];
  if (!PyArg_ParseTuple(args, "nnnnn", p, p + 1, p + 2, p + 3, p + 4)) return nullptr;
  f_append = reinterpret_cast<decltype(f_append)>(p[0]);
  f_read = reinterpret_cast<decltype(f_read)>(p[1]);
  f_paged = reinterpret_cast<decltype(f_paged)>(p[2]);
  f_select = reinterpret_cast<decltype(f_select)>(p[3]);
  f_block = reinterpret_cast<decltype(f_block)>(p[4]);
  Py_RETURN_NONE;
}

#define FAST(f) (PyCFunction)(void (*)(void))(f), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"append_kv8", FAST(append_kv8)},     {"read_kv8", FAST(read_kv8)},
                         {"paged_attn", FAST(paged_attn)},     {"block_select", FAST(block_select)},
                         {"block_attn", FAST(block_attn)},     {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  // The torch and Python that this was compiled against; build.py looks for it in the file.
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", HHR_BUILT_FOR) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
