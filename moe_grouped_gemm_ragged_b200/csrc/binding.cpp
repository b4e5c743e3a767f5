// The calls of _layer.py with their buffers in hand, as a CPython module: the same checks of the
// arguments as there, in a tenth of the time (a small call waits for the host, not for the GPU).
// A function returns the C call's status, or None when something is not as the call needs it or
// has to be made first; _layer.py then goes through its own checks, which name what is wrong. The
// C entry points come from the loaded library by address (bind), so this module links to torch
// only.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <initializer_list>

#include "gg.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Entry {
  const char* name;
  void* address;
};
Entry g_entries[] = {{"gg_gate_topk", nullptr},      {"gg_gate_topk_backward", nullptr},
                     {"gg_unroute", nullptr},        {"gg_unroute_backward", nullptr},
                     {"gg_silu_mul", nullptr},       {"gg_silu_mul_backward", nullptr},
                     {"gg_pack8", nullptr},          {"gg_unpack8", nullptr}};
enum { GATE, GATE_BACKWARD, UNROUTE, UNROUTE_BACKWARD, SILU, SILU_BACKWARD, PACK, UNPACK };

template <typename F>
F* entry(int i) {
  return reinterpret_cast<F*>(g_entries[i].address);
}

// Reads one call's arguments; `ok` falls when one is not as the call needs it.
struct Reader {
  bool ok = true;
  int device = -1;

  // A tensor proper (no subclass) of this type and number of dimensions, contiguous, on the
  // current device; the first one sets the device.
  const Tensor* tensor(PyObject* o, ScalarType type, int64_t dims) {
    if (!ok || !THPVariable_CheckExact(o)) return fail();
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.scalar_type() != type || t.dim() != dims || !t.is_contiguous())
      return fail();
    const int d = t.get_device();
    if (device < 0) {
      if (d != c10::cuda::current_device()) return fail();
      device = d;
    }
    return d == device ? &t : fail();
  }
  void* sized(PyObject* o, ScalarType type, std::initializer_list<int64_t> sizes) {
    const Tensor* t = tensor(o, type, (int64_t)sizes.size());
    if (t == nullptr) return nullptr;
    int64_t i = 0;
    for (const int64_t n : sizes)
      if (t->size(i++) != n) return fail();
    return t->data_ptr();
  }
  void* optional(PyObject* o, ScalarType type, std::initializer_list<int64_t> sizes) {
    return o == Py_None ? nullptr : sized(o, type, sizes);
  }
  // fp32, n values in any shape
  float* values(PyObject* o, int64_t n) {
    if (o == Py_None || !ok) return nullptr;
    if (!THPVariable_CheckExact(o)) return fail();
    const Tensor* t = tensor(o, ScalarType::Float, THPVariable_Unpack(o).dim());
    if (t == nullptr || t->numel() != n) return fail();
    return static_cast<float*>(t->data_ptr());
  }
  // the last of the offsets: the rows in use
  const int32_t* used(PyObject* offs) {
    if (offs == Py_None) return nullptr;
    const Tensor* t = tensor(offs, ScalarType::Int, 1);
    if (t == nullptr || t->numel() == 0) return fail();
    return static_cast<const int32_t*>(t->data_ptr()) + (t->numel() - 1);
  }
  int32_t* status(PyObject* o) {
    if (o == Py_None) return nullptr;
    const Tensor* t = tensor(o, ScalarType::Int, 1);
    return t != nullptr ? static_cast<int32_t*>(t->data_ptr()) : nullptr;
  }
  int64_t integer(PyObject* o) {
    if (!PyLong_CheckExact(o)) return fail(), 0;
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
    if (overflow != 0) fail();
    return v;
  }
  bool truth(PyObject* o) {
    if (o != Py_True && o != Py_False) fail();
    return o == Py_True;
  }
  float real(PyObject* o) {
    if (!PyFloat_CheckExact(o)) return fail(), 0.f;
    return (float)PyFloat_AS_DOUBLE(o);
  }
  cudaStream_t stream(PyObject* o) {
    if (!ok) return nullptr;
    if (o == Py_None)
      return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    return reinterpret_cast<cudaStream_t>(integer(o));
  }
  std::nullptr_t fail() {
    ok = false;
    return nullptr;
  }
};

constexpr ScalarType BF16 = ScalarType::BFloat16, F32 = ScalarType::Float, I32 = ScalarType::Int,
                     E4M3 = ScalarType::Float8_e4m3fn, E8M0 = ScalarType::Float8_e8m0fnu;

int64_t blocks(int64_t cols) { return (cols + 31) / 32; }

// Runs `call` on the arguments: its status, or None. Nothing that torch throws gets past here.
template <int N, typename F>
PyObject* guarded(int which, PyObject* const* a, Py_ssize_t n, const F& call) {
  if (n != N || g_entries[which].address == nullptr) Py_RETURN_NONE;
  try {
    Reader r;
    gg_status s = GG_OK;
    if (!call(r, a, &s)) Py_RETURN_NONE;
    return PyLong_FromLong((long)s);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

// logits, k, score, renorm, scale, bias, num_tokens, topk_ids, weights, status, stream
PyObject* gate_topk(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded<11>(GATE, args, nargs, [](Reader& r, PyObject* const* a, gg_status* s) {
    if (!THPVariable_CheckExact(a[0])) return false;
    const ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
    if (type != BF16 && type != F32) return false;
    const Tensor* x = r.tensor(a[0], type, 2);
    if (x == nullptr) return false;
    const int64_t T = x->size(0), E = x->size(1), k = r.integer(a[1]), score = r.integer(a[2]);
    const int32_t flags =
        (r.truth(a[3]) ? GG_GATE_RENORM : 0) | (type == F32 ? GG_GATE_LOGITS_F32 : 0);
    const float scale = r.real(a[4]);
    if (!r.ok || k < 1 || k > GG_MAX_EXPERTS || E > INT32_MAX ||
        (score != GG_GATE_SOFTMAX && score != GG_GATE_SIGMOID))
      return false;
    const void* bias = r.optional(a[5], F32, {E});
    const void* num = r.optional(a[6], I32, {1});
    void* ids = r.sized(a[7], I32, {T, k});
    void* w = r.sized(a[8], F32, {T, k});
    int32_t* status = r.status(a[9]);
    const cudaStream_t stream = r.stream(a[10]);
    if (!r.ok) return false;
    *s = entry<decltype(gg_gate_topk)>(GATE)(
        x->data_ptr(), T, (int32_t)E, (int32_t)k, static_cast<const float*>(bias),
        (int32_t)score, flags, scale, static_cast<const int32_t*>(num),
        static_cast<int32_t*>(ids), static_cast<float*>(w), status, stream);
    return true;
  });
}

// logits, topk_ids, dweights, dlogits, score, renorm, scale, status, stream
PyObject* gate_topk_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded<9>(GATE_BACKWARD, args, nargs, [](Reader& r, PyObject* const* a, gg_status* s) {
    if (!THPVariable_CheckExact(a[0])) return false;
    const ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
    if (type != BF16 && type != F32) return false;
    const Tensor* x = r.tensor(a[0], type, 2);
    const Tensor* ids = r.tensor(a[1], I32, 2);
    if (x == nullptr || ids == nullptr) return false;
    const int64_t T = x->size(0), E = x->size(1), k = ids->size(1), score = r.integer(a[4]);
    const int32_t flags =
        (r.truth(a[5]) ? GG_GATE_RENORM : 0) | (type == F32 ? GG_GATE_LOGITS_F32 : 0);
    const float scale = r.real(a[6]);
    if (!r.ok || ids->size(0) != T || k > GG_MAX_EXPERTS || E > INT32_MAX ||
        (score != GG_GATE_SOFTMAX && score != GG_GATE_SIGMOID))
      return false;
    const void* dw = r.sized(a[2], F32, {T, k});
    void* dx = r.sized(a[3], type, {T, E});
    int32_t* status = r.status(a[7]);
    const cudaStream_t stream = r.stream(a[8]);
    if (!r.ok) return false;
    *s = entry<decltype(gg_gate_topk_backward)>(GATE_BACKWARD)(
        x->data_ptr(), T, (int32_t)E, (int32_t)k, (int32_t)score, flags, scale,
        static_cast<const int32_t*>(ids->data_ptr()), static_cast<const float*>(dw), dx, status,
        stream);
    return true;
  });
}

// Tokens of row_of with k entries each; false when it does not hold them.
bool tokens(Reader& r, PyObject* row_of, PyObject* slots, const Tensor** rows, int64_t* T,
            int64_t* k) {
  *rows = r.tensor(row_of, I32, 1);
  *k = r.integer(slots);
  if (!r.ok || *k < 1 || *k > INT32_MAX || (*rows)->numel() % *k != 0) return false;
  *T = (*rows)->numel() / *k;
  return true;
}

// Y, row_of, k, out, weights, residual, status, stream
PyObject* unroute(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded<8>(UNROUTE, args, nargs, [](Reader& r, PyObject* const* a, gg_status* s) {
    const Tensor *Y = r.tensor(a[0], BF16, 2), *rows;
    int64_t T, k;
    if (Y == nullptr || !tokens(r, a[1], a[2], &rows, &T, &k)) return false;
    const int64_t N = Y->size(1);
    void* out = r.sized(a[3], BF16, {T, N});
    const void* w = r.optional(a[4], F32, {T, k});
    const void* res = r.optional(a[5], BF16, {T, N});
    int32_t* status = r.status(a[6]);
    const cudaStream_t stream = r.stream(a[7]);
    if (!r.ok) return false;
    *s = entry<decltype(gg_unroute)>(UNROUTE)(
        Y->data_ptr(), Y->size(0), static_cast<const int32_t*>(rows->data_ptr()),
        static_cast<const float*>(w), res, T, (int32_t)k, N, out, status, stream);
    return true;
  });
}

// dout, row_of, k, dY, Y, weights, dweights, offs, zero_tail, status, stream
PyObject* unroute_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded<11>(
      UNROUTE_BACKWARD, args, nargs, [](Reader& r, PyObject* const* a, gg_status* s) {
        const Tensor *d = r.tensor(a[0], BF16, 2), *rows;
        int64_t T, k;
        if (d == nullptr || !tokens(r, a[1], a[2], &rows, &T, &k)) return false;
        const int64_t N = d->size(1);
        const bool zero = r.truth(a[8]);
        PyObject* first = a[3] != Py_None ? a[3] : a[4];
        if (d->size(0) != T || first == Py_None || (a[3] == Py_None && a[6] == Py_None) ||
            (a[6] != Py_None && a[4] == Py_None) || (zero && a[7] == Py_None))
          return false;
        const Tensor* packed = r.tensor(first, BF16, 2);
        if (packed == nullptr) return false;
        const int64_t R = packed->size(0);
        void* dY = r.optional(a[3], BF16, {R, N});
        const void* Y = r.optional(a[4], BF16, {R, N});
        const void* w = r.optional(a[5], F32, {T, k});
        void* dw = r.optional(a[6], F32, {T, k});
        const int32_t* used = r.used(a[7]);
        int32_t* status = r.status(a[9]);
        const cudaStream_t stream = r.stream(a[10]);
        if (!r.ok) return false;
        *s = entry<decltype(gg_unroute_backward)>(UNROUTE_BACKWARD)(
            d->data_ptr(), Y, R, static_cast<const int32_t*>(rows->data_ptr()),
            static_cast<const float*>(w), T, (int32_t)k, N, used, zero ? GG_FLAG_ZERO_TAIL : 0,
            dY, static_cast<float*>(dw), status, stream);
        return true;
      });
}

// Rows of SiLU-and-mul: by row, or by assignment. `first` stands in for an empty row_of.
struct Rows {
  const int32_t* used;
  const int32_t* row_of = nullptr;
  int64_t n_assign = 0, n;
  const float* weights;
  int32_t flags;
  bool read(Reader& r, const Tensor& first, PyObject* offs, PyObject* rows, PyObject* w,
            PyObject* concat, PyObject* zero_tail) {
    const bool zero = r.truth(zero_tail);
    if (zero && offs == Py_None) return false;
    used = r.used(offs);
    n = first.size(0);
    if (rows != Py_None) {
      const Tensor* t = r.tensor(rows, I32, 1);
      if (t == nullptr) return false;
      n = n_assign = t->numel();
      row_of = static_cast<const int32_t*>(n > 0 ? t->data_ptr() : first.data_ptr());
    }
    weights = r.values(w, n);
    flags = (zero ? GG_FLAG_ZERO_TAIL : 0) | (r.truth(concat) ? GG_FLAG_GATE_UP_CONCAT : 0);
    return r.ok;
  }
};

// H, act, offs, row_of, weights, gate_up_concat, zero_tail, H8, H8_scale, status, stream
PyObject* silu_mul(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded<11>(SILU, args, nargs, [](Reader& r, PyObject* const* a, gg_status* s) {
    const Tensor* H = r.tensor(a[0], BF16, 2);
    Rows rows;
    if (H == nullptr || (a[7] == Py_None) != (a[8] == Py_None) ||
        !rows.read(r, *H, a[2], a[3], a[4], a[5], a[6]))
      return false;
    const int64_t R = H->size(0), N = H->size(1);
    void* act = r.sized(a[1], BF16, {R, N / 2});
    void* H8 = r.optional(a[7], E4M3, {R, N});
    void* scale = r.optional(a[8], E8M0, {R, 2 * blocks(N / 2)});
    int32_t* status = r.status(a[9]);
    const cudaStream_t stream = r.stream(a[10]);
    if (!r.ok) return false;
    *s = entry<decltype(gg_silu_mul)>(SILU)(H->data_ptr(), R, N, rows.used, rows.row_of,
                                            rows.n_assign, rows.weights, rows.flags, act, H8,
                                            scale, status, stream);
    return true;
  });
}

// dact, dH, H, H8, H8_scale, offs, row_of, weights, act, dweights, gate_up_concat, zero_tail,
// status, stream
PyObject* silu_mul_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded<14>(SILU_BACKWARD, args, nargs, [](Reader& r, PyObject* const* a, gg_status* s) {
    const Tensor* d = r.tensor(a[0], BF16, 2);
    Rows rows;
    if (d == nullptr || (a[2] == Py_None) == (a[3] == Py_None) ||
        (a[3] == Py_None) != (a[4] == Py_None) ||
        !rows.read(r, *d, a[5], a[6], a[7], a[10], a[11]))
      return false;
    const int64_t R = d->size(0), half = d->size(1), N = 2 * half;
    void* dH = r.sized(a[1], BF16, {R, N});
    const void* H = r.optional(a[2], BF16, {R, N});
    const void* H8 = r.optional(a[3], E4M3, {R, N});
    const void* scale = r.optional(a[4], E8M0, {R, 2 * blocks(half)});
    void* act = r.optional(a[8], BF16, {R, half});
    float* dw = r.values(a[9], rows.n);
    int32_t* status = r.status(a[12]);
    const cudaStream_t stream = r.stream(a[13]);
    if (!r.ok) return false;
    *s = entry<decltype(gg_silu_mul_backward)>(SILU_BACKWARD)(
        d->data_ptr(), H, H8, scale, R, N, rows.used, rows.row_of, rows.n_assign, rows.weights,
        rows.flags, dH, act, dw, status, stream);
    return true;
  });
}

// X, X8, scale, offs, status, stream
PyObject* pack8(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded<6>(PACK, args, nargs, [](Reader& r, PyObject* const* a, gg_status* s) {
    const Tensor* X = r.tensor(a[0], BF16, 2);
    if (X == nullptr) return false;
    const int64_t R = X->size(0), C = X->size(1);
    void* X8 = r.sized(a[1], E4M3, {R, C});
    void* scale = r.sized(a[2], E8M0, {R, blocks(C)});
    const int32_t* used = r.used(a[3]);
    int32_t* status = r.status(a[4]);
    const cudaStream_t stream = r.stream(a[5]);
    if (!r.ok) return false;
    *s = entry<decltype(gg_pack8)>(PACK)(X->data_ptr(), R, C, used, X8, scale, status, stream);
    return true;
  });
}

// X8, scale, X, offs, zero_tail, status, stream
PyObject* unpack8(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded<7>(UNPACK, args, nargs, [](Reader& r, PyObject* const* a, gg_status* s) {
    const Tensor* X8 = r.tensor(a[0], E4M3, 2);
    if (X8 == nullptr) return false;
    const int64_t R = X8->size(0), C = X8->size(1);
    const void* scale = r.sized(a[1], E8M0, {R, blocks(C)});
    void* X = r.sized(a[2], BF16, {R, C});
    const bool zero = r.truth(a[4]);
    if (zero && a[3] == Py_None) return false;
    const int32_t* used = r.used(a[3]);
    int32_t* status = r.status(a[5]);
    const cudaStream_t stream = r.stream(a[6]);
    if (!r.ok) return false;
    *s = entry<decltype(gg_unpack8)>(UNPACK)(X8->data_ptr(), scale, R, C, used,
                                             zero ? GG_FLAG_ZERO_TAIL : 0, X, status, stream);
    return true;
  });
}

// name, address of an entry point of the loaded library
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const char* name = n == 2 ? PyUnicode_AsUTF8(a[0]) : nullptr;
  void* p = name != nullptr ? PyLong_AsVoidPtr(a[1]) : nullptr;
  if (PyErr_Occurred()) return nullptr;
  for (Entry& e : g_entries)
    if (name != nullptr && strcmp(e.name, name) == 0) {
      e.address = p;
      Py_RETURN_NONE;
    }
  PyErr_SetString(PyExc_ValueError, "bind(name, address) of an entry point of gg.h");
  return nullptr;
}

#define GG_METHOD(f) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr }
PyMethodDef g_methods[] = {GG_METHOD(bind),
                           GG_METHOD(gate_topk),
                           GG_METHOD(gate_topk_backward),
                           GG_METHOD(unroute),
                           GG_METHOD(unroute_backward),
                           GG_METHOD(silu_mul),
                           GG_METHOD(silu_mul_backward),
                           GG_METHOD(pack8),
                           GG_METHOD(unpack8),
                           {nullptr, nullptr, 0, nullptr}};
// GG_MODULE: the module's name, which the build makes of the torch it is compiled against
#define GG_NAME2(prefix, name) prefix##name
#define GG_NAME(prefix, name) GG_NAME2(prefix, name)
#define GG_TEXT2(name) #name
#define GG_TEXT(name) GG_TEXT2(name)
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, GG_TEXT(GG_MODULE), nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC GG_NAME(PyInit_, GG_MODULE)() { return PyModule_Create(&g_module); }
