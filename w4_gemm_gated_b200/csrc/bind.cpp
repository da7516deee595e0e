// Native marshalling of the decoder-step calls: tensors in, C-ABI calls out.
//
// These calls take a few microseconds on the GPU, less than the same checks and
// allocations take in the interpreter (attn_decode: 9.8 us of host time there).
// Nothing is computed here.  The module does not link to the kernel library:
// setup() receives its functions' addresses, so that either build of it (the
// device-check build too) is called through the one that is loaded.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>
#include <optional>

#include "spear.h"

namespace {

struct {
  decltype(&spear_kv_write) kv_write;
  decltype(&spear_kv_read) kv_read;
  decltype(&spear_attn_decode) attn_decode;
  decltype(&spear_block_norm) block_norm;
  PyObject* check;  // raises the error of a status
} g = {};

// An argument that was refused: the Python error is set.
struct Refused {};

[[noreturn]] void refuse(PyObject* type, const char* fmt, const char* what) {
  PyErr_Format(type, fmt, what);
  throw Refused();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", what);
  return THPVariable_Unpack(o);
}

const at::Tensor* optional_tensor(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }

int as_int(int64_t n, const char* what) {
  if (n > INT_MAX) refuse(PyExc_ValueError, "%s is too long", what);
  return static_cast<int>(n);
}

double as_double(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}

int64_t as_long(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

const uint16_t* bf16(const at::Tensor* t) { return t ? static_cast<const uint16_t*>(t->data_ptr()) : nullptr; }
uint16_t* bf16_out(const at::Tensor& t) { return static_cast<uint16_t*>(t.data_ptr()); }

// The device and stream of a call: the current stream of the tensors' device,
// whichever device is current, or the stream given, which the outputs are then
// allocated on and whose use of the tensors the allocator is told (of the cache's,
// which come as an address, by the caller).
struct Where {
  c10::DeviceIndex index;
  std::optional<c10::cuda::CUDAStreamGuard> on;
  std::optional<c10::cuda::CUDAGuard> there;
  std::optional<c10::cuda::CUDAStream> given;

  Where(c10::DeviceIndex i, PyObject* stream) : index(i) {
    if (stream != Py_None) {
      auto number = [&](const char* name) {
        PyObject* v = PyObject_GetAttrString(stream, name);
        if (!v) throw Refused();
        const int64_t n = PyLong_AsLongLong(v);
        Py_DECREF(v);
        if (n == -1 && PyErr_Occurred()) throw Refused();
        return n;
      };
      given = c10::cuda::CUDAStream::unpack3(number("stream_id"), static_cast<c10::DeviceIndex>(number("device_index")),
                                             static_cast<c10::DeviceType>(number("device_type")));
      if (given->device_index() != index) refuse(PyExc_ValueError, "%s must be a stream of the tensors' device", "stream");
      on.emplace(*given);
    } else if (c10::cuda::current_device() != index) {
      there.emplace(index);
    }
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(index).stream(); }
  at::Tensor empty(c10::IntArrayRef shape, c10::IntArrayRef strides) const {
    return at::detail::empty_strided_cuda(
        shape, strides, at::TensorOptions().dtype(at::kBFloat16).device(at::Device(at::kCUDA, index)));
  }
  void uses(std::initializer_list<const at::Tensor*> tensors) const {
    if (given)
      for (const at::Tensor* t : tensors)
        if (t) t->record_stream(*given);
  }
};

void done(int status) {
  if (status == SPEAR_OK) return;
  PyObject* r = PyObject_CallFunction(g.check, "i", status);
  Py_XDECREF(r);
  if (r) refuse(PyExc_RuntimeError, "%s", "the call failed");
  throw Refused();
}

bool here(const at::Tensor& t, c10::DeviceIndex index) { return t.is_cuda() && t.get_device() == index; }

// Elements between the rows of t: n rows of heads x dim bf16 values (2-D or 3-D).
int64_t rows(const at::Tensor& t, c10::DeviceIndex index, int64_t n, int64_t heads, int64_t dim, const char* what,
             PyObject* wrong_type = PyExc_TypeError) {
  if (t.scalar_type() != at::kBFloat16) refuse(wrong_type, "%s must be bf16", what);
  const auto s = t.sizes(), d = t.strides();
  const bool ok = s.size() == 3 ? s[0] == n && s[1] == heads && s[2] == dim && d[2] == 1 && (heads == 1 || d[1] == dim)
                                : s.size() == 2 && s[0] == n && s[1] == heads * dim && d[1] == 1;
  if (!ok) refuse(PyExc_ValueError, "%s must have consecutive n_heads x head_dim values in each of its rows", what);
  if (!here(t, index)) refuse(PyExc_ValueError, "%s must live on the cache's device", what);
  return n > 1 ? d[0] : heads * dim;
}

const int* i32(const at::Tensor& t, c10::DeviceIndex index, int64_t n, const char* what) {
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous() || !here(t, index))
    refuse(PyExc_ValueError, "%s must be contiguous int32 values, one per row, on the cache's device", what);
  return static_cast<const int*>(t.data_ptr());
}

void* workspace(const at::Tensor& t, c10::DeviceIndex index) {
  if (!t.is_contiguous() || !here(t, index))
    refuse(PyExc_ValueError, "%s must be contiguous, on the cache's device", "the workspace");
  return t.data_ptr();
}

int64_t first_size(const at::Tensor& t, const char* what) {
  if (t.dim() < 1) refuse(PyExc_ValueError, "%s must have rows", what);
  return t.size(0);
}

struct Cache {
  const spear_kv_cache* c;
  c10::DeviceIndex index;
  Cache(PyObject* addr, PyObject* device)
      : c(reinterpret_cast<const spear_kv_cache*>(as_long(addr))), index(static_cast<c10::DeviceIndex>(as_long(device))) {}
};

void want(Py_ssize_t n, Py_ssize_t wanted) {
  if (n != wanted) refuse(PyExc_TypeError, "%s", "wrong number of arguments");
}

// kv_write(cache address, device, k, v, slots, ws, stream)
PyObject* kv_write(PyObject*, PyObject* const* a, Py_ssize_t na) {
  HANDLE_TH_ERRORS try {
    want(na, 7);
    const Cache c(a[0], a[1]);
    const at::Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v"), &slots = tensor(a[4], "slots"),
                     &ws = tensor(a[5], "ws");
    const int64_t n = first_size(k, "k");
    const int64_t ld_k = rows(k, c.index, n, c.c->n_heads, c.c->head_dim, "k");
    const int64_t ld_v = rows(v, c.index, n, c.c->n_heads, c.c->head_dim, "v");
    const int* s = i32(slots, c.index, n, "slots");
    void* w = workspace(ws, c.index);
    const Where at(c.index, a[6]);
    at.uses({&k, &v, &slots, &ws});
    done(g.kv_write(c.c, bf16(&k), ld_k, bf16(&v), ld_v, s, as_int(n, "k"), w, ws.nbytes(), at.stream()));
    Py_RETURN_NONE;
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// kv_read(cache address, device, slots, ws, k_out, v_out, stream) -> (k_out, v_out)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t na) {
  HANDLE_TH_ERRORS try {
    want(na, 7);
    const Cache c(a[0], a[1]);
    const at::Tensor &slots = tensor(a[2], "slots"), &ws = tensor(a[3], "ws");
    const int64_t n = first_size(slots, "slots"), heads = c.c->n_heads, dim = c.c->head_dim;
    const int* s = i32(slots, c.index, n, "slots");
    void* w = workspace(ws, c.index);
    const Where at(c.index, a[6]);
    at::Tensor out[2];
    for (int i = 0; i < 2; ++i) {
      const char* what = i ? "v_out" : "k_out";
      if (const at::Tensor* t = optional_tensor(a[4 + i], what)) {
        if (rows(*t, c.index, n, heads, dim, what, PyExc_ValueError) != heads * dim)
          refuse(PyExc_ValueError, "%s must be contiguous", what);
        out[i] = *t;
      } else {
        out[i] = at.empty({n, heads, dim}, {heads * dim, dim, 1});
      }
    }
    at.uses({&slots, &ws, &out[0], &out[1]});
    done(g.kv_read(c.c, s, as_int(n, "slots"), bf16_out(out[0]), bf16_out(out[1]), w, ws.nbytes(), at.stream()));
    PyObject* k = a[4] == Py_None ? THPVariable_Wrap(std::move(out[0])) : Py_NewRef(a[4]);
    PyObject* v = a[5] == Py_None ? THPVariable_Wrap(std::move(out[1])) : Py_NewRef(a[5]);
    PyObject* r = PyTuple_Pack(2, k, v);
    Py_DECREF(k);
    Py_DECREF(v);
    return r;
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// attn_decode(cache address, device, q, page_table, seq_lens, ws, scale, out, lse, stream) -> out
PyObject* attn_decode(PyObject*, PyObject* const* a, Py_ssize_t na) {
  HANDLE_TH_ERRORS try {
    want(na, 10);
    const Cache c(a[0], a[1]);
    const at::Tensor &q = tensor(a[2], "q"), &table = tensor(a[3], "page_table"), &lens = tensor(a[4], "seq_lens"),
                     &ws = tensor(a[5], "ws");
    const int64_t n = first_size(q, "q"), dim = c.c->head_dim;
    if (q.dim() != 2 && q.dim() != 3) refuse(PyExc_ValueError, "%s must be 2-D or 3-D", "q");
    const int64_t heads = q.dim() == 3 ? q.size(1) : q.size(1) / dim;
    const int64_t ld_q = rows(q, c.index, n, heads, dim, "q");
    if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != n ||
        (table.stride(1) != 1 && table.size(1) > 1) || !here(table, c.index))
      refuse(PyExc_ValueError, "%s must be n_seqs x max_pages int32 with consecutive rows, on the cache's device",
             "page_table");
    const int pages = as_int(table.size(1), "page_table");
    const int ld_table = n > 1 ? as_int(table.stride(0), "page_table") : pages;
    const int* l = i32(lens, c.index, n, "seq_lens");
    const at::Tensor* lse = optional_tensor(a[8], "lse");
    if (lse && (lse->scalar_type() != at::kFloat || lse->dim() != 2 || lse->size(0) != n || lse->size(1) != heads ||
                !lse->is_contiguous() || !here(*lse, c.index)))
      refuse(PyExc_ValueError, "%s must be contiguous fp32, n_seqs x n_q_heads, on the cache's device", "lse");
    void* w = workspace(ws, c.index);
    const float scale = a[6] == Py_None ? 1.f / std::sqrt(static_cast<float>(dim)) : static_cast<float>(as_double(a[6]));
    const Where at(c.index, a[9]);
    at::Tensor out;
    int64_t ld_out = heads * dim;
    if (const at::Tensor* t = optional_tensor(a[7], "out")) {
      if (t->sizes() != q.sizes()) refuse(PyExc_ValueError, "%s must have q's shape", "out");
      ld_out = rows(*t, c.index, n, heads, dim, "out");
      out = *t;
    } else if (q.dim() == 3) {
      out = at.empty({n, heads, dim}, {heads * dim, dim, 1});
    } else {
      out = at.empty({n, heads * dim}, {heads * dim, 1});
    }
    at.uses({&q, &out, &table, &lens, lse, &ws});
    done(g.attn_decode(c.c, bf16(&q), ld_q, as_int(n, "q"), as_int(heads, "q"), static_cast<const int*>(table.data_ptr()),
                       pages, ld_table, l, scale, bf16_out(out), ld_out,
                       lse ? static_cast<float*>(lse->data_ptr()) : nullptr, w, ws.nbytes(), at.stream()));
    return a[7] == Py_None ? THPVariable_Wrap(std::move(out)) : Py_NewRef(a[7]);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// A contiguous bf16 tensor of M x K (M < 0: K values) on a device, or absent.
const at::Tensor* plain(PyObject* o, int64_t M, int64_t K, c10::DeviceIndex index, const char* what) {
  const at::Tensor* t = optional_tensor(o, what);
  if (!t) return nullptr;
  const auto s = t->sizes();
  if (t->scalar_type() != at::kBFloat16 || !(M < 0 ? s.size() == 1 && s[0] == K : s.size() == 2 && s[0] == M && s[1] == K) ||
      !t->is_contiguous() || !here(*t, index))
    refuse(PyExc_ValueError, "%s must be contiguous bf16 of x's rows' or columns' number, on x's CUDA device", what);
  return t;
}

// block_norm(x, y, pre, post, gate, residual_scale, block_scale, eps, x_out, h, norm, stream) -> (x_out or x, h or None)
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t na) {
  HANDLE_TH_ERRORS try {
    want(na, 12);
    const at::Tensor& x = tensor(a[0], "x");
    if (x.dim() != 2 || !x.is_cuda()) refuse(PyExc_ValueError, "%s must be M x K on a CUDA device", "x");
    const auto index = static_cast<c10::DeviceIndex>(x.get_device());
    const int64_t M = x.size(0), K = x.size(1);
    plain(a[0], M, K, index, "x");
    const at::Tensor *y = plain(a[1], M, K, index, "y"), *pre = plain(a[2], -1, K, index, "pre_weight"),
                     *post = plain(a[3], -1, K, index, "post_weight"), *gate = optional_tensor(a[4], "gate"),
                     *x_out = plain(a[8], M, K, index, "x_out"), *h = plain(a[9], M, K, index, "h");
    int64_t gate_ld = 0;
    if (gate) {
      const auto s = gate->sizes();
      const bool shape = s.size() == 1 ? s[0] == K : s.size() == 2 && s[1] == K && (s[0] == 1 || s[0] == M);
      if (gate->scalar_type() != at::kBFloat16 || !shape || gate->strides().back() != 1 || !here(*gate, index))
        refuse(PyExc_ValueError, "%s must be bf16, K, 1 x K or M x K, with consecutive rows, on x's device", "gate");
      if (s.size() == 2 && s[0] > 1) gate_ld = gate->stride(0);
    }
    const int norm = PyObject_IsTrue(a[10]);
    if (norm < 0) throw Refused();
    const Where at(index, a[11]);
    at::Tensor made_x, made_h;
    if (!x_out && y) {
      made_x = at.empty({M, K}, {K, 1});
      x_out = &made_x;
    }
    if (!norm) {
      h = nullptr;
    } else if (!h) {
      made_h = at.empty({M, K}, {K, 1});
      h = &made_h;
    }
    at.uses({&x, y, pre, post, gate, x_out, h});
    done(g.block_norm(bf16(&x), bf16(y), as_int(M, "x"), as_int(K, "x"), bf16(post), bf16(gate), gate_ld,
                      static_cast<float>(as_double(a[5])), static_cast<float>(as_double(a[6])), bf16(pre),
                      static_cast<float>(as_double(a[7])), x_out ? bf16_out(*x_out) : nullptr,
                      h ? bf16_out(*h) : nullptr, at.stream()));
    PyObject* rx = made_x.defined() ? THPVariable_Wrap(std::move(made_x)) : Py_NewRef(y ? a[8] : a[0]);
    PyObject* rh = made_h.defined() ? THPVariable_Wrap(std::move(made_h)) : Py_NewRef(norm ? a[9] : Py_None);
    PyObject* r = PyTuple_Pack(2, rx, rh);
    Py_DECREF(rx);
    Py_DECREF(rh);
    return r;
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// setup(kv_write, kv_read, attn_decode, block_norm addresses, check)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t na) {
  HANDLE_TH_ERRORS try {
    want(na, 5);
    g.kv_write = reinterpret_cast<decltype(g.kv_write)>(as_long(a[0]));
    g.kv_read = reinterpret_cast<decltype(g.kv_read)>(as_long(a[1]));
    g.attn_decode = reinterpret_cast<decltype(g.attn_decode)>(as_long(a[2]));
    g.block_norm = reinterpret_cast<decltype(g.block_norm)>(as_long(a[3]));
    Py_XDECREF(g.check);
    g.check = Py_NewRef(a[4]);
    Py_RETURN_NONE;
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(setup), FAST(kv_write), FAST(kv_read), FAST(attn_decode), FAST(block_norm),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "Native marshalling of the decoder-step calls.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
