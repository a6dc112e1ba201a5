// CPython binding of the residual norm, the paged cache and the attention: reads sizes, strides and pointers out of
// the tensors, checks what the C entry points cannot see (types, shapes, layouts, devices) and calls them. In C++ because
// the same checks in Python take longer than the smallest of these calls run on the GPU. The entry points' addresses are
// given at start-up, so this module serves whichever build of the library is loaded.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>
#include <string>

#include "../../include/sffn.h"

namespace {

decltype(&sffn_kv_write) p_write = nullptr;
decltype(&sffn_kv_read) p_read = nullptr;
decltype(&sffn_attn) p_attn = nullptr;
decltype(&sffn_add_rmsnorm) p_norm = nullptr;

struct Bad : std::runtime_error {
  using std::runtime_error::runtime_error;
};
[[noreturn]] void bad(const char* where, const char* what) { throw Bad(std::string(where) + ": " + what); }

const at::Tensor& tensor(PyObject* o, const char* where, const char* name) {
  if (!THPVariable_Check(o)) bad(where, (std::string(name) + " is not a tensor").c_str());
  return THPVariable_Unpack(o);
}
const at::Tensor* maybe(PyObject* o, const char* where, const char* name) {
  return o == Py_None ? nullptr : &tensor(o, where, name);
}

constexpr unsigned F32 = 1, F16 = 2, BF16 = 4, I8 = 8, E4M3 = 16;
int type(const at::Tensor& t, unsigned allowed, const char* where, const char* name) {
  int n = -1;
  switch (t.scalar_type()) {
    case at::kFloat: n = SFFN_F32; break;
    case at::kHalf: n = SFFN_F16; break;
    case at::kBFloat16: n = SFFN_BF16; break;
    case at::kChar: n = SFFN_I8; break;
    case at::kFloat8_e4m3fn: n = SFFN_E4M3; break;
    default: break;
  }
  if (n < 0 || !(allowed >> n & 1)) bad(where, (std::string(name) + ": this type is not supported here").c_str());
  return n;
}
void same_device(const at::Tensor& ref, const at::Tensor& t, const char* where) {
  if (t.device() != ref.device()) bad(where, "the tensors are on different devices");
}

// elements between the tokens of t [T, heads, d], whose tokens are dense
int64_t rows(const at::Tensor& t, int64_t heads, int64_t d, const char* where, const char* name) {
  if (t.dim() != 3 || t.size(1) != heads || t.size(2) != d)
    bad(where, (std::string(name) + " is not [tokens, " + std::to_string(heads) + ", " + std::to_string(d) + "]").c_str());
  if (t.size(0) && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d)))
    bad(where, (std::string(name) + ": the heads of a token must be dense").c_str());
  return t.size(0) > 1 ? t.stride(0) : heads * d;
}
int64_t mat(const at::Tensor& t, int64_t T, int64_t D, const char* where, const char* name) {
  if (t.dim() != 2 || t.size(0) != T || t.size(1) != D || (T && t.stride(1) != 1))
    bad(where, (std::string(name) + " is not [" + std::to_string(T) + ", " + std::to_string(D) + "] with dense rows").c_str());
  return T > 1 ? t.stride(0) : D;
}

int as_int(int64_t v, const char* where) {
  if (v < 0 || v > 2147483647) bad(where, "a size does not fit 32 bits");
  return (int)v;
}

struct Cache {
  sffn_kv c;
  const at::Tensor* K;
};
Cache cache(PyObject* kv, const char* where) {
  const Py_ssize_t n = PyTuple_Check(kv) ? PyTuple_GET_SIZE(kv) : -1;
  if (n != 2 && n != 4) bad(where, "the cache is a tuple (K, V) or (K, V, K_scale, V_scale)");
  const at::Tensor &K = tensor(PyTuple_GET_ITEM(kv, 0), where, "K"), &V = tensor(PyTuple_GET_ITEM(kv, 1), where, "V");
  const int ty = type(K, F16 | BF16 | I8 | E4M3, where, "K");
  if (K.dim() != 4 || K.sizes() != V.sizes() || V.scalar_type() != K.scalar_type() || !K.is_contiguous() || !V.is_contiguous())
    bad(where, "K and V are contiguous [pages, heads, page, head size] of one type");
  same_device(K, V, where);
  Cache r{{K.data_ptr(), V.data_ptr(), nullptr, nullptr, ty, as_int(K.size(0), where), as_int(K.size(2), where),
           as_int(K.size(1), where), as_int(K.size(3), where)}, &K};
  if (ty >= SFFN_I8) {
    for (int i = 2; i < 4; ++i) {
      const at::Tensor* s = n == 4 ? maybe(PyTuple_GET_ITEM(kv, i), where, "scale") : nullptr;
      if (!s || s->scalar_type() != at::kFloat || s->sizes() != K.sizes().slice(0, 3) || !s->is_contiguous())
        bad(where, "an 8-bit cache needs contiguous fp32 scales [pages, heads, page]");
      same_device(K, *s, where);
      (i == 2 ? r.c.k_scale : r.c.v_scale) = (float*)s->data_ptr();
    }
  }
  return r;
}

sffn_seqs seqs(PyObject* ocu, PyObject* ol, PyObject* ot, int64_t T, const at::Tensor& ref, const char* where) {
  const at::Tensor &cu = tensor(ocu, where, "cu"), &len = tensor(ol, where, "kv_len"), &tab = tensor(ot, where, "table");
  if (cu.scalar_type() != at::kInt || len.scalar_type() != at::kInt || tab.scalar_type() != at::kInt)
    bad(where, "cu, kv_len and table are int32");
  if (cu.dim() != 1 || len.dim() != 1 || tab.dim() != 2 || cu.size(0) != len.size(0) + 1 || tab.size(0) != len.size(0))
    bad(where, "need cu [S + 1], kv_len [S], table [S, max_pages]");
  const int64_t S = len.size(0), cols = tab.size(1);
  if (!cu.is_contiguous() || !len.is_contiguous() || (cols > 1 && tab.stride(1) != 1))
    bad(where, "cu, kv_len and the rows of table must be dense");
  same_device(ref, cu, where);
  same_device(ref, len, where);
  same_device(ref, tab, where);
  return {(const int32_t*)cu.data_ptr(), (const int32_t*)len.data_ptr(), (const int32_t*)tab.data_ptr(), as_int(S, where),
          as_int(T, where), as_int(cols, where), as_int(S > 1 ? tab.stride(0) : cols, where)};
}

long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Bad("");
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Bad("");
  return v;
}
int int_of(PyObject* o) {              // clamped: the entry points turn both ends away or treat them as "very large"
  const long v = integer(o);
  return v > 2147483647L ? 2147483647 : v < -2147483647L ? -2147483647 : (int)v;
}

// Work goes to the given stream, or to torch's current one of the tensors' device; that device is current meanwhile.
template <class F>
PyObject* call(const at::Tensor& ref, PyObject* stream, const char* where, F&& f) {
  if (!ref.device().is_cuda()) bad(where, "the tensors must be on the GPU");
  const int dev = ref.device().index();
  void* st = stream == Py_None ? (void*)c10::hip::getCurrentHIPStream(dev).stream() : PyLong_AsVoidPtr(stream);
  if (PyErr_Occurred()) throw Bad("");
  const int now = c10::hip::current_device();
  if (now != dev) c10::hip::set_device(dev);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f(st);
  Py_END_ALLOW_THREADS
  if (now != dev) c10::hip::set_device(now);
  return PyLong_FromLong(rc);
}

template <class F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F&& f) {
  try {
    if (have != want) throw Bad("wrong number of arguments");
    return f();
  } catch (const Bad& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (k, v, kv, cu, kv_len, table, stream)
template <bool WRITE>
PyObject* move(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const char* where = WRITE ? "sffn_kv_write" : "sffn_kv_read";
    const Cache c = cache(a[2], where);
    const at::Tensor &k = tensor(a[0], where, "k"), &v = tensor(a[1], where, "v");
    const int ty = type(k, F16 | BF16, where, "k");
    if (v.scalar_type() != k.scalar_type() || v.sizes() != k.sizes()) bad(where, "k and v differ in type or shape");
    const int64_t lk = rows(k, c.c.n_kv_heads, c.c.head_dim, where, "k"), lv = rows(v, c.c.n_kv_heads, c.c.head_dim, where, "v");
    same_device(*c.K, k, where);
    same_device(*c.K, v, where);
    const sffn_seqs q = seqs(a[3], a[4], a[5], k.size(0), *c.K, where);
    return call(*c.K, a[6], where, [&](void* st) {
      return WRITE ? p_write(c.c, q, ty, k.data_ptr(), lk, v.data_ptr(), lv, st)
                   : p_read(c.c, q, ty, k.data_ptr(), lk, v.data_ptr(), lv, st);
    });
  });
}

// (q, kv, cu, kv_len, table, max_q, max_kv, out, ws, scale, window, sinks, lse, stream)
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&] {
    const char* where = "sffn_attn";
    const Cache c = cache(a[1], where);
    const at::Tensor &q = tensor(a[0], where, "q"), &out = tensor(a[7], where, "out");
    const at::Tensor *ws = maybe(a[8], where, "ws"), *lse = maybe(a[12], where, "lse");
    const int ty = type(q, F16 | BF16, where, "q");
    if (q.dim() != 3 || out.scalar_type() != q.scalar_type() || out.sizes() != q.sizes())
      bad(where, "q and out are [tokens, heads, head size] of one type");
    const int64_t T = q.size(0), Hq = q.size(1);
    const int64_t lq = rows(q, Hq, c.c.head_dim, where, "q"), lo = rows(out, Hq, c.c.head_dim, where, "out");
    if (lse && (lse->scalar_type() != at::kFloat || lse->dim() != 2 || lse->size(0) != T || lse->size(1) != Hq || !lse->is_contiguous()))
      bad(where, "lse is contiguous fp32 [tokens, heads]");
    if (ws && !ws->is_contiguous()) bad(where, "the workspace must be contiguous");
    same_device(*c.K, q, where);
    same_device(*c.K, out, where);
    if (lse) same_device(*c.K, *lse, where);
    if (ws) same_device(*c.K, *ws, where);
    const sffn_seqs sq = seqs(a[2], a[3], a[4], T, *c.K, where);
    const int max_q = int_of(a[5]), max_kv = int_of(a[6]), window = int_of(a[10]), sinks = int_of(a[11]);
    const float scale = (float)(a[9] == Py_None ? std::pow((double)c.c.head_dim, -0.5) : number(a[9]));
    const int hq = as_int(Hq, where);
    return call(*c.K, a[13], where, [&](void* st) {
      return p_attn(c.c, sq, ty, q.data_ptr(), lq, hq, max_q, max_kv, scale, window, sinks, out.data_ptr(), lo,
                    lse ? (float*)lse->data_ptr() : nullptr, ws ? ws->data_ptr() : nullptr, ws ? ws->nbytes() : 0, st);
    });
  });
}

// (x, res, w, eps, y, res_out, y_scale, stream)
PyObject* add_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const char* where = "sffn_add_rmsnorm";
    const at::Tensor &x = tensor(a[0], where, "x"), &y = tensor(a[4], where, "y");
    const at::Tensor *res = maybe(a[1], where, "res"), *w = maybe(a[2], where, "w"), *ro = maybe(a[5], where, "res_out"),
                     *ys = maybe(a[6], where, "y_scale");
    if (x.dim() != 2) bad(where, "x is [tokens, D]");
    const int64_t T = x.size(0), D = x.size(1);
    const int xt = type(x, F32 | F16 | BF16, where, "x"), yt = type(y, F32 | F16 | BF16 | I8 | E4M3, where, "y");
    const int rt = res ? type(*res, F32 | F16 | BF16, where, "res") : ro ? type(*ro, F32 | F16 | BF16, where, "res_out") : SFFN_F32;
    if (res && ro && res->scalar_type() != ro->scalar_type()) bad(where, "res and res_out differ in type");
    const int64_t lx = mat(x, T, D, where, "x"), ly = mat(y, T, D, where, "y"), lr = res ? mat(*res, T, D, where, "res") : 0,
                  lro = ro ? mat(*ro, T, D, where, "res_out") : 0;
    if (w && (w->scalar_type() != at::kFloat || w->dim() != 1 || w->size(0) != D || !w->is_contiguous()))
      bad(where, "w is contiguous fp32 [D]");
    if (yt >= SFFN_I8 && (!ys || ys->scalar_type() != at::kFloat || ys->dim() != 1 || ys->size(0) != T || !ys->is_contiguous()))
      bad(where, "an 8-bit y needs y_scale, contiguous fp32 [tokens]");
    same_device(x, y, where);
    for (const at::Tensor* t : {res, w, ro, ys})
      if (t) same_device(x, *t, where);
    const double eps = number(a[3]);
    const int t32 = as_int(T, where), d32 = as_int(D, where);
    return call(x, a[7], where, [&](void* st) {
      return p_norm(xt, x.data_ptr(), lx, rt, res ? res->data_ptr() : nullptr, lr, w ? (const float*)w->data_ptr() : nullptr, eps,
                    t32, d32, yt, y.data_ptr(), ly, yt >= SFFN_I8 ? (float*)ys->data_ptr() : nullptr,
                    ro ? ro->data_ptr() : nullptr, lro, st);
    });
  });
}

// the entry points' addresses: (kv_write, kv_read, attn, add_rmsnorm)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    void* p[4];
    for (int i = 0; i < 4; ++i) {
      p[i] = PyLong_AsVoidPtr(a[i]);
      if (!p[i]) throw Bad("bind: no address");
    }
    p_write = (decltype(p_write))p[0];
    p_read = (decltype(p_read))p[1];
    p_attn = (decltype(p_attn))p[2];
    p_norm = (decltype(p_norm))p[3];
    Py_RETURN_NONE;
  });
}

#define M(name, fn) {name, (PyCFunction)(void (*)(void))(fn), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {M("bind", bind), M("kv_write", move<true>), M("kv_read", move<false>), M("attn", attn),
                         M("add_rmsnorm", add_rmsnorm), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) { return PyModule_Create(&module); }
