// A shorter way into the C ABI for calls whose host time counts (the operators over
// paged caches): what __init__.py checks and passes on through ctypes, 6 to 9 us of a
// call, takes 1 us here.
//
// Each function looks at the arguments as __init__.py does. Where all is as it should
// be, on the current device, it allocates what the caller left out, calls the library
// and gives the result back: a tensor, True, or the library's status where that is not
// 0. Anything else, wrong arguments among it, gives None: __init__.py then goes its own
// way, which says what is wrong. Nothing here throws into Python or keeps a reference.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "rope.h"

namespace {

decltype(&rope_apply_qkv_paged) g_append = nullptr;
decltype(&kv_attention_paged) g_attention = nullptr;
decltype(&kv_attention_paged_workspace) g_workspace = nullptr;
decltype(&kv_keep_paged) g_keep = nullptr;

struct Decline {};  // the arguments are for __init__.py

// An argument that is a tensor, or None.
struct Arg {
  const at::Tensor* t;
  explicit Arg(PyObject* o) : t(nullptr) {
    if (o == Py_None) return;
    if (!THPVariable_Check(o)) throw Decline();
    t = &THPVariable_Unpack(o);
  }
  explicit operator bool() const { return t != nullptr; }
  const at::Tensor& operator*() const { return *t; }
  void* at() const { return t ? t->data_ptr() : nullptr; }
};

int64_t whole(PyObject* o) {
  const long long v = PyLong_Check(o) ? PyLong_AsLongLong(o) : -1;
  if (!PyLong_Check(o) || (v == -1 && PyErr_Occurred())) throw Decline();
  return v;
}
int32_t whole32(PyObject* o) {
  const int64_t v = whole(o);
  if (v != (int32_t)v) throw Decline();
  return (int32_t)v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Decline();
  return v;
}

rope_dtype code_of(at::ScalarType t) {
  if (t == at::kHalf) return ROPE_F16;
  if (t == at::kBFloat16) return ROPE_BF16;
  if (t == at::kFloat) return ROPE_F32;
  throw Decline();
}

void need(bool ok) {
  if (!ok) throw Decline();
}
void fits(const at::Tensor& t, int index, at::ScalarType type, at::IntArrayRef shape) {
  need(t.layout() == at::kStrided && t.is_cuda() && t.get_device() == index && t.scalar_type() == type &&
       t.sizes() == shape && t.is_contiguous());
}

// The batch that all calls describe alike.
struct Pages {
  int64_t P, N, ps, H, stride, B, wide;
  at::ScalarType type;
  Pages(const at::Tensor& like, int index, const Arg& k, const Arg& v, const Arg& table, const Arg& past) {
    type = like.scalar_type();
    need(k && v && table && past && (*k).dim() == 4 && (*table).dim() == 2);
    const auto s = (*k).sizes();
    P = s[0], N = s[1], ps = s[2], H = s[3];
    B = (*table).size(0), wide = (*table).size(1);
    fits(*k, index, type, s);
    fits(*v, index, type, s);
    fits(*table, index, at::kInt, (*table).sizes());
    fits(*past, index, at::kInt, {B});
    stride = N * ps * H;
  }
};

// (tokens, hidden) of a query with or without starts; its leading sizes in lead.
int64_t tokens_of(const at::Tensor& q, int index, const Arg& starts, int64_t B, int64_t* hidden) {
  if (!starts) {
    need(q.dim() == 3 && q.size(0) == B);
    *hidden = q.size(2);
    return B * q.size(1);
  }
  need(q.dim() == 2);
  fits(*starts, index, at::kInt, {B + 1});
  *hidden = q.size(1);
  return q.size(0);
}

template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Decline&) {
  } catch (const std::exception&) {  // (an allocation that failed: __init__.py's raises)
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

PyObject* result(rope_status st, const at::Tensor& out) {
  return st == ROPE_OK ? THPVariable_Wrap(out) : PyLong_FromLong(st);
}

// append(device, stream, query, cos, sin, positions, num_heads, kv_num_heads, k_pages, v_pages, table, past, starts,
//        key, value, interleaved, rotary_dim, q_out, status, q_weight, k_weight, epsilon)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 22 && g_append);
    const int index = whole32(a[0]);
    const Arg q(a[2]), cos(a[3]), sin(a[4]), pos(a[5]), k(a[8]), v(a[9]), table(a[10]), past(a[11]), starts(a[12]),
        key(a[13]), value(a[14]), out(a[17]), status(a[18]), qw(a[19]), kw(a[20]);
    need(q && cos && sin);
    const Pages g(*q, index, k, v, table, past);
    const int32_t nq = whole32(a[6]), nkv = whole32(a[7]), rd = whole32(a[16]);
    const bool packed = !key && !value;
    int64_t hidden;
    const int64_t tokens = tokens_of(*q, index, starts, g.B, &hidden);
    need(nkv == g.N && hidden == (nq + (packed ? 2 * (int64_t)nkv : 0)) * g.H && (*cos).dim() == 2);
    fits(*q, index, g.type, (*q).sizes());
    const int64_t rows = (*cos).size(0);
    fits(*cos, index, g.type, {rows, (rd ? rd : g.H) / 2});
    fits(*sin, index, g.type, {rows, (rd ? rd : g.H) / 2});
    c10::SmallVector<int64_t, 3> shape((*q).sizes().begin(), (*q).sizes().end());
    if (!packed) {
      need(key && value);
      shape.back() = nkv * g.H;
      fits(*key, index, g.type, shape);
      fits(*value, index, g.type, shape);
    }
    if (pos) fits(*pos, index, at::kLong, (*q).sizes().slice(0, shape.size() - 1));
    if (qw || kw) {
      need(qw && kw);
      fits(*qw, index, g.type, {g.H});
      fits(*kw, index, g.type, {g.H});
    }
    if (status) fits(*status, index, at::kInt, (*status).sizes());
    shape.back() = nq * g.H;
    if (out) fits(*out, index, g.type, shape);
    const at::Tensor y = out ? *out : at::empty(shape, (*q).options());
    return result(g_append(code_of(g.type), g.B, tokens, nq, nkv, g.H, q.at(), key.at(), value.at(), qw.at(), kw.at(),
                           (float)real(a[21]), cos.at(), sin.at(), rows, (const int64_t*)pos.at(), (const int32_t*)past.at(),
                           (const int32_t*)starts.at(), (const int32_t*)table.at(), g.wide, whole32(a[15]), rd, y.data_ptr(),
                           k.at(), v.at(), g.P, g.ps, g.stride, (int32_t*)status.at(), (rope_stream_t)whole(a[1])),
                  y);
  });
}

// attention(device, stream, query, k_pages, v_pages, table, past, num_heads, starts, max_query_len, scale, softcap,
//           window, slopes, masks, out, status, workspace)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 18 && g_attention && g_workspace);
    const int index = whole32(a[0]);
    const Arg q(a[2]), k(a[3]), v(a[4]), table(a[5]), past(a[6]), starts(a[8]), slopes(a[13]), masks(a[14]), out(a[15]),
        status(a[16]), ws(a[17]);
    need(bool(q));
    const Pages g(*q, index, k, v, table, past);
    const int32_t nq = whole32(a[7]);
    int64_t hidden;
    const int64_t tokens = tokens_of(*q, index, starts, g.B, &hidden);
    need(hidden == nq * g.H && nq > 0 && g.N > 0);
    fits(*q, index, g.type, (*q).sizes());
    const int64_t all = starts ? tokens : (*q).size(1);
    int64_t most = a[9] == Py_None ? all : whole(a[9]);
    need(starts || most == all);
    if (most > all) most = all;
    if (slopes) fits(*slopes, index, at::kFloat, {nq});
    if (masks) fits(*masks, index, at::kLong, (*q).sizes().slice(0, (*q).dim() - 1));
    if (out) fits(*out, index, g.type, (*q).sizes());
    if (status) fits(*status, index, at::kInt, (*status).sizes());
    if (ws) fits(*ws, index, at::kByte, (*ws).sizes());
    const double scale = a[10] == Py_None ? 1.0 / std::sqrt((double)(g.H > 1 ? g.H : 1)) : real(a[10]);
    const rope_dtype code = code_of(g.type);
    const at::Tensor y = out ? *out : at::empty((*q).sizes(), (*q).options());
    at::Tensor work;
    if (!ws) {
      const int64_t bytes = g_workspace(code, g.B, tokens, most, nq, (int32_t)g.N, g.H, g.ps, g.wide);
      if (bytes > 0) work = at::empty({bytes}, (*q).options().dtype(at::kByte));
    } else {
      work = *ws;
    }
    return result(g_attention(code, g.B, tokens, most, nq, (int32_t)g.N, g.H, q.at(), k.at(), v.at(), g.P, g.ps, g.stride,
                              (const int32_t*)table.at(), g.wide, (const int32_t*)past.at(), (const int32_t*)starts.at(),
                              (float)scale, (float)real(a[11]), whole(a[12]), (const float*)slopes.at(),
                              (const int64_t*)masks.at(), y.data_ptr(), (int32_t*)status.at(),
                              work.defined() ? work.data_ptr() : nullptr, work.defined() ? work.numel() : 0,
                              (rope_stream_t)whole(a[1])),
                  y);
  });
}

// keep(device, stream, k_pages, v_pages, table, past, kept, kept_lens, status)
PyObject* keep(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 9 && g_keep);
    const int index = whole32(a[0]);
    const Arg k(a[2]), v(a[3]), table(a[4]), past(a[5]), kept(a[6]), lens(a[7]), status(a[8]);
    need(k && kept && lens && (*kept).dim() == 2);
    const Pages g(*k, index, k, v, table, past);
    const int64_t most = (*kept).size(1);
    fits(*kept, index, at::kInt, {g.B, most});
    fits(*lens, index, at::kInt, {g.B});
    if (status) fits(*status, index, at::kInt, (*status).sizes());
    const rope_status st =
        g_keep(code_of(g.type), g.B, (int32_t)g.N, g.H, k.at(), v.at(), g.P, g.ps, g.stride, (const int32_t*)table.at(), g.wide,
               (const int32_t*)past.at(), (const int32_t*)kept.at(), most, (const int32_t*)lens.at(), (int32_t*)status.at(),
               (rope_stream_t)whole(a[1]));
    if (st != ROPE_OK) return PyLong_FromLong(st);
    Py_RETURN_TRUE;
  });
}

// bind(addresses of rope_apply_qkv_paged, kv_attention_paged, kv_attention_paged_workspace, kv_keep_paged)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 4);
    g_append = (decltype(g_append))whole(a[0]);
    g_attention = (decltype(g_attention))whole(a[1]);
    g_workspace = (decltype(g_workspace))whole(a[2]);
    g_keep = (decltype(g_keep))whole(a[3]);
    Py_RETURN_TRUE;
  });
}

PyMethodDef methods[] = {{"append", (PyCFunction)(void*)append, METH_FASTCALL, nullptr},
                         {"attention", (PyCFunction)(void*)attention, METH_FASTCALL, nullptr},
                         {"keep", (PyCFunction)(void*)keep, METH_FASTCALL, nullptr},
                         {"bind", (PyCFunction)(void*)bind, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__binding() { return PyModule_Create(&module); }
