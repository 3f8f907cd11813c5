// Argument checks, output allocation and call of the layer operators (the
// norms, the conv backward, the single-token step) for the Python package: a
// CPython module over the C ABI of include/ssd.h.  In serving these calls take
// 3 to 8 us on the GPU, less than the same checks and a ctypes call cost in
// Python (10 to 13 us), so here they are native.  Python keeps the signatures,
// the defaults and the device and stream scope; the raw stream handle comes in
// as the last argument of every function.
//
// Every function returns its result, an int (the library's error code, for the
// caller to raise) or raises: ValueError for a shape, device or layout,
// TypeError for a type.  Shapes and types are checked before devices.

#include <Python.h>
#include <dlfcn.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "../../include/ssd.h"

namespace {

// the library's entry points, looked up by bind()
struct Entry {
  decltype(&ssd_add_norm_fwd) add_norm_fwd;
  decltype(&ssd_add_norm_bwd_workspace_size) add_norm_bwd_ws;
  decltype(&ssd_add_norm_bwd) add_norm_bwd;
  decltype(&ssd_gated_norm_fwd) gated_norm_fwd;
  decltype(&ssd_gated_norm_bwd_workspace_size) gated_norm_bwd_ws;
  decltype(&ssd_gated_norm_bwd) gated_norm_bwd;
  decltype(&ssd_conv1d_bwd_workspace_size) conv1d_bwd_ws;
  decltype(&ssd_conv1d_bwd) conv1d_bwd;
  decltype(&ssd_mixer_step) mixer_step;
} E;

struct Refused {
  PyObject* type;
  std::string msg;
};
[[noreturn]] void bad_value(const std::string& m) { throw Refused{PyExc_ValueError, m}; }
[[noreturn]] void bad_type(const std::string& m) { throw Refused{PyExc_TypeError, m}; }

using Shape = at::IntArrayRef;
using Opt = const at::Tensor*;  // null: None

std::string str(Shape s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}
std::string str(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
  }
}
std::string str(const at::Device& d) { return d.str(); }

Opt opt(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& need(PyObject* o, const char* name) {
  if (o == Py_None) bad_type(std::string(name) + " must be a tensor, got None");
  return *opt(o, name);
}
long long as_int(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
  return v;
}
int as_int32(PyObject* o, const char* name) {
  const long long v = as_int(o);
  if (v < -2147483647LL - 1 || v > 2147483647LL) bad_value(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(v);
}
float as_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
  return static_cast<float>(v);
}

// SSD_F32 or SSD_BF16
int code(at::ScalarType t, const char* name) {
  if (t == at::kFloat) return SSD_F32;
  if (t == at::kBFloat16) return SSD_BF16;
  bad_type(std::string(name) + " must be float32 or bfloat16, got " + str(t));
}
at::ScalarType type_of(int c) { return c == SSD_BF16 ? at::kBFloat16 : at::kFloat; }

struct Spec {
  Opt t;
  const char* name;
  Shape shape;
  at::ScalarType type;
  bool strided;  // rows that lead() looks at
};

// Each tensor of exactly its shape and type, contiguous on ref's GPU.
void check(const at::Tensor& ref, std::initializer_list<Spec> specs) {
  for (const Spec& s : specs) {
    if (!s.t) continue;
    if (s.t->sizes() != s.shape)
      bad_value(std::string(s.name) + " has shape " + str(s.t->sizes()) + ", expected " + str(s.shape));
    if (s.t->scalar_type() != s.type)
      bad_type(std::string(s.name) + " must be " + str(s.type) + ", got " + str(s.t->scalar_type()));
  }
  for (const Spec& s : specs) {
    if (!s.t) continue;
    if (!s.t->is_cuda()) bad_value(std::string(s.name) + " must be a GPU tensor");
    if (s.t->device() != ref.device())
      bad_value(std::string(s.name) + " is on " + str(s.t->device()) + ", expected " + str(ref.device()));
    if (!s.strided && !s.t->is_contiguous()) bad_value(std::string(s.name) + " must be contiguous");
  }
}

// Rows of the last axis of a tensor whose leading axes collapse into one
// evenly spaced axis (contiguous, or a column slice of such rows): their
// stride in elements.
long long lead(const at::Tensor& t, const char* name) {
  const int64_t n = t.size(-1);
  if (t.numel() == 0 || t.is_contiguous()) return n > 0 ? n : 1;
  if (n > 1 && t.stride(-1) != 1) bad_value(std::string(name) + " must have a contiguous last dim");
  int64_t ld = -1, span = 0;
  for (int64_t d = t.dim() - 2; d >= 0; --d) {
    if (t.size(d) == 1) continue;
    if (ld < 0)
      ld = t.stride(d);
    else if (t.stride(d) != span)
      bad_value(std::string(name) + ": its rows must be evenly spaced");
    span = t.stride(d) * t.size(d);
  }
  if (ld < 0) return n;
  if (ld < n)
    bad_value(std::string(name) + ": rows " + std::to_string(ld) + " apart overlap, they have " +
              std::to_string(n) + " elements");
  return ld;
}

template <typename T = void>
T* ptr(Opt t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
at::Tensor fresh(Shape s, at::ScalarType t, const at::Tensor& ref) {
  return at::empty(s, at::TensorOptions().dtype(t).device(ref.device()));
}
at::Tensor scratch(Opt given, size_t bytes, const at::Tensor& ref) {
  if (!given) return fresh({static_cast<int64_t>(bytes < 256 ? 256 : bytes)}, at::kByte, ref);
  check(ref, {{given, "workspace", given->sizes(), at::kByte, false}});
  return *given;
}

int rows_of(const at::Tensor& x, const char* name, int& D) {
  if (x.dim() < 1 || x.size(-1) < 1)
    bad_value(std::string(name) + " must have rows of at least one channel, got shape " + str(x.sizes()));
  const int64_t d = x.size(-1), m = x.numel() / d;
  if (d > 2147483647LL || m > 2147483647LL) bad_value(std::string(name) + " has too many rows or channels");
  D = static_cast<int>(d);
  return static_cast<int>(m);
}

PyObject* wrapped(const at::Tensor& t) { return THPVariable_Wrap(t); }
// the caller's own object where an output was given
PyObject* result(PyObject* given, const at::Tensor& t) {
  if (given == Py_None) return wrapped(t);
  Py_INCREF(given);
  return given;
}
void put(PyObject* d, const char* key, PyObject* v) {
  PyDict_SetItemString(d, key, v);
  Py_DECREF(v);
}
PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

// Runs one entry's body: exceptions become Python errors.
template <typename F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F f) {
  if (have != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  if (!E.mixer_step) {
    PyErr_SetString(PyExc_RuntimeError, "the library is not bound");
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused& r) {
    if (r.type) PyErr_SetString(r.type, r.msg.c_str());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
template <typename F>
int without_gil(F f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS rc = f();
  Py_END_ALLOW_THREADS return rc;
}
void* stream_of(PyObject* o) { return reinterpret_cast<void*>(static_cast<uintptr_t>(as_int(o))); }

// x, w, residual, scale, eps, out, out code or -1, residual_out, residual code or -1, stream
PyObject* add_norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor& x = need(a[0], "x");
    const at::Tensor& w = need(a[1], "w");
    Opt residual = opt(a[2], "residual"), scale = opt(a[3], "scale"), out = opt(a[5], "out"), ro = opt(a[7], "residual_out");
    int D, M = rows_of(x, "x", D), oc = as_int32(a[6], "out_dtype"), rc = as_int32(a[8], "res_dtype");
    const int xc = code(x.scalar_type(), "x");
    if (residual) {
      const int c = code(residual->scalar_type(), "residual");
      if (rc >= 0 && rc != c) bad_type("residual is " + str(residual->scalar_type()) + ", res_dtype " + str(type_of(rc)));
      rc = c;
    } else if (rc < 0) {
      rc = ro ? code(ro->scalar_type(), "residual_out") : SSD_F32;
    }
    if (oc < 0) oc = out ? code(out->scalar_type(), "out") : xc;
    const at::ScalarType rt = type_of(rc), ot = type_of(oc);
    const Shape s = x.sizes(), d = s.slice(s.size() - 1);
    check(x, {{&x, "x", s, x.scalar_type(), false}, {scale, "scale", d, at::kFloat, false},
              {residual, "residual", s, rt, false}, {&w, "w", d, at::kFloat, false},
              {ro, "residual_out", s, rt, false}, {out, "out", s, ot, false}});
    const float eps = as_float(a[4]);
    void* st = stream_of(a[9]);
    const at::Tensor o = out ? *out : fresh(s, ot, x), r = ro ? *ro : fresh(s, rt, x);
    const int e = without_gil([&] {
      return E.add_norm_fwd(ptr(&x), ptr<float>(scale), ptr(residual), ptr<float>(&w), eps, ptr(&r), ptr(&o), M, D,
                            xc, rc, oc, st);
    });
    if (e) return PyLong_FromLong(e);
    PyObject* t = PyTuple_New(2);
    PyTuple_SET_ITEM(t, 0, result(a[5], o));
    PyTuple_SET_ITEM(t, 1, result(a[7], r));
    return t;
  });
}

// dout, r, w, dres, scale, x, eps, x code or -1, workspace, stream
PyObject* add_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor& dout = need(a[0], "dout");
    const at::Tensor& r = need(a[1], "r");
    const at::Tensor& w = need(a[2], "w");
    Opt dres = opt(a[3], "dres"), scale = opt(a[4], "scale"), x = opt(a[5], "x"), given = opt(a[8], "workspace");
    int D, M = rows_of(r, "r", D), xc = as_int32(a[7], "x_dtype");
    if (xc < 0) xc = code((x ? *x : dout).scalar_type(), x ? "x" : "dout");
    const int rc = code(r.scalar_type(), "r"), oc = code(dout.scalar_type(), "dout");
    const Shape s = r.sizes(), d = s.slice(s.size() - 1);
    const at::ScalarType xt = type_of(xc);
    check(r, {{&r, "r", s, r.scalar_type(), false}, {&dout, "dout", s, dout.scalar_type(), false},
              {dres, "dres", s, r.scalar_type(), false}, {x, "x", s, xt, false}, {&w, "w", d, at::kFloat, false},
              {scale, "scale", d, at::kFloat, false}});
    const float eps = as_float(a[6]);
    void* st = stream_of(a[9]);
    const at::Tensor dr = fresh(s, r.scalar_type(), r), dx = fresh(s, xt, r), dw = fresh(d, at::kFloat, r);
    const at::Tensor ds = x ? fresh(d, at::kFloat, r) : at::Tensor();
    const at::Tensor ws = scratch(given, E.add_norm_bwd_ws(M, D), r);
    const int e = without_gil([&] {
      return E.add_norm_bwd(ptr(&dout), ptr(dres), ptr(&r), ptr(x), ptr<float>(scale), ptr<float>(&w), eps, ptr(&dr),
                            ptr(&dx), ptr<float>(&dw), x ? ptr<float>(&ds) : nullptr, M, D, xc, rc, oc, ptr(&ws),
                            ws.nbytes(), st);
    });
    if (e) return PyLong_FromLong(e);
    PyObject* t = PyDict_New();
    put(t, "dresidual", wrapped(dr));
    put(t, "dx", wrapped(dx));
    put(t, "dw", wrapped(dw));
    put(t, "dscale", x ? wrapped(ds) : none());
    return t;
  });
}

// y, z, w, groups, eps, before, out, out code or -1, stream
PyObject* gated_norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor& y = need(a[0], "y");
    const at::Tensor& z = need(a[1], "z");
    const at::Tensor& w = need(a[2], "w");
    Opt out = opt(a[6], "out");
    int D, M = rows_of(y, "y", D), oc = as_int32(a[7], "out_dtype");
    const int groups = as_int32(a[3], "groups"), before = as_int32(a[5], "norm_before_gate");
    const int yc = code(y.scalar_type(), "y"), zc = code(z.scalar_type(), "z");
    if (oc < 0) oc = out ? code(out->scalar_type(), "out") : zc;
    const Shape s = y.sizes(), d = s.slice(s.size() - 1);
    check(y, {{&z, "z", s, z.scalar_type(), true}, {&y, "y", s, y.scalar_type(), false}, {&w, "w", d, at::kFloat, false},
              {out, "out", s, type_of(oc), false}});
    const long long ldz = lead(z, "z");
    const float eps = as_float(a[4]);
    void* st = stream_of(a[8]);
    const at::Tensor o = out ? *out : fresh(s, type_of(oc), y);
    const int e = without_gil([&] {
      return E.gated_norm_fwd(ptr(&y), ptr(&z), ldz, ptr<float>(&w), eps, before, ptr(&o), M, D, groups, yc, zc, oc, st);
    });
    return e ? PyLong_FromLong(e) : result(a[6], o);
  });
}

// dout, y, z, w, groups, eps, before, dz, workspace, stream
PyObject* gated_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor& dout = need(a[0], "dout");
    const at::Tensor& y = need(a[1], "y");
    const at::Tensor& z = need(a[2], "z");
    const at::Tensor& w = need(a[3], "w");
    Opt dz = opt(a[7], "dz"), given = opt(a[8], "workspace");
    int D, M = rows_of(y, "y", D);
    const int groups = as_int32(a[4], "groups"), before = as_int32(a[6], "norm_before_gate");
    const int yc = code(y.scalar_type(), "y"), zc = code(z.scalar_type(), "z"), oc = code(dout.scalar_type(), "dout");
    const Shape s = y.sizes(), d = s.slice(s.size() - 1);
    check(y, {{&z, "z", s, z.scalar_type(), true}, {dz, "dz", s, z.scalar_type(), true},
              {&y, "y", s, y.scalar_type(), false}, {&dout, "dout", s, dout.scalar_type(), false},
              {&w, "w", d, at::kFloat, false}});
    const long long ldz = lead(z, "z");
    const float eps = as_float(a[5]);
    void* st = stream_of(a[9]);
    const at::Tensor gz = dz ? *dz : fresh(s, z.scalar_type(), y);
    const long long lddz = lead(gz, "dz");
    const at::Tensor dy = fresh(s, y.scalar_type(), y), dw = fresh(d, at::kFloat, y);
    const at::Tensor ws = scratch(given, E.gated_norm_bwd_ws(M, D, groups), y);
    const int e = without_gil([&] {
      return E.gated_norm_bwd(ptr(&dout), ptr(&y), ptr(&z), ldz, ptr<float>(&w), eps, before, ptr(&dy), ptr(&gz), lddz,
                              ptr<float>(&dw), M, D, groups, yc, zc, oc, ptr(&ws), ws.nbytes(), st);
    });
    if (e) return PyLong_FromLong(e);
    PyObject* t = PyDict_New();
    put(t, "dy", wrapped(dy));
    put(t, "dz", result(a[7], gz));
    put(t, "dw", wrapped(dw));
    return t;
  });
}

void ndim(const at::Tensor& t, const char* name, int64_t n) {
  if (t.dim() != n)
    bad_value(std::string(name) + " must have " + std::to_string(n) + " dimensions, got shape " + str(t.sizes()));
}
int dim32(int64_t v, const char* name) {
  if (v > 2147483647LL) bad_value(std::string(name) + " is too large");
  return static_cast<int>(v);
}

// xbc, w, dx, dB, dC, bias, state_in, dstate_out, act, dxbc, want_dstate_in, workspace, stream
PyObject* conv1d_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const at::Tensor& xbc = need(a[0], "xbc");
    const at::Tensor& w = need(a[1], "w");
    const at::Tensor& dx = need(a[2], "dx");
    const at::Tensor& dB = need(a[3], "dB");
    const at::Tensor& dC = need(a[4], "dC");
    Opt bias = opt(a[5], "bias"), si = opt(a[6], "state_in"), dso = opt(a[7], "dstate_out"), dxbc = opt(a[9], "dxbc");
    Opt given = opt(a[11], "workspace");
    const int act = as_int32(a[8], "act"), want = PyObject_IsTrue(a[10]);
    if (want < 0) throw Refused{nullptr, ""};
    ndim(xbc, "xbc", 3);
    ndim(dx, "dx", 3);
    ndim(dB, "dB", 3);
    ndim(w, "w", 2);
    const int64_t B = xbc.size(0), T = xbc.size(1), Ch = xbc.size(2), HP = dx.size(2), GN = dB.size(2), K = w.size(1);
    if (Ch != HP + 2 * GN)
      bad_value("xbc has " + std::to_string(Ch) + " channels, HP + 2*GN = " + std::to_string(HP + 2 * GN));
    const int c = code(xbc.scalar_type(), "xbc");
    const at::ScalarType xt = xbc.scalar_type(), f32 = at::kFloat;
    const int64_t sw[] = {Ch, K}, sx[] = {B, T, HP}, sg[] = {B, T, GN}, sc[] = {Ch}, ss[] = {B, K - 1, Ch};
    check(xbc, {{&xbc, "xbc", xbc.sizes(), xt, true}, {dxbc, "dxbc", xbc.sizes(), xt, true}, {&w, "w", sw, f32, false},
                {&dx, "dx", sx, xt, false}, {&dB, "dB", sg, f32, false}, {&dC, "dC", sg, f32, false},
                {bias, "bias", sc, f32, false}, {si, "state_in", ss, f32, false}, {dso, "dstate_out", ss, f32, false}});
    const int b = dim32(B, "the batch"), t_ = dim32(T, "T"), hp = dim32(HP, "HP"), gn = dim32(GN, "GN"), k = dim32(K, "K");
    const long long ld = lead(xbc, "xbc");
    void* st = stream_of(a[12]);
    const at::Tensor g = dxbc ? *dxbc : fresh(xbc.sizes(), xt, xbc);
    const long long lddx = lead(g, "dxbc");
    const at::Tensor dw = fresh(sw, f32, xbc), db = fresh(sc, f32, xbc);
    const at::Tensor ds = want && K > 0 ? fresh(ss, f32, xbc) : at::Tensor();
    const at::Tensor ws = scratch(given, E.conv1d_bwd_ws(b, t_, hp, gn), xbc);
    const int e = without_gil([&] {
      return E.conv1d_bwd(ptr(&xbc), ld, ptr<float>(&w), ptr<float>(bias), ptr<float>(si), act, ptr(&dx), ptr<float>(&dB),
                          ptr<float>(&dC), ptr<float>(dso), ptr(&g), lddx, ptr<float>(&dw), ptr<float>(&db),
                          ds.defined() ? ptr<float>(&ds) : nullptr, b, t_, hp, gn, k, c, ptr(&ws), ws.nbytes(), st);
    });
    if (e) return PyLong_FromLong(e);
    PyObject* t = PyDict_New();
    put(t, "dxbc", result(a[9], g));
    put(t, "dw", wrapped(dw));
    put(t, "dbias", wrapped(db));
    put(t, "dstate_in", ds.defined() ? wrapped(ds) : none());
    return t;
  });
}

// conv_state, h, arrivals, xbc, dt, w, A, bias, D, dt_bias, dt_min, dt_max, slots, act, y, y code, stream
PyObject* mixer_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    const at::Tensor& conv = need(a[0], "conv_state");
    const at::Tensor& h = need(a[1], "h");
    Opt arrivals = opt(a[2], "arrivals");
    const at::Tensor& xbc = need(a[3], "xbc");
    const at::Tensor& dt = need(a[4], "dt");
    const at::Tensor& w = need(a[5], "w");
    const at::Tensor& A = need(a[6], "A");
    Opt bias = opt(a[7], "bias"), D = opt(a[8], "D"), dtb = opt(a[9], "dt_bias"), slots = opt(a[12], "slots"), y = opt(a[14], "y");
    ndim(h, "h", 4);
    ndim(xbc, "xbc", 2);
    ndim(w, "w", 2);
    const int64_t ns = h.size(0), H = h.size(1), P = h.size(2), N = h.size(3), B = xbc.size(0), Ch = xbc.size(1), K = w.size(1);
    if (N <= 0 || Ch <= H * P || (Ch - H * P) % (2 * N))
      bad_value("xbc has " + std::to_string(Ch) + " channels, not H*P + 2*G*N with H=" + std::to_string(H) +
                " P=" + std::to_string(P) + " N=" + std::to_string(N));
    const int64_t G = (Ch - H * P) / (2 * N);
    const at::ScalarType t = xbc.scalar_type(), f32 = at::kFloat;
    const int c = code(t, "xbc"), yc = y ? code(y->scalar_type(), "y") : as_int32(a[15], "y_dtype") == SSD_BF16 ? SSD_BF16 : SSD_F32;
    const int64_t sv[] = {ns, K - 1, Ch}, sa[] = {ns, G}, sd[] = {B, H}, sb[] = {B}, sw[] = {Ch, K}, sh[] = {H}, sc[] = {Ch},
                  sy[] = {B, H, P};
    check(h, {{&xbc, "xbc", xbc.sizes(), t, true}, {&dt, "dt", sd, t, true}, {&h, "h", h.sizes(), f32, false},
              {&conv, "conv_state", sv, f32, false}, {arrivals, "arrivals", sa, at::kInt, false},
              {slots, "slots", sb, at::kInt, false}, {&w, "w", sw, f32, false}, {&A, "A", sh, f32, false},
              {bias, "bias", sc, f32, false}, {D, "D", sh, f32, false}, {dtb, "dt_bias", sh, f32, false},
              {y, "y", sy, type_of(yc), false}});
    const long long ldx = lead(xbc, "xbc"), lddt = lead(dt, "dt");
    const float lo = as_float(a[10]), hi = as_float(a[11]);
    const int act = as_int32(a[13], "act");
    const int ns_ = dim32(ns, "the pool"), b = dim32(B, "the batch"), h_ = dim32(H, "H"), p = dim32(P, "P"),
              g = dim32(G, "G"), n_ = dim32(N, "N"), k = dim32(K, "K");
    void* st = stream_of(a[16]);
    const at::Tensor o = y ? *y : fresh(sy, type_of(yc), h);
    const int e = without_gil([&] {
      return E.mixer_step(ptr<float>(&conv), ptr<float>(&h), ptr<int>(arrivals), ptr<int>(slots), ns_, ptr(&xbc), ldx,
                          ptr(&dt), lddt, ptr<float>(&w), ptr<float>(bias), act, ptr<float>(&A), ptr<float>(D),
                          ptr<float>(dtb), lo, hi, ptr(&o), yc, b, h_, p, g, n_, k, c, st);
    });
    return e ? PyLong_FromLong(e) : result(a[14], o);
  });
}

// bind(path): the library whose entry points the others call
PyObject* bind(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* lib = dlopen(p, RTLD_NOW | RTLD_LOCAL);
  Entry e{};
  bool ok = lib != nullptr;
  auto find = [&](auto& f, const char* name) {
    if (ok) f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(lib, name));
    ok = ok && f;
  };
  find(e.add_norm_fwd, "ssd_add_norm_fwd");
  find(e.add_norm_bwd_ws, "ssd_add_norm_bwd_workspace_size");
  find(e.add_norm_bwd, "ssd_add_norm_bwd");
  find(e.gated_norm_fwd, "ssd_gated_norm_fwd");
  find(e.gated_norm_bwd_ws, "ssd_gated_norm_bwd_workspace_size");
  find(e.gated_norm_bwd, "ssd_gated_norm_bwd");
  find(e.conv1d_bwd_ws, "ssd_conv1d_bwd_workspace_size");
  find(e.conv1d_bwd, "ssd_conv1d_bwd");
  find(e.mixer_step, "ssd_mixer_step");
  if (!ok) {
    const char* why = dlerror();
    PyErr_SetString(PyExc_RuntimeError, why ? why : "an entry point is missing");
    return nullptr;
  }
  E = e;
  return none();
}

#define SSD_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SSD_METHOD(add_norm_fwd),   SSD_METHOD(add_norm_bwd), SSD_METHOD(gated_norm_fwd),
                         SSD_METHOD(gated_norm_bwd), SSD_METHOD(conv1d_bwd),   SSD_METHOD(mixer_step),
                         {"bind", bind, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
