// The binding's calls that a model makes for every token, as a Python extension:
// checks of the tensors, allocation of the results and the call of the C ABI.  One
// token's kernels take 2 to 10 us, and the same work done by the interpreter took 7 to
// 11 us a call.  It holds no computation: the functions it calls are libbqm.so's, whose
// addresses the binding hands over.
//
// Every function returns its result, or the ABI's error code as an integer.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>

#include <cmath>
#include <sstream>

#include "bqm.h"

namespace {

struct Refused {
  std::string what;
};

PyObject *g_device = nullptr, *g_stream = nullptr;   // torch._C._cuda_getDevice, _cuda_getCurrentRawStream

// libbqm.so's functions, by the types that bqm.h declares
#define FUNCTIONS(X) X(fp8_quant) X(fp8_gemm) X(fp8_gemm_grouped) X(moe_route_workspace) X(moe_route) X(moe_combine) \
  X(rope) X(kv_append) X(kv_attention_workspace) X(kv_attention) X(moe_ffn_workspace) X(moe_ffn)
#define DECLARE(f) decltype(&::f) p_##f = nullptr;
FUNCTIONS(DECLARE)
#undef DECLARE

std::string shown(at::IntArrayRef s) {
  std::ostringstream o;
  o << '(';
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << (s.size() == 1 ? ",)" : ")");
  return o.str();
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) throw Refused{std::string(name) + " must be a CUDA/HIP tensor"};
  return THPVariable_Unpack(o);
}

void shape(const at::Tensor &t, at::IntArrayRef want, const char *name) {
  if (t.sizes() != want)
    throw Refused{std::string(name) + " must have shape " + shown(want) + ", got " + shown(t.sizes())};
}

void on_device(const at::Tensor &t, int device, const char *name) {
  if (!t.is_cuda()) throw Refused{std::string(name) + " must be a CUDA/HIP tensor"};
  if (t.get_device() != device)
    throw Refused{std::string(name) + " must be on the current device " + std::to_string(device) + ", got " +
                  t.device().str()};
}

std::string type_name(at::ScalarType s) {
  std::ostringstream o;
  o << s;
  return o.str();
}

// The address of a contiguous tensor of the type on the device.
void *address(const at::Tensor &t, at::ScalarType type, int device, const char *name) {
  on_device(t, device, name);
  if (t.scalar_type() != type)
    throw Refused{std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type())};
  if (!t.is_contiguous()) throw Refused{std::string(name) + " must be contiguous"};
  return t.data_ptr();
}

int type_code(at::ScalarType s, const char *name) {
  switch (s) {
    case at::kFloat: return BQM_F32;
    case at::kBFloat16: return BQM_BF16;
    case at::kHalf: return BQM_F16;
    default:
      throw Refused{std::string(name) + " must be float32, bfloat16 or float16, got " + type_name(s)};
  }
}

// The current device, asked for only with a tensor on some device (there may be none).
int current_device(const at::Tensor &t, const char *name) {
  if (!t.is_cuda()) throw Refused{std::string(name) + " must be a CUDA/HIP tensor"};
  PyObject *r = PyObject_CallNoArgs(g_device);
  if (!r) throw python_error();
  const long d = PyLong_AsLong(r);
  Py_DECREF(r);
  return (int)d;
}

void *current_stream(int device) {
  PyObject *d = PyLong_FromLong(device);
  PyObject *r = d ? PyObject_CallOneArg(g_stream, d) : nullptr;
  Py_XDECREF(d);
  if (!r) throw python_error();
  void *s = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return s;
}

at::Tensor fresh(at::IntArrayRef size, at::ScalarType type, int device) {
  return at::empty(size, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)device)));
}

// The caller's result tensor, or a new one.
at::Tensor result(PyObject *o, at::IntArrayRef size, at::ScalarType type, int device, const char *name) {
  if (o == Py_None) return fresh(size, type, device);
  const at::Tensor &t = tensor(o, name);
  shape(t, size, name);
  address(t, type, device, name);
  return t;
}

int integer(PyObject *o, const char *name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v < INT32_MIN || v > INT32_MAX) throw Refused{std::string(name) + " is out of range"};
  return (int)v;
}

bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

PyObject *code(int rc) { return PyLong_FromLong(rc); }

// A 2-D tensor whose rows are contiguous, and its row stride.
int64_t strided_rows(const at::Tensor &t, const char *name) {
  if (t.dim() != 2) throw Refused{std::string(name) + " must be a 2-D tensor, got " + shown(t.sizes())};
  type_code(t.scalar_type(), name);
  if (t.numel() < 1) throw Refused{std::string(name) + " must not be empty, got " + shown(t.sizes())};
  if (t.size(1) > 1 && t.stride(1) != 1)
    throw Refused{std::string(name) + "'s rows must be contiguous (strides " + shown(t.strides()) + ")"};
  if (t.size(0) > 1 && t.stride(0) < t.size(1))
    throw Refused{std::string(name) + "'s rows must not overlap (strides " + shown(t.strides()) + ")"};
  if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX) throw Refused{std::string(name) + " is too large"};
  return t.stride(0);
}

// x, swiglu, q, scale -> (q, scale)
PyObject *quant(PyObject *const *a) {
  const at::Tensor &x = tensor(a[0], "x");
  const int64_t stride = strided_rows(x, "x");
  const bool swiglu = truth(a[1]);
  const int64_t m = x.size(0), width = x.size(1);
  if (swiglu && width % 2) throw Refused{"x must hold gate and up columns, got " + std::to_string(width)};
  const int64_t k = swiglu ? width / 2 : width, kb = (k + 127) / 128;
  const int dev = current_device(x, "x");
  on_device(x, dev, "x");
  const at::Tensor q = result(a[2], {m, kb * 128}, at::kFloat8_e4m3fn, dev, "q");
  const at::Tensor s = result(a[3], {kb, m}, at::kFloat, dev, "scale");
  const int rc = p_fp8_quant(x.data_ptr(), type_code(x.scalar_type(), "x"), (int)m, (int)k, stride, swiglu,
                             (uint8_t *)q.data_ptr(), (float *)s.data_ptr(), current_stream(dev));
  if (rc) return code(rc);
  PyObject *qo = THPVariable_Wrap(q), *so = THPVariable_Wrap(s);
  return Py_BuildValue("(NN)", qo, so);
}

struct Product {
  int64_t experts = 1, rows = 0, cols = 0, m = 0, kb = 0;
  at::ScalarType type = at::kBFloat16;
  const void *w, *ws, *q, *qs;
};

// w, w_scale, cols, q, q_scale: their shapes, and the type of the result
Product product(PyObject *const *a, bool grouped, PyObject *dtype, PyObject *y) {
  Product p;
  p.cols = integer(a[2], "cols");
  if (p.cols < 1) throw Refused{"cols must be at least 1, got " + std::to_string(p.cols)};
  p.kb = (p.cols + 127) / 128;
  const std::string kp = std::to_string(p.kb * 128);
  const at::Tensor &w = tensor(a[0], "w"), &q = tensor(a[3], "q");
  const int64_t lead = grouped ? 1 : 0;
  if (w.dim() != lead + 2 || w.size(-1) != p.kb * 128 || w.numel() < 1 || w.size(0) > INT32_MAX ||
      w.size(-2) > INT32_MAX)
    throw Refused{std::string("w must have shape [") + (grouped ? "experts, " : "") + "rows, " + kp + "], got " +
                  shown(w.sizes())};
  if (q.dim() != 2 || q.size(1) != p.kb * 128 || q.size(0) < 1 || q.size(0) > INT32_MAX)
    throw Refused{"q must have shape [batch, " + kp + "], got " + shown(q.sizes())};
  p.experts = grouped ? w.size(0) : 1;
  p.rows = w.size(-2);
  p.m = q.size(0);
  const at::Tensor &ws = tensor(a[1], "w_scale"), &qs = tensor(a[4], "q_scale");
  const int64_t nb = (p.rows + 127) / 128;
  if (grouped) shape(ws, {p.experts, nb, p.kb}, "w_scale");
  else shape(ws, {nb, p.kb}, "w_scale");
  shape(qs, {p.kb, p.m}, "q_scale");
  if (dtype != Py_None) {
    if (!THPDtype_Check(dtype)) throw Refused{"dtype must be a torch.dtype"};
    p.type = reinterpret_cast<THPDtype *>(dtype)->scalar_type;
  }
  if (y != Py_None) {
    const at::Tensor &t = tensor(y, "y");
    if (dtype != Py_None && t.scalar_type() != p.type)
      throw Refused{"y must be " + type_name(p.type) + ", got " + type_name(t.scalar_type())};
    p.type = t.scalar_type();
  }
  type_code(p.type, "y");
  return p;
}

// the addresses, once every shape has been checked and the tensors are known to be on a device
int operands(Product &p, PyObject *const *a) {
  const at::Tensor &w = THPVariable_Unpack(a[0]), &ws = THPVariable_Unpack(a[1]);
  const at::Tensor &q = THPVariable_Unpack(a[3]), &qs = THPVariable_Unpack(a[4]);
  const int dev = current_device(q, "q");
  p.w = address(w, at::kFloat8_e4m3fn, dev, "w");
  p.ws = address(ws, at::kFloat, dev, "w_scale");
  p.q = address(q, at::kFloat8_e4m3fn, dev, "q");
  p.qs = address(qs, at::kFloat, dev, "q_scale");
  return dev;
}

// w, w_scale, cols, q, q_scale, dtype, y -> y
PyObject *gemm(PyObject *const *a) {
  Product p = product(a, false, a[5], a[6]);
  const int dev = operands(p, a);
  const at::Tensor y = result(a[6], {p.m, p.rows}, p.type, dev, "y");
  const int rc = p_fp8_gemm((const uint8_t *)p.w, (const float *)p.ws, (int)p.rows, (int)p.cols, (const uint8_t *)p.q,
                            (const float *)p.qs, (int)p.m, y.data_ptr(), type_code(p.type, "y"), current_stream(dev));
  return rc ? code(rc) : THPVariable_Wrap(y);
}

// w, w_scale, cols, q, q_scale, offsets, row_ids, dtype, y -> y
PyObject *grouped(PyObject *const *a) {
  Product p = product(a, true, a[7], a[8]);
  const at::Tensor &off = tensor(a[5], "offsets");
  shape(off, {p.experts + 1}, "offsets");
  int64_t slots = p.m;
  const bool gather = a[6] != Py_None;
  if (gather) {
    const at::Tensor &r = tensor(a[6], "row_ids");
    if (r.dim() != 1 || r.size(0) < 1 || r.size(0) > INT32_MAX)
      throw Refused{"row_ids must have shape [slots], got " + shown(r.sizes())};
    slots = r.size(0);
  }
  const int dev = operands(p, a);
  const void *op = address(off, at::kInt, dev, "offsets");
  const void *rp = gather ? address(THPVariable_Unpack(a[6]), at::kInt, dev, "row_ids") : nullptr;
  const at::Tensor y = result(a[8], {slots, p.rows}, p.type, dev, "y");
  const int rc = p_fp8_gemm_grouped((const uint8_t *)p.w, (const float *)p.ws, (int)p.experts, (int)p.rows,
                                    (int)p.cols, (const uint8_t *)p.q, (const float *)p.qs, (int)p.m,
                                    (const int32_t *)op, (const int32_t *)rp, (int)slots, y.data_ptr(),
                                    type_code(p.type, "y"), current_stream(dev));
  return rc ? code(rc) : THPVariable_Wrap(y);
}

// logits, top, renorm, workspace -> (ids, weights, offsets, row_ids, slots)
PyObject *route(PyObject *const *a) {
  const at::Tensor &x = tensor(a[0], "logits");
  const int64_t stride = strided_rows(x, "logits");
  const int64_t tokens = x.size(0), experts = x.size(1);
  const int top = integer(a[1], "top");
  const int dev = current_device(x, "logits");
  int64_t need = 0;
  int rc = p_moe_route_workspace((int)tokens, (int)experts, top, &need);
  if (rc) return code(rc);
  on_device(x, dev, "logits");
  at::Tensor ws;
  if (a[3] != Py_None) {
    ws = tensor(a[3], "workspace");
    address(ws, at::kByte, dev, "workspace");
    if (ws.numel() < need)
      throw Refused{"workspace must hold at least " + std::to_string(need) + " bytes, got " +
                    std::to_string(ws.numel())};
  } else if (need) {
    ws = fresh({need}, at::kByte, dev);
  }
  const at::Tensor ids = fresh({tokens, top}, at::kInt, dev), weights = fresh({tokens, top}, at::kFloat, dev),
                   offsets = fresh({experts + 1}, at::kInt, dev), rows = fresh({tokens * top}, at::kInt, dev),
                   slots = fresh({tokens, top}, at::kInt, dev);
  rc = p_moe_route(x.data_ptr(), type_code(x.scalar_type(), "logits"), (int)tokens, (int)experts, stride, top,
                   truth(a[2]), (int32_t *)ids.data_ptr(), (float *)weights.data_ptr(), (int32_t *)offsets.data_ptr(),
                   (int32_t *)rows.data_ptr(), (int32_t *)slots.data_ptr(), ws.defined() ? ws.data_ptr() : nullptr,
                   need, current_stream(dev));
  if (rc) return code(rc);
  return Py_BuildValue("(NNNNN)", THPVariable_Wrap(ids), THPVariable_Wrap(weights), THPVariable_Wrap(offsets),
                       THPVariable_Wrap(rows), THPVariable_Wrap(slots));
}

// y, slots, weights, out -> out
PyObject *combine(PyObject *const *a) {
  const at::Tensor &y = tensor(a[0], "y"), &slots = tensor(a[1], "slots"), &weights = tensor(a[2], "weights");
  if (y.dim() != 2 || y.numel() < 1 || y.size(1) > INT32_MAX)
    throw Refused{"y must have shape [rows, d], got " + shown(y.sizes())};
  if (slots.dim() != 2 || slots.numel() < 1 || slots.size(0) > INT32_MAX || slots.size(1) > INT32_MAX)
    throw Refused{"slots must have shape [tokens, top], got " + shown(slots.sizes())};
  shape(weights, slots.sizes(), "weights");
  const int type = type_code(y.scalar_type(), "y");
  const int dev = current_device(y, "y");
  const void *yp = address(y, y.scalar_type(), dev, "y"), *sp = address(slots, at::kInt, dev, "slots"),
             *wp = address(weights, at::kFloat, dev, "weights");
  const at::Tensor out = result(a[3], {slots.size(0), y.size(1)}, y.scalar_type(), dev, "out");
  const int rc = p_moe_combine(yp, type, y.size(0), (int)y.size(1), (const int32_t *)sp, (const float *)wp,
                               (int)slots.size(0), (int)slots.size(1), out.data_ptr(), current_stream(dev));
  return rc ? code(rc) : THPVariable_Wrap(out);
}

double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

// A tensor [tokens, heads, dim] whose rows are contiguous, on the device
struct Heads {
  int tokens, heads, dim, type;
  int64_t ts, hs;
};
Heads heads_of(const at::Tensor &t, const char *name) {
  if (t.dim() != 3 || t.numel() < 1)
    throw Refused{std::string(name) + " must have shape [tokens, heads, dim], got " + shown(t.sizes())};
  if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX || t.size(2) > INT32_MAX) throw Refused{std::string(name) + " is too large"};
  const int type = type_code(t.scalar_type(), name);
  if (t.size(2) > 1 && t.stride(2) != 1)
    throw Refused{std::string(name) + "'s rows must be contiguous (strides " + shown(t.strides()) + ")"};
  return {(int)t.size(0), (int)t.size(1), (int)t.size(2), type, t.stride(0), t.stride(1)};
}

// freqs and positions of `tokens` tokens, or none of both
struct Turns {
  const at::Tensor *positions = nullptr, *freqs = nullptr;
  int rotary = 0;
  const int32_t *p = nullptr;
  const double *f = nullptr;
  Turns(PyObject *po, PyObject *fo, const Heads &x) {
    if (fo == Py_None) {
      if (po != Py_None) throw Refused{"positions come with freqs"};
      return;
    }
    freqs = &tensor(fo, "freqs");
    positions = &tensor(po, "positions");
    if (freqs->dim() != 1 || freqs->numel() < 1 || 2 * freqs->numel() > x.dim)
      throw Refused{"freqs must have shape [rotary / 2], rotary at most " + std::to_string(x.dim) + ", got " + shown(freqs->sizes())};
    shape(*positions, {x.tokens}, "positions");
    rotary = 2 * (int)freqs->numel();
  }
  void addresses(int dev) {
    if (!freqs) return;
    f = (const double *)address(*freqs, at::kDouble, dev, "freqs");
    p = (const int32_t *)address(*positions, at::kInt, dev, "positions");
  }
};

// x, positions, freqs, interleaved, mscale, backward, out -> out
PyObject *rope_call(PyObject *const *a) {
  const at::Tensor &x = tensor(a[0], "x");
  const Heads h = heads_of(x, "x");
  if (a[2] == Py_None) throw Refused{"freqs must be a CUDA/HIP tensor"};
  Turns r(a[1], a[2], h);
  const int dev = current_device(x, "x");
  on_device(x, dev, "x");
  r.addresses(dev);
  at::Tensor y;
  if (a[6] == Py_None) {
    y = fresh(x.sizes(), x.scalar_type(), dev);
  } else {
    y = tensor(a[6], "out");
    shape(y, x.sizes(), "out");
    on_device(y, dev, "out");
    if (y.scalar_type() != x.scalar_type())
      throw Refused{"out must be " + type_name(x.scalar_type()) + ", got " + type_name(y.scalar_type())};
  }
  const Heads o = heads_of(y, "out");
  const int rc = p_rope(x.data_ptr(), h.type, h.tokens, h.heads, h.dim, h.ts, h.hs, r.p, r.f, r.rotary, truth(a[3]),
                        (float)number(a[4]), truth(a[5]), y.data_ptr(), o.ts, o.hs, current_stream(dev));
  return rc ? code(rc) : THPVariable_Wrap(y);
}

// The cache's four tensors and the batch's: a = k, v, k_scale, v_scale; pages, lens, offsets
struct Cache {
  int64_t count, heads;
  uint8_t *k, *v;
  float *ks, *vs;
  int seqs, width;
  int64_t stride;
  const int32_t *pages, *lens, *offsets = nullptr;
  Cache(PyObject *const *a, PyObject *const *b, int64_t dim, int64_t tokens) {
    const at::Tensor &kt = tensor(a[0], "cache.k"), &vt = tensor(a[1], "cache.v");
    const int64_t dp = dim <= 128 ? (dim + 31) / 32 * 32 : (dim + 63) / 64 * 64;
    if (kt.dim() != 4 || kt.size(2) != 64 || kt.size(3) != dp || kt.numel() < 1 || kt.size(0) > INT32_MAX || kt.size(1) > INT32_MAX)
      throw Refused{"cache.k must have shape [pages, heads, 64, " + std::to_string(dp) + "], got " + shown(kt.sizes())};
    count = kt.size(0);
    heads = kt.size(1);
    shape(vt, {count, heads, dp, 64}, "cache.v");
    shape(tensor(a[2], "cache.k_scale"), {count, heads}, "cache.k_scale");
    shape(tensor(a[3], "cache.v_scale"), {count, heads}, "cache.v_scale");
    const at::Tensor &p = tensor(b[0], "pages");
    if (p.dim() != 2 || p.numel() < 1 || p.size(0) > INT32_MAX || p.size(1) > INT32_MAX)
      throw Refused{"pages must have shape [seqs, width], got " + shown(p.sizes())};
    if (p.size(1) > 1 && p.stride(1) != 1) throw Refused{"pages's rows must be contiguous (strides " + shown(p.strides()) + ")"};
    seqs = (int)p.size(0);
    width = (int)p.size(1);
    stride = p.stride(0);
    shape(tensor(b[1], "lens"), {seqs}, "lens");
    if (b[2] != Py_None) shape(tensor(b[2], "offsets"), {seqs + 1}, "offsets");
    else if (tokens != seqs)
      throw Refused{"without offsets there is one token a sequence: " + std::to_string(seqs) + " sequences, got " + std::to_string(tokens)};
  }
  void addresses(PyObject *const *a, PyObject *const *b, int dev) {
    k = (uint8_t *)address(THPVariable_Unpack(a[0]), at::kFloat8_e4m3fn, dev, "cache.k");
    v = (uint8_t *)address(THPVariable_Unpack(a[1]), at::kFloat8_e4m3fn, dev, "cache.v");
    ks = (float *)address(THPVariable_Unpack(a[2]), at::kFloat, dev, "cache.k_scale");
    vs = (float *)address(THPVariable_Unpack(a[3]), at::kFloat, dev, "cache.v_scale");
    const at::Tensor &p = THPVariable_Unpack(b[0]);
    on_device(p, dev, "pages");
    if (p.scalar_type() != at::kInt) throw Refused{"pages must be Int, got " + type_name(p.scalar_type())};
    pages = (const int32_t *)p.data_ptr();
    lens = (const int32_t *)address(THPVariable_Unpack(b[1]), at::kInt, dev, "lens");
    if (b[2] != Py_None) offsets = (const int32_t *)address(THPVariable_Unpack(b[2]), at::kInt, dev, "offsets");
  }
};

// cache.k, cache.v, cache.k_scale, cache.v_scale, pages, lens, offsets, k, v, positions, freqs, interleaved, mscale
PyObject *append(PyObject *const *a) {
  const at::Tensor &k = tensor(a[7], "k"), &v = tensor(a[8], "v");
  const Heads h = heads_of(k, "k");
  shape(v, k.sizes(), "v");
  const Heads g = heads_of(v, "v");
  if (g.type != h.type) throw Refused{"v must be " + type_name(k.scalar_type()) + ", got " + type_name(v.scalar_type())};
  Cache c(a, a + 4, h.dim, h.tokens);
  if (c.heads != h.heads)
    throw Refused{"k must have the cache's " + std::to_string(c.heads) + " heads, got " + shown(k.sizes())};
  Turns r(a[9], a[10], h);
  const int dev = current_device(k, "k");
  on_device(k, dev, "k");
  on_device(v, dev, "v");
  r.addresses(dev);
  c.addresses(a, a + 4, dev);
  return code(p_kv_append(k.data_ptr(), v.data_ptr(), h.type, h.tokens, h.heads, h.dim, h.ts, h.hs, g.ts, g.hs, c.offsets,
                          c.lens, c.seqs, c.pages, c.stride, c.width, r.p, r.f, r.rotary, truth(a[11]), (float)number(a[12]),
                          c.k, c.v, c.ks, c.vs, (int)c.count, current_stream(dev)));
}

// The caller's workspace of at least `need` bytes, or a new one; nothing where none is needed.
at::Tensor scratch(PyObject *o, int64_t need, int dev) {
  if (o == Py_None) return need ? fresh({need}, at::kByte, dev) : at::Tensor();
  const at::Tensor &ws = tensor(o, "workspace");
  address(ws, at::kByte, dev, "workspace");
  if (ws.numel() < need)
    throw Refused{"workspace must hold at least " + std::to_string(need) + " bytes, got " + std::to_string(ws.numel())};
  return ws;
}

// cache.k, cache.v, cache.k_scale, cache.v_scale, pages, lens, offsets, q, scale, window, out, workspace -> out
PyObject *attention(PyObject *const *a) {
  const at::Tensor &q = tensor(a[7], "q");
  const Heads h = heads_of(q, "q");
  Cache c(a, a + 4, h.dim, h.tokens);
  if (h.heads % c.heads)
    throw Refused{"q's heads must be a multiple of the cache's " + std::to_string(c.heads) + ", got " + std::to_string(h.heads)};
  const int window = integer(a[9], "window");
  if (window < 0) throw Refused{"window must be at least 0, got " + std::to_string(window)};
  const float scale = a[8] == Py_None ? (float)(1.0 / std::sqrt((double)h.dim)) : (float)number(a[8]);
  const int dev = current_device(q, "q");
  on_device(q, dev, "q");
  c.addresses(a, a + 4, dev);
  int64_t need = 0;
  int rc = p_kv_attention_workspace(h.tokens, c.seqs, h.heads, (int)c.heads, h.dim, c.width, &need);
  if (rc) return code(rc);
  const at::Tensor ws = scratch(a[11], need, dev);
  const at::Tensor out = result(a[10], q.sizes(), q.scalar_type(), dev, "out");
  rc = p_kv_attention(q.data_ptr(), h.type, h.tokens, h.heads, h.dim, h.ts, h.hs, c.offsets, c.lens, c.seqs, c.pages,
                      c.stride, c.width, c.k, c.v, c.ks, c.vs, (int)c.count, (int)c.heads, scale, window, out.data_ptr(),
                      ws.defined() ? ws.data_ptr() : nullptr, need, current_stream(dev));
  return rc ? code(rc) : THPVariable_Wrap(out);
}

// x, w13, w13_scale, w2, w2_scale, logits, top, renorm, out, workspace -> out
PyObject *few(PyObject *const *a) {
  const at::Tensor &x = tensor(a[0], "x"), &logits = tensor(a[5], "logits");
  const int64_t xs = strided_rows(x, "x"), ls = strided_rows(logits, "logits");
  const int64_t tokens = x.size(0), hidden = x.size(1), experts = logits.size(1);
  if (logits.size(0) != tokens)
    throw Refused{"logits must have shape [" + std::to_string(tokens) + ", experts], got " + shown(logits.sizes())};
  const at::Tensor &w13 = tensor(a[1], "w13"), &w2 = tensor(a[3], "w2");
  const int64_t kb = (hidden + 127) / 128;
  if (w13.dim() != 3 || w13.size(0) != experts || w13.size(1) % 2 || w13.size(2) != kb * 128 || w13.numel() < 1 || w13.size(1) > INT32_MAX)
    throw Refused{"w13 must have shape [" + std::to_string(experts) + ", 2 ffn, " + std::to_string(kb * 128) + "], got " + shown(w13.sizes())};
  const int64_t ffn = w13.size(1) / 2, fb = (ffn + 127) / 128;
  shape(w2, {experts, hidden, fb * 128}, "w2");
  const at::Tensor &s13 = tensor(a[2], "w13_scale"), &s2 = tensor(a[4], "w2_scale");
  shape(s13, {experts, (2 * ffn + 127) / 128, kb}, "w13_scale");
  shape(s2, {experts, kb, fb}, "w2_scale");
  const int top = integer(a[6], "top");
  const int dev = current_device(x, "x");
  int64_t need = 0;
  int rc = p_moe_ffn_workspace((int)tokens, (int)experts, top, (int)hidden, (int)ffn, &need);
  if (rc) return code(rc);
  on_device(x, dev, "x");
  on_device(logits, dev, "logits");
  const void *w13p = address(w13, at::kFloat8_e4m3fn, dev, "w13"), *w2p = address(w2, at::kFloat8_e4m3fn, dev, "w2"),
             *s13p = address(s13, at::kFloat, dev, "w13_scale"), *s2p = address(s2, at::kFloat, dev, "w2_scale");
  const at::Tensor ws = scratch(a[9], need, dev);
  const at::Tensor out = result(a[8], x.sizes(), x.scalar_type(), dev, "out");
  rc = p_moe_ffn(x.data_ptr(), type_code(x.scalar_type(), "x"), (int)tokens, (int)hidden, xs, logits.data_ptr(),
                 type_code(logits.scalar_type(), "logits"), ls, (int)experts, top, truth(a[7]), (const uint8_t *)w13p,
                 (const float *)s13p, (const uint8_t *)w2p, (const float *)s2p, (int)ffn, out.data_ptr(),
                 ws.defined() ? ws.data_ptr() : nullptr, need, current_stream(dev));
  return rc ? code(rc) : THPVariable_Wrap(out);
}

// No exception leaves a call: refusals become ValueError, torch's errors its own.
template <PyObject *(*kCall)(PyObject *const *), int kArgs>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != kArgs || !g_device) {
    PyErr_SetString(PyExc_TypeError, g_device ? "wrong number of arguments" : "the library is not bound");
    return nullptr;
  }
  try {
    return kCall(a);
  } catch (const Refused &r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// {name: address}, _cuda_getDevice, _cuda_getCurrentRawStream
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 3 || !PyDict_Check(a[0])) {
    PyErr_SetString(PyExc_TypeError, "bind takes a dict of addresses and two functions");
    return nullptr;
  }
#define TAKE(f)                                                              \
  {                                                                          \
    PyObject *o = PyDict_GetItemString(a[0], #f);                            \
    void *p = o ? PyLong_AsVoidPtr(o) : nullptr;                             \
    if (!p) {                                                                \
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_KeyError, #f);            \
      return nullptr;                                                        \
    }                                                                        \
    p_##f = reinterpret_cast<decltype(p_##f)>(p);                            \
  }
  FUNCTIONS(TAKE)
#undef TAKE
  Py_INCREF(a[1]);
  Py_INCREF(a[2]);
  g_device = a[1];
  g_stream = a[2];
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {
    {"bind", FAST(bind), METH_FASTCALL, nullptr},
    {"fp8_quant", FAST((&entry<quant, 4>)), METH_FASTCALL, nullptr},
    {"fp8_gemm", FAST((&entry<gemm, 7>)), METH_FASTCALL, nullptr},
    {"fp8_gemm_grouped", FAST((&entry<grouped, 9>)), METH_FASTCALL, nullptr},
    {"moe_route", FAST((&entry<route, 4>)), METH_FASTCALL, nullptr},
    {"moe_combine", FAST((&entry<combine, 4>)), METH_FASTCALL, nullptr},
    {"rope", FAST((&entry<rope_call, 7>)), METH_FASTCALL, nullptr},
    {"kv_append", FAST((&entry<append, 13>)), METH_FASTCALL, nullptr},
    {"kv_attention", FAST((&entry<attention, 12>)), METH_FASTCALL, nullptr},
    {"moe_ffn", FAST((&entry<few, 10>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
