// rglru_torch.cpp -- the binding's checks of the attention block's and the serving operators' tensors, and its calls of the C ABI
// (include/rglru.h), as a CPython module. In Python the checks of a dozen tensors take longer than the
// kernels of a decoding step (17 us against 4 for the norms of 64 tokens); here they are reads of tensor
// fields, and new tensors are made without the arguments of torch.empty (0.5 us each instead of 1.2).
// Nothing is computed here.
//
// Tensors of heads are [..., H, dh] with the heads of a token contiguous and one stride from token to token;
// other tensors are contiguous. Shapes and types are checked first, then the devices: all tensors on one
// GPU. A tensor that does not fit raises ValueError (TypeError if it is none); else the functions return
// the entry point's status. The interpreter's lock is given up for the call, as a full queue may hold it.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <string>

#include "rglru.h"

namespace {

struct Refused {};  // a Python error is set

typedef c10::IntArrayRef Sizes;

[[noreturn]] void refuse(PyObject *kind, const std::string &what) {
  PyErr_SetString(kind, what.c_str());
  throw Refused{};
}

std::string text(Sizes s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

std::string text(c10::ScalarType t) { return std::string("torch.") + torch::getTHPDtype(t)->name; }

// The tensors of one call.
class Call {
 public:
  // The call's first tensor: f32 or bf16.
  const at::Tensor &first(PyObject *o, const char *name, int64_t min_dim) {
    const at::Tensor &t = tensor(o, name);
    io_ = t.scalar_type();
    if (io_ != at::kBFloat16 && io_ != at::kFloat)
      refuse(PyExc_ValueError, std::string(name) + ": unsupported dtype " + text(io_));
    if (t.dim() < min_dim)
      refuse(PyExc_ValueError, std::string(name) + ": expected [..., heads, dh], got shape " + text(t.sizes()));
    return t;
  }
  static const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + ": expected a torch.Tensor");
    return THPVariable_Unpack(o);
  }
  rglru_dtype dtype() const { return io_ == at::kBFloat16 ? RGLRU_BF16 : RGLRU_F32; }
  c10::ScalarType io() const { return io_; }

  // Pointer of a contiguous tensor of this shape (and of this type); NULL for None.
  void *flat(PyObject *o, c10::ScalarType type, Sizes shape, const char *name) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    fits(t, type, shape, name);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + ": must be contiguous");
    return seen(t, name);
  }
  // Pointer and bytes of a workspace: any contiguous tensor.
  void *workspace(PyObject *o, size_t &bytes) {
    bytes = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, "workspace");
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "workspace: must be contiguous");
    bytes = t.nbytes();
    return seen(t, "workspace");
  }
  // Pointer of a tensor of heads of this shape, and the elements from token to token.
  void *heads(PyObject *o, Sizes shape, long long &stride, const char *name) {
    stride = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    fits(t, io_, shape, name);
    const Sizes st = t.strides();
    const size_t n = shape.size();
    const int64_t H = shape[n - 2], dh = shape[n - 1];
    if ((dh > 1 && st[n - 1] != 1) || (H > 1 && st[n - 2] != dh))
      refuse(PyExc_ValueError, std::string(name) + ": the heads of a token must be contiguous");
    int64_t step = H * dh, reach = -1;  // the innermost leading dimension longer than 1 gives the stride
    for (size_t i = n - 2; i-- > 0;) {
      if (shape[i] == 1) continue;
      if (reach < 0)
        step = st[i];
      else if (st[i] != reach)
        refuse(PyExc_ValueError, std::string(name) + ": tokens must be one stride apart");
      reach = st[i] * shape[i];
    }
    if (step < H * dh) refuse(PyExc_ValueError, std::string(name) + ": tokens overlap");
    stride = step;
    return seen(t, name);
  }
  // The entry point's status, once all tensors are on one GPU.
  template <typename F, typename... A> long run(F entry, A... args) const {
    const c10::Device device = tensors_[0].tensor->device();
    for (int i = 0; i < count_; ++i) {
      const at::Tensor &t = *tensors_[i].tensor;
      if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(tensors_[i].name) + ": must be a device tensor");
      if (t.device() != device)
        refuse(PyExc_ValueError,
               std::string(tensors_[i].name) + ": on " + t.device().str() + ", expected " + device.str());
    }
    long status;
    Py_BEGIN_ALLOW_THREADS;
    status = entry(args...);
    Py_END_ALLOW_THREADS;
    return status;
  }

 private:
  static void fits(const at::Tensor &t, c10::ScalarType type, Sizes shape, const char *name) {
    if (t.sizes() != shape)
      refuse(PyExc_ValueError, std::string(name) + ": expected shape " + text(shape) + ", got " + text(t.sizes()));
    if (t.scalar_type() != type)
      refuse(PyExc_ValueError, std::string(name) + ": expected " + text(type) + ", got " + text(t.scalar_type()));
  }
  void *seen(const at::Tensor &t, const char *name) {
    tensors_[count_].tensor = &t;
    tensors_[count_++].name = name;
    return t.data_ptr();
  }
  c10::ScalarType io_ = at::kFloat;
  struct {
    const at::Tensor *tensor;
    const char *name;
  } tensors_[16];  // no operator has more
  int count_ = 0;
};

int as_int(int64_t v, const char *name) {
  if (v > INT_MAX) refuse(PyExc_ValueError, std::string(name) + ": too large");
  return static_cast<int>(v);
}
// An integer argument; larger ones than an int holds as the largest (a window beyond every sequence).
int arg_int(PyObject *o) {
  int overflow = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
  if (v == -1 && !overflow && PyErr_Occurred()) throw Refused{};
  return overflow > 0 || v > INT_MAX ? INT_MAX : overflow < 0 || v < INT_MIN ? INT_MIN : static_cast<int>(v);
}
float arg_float(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return static_cast<float>(v);
}
void *arg_stream(PyObject *o) {
  void *p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Refused{};
  return p;
}

typedef c10::SmallVector<int64_t, 6> Shape;

// q's shape with another number of heads (k's), whose own trailing sizes have to exist.
Shape with_heads(Sizes q, PyObject *other, const char *name) {
  const at::Tensor &t = Call::tensor(other, name);
  if (t.dim() < 2)
    refuse(PyExc_ValueError, std::string(name) + ": expected [..., heads, dh], got shape " + text(t.sizes()));
  Shape s(q.begin(), q.end());
  s[s.size() - 2] = t.size(t.dim() - 2);
  return s;
}

template <typename F> PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F f) {
  try {
    if (got != want) refuse(PyExc_TypeError, "wrong number of arguments");
    return PyLong_FromLong(f());
  } catch (const Refused &) {
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (q, k, v, q_w, k_w, inv_freq, positions, slots, q_out, k_out, k_pages, v_pages, eps, stream)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> long {
    Call c;
    const at::Tensor &q = c.first(a[0], "q", 3);
    const Sizes qs = q.sizes(), lead = qs.slice(0, qs.size() - 2);
    const Shape ks = with_heads(qs, a[1], "k");
    const int64_t Hq = qs[qs.size() - 2], Hkv = ks[ks.size() - 2], dh = qs[qs.size() - 1];
    long long sq, sk, sv = 0, sqo, sko;
    void *pq = c.heads(a[0], qs, sq, "q"), *pk = c.heads(a[1], ks, sk, "k");
    void *pqo = c.heads(a[8], qs, sqo, "q_out"), *pko = c.heads(a[9], ks, sko, "k_out");
    void *pv = nullptr, *kp = nullptr, *vp = nullptr, *slots = nullptr;
    int64_t n_slots = 0;
    if (a[7] != Py_None) {
      if (a[2] == Py_None || a[10] == Py_None || a[11] == Py_None)
        refuse(PyExc_ValueError, "slots: needs v, k_pages and v_pages");
      const at::Tensor &pages = Call::tensor(a[10], "k_pages");
      if (pages.dim() != 4)
        refuse(PyExc_ValueError, "k_pages: expected [pages, page, Hkv, dh], got " + text(pages.sizes()));
      const int64_t pool[] = {pages.size(0), pages.size(1), Hkv, dh};
      n_slots = pool[0] * pool[1];
      pv = c.heads(a[2], ks, sv, "v");
      kp = c.flat(a[10], c.io(), pool, "k_pages");
      vp = c.flat(a[11], c.io(), pool, "v_pages");
      slots = c.flat(a[7], at::kLong, lead, "slots");
    } else if (a[10] != Py_None || a[11] != Py_None) {
      refuse(PyExc_ValueError, "k_pages, v_pages: need slots");
    }
    const int64_t pairs = a[5] == Py_None ? 0 : Call::tensor(a[5], "inv_freq").numel();
    const int64_t vec[] = {dh}, half[] = {pairs};
    const float *qw = static_cast<float *>(c.flat(a[3], at::kFloat, vec, "q_w"));
    const float *kw = static_cast<float *>(c.flat(a[4], at::kFloat, vec, "k_w"));
    const float *fr = static_cast<float *>(c.flat(a[5], at::kFloat, half, "inv_freq"));
    const int *pos = static_cast<int *>(c.flat(a[6], at::kInt, lead, "positions"));
    const int64_t rows = q.numel() / std::max<int64_t>(1, Hq * dh);
    return c.run(rglru_qk_norm_rope, pq, pk, pv, qw, kw, fr, pos, static_cast<long long *>(slots), pqo,
                 pko, kp, vp, as_int(rows, "q"), as_int(Hq, "q"), as_int(Hkv, "k"), as_int(dh, "q"),
                 as_int(2 * pairs, "inv_freq"), sq, sk, sv, sqo, sko, n_slots, arg_float(a[12]),
                 c.dtype(), arg_stream(a[13]));
  });
}

// (q, k, q_w, k_w, inv_freq, positions, dq_out, dk_out, dq, dk, dq_w, dk_w, eps, workspace, stream)
PyObject *qk_norm_rope_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> long {
    Call c;
    const at::Tensor &q = c.first(a[0], "q", 3);
    const Sizes qs = q.sizes(), lead = qs.slice(0, qs.size() - 2);
    const Shape ks = with_heads(qs, a[1], "k");
    const int64_t Hq = qs[qs.size() - 2], Hkv = ks[ks.size() - 2], dh = qs[qs.size() - 1];
    long long s[6];
    void *pq = c.heads(a[0], qs, s[0], "q"), *pk = c.heads(a[1], ks, s[1], "k");
    void *gq = c.heads(a[6], qs, s[2], "dq_out"), *gk = c.heads(a[7], ks, s[3], "dk_out");
    void *dq = c.heads(a[8], qs, s[4], "dq"), *dk = c.heads(a[9], ks, s[5], "dk");
    const int64_t pairs = a[4] == Py_None ? 0 : Call::tensor(a[4], "inv_freq").numel();
    const int64_t vec[] = {dh}, half[] = {pairs};
    const float *qw = static_cast<float *>(c.flat(a[2], at::kFloat, vec, "q_w"));
    const float *kw = static_cast<float *>(c.flat(a[3], at::kFloat, vec, "k_w"));
    const float *fr = static_cast<float *>(c.flat(a[4], at::kFloat, half, "inv_freq"));
    const int *pos = static_cast<int *>(c.flat(a[5], at::kInt, lead, "positions"));
    float *dqw = static_cast<float *>(c.flat(a[10], at::kFloat, vec, "dq_w"));
    float *dkw = static_cast<float *>(c.flat(a[11], at::kFloat, vec, "dk_w"));
    size_t bytes;
    void *ws = c.workspace(a[13], bytes);
    const int64_t rows = q.numel() / std::max<int64_t>(1, Hq * dh);
    return c.run(rglru_qk_norm_rope_backward, pq, pk, qw, kw, fr, pos, gq, gk, dq, dk, dqw, dkw,
                 as_int(rows, "q"), as_int(Hq, "q"), as_int(Hkv, "k"), as_int(dh, "q"),
                 as_int(2 * pairs, "inv_freq"), s[0], s[1], s[2], s[3], s[4], s[5], arg_float(a[12]),
                 c.dtype(), ws, bytes, arg_stream(a[14]));
  });
}

const at::Tensor &batch_of_heads(Call &c, PyObject *o) {
  const at::Tensor &q = c.first(o, "q", 3);
  if (q.dim() != 4) refuse(PyExc_ValueError, "q: expected [B, T, Hq, dh], got shape " + text(q.sizes()));
  return q;
}

// (q, k, v, lens, o, lse, window, sinks, scale, stream)
PyObject *local_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> long {
    Call c;
    const Sizes qs = batch_of_heads(c, a[0]).sizes();
    const Shape ks = with_heads(qs, a[1], "k");
    const int64_t B = qs[0], T = qs[1], Hq = qs[2], Hkv = ks[2], dh = qs[3];
    const int64_t per_seq[] = {B}, rows[] = {B, Hq, T};
    long long sq, sk, sv;
    void *q = c.heads(a[0], qs, sq, "q"), *k = c.heads(a[1], ks, sk, "k"), *v = c.heads(a[2], ks, sv, "v");
    const int *lens = static_cast<int *>(c.flat(a[3], at::kInt, per_seq, "lens"));
    void *o = c.flat(a[4], c.io(), qs, "o");
    float *lse = static_cast<float *>(c.flat(a[5], at::kFloat, rows, "lse"));
    return c.run(rglru_local_attention, q, k, v, lens, o, lse, as_int(B, "q"), as_int(T, "q"),
                 as_int(Hq, "q"), as_int(Hkv, "k"), as_int(dh, "q"), sq, sk, sv, arg_int(a[6]),
                 arg_int(a[7]), arg_float(a[8]), c.dtype(), arg_stream(a[9]));
  });
}

// (q, k, v, lens, o, lse, do, dq, dk, dv, window, sinks, scale, workspace, stream)
PyObject *local_attention_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> long {
    Call c;
    const Sizes qs = batch_of_heads(c, a[0]).sizes();
    const Shape ks = with_heads(qs, a[1], "k");
    const int64_t B = qs[0], T = qs[1], Hq = qs[2], Hkv = ks[2], dh = qs[3];
    const int64_t per_seq[] = {B}, rows[] = {B, Hq, T};
    long long sq, sk, sv, sdq, sdk, sdv;
    void *q = c.heads(a[0], qs, sq, "q"), *k = c.heads(a[1], ks, sk, "k"), *v = c.heads(a[2], ks, sv, "v");
    const int *lens = static_cast<int *>(c.flat(a[3], at::kInt, per_seq, "lens"));
    void *o = c.flat(a[4], c.io(), qs, "o");
    float *lse = static_cast<float *>(c.flat(a[5], at::kFloat, rows, "lse"));
    void *d_o = c.flat(a[6], c.io(), qs, "do");
    void *dq = c.heads(a[7], qs, sdq, "dq"), *dk = c.heads(a[8], ks, sdk, "dk"), *dv = c.heads(a[9], ks, sdv, "dv");
    size_t bytes;
    void *ws = c.workspace(a[13], bytes);
    return c.run(rglru_local_attention_backward, q, k, v, lens, o, lse, d_o, dq, dk, dv, as_int(B, "q"),
                 as_int(T, "q"), as_int(Hq, "q"), as_int(Hkv, "k"), as_int(dh, "q"), sq, sk, sv, sdq,
                 sdk, sdv, arg_int(a[10]), arg_int(a[11]), arg_float(a[12]), c.dtype(), ws, bytes,
                 arg_stream(a[14]));
  });
}

// (q, k_pages, v_pages, block_table, lens, o, window, sinks, scale, workspace, stream)
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> long {
    Call c;
    const at::Tensor &qt = c.first(a[0], "q", 3);
    if (qt.dim() != 3) refuse(PyExc_ValueError, "q: expected [N, Hq, dh], got shape " + text(qt.sizes()));
    const Sizes qs = qt.sizes();
    const at::Tensor &pages = Call::tensor(a[1], "k_pages"), &table = Call::tensor(a[3], "block_table");
    if (pages.dim() != 4)
      refuse(PyExc_ValueError, "k_pages: expected [pages, page, Hkv, dh], got " + text(pages.sizes()));
    if (table.dim() != 2)
      refuse(PyExc_ValueError, "block_table: expected [N, max_pages], got " + text(table.sizes()));
    const int64_t N = qs[0], Hkv = pages.size(2);
    const int64_t pool[] = {pages.size(0), pages.size(1), Hkv, qs[2]}, tab[] = {N, table.size(1)}, per_seq[] = {N};
    long long sq;
    void *q = c.heads(a[0], qs, sq, "q");
    void *kp = c.flat(a[1], c.io(), pool, "k_pages"), *vp = c.flat(a[2], c.io(), pool, "v_pages");
    const int *bt = static_cast<int *>(c.flat(a[3], at::kInt, tab, "block_table"));
    const int *lens = static_cast<int *>(c.flat(a[4], at::kInt, per_seq, "lens"));
    void *o = c.flat(a[5], c.io(), qs, "o");
    size_t bytes;
    void *ws = c.workspace(a[9], bytes);
    return c.run(rglru_paged_attention, q, kp, vp, bt, lens, o, as_int(N, "q"), as_int(qs[1], "q"),
                 as_int(Hkv, "k_pages"), as_int(qs[2], "q"), sq, as_int(pool[0], "k_pages"),
                 as_int(pool[1], "k_pages"), as_int(tab[1], "block_table"), arg_int(a[6]), arg_int(a[7]),
                 arg_float(a[8]), c.dtype(), ws, bytes, arg_stream(a[10]));
  });
}

// ---- serving
constexpr c10::ScalarType kE4m3 = at::kFloat8_e4m3fn, kE8m0 = at::kFloat8_e8m0fnu;

// An e4m3 cache's sizes, from k_pages.
struct Pool {
  int64_t pages[4], scales[3];
};
Pool pool_of(PyObject *k_pages) {
  const at::Tensor &t = Call::tensor(k_pages, "k_pages");
  if (t.dim() != 4) refuse(PyExc_ValueError, "k_pages: expected [pages, page, Hkv, dh], got " + text(t.sizes()));
  Pool p;
  for (int i = 0; i < 4; ++i) p.pages[i] = t.size(i);
  for (int i = 0; i < 3; ++i) p.scales[i] = t.size(i);
  return p;
}
struct Cache {
  void *k, *v, *ks, *vs;
};
Cache cache_of(Call &c, const Pool &p, PyObject *const *a) {  // k_pages, v_pages, k_scales, v_scales
  for (int i = 0; i < 4; ++i) Call::tensor(a[i], "cache");    // (none is optional)
  return {c.flat(a[0], kE4m3, p.pages, "k_pages"), c.flat(a[1], kE4m3, p.pages, "v_pages"),
          c.flat(a[2], kE8m0, p.scales, "k_scales"), c.flat(a[3], kE8m0, p.scales, "v_scales")};
}

// (k, v, slots, k_pages, v_pages, k_scales, v_scales, stream)
PyObject *cache_quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> long {
    Call c;
    const at::Tensor &k = c.first(a[0], "k", 2);
    const Sizes ks = k.sizes(), lead = ks.slice(0, ks.size() - 2);
    const Pool p = pool_of(a[3]);
    if (p.pages[2] != ks[ks.size() - 2] || p.pages[3] != ks[ks.size() - 1])
      refuse(PyExc_ValueError, "k_pages: expected [pages, page, Hkv, dh] of k's heads, got " + text(p.pages));
    long long sk, sv;
    Call::tensor(a[1], "v");
    Call::tensor(a[2], "slots");
    void *pk = c.heads(a[0], ks, sk, "k"), *pv = c.heads(a[1], ks, sv, "v");
    const long long *slots = static_cast<long long *>(c.flat(a[2], at::kLong, lead, "slots"));
    const Cache m = cache_of(c, p, a + 3);
    const int64_t rows = k.numel() / std::max<int64_t>(1, p.pages[2] * p.pages[3]);
    return c.run(rglru_cache_quantize, pk, pv, slots, m.k, m.v, m.ks, m.vs, as_int(rows, "k"),
                 as_int(p.pages[2], "k"), as_int(p.pages[3], "k"), sk, sv,
                 static_cast<long long>(p.pages[0]) * p.pages[1], c.dtype(), arg_stream(a[7]));
  });
}

// (k_pages, v_pages, k_scales, v_scales, block_table, lens, starts, k_out, v_out, zero_rest, stream)
PyObject *cache_dequantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> long {
    Call c;
    const at::Tensor &out = c.first(a[7], "k_out", 3), &table = Call::tensor(a[4], "block_table");
    const Sizes os = out.sizes();
    const Pool p = pool_of(a[0]);
    if (os.size() != 4 || os[2] != p.pages[2] || os[3] != p.pages[3])
      refuse(PyExc_ValueError, "k_out: expected [B, T, Hkv, dh] of the cache's heads, got shape " + text(os));
    if (table.dim() != 2)
      refuse(PyExc_ValueError, "block_table: expected [B, max_pages], got " + text(table.sizes()));
    const int64_t tab[] = {os[0], table.size(1)}, per_seq[] = {os[0]};
    long long sk, sv;
    Call::tensor(a[5], "lens");
    Call::tensor(a[8], "v_out");
    const Cache m = cache_of(c, p, a);
    const int *bt = static_cast<int *>(c.flat(a[4], at::kInt, tab, "block_table"));
    const int *lens = static_cast<int *>(c.flat(a[5], at::kInt, per_seq, "lens"));
    const int *starts = static_cast<int *>(c.flat(a[6], at::kInt, per_seq, "starts"));
    void *ko = c.heads(a[7], os, sk, "k_out"), *vo = c.heads(a[8], os, sv, "v_out");
    return c.run(rglru_cache_dequantize, m.k, m.v, m.ks, m.vs, bt, lens, starts, ko, vo, as_int(os[0], "k_out"),
                 as_int(os[1], "k_out"), as_int(os[2], "k_out"), as_int(os[3], "k_out"), sk, sv,
                 as_int(p.pages[0], "k_pages"), as_int(p.pages[1], "k_pages"), as_int(tab[1], "block_table"),
                 a[9] == Py_True ? 1 : 0, c.dtype(), arg_stream(a[10]));
  });
}

void want_bf16(const Call &c, const char *name) {
  if (c.io() != at::kBFloat16)
    refuse(PyExc_ValueError, std::string(name) + ": expected torch.bfloat16, got " + text(c.io()));
}

// (q, k_pages, v_pages, k_scales, v_scales, block_table, lens, o, window, sinks, scale, workspace, stream)
PyObject *paged_attention_e4m3(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> long {
    Call c;
    const at::Tensor &qt = c.first(a[0], "q", 3), &table = Call::tensor(a[5], "block_table");
    want_bf16(c, "q");
    if (qt.dim() != 3) refuse(PyExc_ValueError, "q: expected [N, Hq, dh], got shape " + text(qt.sizes()));
    const Sizes qs = qt.sizes();
    Pool p = pool_of(a[1]);
    p.pages[3] = qs[2];
    if (table.dim() != 2)
      refuse(PyExc_ValueError, "block_table: expected [N, max_pages], got " + text(table.sizes()));
    const int64_t tab[] = {qs[0], table.size(1)}, per_seq[] = {qs[0]};
    long long sq;
    void *q = c.heads(a[0], qs, sq, "q");
    const Cache m = cache_of(c, p, a + 1);
    const int *bt = static_cast<int *>(c.flat(a[5], at::kInt, tab, "block_table"));
    const int *lens = static_cast<int *>(c.flat(a[6], at::kInt, per_seq, "lens"));
    void *o = c.flat(a[7], c.io(), qs, "o");
    size_t bytes;
    void *ws = c.workspace(a[11], bytes);
    return c.run(rglru_paged_attention_e4m3, q, m.k, m.v, m.ks, m.vs, bt, lens, o, as_int(qs[0], "q"),
                 as_int(qs[1], "q"), as_int(p.pages[2], "k_pages"), as_int(qs[2], "q"), sq,
                 as_int(p.pages[0], "k_pages"), as_int(p.pages[1], "k_pages"), as_int(tab[1], "block_table"),
                 arg_int(a[8]), arg_int(a[9]), arg_float(a[10]), ws, bytes, arg_stream(a[12]));
  });
}

// (q, k_pages, v_pages, k_scales, v_scales, prefix_table, prefix_len, block_table, lens, o, window, sinks, scale,
//  workspace, stream)
PyObject *prefix_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> long {
    Call c;
    const at::Tensor &qt = c.first(a[0], "q", 3), &table = Call::tensor(a[7], "block_table"),
                     &prefix = Call::tensor(a[5], "prefix_table");
    if (qt.dim() != 3) refuse(PyExc_ValueError, "q: expected [N, Hq, dh], got shape " + text(qt.sizes()));
    const Sizes qs = qt.sizes();
    Pool p = pool_of(a[1]);
    p.pages[3] = qs[2];
    if (table.dim() != 2)
      refuse(PyExc_ValueError, "block_table: expected [N, max_pages], got " + text(table.sizes()));
    if (prefix.dim() != 1)
      refuse(PyExc_ValueError, "prefix_table: expected [prefix_pages], got " + text(prefix.sizes()));
    const int64_t tab[] = {qs[0], table.size(1)}, per_seq[] = {qs[0]}, shared[] = {prefix.size(0)}, one[] = {1};
    long long sq;
    void *q = c.heads(a[0], qs, sq, "q");
    if ((a[3] == Py_None) != (a[4] == Py_None)) refuse(PyExc_ValueError, "k_scales, v_scales: both or none");
    const Cache m = a[3] == Py_None ? Cache{c.flat(a[1], c.io(), p.pages, "k_pages"),
                                            c.flat(a[2], c.io(), p.pages, "v_pages"), nullptr, nullptr}
                                    : cache_of(c, p, a + 1);
    const int *pt = static_cast<int *>(c.flat(a[5], at::kInt, shared, "prefix_table"));
    const int *pl = static_cast<int *>(c.flat(a[6], at::kInt, one, "prefix_len"));
    const int *bt = static_cast<int *>(c.flat(a[7], at::kInt, tab, "block_table"));
    const int *lens = static_cast<int *>(c.flat(a[8], at::kInt, per_seq, "lens"));
    void *o = c.flat(a[9], c.io(), qs, "o");
    size_t bytes;
    void *ws = c.workspace(a[13], bytes);
    return c.run(rglru_prefix_attention, q, m.k, m.v, m.ks, m.vs, pt, pl, bt, lens, o, as_int(qs[0], "q"),
                 as_int(qs[1], "q"), as_int(p.pages[2], "k_pages"), as_int(qs[2], "q"), sq,
                 as_int(p.pages[0], "k_pages"), as_int(p.pages[1], "k_pages"), as_int(shared[0], "prefix_table"),
                 as_int(tab[1], "block_table"), arg_int(a[10]), arg_int(a[11]), arg_float(a[12]), c.dtype(), ws, bytes,
                 arg_stream(a[14]));
  });
}

// log_decay: [H], or one value of each row and head.
const float *decays(Call &c, PyObject *o, Sizes lead, int64_t H, int &gated) {
  const at::Tensor &t = Call::tensor(o, "log_decay");
  Shape per_row(lead.begin(), lead.end());
  per_row.push_back(H);
  gated = t.dim() == 1 ? 0 : 1;
  const int64_t per_head[] = {H};
  return static_cast<float *>(c.flat(o, at::kFloat, gated ? Sizes(per_row) : Sizes(per_head), "log_decay"));
}

// (q, k, v, log_decay, lens, state, o, state_out, scale, workspace, stream)
PyObject *linear_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> long {
    Call c;
    const at::Tensor &q = c.first(a[0], "q", 3), &v = Call::tensor(a[2], "v");
    if (q.dim() != 4) refuse(PyExc_ValueError, "q: expected [B, T, Hk, dk], got shape " + text(q.sizes()));
    if (v.dim() != 4) refuse(PyExc_ValueError, "v: expected [B, T, H, dv], got shape " + text(v.sizes()));
    const Sizes qs = q.sizes();
    const int64_t B = qs[0], T = qs[1], Hk = qs[2], dk = qs[3], H = v.size(2), dv = v.size(3);
    const int64_t vs[] = {B, T, H, dv}, st[] = {B, H, dk, dv}, per_seq[] = {B};
    long long sq, sk, sv;
    Call::tensor(a[1], "k");
    void *pq = c.heads(a[0], qs, sq, "q"), *pk = c.heads(a[1], qs, sk, "k"), *pv = c.heads(a[2], vs, sv, "v");
    int gated;
    const float *g = decays(c, a[3], qs.slice(0, 2), H, gated);
    const int *lens = static_cast<int *>(c.flat(a[4], at::kInt, per_seq, "lens"));
    const float *s0 = static_cast<float *>(c.flat(a[5], at::kFloat, st, "state"));
    void *o = c.flat(a[6], c.io(), vs, "o");
    float *so = static_cast<float *>(c.flat(a[7], at::kFloat, st, "state_out"));
    size_t bytes;
    void *ws = c.workspace(a[9], bytes);
    return c.run(rglru_linear_attention, pq, pk, pv, g, lens, s0, o, so, as_int(B, "q"), as_int(T, "q"),
                 as_int(Hk, "q"), as_int(H, "v"), as_int(dk, "q"), as_int(dv, "v"), sq, sk, sv, gated,
                 arg_float(a[8]), c.dtype(), ws, bytes, arg_stream(a[10]));
  });
}

// (q, k, v, log_decay, state, state_out, o, scale, stream)
PyObject *linear_attention_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> long {
    Call c;
    const at::Tensor &q = c.first(a[0], "q", 3), &v = Call::tensor(a[2], "v");
    if (q.dim() != 3) refuse(PyExc_ValueError, "q: expected [N, Hk, dk], got shape " + text(q.sizes()));
    if (v.dim() != 3) refuse(PyExc_ValueError, "v: expected [N, H, dv], got shape " + text(v.sizes()));
    const Sizes qs = q.sizes();
    const int64_t N = qs[0], Hk = qs[1], dk = qs[2], H = v.size(1), dv = v.size(2);
    const int64_t vs[] = {N, H, dv}, st[] = {N, H, dk, dv};
    long long sq, sk, sv;
    Call::tensor(a[1], "k");
    void *pq = c.heads(a[0], qs, sq, "q"), *pk = c.heads(a[1], qs, sk, "k"), *pv = c.heads(a[2], vs, sv, "v");
    int gated;
    const float *g = decays(c, a[3], qs.slice(0, 1), H, gated);
    const float *s0 = static_cast<float *>(c.flat(a[4], at::kFloat, st, "state"));
    float *so = static_cast<float *>(c.flat(a[5], at::kFloat, st, "state_out"));
    void *o = c.flat(a[6], c.io(), vs, "o");
    return c.run(rglru_linear_attention_step, pq, pk, pv, g, s0, so, o, as_int(N, "q"), as_int(Hk, "q"),
                 as_int(H, "v"), as_int(dk, "q"), as_int(dv, "v"), sq, sk, sv, gated, arg_float(a[7]), c.dtype(),
                 arg_stream(a[8]));
  });
}

template <typename F> PyObject *made(F f) {
  try {
    return THPVariable_Wrap(f());
  } catch (const Refused &) {
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (t): an uninitialised contiguous tensor of t's shape, type and device
PyObject *empty_as(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return made([&] {
    if (n != 1) refuse(PyExc_TypeError, "wrong number of arguments");
    const at::Tensor &t = Call::tensor(a[0], "t");
    return at::empty(t.sizes(), t.options().requires_grad(false));
  });
}

// (t, bytes): an uninitialised workspace on t's device
PyObject *empty_bytes(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return made([&] {
    if (n != 2) refuse(PyExc_TypeError, "wrong number of arguments");
    const at::Tensor &t = Call::tensor(a[0], "t");
    const long long bytes = PyLong_AsLongLong(a[1]);
    if (bytes == -1 && PyErr_Occurred()) throw Refused{};
    return at::empty({bytes}, t.options().requires_grad(false).dtype(at::kByte));
  });
}

#define RGLRU_METHOD(f) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {RGLRU_METHOD(qk_norm_rope),    RGLRU_METHOD(qk_norm_rope_backward),
                         RGLRU_METHOD(local_attention), RGLRU_METHOD(local_attention_backward),
                         RGLRU_METHOD(paged_attention), RGLRU_METHOD(cache_quantize),
                         RGLRU_METHOD(cache_dequantize), RGLRU_METHOD(paged_attention_e4m3),
                         RGLRU_METHOD(prefix_attention), RGLRU_METHOD(linear_attention),
                         RGLRU_METHOD(linear_attention_step), RGLRU_METHOD(empty_as),
                         RGLRU_METHOD(empty_bytes),     {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rglru_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rglru_torch() { return PyModule_Create(&module); }
