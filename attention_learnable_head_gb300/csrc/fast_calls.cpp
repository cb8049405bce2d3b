// Native side of the conveniences of attn_sink_step.h (page_plan, qkv_rope,
// qkv_rope_backward, extend) and attn_sink_cache.h (decode_shared, page_bounds,
// select_pages, decode_pages, key_mass, evict): checks the arguments, allocates the outputs and the
// workspace on the current stream and calls the C entry point.  A small call's
// kernels take 3 to 10 us; with these steps in Python (ctypes, torch.empty) the
// host took longer than they did.  A call, host and device, Python -> native:
// page_plan of 128 sequences 28 -> 6.2 us, qkv_rope of 128 tokens into the pages
// 22 -> 6.3 us, qkv_rope_backward with norm 43 -> 11.9 us; the larger calls, bound
// by their kernels, are as before.
//
// Only the plain case is handled here: CUDA tensors of the current device, on its
// current stream, with the expected types, shapes and layouts.  For any other
// call the functions return None, and binding.py goes through its own checks,
// which name what is wrong.  A non-zero status of the library is returned as an
// int.  Each function mirrors the one of its name in binding.py.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "attn_sink_cache.h"
#include "attn_sink_step.h"

namespace {

// The library's entry points (set by init with the addresses ctypes resolved).
decltype(&attn_sink_page_plan) f_plan;
decltype(&attn_sink_qkv_rope) f_rope;
decltype(&attn_sink_qkv_rope_bwd_workspace_size) f_rope_ws;
decltype(&attn_sink_qkv_rope_bwd) f_rope_bwd;
decltype(&attn_sink_extend_workspace_size) f_extend_ws;
decltype(&attn_sink_extend) f_extend;
decltype(&attn_sink_decode_shared_workspace_size) f_shared_ws;
decltype(&attn_sink_decode_shared) f_shared;
decltype(&attn_sink_page_bounds) f_bounds;
decltype(&attn_sink_select_pages_workspace_size) f_select_ws;
decltype(&attn_sink_select_pages) f_select;
decltype(&attn_sink_decode_pages_workspace_size) f_pages_ws;
decltype(&attn_sink_decode_pages) f_pages;
decltype(&attn_sink_key_mass) f_mass;
decltype(&attn_sink_evict_workspace_size) f_evict_ws;
decltype(&attn_sink_evict) f_evict;

// A tensor argument; null for None or anything else.
const at::Tensor* tensor(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// A contiguous tensor of this type and device with these sizes (-1: any)?
bool fits(const at::Tensor* t, at::ScalarType type, c10::Device dev,
          std::initializer_list<int64_t> sizes) {
  if (t == nullptr || t->scalar_type() != type || t->device() != dev ||
      t->dim() != (int64_t)sizes.size() || !t->is_contiguous())
    return false;
  int64_t i = 0;
  for (int64_t s : sizes) {
    const int64_t n = t->size(i++);
    if (n > INT_MAX || (s >= 0 && n != s)) return false;
  }
  return true;
}

// Is the tensor on the current CUDA device?
bool here(const at::Tensor* t) {
  return t != nullptr && t->is_cuda() && t->get_device() == c10::cuda::current_device();
}

// The interpreter lock is given up around allocations and launches, which may wait.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
};

void* current_stream(const at::Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
}

at::Tensor make(const at::Tensor& like, at::ScalarType type, at::IntArrayRef sizes) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(like.device()));
}

// Tensors that live in one buffer, each at a multiple of 256 bytes: a call's small
// outputs from one allocation (an allocation takes the host 0.7 us, a tensor on it
// 0.1 us).
int64_t padded(int64_t bytes) { return (bytes + 255) / 256 * 256; }
at::Tensor part(const at::Tensor& buffer, int64_t at, at::ScalarType type,
                at::IntArrayRef sizes) {
  const caffe2::TypeMeta meta = c10::scalarTypeToTypeMeta(type);
  auto impl = c10::make_intrusive<c10::TensorImpl>(
      c10::TensorImpl::VIEW, c10::Storage(buffer.storage()), buffer.key_set(), meta);
  impl->set_storage_offset(at / (int64_t)meta.itemsize());
  impl->set_sizes_contiguous(sizes);
  return at::Tensor(std::move(impl));
}

// An int argument in [INT_MIN, INT_MAX].
bool integer(PyObject* o, int* out) {
  if (!PyLong_Check(o)) return false;
  int over = 0;
  const long v = PyLong_AsLongAndOverflow(o, &over);
  if (over != 0 || v < INT_MIN || v > INT_MAX) return false;
  *out = (int)v;
  return true;
}
bool real(PyObject* o, float* out) {
  if (!PyFloat_Check(o) && !PyLong_Check(o)) return false;
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  *out = (float)v;
  return true;
}
bool truth(PyObject* o, int* out) {
  if (!PyBool_Check(o)) return false;
  *out = o == Py_True;
  return true;
}

PyObject* none() { Py_RETURN_NONE; }

PyObject* tuple(std::initializer_list<const at::Tensor*> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (r == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor* t : ts) {
    PyObject* o = t != nullptr ? THPVariable_Wrap(*t) : (Py_INCREF(Py_None), Py_None);
    if (o == nullptr) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

void* data(const at::Tensor* t) { return t != nullptr ? t->data_ptr() : nullptr; }
template <typename T>
T* data_as(const at::Tensor* t) {
  return static_cast<T*>(data(t));
}

PyObject* page_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  attn_sink_plan_params p;
  const at::Tensor *cached, *fresh, *free, *table;
  if (n != 7 || !here(cached = tensor(a[0])) || !integer(a[4], &p.page_size) ||
      !integer(a[5], &p.num_pages) || !integer(a[6], &p.max_tokens) || p.max_tokens < 0)
    return none();
  const c10::Device dev = cached->device();
  if (!fits(cached, at::kInt, dev, {-1})) return none();
  const int64_t b = cached->size(0);
  if (!fits(fresh = tensor(a[1]), at::kInt, dev, {b}) ||
      !fits(free = tensor(a[2]), at::kInt, dev, {-1}) ||
      !fits(table = tensor(a[3]), at::kInt, dev, {b, -1}))
    return none();
  p.batch = (int)b;
  p.max_pages = (int)table->size(1);
  p.num_free = (int)free->size(0);
  at::Tensor slots, positions, cu, lens, needed;
  int st;
  {
    const Unlocked unlocked;
    const int64_t at1 = padded(8ll * p.max_tokens), at2 = at1 + padded(4ll * p.max_tokens);
    const int64_t at3 = at2 + padded(4 * (b + 1)), at4 = at3 + padded(4 * b);
    const at::Tensor all = make(*cached, at::kByte, {at4 + 4});
    slots = part(all, 0, at::kLong, {p.max_tokens});
    positions = part(all, at1, at::kInt, {p.max_tokens});
    cu = part(all, at2, at::kInt, {b + 1});
    lens = part(all, at3, at::kInt, {b});
    needed = part(all, at4, at::kInt, {1});
    st = f_plan(&p, data_as<int>(cached), data_as<int>(fresh), data_as<int>(free),
                data_as<int>(table), data_as<long long>(&slots), data_as<int>(&positions),
                data_as<int>(&cu), data_as<int>(&lens), data_as<int>(&needed),
                current_stream(*cached));
  }
  if (st != 0) return PyLong_FromLong(st);
  return tuple({&slots, &positions, &cu, &lens, &needed});
  END_HANDLE_TH_ERRORS
}

// Arguments that qkv_rope and its backward share: qkv, positions, inv_freq,
// heads_q, heads_kv, q_weight, k_weight, eps, pair_axis, interleaved, amplitude.
struct Rope {
  attn_sink_rope_params p;
  const at::Tensor *qkv, *positions, *inv_freq, *q_weight, *k_weight;
  int64_t t, rows;
};

bool rope_args(PyObject* const* a, Rope* r) {
  std::memset(&r->p, 0, sizeof(r->p));
  attn_sink_rope_params& p = r->p;
  r->qkv = tensor(a[0]);
  r->positions = tensor(a[1]);
  r->inv_freq = tensor(a[2]);
  r->q_weight = tensor(a[5]);
  r->k_weight = tensor(a[6]);
  if (!here(r->qkv) || r->positions == nullptr || !integer(a[3], &p.heads_q) ||
      !integer(a[4], &p.heads_kv) || p.heads_q < 1 || p.heads_kv < 1 || p.heads_q > (1 << 20) ||
      p.heads_kv > (1 << 20) || !real(a[7], &p.eps) || !truth(a[9], &p.interleaved) ||
      !real(a[10], &p.amplitude) || (r->q_weight == nullptr && a[5] != Py_None) ||
      (r->k_weight == nullptr && a[6] != Py_None) ||
      (r->q_weight == nullptr) != (r->k_weight == nullptr))
    return false;
  const at::Tensor& x = *r->qkv;
  r->rows = p.heads_q + 2ll * p.heads_kv;
  if (x.scalar_type() != at::kBFloat16 || x.dim() != 3 || x.size(1) != r->rows ||
      x.size(2) != 64 || x.size(0) > INT_MAX)
    return false;
  r->t = x.size(0);
  p.tokens = (int)r->t;
  p.head_dim = 64;
  int64_t stride = r->rows * 64;             // of one token or none: its own means nothing
  if (r->t > 0) {
    if (x.stride(2) != 1 || x.stride(1) != 64) return false;
    if (r->t > 1) stride = x.stride(0);
    if (stride < r->rows * 64 || stride % 8 != 0) return false;
  }
  p.q_stride = p.k_stride = p.v_stride = stride;
  const c10::Device dev = x.device();
  const bool flat = r->positions->dim() == 1;
  if (!flat && r->positions->dim() != 2) return false;
  p.num_axes = flat ? 1 : (int)std::min<int64_t>(r->positions->size(0), INT_MAX);
  if (!(flat ? fits(r->positions, at::kInt, dev, {r->t})
             : fits(r->positions, at::kInt, dev, {-1, r->t})) ||
      !fits(r->inv_freq, at::kFloat, dev, {-1}))
    return false;
  const int64_t pairs = r->inv_freq->size(0);
  if (pairs > 32) return false;
  p.rotary_dim = 2 * (int)pairs;
  if (a[8] == Py_None) {
    if (p.num_axes > 1) return false;
  } else {
    if (!PyList_Check(a[8]) || PyList_GET_SIZE(a[8]) != pairs) return false;
    for (int64_t i = 0; i < pairs; ++i) {
      int axis;
      if (!integer(PyList_GET_ITEM(a[8], i), &axis) || axis < 0 || axis >= p.num_axes ||
          axis > 255)
        return false;
      p.pair_axis[i] = (unsigned char)axis;
    }
  }
  if (r->q_weight != nullptr) {
    const at::ScalarType kind = r->q_weight->scalar_type();
    if ((kind != at::kFloat && kind != at::kBFloat16) || !fits(r->q_weight, kind, dev, {64}) ||
        !fits(r->k_weight, kind, dev, {64}))
      return false;
    p.norm = 1;
    p.weight_bf16 = kind == at::kBFloat16;
  }
  return true;
}

PyObject* qkv_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Rope r;
  if (n != 15 || !rope_args(a, &r)) return none();
  attn_sink_rope_params& p = r.p;
  const c10::Device dev = r.qkv->device();
  const at::Tensor *slots = tensor(a[11]), *kc = tensor(a[12]), *vc = tensor(a[13]);
  int keep = slots == nullptr;
  if (a[14] != Py_None && !truth(a[14], &keep)) return none();
  if (slots != nullptr) {
    if (!fits(slots, at::kLong, dev, {r.t}) ||
        !fits(kc, at::kBFloat16, dev, {-1, -1, p.heads_kv, 64}) ||
        !fits(vc, at::kBFloat16, dev, {kc->size(0), kc->size(1), p.heads_kv, 64}))
      return none();
    p.num_pages = (int)kc->size(0);
    p.page_size = (int)kc->size(1);
  } else if (a[11] != Py_None || a[12] != Py_None || a[13] != Py_None) {
    return none();
  }
  at::Tensor q, k, v;
  int st;
  {
    const Unlocked unlocked;
    q = make(*r.qkv, at::kBFloat16, {r.t, p.heads_q, 64});
    if (keep) {
      k = make(*r.qkv, at::kBFloat16, {r.t, p.heads_kv, 64});
      v = make(*r.qkv, at::kBFloat16, {r.t, p.heads_kv, 64});
    }
    const char* base = data_as<char>(r.qkv);
    const char* kp = base + 128ll * p.heads_q;
    st = f_rope(&p, base, kp, kp + 128ll * p.heads_kv, data_as<int>(r.positions),
                data_as<float>(r.inv_freq), data(r.q_weight), data(r.k_weight),
                data_as<long long>(slots), q.data_ptr(), keep ? k.data_ptr() : nullptr,
                keep ? v.data_ptr() : nullptr, data(kc), data(vc), current_stream(*r.qkv));
  }
  if (st != 0) return PyLong_FromLong(st);
  return tuple({&q, keep ? &k : nullptr, keep ? &v : nullptr});
  END_HANDLE_TH_ERRORS
}

PyObject* qkv_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Rope r;
  if (n != 14 || !rope_args(a, &r)) return none();
  attn_sink_rope_params& p = r.p;
  const c10::Device dev = r.qkv->device();
  const at::Tensor *dq = tensor(a[11]), *dk = tensor(a[12]), *dv = tensor(a[13]);
  if (dq == nullptr) return none();
  const at::ScalarType kind = dq->scalar_type();
  if ((kind != at::kFloat && kind != at::kBFloat16) ||
      !fits(dq, kind, dev, {r.t, p.heads_q, 64}) || !fits(dk, kind, dev, {r.t, p.heads_kv, 64}) ||
      !fits(dv, kind, dev, {r.t, p.heads_kv, 64}))
    return none();
  p.grad_dtype = kind == at::kFloat;
  at::Tensor dqkv, dwq, dwk;
  int st;
  {
    const Unlocked unlocked;
    at::Tensor ws;
    size_t bytes = 0;
    dqkv = make(*r.qkv, at::kBFloat16, {r.t, r.rows, 64});
    if (p.norm) {
      const at::Tensor dw = make(*r.qkv, at::kFloat, {128});
      dwq = part(dw, 0, at::kFloat, {64});
      dwk = part(dw, 256, at::kFloat, {64});
      bytes = f_rope_ws(&p);
      ws = make(*r.qkv, at::kByte, {(int64_t)bytes});
    }
    const char* src = data_as<char>(r.qkv);
    char* dst = data_as<char>(&dqkv);
    const int64_t kq = 128ll * p.heads_q, kk = 128ll * p.heads_kv, row = r.rows * 64;
    st = f_rope_bwd(&p, src, src + kq, data_as<int>(r.positions), data_as<float>(r.inv_freq),
                    data(r.q_weight), data(r.k_weight), data(dq), data(dk), data(dv), dst,
                    dst + kq, dst + kq + kk, row, row, row,
                    p.norm ? data_as<float>(&dwq) : nullptr,
                    p.norm ? data_as<float>(&dwk) : nullptr, p.norm ? ws.data_ptr() : nullptr,
                    bytes, current_stream(*r.qkv));
  }
  if (st != 0) return PyLong_FromLong(st);
  return tuple({&dqkv, p.norm ? &dwq : nullptr, p.norm ? &dwk : nullptr});
  END_HANDLE_TH_ERRORS
}

PyObject* extend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  attn_sink_extend_params p;
  std::memset(&p, 0, sizeof(p));
  const at::Tensor *q, *kc, *vc, *table, *lens, *cu, *sink;
  if (n != 11 || !here(q = tensor(a[0])) || !integer(a[7], &p.window) ||
      !real(a[8], &p.softmax_scale))
    return none();
  const c10::Device dev = q->device();
  if (!fits(q, at::kBFloat16, dev, {-1, -1, 64}) ||
      !fits(kc = tensor(a[1]), at::kBFloat16, dev, {-1, -1, -1, 64}) ||
      !fits(vc = tensor(a[2]), at::kBFloat16, dev, {kc->size(0), kc->size(1), kc->size(2), 64}) ||
      !fits(lens = tensor(a[4]), at::kInt, dev, {-1}) ||
      !fits(table = tensor(a[3]), at::kInt, dev, {lens->size(0), -1}) ||
      !fits(cu = tensor(a[5]), at::kInt, dev, {lens->size(0) + 1}) ||
      !fits(sink = tensor(a[6]), at::kFloat, dev, {q->size(1)}))
    return none();
  p.batch = (int)lens->size(0);
  p.total_q = (int)q->size(0);
  p.heads_q = (int)q->size(1);
  p.heads_kv = (int)kc->size(2);
  p.head_dim = 64;
  p.page_size = (int)kc->size(1);
  p.num_pages = (int)kc->size(0);
  p.max_pages = (int)table->size(1);
  const at::Tensor *given_out = tensor(a[9]), *given_lse = tensor(a[10]);
  if ((a[9] != Py_None && !fits(given_out, at::kBFloat16, dev, {p.total_q, p.heads_q, 64})) ||
      (a[10] != Py_None && !fits(given_lse, at::kFloat, dev, {p.heads_q, p.total_q})))
    return none();
  at::Tensor out, lse;
  int st;
  {
    const Unlocked unlocked;
    out = given_out ? *given_out : make(*q, at::kBFloat16, {p.total_q, p.heads_q, 64});
    lse = given_lse ? *given_lse : make(*q, at::kFloat, {p.heads_q, p.total_q});
    const size_t bytes = f_extend_ws(&p);
    const at::Tensor ws = make(*q, at::kByte, {(int64_t)bytes});
    st = f_extend(&p, data(q), data(kc), data(vc), data_as<int>(table), data_as<int>(lens),
                  data_as<int>(cu), data_as<float>(sink), out.data_ptr(), data_as<float>(&lse),
                  ws.data_ptr(), bytes, current_stream(*q));
  }
  if (st != 0) return PyLong_FromLong(st);
  return tuple({&out, &lse});
  END_HANDLE_TH_ERRORS
}

// A paged cache and its tables: k_cache and (null: none) v_cache [pages, page size, kv
// heads, 64], block_table [B, columns], seq_lens [B]; fills the fields all params have.
template <typename P>
bool paged(const at::Tensor* kc, const at::Tensor* vc, bool values, const at::Tensor* table,
           const at::Tensor* lens, P* p) {
  if (!here(kc)) return false;
  const c10::Device dev = kc->device();
  if (!fits(kc, at::kBFloat16, dev, {-1, -1, -1, 64}) ||
      (values && !fits(vc, at::kBFloat16, dev, {kc->size(0), kc->size(1), kc->size(2), 64})) ||
      !fits(lens, at::kInt, dev, {-1}) || !fits(table, at::kInt, dev, {lens->size(0), -1}))
    return false;
  p->batch = (int)lens->size(0);
  p->heads_kv = (int)kc->size(2);
  p->head_dim = 64;
  p->page_size = (int)kc->size(1);
  p->num_pages = (int)kc->size(0);
  p->max_pages = (int)table->size(1);
  return true;
}

// The caller's own out and lse (null: none), if they are what q's call writes.
bool results(PyObject* o, PyObject* l, const at::Tensor& q, const at::Tensor** out,
             const at::Tensor** lse) {
  *out = tensor(o);
  *lse = tensor(l);
  return (o == Py_None || fits(*out, at::kBFloat16, q.device(), {q.size(0), q.size(1), 64})) &&
         (l == Py_None || fits(*lse, at::kFloat, q.device(), {q.size(1), q.size(0)}));
}

PyObject* decode_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  attn_sink_shared_params p;
  std::memset(&p, 0, sizeof(p));
  const at::Tensor *q, *kc, *vc, *table, *lens, *cu, *prefix, *sink, *given_out, *given_lse;
  if (n != 11 || !paged(kc = tensor(a[1]), vc = tensor(a[2]), true, table = tensor(a[3]),
                        lens = tensor(a[4]), &p) ||
      !real(a[8], &p.softmax_scale))
    return none();
  const c10::Device dev = kc->device();
  if (!fits(q = tensor(a[0]), at::kBFloat16, dev, {p.batch, -1, 64}) ||
      !fits(prefix = tensor(a[6]), at::kInt, dev, {-1}) ||
      !fits(cu = tensor(a[5]), at::kInt, dev, {prefix->size(0) + 1}) ||
      !fits(sink = tensor(a[7]), at::kFloat, dev, {q->size(1)}) ||
      !results(a[9], a[10], *q, &given_out, &given_lse))
    return none();
  p.num_groups = (int)prefix->size(0);
  p.heads_q = (int)q->size(1);
  at::Tensor out, lse;
  int st;
  {
    const Unlocked unlocked;
    out = given_out ? *given_out : make(*q, at::kBFloat16, {p.batch, p.heads_q, 64});
    lse = given_lse ? *given_lse : make(*q, at::kFloat, {p.heads_q, p.batch});
    const size_t bytes = f_shared_ws(&p);
    const at::Tensor ws = make(*q, at::kByte, {(int64_t)bytes});
    st = f_shared(&p, data(q), data(kc), data(vc), data_as<int>(table), data_as<int>(lens),
                  data_as<int>(cu), data_as<int>(prefix), data_as<float>(sink), out.data_ptr(),
                  data_as<float>(&lse), ws.data_ptr(), bytes, current_stream(*q));
  }
  if (st != 0) return PyLong_FromLong(st);
  return tuple({&out, &lse});
  END_HANDLE_TH_ERRORS
}

PyObject* page_bounds(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  attn_sink_bounds_params p;
  const at::Tensor *kc, *table, *cached, *lens, *bounds;
  if (n != 5 || !paged(kc = tensor(a[0]), nullptr, false, table = tensor(a[1]),
                       lens = tensor(a[3]), &p))
    return none();
  const c10::Device dev = kc->device();
  if (!fits(cached = tensor(a[2]), at::kInt, dev, {p.batch}) ||
      !fits(bounds = tensor(a[4]), at::kBFloat16, dev, {p.num_pages, p.heads_kv, 2, 64}))
    return none();
  int st;
  {
    const Unlocked unlocked;
    st = f_bounds(&p, data(kc), data_as<int>(table), data_as<int>(cached), data_as<int>(lens),
                  data(bounds), current_stream(*kc));
  }
  return PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

PyObject* select_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  attn_sink_select_params p;
  const at::Tensor *q, *bounds, *table, *lens;
  if (n != 8 || !here(q = tensor(a[0])) || !integer(a[4], &p.count) || p.count < 1 ||
      !integer(a[5], &p.page_size) || !integer(a[6], &p.keep_first) ||
      !integer(a[7], &p.keep_last))
    return none();
  const c10::Device dev = q->device();
  if (!fits(lens = tensor(a[3]), at::kInt, dev, {-1}) ||
      !fits(q, at::kBFloat16, dev, {lens->size(0), -1, 64}) ||
      !fits(bounds = tensor(a[1]), at::kBFloat16, dev, {-1, -1, 2, 64}) ||
      !fits(table = tensor(a[2]), at::kInt, dev, {lens->size(0), -1}))
    return none();
  p.batch = (int)lens->size(0);
  p.heads_q = (int)q->size(1);
  p.heads_kv = (int)bounds->size(1);
  p.head_dim = 64;
  p.num_pages = (int)bounds->size(0);
  p.max_pages = (int)table->size(1);
  at::Tensor selected;
  int st;
  {
    const Unlocked unlocked;
    selected = make(*q, at::kInt, {p.batch, p.heads_kv, p.count});
    const size_t bytes = f_select_ws(&p);
    const at::Tensor ws = make(*q, at::kByte, {(int64_t)bytes});
    st = f_select(&p, data(q), data(bounds), data_as<int>(table), data_as<int>(lens),
                  data_as<int>(&selected), ws.data_ptr(), bytes, current_stream(*q));
  }
  if (st != 0) return PyLong_FromLong(st);
  return THPVariable_Wrap(selected);
  END_HANDLE_TH_ERRORS
}

PyObject* decode_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  attn_sink_pages_params p;
  const at::Tensor *q, *kc, *vc, *table, *lens, *selected, *sink, *given_out, *given_lse;
  if (n != 10 || !paged(kc = tensor(a[1]), vc = tensor(a[2]), true, table = tensor(a[3]),
                        lens = tensor(a[4]), &p) ||
      !real(a[7], &p.softmax_scale))
    return none();
  const c10::Device dev = kc->device();
  if (!fits(q = tensor(a[0]), at::kBFloat16, dev, {p.batch, -1, 64}) ||
      !fits(selected = tensor(a[5]), at::kInt, dev, {p.batch, p.heads_kv, -1}) ||
      !fits(sink = tensor(a[6]), at::kFloat, dev, {q->size(1)}) ||
      !results(a[8], a[9], *q, &given_out, &given_lse))
    return none();
  p.heads_q = (int)q->size(1);
  p.count = (int)selected->size(2);
  at::Tensor out, lse;
  int st;
  {
    const Unlocked unlocked;
    out = given_out ? *given_out : make(*q, at::kBFloat16, {p.batch, p.heads_q, 64});
    lse = given_lse ? *given_lse : make(*q, at::kFloat, {p.heads_q, p.batch});
    const size_t bytes = f_pages_ws(&p);
    const at::Tensor ws = make(*q, at::kByte, {(int64_t)bytes});
    st = f_pages(&p, data(q), data(kc), data(vc), data_as<int>(table), data_as<int>(lens),
                 data_as<int>(selected), data_as<float>(sink), out.data_ptr(),
                 data_as<float>(&lse), ws.data_ptr(), bytes, current_stream(*q));
  }
  if (st != 0) return PyLong_FromLong(st);
  return tuple({&out, &lse});
  END_HANDLE_TH_ERRORS
}

PyObject* key_mass(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  attn_sink_mass_params p;
  const at::Tensor *q, *kc, *table, *lens, *cu, *lse, *mass;
  if (n != 9 || !paged(kc = tensor(a[1]), nullptr, false, table = tensor(a[2]),
                       lens = tensor(a[3]), &p) ||
      !truth(a[7], &p.accumulate) || !real(a[8], &p.softmax_scale))
    return none();
  const c10::Device dev = kc->device();
  if (!fits(q = tensor(a[0]), at::kBFloat16, dev, {-1, -1, 64}) ||
      !fits(cu = tensor(a[4]), at::kInt, dev, {p.batch + 1ll}) ||
      !fits(lse = tensor(a[5]), at::kFloat, dev, {q->size(1), q->size(0)}) ||
      !fits(mass = tensor(a[6]), at::kFloat, dev, {p.batch, p.heads_kv, -1}))
    return none();
  p.total_q = (int)q->size(0);
  p.heads_q = (int)q->size(1);
  p.max_keys = (int)mass->size(2);
  int st;
  {
    const Unlocked unlocked;
    st = f_mass(&p, data(q), data(kc), data_as<int>(table), data_as<int>(lens),
                data_as<int>(cu), data_as<float>(lse), data_as<float>(mass), current_stream(*q));
  }
  return PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  attn_sink_evict_params p;
  const at::Tensor *kc, *vc, *table, *lens, *mass;
  if (n != 8 || !paged(kc = tensor(a[0]), vc = tensor(a[1]), true, table = tensor(a[2]),
                       lens = tensor(a[3]), &p) ||
      !integer(a[5], &p.budget) || !integer(a[6], &p.keep_first) || !integer(a[7], &p.keep_last) ||
      !fits(mass = tensor(a[4]), at::kFloat, kc->device(), {p.batch, p.heads_kv, -1}) ||
      table->numel() > INT_MAX)
    return none();
  p.max_keys = (int)mass->size(2);
  p.max_freed = (int)table->numel();
  at::Tensor left, fewer, freed, count;
  int st;
  {
    const Unlocked unlocked;
    left = make(*mass, at::kFloat, mass->sizes());
    const int64_t at1 = padded(4ll * p.max_freed), at2 = at1 + padded(4ll * p.batch);
    const at::Tensor all = make(*kc, at::kByte, {at2 + 4});
    freed = part(all, 0, at::kInt, {p.max_freed});
    fewer = part(all, at1, at::kInt, {p.batch});
    count = part(all, at2, at::kInt, {1});
    const size_t bytes = f_evict_ws(&p);
    const at::Tensor ws = make(*kc, at::kByte, {(int64_t)bytes});
    st = f_evict(&p, data(kc), data(vc), data_as<int>(table), data_as<int>(lens),
                 data_as<float>(mass), data_as<float>(&left), data_as<int>(&fewer),
                 data_as<int>(&freed), data_as<int>(&count), ws.data_ptr(), bytes,
                 current_stream(*kc));
  }
  if (st != 0) return PyLong_FromLong(st);
  return tuple({&fewer, &left, &freed, &count});
  END_HANDLE_TH_ERRORS
}

// init(addresses of the entry points, in the order of their declaration above)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kCalls = 16;
  void* f[kCalls];
  if (n != kCalls) {
    PyErr_SetString(PyExc_TypeError, "init takes sixteen addresses");
    return nullptr;
  }
  for (int i = 0; i < kCalls; ++i)
    if ((f[i] = PyLong_AsVoidPtr(a[i])) == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  f_plan = reinterpret_cast<decltype(f_plan)>(f[0]);
  f_rope = reinterpret_cast<decltype(f_rope)>(f[1]);
  f_rope_ws = reinterpret_cast<decltype(f_rope_ws)>(f[2]);
  f_rope_bwd = reinterpret_cast<decltype(f_rope_bwd)>(f[3]);
  f_extend_ws = reinterpret_cast<decltype(f_extend_ws)>(f[4]);
  f_extend = reinterpret_cast<decltype(f_extend)>(f[5]);
  f_shared_ws = reinterpret_cast<decltype(f_shared_ws)>(f[6]);
  f_shared = reinterpret_cast<decltype(f_shared)>(f[7]);
  f_bounds = reinterpret_cast<decltype(f_bounds)>(f[8]);
  f_select_ws = reinterpret_cast<decltype(f_select_ws)>(f[9]);
  f_select = reinterpret_cast<decltype(f_select)>(f[10]);
  f_pages_ws = reinterpret_cast<decltype(f_pages_ws)>(f[11]);
  f_pages = reinterpret_cast<decltype(f_pages)>(f[12]);
  f_mass = reinterpret_cast<decltype(f_mass)>(f[13]);
  f_evict_ws = reinterpret_cast<decltype(f_evict_ws)>(f[14]);
  f_evict = reinterpret_cast<decltype(f_evict)>(f[15]);
  return none();
}

#define FAST(name) {#name, (PyCFunction)(void*)name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(init),     FAST(page_plan), FAST(qkv_rope), FAST(qkv_rope_backward),
                         FAST(extend),   FAST(decode_shared), FAST(page_bounds),
                         FAST(select_pages), FAST(decode_pages), FAST(key_mass), FAST(evict),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "attn_sink_fast", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_attn_sink_fast() { return PyModule_Create(&module); }
