// marshal.cpp -- the common case of the attention calls' argument marshalling, compiled.
//
// A call takes up to twelve tensors, and asking each from Python for its type, device,
// shape, layout and address costs more than the launch (append: 10 of 13.5 us).  Each
// function here checks the common case -- contiguous CUDA tensors on the current device,
// of the types and shapes that the call takes -- makes the C-ABI call and returns its
// status; it returns None, without having done anything, for every other case, and the
// Python binding then goes through the arguments one by one, makes the call or says what
// is wrong.  The arithmetic is the library's; this file only reads tensors' descriptions.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "bitlinear.h"

namespace {

decltype(&bitlinear_rope) g_rope;
decltype(&bitlinear_kv_append) g_append;
decltype(&bitlinear_kv_read) g_read;
decltype(&bitlinear_attention) g_attention;
decltype(&bitlinear_attention_shared) g_shared;
decltype(&bitlinear_kv_summarise) g_summarise;
decltype(&bitlinear_attention_select) g_select;
decltype(&bitlinear_attention_blocks) g_blocks;
decltype(&bitlinear_softmax) g_softmax;
decltype(&bitlinear_verify) g_verify;

constexpr auto kF32 = at::kFloat, kI32 = at::kInt;

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool fits(const at::Tensor* t, int64_t device, at::ScalarType type, int64_t dims) {
  return t && t->is_cuda() && t->get_device() == device && t->scalar_type() == type && t->dim() == dims &&
         t->is_contiguous();
}
bool fits(const at::Tensor* t, int64_t device, at::ScalarType type, at::IntArrayRef shape) {
  return fits(t, device, type, (int64_t)shape.size()) && t->sizes() == shape;
}
template <typename P = void>
P* at_of(const at::Tensor* t) {
  return t ? static_cast<P*>(t->data_ptr()) : nullptr;
}

// The device of a call's first tensor where it is the current one, else -1.
int64_t device_of(const at::Tensor* t) {
  if (!t || !t->is_cuda()) return -1;
  const int64_t d = t->get_device();
  return d == (int64_t)c10::cuda::current_device() ? d : -1;
}

bool integer(PyObject* o, long long* out) {
  if (!PyLong_Check(o)) return false;
  *out = PyLong_AsLongLong(o);
  return !(*out == -1 && PyErr_Occurred());
}
bool real(PyObject* o, double* out) {
  if (!PyFloat_Check(o)) return false;
  *out = PyFloat_AS_DOUBLE(o);
  return true;
}

bool stream_of(PyObject* o, int64_t device, void** out) {
  if (o == Py_None) {
    *out = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    return true;
  }
  PyObject* handle = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  if (!handle) return false;
  long long v = 0;
  const bool ok = integer(handle, &v);
  Py_DECREF(handle);
  *out = reinterpret_cast<void*>(v);
  return ok;
}

// (k, v[, k_step, v_step]) as the C struct.
bool pages_of(PyObject* cache, int64_t device, bitlinear_kv_pages* out) {
  if (!PyTuple_Check(cache)) return false;
  const Py_ssize_t n = PyTuple_GET_SIZE(cache);
  if (n != 2 && n != 4) return false;
  const at::Tensor *k = tensor(PyTuple_GET_ITEM(cache, 0)), *v = tensor(PyTuple_GET_ITEM(cache, 1));
  if (!k) return false;
  const at::ScalarType type = k->scalar_type();
  const int format = type == at::kChar             ? BITLINEAR_KV_INT8
                     : type == at::kFloat8_e4m3fn  ? BITLINEAR_KV_FP8
                     : type == at::kBFloat16       ? BITLINEAR_KV_BF16
                                                   : -1;
  if (format < 0 || !fits(k, device, type, 4) || !fits(v, device, type, k->sizes())) return false;
  const at::Tensor *ks = nullptr, *vs = nullptr;
  if (format == BITLINEAR_KV_BF16) {
    if (n == 4 && (PyTuple_GET_ITEM(cache, 2) != Py_None || PyTuple_GET_ITEM(cache, 3) != Py_None)) return false;
  } else {
    if (n != 4) return false;
    ks = tensor(PyTuple_GET_ITEM(cache, 2));
    vs = tensor(PyTuple_GET_ITEM(cache, 3));
    const at::IntArrayRef rows = k->sizes().slice(0, 3);
    if (!fits(ks, device, kF32, rows) || !fits(vs, device, kF32, rows)) return false;
  }
  for (int i = 1; i < 4; ++i)
    if (k->size(i) > 0x7fffffff) return false;
  *out = bitlinear_kv_pages{at_of(k), at_of(v), at_of<float>(ks), at_of<float>(vs), k->size(0),
                            (int32_t)k->size(1), (int32_t)k->size(2), (int32_t)k->size(3), format};
  return true;
}

// (freq, layout[, amplitude]) as the C struct.
bool spec_of(PyObject* rope, int64_t device, bitlinear_rope_spec* out) {
  if (!PyTuple_Check(rope)) return false;
  const Py_ssize_t n = PyTuple_GET_SIZE(rope);
  if (n != 2 && n != 3) return false;
  const at::Tensor* freq = tensor(PyTuple_GET_ITEM(rope, 0));
  long long layout = 0;
  double amplitude = 1.0;
  if (!fits(freq, device, at::kDouble, 1) || freq->numel() > 4096 || !integer(PyTuple_GET_ITEM(rope, 1), &layout) ||
      layout < 0 || layout > 0x7fff || (n == 3 && !real(PyTuple_GET_ITEM(rope, 2), &amplitude)))
    return false;
  *out = bitlinear_rope_spec{at_of<double>(freq), (int32_t)(2 * freq->numel()), (int32_t)layout, (float)amplitude};
  return true;
}

struct Places {
  const int32_t *positions, *seq, *table;
  int64_t sequences, columns;
};
bool places_of(PyObject* positions, PyObject* table, PyObject* seq, int64_t T, int64_t device, Places* out) {
  const at::Tensor *p = tensor(positions), *t = tensor(table), *s = seq == Py_None ? nullptr : tensor(seq);
  if (!fits(p, device, kI32, at::IntArrayRef(&T, 1)) || !fits(t, device, kI32, 2)) return false;
  if (seq != Py_None && !fits(s, device, kI32, at::IntArrayRef(&T, 1))) return false;
  *out = Places{at_of<int32_t>(p), at_of<int32_t>(s), at_of<int32_t>(t), t->size(0), t->size(1)};
  return true;
}

bool flags_of(PyObject* o, int* out) {
  long long v;
  if (!integer(o, &v) || v < 0 || v > 0xffff) return false;
  *out = (int)v;
  return true;
}

// Runs f(); what it cannot take, a C++ exception or a Python error it met gives None.
template <typename F>
PyObject* common_case(F f) {
  int status = 0;
  bool done = false;
  try {
    done = f(&status);
  } catch (...) {
  }
  if (!done) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  return PyLong_FromLong(status);
}

// Lets other Python threads run while the library enqueues (a launch waits where the queue is
// full, and what it waits for may be a host callback that needs Python).  The caller's
// references keep the tensors.
struct Released {
  PyThreadState* state = PyEval_SaveThread();
  ~Released() { PyEval_RestoreThread(state); }
};

// rope(x, positions, rope, y, flags, stream)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return common_case([&](int* status) {
    if (n != 6) return false;
    const at::Tensor *x = tensor(a[0]), *p = tensor(a[1]), *y = tensor(a[3]);
    const int64_t d = device_of(x);
    bitlinear_rope_spec spec;
    int flags;
    void* stream;
    if (d < 0 || !fits(x, d, kF32, 3) || !fits(y, d, kF32, x->sizes()) || !fits(p, d, kI32, x->sizes().slice(0, 1)) ||
        x->size(1) > 0x7fffffff || x->size(2) > 0x7fffffff || !spec_of(a[2], d, &spec) || !flags_of(a[4], &flags) ||
        !stream_of(a[5], d, &stream))
      return false;
    const int64_t stride = x->size(1) * x->size(2);
    Released released;
    *status = g_rope(at_of<float>(x), stride, x->size(0), (int)x->size(1), (int)x->size(2), at_of<int32_t>(p), &spec,
                     at_of<float>(y), stride, flags, stream);
    return true;
  });
}

// kv_append(k, v, cache, positions, page_table, seq, q, q_out, rope, flags, stream)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return common_case([&](int* status) {
    if (n != 11) return false;
    const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *q = nullptr, *q_out = nullptr;
    const int64_t d = device_of(k);
    bitlinear_kv_pages pages;
    bitlinear_rope_spec spec;
    Places at;
    int flags;
    void* stream;
    if (d < 0 || !fits(k, d, kF32, 3) || !fits(v, d, kF32, k->sizes()) || !pages_of(a[2], d, &pages) ||
        k->size(1) != pages.num_heads || k->size(2) != pages.head_dim)
      return false;
    const int64_t T = k->size(0), stride = k->size(1) * k->size(2);
    if (!places_of(a[3], a[4], a[5], T, d, &at)) return false;
    int64_t heads = 0;
    if (a[6] != Py_None || a[7] != Py_None) {
      q = tensor(a[6]);
      q_out = tensor(a[7]);
      if (!fits(q, d, kF32, 3) || q->size(0) != T || q->size(2) != pages.head_dim || q->size(1) > 0x7fffffff ||
          !fits(q_out, d, kF32, q->sizes()))
        return false;
      heads = q->size(1);
    }
    if ((a[8] != Py_None && !spec_of(a[8], d, &spec)) || !flags_of(a[9], &flags) || !stream_of(a[10], d, &stream))
      return false;
    Released released;
    *status = g_append(at_of<float>(q), heads * pages.head_dim, (int)heads, at_of<float>(q_out), heads * pages.head_dim,
                       at_of<float>(k), stride, at_of<float>(v), stride, T, at.positions, at.seq, at.table, at.columns,
                       at.sequences, at.columns, a[8] == Py_None ? nullptr : &spec, &pages, flags, stream);
    return true;
  });
}

// kv_read(cache, positions, page_table, k_out, v_out, seq, flags, stream)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return common_case([&](int* status) {
    if (n != 8) return false;
    const at::Tensor *k = tensor(a[3]), *v = tensor(a[4]);
    const int64_t d = device_of(k);
    bitlinear_kv_pages pages;
    Places at;
    int flags;
    void* stream;
    if (d < 0 || !fits(k, d, kF32, 3) || !fits(v, d, kF32, k->sizes()) || !pages_of(a[0], d, &pages) ||
        k->size(1) != pages.num_heads || k->size(2) != pages.head_dim ||
        !places_of(a[1], a[2], a[5], k->size(0), d, &at) || !flags_of(a[6], &flags) || !stream_of(a[7], d, &stream))
      return false;
    const int64_t stride = k->size(1) * k->size(2);
    Released released;
    *status = g_read(&pages, k->size(0), at.positions, at.seq, at.table, at.columns, at.sequences, at.columns,
                     at_of<float>(k), stride, at_of<float>(v), stride, flags, stream);
    return true;
  });
}

// attention(q, cache, page_table, lengths, out, workspace, scale, window, flags, stream)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return common_case([&](int* status) {
    if (n != 10) return false;
    const at::Tensor *q = tensor(a[0]), *table = tensor(a[2]), *lengths = tensor(a[3]), *out = tensor(a[4]);
    const at::Tensor* space = a[5] == Py_None ? nullptr : tensor(a[5]);
    const int64_t d = device_of(q);
    bitlinear_kv_pages pages;
    double scale = 0.0;
    long long window;
    int flags;
    void* stream;
    if (d < 0 || !fits(q, d, kF32, 3) || !fits(out, d, kF32, q->sizes()) || !pages_of(a[1], d, &pages) ||
        q->size(2) != pages.head_dim || q->size(1) > 0x7fffffff || !fits(table, d, kI32, 2) ||
        table->size(0) != q->size(0) || !fits(lengths, d, kI32, q->sizes().slice(0, 1)) ||
        (a[5] != Py_None && !fits(space, d, at::kByte, 1)) || (a[6] != Py_None && !real(a[6], &scale)) ||
        !integer(a[7], &window) || !flags_of(a[8], &flags) || !stream_of(a[9], d, &stream))
      return false;
    if (a[6] == Py_None) scale = std::pow((double)pages.head_dim, -0.5);
    const int64_t stride = q->size(1) * q->size(2);
    Released released;
    *status = g_attention(at_of<float>(q), stride, q->size(0), (int)q->size(1), &pages, at_of<int32_t>(table),
                          table->size(1), table->size(1), at_of<int32_t>(lengths), window, (float)scale,
                          at_of<float>(out), stride, at_of(space), space ? (size_t)space->numel() : 0, flags, stream);
    return true;
  });
}

// What the attention calls without a window have in common.
struct Attended {
  const at::Tensor *q, *table, *lengths;
  int64_t device, stride;
  bitlinear_kv_pages pages;
};
bool attended(PyObject* q, PyObject* cache, PyObject* table, PyObject* lengths, Attended* out) {
  out->q = tensor(q);
  out->table = tensor(table);
  out->lengths = tensor(lengths);
  const int64_t d = out->device = device_of(out->q);
  if (d < 0 || !fits(out->q, d, kF32, 3) || !pages_of(cache, d, &out->pages) || out->q->size(2) != out->pages.head_dim ||
      out->q->size(1) > 0x7fffffff || !fits(out->table, d, kI32, 2) || out->table->size(0) != out->q->size(0) ||
      !fits(out->lengths, d, kI32, out->q->sizes().slice(0, 1)))
    return false;
  out->stride = out->q->size(1) * out->q->size(2);
  return true;
}
bool scale_of(PyObject* o, const bitlinear_kv_pages& pages, double* out) {
  if (o == Py_None) {
    *out = std::pow((double)pages.head_dim, -0.5);
    return true;
  }
  return real(o, out);
}
bool listed(PyObject* o, const Attended& a, const at::Tensor** out) {
  const at::Tensor* t = *out = tensor(o);
  return fits(t, a.device, kI32, 3) && t->size(0) == a.q->size(0) && t->size(1) == a.pages.num_heads && t->size(2) <= 0x7fffffff;
}
// (bounds, step) as the C struct.
bool summary_of(PyObject* o, int64_t device, const bitlinear_kv_pages& pages, bitlinear_kv_summary* out) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) return false;
  const at::Tensor *bounds = tensor(PyTuple_GET_ITEM(o, 0)), *step = tensor(PyTuple_GET_ITEM(o, 1));
  const int64_t shape[4] = {pages.num_pages, pages.num_heads, 2, pages.head_dim};
  if (!fits(bounds, device, at::kChar, at::IntArrayRef(shape, 4)) || !fits(step, device, kF32, at::IntArrayRef(shape, 2)))
    return false;
  *out = bitlinear_kv_summary{at_of<int8_t>(bounds), at_of<float>(step)};
  return true;
}

// attention_shared(q, cache, page_table, lengths, shared, out, workspace, scale, flags, stream)
PyObject* attention_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return common_case([&](int* status) {
    if (n != 10) return false;
    Attended t;
    if (!attended(a[0], a[1], a[2], a[3], &t)) return false;
    const at::Tensor *shared = tensor(a[4]), *out = tensor(a[5]), *space = a[6] == Py_None ? nullptr : tensor(a[6]);
    double scale;
    int flags;
    void* stream;
    if (!fits(shared, t.device, kI32, 1) || !fits(out, t.device, kF32, t.q->sizes()) ||
        (a[6] != Py_None && !fits(space, t.device, at::kByte, 1)) || !scale_of(a[7], t.pages, &scale) ||
        !flags_of(a[8], &flags) || !stream_of(a[9], t.device, &stream))
      return false;
    Released released;
    *status = g_shared(at_of<float>(t.q), t.stride, t.q->size(0), (int)t.q->size(1), &t.pages, at_of<int32_t>(t.table),
                       t.table->size(1), t.table->size(1), at_of<int32_t>(t.lengths), at_of<int32_t>(shared), shared->size(0),
                       (float)scale, at_of<float>(out), t.stride, at_of(space), space ? (size_t)space->numel() : 0, flags, stream);
    return true;
  });
}

// kv_summarise(cache, summary, page_table, first, lengths, flags, stream)
PyObject* kv_summarise(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return common_case([&](int* status) {
    if (n != 7) return false;
    const at::Tensor *table = tensor(a[2]), *first = tensor(a[3]), *lengths = tensor(a[4]);
    const int64_t d = device_of(table);
    bitlinear_kv_pages pages;
    bitlinear_kv_summary summary;
    int flags;
    void* stream;
    if (d < 0 || !fits(table, d, kI32, 2) || !pages_of(a[0], d, &pages) || !summary_of(a[1], d, pages, &summary) ||
        !fits(first, d, kI32, table->sizes().slice(0, 1)) || !fits(lengths, d, kI32, table->sizes().slice(0, 1)) ||
        !flags_of(a[5], &flags) || !stream_of(a[6], d, &stream))
      return false;
    Released released;
    *status = g_summarise(&pages, &summary, at_of<int32_t>(table), table->size(1), table->size(0), table->size(1),
                          at_of<int32_t>(first), at_of<int32_t>(lengths), flags, stream);
    return true;
  });
}

// attention_select(q, cache, summary, page_table, lengths, blocks, keep_first, keep_last, flags, stream)
PyObject* attention_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return common_case([&](int* status) {
    if (n != 10) return false;
    Attended t;
    if (!attended(a[0], a[1], a[3], a[4], &t)) return false;
    const at::Tensor* blocks;
    bitlinear_kv_summary summary;
    long long first, last;
    int flags;
    void* stream;
    if (!summary_of(a[2], t.device, t.pages, &summary) || !listed(a[5], t, &blocks) || !integer(a[6], &first) ||
        !integer(a[7], &last) || first < 0 || first > 0x7fffffff || last < 0 || last > 0x7fffffff ||
        !flags_of(a[8], &flags) || !stream_of(a[9], t.device, &stream))
      return false;
    Released released;
    *status = g_select(at_of<float>(t.q), t.stride, t.q->size(0), (int)t.q->size(1), &t.pages, &summary, at_of<int32_t>(t.table),
                       t.table->size(1), t.table->size(1), at_of<int32_t>(t.lengths), (int)first, (int)last,
                       at_of<int32_t>(blocks), (int)blocks->size(2), flags, stream);
    return true;
  });
}

// attention_blocks(q, cache, page_table, lengths, blocks, out, scale, flags, stream)
PyObject* attention_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return common_case([&](int* status) {
    if (n != 9) return false;
    Attended t;
    if (!attended(a[0], a[1], a[2], a[3], &t)) return false;
    const at::Tensor *blocks, *out = tensor(a[5]);
    double scale;
    int flags;
    void* stream;
    if (!listed(a[4], t, &blocks) || !fits(out, t.device, kF32, t.q->sizes()) || !scale_of(a[6], t.pages, &scale) ||
        !flags_of(a[7], &flags) || !stream_of(a[8], t.device, &stream))
      return false;
    Released released;
    *status = g_blocks(at_of<float>(t.q), t.stride, t.q->size(0), (int)t.q->size(1), &t.pages, at_of<int32_t>(t.table),
                       t.table->size(1), t.table->size(1), at_of<int32_t>(t.lengths), at_of<int32_t>(blocks),
                       (int)blocks->size(2), (float)scale, at_of<float>(out), t.stride, flags, stream);
    return true;
  });
}

// softmax(y, p, temperature, flags, stream)
PyObject* softmax(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return common_case([&](int* status) {
    if (n != 5) return false;
    const at::Tensor *y = tensor(a[0]), *p = tensor(a[1]), *temperature = a[2] == Py_None ? nullptr : tensor(a[2]);
    const int64_t d = device_of(y);
    int flags;
    void* stream;
    if (d < 0 || !fits(y, d, kF32, 2) || !fits(p, d, kF32, y->sizes()) ||
        (a[2] != Py_None && !fits(temperature, d, kF32, y->sizes().slice(0, 1))) || !flags_of(a[3], &flags) ||
        !stream_of(a[4], d, &stream))
      return false;
    Released released;
    *status = g_softmax(at_of<float>(y), y->size(0), y->size(1), at_of<float>(temperature), at_of<float>(p), flags, stream);
    return true;
  });
}

// verify(p, q, draft, uniform, tokens, accepted, flags, stream)
PyObject* verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return common_case([&](int* status) {
    if (n != 8) return false;
    const at::Tensor *p = tensor(a[0]), *q = tensor(a[1]), *draft = tensor(a[2]), *uniform = tensor(a[3]);
    const at::Tensor *tokens = tensor(a[4]), *accepted = tensor(a[5]);
    const int64_t d = device_of(p);
    int flags;
    void* stream;
    if (d < 0 || !fits(p, d, kF32, 3) || p->size(1) < 2 || p->size(1) > 0x7fffffff) return false;
    const int64_t B = p->size(0), K = p->size(1) - 1, rows[3] = {B, K, p->size(2)}, all[2] = {B, K + 1};
    if (!fits(q, d, kF32, at::IntArrayRef(rows, 3)) || !fits(draft, d, kI32, at::IntArrayRef(rows, 2)) ||
        !fits(uniform, d, kF32, at::IntArrayRef(all, 2)) || !fits(tokens, d, kI32, at::IntArrayRef(all, 2)) ||
        !fits(accepted, d, kI32, at::IntArrayRef(rows, 1)) || !flags_of(a[6], &flags) || !stream_of(a[7], d, &stream))
      return false;
    Released released;
    *status = g_verify(at_of<float>(p), at_of<float>(q), B, (int)K, p->size(2), at_of<int32_t>(draft), at_of<float>(uniform),
                       at_of<int32_t>(tokens), at_of<int32_t>(accepted), flags, stream);
    return true;
  });
}

// bind_serving(attention_shared, kv_summarise, attention_select, attention_blocks, softmax, verify): their addresses.
PyObject* bind_serving(PyObject*, PyObject* const* a, Py_ssize_t n) {
  long long at[6];
  for (int i = 0; i < 6; ++i)
    if (n != 6 || !integer(a[i], &at[i]) || !at[i]) {
      PyErr_SetString(PyExc_ValueError, "bind_serving takes six addresses");
      return nullptr;
    }
  g_shared = reinterpret_cast<decltype(g_shared)>(at[0]);
  g_summarise = reinterpret_cast<decltype(g_summarise)>(at[1]);
  g_select = reinterpret_cast<decltype(g_select)>(at[2]);
  g_blocks = reinterpret_cast<decltype(g_blocks)>(at[3]);
  g_softmax = reinterpret_cast<decltype(g_softmax)>(at[4]);
  g_verify = reinterpret_cast<decltype(g_verify)>(at[5]);
  Py_RETURN_NONE;
}

// bind(rope, kv_append, kv_read, attention): the addresses of the library's entry points.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  long long at[4];
  for (int i = 0; i < 4; ++i)
    if (n != 4 || !integer(a[i], &at[i]) || !at[i]) {
      PyErr_SetString(PyExc_ValueError, "bind takes four addresses");
      return nullptr;
    }
  g_rope = reinterpret_cast<decltype(g_rope)>(at[0]);
  g_append = reinterpret_cast<decltype(g_append)>(at[1]);
  g_read = reinterpret_cast<decltype(g_read)>(at[2]);
  g_attention = reinterpret_cast<decltype(g_attention)>(at[3]);
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(bind)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(rope)), METH_FASTCALL, nullptr},
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(kv_append)), METH_FASTCALL, nullptr},
    {"kv_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(kv_read)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(attention)), METH_FASTCALL, nullptr},
    {"bind_serving", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(bind_serving)), METH_FASTCALL, nullptr},
    {"attention_shared", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(attention_shared)), METH_FASTCALL, nullptr},
    {"kv_summarise", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(kv_summarise)), METH_FASTCALL, nullptr},
    {"attention_select", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(attention_select)), METH_FASTCALL, nullptr},
    {"attention_blocks", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(attention_blocks)), METH_FASTCALL, nullptr},
    {"softmax", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(softmax)), METH_FASTCALL, nullptr},
    {"verify", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(verify)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "bitlinear_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_bitlinear_marshal(void) { return PyModule_Create(&g_module); }
