// The Python binding's short way into the calls that a serving step makes once per layer.  A small
// step is bound by the host, and checking a call's dozen tensors attribute by attribute in Python
// costs more than its launches (four-token rotary append: 9.7 us a call, of which 5.8 in Python).  Each
// function here checks its arguments against the tensors themselves and calls the library: it
// returns the call's status, or None, having done nothing, when an argument is not what the plain
// case takes (another type, device, layout or shape, a subclass, another current device).  The
// Python code then goes its own way, which says what is wrong or makes the call.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "../../include/pagedkv.h"

namespace {

using at::ScalarType;

struct Unfit {};  // thrown by the checks, turned into None

// The arguments of one call.  The first tensor says which device the others have to be on.
struct Args {
  PyObject* const* at;
  int device = -1;

  const at::Tensor& tensor(int i, ScalarType type) {
    if (!THPVariable_CheckExact(at[i])) throw Unfit();
    const at::Tensor& t = THPVariable_Unpack(at[i]);
    if (!t.is_cuda() || t.layout() != at::kStrided || t.scalar_type() != type) throw Unfit();
    if (device < 0) device = t.get_device();
    if (t.get_device() != device || !t.is_contiguous()) throw Unfit();
    return t;
  }
  bool given(int i) const { return at[i] != Py_None; }
  void* address(int i, ScalarType type) { return tensor(i, type).data_ptr(); }
  void* address_or_null(int i, ScalarType type) { return given(i) ? address(i, type) : nullptr; }
  int32_t number(int i) {
    int overflow = 0;
    const long v = PyLong_Check(at[i]) ? PyLong_AsLongAndOverflow(at[i], &overflow) : -1;
    if (!PyLong_Check(at[i]) || overflow || v < INT32_MIN || v > INT32_MAX) throw Unfit();
    return (int32_t)v;
  }
  float real(int i) {
    if (!PyFloat_Check(at[i])) throw Unfit();
    return (float)PyFloat_AS_DOUBLE(at[i]);
  }
  // A stream's handle, or None for the device's current one; the device has to be the current one.
  void* stream(int i) {
    if (c10::cuda::current_device() != device) throw Unfit();
    if (!given(i)) return c10::cuda::getCurrentCUDAStream(device).stream();
    void* s = PyLong_AsVoidPtr(at[i]);
    if (!s && PyErr_Occurred()) {
      PyErr_Clear();
      throw Unfit();
    }
    return s;
  }
};

int32_t i32(int64_t n) {
  if (n > INT32_MAX) throw Unfit();
  return (int32_t)n;
}
void need(bool ok) {
  if (!ok) throw Unfit();
}
bool is_shape(const at::Tensor& t, std::initializer_list<int64_t> shape) { return t.sizes() == at::IntArrayRef(shape); }

struct Shape {
  int64_t pages, page_size, heads, dim;
};

pkv_pool pool_bf16(Args& a, int i, Shape& s) {
  const at::Tensor &k = a.tensor(i, at::kBFloat16), &v = a.tensor(i + 1, at::kBFloat16);
  need(k.dim() == 4 && v.sizes() == k.sizes());
  s = {k.size(0), k.size(1), k.size(2), k.size(3)};
  return pkv_pool{k.data_ptr(), v.data_ptr(), s.pages, i32(s.page_size), i32(s.heads), i32(s.dim)};
}

pkv_pool_fp8 pool_fp8(Args& a, int i, Shape& s) {
  need(THPVariable_CheckExact(a.at[i]));
  const ScalarType type = THPVariable_Unpack(a.at[i]).scalar_type();
  need(type == at::kFloat8_e4m3fn || type == at::kByte);
  const at::Tensor &k = a.tensor(i, type), &v = a.tensor(i + 1, type);
  const at::Tensor &ks = a.tensor(i + 2, at::kFloat), &vs = a.tensor(i + 3, at::kFloat);
  need(k.dim() == 4 && v.sizes() == k.sizes());
  s = {k.size(0), k.size(1), k.size(2), k.size(3)};
  need(is_shape(ks, {s.pages, s.page_size, s.heads}) && vs.sizes() == ks.sizes());
  return pkv_pool_fp8{k.data_ptr(), v.data_ptr(), (float*)ks.data_ptr(), (float*)vs.data_ptr(),
                      s.pages,      i32(s.page_size), i32(s.heads),      i32(s.dim)};
}

// Makes the call without holding the interpreter (a launch can wait for room in the stream's queue).
template <typename F>
PyObject* status_of(F call) {
  PyThreadState* state = PyEval_SaveThread();
  const int status = call();
  PyEval_RestoreThread(state);
  return PyLong_FromLong(status);
}

template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F body) {
  if (given != wanted) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return body();
  } catch (...) {  // also what torch throws for a tensor without memory of its own
    Py_RETURN_NONE;
  }
}

struct NewRows {
  const void *k, *v;
  const int64_t* slots;
  int32_t n;
};

NewRows new_rows(Args& a, int i, const Shape& s) {  // k_new, v_new, slot_mapping
  const at::Tensor &k = a.tensor(i, at::kBFloat16), &v = a.tensor(i + 1, at::kBFloat16);
  const at::Tensor& slots = a.tensor(i + 2, at::kLong);
  const int64_t n = slots.numel();
  need(is_shape(k, {n, s.heads, s.dim}) && v.sizes() == k.sizes());
  return {k.data_ptr(), v.data_ptr(), (const int64_t*)slots.data_ptr(), i32(n)};
}

// (k_pool, v_pool[, k_scale, v_scale], k_new, v_new, slot_mapping, positions, cos_sin, q, q_out,
//  interleaved, err_word, stream)
template <bool FP8>
PyObject* rotary(PyObject*, PyObject* const* args, Py_ssize_t n) {
  constexpr int p = FP8 ? 4 : 2;
  return guarded(n, p + 10, [&] {
    Args a{args};
    Shape s;
    pkv_pool pool;
    pkv_pool_fp8 pool8;
    if (FP8)
      pool8 = pool_fp8(a, 0, s);
    else
      pool = pool_bf16(a, 0, s);
    const NewRows rows = new_rows(a, p, s);
    const at::Tensor &pos = a.tensor(p + 3, at::kInt), &table = a.tensor(p + 4, at::kFloat);
    need(pos.numel() == rows.n && table.dim() == 2);
    const int64_t width = table.size(1);
    need(width >= 2 && width % 2 == 0 && width <= s.dim);
    void *q = nullptr, *q_out = nullptr;
    int32_t heads = 0;
    if (a.given(p + 5)) {
      const at::Tensor& t = a.tensor(p + 5, at::kBFloat16);
      need(t.dim() == 3 && t.size(0) == rows.n && t.size(2) == s.dim);
      heads = i32(t.size(1));
      q = q_out = t.data_ptr();
      if (a.given(p + 6)) {
        const at::Tensor& o = a.tensor(p + 6, at::kBFloat16);
        need(o.sizes() == t.sizes());
        q_out = o.data_ptr();
      }
    } else {
      need(!a.given(p + 6));
    }
    const int32_t max_position = i32(table.size(0)), R = i32(width), pairs = args[p + 7] == Py_True;
    need(PyBool_Check(args[p + 7]));
    uint32_t* err = (uint32_t*)a.address_or_null(p + 8, at::kInt);
    void* stream = a.stream(p + 9);
    const int32_t* at_pos = (const int32_t*)pos.data_ptr();
    const float* cos_sin = (const float*)table.data_ptr();
    return status_of([&]() -> int {
      if (FP8)
        return pkv_rotary_kv_append_fp8(&pool8, rows.k, rows.v, rows.slots, at_pos, cos_sin, max_position, R, pairs, q,
                                        q_out, heads, rows.n, err, stream);
      return pkv_rotary_kv_append(&pool, rows.k, rows.v, rows.slots, at_pos, cos_sin, max_position, R, pairs, q, q_out,
                                  heads, rows.n, err, stream);
    });
  });
}

// (k_pool, v_pool, k_scale, v_scale, k_new, v_new, slot_mapping, err_word, stream)
PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    Args a{args};
    Shape s;
    const pkv_pool_fp8 pool = pool_fp8(a, 0, s);
    const NewRows rows = new_rows(a, 4, s);
    uint32_t* err = (uint32_t*)a.address_or_null(7, at::kInt);
    void* stream = a.stream(8);
    return status_of([&] { return (int)pkv_kv_append_fp8(&pool, rows.k, rows.v, rows.slots, rows.n, err, stream); });
  });
}

// The rows of an attention call: q, out, lse (or None) at i, i + 1, i + 2.
struct Rows {
  const void* q;
  void* out;
  float* lse;
  int32_t n, heads;
};

Rows attention_rows(Args& a, int i, int64_t dim) {
  const at::Tensor &q = a.tensor(i, at::kBFloat16), &out = a.tensor(i + 1, at::kBFloat16);
  need(q.dim() == 3 && q.size(2) == dim && out.sizes() == q.sizes());
  Rows r{q.data_ptr(), out.data_ptr(), nullptr, i32(q.size(0)), i32(q.size(1))};
  if (a.given(i + 2)) {
    const at::Tensor& lse = a.tensor(i + 2, at::kFloat);
    need(is_shape(lse, {q.size(0), q.size(1)}));
    r.lse = (float*)lse.data_ptr();
  }
  return r;
}

// (k_pool, v_pool, k_scale, v_scale, q, out, lse, kv_indptr, kv_indices, kv_lens, sm_scale, workspace, err_word,
//  max_ctas, stream)
PyObject* decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    Args a{args};
    Shape s;
    const pkv_pool_fp8 pool = pool_fp8(a, 0, s);
    const Rows r = attention_rows(a, 4, s.dim);
    const at::Tensor &indptr = a.tensor(7, at::kInt), &indices = a.tensor(8, at::kInt), &lens = a.tensor(9, at::kInt);
    need(lens.numel() == r.n && indptr.numel() == (int64_t)r.n + 1);
    const float scale = a.real(10);
    const at::Tensor& ws = a.tensor(11, at::kByte);
    uint32_t* err = (uint32_t*)a.address_or_null(12, at::kInt);
    const int32_t max_ctas = a.number(13);
    void* stream = a.stream(14);
    const int32_t *p = (const int32_t*)indptr.data_ptr(), *x = (const int32_t*)indices.data_ptr(),
                  *l = (const int32_t*)lens.data_ptr();
    void* w = ws.data_ptr();
    const size_t bytes = (size_t)ws.numel();
    return status_of([&] {
      return (int)pkv_paged_decode_fp8(&pool, r.q, r.n, r.heads, p, x, l, scale, r.out, r.lse, w, bytes, err, max_ctas,
                                       stream);
    });
  });
}

// (k_pool, v_pool, q, out, lse, qo_indptr, kv_indptr, kv_indices, prefix_lens, tree_mask, max_tree_len,
//  sm_scale, workspace, err_word, stream)
PyObject* tree(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    Args a{args};
    Shape s;
    const pkv_pool pool = pool_bf16(a, 0, s);
    const Rows r = attention_rows(a, 2, s.dim);
    const at::Tensor &qo = a.tensor(5, at::kInt), &indptr = a.tensor(6, at::kInt), &indices = a.tensor(7, at::kInt),
                     &prefix = a.tensor(8, at::kInt), &mask = a.tensor(9, at::kInt);
    const int32_t batch = i32(prefix.numel()), most = a.number(10);
    need(qo.numel() == (int64_t)batch + 1 && indptr.numel() == (int64_t)batch + 1);
    need(mask.dim() == 2 && mask.size(0) == r.n && 32 * mask.size(1) >= most);
    const int32_t words = i32(mask.size(1));
    const float scale = a.real(11);
    const at::Tensor& ws = a.tensor(12, at::kByte);
    uint32_t* err = (uint32_t*)a.address_or_null(13, at::kInt);
    void* stream = a.stream(14);
    const int32_t *o = (const int32_t*)qo.data_ptr(), *p = (const int32_t*)indptr.data_ptr(),
                  *x = (const int32_t*)indices.data_ptr(), *l = (const int32_t*)prefix.data_ptr();
    const void* m = mask.data_ptr();
    void* w = ws.data_ptr();
    const size_t bytes = (size_t)ws.numel();
    return status_of([&] {
      return (int)pkv_paged_tree_attention(&pool, r.q, r.n, o, batch, r.heads, p, x, l, m, words, most, scale, r.out,
                                           r.lse, w, bytes, err, stream);
    });
  });
}

// (k_pool, v_pool, k_scale, v_scale, kv_indptr, kv_indices, kv_lens, out_indptr, k_out, v_out, err_word, stream)
PyObject* gather(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    Args a{args};
    Shape s;
    const pkv_pool_fp8 pool = pool_fp8(a, 0, s);
    const at::Tensor &indptr = a.tensor(4, at::kInt), &indices = a.tensor(5, at::kInt), &lens = a.tensor(6, at::kInt),
                     &to = a.tensor(7, at::kInt);
    const at::Tensor &k = a.tensor(8, at::kBFloat16), &v = a.tensor(9, at::kBFloat16);
    const int32_t batch = i32(lens.numel());
    need(indptr.numel() == (int64_t)batch + 1 && to.numel() == (int64_t)batch + 1);
    need(k.dim() == 3 && k.size(1) == s.heads && k.size(2) == s.dim && v.sizes() == k.sizes());
    const int32_t rows = i32(k.size(0));
    uint32_t* err = (uint32_t*)a.address_or_null(10, at::kInt);
    void* stream = a.stream(11);
    const int32_t *p = (const int32_t*)indptr.data_ptr(), *x = (const int32_t*)indices.data_ptr(),
                  *l = (const int32_t*)lens.data_ptr(), *o = (const int32_t*)to.data_ptr();
    void *ko = k.data_ptr(), *vo = v.data_ptr();
    return status_of([&] { return (int)pkv_paged_gather_fp8(&pool, p, x, l, batch, o, rows, ko, vo, err, stream); });
  });
}

PyMethodDef kMethods[] = {
    {"rotary_kv_append", (PyCFunction)(void (*)())rotary<false>, METH_FASTCALL, nullptr},
    {"rotary_kv_append_fp8", (PyCFunction)(void (*)())rotary<true>, METH_FASTCALL, nullptr},
    {"kv_append_fp8", (PyCFunction)(void (*)())append, METH_FASTCALL, nullptr},
    {"paged_gather_fp8", (PyCFunction)(void (*)())gather, METH_FASTCALL, nullptr},
    {"paged_decode_fp8", (PyCFunction)(void (*)())decode, METH_FASTCALL, nullptr},
    {"paged_tree_attention", (PyCFunction)(void (*)())tree, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_checked", "Checked calls of libpagedkv.so.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__checked() {
  PyObject* m = PyModule_Create(&kModule);
  if (m) PyModule_AddStringConstant(m, "torch_version", PKV_TORCH);  // whose tensors it reads
  return m;
}
