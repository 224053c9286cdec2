// kvp_calls.cpp -- the entry points that take a few microseconds on the GPU, called
// straight with torch tensors: looking at a dozen tensors from Python takes longer
// than the kernels.  A 4-bit decode of four short requests, 5 us on the GPU, kept
// the host busy for 9.1 us a call that way and for 2.7 this way, of which the
// launch is 2; a rotary append, 3.4 us on the GPU, 10.4 and 3.2.
//
// A function here checks the whole call and makes it, or returns None: then the
// Python binding goes through the arguments one by one for the error, or makes
// the call itself.  So what is allowed is said there and nowhere else; here are
// only the conditions under which a call is in order beyond doubt.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "kvp.h"

namespace {

using at::ScalarType;
using at::Tensor;

// One call's arguments, taken in order.  Tensors lie on the current device.
class Args {
 public:
  Args(PyObject* const* a, Py_ssize_t n) : next_(a), end_(a + n), dev_(c10::cuda::current_device()) {}

  // The next argument, a strided CUDA tensor.
  const Tensor* any() {
    PyObject* o = take();
    if (o == nullptr || !THPVariable_Check(o)) return nullptr;
    const Tensor& t = THPVariable_Unpack(o);
    return t.is_cuda() && t.device().index() == dev_ && t.layout() == c10::kStrided ? &t : nullptr;
  }
  // The same, contiguous and of the given type.
  const Tensor* whole(ScalarType type) {
    const Tensor* t = any();
    return t != nullptr && t->scalar_type() == type && t->is_contiguous() ? t : nullptr;
  }
  // An int32 tensor or None, which is null; anything else is not in order.
  bool status(int32_t** p) {
    *p = nullptr;
    if (none()) return true;
    const Tensor* t = whole(ScalarType::Int);
    if (t != nullptr && t->numel() >= 1) *p = t->data_ptr<int32_t>();
    return *p != nullptr;
  }
  bool number(int32_t* x) { return number(take(), x); }
  static bool number(PyObject* o, int32_t* x) {
    if (o == nullptr || !PyLong_Check(o)) return false;
    int over = 0;
    const long v = PyLong_AsLongAndOverflow(o, &over);
    *x = static_cast<int32_t>(v);
    return over == 0 && *x == v;
  }
  bool real(float* x) {
    PyObject* o = take();
    if (o == nullptr || !PyFloat_Check(o)) return false;
    *x = static_cast<float>(PyFloat_AS_DOUBLE(o));
    return true;
  }
  PyObject* take() { return next_ < end_ ? *next_++ : nullptr; }
  bool none() {
    if (next_ < end_ && *next_ == Py_None) {
      ++next_;
      return true;
    }
    return false;
  }
  kvp_stream_t stream() const {
    return reinterpret_cast<kvp_stream_t>(c10::cuda::getCurrentCUDAStream(dev_).stream());
  }

 private:
  PyObject* const* next_;
  PyObject* const* end_;
  c10::DeviceIndex dev_;
};

bool shape(const Tensor* t, std::initializer_list<int64_t> s) {
  return t->sizes() == c10::IntArrayRef(s.begin(), s.size());
}

bool dtype_code(const Tensor* t, kvp_dtype* d) {
  *d = t->scalar_type() == ScalarType::Half ? KVP_F16 : KVP_BF16;
  return t->scalar_type() == ScalarType::Half || t->scalar_type() == ScalarType::BFloat16;
}

bool small(int64_t x) { return x <= INT32_MAX; }

template <class T>
T* ptr(const Tensor* t) {
  return static_cast<T*>(t->data_ptr());
}

// 4-bit pools: codes, pairs of `type`, and their descriptor.
struct Pools {
  const Tensor *kc, *vc, *ks, *vs;
  kvp_cache_desc d;

  bool take(Args& a, ScalarType type) {
    if (!(kc = a.whole(ScalarType::Byte)) || !(vc = a.whole(ScalarType::Byte)) ||
        !(ks = a.whole(type)) || !(vs = a.whole(type)) || kc->dim() != 4)
      return false;
    const int64_t nb = kc->size(0), hkv = kc->size(1), bs = kc->size(2), half = kc->size(3);
    if (!small(nb) || !small(hkv) || !small(bs) || !small(2 * half)) return false;
    d = {static_cast<int32_t>(nb), static_cast<int32_t>(hkv), static_cast<int32_t>(bs),
         static_cast<int32_t>(2 * half)};
    return vc->sizes() == kc->sizes() && shape(ks, {nb, hkv, bs, half / 32, 2}) &&
           vs->sizes() == ks->sizes();
  }
};

// What a call gives: the library's status, or None where it was not made.  No
// C++ exception passes (torch's checks throw).
template <class F>
PyObject* guarded(F&& call) {
  try {
    kvp_status s = KVP_OK;
    if (call(&s)) return PyLong_FromLong(s);
  } catch (...) {
  }
  Py_RETURN_NONE;
}

// Other threads may run Python while a launch is made (given back on the way of an
// exception as well).
class WithoutGil {
 public:
  WithoutGil() : state_(PyEval_SaveThread()) {}
  ~WithoutGil() { PyEval_RestoreThread(state_); }
  WithoutGil(const WithoutGil&) = delete;
  WithoutGil& operator=(const WithoutGil&) = delete;

 private:
  PyThreadState* state_;
};

// key, value, pools, slot_mapping, status
template <bool kRead>
PyObject* rows_int4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&](kvp_status* s) {
    Args a(args, n);
    const Tensor *key, *value, *slots;
    Pools p;
    kvp_dtype dt;
    int32_t* status;
    if (!(key = a.any()) || !dtype_code(key, &dt) || !key->is_contiguous() ||
        !(value = a.whole(key->scalar_type())) || !p.take(a, key->scalar_type()) ||
        !(slots = a.whole(ScalarType::Int)) || slots->dim() != 1 || !a.status(&status))
      return false;
    const int64_t T = slots->size(0);
    if (!small(T) || !shape(key, {T, p.d.num_kv_heads, p.d.head_dim}) ||
        value->sizes() != key->sizes())
      return false;
    const kvp_stream_t st = a.stream();
    const WithoutGil guard;
    *s = kRead ? kvp_read_int4(ptr<void>(key), ptr<void>(value), dt,
                               ptr<uint8_t>(p.kc), ptr<uint8_t>(p.vc),
                               ptr<void>(p.ks), ptr<void>(p.vs),
                               ptr<int32_t>(slots), static_cast<int32_t>(T), p.d,
                               status, st)
               : kvp_append_int4(ptr<void>(key), ptr<void>(value), dt,
                                 ptr<uint8_t>(p.kc), ptr<uint8_t>(p.vc),
                                 ptr<void>(p.ks), ptr<void>(p.vs),
                                 ptr<int32_t>(slots), static_cast<int32_t>(T),
                                 p.d, status, st);
    return true;
  });
}

// out, q, pools, block_tables, context_lens, scale, workspace, partition_blocks,
// phases, status
PyObject* attention_decode_int4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&](kvp_status* s) {
    Args a(args, n);
    const Tensor *out, *q, *tables, *lens, *ws = nullptr;
    Pools p;
    kvp_dtype dt;
    float scale;
    int32_t part, phases, *status;
    if (!(out = a.any()) || !dtype_code(out, &dt) || !out->is_contiguous() ||
        !(q = a.whole(out->scalar_type())) || !p.take(a, out->scalar_type()) ||
        !(tables = a.whole(ScalarType::Int)) || !(lens = a.whole(ScalarType::Int)) ||
        !a.real(&scale))
      return false;
    if (!a.none() && (!(ws = a.any()) || !ws->is_contiguous())) return false;
    if (!a.number(&part) || !a.number(&phases) || !a.status(&status)) return false;
    if (q->dim() != 3 || tables->dim() != 2) return false;
    const int64_t B = q->size(0), Hq = q->size(1), MB = tables->size(1);
    if (!small(B) || !small(Hq) || !small(MB) || !shape(q, {B, Hq, p.d.head_dim}) ||
        out->sizes() != q->sizes() || tables->size(0) != B || !shape(lens, {B}))
      return false;
    const kvp_stream_t st = a.stream();
    const WithoutGil guard;
    *s = kvp_attention_decode_int4(
        ptr<void>(out), ptr<void>(q), dt, ptr<uint8_t>(p.kc), ptr<uint8_t>(p.vc),
        ptr<void>(p.ks), ptr<void>(p.vs), ptr<int32_t>(tables),
        static_cast<int32_t>(MB), ptr<int32_t>(lens), static_cast<int32_t>(B),
        static_cast<int32_t>(Hq), scale, p.d, part,
        ws != nullptr ? ws->data_ptr() : nullptr, ws != nullptr ? ws->nbytes() : 0,
        phases, status, st);
    return true;
  });
}

// Rows [T, heads, dim] with contiguous heads: their token stride.
bool row_stride(const Tensor* t, ScalarType type, int64_t T, int64_t heads, int64_t dim,
                int64_t* stride) {
  if (t->scalar_type() != type || !shape(t, {T, heads, dim}) || t->stride(2) != 1 ||
      (t->stride(1) != dim && heads > 1))
    return false;
  *stride = T > 1 ? t->stride(0) : heads * dim;
  return true;
}

// q_out, q, key, value, pools, cos_sin, positions, slot_mapping, sections,
// interleaved, status
template <bool kInt4>
PyObject* rope_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&](kvp_status* s) {
    Args a(args, n);
    const Tensor *qo, *q, *key, *value, *kc, *vc, *cs, *pos, *slots;
    Pools p;
    kvp_dtype dt;
    if (!(qo = a.any()) || !(q = a.any()) || !(key = a.any()) || !(value = a.any()) ||
        !dtype_code(key, &dt))
      return false;
    const ScalarType type = key->scalar_type();
    kvp_cache_desc d;
    if constexpr (kInt4) {
      if (!p.take(a, type)) return false;
      d = p.d;
    } else {
      if (!(kc = a.whole(type)) || !(vc = a.whole(type)) || kc->dim() != 4 ||
          vc->sizes() != kc->sizes())
        return false;
      for (int i = 0; i < 4; ++i) {
        if (!small(kc->size(i))) return false;
      }
      d = {static_cast<int32_t>(kc->size(0)), static_cast<int32_t>(kc->size(1)),
           static_cast<int32_t>(kc->size(2)), static_cast<int32_t>(kc->size(3))};
    }
    if (!(cs = a.whole(ScalarType::Float)) || cs->dim() != 2 ||
        !(pos = a.whole(ScalarType::Int)) || !(slots = a.whole(ScalarType::Int)) ||
        slots->dim() != 1 || q->dim() != 3)
      return false;
    const int64_t T = slots->size(0), P = cs->size(0), R = cs->size(1), Hq = q->size(1);
    if (!small(T) || !small(P) || !small(R) || !small(Hq)) return false;
    kvp_rope_desc rope = {};
    rope.rotary_dim = static_cast<int32_t>(R);
    PyObject* sections = a.take();
    if (sections == Py_None) {
      rope.num_axes = 1;
      rope.sections[0] = static_cast<int32_t>(R / 2);
    } else {
      const bool list = sections != nullptr && PyList_Check(sections);
      if (sections == nullptr || (!list && !PyTuple_Check(sections))) return false;
      const Py_ssize_t axes = list ? PyList_GET_SIZE(sections) : PyTuple_GET_SIZE(sections);
      if (axes < 1 || axes > 4) return false;
      rope.num_axes = static_cast<int32_t>(axes);
      for (Py_ssize_t i = 0; i < axes; ++i) {
        if (!Args::number(list ? PyList_GET_ITEM(sections, i) : PyTuple_GET_ITEM(sections, i),
                          &rope.sections[i]))
          return false;
      }
    }
    PyObject* interleaved = a.take();
    if (interleaved != Py_True && interleaved != Py_False) return false;
    rope.interleaved = interleaved == Py_True;
    int32_t* status;
    if (!a.status(&status)) return false;
    if (!shape(pos, {rope.num_axes, T}) && !(rope.num_axes == 1 && shape(pos, {T}))) return false;
    int64_t qos, qs, ks, vs;
    if (!row_stride(qo, type, T, Hq, d.head_dim, &qos) ||
        !row_stride(q, type, T, Hq, d.head_dim, &qs) ||
        !row_stride(key, type, T, d.num_kv_heads, d.head_dim, &ks) ||
        !row_stride(value, type, T, d.num_kv_heads, d.head_dim, &vs))
      return false;
    const kvp_stream_t st = a.stream();
    if constexpr (kInt4) {
      const WithoutGil guard;
      *s = kvp_rope_append_int4(
          ptr<void>(qo), qos, ptr<void>(q), qs, ptr<void>(key), ks,
          ptr<void>(value), vs, ptr<uint8_t>(p.kc), ptr<uint8_t>(p.vc),
          ptr<void>(p.ks), ptr<void>(p.vs), ptr<float>(cs),
          static_cast<int32_t>(P), ptr<int32_t>(pos), ptr<int32_t>(slots),
          static_cast<int32_t>(T), static_cast<int32_t>(Hq), rope, d, dt, status,
          st);
    } else {
      const WithoutGil guard;
      *s = kvp_rope_append(
          ptr<void>(qo), qos, ptr<void>(q), qs, ptr<void>(key), ks,
          ptr<void>(value), vs, ptr<void>(kc), ptr<void>(vc), ptr<float>(cs),
          static_cast<int32_t>(P), ptr<int32_t>(pos), ptr<int32_t>(slots),
          static_cast<int32_t>(T), static_cast<int32_t>(Hq), rope, d, dt, status,
          st);
    }
    return true;
  });
}

// block_tables, context_lens, new_lens, free_blocks, free_count, context_lens_out,
// free_count_out, slot_mapping, query_start, positions, status
PyObject* extend_tables(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&](kvp_status* s) {
    Args a(args, n);
    const Tensor* t[9];
    for (auto& x : t) {
      if (!(x = a.whole(ScalarType::Int))) return false;
    }
    const Tensor* pos = nullptr;
    int32_t* status;
    if (!a.none() && !(pos = a.whole(ScalarType::Int))) return false;
    if (!a.status(&status) || t[0]->dim() != 2 || t[3]->dim() != 1 || t[7]->dim() != 1) return false;
    const int64_t B = t[0]->size(0), MB = t[0]->size(1), NB = t[3]->size(0), T = t[7]->size(0);
    if (!small(B) || !small(MB) || !small(NB) || !small(T) || !shape(t[1], {B}) ||
        !shape(t[2], {B}) || !shape(t[4], {1}) || !shape(t[5], {B}) || !shape(t[6], {1}) ||
        !shape(t[8], {B + 1}) || (pos != nullptr && !shape(pos, {T})))
      return false;
    const kvp_stream_t st = a.stream();
    const WithoutGil guard;
    *s = kvp_extend_tables(
        ptr<int32_t>(t[0]), static_cast<int32_t>(MB), ptr<int32_t>(t[1]),
        ptr<int32_t>(t[2]), static_cast<int32_t>(B), ptr<int32_t>(t[3]),
        ptr<int32_t>(t[4]), static_cast<int32_t>(NB), ptr<int32_t>(t[5]),
        ptr<int32_t>(t[6]), ptr<int32_t>(t[7]), static_cast<int32_t>(T),
        ptr<int32_t>(t[8]), pos != nullptr ? ptr<int32_t>(pos) : nullptr, status,
        st);
    return true;
  });
}

// block_tables, context_lens, finished, free_blocks, free_count, context_lens_out,
// free_count_out, status
PyObject* release_tables(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&](kvp_status* s) {
    Args a(args, n);
    const Tensor* t[7];
    for (auto& x : t) {
      if (!(x = a.whole(ScalarType::Int))) return false;
    }
    int32_t* status;
    if (!a.status(&status) || t[0]->dim() != 2 || t[3]->dim() != 1) return false;
    const int64_t B = t[0]->size(0), MB = t[0]->size(1), NB = t[3]->size(0);
    if (!small(B) || !small(MB) || !small(NB) || !shape(t[1], {B}) || !shape(t[2], {B}) ||
        !shape(t[4], {1}) || !shape(t[5], {B}) || !shape(t[6], {1}))
      return false;
    const kvp_stream_t st = a.stream();
    const WithoutGil guard;
    *s = kvp_release_tables(
        ptr<int32_t>(t[0]), static_cast<int32_t>(MB), ptr<int32_t>(t[1]),
        ptr<int32_t>(t[2]), static_cast<int32_t>(B), ptr<int32_t>(t[3]),
        ptr<int32_t>(t[4]), static_cast<int32_t>(NB), ptr<int32_t>(t[5]),
        ptr<int32_t>(t[6]), status, st);
    return true;
  });
}

#define KVP_METHOD(name, f) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {KVP_METHOD("append_int4", (&rows_int4<false>)),
                          KVP_METHOD("read_int4", (&rows_int4<true>)),
                          KVP_METHOD("attention_decode_int4", &attention_decode_int4),
                          KVP_METHOD("rope_append", (&rope_append<false>)),
                          KVP_METHOD("rope_append_int4", (&rope_append<true>)),
                          KVP_METHOD("extend_tables", &extend_tables),
                          KVP_METHOD("release_tables", &release_tables),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_kvp_calls", nullptr, -1, kMethods,
                       nullptr,               nullptr,      nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvp_calls() { return PyModule_Create(&kModule); }
