// kv_py.cpp -- the 4-bit cache's calls from Python in one step: checks of the tensors,
// allocation of the results, and the call of the C entry point on the current stream.
//
// A decoding step's calls run 3 to 9 us on the GPU, less than the same work takes as
// single Python statements (torch.empty alone is 1.4 us, and twice that after a
// launch has run the driver's code).  These functions take the ordinary call: buffers to
// be allocated, on the current device and stream.  For any other, and for
// arguments that do not fit together, they return None and do nothing: mxfa.py then
// goes through its own checks, which name what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstring>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mxfa.h"

namespace {

// What KvCache keeps of its checked tensors, as bytes.
struct Cache {
  mxfa_kv_cache c;
  int64_t index;
};

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A contiguous tensor of this type on CUDA device `index`.
bool flat(const at::Tensor* t, at::ScalarType type, int64_t index) {
  return t && t->scalar_type() == type && t->is_cuda() && t->get_device() == index && t->is_contiguous();
}

// bf16 [tokens][heads][128] with the heads of a token one after another; `stride` gets
// the elements between tokens.
bool rows(const at::Tensor* x, int64_t heads, int64_t index, int64_t& stride) {
  if (!x || x->scalar_type() != at::kBFloat16 || x->dim() != 3 || !x->is_cuda() || x->get_device() != index) return false;
  const auto size = x->sizes(), step = x->strides();
  if (size[0] == 0 || size[1] != heads || size[2] != 128) return false;
  if (step[2] != 1 || (heads > 1 && step[1] != 128)) return false;
  stride = size[0] > 1 ? step[0] : heads * 128;
  return true;
}

const Cache* cache_of(PyObject* o) {
  if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != Py_ssize_t(sizeof(Cache))) return nullptr;
  return reinterpret_cast<const Cache*>(PyBytes_AS_STRING(o));
}

bool current(int64_t index) { return c10::cuda::current_device() == index; }
mxfa_stream_t stream(int64_t index) {
  return reinterpret_cast<mxfa_stream_t>(c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(index)).stream());
}

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, int64_t index) {
  return at::Tensor(at::detail::empty_cuda(size, type, at::Device(at::kCUDA, c10::DeviceIndex(index)), std::nullopt));
}

// A nonzero status goes back as a number, which mxfa.py raises.
PyObject* failed(mxfa_status s) { return PyLong_FromLong(s); }

PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(Py_ssize_t(ts.size()));
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = r ? THPVariable_Wrap(t) : nullptr;
    if (!o) {
      Py_XDECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// No C++ exception crosses into the interpreter.
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    return nullptr;
  }
}

// cache(k, v, k_sf, v_sf, fmt, k_scale, v_scale) -> (bytes, H, page, index)
PyObject* cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 7) Py_RETURN_NONE;
    const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *ksf = tensor(a[2]), *vsf = tensor(a[3]);
    const long fmt = PyLong_Check(a[4]) ? PyLong_AsLong(a[4]) : -1;
    if (!k || !v || !ksf || !vsf || !k->is_cuda() || (fmt != MXFA_KV_MXFP4 && fmt != MXFA_KV_NVFP4)) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    const int64_t index = k->get_device();
    for (const at::Tensor* t : {k, v, ksf, vsf})
      if (!flat(t, at::kByte, index) || t->dim() != 4) Py_RETURN_NONE;
    const auto size = k->sizes();
    const int64_t sf = fmt == MXFA_KV_MXFP4 ? 4 : 8;
    if (size[3] != 64 || v->sizes() != size || ksf->sizes() != vsf->sizes() || ksf->size(0) != size[0] ||
        ksf->size(1) != size[1] || ksf->size(2) != size[2] || ksf->size(3) != sf || size[0] < 1 || size[1] < 1 ||
        size[1] > 65536 || size[2] < 1 || size[2] > 128)
      Py_RETURN_NONE;
    Cache x;
    std::memset(&x, 0, sizeof(x));
    if (fmt == MXFA_KV_NVFP4) {
      const at::Tensor *ks = tensor(a[5]), *vs = tensor(a[6]);
      if (!flat(ks, at::kFloat, index) || !flat(vs, at::kFloat, index) || ks->numel() != 1 || vs->numel() != 1) Py_RETURN_NONE;
      x.c.k_scale = static_cast<const float*>(ks->data_ptr());
      x.c.v_scale = static_cast<const float*>(vs->data_ptr());
    }
    x.c.k = static_cast<uint8_t*>(k->data_ptr());
    x.c.v = static_cast<uint8_t*>(v->data_ptr());
    x.c.k_sf = static_cast<uint8_t*>(ksf->data_ptr());
    x.c.v_sf = static_cast<uint8_t*>(vsf->data_ptr());
    x.c.num_blocks = size[0];
    x.c.page = int(size[2]);
    x.c.H = int(size[1]);
    x.c.D = 128;
    x.c.fmt = int(fmt);
    x.index = index;
    return Py_BuildValue("(y#LLL)", reinterpret_cast<const char*>(&x), Py_ssize_t(sizeof(x)), (long long)(size[1]),
                         (long long)(size[2]), (long long)(index));
  });
}

// append(cache, k, v, slots) -> status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Cache* c = n == 4 ? cache_of(a[0]) : nullptr;
    if (!c) Py_RETURN_NONE;
    const at::Tensor *k = tensor(a[1]), *v = tensor(a[2]), *slots = tensor(a[3]);
    int64_t ks, vs;
    if (!rows(k, c->c.H, c->index, ks) || !rows(v, c->c.H, c->index, vs) || !flat(slots, at::kLong, c->index)) Py_RETURN_NONE;
    const int64_t T = k->size(0);
    if (v->size(0) != T || slots->numel() != T || !current(c->index)) Py_RETURN_NONE;
    return PyLong_FromLong(mxfa_kv_append(&c->c, k->data_ptr(), v->data_ptr(), ks, vs, T,
                                          static_cast<const int64_t*>(slots->data_ptr()), stream(c->index)));
  });
}

// load(cache, slots) -> (k, v), or a status
PyObject* load(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Cache* c = n == 2 ? cache_of(a[0]) : nullptr;
    if (!c) Py_RETURN_NONE;
    const at::Tensor* slots = tensor(a[1]);
    if (!flat(slots, at::kLong, c->index) || slots->numel() == 0 || !current(c->index)) Py_RETURN_NONE;
    const int64_t T = slots->numel(), size[3] = {T, c->c.H, 128};
    at::Tensor k = empty(size, at::kBFloat16, c->index), v = empty(size, at::kBFloat16, c->index);
    const mxfa_status s = mxfa_kv_load(&c->c, static_cast<const int64_t*>(slots->data_ptr()), T, k.data_ptr(), v.data_ptr(),
                                       stream(c->index));
    return s ? failed(s) : tuple_of({k, v});
  });
}

bool number(PyObject* o, int64_t& x) {
  if (!PyLong_Check(o)) return false;
  int over = 0;
  x = PyLong_AsLongLongAndOverflow(o, &over);
  return !over;
}

// plan(ctx_lens, new_lens, block_table, free_ring, ring_state, page, tokens) -> (cu_q, kv_lens, slots,
// positions, ring_state), or a status
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* ctx = n == 7 ? tensor(a[0]) : nullptr;
    int64_t page, tokens;
    if (!ctx || !ctx->is_cuda() || !number(a[5], page) || !number(a[6], tokens)) Py_RETURN_NONE;
    const int64_t index = ctx->get_device(), R = ctx->numel();
    const at::Tensor *add = tensor(a[1]), *table = tensor(a[2]), *ring = tensor(a[3]), *state = tensor(a[4]);
    if (!flat(ctx, at::kInt, index) || !flat(add, at::kInt, index) || !flat(table, at::kInt, index) ||
        !flat(ring, at::kInt, index) || !flat(state, at::kLong, index))
      Py_RETURN_NONE;
    const int64_t most = int64_t(1) << 31;
    if (add->numel() != R || table->dim() != 2 || table->size(0) != R || state->numel() != 3 || R >= most || tokens < 0 ||
        tokens >= most || table->size(1) >= most || page < 0 || page > 128 || !current(index))
      Py_RETURN_NONE;
    at::Tensor cu = empty({R + 1}, at::kInt, index), kv = empty({R}, at::kInt, index), slots = empty({tokens}, at::kLong, index),
               pos = empty({tokens}, at::kInt, index), out = empty({3}, at::kLong, index);
    auto i32 = [](const at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); };
    auto i64 = [](const at::Tensor& t) { return static_cast<int64_t*>(t.data_ptr()); };
    const mxfa_status s = mxfa_kv_plan(i32(*ctx), i32(*add), int(R), i32(*table), int(table->size(1)), i32(*ring),
                                       ring->numel(), i64(*state), i64(out), int(page), tokens, i32(cu), i32(kv),
                                       i64(slots), i32(pos), stream(index));
    return s ? failed(s) : tuple_of({cu, kv, slots, pos, out});
  });
}

// attention(q, cache, cu_q, kv_lens, block_table, max_q, scale, causal) -> (o, lse), or a status
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Cache* c = n == 8 ? cache_of(a[1]) : nullptr;
    if (!c) Py_RETURN_NONE;
    const at::Tensor *q = tensor(a[0]), *cu = tensor(a[2]), *kv = tensor(a[3]), *table = tensor(a[4]);
    int64_t max_q, qs;
    if (!q || q->dim() != 3 || !number(a[5], max_q) || !PyFloat_Check(a[6]) || !PyBool_Check(a[7])) Py_RETURN_NONE;
    const int64_t T = q->size(0), Hq = q->size(1), index = c->index, most = int64_t(1) << 31;
    if (Hq == 0 || Hq % c->c.H || !rows(q, Hq, index, qs)) Py_RETURN_NONE;
    if (!flat(cu, at::kInt, index) || !flat(kv, at::kInt, index) || !flat(table, at::kInt, index)) Py_RETURN_NONE;
    const int64_t R = kv->numel();
    if (R == 0 || cu->numel() != R + 1 || table->dim() != 2 || table->size(0) != R || R >= most || Hq >= most ||
        max_q < 0 || max_q >= most || table->size(1) >= most || !current(index))
      Py_RETURN_NONE;
    at::Tensor o = empty(q->sizes(), at::kBFloat16, index), lse = empty({Hq, T}, at::kFloat, index), ws;
    const size_t bytes = mxfa_kv_attn_workspace_size(int(R), int(max_q), table->size(1) * c->c.page, int(Hq), c->c.H);
    if (bytes) ws = empty({int64_t(bytes)}, at::kByte, index);
    auto i32 = [](const at::Tensor* t) { return static_cast<const int32_t*>(t->data_ptr()); };
    const mxfa_status s = mxfa_kv_attn(&c->c, q->data_ptr(), qs, T, i32(cu), i32(kv), int(R), i32(table), int(table->size(1)),
                                       int(max_q), int(Hq), float(PyFloat_AS_DOUBLE(a[6])), a[7] == Py_True, o.data_ptr(),
                                       static_cast<float*>(lse.data_ptr()), bytes ? ws.data_ptr() : nullptr, bytes,
                                       stream(index));
    return s ? failed(s) : tuple_of({o, lse});
  });
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(cache), METHOD(append), METHOD(load), METHOD(plan), METHOD(attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "kv_py", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kv_py() { return PyModule_Create(&module); }
