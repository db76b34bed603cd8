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

const int32_t* i32(const at::Tensor* t) { return static_cast<const int32_t*>(t->data_ptr()); }
int32_t* i32(at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }
const int64_t* i64(const at::Tensor* t) { return static_cast<const int64_t*>(t->data_ptr()); }

// What the forms of attention over the cache have in common: q, cache, cu_q, kv_lens, block_table, max_q, scale.
struct Attn {
  const Cache* c;
  const at::Tensor *q, *cu, *kv, *table;
  int64_t max_q, qs, T, Hq, R, most;
  float scale;
  at::Tensor o, lse, ws;
};
constexpr int64_t kMost = int64_t(1) << 31;

// Reads the first seven arguments of a call; false where they do not fit.
bool attn_args(PyObject* const* a, Attn& x) {
  x.c = cache_of(a[1]);
  if (!x.c) return false;
  x.q = tensor(a[0]), x.cu = tensor(a[2]), x.kv = tensor(a[3]), x.table = tensor(a[4]);
  if (!x.q || x.q->dim() != 3 || !number(a[5], x.max_q) || !PyFloat_Check(a[6])) return false;
  const int64_t index = x.c->index;
  x.T = x.q->size(0), x.Hq = x.q->size(1);
  if (x.Hq == 0 || x.Hq % x.c->c.H || !rows(x.q, x.Hq, index, x.qs)) return false;
  if (!flat(x.cu, at::kInt, index) || !flat(x.kv, at::kInt, index) || !flat(x.table, at::kInt, index)) return false;
  x.R = x.kv->numel();
  if (x.R == 0 || x.cu->numel() != x.R + 1 || x.table->dim() != 2 || x.table->size(0) != x.R || x.R >= kMost || x.Hq >= kMost ||
      x.max_q < 0 || x.max_q >= kMost || x.table->size(1) >= kMost || !current(index))
    return false;
  x.most = x.table->size(1) * x.c->c.page;
  x.scale = float(PyFloat_AS_DOUBLE(a[6]));
  return true;
}
// The results, and a workspace of so many bytes (NULL for none).
void* attn_buffers(Attn& x, size_t bytes) {
  const int64_t index = x.c->index;
  x.o = empty(x.q->sizes(), at::kBFloat16, index);
  x.lse = empty({x.Hq, x.T}, at::kFloat, index);
  if (!bytes) return nullptr;
  x.ws = empty({int64_t(bytes)}, at::kByte, index);
  return x.ws.data_ptr();
}

// attention(q, cache, cu_q, kv_lens, block_table, max_q, scale, causal) -> (o, lse), or a status
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Attn x;
    if (n != 8 || !attn_args(a, x) || !PyBool_Check(a[7])) Py_RETURN_NONE;
    const size_t bytes = mxfa_kv_attn_workspace_size(int(x.R), int(x.max_q), x.most, int(x.Hq), x.c->c.H);
    void* const ws = attn_buffers(x, bytes);
    const mxfa_status s = mxfa_kv_attn(&x.c->c, x.q->data_ptr(), x.qs, x.T, i32(x.cu), i32(x.kv), int(x.R), i32(x.table), int(x.table->size(1)),
                                       int(x.max_q), int(x.Hq), x.scale, a[7] == Py_True, x.o.data_ptr(),
                                       static_cast<float*>(x.lse.data_ptr()), ws, bytes, stream(x.c->index));
    return s ? failed(s) : tuple_of({x.o, x.lse});
  });
}

// window(q, cache, cu_q, kv_lens, block_table, max_q, scale, window, sinks) -> (o, lse), or a status
PyObject* window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Attn x;
    int64_t w, sinks;
    if (n != 9 || !attn_args(a, x) || !number(a[7], w) || !number(a[8], sinks) || w < 1 || w >= kMost || sinks < 0 || sinks >= kMost) Py_RETURN_NONE;
    const size_t bytes = mxfa_kv_attn_window_workspace_size(int(x.R), int(x.max_q), x.most, int(x.Hq), x.c->c.H, int(w), int(sinks));
    void* const ws = attn_buffers(x, bytes);
    const mxfa_status s = mxfa_kv_attn_window(&x.c->c, x.q->data_ptr(), x.qs, x.T, i32(x.cu), i32(x.kv), int(x.R), i32(x.table),
                                              int(x.table->size(1)), int(x.max_q), int(x.Hq), x.scale, int(w), int(sinks), x.o.data_ptr(),
                                              static_cast<float*>(x.lse.data_ptr()), ws, bytes, stream(x.c->index));
    return s ? failed(s) : tuple_of({x.o, x.lse});
  });
}

// shared(q, cache, cu_q, kv_lens, block_table, max_q, scale, group_starts, prefix_lens, max_group_q, share) -> (o, lse), or a status
PyObject* shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Attn x;
    int64_t most, share;
    if (n != 11 || !attn_args(a, x) || !number(a[9], most) || most < 0 || most >= kMost || !number(a[10], share) || share < 0 || share > 2)
      Py_RETURN_NONE;
    const at::Tensor *starts = tensor(a[7]), *prefix = tensor(a[8]);
    if (!flat(starts, at::kInt, x.c->index) || !flat(prefix, at::kInt, x.c->index)) Py_RETURN_NONE;
    const int64_t groups = prefix->numel();
    if (groups == 0 || groups >= kMost || starts->numel() != groups + 1) Py_RETURN_NONE;
    const size_t bytes = mxfa_kv_attn_shared_workspace_size_mode(int(x.R), int(groups), x.T, int(x.max_q), int(most), x.most, int(x.Hq),
                                                                 x.c->c.H, int(share));
    void* const ws = attn_buffers(x, bytes);
    const mxfa_status s = mxfa_kv_attn_shared(&x.c->c, x.q->data_ptr(), x.qs, x.T, i32(x.cu), i32(x.kv), int(x.R), i32(x.table),
                                              int(x.table->size(1)), int(x.max_q), int(x.Hq), x.scale, i32(starts), i32(prefix), int(groups),
                                              int(most), int(share), x.o.data_ptr(), static_cast<float*>(x.lse.data_ptr()), ws, bytes, stream(x.c->index));
    return s ? failed(s) : tuple_of({x.o, x.lse});
  });
}

// turns, interleaved, gain -> a rotation
bool rotation(PyObject* const* a, int64_t index, mxfa_rotation& r) {
  const at::Tensor* turns = tensor(a[0]);
  if (!flat(turns, at::kLong, index) || turns->numel() < 1 || turns->numel() > 64 || !PyBool_Check(a[1]) || !PyFloat_Check(a[2])) return false;
  r.turns = i64(turns);
  r.rot = int(2 * turns->numel());
  r.layout = a[1] == Py_True ? MXFA_ROPE_INTERLEAVED : MXFA_ROPE_HALF;
  r.gain = PyFloat_AS_DOUBLE(a[2]);
  return true;
}
PyObject* wrapped(const at::Tensor& t) { return THPVariable_Wrap(t); }

// rope(x, turns, interleaved, gain, positions, inverse) -> y, or a status
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* x = n == 6 ? tensor(a[0]) : nullptr;
    int64_t inverse, xs;
    if (!x || x->dim() != 3 || !x->is_cuda() || !number(a[5], inverse)) Py_RETURN_NONE;
    const int64_t index = x->get_device(), T = x->size(0), H = x->size(1);
    const at::Tensor* pos = tensor(a[4]);
    mxfa_rotation r;
    if (H == 0 || H >= kMost || !rows(x, H, index, xs) || !flat(pos, at::kInt, index) || pos->numel() != T || !rotation(a + 1, index, r) ||
        !current(index))
      Py_RETURN_NONE;
    at::Tensor y = empty(x->sizes(), at::kBFloat16, index);
    const mxfa_status s = mxfa_rope(x->data_ptr(), xs, y.data_ptr(), H * 128, i32(pos), T, int(H), 128, &r, inverse ? 1 : 0, stream(index));
    return s ? failed(s) : wrapped(y);
  });
}

// append_rope(cache, q, k, v, turns, interleaved, gain, positions, slots, out or None) -> q turned, or a status
PyObject* append_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Cache* c = n == 10 ? cache_of(a[0]) : nullptr;
    if (!c) Py_RETURN_NONE;
    const at::Tensor *q = tensor(a[1]), *k = tensor(a[2]), *v = tensor(a[3]), *pos = tensor(a[7]), *slots = tensor(a[8]);
    if (!q || q->dim() != 3 || q->size(1) == 0 || q->size(1) >= kMost) Py_RETURN_NONE;
    const int64_t index = c->index, T = q->size(0), Hq = q->size(1);
    int64_t qs, ks, vs, ys = Hq * 128;
    mxfa_rotation r;
    if (!rows(q, Hq, index, qs) || !rows(k, c->c.H, index, ks) || !rows(v, c->c.H, index, vs) || !flat(pos, at::kInt, index) ||
        !flat(slots, at::kLong, index) || !rotation(a + 4, index, r))
      Py_RETURN_NONE;
    if (k->size(0) != T || v->size(0) != T || pos->numel() != T || slots->numel() != T || !current(index)) Py_RETURN_NONE;
    at::Tensor made;
    const at::Tensor* y = &made;
    if (a[9] == Py_None) {
      made = empty(q->sizes(), at::kBFloat16, index);
    } else {
      y = tensor(a[9]);
      if (!rows(y, Hq, index, ys) || y->size(0) != T) Py_RETURN_NONE;
    }
    const mxfa_status s = mxfa_kv_append_rope(&c->c, q->data_ptr(), qs, int(Hq), k->data_ptr(), ks, v->data_ptr(), vs, T, i32(pos), i64(slots), &r,
                                              y->data_ptr(), ys, stream(index));
    if (s) return failed(s);
    if (a[9] == Py_None) return wrapped(made);
    Py_INCREF(a[9]);
    return a[9];
  });
}

// What fork and free have in common: block_table, three lists, refs, free_ring, ring_state.
struct Pages {
  const at::Tensor *table, *l[3], *refs, *ring, *state;
  int64_t index, F;
};
bool pages_args(PyObject* const* a, Pages& x) {
  x.table = tensor(a[0]), x.refs = tensor(a[4]), x.ring = tensor(a[5]), x.state = tensor(a[6]);
  if (!x.table || !x.table->is_cuda() || x.table->dim() != 2) return false;
  x.index = x.table->get_device();
  for (int i = 0; i < 3; i++) {
    x.l[i] = tensor(a[1 + i]);
    if (!flat(x.l[i], at::kInt, x.index)) return false;
    x.F = x.l[0]->numel();
    if (x.l[i]->numel() != x.F) return false;
  }
  return flat(x.table, at::kInt, x.index) && flat(x.refs, at::kInt, x.index) && flat(x.ring, at::kInt, x.index) &&
         flat(x.state, at::kLong, x.index) && x.state->numel() == 3 && x.table->size(0) < kMost && x.table->size(1) < kMost && x.F < kMost &&
         current(x.index);
}

// fork(block_table, src, dst, lens, refs, free_ring, ring_state, page, gap_first or None, gap_end or None) ->
// (from, to, lens, ring_state), or a status
PyObject* fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Pages x;
    int64_t page;
    if (n != 10 || !pages_args(a, x) || !number(a[7], page) || page < 0 || page > 128) Py_RETURN_NONE;
    const int32_t* gap[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; i++) {
      if (a[8 + i] == Py_None) continue;
      const at::Tensor* t = tensor(a[8 + i]);
      if (!flat(t, at::kInt, x.index) || t->numel() != x.F) Py_RETURN_NONE;
      gap[i] = i32(t);
    }
    at::Tensor from = empty({x.F}, at::kInt, x.index), to = empty({x.F}, at::kInt, x.index), lens = empty({x.F}, at::kInt, x.index),
               out = empty({3}, at::kLong, x.index);
    const mxfa_status s = mxfa_kv_fork_gap(static_cast<int32_t*>(x.table->data_ptr()), int(x.table->size(0)), int(x.table->size(1)),
                                           i32(x.l[0]), i32(x.l[1]), i32(x.l[2]), gap[0], gap[1], int(x.F),
                                           static_cast<int32_t*>(x.refs->data_ptr()), x.refs->numel(), i32(x.ring), x.ring->numel(), i64(x.state),
                                           static_cast<int64_t*>(out.data_ptr()), int(page), i32(from), i32(to), i32(lens), stream(x.index));
    return s ? failed(s) : tuple_of({from, to, lens, out});
  });
}

// free(block_table, rows, first, end, refs, free_ring, ring_state) -> ring_state, or a status
PyObject* free_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Pages x;
    if (n != 7 || !pages_args(a, x)) Py_RETURN_NONE;
    at::Tensor out = empty({3}, at::kLong, x.index);
    const mxfa_status s = mxfa_kv_free(i32(x.table), int(x.table->size(0)), int(x.table->size(1)), i32(x.l[0]), i32(x.l[1]), i32(x.l[2]), int(x.F),
                                       static_cast<int32_t*>(x.refs->data_ptr()), x.refs->numel(), static_cast<int32_t*>(x.ring->data_ptr()),
                                       x.ring->numel(), i64(x.state), static_cast<int64_t*>(out.data_ptr()), stream(x.index));
    return s ? failed(s) : wrapped(out);
  });
}

// copy_blocks(cache, from, to) -> status
PyObject* copy_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Cache* c = n == 3 ? cache_of(a[0]) : nullptr;
    if (!c) Py_RETURN_NONE;
    const at::Tensor *from = tensor(a[1]), *to = tensor(a[2]);
    if (!flat(from, at::kInt, c->index) || !flat(to, at::kInt, c->index) || from->numel() != to->numel() || from->numel() == 0 ||
        from->numel() >= kMost || !current(c->index))
      Py_RETURN_NONE;
    return PyLong_FromLong(mxfa_kv_copy_blocks(&c->c, i32(from), i32(to), int(from->numel()), stream(c->index)));
  });
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(cache), METHOD(append), METHOD(load), METHOD(plan), METHOD(attention),
                         METHOD(window), METHOD(shared), METHOD(rope), METHOD(append_rope), METHOD(fork), METHOD(free_pages),
                         METHOD(copy_blocks), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "kv_py", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kv_py() { return PyModule_Create(&module); }
