// pkv_binding.cpp -- Python arguments of the rotated appends, of latent
// attention, of attention weights and of eviction, checked and handed to libpkv's
// entry points.
//
// A decode step's append is 2 us of GPU work.  Its checks of a dozen tensors
// and the marshalling of 18 arguments took 13 us through Python and ctypes (20
// between other calls, which have the caches), and take 2.7 (6.5) here, where a
// check is a few loads from the tensor's own fields.  The entry points are
// those of the library that the package has loaded, by address (bind), so
// status words and counts are the same ones.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>
#include <optional>
#include <type_traits>

#include "pkv.h"

namespace {

constexpr int64_t kLatentDim = 512, kLatentRope = 64, kLatentRow = kLatentDim + kLatentRope;

struct Raised {};  // a Python error is set

#define RAISE(type, ...)                         \
  do {                                           \
    PyErr_Format(PyExc_##type, __VA_ARGS__);     \
    throw Raised{};                              \
  } while (0)

decltype(&pkv_write_rope) g_write_rope;
decltype(&pkv_write_rope_fp8) g_write_rope_fp8;
decltype(&pkv_write_rope_axes) g_write_rope_axes;
decltype(&pkv_write_rope_axes_fp8) g_write_rope_axes_fp8;
decltype(&pkv_write_latent) g_write_latent;
decltype(&pkv_attend_latent) g_attend_latent;
decltype(&pkv_attend_latent_workspace_size) g_workspace_size;
decltype(&pkv_weigh) g_weigh;
decltype(&pkv_weigh_fp8) g_weigh_fp8;
decltype(&pkv_weigh_workspace_size) g_weigh_size;
decltype(&pkv_evict) g_evict;
decltype(&pkv_evict_fp8) g_evict_fp8;
decltype(&pkv_evict_workspace_size) g_evict_size;
PyObject* g_error;  // PkvError

const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    default: return "torch.uint8";
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) RAISE(TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

void need_dtype(PyObject* o, const at::Tensor& t, const char* name, at::ScalarType dtype) {
  if (t.scalar_type() == dtype) return;
  PyObject* got = PyObject_GetAttrString(o, "dtype");
  if (got) PyErr_Format(PyExc_TypeError, "%s must be %s, got %S", name, name_of(dtype), got);
  Py_XDECREF(got);
  throw Raised{};
}

void need_device(const at::Tensor& t, const char* name, int index) {
  if (!t.is_cuda()) RAISE(ValueError, "%s must be a CUDA tensor", name);
  if (t.get_device() != index)
    RAISE(ValueError, "%s is on cuda:%d, not on cuda:%d like the cache", name, int(t.get_device()), index);
}

[[noreturn]] void bad_shape(PyObject* o, const char* name, const char* want) {
  PyObject* got = PyObject_GetAttrString(o, "shape");
  if (got) PyErr_Format(PyExc_ValueError, "%s must be %s, got shape %S", name, want, got);
  Py_XDECREF(got);
  throw Raised{};
}

// A contiguous tensor of this type and number of dimensions on device `index`.
const at::Tensor& take(PyObject* o, const char* name, at::ScalarType dtype, int ndim, int index) {
  const at::Tensor& t = tensor(o, name);
  need_dtype(o, t, name, dtype);
  need_device(t, name, index);
  if (!t.is_contiguous()) RAISE(ValueError, "%s must be contiguous", name);
  if (t.dim() != ndim) bad_shape(o, name, ndim == 1 ? "[n]" : ndim == 2 ? "[n, m]" : ndim == 3 ? "of 3 dimensions"
                                                                                            : "of 4 dimensions");
  return t;
}

int32_t i32(int64_t v, const char* name) {
  if (v < 0 || v > INT32_MAX) RAISE(ValueError, "%s has more than 2^31 - 1 of something", name);
  return int32_t(v);
}

template <class T>
T* in(const at::Tensor& t) {
  return const_cast<T*>(static_cast<const T*>(t.const_data_ptr()));
}
template <class T>
T* inout(const at::Tensor& t) {
  return static_cast<T*>(t.mutable_data_ptr());
}

// bf16 [tokens, heads, dim], or [tokens, dim] where heads is 0: a token's
// elements contiguous, any token stride that keeps 16-byte alignment.
struct Rows {
  const pkv_bf16* at;
  int64_t stride;
};
Rows take_rows(PyObject* o, const char* name, int64_t tokens, int64_t heads, int64_t dim, int index) {
  const at::Tensor& t = tensor(o, name);
  need_dtype(o, t, name, at::kBFloat16);
  need_device(t, name, index);
  const int nd = heads ? 3 : 2;
  if (t.dim() != nd || t.size(0) != tokens || t.size(nd - 1) != dim || (heads && t.size(1) != heads))
    bad_shape(o, name, heads ? "[tokens, heads, head_dim] like the cache and the other inputs" : "[tokens, dim] of its part");
  if (t.stride(nd - 1) != 1 || (heads > 1 && t.stride(1) != dim))
    RAISE(ValueError, "a token's elements of %s must be contiguous", name);
  const int64_t row = dim * (heads ? heads : 1);
  if (tokens < 2) return {in<pkv_bf16>(t), row};
  if (t.stride(0) < row || t.stride(0) % 8)
    RAISE(ValueError, "%s's token stride must be a multiple of 8 elements and no less than a token", name);
  return {in<pkv_bf16>(t), t.stride(0)};
}

// The stream of a call: the argument's, or the device's current one.
struct Stream {
  std::optional<c10::cuda::CUDAStream> given;
  pkv_stream_t handle;
  Stream(PyObject* o, int index) {
    if (o == Py_None) {
      handle = c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(index)).stream();
      return;
    }
    PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
    if (!h) throw Raised{};
    handle = static_cast<pkv_stream_t>(PyLong_AsVoidPtr(h));
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Raised{};
    given = c10::cuda::getStreamFromExternal(handle, c10::DeviceIndex(index));
  }
  // an uninitialised tensor that belongs to the stream it is used on
  at::Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, int index) const {
    c10::cuda::OptionalCUDAStreamGuard guard;
    if (given) guard.reset_stream(*given);
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(c10::Device(at::kCUDA, c10::DeviceIndex(index))));
  }
};

// Without the interpreter's lock for as long as it lives, however that ends.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// call(): the entry point's code, with device `index` current.
template <class F>
void run(const char* what, int index, F call) {
  int code;
  {
    c10::cuda::CUDAGuard guard{c10::DeviceIndex(index)};
    Unlocked unlocked;
    code = call();
  }
  if (code != PKV_OK) {
    PyObject* args = Py_BuildValue("(is)", code, what);
    if (args) PyErr_SetObject(g_error, args);
    Py_XDECREF(args);
    throw Raised{};
  }
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

int device_of(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return int(v);
}

double number_of(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    if (PyErr_ExceptionMatches(PyExc_TypeError))
      RAISE(TypeError, "%s must be a float, got %s", name, Py_TYPE(o)->tp_name);
    throw Raised{};
  }
  return v;
}

int64_t whole_of(PyObject* whole) {  // takes over the reference
  if (!whole) throw Raised{};
  int overflow = 0;
  const int64_t v = PyLong_AsLongLongAndOverflow(whole, &overflow);
  Py_DECREF(whole);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return overflow > 0 ? INT64_MAX : overflow < 0 ? INT64_MIN : v;
}

// A host-side bound: what is negative counts as 0, what is above `top` as top.
int64_t bound_of(PyObject* o, int64_t top) { return std::clamp<int64_t>(whole_of(PyNumber_Long(o)), 0, top); }

int64_t int_of(PyObject* o, const char* name) {
  if (!PyIndex_Check(o)) RAISE(TypeError, "%s must be an int, got %s", name, Py_TYPE(o)->tp_name);
  return whole_of(PyNumber_Index(o));
}

pkv_rope rope_of(PyObject* o, PyObject* interleaved, int index) {
  const at::Tensor& t = take(o, "cos_sin", at::kFloat, 2, index);
  return {in<float>(t), i32(t.size(0), "cos_sin"), i32(t.size(1), "cos_sin"), truth(interleaved)};
}

PyObject* result(PyObject* given, const at::Tensor& made) {
  if (made.defined()) return THPVariable_Wrap(made);
  return Py_NewRef(given);
}

void need_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) RAISE(TypeError, "%zd arguments, not %zd", want, n);
}

// The axis of each of `pairs` pairs: bytes, or a list or tuple of numbers.
void axes_of(PyObject* o, int64_t pairs, uint8_t* axis) {
  if (PyBytes_Check(o)) {
    if (PyBytes_GET_SIZE(o) != pairs) RAISE(ValueError, "axes must name the axis of each of rotary_dim / 2 pairs");
    const char* at = PyBytes_AS_STRING(o);
    for (int64_t i = 0; i < pairs; ++i) axis[i] = uint8_t(at[i]);
    return;
  }
  if (!PyList_Check(o) && !PyTuple_Check(o))
    RAISE(TypeError, "axes must be bytes, a list or a tuple, got %s", Py_TYPE(o)->tp_name);
  if (PySequence_Fast_GET_SIZE(o) != pairs)
    RAISE(ValueError, "axes must name the axis of each of rotary_dim / 2 pairs");
  for (int64_t i = 0; i < pairs; ++i) {
    PyObject* item = PySequence_Fast_GET_ITEM(o, i);
    const long v = PyLong_AsLong(item);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v < 0 || v > UINT8_MAX) RAISE(ValueError, "axes must be axes of positions");
    axis[i] = uint8_t(v);
  }
}

// (index, stream, k_new, v_new, positions, cos_sin, slot_mapping, k_cache,
//  v_cache, q, q_out, interleaved[, k_scale, v_scale][, axes])
template <bool F8, bool AXES>
PyObject* write_rope(PyObject* const* a, Py_ssize_t n) {
  need_args(n, (F8 ? 14 : 12) + AXES);
  const int index = device_of(a[0]);
  constexpr at::ScalarType kind = F8 ? at::kByte : at::kBFloat16;
  const at::Tensor& kc = take(a[7], "k_cache", kind, 4, index);
  const at::Tensor& vc = take(a[8], "v_cache", kind, 4, index);
  if (kc.sizes() != vc.sizes()) RAISE(ValueError, "k_cache and v_cache shapes disagree");
  uint8_t *ks = nullptr, *vs = nullptr;
  if constexpr (F8) {
    const at::Tensor& s = take(a[12], "k_scale", at::kByte, 3, index);
    const at::Tensor& u = take(a[13], "v_scale", at::kByte, 3, index);
    if (s.sizes() != kc.sizes().slice(0, 3) || u.sizes() != s.sizes())
      RAISE(ValueError, "FP8 pools must be codes [NB, Hkv, P, D] and scales [NB, Hkv, P]");
    ks = inout<uint8_t>(s);
    vs = inout<uint8_t>(u);
  }
  const at::Tensor& k_new = tensor(a[2], "k_new");
  const int64_t T = k_new.dim() ? k_new.size(0) : -1, hkv = kc.size(1), D = kc.size(3);
  const Rows k = take_rows(a[2], "k_new", T, hkv, D, index), v = take_rows(a[3], "v_new", T, hkv, D, index);
  const at::Tensor& pos = AXES ? tensor(a[4], "positions") : take(a[4], "positions", at::kLong, 1, index);
  if constexpr (AXES) {  // [num_axes, T], a slice of a longer buffer or one row for all axes too
    need_dtype(a[4], pos, "positions", at::kLong);
    need_device(pos, "positions", index);
    if (pos.dim() != 2) bad_shape(a[4], "positions", "[axes, tokens]");
    if (T > 1 && pos.stride(1) != 1) RAISE(ValueError, "an axis's positions must be contiguous");
  }
  const at::Tensor& slots = take(a[6], "slot_mapping", at::kLong, 1, index);
  if (pos.size(AXES ? 1 : 0) != T || slots.size(0) != T)
    RAISE(ValueError, "k_new, positions and slot_mapping disagree on the number of tokens");
  const pkv_rope rope = rope_of(a[5], a[11], index);
  uint8_t axis[128];
  pkv_rope_axes several{};
  if constexpr (AXES) {
    if (pos.size(0) < 1 || pos.size(0) > PKV_MAX_AXES) RAISE(ValueError, "positions must have 1 to %d axes", PKV_MAX_AXES);
    if (rope.rotary_dim > int32_t(2 * sizeof axis)) bad_shape(a[5], "cos_sin", "[max_position, rotary_dim]");
    axes_of(a[F8 ? 14 : 12], rope.rotary_dim / 2, axis);
    for (int32_t i = 0; i < rope.rotary_dim / 2; ++i)
      if (axis[i] >= pos.size(0)) RAISE(ValueError, "axes must be axes of positions");
    several = {rope.cos_sin, rope.max_position, rope.rotary_dim, rope.interleaved, int32_t(pos.size(0)), axis};
  }
  const Stream stream(a[1], index);
  Rows q{nullptr, 0};
  pkv_bf16* q_out = nullptr;
  int64_t hq = hkv;
  at::Tensor made;
  if (a[9] != Py_None) {
    const at::Tensor& t = tensor(a[9], "q");
    hq = t.dim() == 3 ? t.size(1) : 0;
    q = take_rows(a[9], "q", T, hq, D, index);
    if (hq == 0) bad_shape(a[9], "q", "[tokens, Hq, head_dim]");
    if (a[10] == Py_None) {
      made = stream.fresh(t.sizes(), at::kBFloat16, index);
      q_out = inout<pkv_bf16>(made);
    } else {
      const at::Tensor& o = take(a[10], "q_out", at::kBFloat16, 3, index);
      if (o.sizes() != t.sizes()) RAISE(ValueError, "q_out must have q's shape");
      q_out = inout<pkv_bf16>(o);
    }
  } else if (a[10] != Py_None) {
    RAISE(ValueError, "q_out without q");
  }
  const pkv_desc desc{i32(kc.size(0), "k_cache"), i32(kc.size(2), "k_cache"), i32(hkv, "k_cache"),
                      i32(hq, "q"),               i32(D, "k_cache"),          1};
  const int64_t *p = in<int64_t>(pos), *s = in<int64_t>(slots);
  [[maybe_unused]] const int64_t ps = AXES ? pos.stride(0) : 0;
  if constexpr (F8) {
    auto *kp = inout<pkv_fp8>(kc), *vp = inout<pkv_fp8>(vc);
    run(AXES ? "pkv_write_rope_axes_fp8" : "pkv_write_rope_fp8", index, [&] {
      if constexpr (AXES)
        return g_write_rope_axes_fp8(q.at, k.at, v.at, q.stride, k.stride, v.stride, p, ps, s, T, &several,
                                     q_out, kp, vp, ks, vs, &desc, stream.handle);
      return g_write_rope_fp8(q.at, k.at, v.at, q.stride, k.stride, v.stride, p, s, T, &rope, q_out, kp, vp, ks, vs,
                              &desc, stream.handle);
    });
  } else {
    auto *kp = inout<pkv_bf16>(kc), *vp = inout<pkv_bf16>(vc);
    run(AXES ? "pkv_write_rope_axes" : "pkv_write_rope", index, [&] {
      if constexpr (AXES)
        return g_write_rope_axes(q.at, k.at, v.at, q.stride, k.stride, v.stride, p, ps, s, T, &several,
                                 q_out, kp, vp, &desc, stream.handle);
      return g_write_rope(q.at, k.at, v.at, q.stride, k.stride, v.stride, p, s, T, &rope, q_out, kp, vp, &desc,
                          stream.handle);
    });
  }
  return result(a[10], made);
}

// (index, stream, c_new, k_pe, positions, cos_sin, slot_mapping, latent_cache,
//  q_pe, q_out, interleaved)
PyObject* write_latent(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 11);
  const int index = device_of(a[0]);
  const at::Tensor& pool = take(a[7], "latent_cache", at::kBFloat16, 3, index);
  const at::Tensor& c_new = tensor(a[2], "c_new");
  const int64_t T = c_new.dim() ? c_new.size(0) : -1;
  const Rows c = take_rows(a[2], "c_new", T, 0, kLatentDim, index);
  const Rows k = take_rows(a[3], "k_pe", T, 0, kLatentRope, index);
  const at::Tensor& pos = take(a[4], "positions", at::kLong, 1, index);
  const at::Tensor& slots = take(a[6], "slot_mapping", at::kLong, 1, index);
  if (pos.size(0) != T || slots.size(0) != T)
    RAISE(ValueError, "c_new, positions and slot_mapping disagree on the number of tokens");
  const pkv_rope rope = rope_of(a[5], a[10], index);
  const Stream stream(a[1], index);
  const pkv_bf16* q_pe = nullptr;
  pkv_bf16* q_out = nullptr;
  int64_t heads = 1, qs = 0, hs = 0;
  at::Tensor made;
  if (a[8] != Py_None) {
    const at::Tensor& t = tensor(a[8], "q_pe");
    need_dtype(a[8], t, "q_pe", at::kBFloat16);
    need_device(t, "q_pe", index);
    if (t.dim() != 3 || t.size(0) != T || t.size(2) != kLatentRope || t.stride(2) != 1)
      bad_shape(a[8], "q_pe", "[tokens, H, 64] with contiguous rows");
    heads = t.size(1);
    hs = heads > 1 ? t.stride(1) : kLatentRope;
    qs = T > 1 ? t.stride(0) : std::max<int64_t>(heads, 1) * hs;
    if (hs < kLatentRope || hs % 8 || qs < (heads - 1) * hs + kLatentRope || qs % 8)
      RAISE(ValueError, "q_pe's strides must be multiples of 8 elements and its rows must not overlap");
    q_pe = in<pkv_bf16>(t);
    const int64_t shape[3] = {T, heads, kLatentRow};
    if (a[9] == Py_None) {
      made = stream.fresh(shape, at::kBFloat16, index);
      q_out = inout<pkv_bf16>(made);
    } else {
      const at::Tensor& o = take(a[9], "q_out", at::kBFloat16, 3, index);
      if (o.sizes() != at::IntArrayRef(shape)) bad_shape(a[9], "q_out", "[tokens, H, 576]");
      q_out = inout<pkv_bf16>(o);
    }
  } else if (a[9] != Py_None) {
    RAISE(ValueError, "q_out without q_pe");
  }
  const pkv_desc desc{i32(pool.size(0), "latent_cache"), i32(pool.size(1), "latent_cache"), 1, i32(heads, "q_pe"),
                      i32(pool.size(2), "latent_cache"), 1};
  const int64_t *p = in<int64_t>(pos), *s = in<int64_t>(slots);
  auto* cache = inout<pkv_bf16>(pool);
  run("pkv_write_latent", index, [&] {
    return g_write_latent(c.at, k.at, q_pe, c.stride, k.stride, qs, hs, p, s, T, &rope, q_out, cache, &desc,
                          stream.handle);
  });
  return result(a[9], made);
}

// (index, stream, q, latent_cache, block_tables, seq_lens, query_start_loc,
//  scale, out, workspace, max_query_len)
PyObject* attend_latent(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 11);
  const int index = device_of(a[0]);
  const at::Tensor& pool = take(a[3], "latent_cache", at::kBFloat16, 3, index);
  const at::Tensor& q = take(a[2], "q", at::kBFloat16, 3, index);
  const at::Tensor& tables = take(a[4], "block_tables", at::kInt, 2, index);
  const at::Tensor& lens = take(a[5], "seq_lens", at::kInt, 1, index);
  const at::Tensor& qsl = take(a[6], "query_start_loc", at::kInt, 1, index);
  const int64_t B = lens.size(0);
  if (qsl.size(0) != B + 1 || tables.size(0) != B)
    RAISE(ValueError, "seq_lens [B], query_start_loc [B+1] and block_tables [B, M] disagree");
  if (pool.size(2) != q.size(2)) RAISE(ValueError, "latent_cache and q rows disagree");
  const double scale = number_of(a[7], "scale");
  const int32_t max_query_len = int32_t(bound_of(a[10], INT32_MAX));
  const pkv_desc desc{i32(pool.size(0), "latent_cache"), i32(pool.size(1), "latent_cache"), 1, i32(q.size(1), "q"),
                      i32(q.size(2), "q"),               i32(tables.size(1), "block_tables")};
  const int32_t seqs = i32(B, "seq_lens"), tokens = i32(q.size(0), "q");
  const Stream stream(a[1], index);
  const int64_t shape[3] = {q.size(0), q.size(1), kLatentDim};
  at::Tensor made, scratch;
  pkv_bf16* out;
  if (a[8] == Py_None) {
    made = stream.fresh(shape, at::kBFloat16, index);
    out = inout<pkv_bf16>(made);
  } else {
    const at::Tensor& o = take(a[8], "out", at::kBFloat16, 3, index);
    if (o.sizes() != at::IntArrayRef(shape)) bad_shape(a[8], "out", "[tokens, H, 512]");
    out = inout<pkv_bf16>(o);
  }
  if (a[9] == Py_None) {
    size_t bytes = 0;
    run("pkv_attend_latent_workspace_size", index,
        [&] { return g_workspace_size(&desc, seqs, tokens, &bytes); });
    scratch = stream.fresh({int64_t(bytes)}, at::kByte, index);
  } else {
    scratch = take(a[9], "workspace", at::kByte, 1, index);
  }
  void* ws = inout<void>(scratch);
  const size_t ws_bytes = size_t(scratch.size(0));
  // (here, with the interpreter's lock: a tensor without memory of its own raises)
  const auto *qp = in<pkv_bf16>(q), *cache = in<pkv_bf16>(pool);
  const int32_t *bt = in<int32_t>(tables), *sl = in<int32_t>(lens), *starts = in<int32_t>(qsl);
  run("pkv_attend_latent", index, [&] {
    return g_attend_latent(qp, cache, bt, sl, starts, seqs, tokens, max_query_len, float(scale), out, ws, ws_bytes,
                           &desc, stream.handle);
  });
  return result(a[8], made);
}

// An int32 number a sequence, or nothing.
const int32_t* per_sequence(PyObject* o, const char* name, int64_t seqs, int index) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = take(o, name, at::kInt, 1, index);
  if (t.size(0) != seqs) RAISE(ValueError, "%s must have a number for each sequence", name);
  return in<int32_t>(t);
}

// (index, stream, q, k_cache, scores, block_tables, seq_lens, query_start_loc,
//  scale, decay, first, scored, workspace, max_query_len, num_keys[, k_scale])
template <bool F8>
PyObject* weigh(PyObject* const* a, Py_ssize_t n) {
  need_args(n, F8 ? 16 : 15);
  const int index = device_of(a[0]);
  const at::Tensor& kc = take(a[3], "k_cache", F8 ? at::kByte : at::kBFloat16, 4, index);
  const at::Tensor& q = take(a[2], "q", at::kBFloat16, 3, index);
  const at::Tensor& scores = take(a[4], "scores", at::kFloat, 3, index);
  const at::Tensor& tables = take(a[5], "block_tables", at::kInt, 2, index);
  const at::Tensor& lens = take(a[6], "seq_lens", at::kInt, 1, index);
  const at::Tensor& qsl = take(a[7], "query_start_loc", at::kInt, 1, index);
  const int64_t B = lens.size(0);
  if (qsl.size(0) != B + 1 || tables.size(0) != B)
    RAISE(ValueError, "seq_lens [B], query_start_loc [B+1] and block_tables [B, M] disagree");
  if (kc.size(3) != q.size(2)) RAISE(ValueError, "k_cache and q shapes disagree");
  if (scores.sizes() != kc.sizes().slice(0, 3)) RAISE(ValueError, "scores must be [NB, Hkv, P] like k_cache");
  [[maybe_unused]] const uint8_t* ks = nullptr;
  if constexpr (F8) {
    const at::Tensor& s = take(a[15], "k_scale", at::kByte, 3, index);
    if (s.sizes() != kc.sizes().slice(0, 3))
      RAISE(ValueError, "FP8 pools must be codes [NB, Hkv, P, D] and scales [NB, Hkv, P]");
    ks = in<uint8_t>(s);
  }
  const float scale = float(number_of(a[8], "scale")), decay = float(number_of(a[9], "decay"));
  const int32_t* first = per_sequence(a[10], "first", B, index);
  const int32_t* scored = per_sequence(a[11], "scored", B, index);
  const int32_t most = int32_t(std::clamp<int64_t>(int_of(a[13], "max_query_len"), 0, INT32_MAX));
  const int64_t keys = std::max<int64_t>(int_of(a[14], "num_keys"), 0);
  const pkv_desc desc{i32(kc.size(0), "k_cache"), i32(kc.size(2), "k_cache"), i32(kc.size(1), "k_cache"),
                      i32(q.size(1), "q"),        i32(kc.size(3), "k_cache"), i32(tables.size(1), "block_tables")};
  const int32_t seqs = i32(B, "seq_lens"), tokens = i32(q.size(0), "q");
  const Stream stream(a[1], index);
  at::Tensor scratch;
  if (a[12] == Py_None) {
    size_t bytes = 0;
    run("pkv_weigh_workspace_size", index, [&] { return g_weigh_size(&desc, seqs, tokens, most, keys, &bytes); });
    scratch = stream.fresh({int64_t(bytes)}, at::kByte, index);
  } else {
    scratch = take(a[12], "workspace", at::kByte, 1, index);
  }
  void* ws = inout<void>(scratch);
  const size_t ws_bytes = size_t(scratch.size(0));
  const auto* qp = in<pkv_bf16>(q);
  auto* sp = inout<float>(scores);
  const int32_t *bt = in<int32_t>(tables), *sl = in<int32_t>(lens), *starts = in<int32_t>(qsl);
  if constexpr (F8) {
    const auto* kp = in<pkv_fp8>(kc);
    run("pkv_weigh_fp8", index, [&] {
      return g_weigh_fp8(qp, kp, ks, sp, bt, sl, starts, first, scored, seqs, tokens, most, keys, scale, decay, ws,
                         ws_bytes, &desc, stream.handle);
    });
  } else {
    const auto* kp = in<pkv_bf16>(kc);
    run("pkv_weigh", index, [&] {
      return g_weigh(qp, kp, sp, bt, sl, starts, first, scored, seqs, tokens, most, keys, scale, decay, ws, ws_bytes,
                     &desc, stream.handle);
    });
  }
  return Py_NewRef(Py_None);
}

// (index, stream, k_cache, v_cache, scores, block_tables, seq_lens, keep,
//  first, recent, new_lens, workspace[, k_scale, v_scale])
template <bool F8>
PyObject* evict(PyObject* const* a, Py_ssize_t n) {
  need_args(n, F8 ? 14 : 12);
  const int index = device_of(a[0]);
  constexpr at::ScalarType kind = F8 ? at::kByte : at::kBFloat16;
  const at::Tensor& kc = take(a[2], "k_cache", kind, 4, index);
  const at::Tensor& vc = take(a[3], "v_cache", kind, 4, index);
  if (kc.sizes() != vc.sizes()) RAISE(ValueError, "k_cache and v_cache shapes disagree");
  const at::Tensor& scores = take(a[4], "scores", at::kFloat, 3, index);
  if (scores.sizes() != kc.sizes().slice(0, 3)) RAISE(ValueError, "scores must be [NB, Hkv, P] like k_cache");
  uint8_t *ks = nullptr, *vs = nullptr;
  if constexpr (F8) {
    const at::Tensor& s = take(a[12], "k_scale", at::kByte, 3, index);
    const at::Tensor& u = take(a[13], "v_scale", at::kByte, 3, index);
    if (s.sizes() != kc.sizes().slice(0, 3) || u.sizes() != s.sizes())
      RAISE(ValueError, "FP8 pools must be codes [NB, Hkv, P, D] and scales [NB, Hkv, P]");
    ks = inout<uint8_t>(s);
    vs = inout<uint8_t>(u);
  }
  const at::Tensor& tables = take(a[5], "block_tables", at::kInt, 2, index);
  const at::Tensor& lens = take(a[6], "seq_lens", at::kInt, 1, index);
  const int64_t B = lens.size(0);
  if (tables.size(0) != B) RAISE(ValueError, "seq_lens [B] and block_tables [B, M] disagree");
  if (a[7] == Py_None) RAISE(TypeError, "keep must be a torch.Tensor");
  const int32_t* keep = per_sequence(a[7], "keep", B, index);
  const int32_t* first = per_sequence(a[8], "first", B, index);
  const int64_t recent = int_of(a[9], "recent");
  if (recent < 0) RAISE(ValueError, "recent must not be negative");
  const int32_t last = int32_t(std::min<int64_t>(recent, INT32_MAX));
  const pkv_desc desc{i32(kc.size(0), "k_cache"), i32(kc.size(2), "k_cache"), i32(kc.size(1), "k_cache"),
                      i32(kc.size(1), "k_cache"), i32(kc.size(3), "k_cache"), i32(tables.size(1), "block_tables")};
  const int32_t seqs = i32(B, "seq_lens");
  const Stream stream(a[1], index);
  at::Tensor made, scratch;
  int32_t* out;
  if (a[10] == Py_None) {
    made = stream.fresh({B}, at::kInt, index);
    out = inout<int32_t>(made);
  } else {
    const at::Tensor& o = take(a[10], "new_lens", at::kInt, 1, index);
    if (o.size(0) != B) RAISE(ValueError, "new_lens must have a number for each sequence");
    out = inout<int32_t>(o);
  }
  if (a[11] == Py_None) {
    size_t bytes = 0;
    run("pkv_evict_workspace_size", index, [&] { return g_evict_size(&desc, seqs, &bytes); });
    scratch = stream.fresh({int64_t(bytes)}, at::kByte, index);
  } else {
    scratch = take(a[11], "workspace", at::kByte, 1, index);
  }
  void* ws = inout<void>(scratch);
  const size_t ws_bytes = size_t(scratch.size(0));
  auto* sp = inout<float>(scores);
  const int32_t *bt = in<int32_t>(tables), *sl = in<int32_t>(lens);
  if constexpr (F8) {
    auto *kp = inout<pkv_fp8>(kc), *vp = inout<pkv_fp8>(vc);
    run("pkv_evict_fp8", index, [&] {
      return g_evict_fp8(kp, vp, ks, vs, sp, bt, sl, keep, first, last, seqs, out, ws, ws_bytes, &desc, stream.handle);
    });
  } else {
    auto *kp = inout<pkv_bf16>(kc), *vp = inout<pkv_bf16>(vc);
    run("pkv_evict", index, [&] {
      return g_evict(kp, vp, sp, bt, sl, keep, first, last, seqs, out, ws, ws_bytes, &desc, stream.handle);
    });
  }
  return result(a[10], made);
}

// (PkvError, addresses of the entry points in the order below)
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 14);
  Py_ssize_t next = 1;
  auto take_address = [&](auto& entry) {
    void* at = PyLong_AsVoidPtr(a[next++]);
    if (PyErr_Occurred()) throw Raised{};
    entry = reinterpret_cast<std::remove_reference_t<decltype(entry)>>(at);
  };
  take_address(g_write_rope);
  take_address(g_write_rope_fp8);
  take_address(g_write_rope_axes);
  take_address(g_write_rope_axes_fp8);
  take_address(g_write_latent);
  take_address(g_attend_latent);
  take_address(g_workspace_size);
  take_address(g_weigh);
  take_address(g_weigh_fp8);
  take_address(g_weigh_size);
  take_address(g_evict);
  take_address(g_evict_fp8);
  take_address(g_evict_size);
  Py_XSETREF(g_error, Py_NewRef(a[0]));
  return Py_NewRef(Py_None);
}

// No C++ exception leaves an entry point.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(args, n);
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<bind>("bind"),
                           method<write_rope<false, false>>("write_rope"),
                           method<write_rope<true, false>>("write_rope_fp8"),
                           method<write_rope<false, true>>("write_rope_axes"),
                           method<write_rope<true, true>>("write_rope_axes_fp8"),
                           method<weigh<false>>("weigh"),
                           method<weigh<true>>("weigh_fp8"),
                           method<evict<false>>("evict"),
                           method<evict<true>>("evict_fp8"),
                           method<write_latent>("write_latent"),
                           method<attend_latent>("attend_latent"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_pkv_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__pkv_binding() { return PyModule_Create(&g_module); }
