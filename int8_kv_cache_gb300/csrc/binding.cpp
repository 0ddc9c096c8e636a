// The compiled half of the Python binding, for the calls of a decode step:
// rope_and_cache, gather_cache and paged_decode_mx4.  It checks the tensors, makes
// the outputs that were not passed and calls the C entry point of the same name on
// the current stream; the same in Python costs about ten times as long (10 us a
// call on Grace, more than the kernels of a small step).  A status other than
// I8KV_OK comes back as an int, which the Python side turns into its exception.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <optional>
#include <string>

#include "../../include/int8kv.h"

namespace {

struct Refusal {
  PyObject* type;
  std::string text;
};
[[noreturn]] void refuse(PyObject* type, const std::string& text) { throw Refusal{type, text}; }

std::string text_of(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

const at::Tensor& tensor_of(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

void check_type(const at::Tensor& t, const char* name, at::ScalarType dt) {
  if (t.scalar_type() != dt)
    refuse(PyExc_TypeError, std::string(name) + ": expected " + c10::toString(dt) + ", got " +
                                c10::toString(t.scalar_type()));
}

void check_device(const at::Tensor& t, const char* name, int dev) {
  if (!t.is_cuda() || t.get_device() != dev)
    refuse(PyExc_ValueError, std::string(name) + " is on " + t.device().str() +
                                 ", but the library works on the current device, cuda:" +
                                 std::to_string(dev));
}

// Device pointer of a dense tensor; nullptr for None.
void* dense(PyObject* o, const char* name, at::ScalarType dt, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor_of(o, name);
  check_type(t, name, dt);
  check_device(t, name, dev);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
  return t.data_ptr();
}

// The same of a given shape.
void* shaped(PyObject* o, const char* name, at::ScalarType dt, int dev, at::IntArrayRef shape) {
  void* p = dense(o, name, dt, dev);
  if (o != Py_None && THPVariable_Unpack(o).sizes() != shape)
    refuse(PyExc_ValueError, std::string(name) + ": expected shape " + text_of(shape) + ", got " +
                                 text_of(THPVariable_Unpack(o).sizes()));
  return p;
}

// New rows [T, H, D] fp16: heads contiguous, tokens any distance apart.
struct Rows {
  const uint16_t* p;
  int64_t heads, stride;
};
Rows rows_of(PyObject* o, const char* name, int dev, int64_t T, int64_t D) {
  const at::Tensor& t = tensor_of(o, name);
  check_type(t, name, at::kHalf);
  check_device(t, name, dev);
  if (t.dim() != 3 || t.size(0) != T || t.size(2) != D)
    refuse(PyExc_ValueError, std::string(name) + ": expected [" + std::to_string(T) + ", heads, " +
                                 std::to_string(D) + "], got " + text_of(t.sizes()));
  if (t.numel() != 0 && ((t.stride(2) != 1 && D > 1) || (t.stride(1) != D && t.size(1) > 1)))
    refuse(PyExc_ValueError, std::string(name) + ": the heads of a token must be contiguous");
  return Rows{static_cast<const uint16_t*>(t.data_ptr()), t.size(1), t.stride(0)};
}

struct Cache {
  void *k, *v;
  int32_t dtype, block_size;
  int64_t slots, Hkv, D, blocks;
};
Cache mx4_of(PyObject* o, const char* name, int dev) {
  Cache c{};
  const at::Tensor& t = tensor_of(o, name);
  c.k = dense(o, name, at::kByte, dev);
  if (t.dim() != 4 || t.size(3) % 18 != 0)
    refuse(PyExc_ValueError, std::string(name) +
                                 ": expected [num_blocks, Hkv, block_size / 16, 18 * D], got " +
                                 text_of(t.sizes()));
  c.dtype = I8KV_CACHE_MX4;
  c.blocks = t.size(0);
  c.Hkv = t.size(1);
  c.block_size = static_cast<int32_t>(16 * t.size(2));
  c.D = t.size(3) / 18;
  c.slots = c.blocks * c.block_size;
  return c;
}
// The cache type: an MX4 record cache has no v_cache of its own.
int32_t cache_type(PyObject* k, PyObject* v) {
  const at::Tensor& t = tensor_of(k, "k_cache");
  if (v == Py_None) {
    check_type(t, "k_cache (no v_cache: an MX4 cache)", at::kByte);
    return I8KV_CACHE_MX4;
  }
  switch (t.scalar_type()) {
    case at::kChar: return I8KV_CACHE_INT8;
    case at::kByte:
    case at::kFloat8_e4m3fn: return I8KV_CACHE_FP8;
    case at::kHalf: return I8KV_CACHE_FP16;
    default:
      refuse(PyExc_TypeError, std::string("unsupported cache dtype ") + c10::toString(t.scalar_type()));
  }
}
Cache cache_of(PyObject* k, PyObject* v, int32_t dtype, int dev) {
  if (dtype == I8KV_CACHE_MX4) return mx4_of(k, "k_cache", dev);
  Cache c{};
  c.dtype = dtype;
  const at::Tensor& t = tensor_of(k, "k_cache");
  if (t.dim() != 3 && t.dim() != 4)
    refuse(PyExc_ValueError,
           "k_cache: expected [num_slots, Hkv, D] or [num_blocks, block_size, Hkv, D], got " +
               text_of(t.sizes()));
  c.k = dense(k, "k_cache", t.scalar_type(), dev);
  c.v = shaped(v, "v_cache", t.scalar_type(), dev, t.sizes());
  c.Hkv = t.size(-2);
  c.D = t.size(-1);
  c.block_size = 16;
  c.slots = c.Hkv * c.D > 0 ? t.numel() / (c.Hkv * c.D) : 0;
  return c;
}

struct Scales {
  const float *k, *v;
};
Scales scales_of(PyObject* k, PyObject* v, int32_t kind, const Cache& c, int dev) {
  if (c.dtype == I8KV_CACHE_FP16) return Scales{nullptr, nullptr};
  if (k == Py_None || v == Py_None)
    refuse(PyExc_ValueError, "k_scale and v_scale are needed for a quantised cache");
  const int64_t n = kind == I8KV_SCALE_PER_CHANNEL ? c.Hkv * c.D : 1;
  const auto one = [&](PyObject* o, const char* name) {
    const float* p = static_cast<const float*>(dense(o, name, at::kFloat, dev));
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.numel() != n)
      refuse(PyExc_ValueError, std::string(name) + ": expected " + std::to_string(n) +
                                   " values, got " + std::to_string(t.numel()));
    // [Hkv, D] or the same in a row, dimensions of one aside: the channels are the last
    int64_t last = 1;
    for (const int64_t d : t.sizes()) last = d != 1 ? d : last;
    if (n > 1 && last != c.D && last != n)
      refuse(PyExc_ValueError, std::string(name) + ": expected shape " + text_of({c.Hkv, c.D}) +
                                   ", got " + text_of(t.sizes()));
    return p;
  };
  return Scales{one(k, "k_scale"), one(v, "v_scale")};
}

int32_t int_of(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, std::string(name) + " must be an int");
  }
  if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " is out of range");
  return static_cast<int32_t>(v);
}
float float_of(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, std::string(name) + " must be a number");
  }
  return static_cast<float>(v);
}
int32_t size32(int64_t v, const char* name) {
  if (v > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " is too large");
  return static_cast<int32_t>(v);
}

// The stream to work on: None is the current one, else a cudaStream_t as an int, which
// is then current for the outputs made here (their memory must not be in use on another).
struct Stream {
  void* handle;
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  Stream(PyObject* o, int dev) {
    const auto index = static_cast<c10::DeviceIndex>(dev);
    if (o == Py_None) {
      handle = c10::cuda::getCurrentCUDAStream(index).stream();
    } else {
      handle = PyLong_AsVoidPtr(o);
      guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), index));
    }
  }
};

// The interpreter runs other threads while the C entry point enqueues: a launch waits where the
// queue of launches is full.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// The current device; a tensor on the host is refused before the device is asked for.
int device_of(PyObject* o, const char* name) {
  const at::Tensor& t = tensor_of(o, name);
  if (!t.is_cuda())
    refuse(PyExc_ValueError,
           std::string(name) + " is on " + t.device().str() + ", not on the current device");
  return static_cast<int>(c10::cuda::current_device());
}

PyObject* status(i8kv_status s) { return PyLong_FromLong(s); }

bool wrong_count(const char* name, Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return false;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, got);
  return true;
}

// (q, k_new, v_new, positions, cos_sin, slot_mapping, k_cache, v_cache, k_scale, v_scale,
//  scale_kind, interleaved, q_out, flags, stream)
PyObject* py_rope_and_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (wrong_count("rope_and_cache", n, 15)) return nullptr;
  try {
    const int32_t dtype = cache_type(a[6], a[7]);
    const int dev = device_of(a[6], "k_cache");
    const Cache c = cache_of(a[6], a[7], dtype, dev);
    const at::Tensor& kt = tensor_of(a[1], "k_new");
    if (kt.dim() != 3) refuse(PyExc_ValueError, "k_new: expected [T, Hkv, D], got " + text_of(kt.sizes()));
    const int64_t T = kt.size(0);
    const Rows k = rows_of(a[1], "k_new", dev, T, c.D), v = rows_of(a[2], "v_new", dev, T, c.D);
    if (k.heads != c.Hkv || v.heads != c.Hkv)
      refuse(PyExc_ValueError, "k_new / v_new have " + std::to_string(k.heads) + " / " +
                                   std::to_string(v.heads) + " heads, the cache " + std::to_string(c.Hkv));
    const void* pos = nullptr;
    const void* cs = nullptr;
    int64_t max_pos = 0, R = 0;
    if (a[4] != Py_None) {
      cs = dense(a[4], "cos_sin", at::kFloat, dev);
      const at::Tensor& t = THPVariable_Unpack(a[4]);
      if (t.dim() != 2) refuse(PyExc_ValueError, "cos_sin must be [max_pos, rot_dim]");
      max_pos = t.size(0);
      R = t.size(1);
      pos = shaped(a[3], "positions", at::kInt, dev, {T});
    }
    const void* slots = shaped(a[5], "slot_mapping", at::kInt, dev, {T});
    const int32_t kind = int_of(a[10], "scale_kind");
    const Scales s = scales_of(a[8], a[9], kind, c, dev);
    const int style = PyObject_IsTrue(a[11]);
    if (style < 0) return nullptr;
    void* flags = dense(a[13], "flags", at::kInt, dev);
    const Stream stream(a[14], dev);
    Rows q{nullptr, 0, 0};
    PyObject* out = a[12];
    at::Tensor made;
    void* qo = nullptr;
    if (a[0] != Py_None) {
      q = rows_of(a[0], "q", dev, T, c.D);
      if (out == Py_None) {
        made = at::empty({T, q.heads, c.D}, THPVariable_Unpack(a[0]).options());
        qo = made.data_ptr();
      } else {
        qo = shaped(out, "q_out", at::kHalf, dev, {T, q.heads, c.D});
      }
    } else if (out != Py_None) {
      refuse(PyExc_ValueError, "q_out without q");
    }
    const int32_t tokens = size32(T, "T"), Hq = size32(q.heads, "Hq"), Hkv = size32(c.Hkv, "Hkv");
    const int32_t D = size32(c.D, "D"), rot = size32(R, "rot_dim");
    const i8kv_status st = [&] {
      const Unlocked other_threads_run;
      return rope_and_cache(q.p, q.stride, k.p, k.stride, v.p, v.stride,
                            static_cast<const int32_t*>(pos), static_cast<const float*>(cs), max_pos,
                            rot, style ? I8KV_ROPE_INTERLEAVED : I8KV_ROPE_HALVES,
                            static_cast<const int32_t*>(slots), tokens, Hq, Hkv, D,
                            static_cast<uint16_t*>(qo), c.k, c.v, c.dtype, c.slots, c.block_size,
                            s.k, s.v, kind, static_cast<uint32_t*>(flags), stream.handle);
    }();
    if (st != I8KV_OK) return status(st);
    if (made.defined()) return THPVariable_Wrap(made);
    return Py_NewRef(out);
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (slot_mapping, k_cache, v_cache, k_scale, v_scale, scale_kind, k_out, v_out, flags, stream)
PyObject* py_gather_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (wrong_count("gather_cache", n, 10)) return nullptr;
  try {
    const int32_t dtype = cache_type(a[1], a[2]);
    const int dev = device_of(a[1], "k_cache");
    const Cache c = cache_of(a[1], a[2], dtype, dev);
    const void* slots = dense(a[0], "slot_mapping", at::kInt, dev);
    const at::Tensor& t = tensor_of(a[0], "slot_mapping");
    if (t.dim() != 1) refuse(PyExc_ValueError, "slot_mapping: expected [N], got " + text_of(t.sizes()));
    const int64_t N = t.size(0);
    const int32_t kind = int_of(a[5], "scale_kind");
    const Scales s = scales_of(a[3], a[4], kind, c, dev);
    void* flags = dense(a[8], "flags", at::kInt, dev);
    const Stream stream(a[9], dev);
    const auto options = THPVariable_Unpack(a[1]).options().dtype(at::kHalf);
    at::Tensor made[2];
    void* p[2];
    const char* names[2] = {"k_out", "v_out"};
    for (int i = 0; i < 2; ++i) {
      if (a[6 + i] == Py_None) {
        made[i] = at::empty({N, c.Hkv, c.D}, options);
        p[i] = made[i].data_ptr();
      } else {
        p[i] = shaped(a[6 + i], names[i], at::kHalf, dev, {N, c.Hkv, c.D});
      }
    }
    const int32_t rows = size32(N, "N"), Hkv = size32(c.Hkv, "Hkv"), D = size32(c.D, "D");
    const i8kv_status st = [&] {
      const Unlocked other_threads_run;
      return gather_cache(static_cast<const int32_t*>(slots), rows, Hkv, D, c.k, c.v, c.dtype,
                          c.slots, c.block_size, s.k, s.v, kind, static_cast<uint16_t*>(p[0]),
                          static_cast<uint16_t*>(p[1]), static_cast<uint32_t*>(flags),
                          stream.handle);
    }();
    if (st != I8KV_OK) return status(st);
    PyObject* r = PyTuple_New(2);
    if (r == nullptr) return nullptr;
    for (int i = 0; i < 2; ++i)
      PyTuple_SET_ITEM(r, i, made[i].defined() ? THPVariable_Wrap(made[i]) : Py_NewRef(a[6 + i]));
    return r;
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (q, cache, k_scale, v_scale, scale_kind, block_table, seq_lens, softmax_scale, head_sink,
//  num_splits, chunk, workspace, out, lse, flags, stream, partials_only, softcap, window)
PyObject* py_paged_decode_mx4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (wrong_count("paged_decode_mx4", n, 19)) return nullptr;
  try {
    check_type(tensor_of(a[1], "cache"), "cache", at::kByte);
    const int dev = device_of(a[1], "cache");
    const Cache c = mx4_of(a[1], "cache", dev);
    const void* q = dense(a[0], "q", at::kHalf, dev);
    const at::Tensor& qt = tensor_of(a[0], "q");
    if (qt.dim() != 3 || qt.size(2) != c.D)
      refuse(PyExc_ValueError, "q: expected [B, Hq, " + std::to_string(c.D) + "], got " + text_of(qt.sizes()));
    const int64_t B = qt.size(0), Hq = qt.size(1);
    const void* table = dense(a[5], "block_table", at::kInt, dev);
    const at::Tensor& bt = tensor_of(a[5], "block_table");
    if (bt.dim() != 2 || bt.size(0) != B)
      refuse(PyExc_ValueError, "block_table: expected [" + std::to_string(B) + ", max_blocks], got " +
                                   text_of(bt.sizes()));
    tensor_of(a[6], "seq_lens");
    const void* lens = shaped(a[6], "seq_lens", at::kInt, dev, {B});
    const int32_t kind = int_of(a[4], "scale_kind");
    const Scales s = scales_of(a[2], a[3], kind, c, dev);
    const void* sink = shaped(a[8], "head_sink", at::kFloat, dev, {Hq});
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (a[11] != Py_None) {
      const at::Tensor& w = tensor_of(a[11], "workspace");
      ws = dense(a[11], "workspace", w.scalar_type(), dev);
      ws_bytes = w.nbytes();
    }
    void* lse = shaped(a[13], "lse", at::kFloat, dev, {B, Hq});
    void* flags = dense(a[14], "flags", at::kInt, dev);
    const int partials = PyObject_IsTrue(a[16]);
    if (partials < 0) return nullptr;
    const Stream stream(a[15], dev);
    at::Tensor made;
    void* out = nullptr;
    if (!partials) {
      if (a[12] == Py_None) {
        made = at::empty({B, Hq, c.D}, qt.options());
        out = made.data_ptr();
      } else {
        out = shaped(a[12], "out", at::kHalf, dev, qt.sizes());
      }
    }
    const int32_t rows = size32(B, "B"), heads = size32(Hq, "Hq"), Hkv = size32(c.Hkv, "Hkv");
    const int32_t D = size32(c.D, "D"), max_blocks = size32(bt.size(1), "max_blocks");
    const float sigma = float_of(a[7], "softmax_scale"), softcap = float_of(a[17], "softcap");
    const int32_t window = int_of(a[18], "window"), splits = int_of(a[9], "num_splits");
    const int32_t chunk = int_of(a[10], "chunk");
    const i8kv_status st = [&] {
      const Unlocked other_threads_run;
      return paged_decode_mx4(static_cast<const uint16_t*>(q), c.k, s.k, s.v, kind,
                              static_cast<const int32_t*>(table), static_cast<const int32_t*>(lens),
                              rows, heads, Hkv, D, c.block_size, max_blocks, c.blocks, sigma,
                              static_cast<const float*>(sink), softcap, window, splits, chunk, ws,
                              ws_bytes, static_cast<uint16_t*>(out), static_cast<float*>(lse),
                              static_cast<uint32_t*>(flags), stream.handle);
    }();
    if (st != I8KV_OK) return status(st);
    if (made.defined()) return THPVariable_Wrap(made);
    return Py_NewRef(partials ? Py_None : a[12]);
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"rope_and_cache", reinterpret_cast<PyCFunction>(py_rope_and_cache), METH_FASTCALL, nullptr},
    {"gather_cache", reinterpret_cast<PyCFunction>(py_gather_cache), METH_FASTCALL, nullptr},
    {"paged_decode_mx4", reinterpret_cast<PyCFunction>(py_paged_decode_mx4), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
