// Python face of the MXFP4 entry points (module _mxfp4): argument checks,
// output and workspace allocation, the current stream, and the call.
//
// The calls are short: a decoding step's kernels take a few microseconds, and
// in Python the checks, allocations and ctypes conversions of one call took
// 9-21 us on the GPU's host.  PyTorch still provides device memory and
// streams only; the C functions come by address from the loaded library
// (bind), so this module links against no kernel.
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <optional>
#include <string>

#include "mxfp4.h"

namespace {

using at::Tensor;

struct Api {
  decltype(&mxfp4_quantize) quantize;
  decltype(&mxfp4_dequantize) dequantize;
  decltype(&mxfp4_gemm) gemm;
  decltype(&mxfp4_linear_workspace_bytes) linear_workspace_bytes;
  decltype(&mxfp4_linear) linear;
  decltype(&mxfp4_cache_write) cache_write;
  decltype(&mxfp4_cache_read) cache_read;
  decltype(&mxfp4_attention_workspace_bytes) attention_workspace_bytes;
  decltype(&mxfp4_cache_attention) cache_attention;
};
Api api = {};
PyObject* check_fn = nullptr;  // _lib.check: raises for a status

// A Python exception is set; unwinds to the function's boundary.
struct Raised {};

[[noreturn]] void bad(const char* msg) {
  PyErr_SetString(PyExc_ValueError, msg);
  throw Raised();
}
[[noreturn]] void bad(const std::string& msg) { bad(msg.c_str()); }

constexpr const char* kOneDevice = "tensors must be on one CUDA device";

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
int64_t whole(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
at::ScalarType scalar_type(PyObject* o) {
  if (!THPDtype_Check(o)) bad("dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}
int32_t code_of(at::ScalarType t, const char* name, bool fp32 = true) {
  if (t == at::kBFloat16) return MXFP4_BF16;
  if (t == at::kHalf) return MXFP4_FP16;
  if (t == at::kFloat && fp32) return MXFP4_FP32;
  bad(std::string(name) + (fp32 ? " must be bfloat16, float16 or float32" : " must be bfloat16 or float16"));
}
c10::DeviceIndex cuda_index(const Tensor& t) {
  if (!t.is_cuda()) bad("tensors must be on a CUDA device");
  return t.get_device();
}
void on(const Tensor& t, c10::DeviceIndex dev) {
  if (!t.is_cuda() || t.get_device() != dev) bad(kOneDevice);
}
Tensor empty(at::IntArrayRef sizes, at::ScalarType t, c10::DeviceIndex dev) {
  return at::detail::empty_cuda(sizes, t, at::Device(at::kCUDA, dev), std::nullopt);
}
// Where a call runs: the current stream, or the given one, which is then the
// current one for the call, so that the workspaces it takes and gives back and
// the outputs it allocates belong to the stream that works in them.
class Launch {
 public:
  Launch(PyObject* stream, c10::DeviceIndex dev) : device_(dev), caller_(c10::cuda::getCurrentCUDAStream(dev)) {
    cudaStream_t s = caller_.stream();
    if (stream != Py_None) {
      PyObject* h = PyObject_GetAttrString(stream, "cuda_stream");
      if (!h) throw Raised();
      const unsigned long long v = PyLong_AsUnsignedLongLong(h);
      Py_DECREF(h);
      if (PyErr_Occurred()) throw Raised();
      if (reinterpret_cast<cudaStream_t>(v) != s) {
        s = reinterpret_cast<cudaStream_t>(v);
        guard_.emplace(s == nullptr ? c10::cuda::getDefaultCUDAStream(dev) : c10::cuda::getStreamFromExternal(s, dev));
      }
    }
    handle_ = reinterpret_cast<nvfp4_stream_t>(s);
  }
  nvfp4_stream_t handle() const { return handle_; }
  // The tensor for the caller, who uses a new one on the stream that was current
  // (`given`: it is the caller's own).
  PyObject* result(const Tensor& t, bool given = false) const {
    if (guard_ && !given && t.numel() > 0)
      c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), caller_);
    return THPVariable_Wrap(t);
  }

 private:
  c10::cuda::CUDAGuard device_;
  c10::cuda::CUDAStream caller_;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
  nvfp4_stream_t handle_;
};
void done(nvfp4_status st, const char* name) {
  if (st == NVFP4_OK) return;
  PyObject* r = PyObject_CallFunction(check_fn, "is", int(st), name);
  Py_XDECREF(r);
  if (r) PyErr_SetString(PyExc_RuntimeError, name);  // not reached: check raises
  throw Raised();
}
uint32_t* status_of(PyObject* o, c10::DeviceIndex dev) {
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(o, "status");
  on(t, dev);
  if (t.element_size() < 4 || t.numel() < 1) bad("status must hold 32 bits");
  return static_cast<uint32_t*>(t.data_ptr());
}

// The operators have no backward pass: a result that looked differentiable would
// cut the graph silently.  (Codes and scales are whole numbers, which have none.)
void no_graph(const Tensor& t, const char* name) {
  if (t.requires_grad() && at::GradMode::is_enabled())
    bad(std::string(name) + " requires a gradient, which this operator does not have: detach it, or call under "
        "torch.no_grad()");
}

struct Mat {
  int32_t code;
  int64_t rows, cols, ld;
};
Mat matrix(const Tensor& x, const char* name) {
  Mat m;
  m.code = code_of(x.scalar_type(), name);
  if (x.dim() != 2) bad(std::string(name) + " must be a 2-D tensor");
  m.rows = x.size(0), m.cols = x.size(1);
  if (x.stride(1) != 1 && m.cols > 1) bad(std::string(name) + " must have unit stride along its rows");
  m.ld = m.rows > 1 ? x.stride(0) : m.cols;
  return m;
}

struct Mx {
  const Tensor& q;
  const Tensor& s;
  int64_t rows, cols;
};
// The MXFP4 matrix in args[0..3], whose buffers can hold its rows and columns.
Mx mx(PyObject* const* a, const char* name) {
  Mx m{tensor(a[0], name), tensor(a[1], name), whole(a[2]), whole(a[3])};
  if (m.q.scalar_type() != at::kByte || m.s.scalar_type() != at::kByte || !m.q.is_contiguous() ||
      !m.s.is_contiguous())
    bad(std::string(name) + ".qdata and " + name + ".scales must be contiguous uint8 tensors");
  if (m.rows < 1 || m.cols < 1) bad(std::string(name) + " must have rows and columns");
  const int64_t groups = (m.cols + 127) / 128;
  if (m.q.numel() < m.rows * groups * 64 || m.s.numel() < (m.rows + 127) / 128 * groups * 512)
    bad(std::string(name) + "'s buffers are too small for [" + std::to_string(m.rows) + ", " + std::to_string(m.cols) +
        "]");
  on(m.s, cuda_index(m.q));
  return m;
}

struct Out {
  Tensor t;
  int32_t code;
  int64_t ld;
};
// The given output, checked, or a new one.
Out output(PyObject* o, int64_t rows, int64_t cols, PyObject* dtype, at::ScalarType fallback, c10::DeviceIndex dev) {
  if (o == Py_None) {
    const at::ScalarType t = dtype == Py_None ? fallback : scalar_type(dtype);
    const int32_t code = code_of(t, "dtype");
    return {empty({rows, cols}, t, dev), code, cols};
  }
  const Tensor& t = tensor(o, "out");
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    bad("out must be [" + std::to_string(rows) + ", " + std::to_string(cols) + "]");
  on(t, dev);
  const Mat m = matrix(t, "out");
  return {t, m.code, m.ld};
}

struct Cache {
  mxfp4_cache c;
  c10::DeviceIndex dev;
};
// The cache in args[0..3]: codes and scales of keys, codes and scales of values.
Cache cache(PyObject* const* a) {
  const Tensor &k = tensor(a[0], "cache.k_codes"), &ks = tensor(a[1], "cache.k_scales"),
               &v = tensor(a[2], "cache.v_codes"), &vs = tensor(a[3], "cache.v_scales");
  if (k.dim() != 4 || v.dim() != 4 || ks.dim() != 4 || vs.dim() != 4)
    bad("cache codes must be [pages, kv_heads, page_size, dim / 2], scales [pages, kv_heads, page_size, dim / 32]");
  for (int i = 0; i < 4; ++i)
    if (v.size(i) != k.size(i) || ks.size(i) != (i < 3 ? k.size(i) : k.size(3) / 16) || vs.size(i) != ks.size(i))
      bad("the cache's codes and scales do not fit together");
  if (k.numel() == 0) bad("the cache must have pages, kv_heads, a page_size and a dim");
  const c10::DeviceIndex dev = cuda_index(k);
  for (const Tensor* t : {&k, &ks, &v, &vs}) {
    if (t->scalar_type() != at::kByte || !t->is_contiguous())
      bad("the cache's buffers must be contiguous uint8 tensors");
    on(*t, dev);
  }
  auto narrow = [](int64_t n) { return int32_t(n < 0x7FFFFFFF ? n : 0x7FFFFFFF); };
  return {{k.data_ptr(), ks.data_ptr(), v.data_ptr(), vs.data_ptr(), k.size(0), narrow(k.size(2)), narrow(k.size(1)),
           narrow(k.size(3) * 2), 0},
          dev};
}

const Tensor& ints(PyObject* o, at::ScalarType t, int dims, const char* name, c10::DeviceIndex dev) {
  const Tensor& x = tensor(o, name);
  if (x.scalar_type() != t || x.dim() != dims || !x.is_contiguous())
    bad(std::string(name) + " must be a contiguous " + std::to_string(dims) + "-D " +
        (t == at::kInt ? "int32" : "int64") + " tensor");
  on(x, dev);
  return x;
}

const Tensor& heads_of(PyObject* o, const mxfp4_cache& c, const char* name, c10::DeviceIndex dev) {
  const Tensor& x = tensor(o, name);
  if (x.dim() != 3 || x.size(1) != c.kv_heads || x.size(2) != c.dim)
    bad(std::string(name) + " must be [tokens, " + std::to_string(c.kv_heads) + ", " + std::to_string(c.dim) + "]");
  if (x.stride(2) != 1) bad(std::string(name) + " must have unit stride along its last dimension");
  on(x, dev);
  return x;
}

// quantize(x, qdata | None, scales | None, stream) -> (qdata, scales, rows, cols)
PyObject* quantize(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const Mat m = matrix(x, "x");
  const c10::DeviceIndex dev = cuda_index(x);
  const Launch on_stream(a[3], dev);
  Tensor q, s;
  if (a[1] == Py_None) {
    const int64_t groups = (m.cols + 127) / 128;
    q = empty({m.rows, groups * 64}, at::kByte, dev);
    s = empty({(m.rows + 127) / 128 * groups * 512}, at::kByte, dev);
  } else {
    PyObject* sizes[4] = {a[1], a[2], PyLong_FromLongLong(m.rows), PyLong_FromLongLong(m.cols)};
    const Mx out = mx(sizes, "out");
    Py_DECREF(sizes[2]), Py_DECREF(sizes[3]);
    on(out.q, dev);
    q = out.q, s = out.s;
  }
  if (m.rows > 0 && m.cols > 0)
    done(api.quantize(x.data_ptr(), m.code, m.rows, m.cols, m.ld, q.data_ptr(), s.data_ptr(), on_stream.handle()),
         "mxfp4_quantize");
  const bool given = a[1] != Py_None;
  return Py_BuildValue("NNLL", on_stream.result(q, given), on_stream.result(s, given), (long long)m.rows,
                       (long long)m.cols);
}

// dequantize(qdata, scales, rows, cols, dtype, out | None, stream) -> out
PyObject* dequantize(PyObject* const* a) {
  const int64_t rows = whole(a[2]), cols = whole(a[3]);
  const c10::DeviceIndex dev = cuda_index(tensor(a[0], "t.qdata"));
  const Launch on_stream(a[6], dev);
  Out o = output(a[5], rows, cols, a[4], at::kBFloat16, dev);
  if (rows > 0 && cols > 0) {
    const Mx t = mx(a, "t");
    done(api.dequantize(t.q.data_ptr(), t.s.data_ptr(), rows, cols, o.t.data_ptr(), o.code, o.ld,
                        on_stream.handle()),
         "mxfp4_dequantize");
  }
  return on_stream.result(o.t, a[5] != Py_None);
}

// gemm(a: qdata, scales, rows, cols, w: qdata, scales, rows, cols, dtype, out | None, status | None, stream) -> out
PyObject* gemm(PyObject* const* a) {
  const Mx x = mx(a, "a"), w = mx(a + 4, "w");
  if (x.cols != w.cols) bad("activation and weight K differ");
  const c10::DeviceIndex dev = cuda_index(x.q);
  on(w.q, dev);
  const Launch on_stream(a[11], dev);
  Out o = output(a[9], x.rows, w.rows, a[8], at::kBFloat16, dev);
  done(api.gemm(x.q.data_ptr(), x.s.data_ptr(), w.q.data_ptr(), w.s.data_ptr(), x.rows, w.rows, x.cols,
                o.t.data_ptr(), o.code, o.ld, status_of(a[10], dev), on_stream.handle()),
       "mxfp4_gemm");
  return on_stream.result(o.t, a[9] != Py_None);
}

// linear(x, w: qdata, scales, rows, cols, dtype | None, out | None, status | None, stream) -> out
PyObject* linear(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const Mat m = matrix(x, "x");
  no_graph(x, "x");
  const Mx w = mx(a + 1, "w");
  if (m.cols != w.cols) bad("activation and weight K differ");
  const c10::DeviceIndex dev = cuda_index(x);
  on(w.q, dev);
  const Launch on_stream(a[8], dev);
  Out o = output(a[6], m.rows, w.rows, a[5], x.scalar_type(), dev);
  if (m.rows > 0) {
    const int64_t need = api.linear_workspace_bytes(m.rows, m.cols);
    Tensor ws;
    if (need > 0) ws = empty({need}, at::kByte, dev);
    done(api.linear(x.data_ptr(), m.code, m.rows, m.ld, w.q.data_ptr(), w.s.data_ptr(), w.rows, m.cols,
                    o.t.data_ptr(), o.code, o.ld, need > 0 ? ws.data_ptr() : nullptr, need, status_of(a[7], dev),
                    on_stream.handle()),
         "mxfp4_linear");
  }
  return on_stream.result(o.t, a[6] != Py_None);
}

// cache_write(cache x 4, k, v, slots, stream)
PyObject* cache_write(PyObject* const* a) {
  const Cache c = cache(a);
  const Tensor &k = heads_of(a[4], c.c, "k", c.dev), &v = heads_of(a[5], c.c, "v", c.dev);
  if (k.scalar_type() != v.scalar_type() || k.size(0) != v.size(0))
    bad("k and v must have one type and one number of tokens");
  const Tensor& slots = ints(a[6], at::kLong, 1, "slots", c.dev);
  if (slots.size(0) != k.size(0)) bad("slots must have an entry for each token");
  const int32_t code = code_of(k.scalar_type(), "k");
  const Launch on_stream(a[7], c.dev);
  done(api.cache_write(&c.c, k.data_ptr(), v.data_ptr(), code, k.size(0), k.stride(0), k.stride(1), v.stride(0),
                       v.stride(1), static_cast<const int64_t*>(slots.data_ptr()), on_stream.handle()),
       "mxfp4_cache_write");
  Py_RETURN_NONE;
}

// cache_read(cache x 4, table, starts, total, dtype, stream) -> (k, v)
PyObject* cache_read(PyObject* const* a) {
  const Cache c = cache(a);
  const Tensor &table = ints(a[4], at::kInt, 2, "table", c.dev), &starts = ints(a[5], at::kInt, 1, "starts", c.dev);
  const int64_t total = whole(a[6]);
  const at::ScalarType t = scalar_type(a[7]);
  const int32_t code = code_of(t, "dtype");
  if (starts.size(0) != table.size(0) + 1) bad("starts must have an entry for each sequence and one more");
  if (total < 0) bad("total must not be negative");
  if (total > 0 && table.size(0) == 0) bad("total must be 0 without sequences");
  const Launch on_stream(a[8], c.dev);
  Tensor k = empty({total, c.c.kv_heads, c.c.dim}, t, c.dev), v = empty({total, c.c.kv_heads, c.c.dim}, t, c.dev);
  done(api.cache_read(&c.c, static_cast<const int32_t*>(table.data_ptr()), table.size(1), table.size(0),
                      static_cast<const int32_t*>(starts.data_ptr()), total, k.data_ptr(), v.data_ptr(), code,
                      on_stream.handle()),
       "mxfp4_cache_read");
  return Py_BuildValue("NN", on_stream.result(k), on_stream.result(v));
}

// cache_attention(q, cache x 4, table, lens, q_starts | None, max_queries | None, scale | None, causal, window, sinks,
//                 out | None, lse | None, status | None, stream) -> out
PyObject* cache_attention(PyObject* const* a) {
  const Cache c = cache(a + 1);
  const Tensor& q = tensor(a[0], "q");
  if (q.dim() != 3 || q.size(2) != c.c.dim || q.size(1) == 0 || q.size(1) % c.c.kv_heads != 0)
    bad("q must be [total, multiple of " + std::to_string(c.c.kv_heads) + ", " + std::to_string(c.c.dim) + "]");
  if (q.stride(2) != 1) bad("q must have unit stride along its last dimension");
  no_graph(q, "q");
  on(q, c.dev);
  const Tensor &table = ints(a[5], at::kInt, 2, "table", c.dev), &lens = ints(a[6], at::kInt, 1, "lens", c.dev);
  const int64_t seqs = lens.size(0), total = q.size(0), heads = q.size(1);
  if (table.size(0) != seqs) bad("table must have a row for each sequence");
  mxfp4_attention g = {};
  g.dtype = code_of(q.scalar_type(), "q", false);
  int64_t most = a[8] == Py_None ? total : whole(a[8]);
  if (a[7] == Py_None) {
    if (total != seqs || (a[8] != Py_None && most != 1)) bad("without q_starts every sequence has one query");
    most = 1;
  } else {
    const Tensor& starts = ints(a[7], at::kInt, 1, "q_starts", c.dev);
    if (starts.size(0) != seqs + 1) bad("q_starts must have an entry for each sequence and one more");
    g.q_starts = static_cast<const int32_t*>(starts.data_ptr());
    most = most < total ? most : total;
  }
  const int64_t window = whole(a[11]), sinks = whole(a[12]);
  if (most < 0 || window < 0 || sinks < 0) bad("max_queries, window and sinks must not be negative");
  if (total > 0 && (seqs == 0 || most == 0)) bad("q has rows, but lens or max_queries leave no query");
  if (total > 0x7FFFFFFF || seqs > 0x7FFFFFFF || heads > 0x7FFFFFFF) bad("q is too large");
  if (a[9] == Py_None) {
    g.scale = float(1.0 / std::sqrt(double(c.c.dim)));
  } else {
    const double s = PyFloat_AsDouble(a[9]);
    if (s == -1.0 && PyErr_Occurred()) throw Raised();
    g.scale = float(s);
  }
  const int causal = PyObject_IsTrue(a[10]);
  if (causal < 0) throw Raised();
  const Launch on_stream(a[16], c.dev);
  Tensor out;
  if (a[13] == Py_None) {
    out = empty({total, heads, c.c.dim}, q.scalar_type(), c.dev);
  } else {
    out = tensor(a[13], "out");
    if (out.dim() != 3 || out.size(0) != total || out.size(1) != heads || out.size(2) != c.c.dim ||
        out.scalar_type() != q.scalar_type() || out.stride(2) != 1)
      bad("out must have q's shape and type and unit stride along its last dimension");
    if ((total > 1 && out.stride(0) == 0) || (heads > 1 && out.stride(1) == 0)) bad("out must not overlap itself");
    on(out, c.dev);
  }
  if (a[14] != Py_None) {
    const Tensor& lse = tensor(a[14], "lse");
    if (lse.scalar_type() != at::kFloat || lse.dim() != 2 || lse.size(0) != total || lse.size(1) != heads ||
        !lse.is_contiguous())
      bad("lse must be a contiguous float32 [total, q_heads] tensor");
    on(lse, c.dev);
    g.lse = static_cast<float*>(lse.data_ptr());
  }
  if (total > 0 && seqs > 0 && most > 0) {
    const int64_t need = api.attention_workspace_bytes(c.c.kv_heads, int32_t(heads), c.c.dim, int32_t(most));
    Tensor ws = empty({need}, at::kByte, c.dev);
    g.q = q.data_ptr(), g.out = out.data_ptr();
    g.table = static_cast<const int32_t*>(table.data_ptr());
    g.lens = static_cast<const int32_t*>(lens.data_ptr());
    g.workspace = ws.data_ptr();
    g.dev_status = status_of(a[15], c.dev);
    g.q_st = q.stride(0), g.q_sh = q.stride(1), g.o_st = out.stride(0), g.o_sh = out.stride(1);
    g.table_ld = table.size(1);
    g.workspace_bytes = need;
    g.seqs = int32_t(seqs), g.total_q = int32_t(total), g.max_queries = int32_t(most), g.q_heads = int32_t(heads);
    g.causal = causal;
    g.window = int32_t(window < 0x7FFFFFFF ? window : 0x7FFFFFFF);
    g.sinks = int32_t(sinks < 0x7FFFFFFF ? sinks : 0x7FFFFFFF);
    done(api.cache_attention(&c.c, &g, on_stream.handle()), "mxfp4_cache_attention");
  }
  return on_stream.result(out, a[13] != Py_None);
}

// Every function takes a fixed number of positional arguments, and no C++
// exception leaves it.
template <PyObject* (*kFn)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "%d arguments are needed", kArgs);
    return nullptr;
  }
  if (check_fn == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
    return nullptr;
  }
  try {
    return kFn(args);
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// bind(check, address of each C function in the order of Api)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kFns = sizeof(Api) / sizeof(void*);
  if (n != kFns + 1) {
    PyErr_SetString(PyExc_TypeError, "bind: wrong number of functions");
    return nullptr;
  }
  void* p[kFns];
  for (int i = 0; i < kFns; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null function");
      return nullptr;
    }
  }
  memcpy(&api, p, sizeof(api));
  Py_XDECREF(check_fn);
  check_fn = a[0];
  Py_INCREF(check_fn);
  Py_RETURN_NONE;
}

#define ENTRY(name, args) {#name, (PyCFunction)(void*)entry<name, args>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", (PyCFunction)(void*)bind, METH_FASTCALL, nullptr},
                         ENTRY(quantize, 4),
                         ENTRY(dequantize, 7),
                         ENTRY(gemm, 12),
                         ENTRY(linear, 9),
                         ENTRY(cache_write, 8),
                         ENTRY(cache_read, 9),
                         ENTRY(cache_attention, 17),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mxfp4", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mxfp4() { return PyModule_Create(&module); }
