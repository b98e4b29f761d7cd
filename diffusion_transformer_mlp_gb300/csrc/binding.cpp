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
  decltype(&mxfp4_attention_shared_call_workspace_bytes) attention_shared_call_workspace_bytes;
  decltype(&mxfp4_cache_attention_shared) cache_attention_shared;
  decltype(&head_norm_rotary) norm_rotary;
  decltype(&mxfp4_cache_write_rotary) cache_write_rotary;
  decltype(&mxfp4_pages_workspace_bytes) pages_workspace_bytes;
  decltype(&mxfp4_pages_select) pages_select;
  decltype(&mxfp4_pages_extend) pages_extend;
  decltype(&mxfp4_pages_compact) pages_compact;
  decltype(&mxfp4_cache_copy) cache_copy;
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
// cache_attention_shared(the same, groups, shared, max_group | None, always) -> out
PyObject* attend(PyObject* const* a, bool with_groups) {
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
  mxfp4_shared s = {};
  if (with_groups) {
    const Tensor &groups = ints(a[17], at::kInt, 1, "groups", c.dev), &shared = ints(a[18], at::kInt, 1, "shared", c.dev);
    if (groups.size(0) != shared.size(0) + 1) bad("groups must have an entry for each group and one more");
    if (shared.size(0) > 0x7FFFFFFF) bad("too many groups");
    const int64_t most_group = a[19] == Py_None ? total : whole(a[19]);
    if (most_group < 0) bad("max_group must not be negative");
    if (total > 0 && shared.size(0) > 0 && most_group == 0) bad("q has rows, but max_group leaves no query");
    s.groups = static_cast<const int32_t*>(groups.data_ptr()), s.shared = static_cast<const int32_t*>(shared.data_ptr());
    s.always = PyObject_IsTrue(a[20]);
    if (s.always < 0) throw Raised();
    s.count = int32_t(shared.size(0)), s.max_group = int32_t(most_group < total ? most_group : total);
  }
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
    g.table_ld = table.size(1);
    g.seqs = int32_t(seqs), g.total_q = int32_t(total), g.max_queries = int32_t(most), g.q_heads = int32_t(heads);
    const int64_t need =
        with_groups ? api.attention_shared_call_workspace_bytes(&c.c, &g, &s)
                    : api.attention_workspace_bytes(c.c.kv_heads, int32_t(heads), c.c.dim, int32_t(most));
    Tensor ws = empty({need}, at::kByte, c.dev);
    g.q = q.data_ptr(), g.out = out.data_ptr();
    g.table = static_cast<const int32_t*>(table.data_ptr());
    g.lens = static_cast<const int32_t*>(lens.data_ptr());
    g.workspace = ws.data_ptr();
    g.dev_status = status_of(a[15], c.dev);
    g.q_st = q.stride(0), g.q_sh = q.stride(1), g.o_st = out.stride(0), g.o_sh = out.stride(1);
    g.workspace_bytes = need;
    g.causal = causal;
    g.window = int32_t(window < 0x7FFFFFFF ? window : 0x7FFFFFFF);
    g.sinks = int32_t(sinks < 0x7FFFFFFF ? sinks : 0x7FFFFFFF);
    if (with_groups)
      done(api.cache_attention_shared(&c.c, &g, &s, on_stream.handle()), "mxfp4_cache_attention_shared");
    else
      done(api.cache_attention(&c.c, &g, on_stream.handle()), "mxfp4_cache_attention");
  }
  return on_stream.result(out, a[13] != Py_None);
}
PyObject* cache_attention(PyObject* const* a) { return attend(a, false); }
PyObject* cache_attention_shared(PyObject* const* a) { return attend(a, true); }

struct Rotary {
  mxfp4_rotary r;
  int32_t weight_code;
  float eps;
};
// The rotation and the norm in args: turns, axis | None, interleaved, positions, q_weight | None, k_weight | None, eps.
Rotary rotary_of(PyObject* const* a, const Tensor& x, c10::DeviceIndex dev) {
  Rotary o = {};
  const Tensor& turns = ints(a[0], at::kLong, 1, "rotary.turns", dev);
  if (turns.size(0) > 0x7FFFFFFF) bad("rotary.turns is too large");
  o.r.turns = static_cast<const int64_t*>(turns.data_ptr());
  o.r.pairs = int32_t(turns.size(0));
  if (a[1] != Py_None) {
    const Tensor& axis = ints(a[1], at::kInt, 1, "rotary.axis", dev);
    if (axis.size(0) != turns.size(0)) bad("rotary.axis must have an entry for each of rotary.turns");
    o.r.axis = static_cast<const int32_t*>(axis.data_ptr());
  }
  o.r.interleaved = PyObject_IsTrue(a[2]);
  if (o.r.interleaved < 0) throw Raised();
  const Tensor& pos = tensor(a[3], "positions");
  if (pos.scalar_type() != at::kInt || !pos.is_contiguous() || pos.dim() < 1 || pos.dim() > 2 ||
      pos.size(0) != x.size(0) || (pos.dim() == 2 && (pos.size(1) < 1 || pos.size(1) > 65536)))
    bad("positions must be a contiguous int32 [tokens] or [tokens, axes] tensor");
  on(pos, dev);
  o.r.positions = static_cast<const int32_t*>(pos.data_ptr());
  o.r.axes = pos.dim() == 2 ? int32_t(pos.size(1)) : 1;
  o.weight_code = code_of(x.scalar_type(), "q");
  bool one = false;
  for (int i = 4; i < 6; ++i) {
    if (a[i] == Py_None) continue;
    const char* name = i == 4 ? "q_weight" : "k_weight";
    const Tensor& w = tensor(a[i], name);
    if (w.dim() != 1 || w.size(0) != x.size(2) || !w.is_contiguous())
      bad(std::string(name) + " must be a contiguous [" + std::to_string(x.size(2)) + "] tensor");
    if (w.scalar_type() != x.scalar_type() && w.scalar_type() != at::kFloat)
      bad(std::string(name) + " must be float32 or of the heads' type");
    const int32_t code = code_of(w.scalar_type(), name);
    if (one && code != o.weight_code) bad("q_weight and k_weight must have one type");
    one = true, o.weight_code = code;
    no_graph(w, name);
    on(w, dev);
  }
  const double eps = PyFloat_AsDouble(a[6]);
  if (eps == -1.0 && PyErr_Occurred()) throw Raised();
  o.eps = float(eps);
  return o;
}
// Heads [tokens, heads, dim] of one type; the sizes are checked against `like`.
mxfp4_heads heads_in(const Tensor& x, const Tensor& like, const char* name, c10::DeviceIndex dev) {
  if (x.dim() != 3 || x.size(0) != like.size(0) || x.size(2) != like.size(2) || x.scalar_type() != like.scalar_type())
    bad(std::string(name) + " must be [tokens, heads, dim], of one type and with the tokens and dim of q");
  if (x.stride(2) != 1 && x.size(2) > 1) bad(std::string(name) + " must have unit stride along its last dimension");
  if (x.size(1) > 65535) bad(std::string(name) + " has too many heads");
  no_graph(x, name);
  on(x, dev);
  mxfp4_heads h = {};
  h.x = x.data_ptr(), h.st = x.stride(0), h.sh = x.stride(1), h.heads = int32_t(x.size(1));
  return h;
}
const void* weight_at(PyObject* o) { return o == Py_None ? nullptr : THPVariable_Unpack(o).data_ptr(); }
// Where the heads go: the given tensor, checked, or a new one.
Tensor heads_out(PyObject* o, const Tensor& x, const char* name, c10::DeviceIndex dev, mxfp4_heads& h) {
  Tensor t;
  if (o == Py_None) {
    t = empty({x.size(0), x.size(1), x.size(2)}, x.scalar_type(), dev);
  } else {
    t = tensor(o, name);
    if (t.dim() != 3 || t.sizes() != x.sizes() || t.scalar_type() != x.scalar_type() || t.stride(2) != 1)
      bad(std::string(name) + " must have the heads' shape and type and unit stride along its last dimension");
    if ((t.size(0) > 1 && t.stride(0) == 0) || (t.size(1) > 1 && t.stride(1) == 0))
      bad(std::string(name) + " must not overlap itself");
    if (t.data_ptr() == x.data_ptr() && t.strides() != x.strides() && x.numel() > 0)
      bad(std::string(name) + " may be the heads themselves only with their strides");
    on(t, dev);
    no_graph(t, name);
  }
  h.out = t.data_ptr(), h.o_st = t.stride(0), h.o_sh = t.stride(1);
  return t;
}

// norm_rotary(q, k | None, turns, axis | None, interleaved, positions, q_weight | None, k_weight | None, eps,
//             q_out | None, k_out | None, stream) -> (q_out, k_out | None)
PyObject* norm_rotary(PyObject* const* a) {
  const Tensor& q = tensor(a[0], "q");
  const c10::DeviceIndex dev = cuda_index(q);
  const bool both = a[1] != Py_None;
  if (q.dim() != 3) bad("q must be [tokens, heads, dim]");
  const int32_t code = code_of(q.scalar_type(), "q");
  mxfp4_heads hq = heads_in(q, q, "q", dev), hk = {};
  if (both) hk = heads_in(tensor(a[1], "k"), q, "k", dev);
  else if (a[7] != Py_None || a[10] != Py_None) bad("k_weight and k_out are for a k");
  const Rotary r = rotary_of(a + 2, q, dev);
  hq.weight = weight_at(a[6]), hk.weight = weight_at(a[7]);
  if (q.size(2) > 256) bad("dim must be a multiple of 16 up to 256");
  const Launch on_stream(a[11], dev);
  Tensor tq = heads_out(a[9], q, "q_out", dev, hq), tk;
  if (both) tk = heads_out(a[10], THPVariable_Unpack(a[1]), "k_out", dev, hk);
  done(api.norm_rotary(&hq, both ? &hk : nullptr, &r.r, code, r.weight_code, q.size(0), int32_t(q.size(2)), r.eps,
                       on_stream.handle()),
       "head_norm_rotary");
  PyObject* ok = Py_None;
  if (both) ok = on_stream.result(tk, a[10] != Py_None);
  else Py_INCREF(ok);
  return Py_BuildValue("NN", on_stream.result(tq, a[9] != Py_None), ok);
}

// cache_write_rotary(cache x 4, q, k, v, slots, turns, axis | None, interleaved, positions, q_weight | None,
//                    k_weight | None, eps, q_out | None, stream) -> q_out
PyObject* cache_write_rotary(PyObject* const* a) {
  const Cache c = cache(a);
  const Tensor& q = tensor(a[4], "q");
  if (q.dim() != 3 || q.size(2) != c.c.dim) bad("q must be [tokens, heads, " + std::to_string(c.c.dim) + "]");
  const int32_t code = code_of(q.scalar_type(), "q", false);
  mxfp4_heads hq = heads_in(q, q, "q", c.dev), hk = heads_in(heads_of(a[5], c.c, "k", c.dev), q, "k", c.dev),
              hv = heads_in(heads_of(a[6], c.c, "v", c.dev), q, "v", c.dev);
  const Tensor& slots = ints(a[7], at::kLong, 1, "slots", c.dev);
  if (slots.size(0) != q.size(0)) bad("slots must have an entry for each token");
  const Rotary r = rotary_of(a + 8, q, c.dev);
  hq.weight = weight_at(a[12]), hk.weight = weight_at(a[13]);
  const Launch on_stream(a[16], c.dev);
  Tensor out = heads_out(a[15], q, "q_out", c.dev, hq);
  done(api.cache_write_rotary(&c.c, &hq, &hk, &hv, static_cast<const int64_t*>(slots.data_ptr()), &r.r, code,
                              r.weight_code, q.size(0), r.eps, on_stream.handle()),
       "mxfp4_cache_write_rotary");
  return on_stream.result(out, a[15] != Py_None);
}

struct Pages {
  mxfp4_pages p;
  c10::DeviceIndex dev;
};
// The pages in args[0..3]: refs, table, lens, page_size.
Pages pages_of(PyObject* const* a) {
  const c10::DeviceIndex dev = cuda_index(tensor(a[0], "pages.refs"));
  const Tensor &refs = ints(a[0], at::kInt, 1, "pages.refs", dev), &table = ints(a[1], at::kInt, 2, "pages.table", dev),
               &lens = ints(a[2], at::kInt, 1, "pages.lens", dev);
  if (table.size(0) != lens.size(0)) bad("pages.table must have a row for each of pages.lens");
  if (refs.numel() == 0 || table.numel() == 0) bad("there must be pages, rows and room in the rows");
  if (lens.size(0) > 0x7FFFFFFF) bad("pages.table has too many rows");
  const int64_t size = whole(a[3]);
  if (size < 1 || size > 0x7FFFFFFF) bad("page_size must be 16, 32, 64, 128 or 256");
  return {{static_cast<int32_t*>(refs.data_ptr()), static_cast<int32_t*>(table.data_ptr()),
           static_cast<int32_t*>(lens.data_ptr()), refs.size(0), table.size(1), int32_t(lens.size(0)), int32_t(size)},
          dev};
}

// pages_select(pages x 4, sources, stream)
PyObject* pages_select(PyObject* const* a) {
  const Pages g = pages_of(a);
  const Tensor& sources = ints(a[4], at::kInt, 1, "sources", g.dev);
  if (sources.size(0) != g.p.rows) bad("sources must have an entry for each row");
  const Launch on_stream(a[5], g.dev);
  const int64_t need = api.pages_workspace_bytes(&g.p);
  Tensor ws = empty({need}, at::kByte, g.dev);
  done(api.pages_select(&g.p, static_cast<const int32_t*>(sources.data_ptr()), ws.data_ptr(), need, on_stream.handle()),
       "mxfp4_pages_select");
  Py_RETURN_NONE;
}

// pages_extend(pages x 4, counts, total, stream) -> (slots, copies, missing)
PyObject* pages_extend(PyObject* const* a) {
  const Pages g = pages_of(a);
  const Tensor& counts = ints(a[4], at::kInt, 1, "counts", g.dev);
  if (counts.size(0) != g.p.rows) bad("counts must have an entry for each row");
  const int64_t total = whole(a[5]);
  if (total < 0 || total > 0x7FFFFFFF) bad("total must be from 0 to 2^31 - 1");
  const Launch on_stream(a[6], g.dev);
  const int64_t need = api.pages_workspace_bytes(&g.p);
  Tensor ws = empty({need}, at::kByte, g.dev), slots = empty({total}, at::kLong, g.dev),
         copies = empty({int64_t(g.p.rows), 2}, at::kInt, g.dev), missing = empty({1}, at::kInt, g.dev);
  done(api.pages_extend(&g.p, static_cast<const int32_t*>(counts.data_ptr()), total,
                        static_cast<int64_t*>(slots.data_ptr()), static_cast<int32_t*>(copies.data_ptr()),
                        static_cast<int32_t*>(missing.data_ptr()), ws.data_ptr(), need, on_stream.handle()),
       "mxfp4_pages_extend");
  return Py_BuildValue("NNN", on_stream.result(slots), on_stream.result(copies), on_stream.result(missing));
}

// pages_compact(pages x 4, stream) -> (moves, used)
PyObject* pages_compact(PyObject* const* a) {
  const Pages g = pages_of(a);
  const Launch on_stream(a[4], g.dev);
  const int64_t need = api.pages_workspace_bytes(&g.p);
  Tensor ws = empty({need}, at::kByte, g.dev), moves = empty({g.p.pages / 2, 2}, at::kInt, g.dev),
         used = empty({1}, at::kInt, g.dev);
  done(api.pages_compact(&g.p, static_cast<int32_t*>(moves.data_ptr()), static_cast<int32_t*>(used.data_ptr()),
                         ws.data_ptr(), need, on_stream.handle()),
       "mxfp4_pages_compact");
  return Py_BuildValue("NN", on_stream.result(moves), on_stream.result(used));
}

// cache_copy(cache x 4, source x 4, pairs, stream)
PyObject* cache_copy(PyObject* const* a) {
  const Cache c = cache(a), s = cache(a + 4);
  if (c.dev != s.dev) bad(kOneDevice);
  const Tensor& pairs = ints(a[8], at::kInt, 2, "pairs", c.dev);
  if (pairs.size(1) != 2) bad("pairs must be [n, 2]");
  const Launch on_stream(a[9], c.dev);
  done(api.cache_copy(&c.c, &s.c, static_cast<const int32_t*>(pairs.data_ptr()), pairs.size(0), on_stream.handle()),
       "mxfp4_cache_copy");
  Py_RETURN_NONE;
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
                         ENTRY(cache_attention_shared, 21),
                         ENTRY(norm_rotary, 12),
                         ENTRY(cache_write_rotary, 17),
                         ENTRY(pages_select, 6),
                         ENTRY(pages_extend, 7),
                         ENTRY(pages_compact, 5),
                         ENTRY(cache_copy, 10),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mxfp4", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mxfp4() { return PyModule_Create(&module); }
