// binding.cpp -- the torch-facing calls whose kernels take a few microseconds (single-token
// products, page plans, the 8-bit cache): argument checks, result tensors, the stream and the
// workspace in C++, then the entry point of the C ABI.  The same call through ctypes costs
// 10 to 25 us of Python, several times the kernel.
//
// No step of any operation is computed here.  ops.py documents the functions; they raise
// ValueError and TypeError for tensors that do not fit, and NVFP4Error for what the library
// refuses.
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <map>
#include <string>
#include <utility>

#include "../../include/nvfp4.h"

namespace {

struct Library {
  decltype(&nvfp4_codes_bytes) codes_bytes;
  decltype(&nvfp4_sf_bytes) sf_bytes;
  decltype(&nvfp4_gemv) gemv;
  decltype(&nvfp4_plan_pages) plan_pages;
  decltype(&nvfp4_kv8_append) append;
  decltype(&nvfp4_kv8_attention_scratch_bytes) scratch_bytes;
  decltype(&nvfp4_kv8_attention) attention;
} lib = {};
PyObject* error_class = nullptr;       // NVFP4Error
PyObject* workspace_fn = nullptr;      // ops.workspace

struct Refused {};                     // a Python error is set

[[noreturn]] void refuse(PyObject* kind, const std::string& what) {
  PyErr_SetString(kind, what.c_str());
  throw Refused();
}

void initialised() {
  if (!error_class) refuse(PyExc_RuntimeError, "init has not been called");
}

void check(nvfp4_status st, const char* what) {
  if (st == NVFP4_OK) return;
  PyObject* e = PyObject_CallFunction(error_class, "is", int(st), what);
  if (e) {
    PyErr_SetObject(error_class, e);
    Py_DECREF(e);
  }
  throw Refused();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

int32_t int32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX)
    refuse(PyExc_ValueError, std::string(name) + " does not fit 32 bits");
  return int32_t(v);
}

// The device of a call: the current stream, and the device made current where it is not.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;
  On(const at::Tensor& t, const char* what) {
    initialised();
    if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(what) + " takes CUDA tensors");
    if (t.get_device() != c10::cuda::current_device()) guard.set_index(t.get_device());
    stream = c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
  }
};

// ws, or (None) the stream's own workspace, which ops.workspace keeps.
at::Tensor workspace(PyObject* ws, const at::Tensor& like, const On& on) {
  if (ws != Py_None) {
    const at::Tensor& t = tensor(ws, "ws");
    if (t.device() != like.device() || t.scalar_type() != at::kByte || !t.is_contiguous())
      refuse(PyExc_ValueError, "ws must be a contiguous uint8 tensor on the tensors' device");
    return t;
  }
  if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) {
    // a workspace apart from the stream's own
    PyObject* t = PyObject_CallFunction(workspace_fn, "s", like.device().str().c_str());
    if (!t) throw Refused();
    const at::Tensor ws = THPVariable_Unpack(t);
    Py_DECREF(t);
    return ws;
  }
  // as long-lived as the streams: never freed, or it would be after the CUDA context
  static auto& known = *new std::map<std::pair<int, void*>, at::Tensor>;
  const std::pair<int, void*> key(like.get_device(), on.stream);
  auto it = known.find(key);
  if (it == known.end()) {
    PyObject* t = PyObject_CallFunction(workspace_fn, "s", like.device().str().c_str());
    if (!t) throw Refused();
    it = known.emplace(key, THPVariable_Unpack(t)).first;
    Py_DECREF(t);
  }
  return it->second;
}

int32_t dtype_code(at::ScalarType t) {
  if (t == at::kBFloat16) return NVFP4_BF16;
  if (t == at::kFloat) return NVFP4_FP32;
  refuse(PyExc_TypeError, std::string("unsupported dtype ") + toString(t));
}

// torch gives any stride for a dimension of one
int64_t row_stride(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

void int32_tensor(const at::Tensor& t, const at::Device& dev, const char* name, int dims = 1) {
  if (t.scalar_type() != at::kInt || t.device() != dev || t.dim() != dims)
    refuse(PyExc_ValueError, std::string(name) + " must be an int32 tensor of " +
                                 std::to_string(dims) + " dimension(s) on " + dev.str());
  if (dims == 1 ? !t.is_contiguous() : t.size(1) > 1 && t.stride(1) != 1)
    refuse(PyExc_ValueError, std::string(name) + (dims == 1 ? " must be contiguous"
                                                             : " must have unit column stride"));
}

// Allocations and launches may wait for the GPU, and the GPU for another Python thread.
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

// A refusal or a torch error becomes the Python error.
#define NVFP4_CALL(...)           \
  HANDLE_TH_ERRORS try __VA_ARGS__ \
  catch (const Refused&) {        \
    return nullptr;               \
  }                               \
  END_HANDLE_TH_ERRORS

void count(Py_ssize_t have, Py_ssize_t want) {
  if (have != want) refuse(PyExc_TypeError, "wrong number of arguments");
}

// The buffers of an NVFP4 tensor of rows x cols, whose attributes are public.
nvfp4_tensor weights(const at::Tensor& codes, const at::Tensor& sf, const at::Tensor& s_t,
                     int64_t rows, int64_t cols, int32_t sf_layout) {
  initialised();
  if (rows < 0 || cols < 0 || rows > INT32_MAX || cols > INT32_MAX)
    refuse(PyExc_ValueError, "rows and cols of the weights must fit 31 bits");
  for (const at::Tensor* t : {&codes, &sf})
    if (t->scalar_type() != at::kByte || !t->is_contiguous())
      refuse(PyExc_ValueError, "codes and sf of the weights must be contiguous uint8 tensors");
  if (size_t(codes.numel()) < lib.codes_bytes(rows, cols) ||
      size_t(sf.numel()) < lib.sf_bytes(rows, cols, sf_layout))
    refuse(PyExc_ValueError, "codes or sf of the weights are too short for their rows and cols");
  if (s_t.scalar_type() != at::kFloat || s_t.numel() != 1)
    refuse(PyExc_ValueError, "s_t of the weights must be one fp32 element");
  return {static_cast<uint8_t*>(codes.data_ptr()), static_cast<uint8_t*>(sf.data_ptr()),
          static_cast<float*>(s_t.data_ptr()), rows, cols, sf_layout};
}

// ------------------------------------------------------------------ gemv
// (x, codes, sf, s_t, rows, cols, sf_layout, out_dtype, out, act)
PyObject* gemv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NVFP4_CALL({
    count(n, 10);
    const at::Tensor& x = tensor(a[0], "x");
    const at::Tensor &codes = tensor(a[1], "codes"), &sf = tensor(a[2], "sf"),
                     &s_t = tensor(a[3], "s_t");
    const int64_t rows = integer(a[4]), cols = integer(a[5]);
    if (x.dim() != 2 || x.stride(1) != 1 || x.size(1) != cols)
      refuse(PyExc_ValueError,
             "gemv expects a 2-D tensor of " + std::to_string(cols) + " unit-stride columns");
    if (x.device() != codes.device() || sf.device() != codes.device() ||
        s_t.device() != codes.device())
      refuse(PyExc_ValueError, "x and w must be on one device");
    const nvfp4_tensor w = weights(codes, sf, s_t, rows, cols, int32(a[6], "sf_layout"));
    const int32_t x_code = dtype_code(x.scalar_type());
    at::Tensor out;
    if (a[8] != Py_None) {
      out = tensor(a[8], "out");
      if (out.dim() != 2 || out.size(0) != x.size(0) || out.size(1) < rows || out.stride(1) != 1 ||
          out.device() != x.device())
        refuse(PyExc_ValueError, "out must have " + std::to_string(x.size(0)) +
                                     " rows of at least " + std::to_string(rows) +
                                     " unit-stride columns on x's device");
      dtype_code(out.scalar_type());
    }
    const On on(x, "gemv");
    at::ScalarType type = at::kFloat;
    if (out.defined())
      type = out.scalar_type();
    else if (THPDtype_Check(a[7]))
      type = reinterpret_cast<THPDtype*>(a[7])->scalar_type;
    else
      refuse(PyExc_TypeError, "out_dtype must be a torch.dtype");
    const int32_t y_code = dtype_code(type), act = int32(a[9], "act");
    nvfp4_status st;
    {
      const NoGil no_gil;
      if (!out.defined()) out = at::empty({x.size(0), rows}, x.options().dtype(type));
      st = lib.gemv(x.data_ptr(), x_code, x.size(0), row_stride(x), &w, out.data_ptr(), y_code,
                    row_stride(out), act, on.stream);
    }
    check(st, "nvfp4_gemv");
    return THPVariable_Wrap(out);
  })
}

// ------------------------------------------------------------------ plan_pages
// (cached_lens, new_lens, block_table, free_pages, free_head, page_tokens, n_pages, max_new, ws)
// -> (seq_lens, cu_new, slot_map, free_head)
PyObject* plan_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NVFP4_CALL({
    count(n, 9);
    const at::Tensor &cached = tensor(a[0], "cached_lens"), &fresh = tensor(a[1], "new_lens"),
                     &table = tensor(a[2], "block_table"), &free_pages = tensor(a[3], "free_pages"),
                     &head = tensor(a[4], "free_head");
    const at::Device dev = table.device();
    int32_tensor(cached, dev, "cached_lens");
    int32_tensor(fresh, dev, "new_lens");
    int32_tensor(table, dev, "block_table", 2);
    int32_tensor(free_pages, dev, "free_pages");
    int32_tensor(head, dev, "free_head");
    const int64_t batch = table.size(0), pages = table.size(1);
    if (cached.size(0) != batch || fresh.size(0) != batch || head.size(0) != 1)
      refuse(PyExc_ValueError,
             "plan_pages: cached_lens and new_lens must be [batch], block_table [batch, "
             "max_pages], free_head [1]");
    const int32_t max_new = int32(a[7], "max_new");
    if (max_new < 0) refuse(PyExc_ValueError, "max_new must not be negative");
    if (batch > INT32_MAX || pages > INT32_MAX || free_pages.size(0) > INT32_MAX)
      refuse(PyExc_ValueError, "plan_pages: more than 2^31 entries");
    const On on(table, "plan_pages");
    const at::Tensor ws = workspace(a[8], table, on);
    // the results are parts of one allocation, each on a 16-byte boundary (an allocation costs
    // as much as half a launch)
    const int64_t at_cu = (batch + 3) / 4 * 4, at_slots = at_cu + (batch + 4) / 4 * 4,
                  at_head = at_slots + (int64_t(max_new) + 3) / 4 * 4;
    const int32_t page_tokens = int32(a[5], "page_tokens"), n_pages = int32(a[6], "n_pages");
    at::Tensor mem;
    {
      const NoGil no_gil;
      mem = at::empty({at_head + 1}, table.options());
    }
    auto part = [&mem](int64_t from, int64_t n) {
      at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(mem.storage()),
                                                              mem.key_set(), mem.dtype());
      t.unsafeGetTensorImpl()->set_storage_offset(from);
      t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
      return t;
    };
    const at::Tensor seq = part(0, batch), cu = part(at_cu, batch + 1),
                     slots = part(at_slots, max_new), head_out = part(at_head, 1);
    auto p = [](const at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); };
    nvfp4_status st;
    {
      const NoGil no_gil;
      st = lib.plan_pages(p(cached), p(fresh), int32_t(batch), p(table), row_stride(table),
                          int32_t(pages), p(free_pages), int32_t(free_pages.size(0)), p(head),
                          page_tokens, n_pages, p(seq), p(cu), p(slots), max_new, p(head_out),
                          ws.data_ptr(), size_t(ws.numel()), on.stream);
    }
    check(st, "nvfp4_plan_pages");
    PyObject* r = PyTuple_New(4);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(seq));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(cu));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(slots));
    PyTuple_SET_ITEM(r, 3, THPVariable_Wrap(head_out));
    return r;
  })
}

// (bytes, device index) -> a uint8 tensor of zeros that belongs to no graph, also while the current
// stream is being captured: allocated and filled on a stream that is not, and waited for.
PyObject* zeros_outside_capture(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NVFP4_CALL({
    count(n, 2);
    const int64_t bytes = integer(a[0]), index = integer(a[1]);
    at::Tensor t;
    {
      const NoGil no_gil;
      const auto device = static_cast<c10::DeviceIndex>(index);
      const c10::cuda::CUDAStreamCaptureModeGuard relaxed(cudaStreamCaptureModeRelaxed);
      for (int i = 0; i < 64 && !t.defined(); ++i) {   // more than the pool has
        const c10::cuda::CUDAStream side = c10::cuda::getStreamFromPool(false, device);
        const c10::cuda::CUDAStreamGuard guard(side);
        if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None)
          continue;
        t = at::zeros({bytes}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, device));
        side.synchronize();
      }
    }
    if (!t.defined()) refuse(PyExc_RuntimeError, "every stream is being captured");
    return THPVariable_Wrap(t);
  })
}

// ------------------------------------------------------------------ the 8-bit cache
struct Cache {
  nvfp4_kv8_cache c;
  at::Device dev;
};

// (k_codes, v_codes, k_scale, v_scale), checked every time: the attributes are public.
Cache cache_of(PyObject* const* a) {
  const at::Tensor &k = tensor(a[0], "k_codes"), &v = tensor(a[1], "v_codes"),
                   &ks = tensor(a[2], "k_scale"), &vs = tensor(a[3], "v_scale");
  if (k.dim() != 4 || v.sizes() != k.sizes())
    refuse(PyExc_ValueError, "codes must be [n_pages, kv_heads, page_tokens, head_dim]");
  for (const at::Tensor* t : {&k, &v})
    if (t->scalar_type() != at::kFloat8_e4m3fn || !t->is_contiguous() || t->device() != k.device())
      refuse(PyExc_ValueError, "codes must be contiguous float8_e4m3fn tensors on one device");
  for (const at::Tensor* t : {&ks, &vs})
    if (t->scalar_type() != at::kFloat || t->dim() != 2 || t->size(0) != k.size(0) ||
        t->size(1) != k.size(1) || !t->is_contiguous() || t->device() != k.device())
      refuse(PyExc_ValueError, "scales must be contiguous fp32 tensors [n_pages, kv_heads]");
  for (int d = 0; d < 4; ++d)
    if (k.size(d) > INT32_MAX) refuse(PyExc_ValueError, "cache dimensions must fit 32 bits");
  return {{static_cast<uint8_t*>(k.data_ptr()), static_cast<uint8_t*>(v.data_ptr()),
           static_cast<float*>(ks.data_ptr()), static_cast<float*>(vs.data_ptr()),
           int32_t(k.size(0)), int32_t(k.size(2)), int32_t(k.size(1)), int32_t(k.size(3))},
          k.device()};
}

// The token stride of a bf16 tensor [tokens, heads, head_dim] or [tokens, heads * head_dim]
// whose tokens are contiguous.
int64_t token_stride(const Cache& c, const at::Tensor& t, int64_t heads, const char* name) {
  const int64_t d = c.c.head_dim;
  const bool ok = t.dim() == 3 ? t.size(1) == heads && t.size(2) == d && t.stride(2) == 1 &&
                                     (heads == 1 || t.stride(1) == d)
                               : t.dim() == 2 && t.size(1) == heads * d && t.stride(1) == 1;
  if (!ok || t.scalar_type() != at::kBFloat16 || t.device() != c.dev)
    refuse(PyExc_ValueError, std::string(name) + " must be a bf16 tensor [tokens, " +
                                 std::to_string(heads) + ", " + std::to_string(d) + "] on " +
                                 c.dev.str() + ", contiguous inside a token");
  return t.size(0) > 1 ? t.stride(0) : heads * d;
}

// (k_codes, v_codes, k_scale, v_scale) -> the codes' shape
PyObject* kv8_shape(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NVFP4_CALL({
    count(n, 4);
    const Cache c = cache_of(a);
    return Py_BuildValue("iiii", c.c.n_pages, c.c.kv_heads, c.c.page_tokens, c.c.head_dim);
  })
}

// (k_codes, v_codes, k_scale, v_scale, k, v, slot_map, ws)
PyObject* kv8_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NVFP4_CALL({
    count(n, 8);
    const Cache c = cache_of(a);
    const at::Tensor &k = tensor(a[4], "k"), &v = tensor(a[5], "v"),
                     &slots = tensor(a[6], "slot_map");
    const int64_t stride = token_stride(c, k, c.c.kv_heads, "k");
    const int64_t tokens = k.size(0);
    if (token_stride(c, v, c.c.kv_heads, "v") != stride || v.size(0) != tokens)
      refuse(PyExc_ValueError, "k and v must share their tokens and a token stride");
    int32_tensor(slots, c.dev, "slot_map");
    if (slots.size(0) < tokens)
      refuse(PyExc_ValueError,
             "slot_map must have at least " + std::to_string(tokens) + " entries");
    const On on(k, "append");
    const at::Tensor ws = workspace(a[7], k, on);
    nvfp4_status st;
    {
      const NoGil no_gil;
      st = lib.append(&c.c, k.data_ptr(), v.data_ptr(), stride, tokens,
                      static_cast<const int32_t*>(slots.data_ptr()), ws.data_ptr(),
                      size_t(ws.numel()), on.stream);
    }
    check(st, "nvfp4_kv8_append");
    Py_RETURN_NONE;
  })
}

// (k_codes, v_codes, k_scale, v_scale, q, cu_q, seq_lens, block_table, max_q, max_kv, causal,
//  scale, out, return_lse, ws) -> out or (out, lse); None for the defaults of max_q, max_kv,
// scale, out and ws
PyObject* kv8_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NVFP4_CALL({
    count(n, 15);
    const Cache c = cache_of(a);
    const at::Tensor &q = tensor(a[4], "q"), &cu = tensor(a[5], "cu_q"),
                     &lens = tensor(a[6], "seq_lens"), &table = tensor(a[7], "block_table");
    const int64_t d = c.c.head_dim;
    if (q.dim() != 3 || q.size(2) != d)
      refuse(PyExc_ValueError, "q must be [tokens, q_heads, " + std::to_string(d) + "]");
    const int64_t tokens = q.size(0), heads = q.size(1);
    const int64_t stride = token_stride(c, q, heads, "q");
    int32_tensor(cu, c.dev, "cu_q");
    int32_tensor(lens, c.dev, "seq_lens");
    int32_tensor(table, c.dev, "block_table", 2);
    const int64_t batch = table.size(0), pages = table.size(1);
    if (cu.size(0) != batch + 1 || lens.size(0) != batch)
      refuse(PyExc_ValueError,
             "attention: cu_q must be [batch + 1], seq_lens [batch] and block_table [batch, "
             "pages]");
    if (batch > INT32_MAX || pages > INT32_MAX || heads > INT32_MAX || tokens > INT32_MAX)
      refuse(PyExc_ValueError, "attention: dimensions must fit 32 bits");
    at::Tensor out, lse, scratch;
    int64_t out_stride = heads * d;
    if (a[12] != Py_None) {
      out = tensor(a[12], "out");
      if (out.sizes() != q.sizes()) refuse(PyExc_ValueError, "out must have q's shape");
      out_stride = token_stride(c, out, heads, "out");
    }
    auto bound = [](PyObject* o, int64_t most, const char* name) {
      return o == Py_None ? int32_t(std::clamp<int64_t>(most, 1, INT32_MAX)) : int32(o, name);
    };
    const nvfp4_kv8_batch b = {static_cast<const int32_t*>(cu.data_ptr()),
                               static_cast<const int32_t*>(lens.data_ptr()),
                               static_cast<const int32_t*>(table.data_ptr()),
                               row_stride(table),
                               int32_t(batch),
                               int32_t(pages),
                               bound(a[8], tokens, "max_q"),
                               bound(a[9], pages * c.c.page_tokens, "max_kv")};
    const int causal = PyObject_IsTrue(a[10]);
    if (causal < 0) throw Refused();
    float scale = float(1.0 / std::sqrt(double(d)));
    if (a[11] != Py_None) {
      scale = float(PyFloat_AsDouble(a[11]));
      if (PyErr_Occurred()) throw Refused();
    }
    const On on(q, "attention");
    const int want_lse = PyObject_IsTrue(a[13]);
    if (want_lse < 0) throw Refused();
    const at::Tensor ws = workspace(a[14], q, on);
    nvfp4_status st = NVFP4_OK;
    {
      const NoGil no_gil;
      if (!out.defined()) out = at::empty({tokens, heads, d}, q.options());
      if (want_lse) lse = at::empty({tokens, heads}, q.options().dtype(at::kFloat));
      if (batch > 0) {   // (no requests, as a plan may have them: no rows to write)
        const size_t need = lib.scratch_bytes(&c.c, &b, tokens, int32_t(heads), causal);
        // a tensor of the call's own: calls on other streams and captured graphs share nothing
        if (need) scratch = at::empty({int64_t(need)}, q.options().dtype(at::kByte));
        st = lib.attention(&c.c, &b, q.data_ptr(), stride, tokens, int32_t(heads), causal, scale,
                           out.data_ptr(), out_stride,
                           want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr,
                           need ? scratch.data_ptr() : nullptr, need, ws.data_ptr(),
                           size_t(ws.numel()), on.stream);
      }
    }
    check(st, "nvfp4_kv8_attention");
    if (!want_lse) return THPVariable_Wrap(out);
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(out));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(lse));
    return r;
  })
}

// (path of libnvfp4.so, NVFP4Error, ops.workspace)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NVFP4_CALL({
    count(n, 3);
    const char* path = PyUnicode_AsUTF8(a[0]);
    if (!path) return nullptr;
    void* h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!h) refuse(PyExc_ImportError, dlerror());
    auto get = [h](auto& f, const char* name) {
      f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(dlsym(h, name));
      if (!f) refuse(PyExc_ImportError, std::string("libnvfp4.so has no ") + name);
    };
    get(lib.codes_bytes, "nvfp4_codes_bytes");
    get(lib.sf_bytes, "nvfp4_sf_bytes");
    get(lib.gemv, "nvfp4_gemv");
    get(lib.plan_pages, "nvfp4_plan_pages");
    get(lib.append, "nvfp4_kv8_append");
    get(lib.scratch_bytes, "nvfp4_kv8_attention_scratch_bytes");
    get(lib.attention, "nvfp4_kv8_attention");
    Py_INCREF(a[1]);
    Py_INCREF(a[2]);
    error_class = a[1];
    workspace_fn = a[2];
    Py_RETURN_NONE;
  })
}

template <PyObject* (*kF)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kF)), METH_FASTCALL,
          nullptr};
}

PyMethodDef methods[] = {method<init>("init"),
                         method<gemv>("gemv"),
                         method<plan_pages>("plan_pages"),
                         method<zeros_outside_capture>("zeros_outside_capture"),
                         method<kv8_shape>("kv8_shape"),
                         method<kv8_append>("kv8_append"),
                         method<kv8_attention>("kv8_attention"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", NVFP4_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
