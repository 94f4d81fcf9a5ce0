// Argument marshalling of moe_rms_norm, moe_kv_append and moe_paged_attention for torch tensors:
// the checks, the outputs and the argument structs of binding.py's entry points, compiled. A
// decode step calls these with a few microseconds of GPU work each, and the same checks through
// ctypes took 10 to 16 us a call. The library is reached through the addresses that bind() is
// given, so this module does not depend on where libgbmoe.so lies.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/gbmoe.h"

namespace {

decltype(&moe_rms_norm) rms_norm_fn;
decltype(&moe_kv_append) kv_append_fn;
decltype(&moe_paged_attention) attention_fn;
PyObject* error_type;  // GbmoeError(entry point, code)

// A new reference when the object dies; unlike a raw pointer it survives the exceptions below.
struct Ref {
  PyObject* p;
  explicit Ref(PyObject* x) : p(x) {}
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  ~Ref() { Py_XDECREF(p); }
  PyObject* take() {
    PyObject* x = p;
    p = nullptr;
    return x;
  }
};

const at::Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}
void* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw python_error();
  return p;
}

// The call's stream: the stream argument, a torch.cuda.Stream, or (None) the current one of t's
// device. New outputs are allocated with it as the current stream: the allocator orders a block's
// reuse by the stream it was allocated on, and on another one than the kernel's, work still queued
// there could meet the kernel's writes in the same memory.
// The kernels launch on the current device, so t's is made that one for the call.
struct CallStream {
  c10::cuda::CUDAGuard device;
  gbmoe_stream_t handle;
  c10::cuda::OptionalCUDAStreamGuard guard;
  CallStream(const at::Tensor& t, PyObject* stream) : device(t.device()) {
    const auto now = c10::cuda::getCurrentCUDAStream(t.get_device());
    handle = now.stream();
    if (stream == Py_None) return;
    const Ref number(PyObject_GetAttrString(stream, "cuda_stream"));
    if (!number.p) throw python_error();
    handle = static_cast<gbmoe_stream_t>(address(number.p));
    if (handle != now.stream())
      guard.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle),
                                                          t.device().index()));
  }
};

// A size as the C ABI's 32-bit number.
int32_t size32(const at::Tensor& t, int d, const char* name) {
  const int64_t n = t.size(d);
  TORCH_CHECK_VALUE(n <= INT32_MAX, name, " has ", n, " in dimension ", d, ", more than 32 bits hold");
  return (int32_t)n;
}

// A kernel reads all its tensors from one device, `like`'s.
void check_device(const at::Tensor& t, const char* name, const at::Tensor& like) {
  TORCH_CHECK_VALUE(t.device() == like.device(), name, " is on ", t.device(),
                    ", the call's other tensors are on ", like.device());
}

// Row stride of a bf16 [T, cols] or [T, heads, dim] tensor with contiguous rows, on like's CUDA
// device.
int64_t row_stride(const at::Tensor& t, const char* name, int64_t T, int64_t cols,
                   const at::Tensor& like) {
  const int64_t d = t.dim();
  TORCH_CHECK_VALUE((d == 2 || d == 3) && t.is_cuda() && t.scalar_type() == at::kBFloat16 &&
                        t.size(0) == T && t.numel() == T * cols && t.stride(d - 1) == 1 &&
                        (d == 2 || t.stride(1) == t.size(2)),
                    name, " must be a CUDA bfloat16 tensor of ", T, " rows of ", cols,
                    " contiguous columns");
  check_device(t, name, like);
  return T > 1 ? t.stride(0) : cols;
}

// An output: none until it is wanted; then the given tensor, checked, or (None) a new contiguous
// one, which make() allocates. As all addresses it is taken once every argument has been checked.
class Out {
 public:
  Out() : obj_(Py_NewRef(Py_None)) {}
  void want(PyObject* given, const char* name, const at::Tensor& like, at::IntArrayRef shape,
            at::ScalarType dtype) {
    if (given == Py_None) {
      shape_ = shape;
      dtype_ = dtype;
      fresh_ = true;
      return;
    }
    const at::Tensor& t = tensor(given, name);
    TORCH_CHECK_VALUE(t.is_cuda() && t.scalar_type() == dtype && t.is_contiguous() &&
                          t.sizes() == shape,
                      name, " must be a contiguous CUDA ", dtype, " tensor of shape ", shape);
    check_device(t, name, like);
    Py_INCREF(given);
    Py_SETREF(obj_.p, given);
  }
  void make(const at::Tensor& like) {
    if (!fresh_) {
      if (obj_.p != Py_None) ptr_ = THPVariable_Unpack(obj_.p).data_ptr();
      return;
    }
    at::Tensor t = at::empty(shape_, like.options().dtype(dtype_));
    ptr_ = t.data_ptr();
    PyObject* o = THPVariable_Wrap(std::move(t));
    if (!o) throw python_error();
    Py_SETREF(obj_.p, o);
  }
  template <class T = void>
  T* ptr() const {
    return static_cast<T*>(ptr_);
  }
  PyObject* obj() const { return obj_.p; }
  PyObject* take() { return obj_.take(); }

 private:
  Ref obj_;
  void* ptr_ = nullptr;
  bool fresh_ = false;
  at::DimVector shape_;
  at::ScalarType dtype_ = at::kFloat;
};

PyObject* failed(const char* fn, int code) {
  Ref e(PyObject_CallFunction(error_type, "si", fn, code));
  if (e.p) PyErr_SetObject(error_type, e.p);
  return nullptr;
}
bool arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments instead of %zd", n, want);
  return false;
}

// bind(address of moe_rms_norm, of moe_kv_append, of moe_paged_attention, GbmoeError)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 4)) return nullptr;
  rms_norm_fn = reinterpret_cast<decltype(rms_norm_fn)>(address(a[0]));
  kv_append_fn = reinterpret_cast<decltype(kv_append_fn)>(address(a[1]));
  attention_fn = reinterpret_cast<decltype(attention_fn)>(address(a[2]));
  Py_INCREF(a[3]);
  Py_XSETREF(error_type, a[3]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// rms_norm(x, weight, eps, residual, want bf16, want codes, y, residual_out, q, scale, stream)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 11)) return nullptr;
  const at::Tensor& x = tensor(a[0], "x");
  const at::Tensor& w = tensor(a[1], "weight");
  TORCH_CHECK_VALUE(x.dim() == 2, "x must have two dimensions");
  const int32_t T = size32(x, 0, "x"), H = size32(x, 1, "x");
  gbmoe_rms_norm_args_t g = {};
  g.x_stride = row_stride(x, "x", T, H, x);
  TORCH_CHECK_VALUE(w.is_cuda() && w.scalar_type() == at::kBFloat16 && w.dim() == 1 &&
                        w.size(0) == H && w.is_contiguous(),
                    "weight must be a contiguous CUDA bfloat16 tensor of H columns");
  check_device(w, "weight", x);
  g.eps = (float)PyFloat_AsDouble(a[2]);
  if (PyErr_Occurred()) return nullptr;
  Out y, ro, q, scale;
  if (a[3] != Py_None) {
    const at::Tensor& r = tensor(a[3], "residual");
    g.residual_stride = row_stride(r, "residual", T, H, x);
    ro.want(a[7], "residual_out", x, {T, H}, at::kBFloat16);
  }
  if (a[4] == Py_True) y.want(a[6], "y", x, {T, H}, at::kBFloat16);
  if (a[5] == Py_True) {
    q.want(a[8], "q", x, {T, H}, at::kFloat8_e4m3fn);
    scale.want(a[9], "scale", x, {H / 128, T}, at::kFloat);
  }
  const CallStream stream(x, a[10]);
  for (Out* o : {&y, &ro, &q, &scale}) o->make(x);
  g.x = x.data_ptr();
  if (a[3] != Py_None) g.residual = THPVariable_Unpack(a[3]).data_ptr();
  g.weight = w.data_ptr();
  g.y = y.ptr();
  g.residual_out = ro.ptr();
  g.q = q.ptr<uint8_t>();
  g.scale = scale.ptr<float>();
  const int code = rms_norm_fn(T, H, &g, stream.handle);
  if (code) return failed("moe_rms_norm", code);
  Ref r(PyTuple_New(4));
  if (!r.p) return nullptr;
  PyTuple_SET_ITEM(r.p, 0, y.take());
  PyTuple_SET_ITEM(r.p, 1, ro.take());
  PyTuple_SET_ITEM(r.p, 2, q.take());
  PyTuple_SET_ITEM(r.p, 3, scale.take());
  return r.take();
  END_HANDLE_TH_ERRORS
}

// Checks of (k_cache, v_cache, block_table, cu_seqlens_q, kv_lens), which lie on ws's device.
void check_paged(const gbmoe_attn_config_t& c, PyObject* const* a, const at::Tensor& ws) {
  const at::Tensor& k = tensor(a[0], "k_cache");
  const at::Tensor& v = tensor(a[1], "v_cache");
  const at::ScalarType t = k.scalar_type();
  TORCH_CHECK_VALUE(
      k.dim() == 4 && k.size(1) == c.page_size && k.size(2) == c.num_kv_heads &&
          k.size(3) == c.head_dim && v.sizes() == k.sizes() && v.strides() == k.strides() &&
          k.stride(3) == 1 && v.scalar_type() == t && k.is_cuda() && v.is_cuda() &&
          (c.cache_type == GBMOE_CACHE_BF16 ? t == at::kBFloat16
                                            : t == at::kFloat8_e4m3fn || t == at::kByte),
      "k_cache and v_cache must be CUDA tensors [num_pages, page_size, num_kv_heads, head_dim] of "
      "the configured type and equal strides, contiguous in head_dim");
  const at::Tensor& table = tensor(a[2], "block_table");
  const at::Tensor& cu = tensor(a[3], "cu_seqlens_q");
  const at::Tensor& lens = tensor(a[4], "kv_lens");
  TORCH_CHECK_VALUE(lens.dim() == 1 && table.dim() == 2 && cu.dim() == 1 &&
                        table.size(0) == lens.size(0) && cu.size(0) == lens.size(0) + 1,
                    "block_table must be [S, max_pages], cu_seqlens_q [S + 1], kv_lens [S]");
  for (const at::Tensor* x : {&table, &cu, &lens})
    TORCH_CHECK_VALUE(x->scalar_type() == at::kInt && x->is_cuda() && x->is_contiguous(),
                      "block_table, cu_seqlens_q and kv_lens must be contiguous CUDA int32 tensors");
  size32(k, 0, "k_cache");
  size32(lens, 0, "kv_lens");
  size32(table, 1, "block_table");
  check_device(k, "k_cache", ws);
  check_device(v, "v_cache", ws);
  check_device(table, "block_table", ws);
  check_device(cu, "cu_seqlens_q", ws);
  check_device(lens, "kv_lens", ws);
}

// The paged batch of the same, checked before.
gbmoe_paged_kv_t paged(PyObject* const* a) {
  const at::Tensor &k = THPVariable_Unpack(a[0]), &v = THPVariable_Unpack(a[1]),
                   &table = THPVariable_Unpack(a[2]), &cu = THPVariable_Unpack(a[3]),
                   &lens = THPVariable_Unpack(a[4]);
  // the stride of a dimension of one element is never used: any valid number
  auto stride = [&](int d) { return k.size(d) > 1 ? k.stride(d) : k.size(3); };
  gbmoe_paged_kv_t p = {};
  p.k_cache = k.data_ptr();
  p.v_cache = v.data_ptr();
  p.page_stride = stride(0);
  p.token_stride = stride(1);
  p.head_stride = stride(2);
  p.num_pages = (int32_t)k.size(0);
  p.num_seqs = (int32_t)lens.size(0);
  p.block_table_stride = (int32_t)table.size(1);
  p.block_table = table.data_ptr<int>();
  p.cu_seqlens_q = cu.data_ptr<int>();
  p.kv_lens = lens.data_ptr<int>();
  return p;
}

// kv_append(config address, workspace, q, k, v, k_cache, v_cache, block_table,
//           cu_seqlens_q, kv_lens, cos_sin, interleaved, q_out, stream)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 14)) return nullptr;
  const auto& c = *static_cast<const gbmoe_attn_config_t*>(address(a[0]));
  const at::Tensor& ws = tensor(a[1], "workspace");
  check_paged(c, a + 5, ws);
  const at::Tensor& q = tensor(a[2], "q");
  const at::Tensor& k = tensor(a[3], "k");
  const at::Tensor& v = tensor(a[4], "v");
  TORCH_CHECK_VALUE(q.dim() > 0, "q must have rows");
  const int32_t T = size32(q, 0, "q");
  const int64_t hq = c.num_q_heads, hkv = c.num_kv_heads, d = c.head_dim;
  gbmoe_kv_append_args_t g = {};
  g.q_stride = row_stride(q, "q", T, hq * d, ws);
  g.k_stride = row_stride(k, "k", T, hkv * d, ws);
  g.v_stride = row_stride(v, "v", T, hkv * d, ws);
  if (a[10] != Py_None) {
    const at::Tensor& cs = tensor(a[10], "cos_sin");
    TORCH_CHECK_VALUE(cs.is_cuda() && cs.scalar_type() == at::kFloat && cs.dim() == 2 &&
                          cs.is_contiguous(),
                      "cos_sin must be a contiguous CUDA float32 tensor [max_position, rotary_dim]");
    check_device(cs, "cos_sin", ws);
    g.max_position = size32(cs, 0, "cos_sin");
    g.rotary_dim = size32(cs, 1, "cos_sin");
  }
  g.interleaved = PyObject_IsTrue(a[11]);
  if (g.interleaved < 0) return nullptr;
  Out out;
  out.want(a[12], "q_out", q, {T, hq, d}, at::kBFloat16);
  const CallStream stream(q, a[13]);
  out.make(q);
  const gbmoe_paged_kv_t p = paged(a + 5);
  g.q = q.data_ptr();
  g.k = k.data_ptr();
  g.v = v.data_ptr();
  if (a[10] != Py_None) g.cos_sin = THPVariable_Unpack(a[10]).data_ptr<float>();
  g.q_out = out.ptr();
  g.workspace = ws.data_ptr();
  const int code = kv_append_fn(&c, T, &p, &g, stream.handle);
  return code ? failed("moe_kv_append", code) : out.take();
  END_HANDLE_TH_ERRORS
}

// attention(config address, workspace, q, k_cache, v_cache, block_table, cu_seqlens_q, kv_lens, out,
//           lse (None, True or a tensor), stream)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 11)) return nullptr;
  const auto& c = *static_cast<const gbmoe_attn_config_t*>(address(a[0]));
  const at::Tensor& ws = tensor(a[1], "workspace");
  check_paged(c, a + 3, ws);
  const at::Tensor& q = tensor(a[2], "q");
  TORCH_CHECK_VALUE(q.dim() > 0, "q must have rows");
  const int32_t T = size32(q, 0, "q");
  const int64_t hq = c.num_q_heads, d = c.head_dim;
  const int64_t stride = row_stride(q, "q", T, hq * d, ws);
  Out out, lse;
  out.want(a[8], "out", q, {T, hq, d}, at::kBFloat16);
  if (a[9] != Py_None)
    lse.want(a[9] == Py_True ? Py_None : a[9], "lse", q, {T, hq}, at::kFloat);
  const CallStream stream(q, a[10]);
  out.make(q);
  lse.make(q);
  const gbmoe_paged_kv_t p = paged(a + 3);
  const int code = attention_fn(&c, T, &p, q.data_ptr(), stride, out.ptr(),
                                lse.ptr<float>(), ws.data_ptr(), ws.nbytes(), stream.handle);
  if (code) return failed("moe_paged_attention", code);
  if (a[9] == Py_None) return out.take();
  return PyTuple_Pack(2, out.obj(), lse.obj());
  END_HANDLE_TH_ERRORS
}

#define GBMOE_METHOD(f) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GBMOE_METHOD(bind), GBMOE_METHOD(rms_norm), GBMOE_METHOD(kv_append),
                         GBMOE_METHOD(attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&module); }
