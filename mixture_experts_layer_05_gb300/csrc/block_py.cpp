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
struct CallStream {
  gbmoe_stream_t handle;
  c10::cuda::OptionalCUDAStreamGuard guard;
  CallStream(const at::Tensor& t, PyObject* stream) {
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

// Row stride of a CUDA bf16 [T, cols] or [T, heads, dim] tensor with contiguous rows.
int64_t row_stride(const at::Tensor& t, const char* name, int64_t T, int64_t cols) {
  const int64_t d = t.dim();
  TORCH_CHECK_VALUE((d == 2 || d == 3) && t.is_cuda() && t.scalar_type() == at::kBFloat16 &&
                        t.size(0) == T && t.numel() == T * cols && t.stride(d - 1) == 1 &&
                        (d == 2 || t.stride(1) == t.size(2)),
                    name, " must be a CUDA bfloat16 tensor of ", T, " rows of ", cols,
                    " contiguous columns");
  return T > 1 ? t.stride(0) : cols;
}

// The given output, checked, or a new contiguous tensor; a new reference.
struct Out {
  Ref obj;
  void* ptr;
  static PyObject* get(PyObject* given, const char* name, const at::Tensor& like,
                       at::IntArrayRef shape, at::ScalarType dtype, void** ptr) {
    if (given == Py_None) {
      at::Tensor t = at::empty(shape, like.options().dtype(dtype));
      *ptr = t.data_ptr();
      return THPVariable_Wrap(std::move(t));
    }
    const at::Tensor& t = tensor(given, name);
    TORCH_CHECK_VALUE(t.is_cuda() && t.scalar_type() == dtype && t.is_contiguous() &&
                          t.sizes() == shape,
                      name, " must be a contiguous CUDA ", dtype, " tensor of shape ", shape);
    *ptr = t.data_ptr();
    Py_INCREF(given);
    return given;
  }
  Out() : obj(Py_NewRef(Py_None)), ptr(nullptr) {}
  Out(PyObject* given, const char* name, const at::Tensor& like, at::IntArrayRef shape,
      at::ScalarType dtype)
      : obj(nullptr), ptr(nullptr) {
    obj.p = get(given, name, like, shape, dtype, &ptr);
    if (!obj.p) throw python_error();
  }
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
  const int64_t T = x.size(0), H = x.size(1);
  gbmoe_rms_norm_args_t g = {};
  g.x = x.data_ptr();
  g.x_stride = row_stride(x, "x", T, H);
  TORCH_CHECK_VALUE(w.is_cuda() && w.scalar_type() == at::kBFloat16 && w.dim() == 1 &&
                        w.size(0) == H && w.is_contiguous(),
                    "weight must be a contiguous CUDA bfloat16 tensor of H columns");
  g.weight = w.data_ptr();
  g.eps = (float)PyFloat_AsDouble(a[2]);
  if (PyErr_Occurred()) return nullptr;
  const CallStream stream(x, a[10]);
  Out y, ro, q, scale;
  if (a[3] != Py_None) {
    const at::Tensor& r = tensor(a[3], "residual");
    g.residual_stride = row_stride(r, "residual", T, H);
    g.residual = r.data_ptr();
    Py_SETREF(ro.obj.p, Out::get(a[7], "residual_out", x, {T, H}, at::kBFloat16, &ro.ptr));
    if (!ro.obj.p) return nullptr;
  }
  if (a[4] == Py_True) {
    Py_SETREF(y.obj.p, Out::get(a[6], "y", x, {T, H}, at::kBFloat16, &y.ptr));
    if (!y.obj.p) return nullptr;
  }
  if (a[5] == Py_True) {
    Py_SETREF(q.obj.p, Out::get(a[8], "q", x, {T, H}, at::kFloat8_e4m3fn, &q.ptr));
    if (!q.obj.p) return nullptr;
    Py_SETREF(scale.obj.p, Out::get(a[9], "scale", x, {H / 128, T}, at::kFloat, &scale.ptr));
    if (!scale.obj.p) return nullptr;
  }
  g.y = y.ptr;
  g.residual_out = ro.ptr;
  g.q = static_cast<decltype(g.q)>(q.ptr);
  g.scale = static_cast<float*>(scale.ptr);
  const int code = rms_norm_fn((int32_t)T, (int32_t)H, &g, stream.handle);
  if (code) return failed("moe_rms_norm", code);
  Ref r(PyTuple_New(4));
  if (!r.p) return nullptr;
  PyTuple_SET_ITEM(r.p, 0, y.obj.take());
  PyTuple_SET_ITEM(r.p, 1, ro.obj.take());
  PyTuple_SET_ITEM(r.p, 2, q.obj.take());
  PyTuple_SET_ITEM(r.p, 3, scale.obj.take());
  return r.take();
  END_HANDLE_TH_ERRORS
}

// The paged batch from (k_cache, v_cache, block_table, cu_seqlens_q, kv_lens).
gbmoe_paged_kv_t paged(const gbmoe_attn_config_t& c, PyObject* const* a) {
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

// kv_append(config address, workspace address, q, k, v, k_cache, v_cache, block_table,
//           cu_seqlens_q, kv_lens, cos_sin, interleaved, q_out, stream)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 14)) return nullptr;
  const auto& c = *static_cast<const gbmoe_attn_config_t*>(address(a[0]));
  const gbmoe_paged_kv_t p = paged(c, a + 5);
  const at::Tensor& q = tensor(a[2], "q");
  const at::Tensor& k = tensor(a[3], "k");
  const at::Tensor& v = tensor(a[4], "v");
  TORCH_CHECK_VALUE(q.dim() > 0, "q must have rows");
  const int64_t T = q.size(0), hq = c.num_q_heads, hkv = c.num_kv_heads, d = c.head_dim;
  gbmoe_kv_append_args_t g = {};
  g.q = q.data_ptr();
  g.k = k.data_ptr();
  g.v = v.data_ptr();
  g.q_stride = row_stride(q, "q", T, hq * d);
  g.k_stride = row_stride(k, "k", T, hkv * d);
  g.v_stride = row_stride(v, "v", T, hkv * d);
  const CallStream stream(q, a[13]);
  Out out(a[12], "q_out", q, {T, hq, d}, at::kBFloat16);
  if (a[10] != Py_None) {
    const at::Tensor& cs = tensor(a[10], "cos_sin");
    TORCH_CHECK_VALUE(cs.is_cuda() && cs.scalar_type() == at::kFloat && cs.dim() == 2 &&
                          cs.is_contiguous(),
                      "cos_sin must be a contiguous CUDA float32 tensor [max_position, rotary_dim]");
    g.cos_sin = cs.data_ptr<float>();
    g.max_position = (int32_t)cs.size(0);
    g.rotary_dim = (int32_t)cs.size(1);
  }
  g.interleaved = PyObject_IsTrue(a[11]);
  g.q_out = out.ptr;
  g.workspace = address(a[1]);
  const int code = kv_append_fn(&c, (int32_t)T, &p, &g, stream.handle);
  return code ? failed("moe_kv_append", code) : out.obj.take();
  END_HANDLE_TH_ERRORS
}

// attention(config address, workspace address, workspace bytes, q, k_cache, v_cache, block_table,
//           cu_seqlens_q, kv_lens, out, lse (None, True or a tensor), stream)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 12)) return nullptr;
  const auto& c = *static_cast<const gbmoe_attn_config_t*>(address(a[0]));
  const size_t bytes = PyLong_AsSize_t(a[2]);
  if (PyErr_Occurred()) return nullptr;
  const gbmoe_paged_kv_t p = paged(c, a + 4);
  const at::Tensor& q = tensor(a[3], "q");
  TORCH_CHECK_VALUE(q.dim() > 0, "q must have rows");
  const int64_t T = q.size(0), hq = c.num_q_heads, d = c.head_dim;
  const int64_t stride = row_stride(q, "q", T, hq * d);
  const CallStream stream(q, a[11]);
  Out out(a[9], "out", q, {T, hq, d}, at::kBFloat16);
  Out lse;
  if (a[10] != Py_None) {
    Py_SETREF(lse.obj.p, Out::get(a[10] == Py_True ? Py_None : a[10], "lse", q, {T, hq}, at::kFloat,
                                  &lse.ptr));
    if (!lse.obj.p) return nullptr;
  }
  const int code = attention_fn(&c, (int32_t)T, &p, q.data_ptr(), stride, out.ptr,
                                static_cast<float*>(lse.ptr), address(a[1]), bytes, stream.handle);
  if (code) return failed("moe_paged_attention", code);
  if (a[10] == Py_None) return out.obj.take();
  return PyTuple_Pack(2, out.obj.p, lse.obj.p);
  END_HANDLE_TH_ERRORS
}

#define GBMOE_METHOD(f) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GBMOE_METHOD(bind), GBMOE_METHOD(rms_norm), GBMOE_METHOD(kv_append),
                         GBMOE_METHOD(attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&module); }
