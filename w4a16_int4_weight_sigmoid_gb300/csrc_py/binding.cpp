// Python binding of the expert-order rows and the MXFP4 operators: tensor
// checks and argument marshalling in C++.  A call of the Python binding spent
// 4 to 5 us on the host on its checks and the ctypes conversions, more than
// the launch and most of these kernels at decoding sizes; here they take a
// few tenths.  Every function returns the C entry point's status and raises
// TypeError or ValueError, before anything is launched, for tensors that the
// entry point, which sees raw pointers, cannot check.
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "chord_moe.h"

namespace {

// A Python exception is set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(type, fmt, ap);
  va_end(ap);
  throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be a CUDA tensor", name);
  return t;
}

int dtype_code(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return CHORD_DTYPE_BF16;
    case at::kHalf: return CHORD_DTYPE_FP16;
    case at::kFloat: return CHORD_DTYPE_FP32;
    default: raise(PyExc_TypeError, "%s must be bfloat16, float16 or float32, got %s", name, t.dtype().name().data());
  }
}

// A matrix of rows with unit column stride.
struct Rows {
  void* p;
  int dtype;
  int64_t n, h, stride;
  Rows(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    dtype = dtype_code(t, name);
    // (strides mean nothing without elements)
    if (t.dim() != 2 || (t.size(0) > 0 && t.size(1) > 1 && t.stride(1) != 1))
      raise(PyExc_ValueError, "%s must be a matrix of rows with unit column stride", name);
    p = t.data_ptr();
    n = t.size(0);
    h = t.size(1);
    // the row stride of a single row means nothing
    stride = n > 1 ? t.stride(0) : std::max<int64_t>(t.stride(0), h);
  }
  // The same type and row length as `r`, and `rows` rows where given.
  Rows(PyObject* o, const char* name, const Rows& r, int64_t rows = -1) : Rows(o, name) {
    if (dtype != r.dtype) raise(PyExc_TypeError, "%s is of another type", name);
    if (h != r.h) raise(PyExc_ValueError, "%s's rows hold %lld values, need %lld", name, (long long)h, (long long)r.h);
    if (rows >= 0 && n != rows)
      raise(PyExc_ValueError, "%s has %lld rows, need %lld", name, (long long)n, (long long)rows);
  }
};

// A contiguous tensor of `n` values (any number when negative) of one type.
template <typename T>
T* values(PyObject* o, at::ScalarType type, int64_t n, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s must be %s, got %s", name, at::toString(type), t.dtype().name().data());
  if (!t.is_contiguous() || (n >= 0 && t.numel() != n))
    raise(PyExc_ValueError, "%s must hold %lld contiguous values", name, (long long)n);
  return static_cast<T*>(t.data_ptr());
}
int32_t* ints(PyObject* o, int64_t n, const char* name) { return values<int32_t>(o, at::kInt, n, name); }
uint8_t* bytes(PyObject* o, int64_t n, const char* name) { return values<uint8_t>(o, at::kByte, n, name); }
size_t numel(PyObject* o) { return static_cast<size_t>(THPVariable_Unpack(o).numel()); }

// A [tokens, topk] FP32 matrix of routing weights.
const float* weights(PyObject* o, int64_t& M, int64_t& k) {
  const float* w = values<float>(o, at::kFloat, -1, "topk_weights");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.dim() != 2) raise(PyExc_ValueError, "topk_weights must be [tokens, topk]");
  M = t.size(0);
  k = t.size(1);
  return w;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
// An int parameter of the C ABI; sizes beyond it are refused.
int narrow(int64_t v, const char* name) {
  if (v < INT_MIN || v > INT_MAX) raise(PyExc_ValueError, "%s=%lld does not fit 32 bits", name, (long long)v);
  return static_cast<int>(v);
}
size_t size(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < 0) raise(PyExc_ValueError, "%s=%lld < 0", name, (long long)v);
  return static_cast<size_t>(v);
}
// None: the current stream; otherwise a raw handle.
void* stream(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  return reinterpret_cast<void*>(integer(o));
}

int permute(PyObject* const* a) {
  const Rows x(a[0], "x"), out(a[5], "out", x);
  const int k = narrow(integer(a[4]), "topk"), M = narrow(x.n, "tokens");
  return chord_moe_permute(x.p, x.dtype, x.stride, ints(a[1], x.n * k, "sorted_positions"),
                           ints(a[2], out.n, "sorted_token_ids"), ints(a[3], 1, "num_tokens_post_padded"), M, k,
                           narrow(x.h, "row length"), out.n, out.p, out.stride, stream(a[6]));
}

int permute_backward(PyObject* const* a) {
  const Rows dout(a[0], "dout"), dx(a[3], "dx", dout);
  const int k = narrow(integer(a[2]), "topk");
  return chord_moe_permute_backward(dout.p, dout.dtype, dout.stride, ints(a[1], dx.n * k, "sorted_positions"),
                                    narrow(dx.n, "tokens"), k, narrow(dx.h, "row length"), dout.n, dx.p, dx.stride,
                                    stream(a[4]));
}

int unpermute(PyObject* const* a) {
  int64_t M, k;
  const Rows y(a[0], "y");
  const float* w = weights(a[1], M, k);
  const Rows out(a[3], "out", y, M);
  return chord_moe_unpermute(y.p, y.dtype, y.stride, w, ints(a[2], M * k, "sorted_positions"), narrow(M, "tokens"),
                             narrow(k, "topk"), narrow(y.h, "row length"), y.n, out.p, out.stride, stream(a[4]));
}

int unpermute_backward(PyObject* const* a) {
  int64_t M, k;
  const float* w = weights(a[2], M, k);
  const Rows dout(a[0], "dout"), y(a[1], "y", dout), dy(a[6], "dy", dout, y.n);
  if (dout.n != M) raise(PyExc_ValueError, "dout has %lld rows, need %lld", (long long)dout.n, (long long)M);
  return chord_moe_unpermute_backward(
      dout.p, y.p, dout.dtype, dout.stride, y.stride, w, ints(a[3], M * k, "sorted_positions"),
      ints(a[4], y.n, "sorted_token_ids"), ints(a[5], 1, "num_tokens_post_padded"), narrow(M, "tokens"),
      narrow(k, "topk"), narrow(y.h, "row length"), y.n, dy.p, dy.stride,
      values<float>(a[7], at::kFloat, M * k, "dweights"), stream(a[8]));
}

int quantize(PyObject* const* a) {
  const Rows x(a[0], "x");
  return chord_mxfp4_quantize(x.p, x.dtype, x.stride, x.n, narrow(x.h, "K"), bytes(a[1], x.n * x.h / 2, "codes"),
                              bytes(a[2], x.n * x.h / 32, "scales"), stream(a[3]));
}

int dequantize(PyObject* const* a) {
  const Rows out(a[2], "out");
  return chord_mxfp4_dequantize(bytes(a[0], out.n * out.h / 2, "codes"), bytes(a[1], out.n * out.h / 32, "scales"),
                                out.n, narrow(out.h, "K"), out.p, out.dtype, out.stride, stream(a[3]));
}

int quantize_rows(PyObject* const* a) {
  const Rows x(a[0], "x");
  const int k = narrow(integer(a[2]), "topk");
  const int32_t* pos = a[1] == Py_None ? nullptr : ints(a[1], x.n * k, "sorted_positions");
  const int32_t* total = a[3] == Py_None ? nullptr : ints(a[3], 1, "num_tokens_post_padded");
  uint8_t* rows = bytes(a[5], -1, "rows");
  return chord_mxfp4_quantize_rows(x.p, x.dtype, x.stride, narrow(x.n, "tokens"), narrow(x.h, "K"), pos, k, total,
                                   size(a[4], "capacity"), rows, numel(a[5]), stream(a[6]));
}

int moe_gemm(PyObject* const* a) {
  const int E = narrow(integer(a[2]), "E_local"), N = narrow(integer(a[3]), "N"), K = narrow(integer(a[4]), "K");
  const size_t capacity = size(a[7], "capacity");
  const int epilogue = narrow(integer(a[8]), "epilogue");
  const int64_t cols = epilogue == CHORD_EPI_SILU_MUL ? N / 2 : N;
  const uint8_t* rows = bytes(a[0], -1, "rows");
  const uint8_t* packed = bytes(a[1], -1, "packed_w");
  if (numel(a[1]) < chord_mxfp4_prepack_bytes(E, N, K))
    raise(PyExc_ValueError, "packed_w is smaller than E_local, N and K need");
  const at::Tensor& C = tensor(a[9], "C");
  if (C.scalar_type() != at::kBFloat16 || C.dim() != 2 || C.size(0) != static_cast<int64_t>(capacity) ||
      C.size(1) != cols || !C.is_contiguous())
    raise(PyExc_ValueError, "C must be contiguous bfloat16 [%zu, %lld]", capacity, (long long)cols);
  void* ws = bytes(a[10], -1, "workspace");
  int* status = a[11] == Py_None ? nullptr : ints(a[11], 1, "dev_status");
  return chord_mxfp4_moe_gemm(rows, numel(a[0]), packed, E, N, K, ints(a[5], E, "expert_counts"),
                              ints(a[6], E + 1LL, "expert_offsets"), capacity, epilogue,
                              static_cast<chord_bf16*>(C.data_ptr()), ws, numel(a[10]), status, stream(a[12]));
}

template <int (*kCall)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "%d arguments are needed, got %zd", kArgs, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(kCall(args));
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <int (*kCall)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<kCall, kArgs>)), METH_FASTCALL,
          nullptr};
}

PyMethodDef kMethods[] = {
    method<permute, 7>("permute"),
    method<permute_backward, 5>("permute_backward"),
    method<unpermute, 5>("unpermute"),
    method<unpermute_backward, 9>("unpermute_backward"),
    method<quantize, 4>("quantize"),
    method<dequantize, 4>("dequantize"),
    method<quantize_rows, 7>("quantize_rows"),
    method<moe_gemm, 13>("moe_gemm"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_chord", "Checked calls of the chord_moe library.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__chord(void) { return PyModule_Create(&kModule); }
