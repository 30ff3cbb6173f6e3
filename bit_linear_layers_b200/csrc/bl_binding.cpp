// Native binding of the full-precision operators (bl_layer_norm,
// bl_embedding, bl_grad_clip and their gradients): argument checks, output
// and workspace allocation through torch's allocator, the current stream,
// then the entry point of the C ABI.
//
// These calls are short (a few microseconds on the GPU at one token), so what
// the host does per call shows: through ctypes a lookup of 16 tokens took
// 13.4 us of host time and clipping 180 tensors 240 us, nearly all of it
// reading tensors' attributes one by one.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>
#include <vector>

#include "bitlinear.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

py::handle g_error;  // the package's BitLinearError(name, status)

void check(const char* name, int rc) {
  if (rc == BL_OK) return;
  py::object e = py::reinterpret_borrow<py::object>(g_error)(name, rc);
  PyErr_SetObject(g_error.ptr(), e.ptr());
  throw py::error_already_set();
}

template <typename... Parts>
[[noreturn]] void refuse(const Parts&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  throw py::value_error(s.str());
}

void on_device(const Tensor& t, const char* name, const at::Device& dev) {
  if (!t.is_cuda()) refuse(name, " must be a CUDA tensor");
  if (t.device() != dev) refuse(name, " must be a CUDA tensor on ", dev);
}

int type_code(const Tensor& t, const char* name, const at::Device& dev) {
  on_device(t, name, dev);
  if (t.scalar_type() == at::kBFloat16) return BL_TYPE_BF16;
  if (t.scalar_type() == at::kFloat) return BL_TYPE_F32;
  refuse(name, " must be bfloat16 or float32, got ", t.scalar_type());
}

int id_code(const Tensor& t, const at::Device& dev) {
  on_device(t, "ids", dev);
  if (t.scalar_type() == at::kInt) return BL_IDS_I32;
  if (t.scalar_type() == at::kLong) return BL_IDS_I64;
  refuse("ids must be int32 or int64, got ", t.scalar_type());
}

// ids in the order of their shape: as they are where they lie so, else a copy (a few bytes for each row of D
// columns that is looked up or added); made under the device's guard, on the current stream
Tensor dense_ids(const Tensor& t) { return t.is_contiguous() ? t : t.contiguous(); }

// row pitch of an [M, K] tensor whose rows are dense
int64_t row_pitch(const Tensor& t, int64_t M, int64_t K, const char* name) {
  if (t.dim() != 2 || t.size(0) != M || t.size(1) != K) refuse(name, " must be [", M, ", ", K, "], got ", t.sizes());
  const int64_t ld = t.stride(0);
  if ((t.stride(1) != 1 && K > 1) || (ld < K && M > 1)) refuse(name, " must have dense rows that do not overlap");
  return std::max(ld, K);
}

// pointer of a dense fp32 vector of n elements (none: null)
float* vec(const OptTensor& t, int64_t n, const char* name, const at::Device& dev) {
  if (!t) return nullptr;
  on_device(*t, name, dev);
  if (t->scalar_type() != at::kFloat || t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
    refuse(name, " must be a contiguous float32 tensor of shape [", n, "]");
  return t->data_ptr<float>();
}

Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const at::Device& dev) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(dev));
}

Tensor workspace(int op, int64_t M, int64_t N, int64_t K, const at::Device& dev, const OptTensor& ws) {
  if (!ws) return empty({static_cast<int64_t>(bl_workspace_bytes(op, M, N, K))}, at::kByte, dev);
  on_device(*ws, "ws", dev);
  if (ws->scalar_type() != at::kByte || !ws->is_contiguous()) refuse("ws must be a contiguous uint8 tensor");
  return *ws;
}

void* stream_of(const at::Device& dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

py::object layer_norm(const Tensor& x, const OptTensor& weight, const OptTensor& bias, double eps, OptTensor out,
                      std::optional<at::ScalarType> out_dtype, bool stats, OptTensor mean, OptTensor rstd) {
  const at::Device dev = x.device();
  const int xt = type_code(x, "x", dev);
  if (x.dim() != 2) refuse("x must be [M, K], got ", x.sizes());
  const int64_t M = x.size(0), K = x.size(1);
  const int64_t ldx = row_pitch(x, M, K, "x");
  const c10::cuda::CUDAGuard guard(dev);
  if (!out)
    out = empty({M, K}, out_dtype.value_or(x.scalar_type()), dev);
  else if (out_dtype && out->scalar_type() != *out_dtype)
    refuse("out must be ", *out_dtype, ", got ", out->scalar_type());
  const int yt = type_code(*out, "out", dev);
  const int64_t ldy = row_pitch(*out, M, K, "out");
  if (stats && !mean) mean = empty({M}, at::kFloat, dev);
  if (stats && !rstd) rstd = empty({M}, at::kFloat, dev);
  check("bl_layer_norm",
        bl_layer_norm(x.const_data_ptr(), xt, ldx, vec(weight, K, "weight", dev), vec(bias, K, "bias", dev),
                      out->data_ptr(), yt, ldy, vec(mean, M, "mean", dev), vec(rstd, M, "rstd", dev), M, K,
                      static_cast<float>(eps), stream_of(dev)));
  if (!stats) return py::cast(*out);
  return py::make_tuple(*out, *mean, *rstd);
}

py::tuple layer_norm_backward(const Tensor& x, const OptTensor& weight, const Tensor& mean, const Tensor& rstd,
                              const Tensor& dy, bool want_dx, bool want_dw, OptTensor dx, OptTensor dweight,
                              OptTensor dbias, const OptTensor& ws) {
  const at::Device dev = x.device();
  const int xt = type_code(x, "x", dev), gt = type_code(dy, "dy", dev);
  if (x.dim() != 2) refuse("x must be [M, K], got ", x.sizes());
  const int64_t M = x.size(0), K = x.size(1);
  const int64_t ldx = row_pitch(x, M, K, "x"), lddy = row_pitch(dy, M, K, "dy");
  const c10::cuda::CUDAGuard guard(dev);
  int64_t lddx = K;
  if (!want_dx) {
    dx = std::nullopt;
  } else if (!dx) {
    dx = empty({M, K}, x.scalar_type(), dev);
  } else {
    if (type_code(*dx, "dx", dev) != xt) refuse("dx must be ", x.scalar_type(), ", got ", dx->scalar_type());
    lddx = row_pitch(*dx, M, K, "dx");
  }
  Tensor w;
  if (want_dw) {
    if (!dweight) dweight = empty({K}, at::kFloat, dev);
    if (!dbias) dbias = empty({K}, at::kFloat, dev);
    w = workspace(BL_OP_LAYER_NORM_BACKWARD, M, 0, K, dev, ws);
  } else {
    dweight = dbias = std::nullopt;
  }
  check("bl_layer_norm_backward",
        bl_layer_norm_backward(x.const_data_ptr(), xt, ldx, vec(weight, K, "weight", dev), vec(mean, M, "mean", dev),
                               vec(rstd, M, "rstd", dev), dy.const_data_ptr(), gt, lddy, dx ? dx->data_ptr() : nullptr,
                               lddx, vec(dweight, K, "dweight", dev), vec(dbias, K, "dbias", dev), M, K,
                               want_dw ? w.data_ptr() : nullptr, want_dw ? static_cast<size_t>(w.numel()) : 0,
                               stream_of(dev)));
  return py::make_tuple(dx, dweight, dbias);
}

Tensor embedding(const Tensor& ids, const Tensor& table, double scale, OptTensor out,
                 std::optional<at::ScalarType> out_dtype) {
  const at::Device dev = table.device();
  const int tt = type_code(table, "table", dev), it = id_code(ids, dev);
  if (table.dim() != 2 || !table.is_contiguous()) refuse("table must be a contiguous [V, D] tensor");
  const int64_t V = table.size(0), D = table.size(1);
  std::vector<int64_t> shape(ids.sizes().begin(), ids.sizes().end());
  shape.push_back(D);
  const c10::cuda::CUDAGuard guard(dev);
  if (!out)
    out = empty(shape, out_dtype.value_or(table.scalar_type()), dev);
  else if (out_dtype && out->scalar_type() != *out_dtype)
    refuse("out must be ", *out_dtype, ", got ", out->scalar_type());
  const int yt = type_code(*out, "out", dev);
  if (out->sizes() != at::IntArrayRef(shape) || !out->is_contiguous())
    refuse("out must be a contiguous tensor of shape ", at::IntArrayRef(shape));
  const Tensor id = dense_ids(ids);
  check("bl_embedding", bl_embedding(id.const_data_ptr(), it, table.const_data_ptr(), tt, out->data_ptr(), yt,
                                     ids.numel(), V, D, static_cast<float>(scale), stream_of(dev)));
  return *out;
}

Tensor embedding_backward(const Tensor& ids, const Tensor& dy, int64_t V, double scale,
                          std::optional<int64_t> padding_id, OptTensor out, std::optional<at::ScalarType> out_dtype,
                          bool accumulate, const OptTensor& ws) {
  const at::Device dev = dy.device();
  const int gt = type_code(dy, "dy", dev), it = id_code(ids, dev);
  if (dy.dim() != ids.dim() + 1 || !dy.is_contiguous() || dy.sizes().slice(0, size_t(ids.dim())) != ids.sizes())
    refuse("dy must be a contiguous [*ids.shape, D] tensor, got ", dy.sizes(), " for ids ", ids.sizes());
  const int64_t D = dy.size(-1), T = ids.numel();
  if (padding_id && (*padding_id < 0 || *padding_id >= V)) refuse("padding_id must be in [0, ", V, "), got ", *padding_id);
  const c10::cuda::CUDAGuard guard(dev);
  if (!out) {
    if (accumulate) refuse("accumulate=True adds to `out`: give it");
    out = empty({std::max<int64_t>(V, 0), D}, out_dtype.value_or(at::kFloat), dev);
  } else if (out_dtype && out->scalar_type() != *out_dtype) {
    refuse("out must be ", *out_dtype, ", got ", out->scalar_type());
  }
  const int tt = type_code(*out, "out", dev);
  if (out->dim() != 2 || out->size(0) != V || out->size(1) != D || !out->is_contiguous())
    refuse("out must be a contiguous tensor of shape [", V, ", ", D, "]");
  const Tensor w = workspace(BL_OP_EMBEDDING_BACKWARD, T, V, D, dev, ws);
  const Tensor id = dense_ids(ids);
  check("bl_embedding_backward",
        bl_embedding_backward(id.const_data_ptr(), it, dy.const_data_ptr(), gt, out->data_ptr(), tt, T, V, D,
                              static_cast<float>(scale), padding_id.value_or(-1), accumulate ? BL_EMBED_ACCUMULATE : 0u,
                              w.data_ptr(), static_cast<size_t>(w.numel()), stream_of(dev)));
  return *out;
}

const Tensor& tensor_at(const py::list& l, size_t i, const char* name) {
  PyObject* o = PyList_GET_ITEM(l.ptr(), static_cast<Py_ssize_t>(i));
  if (!THPVariable_Check(o)) refuse(name, " must be tensors");
  return THPVariable_Unpack(o);
}

// `outs`: a list of tensors or None, or None for the tensors themselves;
// norm_only: nothing is written
py::tuple grad_clip(const py::list& tensors, const std::optional<py::list>& outs, bool norm_only, double max_norm,
                    OptTensor stats, const OptTensor& ws) {
  const size_t n = tensors.size();
  if (n == 0) refuse("no tensors");
  if (n > (1u << 30)) refuse("too many tensors");
  if (outs && outs->size() != n) refuse(outs->size(), " outputs for ", n, " tensors");
  const at::Device dev = tensor_at(tensors, 0, "tensors").device();
  std::vector<bl_grad_tensor> rows(n);
  for (size_t i = 0; i < n; ++i) {
    const Tensor& t = tensor_at(tensors, i, "tensors");
    const int code = type_code(t, "tensors", dev);
    // the elements' order does not matter, only that they fill one run of memory
    if (t.layout() != at::kStrided || !t.is_non_overlapping_and_dense()) refuse("tensors must be dense");
    bl_grad_tensor& r = rows[i];
    r.numel = t.numel();
    r.type = code;
    r.g = t.const_data_ptr();
    r.out = nullptr;
    if (norm_only) continue;
    if (!outs) {
      r.out = t.data_ptr();
    } else if (PyList_GET_ITEM(outs->ptr(), static_cast<Py_ssize_t>(i)) != Py_None) {
      const Tensor& o = tensor_at(*outs, i, "outputs");
      if (!o.is_cuda() || o.device() != dev || o.scalar_type() != t.scalar_type() || o.numel() != r.numel ||
          !((t.is_contiguous() && o.is_contiguous()) || (o.sizes() == t.sizes() && o.strides() == t.strides())))
        refuse("an output must be a dense tensor of its gradient's type, size, layout and device");
      r.out = o.data_ptr();
    }
  }
  const c10::cuda::CUDAGuard guard(dev);
  if (!stats) stats = empty({2}, at::kFloat, dev);
  float* st = vec(stats, 2, "stats", dev);
  const Tensor w = workspace(BL_OP_GRAD_CLIP, static_cast<int64_t>(n), 0, 0, dev, ws);
  check("bl_grad_clip", bl_grad_clip(rows.data(), static_cast<int>(n), static_cast<float>(max_norm), st, w.data_ptr(),
                                     static_cast<size_t>(w.numel()), stream_of(dev)));
  return py::make_tuple(stats->select(0, 0), stats->select(0, 1));
}

}  // namespace

PYBIND11_MODULE(_native, m) {
  m.def("set_error", [](py::object e) { g_error = e.release(); });
  m.def("layer_norm", &layer_norm);
  m.def("layer_norm_backward", &layer_norm_backward);
  m.def("embedding", &embedding);
  m.def("embedding_backward", &embedding_backward);
  m.def("grad_clip", &grad_clip);
}
