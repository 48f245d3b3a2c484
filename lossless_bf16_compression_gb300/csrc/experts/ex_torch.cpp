// ex_torch.cpp -- the Python module _experts: the entry points of zc_moe.h, zc_router.h and zc_int4.h on torch
// tensors.
//
// What a call from Python costs is its checks, its outputs and its launch.  Here they take 4 us (8-bit
// blocks of 777 x 1000); the same steps made from Python one by one took 14, more than most kernels of a
// decode step.  Arguments are checked and outputs made on the current device and stream.  Host code
// only; the library's functions come from the copy of libzc.so that the process has loaded.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <Python.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>
#include <optional>
#include <string>

#include "zc_int4.h"
#include "zc_router.h"

namespace {

using at::Tensor;

#define FUNCTIONS(X)                                                                                        \
  X(zc_moe_sort_workspace) X(zc_moe_sort) X(zc_moe_dispatch) X(zc_moe_combine) X(zc_moe_combine_grad)       \
  X(zc_fp8_quantize) X(zc_fp8_scale_values) X(zc_fp8_column_blocks) X(zc_fp8_quantize_columns)              \
  X(zc_fp8_quantize_weight) X(zc_fp8_matmul_workspace) X(zc_fp8_matmul) X(zc_fp8_weight_grad)             \
  X(zc_moe_route) X(zc_moe_balance_workspace) X(zc_moe_balance) X(zc_moe_route_grad)                        \
  X(zc_int4_quantize) X(zc_int4_values) X(zc_int4_matmul)
struct {
#define MEMBER(f) decltype(&::f) f;
  FUNCTIONS(MEMBER)
#undef MEMBER
  PyObject* error;  // the class of a library error: (code, what)
} lib;

void call(int rc, const char* what) {
  if (rc == ZC_OK) return;
  PyObject* e = PyObject_CallFunction(lib.error, "is", rc, what);
  if (e != nullptr) {
    PyErr_SetObject(lib.error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

// ------------------------------------------------------------------ arguments

constexpr unsigned bit(at::ScalarType t) { return 1u << static_cast<unsigned>(t); }
constexpr unsigned kRows = bit(at::kBFloat16) | bit(at::kHalf) | bit(at::kFloat), kFloats = bit(at::kFloat),
                   kInts = bit(at::kInt), kIds = bit(at::kInt) | bit(at::kLong), kBytes = bit(at::kByte);

std::string names(unsigned types) {
  std::string s;
  for (unsigned i = 0; i < 32; ++i)
    if (types >> i & 1) s += (s.empty() ? "" : ", ") + std::string(c10::toString(static_cast<at::ScalarType>(i)));
  return s;
}

// The current device, asked for after the first argument turns out to be on a GPU.
class Device {
  mutable c10::DeviceIndex n_ = -1;

 public:
  c10::DeviceIndex number() const { return n_ < 0 ? n_ = c10::cuda::current_device() : n_; }
};

// A tensor on the current device, of one of the types, with `dim` dimensions (0: any).  One that requires a
// gradient is refused while gradients are recorded: results have no history, so training would lose it unseen.
const Tensor& tensor(PyObject* o, const char* name, const Device& device, unsigned types, int64_t dim) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a CUDA tensor");
  const Tensor& t = THPVariable_Unpack(o);
  TORCH_CHECK_TYPE(t.is_cuda(), name, " must be a CUDA tensor");
  const auto type = static_cast<unsigned>(t.scalar_type());
  TORCH_CHECK_TYPE(type < 32 && (types >> type & 1), name, " has dtype ", t.scalar_type(), ", expected one of ",
                   names(types));
  TORCH_CHECK_VALUE(dim == 0 || t.dim() == dim, name, " must have ", dim, " dimensions, got ", t.sizes());
  TORCH_CHECK_VALUE(t.get_device() == device.number(), name, " is on ", t.device(), ", not on the current device");
  // (asked in this order, since few tensors require a gradient)
  TORCH_CHECK(!t.requires_grad() || !c10::GradMode::is_enabled(), name, " requires a gradient, which this call would not "
              "pass on: its gradient is a call of its own (detach the tensor, or call under torch.no_grad or in a "
              "torch.autograd.Function)");
  return t;
}
int64_t number(PyObject* o) {
  const Py_ssize_t v = PyLong_AsSsize_t(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
void expect(Py_ssize_t n, Py_ssize_t of) { TORCH_CHECK_TYPE(n == of, "expected ", of, " arguments, got ", n); }

int type_of(at::ScalarType t) { return t == at::kBFloat16 ? ZC_TYPE_BF16 : t == at::kHalf ? ZC_TYPE_FP16 : ZC_TYPE_FP32; }

// Rows of contiguous values a pitch apart (copied when they are not laid out so).
struct Rows {
  Tensor t;
  int64_t rows, cols;
  size_t pitch;
  explicit Rows(const Tensor& from) : t(from), rows(from.size(0)), cols(from.size(1)) {
    if ((cols > 1 && t.stride(1) != 1) || (rows > 1 && t.stride(0) < cols)) t = t.contiguous();
    pitch = static_cast<size_t>(rows > 1 ? t.stride(0) : cols);
  }
  const void* data() const { return t.data_ptr(); }
  int type() const { return type_of(t.scalar_type()); }
};
Rows rows_of(PyObject* o, const char* name, const Device& device, int64_t rows = -1, int64_t cols = -1,
             unsigned types = kRows) {
  const Tensor& t = tensor(o, name, device, types, 2);
  TORCH_CHECK_VALUE((rows < 0 || t.size(0) == rows) && t.size(1) >= 1 && (cols < 0 || t.size(1) == cols), name,
                    " must be [", rows < 0 ? "rows" : std::to_string(rows), ", ",
                    cols < 0 ? "columns" : std::to_string(cols), "], got ", t.sizes());
  return Rows(t);
}

Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const Tensor& like) {
  return at::detail::empty_cuda(sizes, type, like.device(), std::nullopt);
}
cudaStream_t current(const Device& device) { return c10::cuda::getCurrentCUDAStream(device.number()).stream(); }

PyObject* results(std::initializer_list<const Tensor*> ts) {  // null: None
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (r == nullptr) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor* t : ts) {
    PyObject* o = t != nullptr ? THPVariable_Wrap(*t) : Py_NewRef(Py_None);
    if (o == nullptr) {
      Py_DECREF(r);
      throw python_error();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// ------------------------------------------------------------------ the order by expert

struct Ids {
  Tensor t;
  int64_t tokens, k, experts;
  Ids(PyObject* o, PyObject* n, const Device& device) {
    t = tensor(o, "experts_of", device, kIds, 2);
    experts = number(n);
    TORCH_CHECK_VALUE(experts >= 1 && experts <= ZC_MOE_MAX_EXPERTS, "num_experts must be 1 to ", ZC_MOE_MAX_EXPERTS,
                      ", got ", experts);
    tokens = t.size(0);
    k = t.size(1);
    TORCH_CHECK_VALUE(k >= 1 && k <= ZC_MOE_MAX_K, "experts_of must have 1 to ", ZC_MOE_MAX_K, " columns, got ", k);
    t = t.contiguous();
  }
  Tensor workspace() const {
    const size_t n = lib.zc_moe_sort_workspace(static_cast<size_t>(tokens * k), static_cast<int>(experts));
    return n ? empty({static_cast<int64_t>(n)}, at::kByte, t) : Tensor();
  }
};
struct Plan {
  const Tensor &position, &offsets;
  int64_t tokens, k, experts;
  Plan(PyObject* p, PyObject* o, const Device& device)
      : position(tensor(p, "plan.position", device, kInts, 2)), offsets(tensor(o, "plan.offsets", device, kInts, 1)) {
    TORCH_CHECK_VALUE(position.is_contiguous() && offsets.is_contiguous(), "a plan's tensors must be contiguous");
    tokens = position.size(0);
    k = position.size(1);
    experts = offsets.size(0) - 1;
    TORCH_CHECK_VALUE(experts >= 1 && experts <= ZC_MOE_MAX_EXPERTS && k >= 1 && k <= ZC_MOE_MAX_K, "a plan has 1 to ",
                      ZC_MOE_MAX_EXPERTS, " experts and 1 to ", ZC_MOE_MAX_K, " slots a token, got ", experts, " and ", k);
  }
  Tensor weights(PyObject* w, const Device& device) const {
    const Tensor& t = tensor(w, "weights", device, kFloats, 2);
    TORCH_CHECK_VALUE(t.sizes() == position.sizes(), "weights must have the shape ", position.sizes(), ", got ", t.sizes());
    return t.contiguous();
  }
};

PyObject* sort(PyObject*, PyObject* const* a, Py_ssize_t n) {  // experts_of, num_experts
  HANDLE_TH_ERRORS
  expect(n, 2);
  const Device device;
  const Ids ids(a[0], a[1], device);
  const Tensor position = empty({ids.tokens, ids.k}, at::kInt, ids.t), offsets = empty({ids.experts + 1}, at::kInt, ids.t);
  const Tensor scratch = ids.workspace();
  call(lib.zc_moe_sort(ids.t.data_ptr(), static_cast<int>(ids.t.element_size()), ids.tokens, static_cast<int>(ids.k),
                       static_cast<int>(ids.experts), position.data_ptr<int>(), offsets.data_ptr<int>(),
                       scratch.defined() ? scratch.data_ptr() : nullptr, current(device)),
       "zc_moe_sort");
  return results({&position, &offsets});
  END_HANDLE_TH_ERRORS
}

PyObject* dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {  // x, experts_of, num_experts
  HANDLE_TH_ERRORS
  expect(n, 3);
  const Device device;
  const Ids ids(a[1], a[2], device);
  const Rows x = rows_of(a[0], "x", device, ids.tokens);
  const Tensor rows = empty({ids.tokens * ids.k, x.cols}, x.t.scalar_type(), x.t);
  const Tensor position = empty({ids.tokens, ids.k}, at::kInt, x.t), offsets = empty({ids.experts + 1}, at::kInt, x.t);
  const Tensor scratch = ids.workspace();
  call(lib.zc_moe_dispatch(x.data(), x.pitch, x.type(), ids.t.data_ptr(), static_cast<int>(ids.t.element_size()),
                           ids.tokens, static_cast<int>(ids.k), static_cast<int>(ids.experts), x.cols, rows.data_ptr(),
                           x.cols, position.data_ptr<int>(), offsets.data_ptr<int>(),
                           scratch.defined() ? scratch.data_ptr() : nullptr, current(device)),
       "zc_moe_dispatch");
  return results({&rows, &position, &offsets});
  END_HANDLE_TH_ERRORS
}

PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n) {  // rows, weights or None, position, offsets
  HANDLE_TH_ERRORS
  expect(n, 4);
  const Device device;
  const Plan plan(a[2], a[3], device);
  const bool weighted = a[1] != Py_None;
  const Rows rows = rows_of(a[0], weighted ? "rows" : "d_rows", device, plan.tokens * plan.k);
  const Tensor weights = weighted ? plan.weights(a[1], device) : Tensor();
  const Tensor out = empty({plan.tokens, rows.cols}, rows.t.scalar_type(), rows.t);
  call(lib.zc_moe_combine(rows.data(), rows.pitch, rows.type(), weighted ? weights.data_ptr<float>() : nullptr,
                          plan.position.data_ptr<int>(), plan.offsets.data_ptr<int>(), plan.tokens,
                          static_cast<int>(plan.k), static_cast<int>(plan.experts), rows.cols, out.data_ptr(), rows.cols,
                          current(device)),
       "zc_moe_combine");
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

PyObject* combine_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {  // d_out, rows, weights, position, offsets
  HANDLE_TH_ERRORS
  expect(n, 5);
  const Device device;
  const Plan plan(a[3], a[4], device);
  const Tensor weights = plan.weights(a[2], device);
  const Rows rows = rows_of(a[1], "rows", device, plan.tokens * plan.k);
  const Rows d_out = rows_of(a[0], "d_out", device, plan.tokens, rows.cols, bit(rows.t.scalar_type()));
  const Tensor d_rows = empty({rows.rows, rows.cols}, rows.t.scalar_type(), rows.t);
  const Tensor d_weights = empty({plan.tokens, plan.k}, at::kFloat, rows.t);
  call(lib.zc_moe_combine_grad(d_out.data(), d_out.pitch, rows.data(), rows.pitch, rows.type(),
                               weights.data_ptr<float>(), plan.position.data_ptr<int>(), plan.offsets.data_ptr<int>(),
                               plan.tokens, static_cast<int>(plan.k), static_cast<int>(plan.experts), rows.cols,
                               d_rows.data_ptr(), rows.cols, d_weights.data_ptr<float>(), current(device)),
       "zc_moe_combine_grad");
  return results({&d_rows, &d_weights});
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ 8-bit blocks

constexpr int64_t kBlock = ZC_FP8_BLOCK;
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Blocks {  // values and scales of rows x cols, or of one such matrix for each group
  Tensor data, scales;
  Blocks(int64_t groups, int64_t rows, int64_t cols, const Tensor& like) {
    const int64_t blocks = ceil_div(cols, kBlock), d[3] = {groups, rows, blocks * kBlock},
                  s[4] = {groups, ceil_div(blocks, 4), rows, 4};
    const int skip = groups == 0 ? 1 : 0;
    data = empty(at::IntArrayRef(d + skip, 3 - skip), at::kByte, like);
    scales = empty(at::IntArrayRef(s + skip, 4 - skip), at::kByte, like);
  }
};

// The groups' starts, or null for one group of all the rows.
const int* starts(PyObject* o, const Device& device, int64_t* groups) {
  *groups = 1;
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(o, "offsets", device, kInts, 1);
  TORCH_CHECK_VALUE(t.size(0) >= 2 && t.size(0) <= ZC_MOE_MAX_EXPERTS + 1, "offsets must have 2 to ",
                    ZC_MOE_MAX_EXPERTS + 1, " entries");
  TORCH_CHECK_VALUE(t.is_contiguous(), "offsets must be contiguous");
  *groups = t.size(0) - 1;
  return t.data_ptr<int>();
}

PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {  // x, format
  HANDLE_TH_ERRORS
  expect(n, 2);
  const Device device;
  const Rows x = rows_of(a[0], "x", device);
  const Blocks q(0, x.rows, x.cols, x.t);
  call(lib.zc_fp8_quantize(x.data(), x.pitch, x.type(), x.rows, x.cols, static_cast<int>(number(a[1])),
                           q.data.data_ptr(), q.scales.data_ptr(), current(device)),
       "zc_fp8_quantize");
  return results({&q.data, &q.scales});
  END_HANDLE_TH_ERRORS
}

PyObject* quantize_columns(PyObject*, PyObject* const* a, Py_ssize_t n) {  // x, offsets or None, format
  HANDLE_TH_ERRORS
  expect(n, 3);
  const Device device;
  const Rows x = rows_of(a[0], "x", device);
  int64_t groups;
  const int* at = starts(a[1], device, &groups);
  const auto capacity = static_cast<int64_t>(lib.zc_fp8_column_blocks(x.rows, static_cast<int>(groups)));
  const Blocks q(0, x.cols, capacity * kBlock, x.t);
  const Tensor first = empty({groups + 1}, at::kInt, x.t);
  call(lib.zc_fp8_quantize_columns(x.data(), x.pitch, x.type(), x.rows, x.cols, static_cast<int>(groups), at,
                                   static_cast<int>(number(a[2])), q.data.data_ptr(), q.scales.data_ptr(),
                                   first.data_ptr<int>(), current(device)),
       "zc_fp8_quantize_columns");
  return results({&q.data, &q.scales, &first});
  END_HANDLE_TH_ERRORS
}

PyObject* quantize_weight(PyObject*, PyObject* const* a, Py_ssize_t n) {  // w, format, transposed
  HANDLE_TH_ERRORS
  expect(n, 3);
  const Device device;
  Tensor w = tensor(a[0], "w", device, kRows, 0);
  const int64_t dim = w.dim();
  TORCH_CHECK_VALUE((dim == 2 || dim == 3) && w.numel() > 0, "w must be [n, k] or [experts, n, k], got ", w.sizes());
  const int64_t groups = dim == 3 ? w.size(0) : 0, rows = w.size(dim - 2), cols = w.size(dim - 1);
  TORCH_CHECK_VALUE(groups <= ZC_MOE_MAX_EXPERTS, "at most ", ZC_MOE_MAX_EXPERTS, " experts");
  w = w.contiguous();
  const bool transposed = a[2] == Py_True;
  const Blocks q(groups, rows, cols, w);
  std::optional<Blocks> t;
  if (transposed) t.emplace(groups, cols, rows, w);
  call(lib.zc_fp8_quantize_weight(w.data_ptr(), type_of(w.scalar_type()), static_cast<int>(groups ? groups : 1), rows,
                                  cols, static_cast<int>(number(a[1])), q.data.data_ptr(), q.scales.data_ptr(),
                                  t ? t->data.data_ptr() : nullptr, t ? t->scales.data_ptr() : nullptr, current(device)),
       "zc_fp8_quantize_weight");
  return results({&q.data, &q.scales, t ? &t->data : nullptr, t ? &t->scales : nullptr});
  END_HANDLE_TH_ERRORS
}

PyObject* scale_values(PyObject*, PyObject* const* a, Py_ssize_t n) {  // scales
  HANDLE_TH_ERRORS
  expect(n, 1);
  const Device device;
  const Tensor& scales = tensor(a[0], "scales", device, kBytes, 0);
  TORCH_CHECK_VALUE(scales.is_contiguous() && scales.numel() % 4 == 0, "scales must be contiguous words of four bytes, got ",
                    scales.sizes());
  const Tensor out = empty(scales.sizes(), at::kFloat, scales);
  call(lib.zc_fp8_scale_values(scales.data_ptr(), static_cast<size_t>(scales.numel()) / 4, out.data_ptr<float>(),
                               current(device)),
       "zc_fp8_scale_values");
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

PyObject* values(PyObject*, PyObject* const* a, Py_ssize_t n) {  // data, format, columns
  HANDLE_TH_ERRORS
  expect(n, 3);
  TORCH_CHECK_TYPE(THPVariable_Check(a[0]), "data must be a tensor");
  const Tensor v = THPVariable_Unpack(a[0]).view(number(a[1]) == ZC_FP8_E4M3 ? at::kFloat8_e4m3fn : at::kFloat8_e5m2);
  const int64_t cols = number(a[2]);
  return THPVariable_Wrap(v.size(-1) == cols ? v : v.narrow(-1, 0, cols));
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ products

// A matrix in blocks: its values, scales, format and columns, four arguments.
struct Operand {
  const Tensor &data, &scales;
  int format;
  int64_t cols;
  Operand(PyObject* const* a, const char* name, const Device& device, int64_t dim)
      : data(tensor(a[0], name, device, kBytes, dim)), scales(tensor(a[1], "scales", device, kBytes, 0)),
        format(static_cast<int>(number(a[2]))), cols(number(a[3])) {
    // A Matrix is checked when it is made, but its tensors can be exchanged: what the kernels read is looked at here.
    const bool grouped = data.dim() == 3;
    const int64_t blocks = ceil_div(cols, kBlock);
    TORCH_CHECK_VALUE(cols >= 0 && (grouped || data.dim() == 2) && data.size(-1) == blocks * kBlock &&
                          scales.numel() == (grouped ? data.size(0) : 1) * data.size(-2) * ceil_div(blocks, 4) * 4 &&
                          data.is_contiguous() && scales.is_contiguous(),
                      name, " must hold contiguous rows of ", cols, " values and a scale for each block, got ",
                      data.sizes(), " and scales ", scales.sizes());
  }
};
at::ScalarType out_type(PyObject* o) { return number(o) == ZC_TYPE_FP32 ? at::kFloat : at::kBFloat16; }

PyObject* matmul(PyObject*, PyObject* const* args, Py_ssize_t n) {  // a, b, offsets or None, type of out
  HANDLE_TH_ERRORS
  expect(n, 10);
  const Device device;
  const Operand a(args, "a", device, 2), b(args + 4, "b", device, 0);
  int64_t groups;
  const int* at = starts(args[8], device, &groups);
  TORCH_CHECK_VALUE(a.cols == b.cols && a.cols >= 1, "a has rows of ", a.cols, " values, b of ", b.cols);
  TORCH_CHECK_VALUE((b.data.dim() == 3 ? b.data.size(0) : 1) == groups, "b must hold ", groups, " matrices, got ",
                    b.data.sizes());
  const int64_t rows = a.data.size(0), width = b.data.size(-2);
  const at::ScalarType type = out_type(args[9]);
  const Tensor out = empty({rows, width}, type, a.data);
  const size_t need = lib.zc_fp8_matmul_workspace(rows, static_cast<int>(groups), width, a.cols);
  const Tensor scratch = need ? empty({static_cast<int64_t>(need)}, at::kByte, a.data) : Tensor();
  call(lib.zc_fp8_matmul(a.data.data_ptr(), a.scales.data_ptr(), a.format, rows, b.data.data_ptr(), b.scales.data_ptr(),
                         b.format, static_cast<int>(groups), width, a.cols, at, out.data_ptr(), width, type_of(type),
                         need ? scratch.data_ptr() : nullptr, current(device)),
       "zc_fp8_matmul");
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

PyObject* weight_grad(PyObject*, PyObject* const* args, Py_ssize_t n) {  // dy, x, the first block of each group, type
  HANDLE_TH_ERRORS
  expect(n, 10);
  const Device device;
  const Operand dy(args, "dy", device, 2), x(args + 4, "x", device, 2);
  int64_t groups;
  const int* at = starts(args[8], device, &groups);
  TORCH_CHECK_VALUE(at != nullptr && dy.cols == x.cols, "dy and x must have the same groups");
  const at::ScalarType type = out_type(args[9]);
  const Tensor out = empty({groups, dy.data.size(0), x.data.size(0)}, type, x.data);
  call(lib.zc_fp8_weight_grad(dy.data.data_ptr(), dy.scales.data_ptr(), dy.format, x.data.data_ptr(),
                              x.scales.data_ptr(), x.format, ceil_div(x.cols, kBlock), static_cast<int>(groups), out.size(1),
                              out.size(2), at, out.data_ptr(), type_of(type), current(device)),
       "zc_fp8_weight_grad");
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ the router

struct Logits : Rows {
  Logits(PyObject* o, const Device& device, int64_t tokens = -1) : Rows(rows_of(o, "logits", device, tokens)) {
    TORCH_CHECK_VALUE(cols <= ZC_MOE_MAX_EXPERTS, "logits must have 1 to ", ZC_MOE_MAX_EXPERTS, " columns, got ", cols);
  }
};
// What a routing chose: int32 (that is what moe.route returns), rows of k.
Tensor chosen(PyObject* o, const Device& device) {
  const Tensor& t = tensor(o, "experts_of", device, kInts, 2);
  TORCH_CHECK_VALUE(t.size(1) >= 1 && t.size(1) <= ZC_MOE_MAX_K, "experts_of must have 1 to ", ZC_MOE_MAX_K,
                    " columns, got ", t.size(1));
  return t.contiguous();
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(v);
}

PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {  // logits, k, score, normalize, scale
  HANDLE_TH_ERRORS
  expect(n, 5);
  const Device device;
  const Logits x(a[0], device);
  const int64_t k = number(a[1]);
  TORCH_CHECK_VALUE(k >= 1 && k <= ZC_MOE_MAX_K && k <= x.cols, "k must be 1 to ",
                    std::min<int64_t>(ZC_MOE_MAX_K, x.cols), ", got ", k);
  const Tensor weights = empty({x.rows, k}, at::kFloat, x.t), ids = empty({x.rows, k}, at::kInt, x.t);
  call(lib.zc_moe_route(x.data(), x.pitch, x.type(), x.rows, static_cast<int>(x.cols), static_cast<int>(k),
                        static_cast<int>(number(a[2])), a[3] == Py_True, real(a[4]), weights.data_ptr<float>(),
                        ids.data_ptr<int>(), current(device)),
       "zc_moe_route");
  return results({&weights, &ids});
  END_HANDLE_TH_ERRORS
}

PyObject* balance(PyObject*, PyObject* const* a, Py_ssize_t n) {  // logits, experts_of, score
  HANDLE_TH_ERRORS
  expect(n, 3);
  const Device device;
  const Tensor ids = chosen(a[1], device);
  const Logits x(a[0], device, ids.size(0));
  const Tensor loss = empty({}, at::kFloat, x.t), counts = empty({x.cols}, at::kInt, x.t),
               slope = empty({x.cols}, at::kFloat, x.t);
  const size_t need = lib.zc_moe_balance_workspace(x.rows, static_cast<int>(x.cols));
  const Tensor scratch = need ? empty({static_cast<int64_t>(need)}, at::kByte, x.t) : Tensor();
  call(lib.zc_moe_balance(x.data(), x.pitch, x.type(), ids.data_ptr<int>(), x.rows, static_cast<int>(x.cols),
                          static_cast<int>(ids.size(1)), static_cast<int>(number(a[2])), loss.data_ptr<float>(),
                          counts.data_ptr<int>(), slope.data_ptr<float>(), need ? scratch.data_ptr() : nullptr,
                          current(device)),
       "zc_moe_balance");
  return results({&loss, &counts, &slope});
  END_HANDLE_TH_ERRORS
}

// logits, d_weights or None, experts_of or None, d_loss or None, slope or None, score, normalize, scale
PyObject* route_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 8);
  const Device device;
  const Logits x(a[0], device);
  Tensor d_weights, ids, slope, d_loss;
  if (a[1] != Py_None) {
    ids = chosen(a[2], device);
    d_weights = tensor(a[1], "d_weights", device, kFloats, 2).contiguous();
    TORCH_CHECK_VALUE(ids.size(0) == x.rows, "experts_of must have ", x.rows, " rows, got ", ids.size(0));
    TORCH_CHECK_VALUE(d_weights.sizes() == ids.sizes(), "d_weights must have the shape ", ids.sizes(), ", got ",
                      d_weights.sizes());
  }
  if (a[3] != Py_None) {
    d_loss = tensor(a[3], "d_loss", device, kFloats, 0);
    TORCH_CHECK_VALUE(d_loss.numel() == 1, "d_loss must have one element, got ", d_loss.sizes());
    slope = tensor(a[4], "slope", device, kFloats, 1).contiguous();
    TORCH_CHECK_VALUE(slope.size(0) == x.cols, "slope must have ", x.cols, " elements, got ", slope.sizes());
  }
  const Tensor d = empty({x.rows, x.cols}, x.t.scalar_type(), x.t);
  call(lib.zc_moe_route_grad(ids.defined() ? d_weights.data_ptr<float>() : nullptr,
                             ids.defined() ? ids.data_ptr<int>() : nullptr,
                             slope.defined() ? d_loss.data_ptr<float>() : nullptr,
                             slope.defined() ? slope.data_ptr<float>() : nullptr, x.data(), x.pitch, x.type(), x.rows,
                             static_cast<int>(x.cols), ids.defined() ? static_cast<int>(ids.size(1)) : 1,
                             static_cast<int>(number(a[5])), a[6] == Py_True, real(a[7]), d.data_ptr(), x.cols,
                             current(device)),
       "zc_moe_route_grad");
  return THPVariable_Wrap(d);
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ 4-bit weights

// Records and scales of n x k weights, or of one such matrix for each group; checked at every call, since a Matrix's
// tensors can be exchanged.
struct Weights4 {
  const Tensor &data, &scales;
  int64_t n, k, groups;
  Weights4(PyObject* const* a, const Device& device)
      : data(tensor(a[0], "data", device, kBytes, 0)), scales(tensor(a[1], "scales", device, bit(at::kBFloat16), 0)),
        n(number(a[2])), k(number(a[3])) {
    const int64_t dim = data.dim();
    groups = dim == 4 ? data.size(0) : 1;
    const int64_t tiles = ceil_div(n, ZC_INT4_ROWS), blocks = ceil_div(k, ZC_INT4_GROUP);
    TORCH_CHECK_VALUE(n >= 1 && k >= 1 && (dim == 3 || dim == 4) && data.size(dim - 3) == tiles &&
                          data.size(dim - 2) == blocks && data.size(dim - 1) == ZC_INT4_GROUP * ZC_INT4_ROWS / 2 &&
                          scales.numel() == groups * tiles * blocks * ZC_INT4_ROWS && data.is_contiguous() &&
                          scales.is_contiguous(),
                      "the records and scales of ", n, " x ", k, " weights do not have the shapes ", data.sizes(), " and ",
                      scales.sizes());
    TORCH_CHECK_VALUE(groups >= 1 && groups <= ZC_MOE_MAX_EXPERTS, "1 to ", ZC_MOE_MAX_EXPERTS, " experts, got ", groups);
  }
};

PyObject* quantize4(PyObject*, PyObject* const* a, Py_ssize_t n) {  // w
  HANDLE_TH_ERRORS
  expect(n, 1);
  const Device device;
  Tensor w = tensor(a[0], "w", device, kRows, 0);
  const int64_t dim = w.dim();
  TORCH_CHECK_VALUE((dim == 2 || dim == 3) && w.numel() > 0, "w must be [n, k] or [experts, n, k], got ", w.sizes());
  const int64_t groups = dim == 3 ? w.size(0) : 1, rows = w.size(dim - 2), cols = w.size(dim - 1);
  TORCH_CHECK_VALUE(groups <= ZC_MOE_MAX_EXPERTS, "at most ", ZC_MOE_MAX_EXPERTS, " experts");
  w = w.contiguous();
  const int64_t tiles = ceil_div(rows, ZC_INT4_ROWS), blocks = ceil_div(cols, ZC_INT4_GROUP), skip = dim == 3 ? 0 : 1;
  const int64_t d[4] = {groups, tiles, blocks, ZC_INT4_GROUP * ZC_INT4_ROWS / 2}, s[4] = {groups, tiles, blocks, ZC_INT4_ROWS};
  const Tensor data = empty(at::IntArrayRef(d + skip, 4 - skip), at::kByte, w),
               scales = empty(at::IntArrayRef(s + skip, 4 - skip), at::kBFloat16, w);
  call(lib.zc_int4_quantize(w.data_ptr(), type_of(w.scalar_type()), static_cast<int>(groups), rows, cols, data.data_ptr(),
                            scales.data_ptr(), current(device)),
       "zc_int4_quantize");
  return results({&data, &scales});
  END_HANDLE_TH_ERRORS
}

constexpr at::ScalarType kTypes[] = {at::kBFloat16, at::kHalf, at::kFloat};  // by ZC_TYPE_*
at::ScalarType type_at(PyObject* o) {
  const int64_t i = number(o);
  TORCH_CHECK_VALUE(i >= 0 && i < 3, "no such type: ", i);
  return kTypes[i];
}

PyObject* values4(PyObject*, PyObject* const* a, Py_ssize_t n) {  // data, scales, n, k, type
  HANDLE_TH_ERRORS
  expect(n, 5);
  const Device device;
  const Weights4 w(a, device);
  const at::ScalarType type = type_at(a[4]);
  const int64_t d[3] = {w.groups, w.n, w.k}, skip = w.data.dim() == 4 ? 0 : 1;
  const Tensor out = empty(at::IntArrayRef(d + skip, 3 - skip), type, w.data);
  call(lib.zc_int4_values(w.data.data_ptr(), w.scales.data_ptr(), static_cast<int>(w.groups), w.n, w.k, type_of(type),
                          out.data_ptr(), current(device)),
       "zc_int4_values");
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

PyObject* matmul4(PyObject*, PyObject* const* a, Py_ssize_t n) {  // x, data, scales, n, k, offsets or None, type or None
  HANDLE_TH_ERRORS
  expect(n, 7);
  const Device device;
  const Weights4 w(a + 1, device);
  const Rows x = rows_of(a[0], "x", device, -1, w.k);
  int64_t groups;
  const int* at = starts(a[5], device, &groups);
  TORCH_CHECK_VALUE(w.groups == groups, "the weights must be of ", groups, " experts, got ", w.data.sizes());
  const at::ScalarType type = a[6] == Py_None ? x.t.scalar_type() : type_at(a[6]);
  const Tensor out = empty({x.rows, w.n}, type, x.t);
  call(lib.zc_int4_matmul(x.data(), x.pitch, x.type(), x.rows, w.data.data_ptr(), w.scales.data_ptr(),
                          static_cast<int>(groups), w.n, w.k, at, out.data_ptr(), w.n, type_of(type), current(device)),
       "zc_int4_matmul");
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ the module

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {  // the loaded library's handle, the class of its errors
  HANDLE_TH_ERRORS
  expect(n, 2);
  void* handle = PyLong_AsVoidPtr(a[0]);
  if (handle == nullptr && PyErr_Occurred()) throw python_error();
#define FIND(f)                                                       \
  lib.f = reinterpret_cast<decltype(lib.f)>(dlsym(handle, #f));      \
  TORCH_CHECK(lib.f != nullptr, "libzc.so has no " #f ": build it again");
  FUNCTIONS(FIND)
#undef FIND
  lib.error = Py_NewRef(a[1]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef method(const char* name, Fast f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method("bind", bind),
                         method("sort", sort),
                         method("dispatch", dispatch),
                         method("combine", combine),
                         method("combine_grad", combine_grad),
                         method("quantize", quantize),
                         method("quantize_columns", quantize_columns),
                         method("quantize_weight", quantize_weight),
                         method("scale_values", scale_values),
                         method("values", values),
                         method("matmul", matmul),
                         method("weight_grad", weight_grad),
                         method("route", route),
                         method("balance", balance),
                         method("route_grad", route_grad),
                         method("quantize4", quantize4),
                         method("values4", values4),
                         method("matmul4", matmul4),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_experts", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__experts() { return PyModule_Create(&module); }
