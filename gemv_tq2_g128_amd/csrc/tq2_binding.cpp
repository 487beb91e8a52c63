// Python module `_binding`: torch tensors into the argument structs of tq2_attn.h,
// tq2_q4.h, tq2_moe.h and tq2_sample.h, and the call on the tensors' device and its current stream.
//
// A decode step makes a handful of these calls on small tensors, whose kernels
// take 3 to 10 us: reading the tensors' types, shapes and strides from Python
// took 7 us of an append's 11, here it takes under one.  Argument marshalling
// only: every check that the C entry points make is left to them, and their
// status is returned where it is not TQ2_OK.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>
#include <optional>
#include <string>

#include <ATen/ops/empty.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tq2.h"
#include "tq2_attn.h"
#include "tq2_moe.h"
#include "tq2_q4.h"
#include "tq2_sample.h"

namespace {

// A Python exception to be: caught at each entry.
struct Refusal {
  PyObject* type;
  std::string text;
};

[[noreturn]] void refuse(const std::string& text) { throw Refusal{PyExc_ValueError, text}; }

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw Refusal{PyExc_TypeError, std::string(what) + " must be a torch.Tensor"};
  return THPVariable_Unpack(o);
}

const at::Tensor* maybe(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }

int64_t integer(PyObject* o, const char* what) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refusal{PyExc_TypeError, std::string(what) + " must be an integer"};
  }
  return v;
}

double real(PyObject* o, const char* what) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refusal{PyExc_TypeError, std::string(what) + " must be a number"};
  }
  return v;
}

const char* name_of(at::ScalarType t) { return c10::toString(t); }

void typed(const at::Tensor& t, at::ScalarType type, const char* what) {
  if (t.scalar_type() != type)
    refuse(std::string(what) + " must have dtype " + name_of(type) + ", got " + name_of(t.scalar_type()));
}

// The device all tensors of a call share: a kernel reads and writes only memory
// of the device it runs on.
struct Device {
  int index;

  Device(const at::Tensor& t, const char* what) : index(-1) {
    if (!t.is_cuda()) refuse(std::string(what) + " must be a device tensor");
    index = t.get_device();
  }
  void holds(const at::Tensor& t, const char* what) const {
    if (!t.is_cuda()) refuse(std::string(what) + " must be a device tensor");
    if (t.get_device() != index)
      refuse(std::string(what) + " is on " + t.device().str() + ", the other tensors on cuda:" + std::to_string(index));
  }
  // The address of a contiguous tensor of this type and size; nullptr for None.
  template <class T>
  T* plain(const at::Tensor* t, at::ScalarType type, int64_t numel, const char* what) const {
    if (!t) return nullptr;
    holds(*t, what);
    typed(*t, type, what);
    if (t->numel() != numel || !t->is_contiguous())
      refuse(std::string(what) + " must be contiguous with " + std::to_string(numel) + " elements");
    return static_cast<T*>(t->data_ptr());
  }
  // A [tokens, heads, head_dim] tensor: its address, and its strides.
  void* rows(const at::Tensor& t, at::ScalarType type, int64_t tokens, int64_t heads, int64_t dim, const char* what,
             int64_t* token_stride, int64_t* head_stride) const {
    holds(t, what);
    typed(t, type, what);
    if (t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads || t.size(2) != dim)
      refuse(std::string(what) + " must be [" + std::to_string(tokens) + ", " + std::to_string(heads) + ", " +
             std::to_string(dim) + "]");
    if (t.stride(2) != 1) refuse(std::string(what) + " must have contiguous components");
    *token_stride = t.stride(0);
    *head_stride = t.stride(1);
    return t.data_ptr();
  }
  // Run a call with this device current, on its current stream.
  template <class Call>
  int launch(Call call) const {
    const c10::hip::OptionalHIPGuard guard(c10::hip::current_device() == index
                                               ? std::optional<c10::DeviceIndex>()
                                               : std::optional<c10::DeviceIndex>(c10::DeviceIndex(index)));
    void* stream = c10::hip::getCurrentHIPStream(c10::DeviceIndex(index)).stream();
    return call(stream);
  }
};

// TQ2_TYPE_* of a dtype, or -1, which the entry points refuse.
int64_t type_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return TQ2_TYPE_F32;
    case at::kHalf: return TQ2_TYPE_F16;
    case at::kBFloat16: return TQ2_TYPE_BF16;
    case at::kFloat8_e4m3fn: return TQ2_TYPE_E4M3;
    default: return -1;
  }
}

// The cache and the new tokens' place in it.  args: k_cache, v_cache, kv_len,
// table, cu_q, k_scale, v_scale.
tq2_paged_cache cache_of(const Device& dev, PyObject* const* args, at::ScalarType act, int64_t tokens,
                         int64_t q_heads, int64_t dim) {
  const at::Tensor &k = tensor(args[0], "k_cache"), &v = tensor(args[1], "v_cache");
  const at::Tensor &lens = tensor(args[2], "kv_len"), &table = tensor(args[3], "table");
  if (k.dim() != 4 || v.sizes() != k.sizes())
    refuse("k_cache and v_cache must be [pages, kv_heads, page, head_dim]");
  if (k.size(3) != dim) refuse("head_dim is " + std::to_string(dim) + ", that of the cache " + std::to_string(k.size(3)));
  const at::ScalarType kind = k.scalar_type();
  if (v.scalar_type() != kind || (kind != at::kHalf && kind != at::kBFloat16 && kind != at::kFloat8_e4m3fn))
    refuse("k_cache and v_cache must have one dtype of float16, bfloat16 and float8_e4m3fn");
  dev.holds(k, "k_cache");
  dev.holds(v, "v_cache");
  dev.holds(table, "table");
  if (k.stride(3) != 1 || v.stride(3) != 1) refuse("k_cache and v_cache must have contiguous components");
  if (table.dim() != 2 || table.scalar_type() != at::kInt || (table.size(1) > 1 && table.stride(1) != 1))
    refuse("table must be an int32 matrix with contiguous rows");
  tq2_paged_cache c;
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.kv_heads = k.size(1);
  c.batch = table.size(0);
  c.k_scale = dev.plain<const float>(maybe(args[5], "k_scale"), at::kFloat, c.kv_heads, "k_scale");
  c.v_scale = dev.plain<const float>(maybe(args[6], "v_scale"), at::kFloat, c.kv_heads, "v_scale");
  c.table = static_cast<const int32_t*>(table.data_ptr());
  c.kv_len = dev.plain<const int32_t>(&lens, at::kInt, c.batch, "kv_len");
  c.cu_q = dev.plain<const int32_t>(maybe(args[4], "cu_q"), at::kInt, c.batch + 1, "cu_q");
  c.tokens = tokens;
  c.pages = k.size(0);
  c.page = k.size(2);
  c.table_cols = table.size(1);
  c.table_stride = table.stride(0);
  c.q_heads = q_heads;
  c.head_dim = dim;
  c.act_type = type_of(act);
  c.cache_type = type_of(kind);
  c.k_page_stride = k.stride(0);
  c.k_head_stride = k.stride(1);
  c.k_token_stride = k.stride(2);
  c.v_page_stride = v.stride(0);
  c.v_head_stride = v.stride(1);
  c.v_token_stride = v.stride(2);
  return c;
}

PyObject* new_ref(PyObject* o) {
  Py_INCREF(o);
  return o;
}

PyObject* status_or(int status, PyObject* out) {
  if (status == TQ2_OK) return out;
  Py_DECREF(out);
  return PyLong_FromLong(status);
}

PyObject* kv_append(PyObject* const* args) {
  const at::Tensor &k = tensor(args[0], "k"), &v = tensor(args[1], "v");
  const at::Tensor* q = maybe(args[9], "q");
  const at::Tensor* q_out = maybe(args[10], "q_out");
  if (k.dim() != 3) refuse("k must be [tokens, kv_heads, head_dim]");
  const Device dev(k, "k");
  const at::ScalarType act = k.scalar_type();
  const int64_t tokens = k.size(0), kv_heads = k.size(1), dim = k.size(2);
  tq2_kv_append_args a{};
  if (q && q->dim() != 3) refuse("q must be [tokens, q_heads, head_dim]");
  if (q_out && !q) refuse("q_out without q");
  const int64_t q_heads = q ? q->size(1) : kv_heads;
  a.cache = cache_of(dev, args + 2, act, tokens, q_heads, dim);
  if (a.cache.kv_heads != kv_heads) refuse("k must have " + std::to_string(a.cache.kv_heads) + " heads for this cache");
  a.k = dev.rows(k, act, tokens, kv_heads, dim, "k", &a.k_token_stride, &a.k_head_stride);
  a.v = dev.rows(v, act, tokens, kv_heads, dim, "v", &a.v_token_stride, &a.v_head_stride);
  at::Tensor made;
  if (q) {
    a.q = dev.rows(*q, act, tokens, q_heads, dim, "q", &a.q_token_stride, &a.q_head_stride);
    if (!q_out) {
      made = at::empty(q->sizes(), q->options());
      q_out = &made;
    }
    a.q_out = dev.rows(*q_out, act, tokens, q_heads, dim, "q_out", &a.q_out_token_stride, &a.q_out_head_stride);
  }
  const at::Tensor* freqs = maybe(args[11], "freqs");
  const at::Tensor* positions = maybe(args[12], "positions");
  const int64_t half = freqs ? freqs->numel() : 0;
  a.rot = 2 * half;
  a.axes = positions && positions->dim() == 2 ? positions->size(0) : 1;
  a.section[0] = half;
  if (args[13] != Py_None) {
    const Py_ssize_t n = PySequence_Size(args[13]);
    if (n < 0) {
      PyErr_Clear();
      throw Refusal{PyExc_TypeError, "sections must be a sequence of integers"};
    }
    if (n != a.axes || n > 3) refuse("positions must be [tokens] or [axes, tokens], with one section for each of at most 3 axes");
    for (Py_ssize_t i = 0; i < n; ++i) {
      PyObject* item = PySequence_GetItem(args[13], i);
      if (!item) {
        PyErr_Clear();
        throw Refusal{PyExc_TypeError, "sections must be a sequence of integers"};
      }
      const long long width = PyLong_AsLongLong(item);
      Py_DECREF(item);
      if (width == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refusal{PyExc_TypeError, "sections must be a sequence of integers"};
      }
      a.section[i] = width;
    }
  } else if (a.axes != 1) {
    refuse("positions must be [tokens] or [axes, tokens], with one section for each of at most 3 axes");
  }
  const int truth = PyObject_IsTrue(args[14]);
  if (truth < 0) {
    PyErr_Clear();
    throw Refusal{PyExc_TypeError, "interleaved must be a truth value"};
  }
  a.interleaved = truth;
  a.freqs = dev.plain<const double>(freqs, at::kDouble, half, "freqs");
  a.positions = dev.plain<const int32_t>(positions, at::kInt, a.axes * tokens, "positions");
  a.q_norm = dev.plain<const float>(maybe(args[15], "q_norm"), at::kFloat, dim, "q_norm");
  a.k_norm = dev.plain<const float>(maybe(args[16], "k_norm"), at::kFloat, dim, "k_norm");
  a.eps = real(args[17], "eps");
  const int status = dev.launch([&](void* stream) { return tq2_kv_append(&a, stream); });
  if (status != TQ2_OK || !q) return status_or(status, new_ref(Py_None));
  return made.defined() ? THPVariable_Wrap(made) : new_ref(args[10]);
}

PyObject* paged_attention(PyObject* const* args) {
  const at::Tensor& q = tensor(args[0], "q");
  if (q.dim() != 3) refuse("q must be [tokens, q_heads, head_dim]");
  const Device dev(q, "q");
  const at::ScalarType act = q.scalar_type();
  const int64_t tokens = q.size(0), q_heads = q.size(1), dim = q.size(2);
  tq2_paged_attention_args a{};
  a.cache = cache_of(dev, args + 1, act, tokens, q_heads, dim);
  a.q = dev.rows(q, act, tokens, q_heads, dim, "q", &a.q_token_stride, &a.q_head_stride);
  a.max_q = args[8] != Py_None ? integer(args[8], "max_q") : (a.cache.cu_q ? tokens : 1);
  const int64_t room = a.cache.table_cols * a.cache.page;
  a.max_kv = args[9] != Py_None ? integer(args[9], "max_kv") : (room < INT32_MAX ? room : INT32_MAX);
  a.window = integer(args[10], "window");
  a.scale = args[11] != Py_None ? real(args[11], "scale") : 1.0 / std::sqrt(double(dim));
  const at::Tensor* out = maybe(args[12], "out");
  at::Tensor made, workspace;
  if (!out) {
    made = at::empty(q.sizes(), q.options());
    out = &made;
  }
  a.out = dev.rows(*out, act, tokens, q_heads, dim, "out", &a.out_token_stride, &a.out_head_stride);
  a.workspace_bytes = int64_t(tq2_paged_attention_workspace_bytes(&a));
  if (a.workspace_bytes > 0) {
    workspace = at::empty({a.workspace_bytes}, q.options().dtype(at::kByte));
    a.workspace = workspace.data_ptr();
  }
  const int status = dev.launch([&](void* stream) { return tq2_paged_attention(&a, stream); });
  if (status != TQ2_OK) return PyLong_FromLong(status);
  return made.defined() ? THPVariable_Wrap(made) : new_ref(args[12]);
}

PyObject* q4_gemv(PyObject* const* args) {
  const at::Tensor &codes = tensor(args[0], "codes"), &scales = tensor(args[1], "scales"), &x = tensor(args[2], "x");
  if (codes.dim() != 2 || scales.dim() != 2 || (x.dim() != 1 && x.dim() != 2))
    refuse("codes and scales must be matrices, x a matrix or a vector");
  const int64_t n = codes.size(0), k = 2 * codes.size(1), m = x.dim() == 2 ? x.size(0) : 1, per_row = scales.size(1);
  const int64_t group = per_row > 0 && k % per_row == 0 ? k / per_row : 0;
  if (group != 32 && group != 64 && group != 128)
    refuse("scales must be [n, k / group] with a group of 32, 64 or 128");
  const Device dev(x, "x");
  const auto* cp = dev.plain<const void>(&codes, at::kByte, n * k / 2, "codes");
  const auto* sp = dev.plain<const void>(&scales, at::kHalf, n * per_row, "scales");
  const float* xp = dev.plain<const float>(&x, at::kFloat, m * k, "x");
  const float* rp = dev.plain<const float>(maybe(args[3], "residual"), at::kFloat, m * n, "residual");
  const at::Tensor* out = maybe(args[4], "out");
  at::Tensor made;
  if (!out) {
    made = x.dim() == 2 ? at::empty({m, n}, x.options()) : at::empty({n}, x.options());
    out = &made;
  }
  float* op = dev.plain<float>(out, at::kFloat, m * n, "out");
  const int status =
      dev.launch([&](void* stream) { return tq2_q4_gemv(cp, sp, xp, rp, op, m, n, k, int(group), stream); });
  if (status != TQ2_OK) return PyLong_FromLong(status);
  return made.defined() ? THPVariable_Wrap(made) : new_ref(args[4]);
}

// A contiguous matrix of activations: its address.
void* matrix(const Device& dev, const at::Tensor& t, at::ScalarType type, int64_t rows, int64_t cols, const char* what) {
  return dev.plain<void>(&t, type, rows * cols, what);
}

int64_t act_type_of(const at::Tensor& t, const char* what) {
  const at::ScalarType k = t.scalar_type();
  if (k != at::kFloat && k != at::kHalf && k != at::kBFloat16)
    refuse(std::string(what) + " must have dtype Float, Half or BFloat16, got " + name_of(k));
  return type_of(k);
}

PyObject* moe_route(PyObject* const* args) {
  const at::Tensor &x = tensor(args[0], "x"), &w = tensor(args[1], "weight");
  if (x.dim() != 2 || w.dim() != 2 || w.size(1) != x.size(1))
    refuse("x must be [tokens, hidden] and weight [experts, hidden]");
  const Device dev(x, "x");
  tq2_moe_route_args a{};
  a.tokens = x.size(0);
  a.hidden = x.size(1);
  a.experts = w.size(0);
  a.top_k = integer(args[2], "top_k");
  a.act_type = act_type_of(x, "x");
  a.weight_type = act_type_of(w, "weight");
  a.x = matrix(dev, x, x.scalar_type(), a.tokens, a.hidden, "x");
  a.weight = matrix(dev, w, w.scalar_type(), a.experts, a.hidden, "weight");
  a.bias = dev.plain<const float>(maybe(args[3], "bias"), at::kFloat, a.experts, "bias");
  a.scoring = integer(args[4], "scoring");
  a.renormalize = args[5] == Py_True;
  a.scale = real(args[6], "scale");
  const at::Tensor *weights = maybe(args[7], "weights"), *ids = maybe(args[8], "ids");
  // The entry point refuses these sizes; no tensor is made for them.
  if (a.top_k < 1 || a.top_k > a.experts) return PyLong_FromLong(TQ2_ERR_INVALID);
  at::Tensor made_weights, made_ids;
  if (!weights) {
    made_weights = at::empty({a.tokens, a.top_k}, x.options().dtype(at::kFloat));
    weights = &made_weights;
  }
  if (!ids) {
    made_ids = at::empty({a.tokens, a.top_k}, x.options().dtype(at::kInt));
    ids = &made_ids;
  }
  a.weights = dev.plain<float>(weights, at::kFloat, a.tokens * a.top_k, "weights");
  a.ids = dev.plain<int32_t>(ids, at::kInt, a.tokens * a.top_k, "ids");
  a.workspace_bytes = int64_t(tq2_moe_route_workspace_bytes(&a));
  at::Tensor workspace;
  if (a.workspace_bytes > 0) {
    workspace = at::empty({a.workspace_bytes}, x.options().dtype(at::kByte));
    a.workspace = workspace.data_ptr();
  }
  const int status = dev.launch([&](void* stream) { return tq2_moe_route(&a, stream); });
  if (status != TQ2_OK) return PyLong_FromLong(status);
  PyObject* first = made_weights.defined() ? THPVariable_Wrap(made_weights) : new_ref(args[7]);
  PyObject* second = made_ids.defined() ? THPVariable_Wrap(made_ids) : new_ref(args[8]);
  PyObject* both = PyTuple_Pack(2, first, second);
  Py_DECREF(first);
  Py_DECREF(second);
  return both;
}

// The experts' rows of one projection: 4-bit codes and scales, or a ternary weight.
struct Projection {
  const void* codes;
  const void* scales;
};

Projection projection(const Device& dev, PyObject* codes_arg, PyObject* scales_arg, int64_t experts, int64_t n,
                      int64_t k, int64_t group, const std::string& what) {
  const at::Tensor& codes = tensor(codes_arg, what.c_str());
  const at::Tensor* scales = maybe(scales_arg, (what + "'s scales").c_str());
  if (!scales)
    return {dev.plain<const void>(&codes, at::kByte, int64_t(tq2_soa_bytes(experts * n, k)), what.c_str()), nullptr};
  if (codes.dim() != 3 || codes.size(0) != experts || codes.size(1) != n || codes.size(2) * 2 != k)
    refuse(what + "'s codes must be [" + std::to_string(experts) + ", " + std::to_string(n) + ", " +
           std::to_string(k / 2) + "]");
  if (scales->dim() != 3 || scales->size(0) != experts || scales->size(1) != n || scales->size(2) * group != k)
    refuse(what + "'s scales must be [" + std::to_string(experts) + ", " + std::to_string(n) + ", " +
           std::to_string(k) + " / group], of one group for gate_up and down");
  return {dev.plain<const void>(&codes, at::kByte, codes.numel(), (what + "'s codes").c_str()),
          dev.plain<const void>(scales, at::kHalf, scales->numel(), (what + "'s scales").c_str())};
}

PyObject* moe_experts(PyObject* const* args) {
  const at::Tensor &x = tensor(args[0], "x"), &gate_up = tensor(args[1], "gate_up");
  const at::Tensor &ids = tensor(args[5], "ids"), &weights = tensor(args[6], "weights");
  const at::Tensor *up_scales = maybe(args[2], "gate_up's scales"), *down_scales = maybe(args[4], "down's scales");
  if (x.dim() != 2 || ids.dim() != 2 || ids.size(0) != x.size(0) || weights.sizes() != ids.sizes())
    refuse("x must be [tokens, hidden], ids and weights [tokens, top_k]");
  if ((up_scales != nullptr) != (down_scales != nullptr)) refuse("gate_up and down must have one format");
  const Device dev(x, "x");
  tq2_moe_experts_args a{};
  a.tokens = x.size(0);
  a.hidden = x.size(1);
  a.top_k = ids.size(1);
  a.act_type = act_type_of(x, "x");
  if (up_scales) {
    a.format = TQ2_MOE_Q4;
    if (gate_up.dim() != 3 || up_scales->dim() != 3 || up_scales->size(2) < 1 || a.hidden % up_scales->size(2))
      refuse("gate_up must be codes [experts, 2 * inter, hidden / 2] and scales [experts, 2 * inter, hidden / group]");
    a.experts = gate_up.size(0);
    a.inter = gate_up.size(1) / 2;
    a.group = a.hidden / up_scales->size(2);
    if (args[7] != Py_None && integer(args[7], "experts") != a.experts)
      refuse("experts is not what gate_up has");
  } else {
    a.format = TQ2_MOE_TERNARY;
    a.group = 128;
    if (args[7] == Py_None) refuse("ternary weights need experts");
    a.experts = integer(args[7], "experts");
    const at::Tensor& down = tensor(args[3], "down");
    // 17 bytes hold 64 weights: down tells inter.
    const int64_t row = a.experts > 0 ? a.experts * a.hidden * 17 : 0;
    a.inter = row > 0 ? down.numel() * 64 / row : 0;
  }
  // The entry point refuses these sizes before any pointer; the shapes of weights are not compared for them.
  if (a.tokens > TQ2_MOE_MAX_TOKENS || a.experts < 1 || a.experts > TQ2_MOE_MAX_EXPERTS || a.hidden < 1 ||
      a.hidden > TQ2_MOE_MAX_DIM || a.inter < 1 || a.inter > TQ2_MOE_MAX_DIM || a.hidden % 128 || a.inter % 128) {
    if (a.format == TQ2_MOE_TERNARY && a.experts >= 1 && a.hidden % 128 == 0 && a.inter % 128)
      refuse("down is not a ternary weight of experts * hidden rows");
    return PyLong_FromLong(tq2_moe_experts(&a, nullptr));
  }
  const Projection up = projection(dev, args[1], args[2], a.experts, 2 * a.inter, a.hidden, a.group, "gate_up");
  const Projection down = projection(dev, args[3], args[4], a.experts, a.hidden, a.inter, a.group, "down");
  a.gate_up = up.codes;
  a.gate_up_scales = up.scales;
  a.down = down.codes;
  a.down_scales = down.scales;
  a.x = matrix(dev, x, x.scalar_type(), a.tokens, a.hidden, "x");
  const at::Tensor* residual = maybe(args[8], "residual");
  if (residual) a.residual = matrix(dev, *residual, x.scalar_type(), a.tokens, a.hidden, "residual");
  a.ids = dev.plain<const int32_t>(&ids, at::kInt, a.tokens * a.top_k, "ids");
  a.weights = dev.plain<const float>(&weights, at::kFloat, a.tokens * a.top_k, "weights");
  const at::Tensor* out = maybe(args[9], "out");
  at::Tensor made, workspace;
  if (!out) {
    made = at::empty(x.sizes(), x.options());
    out = &made;
  }
  a.out = matrix(dev, *out, x.scalar_type(), a.tokens, a.hidden, "out");
  a.workspace_bytes = int64_t(tq2_moe_experts_workspace_bytes(&a));
  if (a.workspace_bytes > 0) {
    workspace = at::empty({a.workspace_bytes}, x.options().dtype(at::kByte));
    a.workspace = workspace.data_ptr();
  }
  const int status = dev.launch([&](void* stream) { return tq2_moe_experts(&a, stream); });
  if (status != TQ2_OK) return PyLong_FromLong(status);
  return made.defined() ? THPVariable_Wrap(made) : new_ref(args[9]);
}

// A setting of a row: a number for all rows, or a tensor of one for each.
template <class T>
const T* setting(const Device& dev, PyObject* o, at::ScalarType type, int64_t rows, const char* what) {
  return THPVariable_Check(o) ? dev.plain<const T>(&THPVariable_Unpack(o), type, rows, what) : nullptr;
}

PyObject* sample(PyObject* const* args) {
  const at::Tensor &logits = tensor(args[0], "logits"), &u = tensor(args[1], "u");
  if (logits.dim() != 2) refuse("logits must be [rows, vocab]");
  const Device dev(logits, "logits");
  tq2_sample_args a{};
  a.rows = logits.size(0);
  a.vocab = logits.size(1);
  a.row_stride = a.rows > 1 ? logits.stride(0) : a.vocab;
  if (a.vocab > 1 && logits.stride(1) != 1) refuse("logits must have contiguous rows");
  a.logits_type = act_type_of(logits, "logits");
  a.logits = logits.data_ptr();
  a.u = dev.plain<const float>(&u, at::kFloat, a.rows, "u");
  a.temperatures = setting<float>(dev, args[2], at::kFloat, a.rows, "temperature");
  if (!a.temperatures) a.temperature = real(args[2], "temperature");
  a.top_ks = setting<int32_t>(dev, args[3], at::kInt, a.rows, "top_k");
  if (!a.top_ks) a.top_k = integer(args[3], "top_k");
  a.top_ps = setting<float>(dev, args[4], at::kFloat, a.rows, "top_p");
  if (!a.top_ps) a.top_p = real(args[4], "top_p");
  a.min_ps = setting<float>(dev, args[5], at::kFloat, a.rows, "min_p");
  if (!a.min_ps) a.min_p = real(args[5], "min_p");
  const at::Tensor* out = maybe(args[6], "out");
  at::Tensor made, workspace;
  if (!out) {
    made = at::empty({a.rows}, logits.options().dtype(at::kInt));
    out = &made;
  }
  a.ids = dev.plain<int32_t>(out, at::kInt, a.rows, "out");
  a.logprob = dev.plain<float>(maybe(args[7], "logprob"), at::kFloat, a.rows, "logprob");
  a.workspace_bytes = int64_t(tq2_sample_workspace_bytes(&a));
  if (a.workspace_bytes > 0) {
    workspace = at::empty({a.workspace_bytes}, logits.options().dtype(at::kByte));
    a.workspace = workspace.data_ptr();
  }
  const int status = dev.launch([&](void* stream) { return tq2_sample(&a, stream); });
  if (status != TQ2_OK) return PyLong_FromLong(status);
  return made.defined() ? THPVariable_Wrap(made) : new_ref(args[6]);
}

// An entry with `count` positional arguments; no C++ exception leaves it.
template <PyObject* (*body)(PyObject* const*), int count>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != count) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", count, n);
    return nullptr;
  }
  try {
    return body(args);
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    PyErr_Clear();
    PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

PyMethodDef methods[] = {
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<kv_append, 18>)), METH_FASTCALL,
     "k, v, k_cache, v_cache, kv_len, table, cu_q, k_scale, v_scale, q, q_out, freqs, positions, sections, "
     "interleaved, q_norm, k_norm, eps -> q_out, or a status"},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<paged_attention, 13>)),
     METH_FASTCALL,
     "q, k_cache, v_cache, kv_len, table, cu_q, k_scale, v_scale, max_q, max_kv, window, scale, out -> out, or a "
     "status"},
    {"q4_gemv", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<q4_gemv, 5>)), METH_FASTCALL,
     "codes, scales, x, residual, out -> out, or a status"},
    {"moe_route", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<moe_route, 9>)), METH_FASTCALL,
     "x, weight, top_k, bias, scoring, renormalize, scale, weights, ids -> (weights, ids), or a status"},
    {"moe_experts", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<moe_experts, 10>)), METH_FASTCALL,
     "x, gate_up, its scales, down, its scales, ids, weights, experts, residual, out -> out, or a status"},
    {"sample", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<sample, 8>)), METH_FASTCALL,
     "logits, u, temperature, top_k, top_p, min_p, out, logprob -> out, or a status"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
