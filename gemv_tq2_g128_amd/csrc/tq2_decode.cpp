// Python module `_decode`: the calls of tq2_moe.h and tq2_sample.h on tensors (tq2_binding.h).
#include "tq2_binding.h"

#include "tq2_moe.h"
#include "tq2_sample.h"

namespace {

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

PyMethodDef methods[] = {
    {"moe_route", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<moe_route, 9>)), METH_FASTCALL,
     "x, weight, top_k, bias, scoring, renormalize, scale, weights, ids -> (weights, ids), or a status"},
    {"moe_experts", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<moe_experts, 10>)), METH_FASTCALL,
     "x, gate_up, its scales, down, its scales, ids, weights, experts, residual, out -> out, or a status"},
    {"sample", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<sample, 8>)), METH_FASTCALL,
     "logits, u, temperature, top_k, top_p, min_p, out, logprob -> out, or a status"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decode", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode(void) { return PyModule_Create(&module); }
