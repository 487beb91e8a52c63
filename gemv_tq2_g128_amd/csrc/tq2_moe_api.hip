// C ABI of the mixture-of-experts operators (tq2_moe.h): argument checks, device check, launch.  Same error policy as
// tq2_api.hip: every failure is a status.
#include "tq2_host.h"
#include "tq2_internal.h"
#include "tq2_moe_internal.h"

#include <cmath>

namespace {

using tq2::aligned;
using tq2::check_device;
using tq2::launch_status;
using tq2::overlaps;

bool size_ok(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }
bool float_type(int64_t t) { return t == TQ2_TYPE_F32 || t == TQ2_TYPE_F16 || t == TQ2_TYPE_BF16; }
size_t bytes_of(int64_t type) { return type == TQ2_TYPE_F32 ? 4 : 2; }

int check_route_sizes(const tq2_moe_route_args& a) {
  if (!size_ok(a.tokens, 0, TQ2_MOE_MAX_ROUTE_TOKENS) || !size_ok(a.hidden, 1, TQ2_MOE_MAX_DIM) ||
      !size_ok(a.top_k, 1, TQ2_MOE_MAX_TOP_K) || !size_ok(a.experts, a.top_k, TQ2_MOE_MAX_EXPERTS))
    return TQ2_ERR_INVALID;
  if (!float_type(a.act_type) || !float_type(a.weight_type)) return TQ2_ERR_INVALID;
  if (a.scoring != TQ2_MOE_SOFTMAX && a.scoring != TQ2_MOE_SIGMOID) return TQ2_ERR_INVALID;
  if (a.hidden % 8) return TQ2_ERR_SHAPE;
  return TQ2_OK;
}

size_t route_workspace(const tq2_moe_route_args& a) {
  return size_t(tq2::route_parts(a.tokens, a.experts, a.hidden)) * size_t(a.tokens) * size_t(a.experts) * 8;
}

int check_experts_sizes(const tq2_moe_experts_args& a) {
  if (!size_ok(a.tokens, 0, TQ2_MOE_MAX_TOKENS) || !size_ok(a.top_k, 1, TQ2_MOE_MAX_TOP_K) ||
      !size_ok(a.experts, 1, TQ2_MOE_MAX_EXPERTS) || !size_ok(a.hidden, 1, TQ2_MOE_MAX_DIM) ||
      !size_ok(a.inter, 1, TQ2_MOE_MAX_DIM))
    return TQ2_ERR_INVALID;
  if (!float_type(a.act_type)) return TQ2_ERR_INVALID;
  if (a.format == TQ2_MOE_TERNARY) {
    if (a.group != 128) return TQ2_ERR_INVALID;
  } else if (a.format != TQ2_MOE_Q4 || (a.group != 32 && a.group != 64 && a.group != 128)) {
    return TQ2_ERR_INVALID;
  }
  if (a.hidden % 128 || a.inter % 128) return TQ2_ERR_SHAPE;
  return TQ2_OK;
}

}  // namespace

extern "C" {

size_t tq2_moe_route_workspace_bytes(const tq2_moe_route_args* args) {
  if (!args || check_route_sizes(*args) != TQ2_OK || args->tokens == 0) return 0;
  return route_workspace(*args);
}

int tq2_moe_route(const tq2_moe_route_args* args, void* stream) {
  if (!args) return TQ2_ERR_INVALID;
  const tq2_moe_route_args& a = *args;
  int st = check_route_sizes(a);
  if (st != TQ2_OK) return st;
  if (!std::isfinite(a.scale)) return TQ2_ERR_INVALID;
  if (a.tokens == 0) return TQ2_OK;
  const size_t need = route_workspace(a);
  if (!a.x || !a.weight || !a.weights || !a.ids || !a.workspace || a.workspace_bytes < 0 ||
      size_t(a.workspace_bytes) < need)
    return TQ2_ERR_INVALID;
  if (!aligned(a.x, 16) || !aligned(a.weight, 16) || !aligned(a.workspace, 16) || !aligned(a.bias, 4) ||
      !aligned(a.weights, 4) || !aligned(a.ids, 4))
    return TQ2_ERR_ALIGN;
  struct {
    const void* p;
    size_t n;
  } in[] = {{a.x, size_t(a.tokens) * a.hidden * bytes_of(a.act_type)},
            {a.weight, size_t(a.experts) * a.hidden * bytes_of(a.weight_type)},
            {a.bias, size_t(a.experts) * 4}};
  const size_t chosen = size_t(a.tokens) * a.top_k * 4;
  for (const auto& i : in)
    if (overlaps(a.weights, chosen, i.p, i.n) || overlaps(a.ids, chosen, i.p, i.n) ||
        overlaps(a.workspace, need, i.p, i.n))
      return TQ2_ERR_ALIAS;
  if (overlaps(a.weights, chosen, a.ids, chosen) || overlaps(a.workspace, need, a.weights, chosen) ||
      overlaps(a.workspace, need, a.ids, chosen))
    return TQ2_ERR_ALIAS;
  st = check_device();
  if (st != TQ2_OK) return st;
  return launch_status(tq2::launch_moe_route(a, static_cast<hipStream_t>(stream)));
}

size_t tq2_moe_experts_workspace_bytes(const tq2_moe_experts_args* args) {
  if (!args || check_experts_sizes(*args) != TQ2_OK || args->tokens == 0) return 0;
  return tq2::plan_moe(*args).workspace;
}

int tq2_moe_experts(const tq2_moe_experts_args* args, void* stream) {
  if (!args) return TQ2_ERR_INVALID;
  const tq2_moe_experts_args& a = *args;
  int st = check_experts_sizes(a);
  if (st != TQ2_OK) return st;
  if (a.tokens == 0) return TQ2_OK;
  const bool q4 = a.format == TQ2_MOE_Q4;
  const tq2::MoePlan plan = tq2::plan_moe(a);
  if (!a.x || !a.out || !a.ids || !a.weights || !a.gate_up || !a.down || q4 != (a.gate_up_scales != nullptr) ||
      q4 != (a.down_scales != nullptr) || !a.workspace || a.workspace_bytes < 0 ||
      size_t(a.workspace_bytes) < plan.workspace)
    return TQ2_ERR_INVALID;
  if (!aligned(a.x, 16) || !aligned(a.residual, 16) || !aligned(a.out, 16) || !aligned(a.gate_up, 16) ||
      !aligned(a.gate_up_scales, 16) || !aligned(a.down, 16) || !aligned(a.down_scales, 16) ||
      !aligned(a.workspace, 16) || !aligned(a.ids, 4) || !aligned(a.weights, 4))
    return TQ2_ERR_ALIGN;
  const size_t rows = size_t(a.tokens) * a.hidden * bytes_of(a.act_type), pairs = size_t(a.tokens) * a.top_k * 4;
  const int64_t up_rows = 2 * a.experts * a.inter, down_rows = a.experts * a.hidden;
  const auto weight_bytes = [&](int64_t n, int64_t k) {
    return q4 ? size_t(n) * size_t(k / 2) : tq2::soa_bytes(n, k);
  };
  const auto scale_bytes = [&](int64_t n, int64_t k) { return size_t(n) * size_t(k / a.group) * 2; };
  struct {
    const void* p;
    size_t n;
  } in[] = {{a.gate_up, weight_bytes(up_rows, a.hidden)},
            {a.gate_up_scales, scale_bytes(up_rows, a.hidden)},
            {a.down, weight_bytes(down_rows, a.inter)},
            {a.down_scales, scale_bytes(down_rows, a.inter)},
            {a.ids, pairs},
            {a.weights, pairs}};
  for (const auto& i : in)
    if (overlaps(a.out, rows, i.p, i.n) || overlaps(a.workspace, plan.workspace, i.p, i.n)) return TQ2_ERR_ALIAS;
  for (const void* p : {a.x, a.residual})
    if ((p != a.out && overlaps(a.out, rows, p, rows)) || overlaps(a.workspace, plan.workspace, p, rows))
      return TQ2_ERR_ALIAS;
  if (overlaps(a.workspace, plan.workspace, a.out, rows)) return TQ2_ERR_ALIAS;
  st = check_device();
  if (st != TQ2_OK) return st;
  return launch_status(tq2::launch_moe_experts(a, plan, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
