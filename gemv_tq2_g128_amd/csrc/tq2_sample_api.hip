// C ABI of the token choice (tq2_sample.h): argument checks, device check, launch.  Same error policy as tq2_api.hip:
// every failure is a status.
#include "tq2_host.h"
#include "tq2_sample_internal.h"

namespace {

using tq2::aligned;
using tq2::check_device;
using tq2::launch_status;
using tq2::overlaps;

bool size_ok(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

int check_sizes(const tq2_sample_args& a) {
  if (!size_ok(a.rows, 0, TQ2_SAMPLE_MAX_ROWS) || !size_ok(a.vocab, 1, TQ2_SAMPLE_MAX_VOCAB)) return TQ2_ERR_INVALID;
  if (a.logits_type != TQ2_TYPE_F32 && a.logits_type != TQ2_TYPE_F16 && a.logits_type != TQ2_TYPE_BF16)
    return TQ2_ERR_INVALID;
  if (a.rows > 1 && !size_ok(a.row_stride, 0, int64_t(1) << 40)) return TQ2_ERR_INVALID;
  return TQ2_OK;
}

}  // namespace

extern "C" {

size_t tq2_sample_workspace_bytes(const tq2_sample_args* args) {
  if (!args || check_sizes(*args) != TQ2_OK || args->rows == 0) return 0;
  return tq2::sample_workspace(args->rows, args->vocab, args->logits_type);
}

int tq2_sample(const tq2_sample_args* args, void* stream) {
  if (!args) return TQ2_ERR_INVALID;
  const tq2_sample_args& a = *args;
  int st = check_sizes(a);
  if (st != TQ2_OK) return st;
  if ((!a.temperatures && !(a.temperature >= 0.0)) || (!a.top_ps && a.top_p != a.top_p) ||
      (!a.min_ps && a.min_p != a.min_p))
    return TQ2_ERR_INVALID;
  if (a.rows == 0) return TQ2_OK;
  const size_t need = tq2::sample_workspace(a.rows, a.vocab, a.logits_type);
  if (!a.logits || !a.u || !a.ids || !a.workspace || a.workspace_bytes < 0 || size_t(a.workspace_bytes) < need)
    return TQ2_ERR_INVALID;
  const size_t element = a.logits_type == TQ2_TYPE_F32 ? 4 : 2, row = size_t(a.rows) * 4;
  if (!aligned(a.logits, element) || !aligned(a.workspace, 16)) return TQ2_ERR_ALIGN;
  struct {
    const void* p;
    size_t n;
  } in[] = {{a.logits, (size_t(a.rows - 1) * size_t(a.rows > 1 ? a.row_stride : 0) + size_t(a.vocab)) * element},
            {a.u, row},
            {a.temperatures, row},
            {a.top_ks, row},
            {a.top_ps, row},
            {a.min_ps, row}};
  for (const auto& i : in)
    if (i.p != a.logits && !aligned(i.p, 4)) return TQ2_ERR_ALIGN;
  if (!aligned(a.ids, 4) || !aligned(a.logprob, 4)) return TQ2_ERR_ALIGN;
  for (const auto& i : in)
    if (overlaps(a.ids, row, i.p, i.n) || overlaps(a.logprob, row, i.p, i.n) || overlaps(a.workspace, need, i.p, i.n))
      return TQ2_ERR_ALIAS;
  if (overlaps(a.ids, row, a.logprob, row) || overlaps(a.workspace, need, a.ids, row) ||
      overlaps(a.workspace, need, a.logprob, row))
    return TQ2_ERR_ALIAS;
  st = check_device();
  if (st != TQ2_OK) return st;
  return launch_status(tq2::launch_sample(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
