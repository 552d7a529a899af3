// Selection of experts and its gradient (select.h), as C entry points.
#include "select.h"

#include <algorithm>
#include <cmath>

using namespace moe;

namespace {

moe_status check_selection(const moe_selection* s) {
  if (!s) return fail(MOE_ERR_INVALID_ARGUMENT, "selection is NULL");
  if (s->T < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "T must be >= 1 (got %d)", s->T);
  if (s->E < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "E must be >= 1 (got %d)", s->E);
  if (s->E > kSelMaxE) return fail(MOE_ERR_UNSUPPORTED, "E > %d is not supported (got %d)", kSelMaxE, s->E);
  if (s->top_k < 1 || s->top_k > s->E)
    return fail(MOE_ERR_INVALID_ARGUMENT, "top_k must be in [1, E] (got %d)", s->top_k);
  if (s->top_k > kSelMaxK) return fail(MOE_ERR_UNSUPPORTED, "top_k > %d is not supported (got %d)", kSelMaxK, s->top_k);
  if (s->scoring != MOE_SCORING_SOFTMAX && s->scoring != MOE_SCORING_SIGMOID)
    return fail(MOE_ERR_INVALID_ARGUMENT, "unknown scoring %d", s->scoring);
  if (s->n_group < 1 || s->E % s->n_group)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n_group must divide E (got %d)", s->n_group);
  if (s->n_group > kSelMaxGroups)
    return fail(MOE_ERR_UNSUPPORTED, "n_group > %d is not supported (got %d)", kSelMaxGroups, s->n_group);
  if (s->topk_group < 1 || s->topk_group > s->n_group)
    return fail(MOE_ERR_INVALID_ARGUMENT, "topk_group must be in [1, n_group] (got %d)", s->topk_group);
  const int per = s->E / s->n_group;
  if (s->group_top < 1 || s->group_top > 2 || (s->n_group > 1 && s->group_top > per))
    return fail(MOE_ERR_INVALID_ARGUMENT, "group_top must be 1 or 2 and within a group's %d experts (got %d)", per,
                s->group_top);
  if (s->top_k > s->topk_group * per)
    return fail(MOE_ERR_INVALID_ARGUMENT, "top_k is %d, the topk_group groups hold %d experts", s->top_k,
                s->topk_group * per);
  if (!std::isfinite(s->scale)) return fail(MOE_ERR_INVALID_ARGUMENT, "scale must be finite");
  return MOE_OK;
}

SelArgs sel_args(const moe_selection* s) {
  SelArgs a{};
  a.T = s->T; a.E = s->E; a.k = s->top_k;
  a.sigmoid = s->scoring == MOE_SCORING_SIGMOID;
  a.groups = s->n_group; a.keep = s->topk_group; a.top = s->group_top;
  a.renorm = s->renormalize != 0;
  a.per = s->E / s->n_group;
  a.per_inv = 1.0f / (float)a.per;
  const int lanes = s->E <= 256 ? 32 : 64, v = s->E <= 128 ? 2 : 4, in = a.per / v;
  while (s->n_group << (a.lanes_log2 + 1) <= lanes) ++a.lanes_log2;
  if (s->E <= 256 && a.per % v == 0 && in <= 32 && (in & (in - 1)) == 0) {
    a.direct = 1;
    a.lanes_log2 = 0;
    while (1 << a.lanes_log2 < in) ++a.lanes_log2;
  }
  a.tol = a.sigmoid ? 0x1p-21f : 0x1p-19f;
  a.scale = s->scale;
  return a;
}

unsigned sel_grid(long T, int cus) { return (unsigned)std::min((T + kSelWaves - 1) / kSelWaves, (long)cus * 8); }

// Experts of a token in 32 lanes, V at a time.
constexpr long kSelLaunch = 1l << 26;              // tokens of a launch (a grid has less than 2^32 threads)
template <int V>
moe_status launch_pair(SelArgs a, hipStream_t st) {
  for (long left = a.T; left > 0; left -= kSelLaunch) {
    a.T = std::min(left, kSelLaunch);
    const dim3 grid((unsigned)((a.T + 2 * kSelWaves - 1) / (2 * kSelWaves))), wg(64 * kSelWaves);
    if (a.keep < a.groups) {
      if (a.sigmoid) hipLaunchKernelGGL((k_select_pair<V, 1, 1>), grid, wg, 0, st, a);
      else hipLaunchKernelGGL((k_select_pair<V, 0, 1>), grid, wg, 0, st, a);
    } else {
      if (a.sigmoid) hipLaunchKernelGGL((k_select_pair<V, 1, 0>), grid, wg, 0, st, a);
      else hipLaunchKernelGGL((k_select_pair<V, 0, 0>), grid, wg, 0, st, a);
    }
    HIP_TRY(hipGetLastError());
    a.logits += a.T * a.E;
    a.ids += a.T * a.k;
    a.w += a.T * a.k;
  }
  return MOE_OK;
}

template <int NV>
moe_status launch_select(const SelArgs& a, int cus, hipStream_t st) {
  // (as many workgroups as fit: each wave has the bias's largest once)
  const dim3 grid(std::min(sel_grid(a.T, cus), (unsigned)cus * (NV == 16 ? 4 : 6))), wg(64 * kSelWaves);
  if (a.keep < a.groups) {
    if (a.sigmoid) hipLaunchKernelGGL((k_select<NV, 1, 1>), grid, wg, 0, st, a);
    else hipLaunchKernelGGL((k_select<NV, 0, 1>), grid, wg, 0, st, a);
  } else {
    if (a.sigmoid) hipLaunchKernelGGL((k_select<NV, 1, 0>), grid, wg, 0, st, a);
    else hipLaunchKernelGGL((k_select<NV, 0, 0>), grid, wg, 0, st, a);
  }
  HIP_TRY(hipGetLastError());
  return MOE_OK;
}

template <int SPLIT, int DENSE>
moe_status launch_bwd(const SelArgs& a, int cus, hipStream_t st) {
  const dim3 grid(sel_grid((a.T + 3) / 4, cus)), wg(64 * kSelWaves);
  if (a.E <= 256) hipLaunchKernelGGL((k_select_bwd<4, SPLIT, DENSE>), grid, wg, 0, st, a);
  else if (a.E <= 512) hipLaunchKernelGGL((k_select_bwd<8, SPLIT, DENSE>), grid, wg, 0, st, a);
  else hipLaunchKernelGGL((k_select_bwd<16, SPLIT, DENSE>), grid, wg, 0, st, a);
  HIP_TRY(hipGetLastError());
  return MOE_OK;
}

}  // namespace

namespace moe {

moe_status launch_select_bwd(const SelArgs& a, int cus, hipStream_t st) {
  if (!a.sigmoid && !a.renorm) return a.hi ? launch_bwd<1, 1>(a, cus, st) : launch_bwd<0, 1>(a, cus, st);
  return a.hi ? launch_bwd<1, 0>(a, cus, st) : launch_bwd<0, 0>(a, cus, st);
}

moe_status select_bwd_args(const moe_selection* s, const float* logits, const int32_t* topk_ids, SelArgs* out) {
  TRY(check_selection(s));
  TRY(check_ptr(logits, "logits"));
  TRY(check_ptr(topk_ids, "topk_ids"));
  *out = sel_args(s);
  out->logits = logits;
  out->ids_in = topk_ids;
  return MOE_OK;
}

}  // namespace moe

extern "C" {

moe_status moe_select_experts(const moe_selection* s, const float* logits, const float* bias, int32_t* topk_ids,
                              float* topk_weights, moe_stream_t stream) {
  TRY(check_selection(s));
  TRY(check_ptr(logits, "logits"));
  TRY(check_ptr(bias, "bias", false));
  TRY(check_ptr(topk_ids, "topk_ids"));
  TRY(check_ptr(topk_weights, "topk_weights"));
  const size_t in = (size_t)s->T * s->E * 4, out = (size_t)s->T * s->top_k * 4;
  if (overlap(logits, in, topk_ids, out) || overlap(logits, in, topk_weights, out) ||
      overlap(bias, (size_t)s->E * 4, topk_ids, out) || overlap(bias, (size_t)s->E * 4, topk_weights, out) ||
      overlap(topk_ids, out, topk_weights, out))
    return fail(MOE_ERR_INVALID_ARGUMENT, "an output overlaps an input or the other output");
  DevInfo di;
  TRY(device_info(&di));
  SelArgs a = sel_args(s);
  a.logits = logits; a.bias = bias; a.ids = topk_ids; a.w = topk_weights;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.E <= 128) return launch_pair<2>(a, st);
  if (a.E <= 256) return launch_pair<4>(a, st);
  if (a.E <= 512) return launch_select<8>(a, di.cus, st);
  return launch_select<16>(a, di.cus, st);
}

moe_status moe_select_experts_backward(const moe_selection* s, const float* logits, const int32_t* topk_ids,
                                       const float* dweights, float* dlogits, moe_stream_t stream) {
  SelArgs a;
  TRY(select_bwd_args(s, logits, topk_ids, &a));
  TRY(check_ptr(dweights, "dweights"));
  TRY(check_ptr(dlogits, "dlogits"));
  const size_t all = (size_t)s->T * s->E * 4, sel = (size_t)s->T * s->top_k * 4;
  if (overlap(dlogits, all, logits, all) || overlap(dlogits, all, topk_ids, sel) || overlap(dlogits, all, dweights, sel))
    return fail(MOE_ERR_INVALID_ARGUMENT, "dlogits overlaps an input");
  DevInfo di;
  TRY(device_info(&di));
  a.dw = dweights;
  a.dl = dlogits;
  return launch_select_bwd(a, di.cus, static_cast<hipStream_t>(stream));
}

}  // extern "C"
