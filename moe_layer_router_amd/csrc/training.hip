// The operators around the layer in a training step, as C entry points:
// layer norm in front of it (norm.h), the load-balance loss of its router
// (balance.h) and the orthogonalised update of its weights
// (orthogonalize.h).
#include "host.h"
#include "balance.h"
#include "norm.h"

#include <algorithm>

using namespace moe;

namespace {

// ----------------------------------------------------------------- layer norm
moe_status check_norm_shape(int32_t T, int32_t H) {
  if (T < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "T must be >= 1 (got %d)", T);
  if (H < 128 || H % 128) return fail(MOE_ERR_INVALID_ARGUMENT, "H must be a positive multiple of 128 (got %d)", H);
  if (H > 16384) return fail(MOE_ERR_UNSUPPORTED, "H > 16384 is not supported (got %d)", H);
  return MOE_OK;
}

// Threads of a row and chunks of 8 channels per thread: a wave per row while
// the row fits its registers (no barrier in the sums), a workgroup above.
template <int IN, int OUT, int TPR, int R>
moe_status launch_norm(const LnArgs& a, int cus, hipStream_t st) {
  constexpr int RPW = ln_threads(TPR) / TPR;
  // several rows per workgroup once every CU has 8 of them, so that gamma and
  // beta are read once for many rows
  const long rows = (a.T + RPW - 1) / RPW;
  const unsigned grid = (unsigned)std::min(rows, (long)cus * (ln_threads(TPR) > 256 ? 4 : 8));
  hipLaunchKernelGGL((k_layer_norm<IN, OUT, TPR, R>), dim3(grid), dim3(ln_threads(TPR)), 0, st, a);
  HIP_TRY(hipGetLastError());
  return MOE_OK;
}
template <int IN, int OUT>
moe_status launch_norm(const LnArgs& a, int cus, hipStream_t st) {
  if (a.H <= 512) return launch_norm<IN, OUT, 64, 1>(a, cus, st);
  if (a.H <= 1024) return launch_norm<IN, OUT, 64, 2>(a, cus, st);
  if (a.H <= 2048) return launch_norm<IN, OUT, 64, 4>(a, cus, st);
  if (a.H <= 4096) return launch_norm<IN, OUT, 256, 2>(a, cus, st);
  if (a.H <= 8192) return launch_norm<IN, OUT, 256, 4>(a, cus, st);
  return launch_norm<IN, OUT, 512, 4>(a, cus, st);
}
template <int IN>
moe_status launch_norm(const LnArgs& a, int out_dtype, int cus, hipStream_t st) {
  if (out_dtype == MOE_DTYPE_BF16) return launch_norm<IN, LN_BF16>(a, cus, st);
  if (out_dtype == MOE_DTYPE_F32) return launch_norm<IN, LN_F32>(a, cus, st);
  return launch_norm<IN, LN_FP8>(a, cus, st);
}

// The backward kernel's row layout for H: threads of a row (two chunks per
// thread above one wave's registers).
int norm_bwd_tpr(int H) { return H <= 1024 ? 64 : H <= 4096 ? 256 : H <= 8192 ? 512 : 1024; }

// Workgroups of the backward kernel on `cus` CUs: each writes one partial
// row of dgamma and dbeta.  One per CU, or two once each has 8 rows.
int norm_bwd_groups(long T, int H, int cus) {
  const int tpr = norm_bwd_tpr(H), rpw = ln_threads(tpr) / tpr;
  const long rows = (T + rpw - 1) / rpw;
  if (rows <= cus) return (int)rows;
  return rows >= 16L * cus && tpr < 1024 ? 2 * cus : cus;
}
constexpr int kNormBwdMaxGroups = 2 * 512;          // (workspace: on any device)

template <int XD, int DYD, int TPR, int R>
moe_status launch_norm_bwd(const LnBwdArgs& a, int groups, hipStream_t st) {
  hipLaunchKernelGGL((k_layer_norm_bwd<XD, DYD, TPR, R>), dim3(groups), dim3(ln_threads(TPR)), 0, st, a);
  HIP_TRY(hipGetLastError());
  return MOE_OK;
}
template <int XD, int DYD>
moe_status launch_norm_bwd(const LnBwdArgs& a, int groups, hipStream_t st) {
  if (a.H <= 512) return launch_norm_bwd<XD, DYD, 64, 1>(a, groups, st);
  if (a.H <= 1024) return launch_norm_bwd<XD, DYD, 64, 2>(a, groups, st);
  if (a.H <= 2048) return launch_norm_bwd<XD, DYD, 256, 1>(a, groups, st);
  if (a.H <= 4096) return launch_norm_bwd<XD, DYD, 256, 2>(a, groups, st);
  if (a.H <= 8192) return launch_norm_bwd<XD, DYD, 512, 2>(a, groups, st);
  return launch_norm_bwd<XD, DYD, 1024, 2>(a, groups, st);
}

// --------------------------------------------------------------- balance loss
struct BalLayout {
  int cb, tb, nc, nt, gx, gy;        // tokens per block, blocks, and the last kernel's grid
  size_t rowcnt, rown, rowp, lpart, done, total;
};

BalLayout bal_layout(int T, int E, int k, int S) {
  BalLayout L{};
  // count blocks of about 8192 ids, at most 64: the token kernel adds up a
  // sequence's rows of counts in every workgroup
  const long nc = std::min(64L, std::max(1L, (long)T * k / 8192));
  L.cb = (int)((T + nc - 1) / nc);
  L.nc = (T + L.cb - 1) / L.cb;
  // token blocks: about 1024 workgroups of whole passes (16 or 4 tokens)
  const int g = E <= 256 ? 16 : 4;
  L.tb = (int)(((long)T + 1023) / 1024 + g - 1) / g * g;
  L.nt = (T + L.tb - 1) / L.tb;
  L.gx = (E + 63) / 64;
  L.gy = std::min(S, 512);
  size_t o = 0;
  L.done = o; o = align256(o + 4);
  L.rown = o; o = align256(o + ((size_t)L.nc + S) * 4);
  L.lpart = o; o = align256(o + (size_t)L.gx * L.gy * 8);
  L.rowcnt = o; o = align256(o + ((size_t)L.nc + S) * E * 4);
  L.rowp = o; o = align256(o + ((size_t)L.nt + S) * E * 4);
  L.total = o;
  return L;
}

moe_status check_balance(int32_t T, int32_t E, int32_t k, int32_t S) {
  if (T < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "T must be >= 1 (got %d)", T);
  if (E < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "E must be >= 1 (got %d)", E);
  if (k < 1 || k > E) return fail(MOE_ERR_INVALID_ARGUMENT, "top_k must be in [1, E] (got %d)", k);
  if (S < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "n_seq must be >= 1 (got %d)", S);
  if (E > 1024) return fail(MOE_ERR_UNSUPPORTED, "E > 1024 is not supported (got %d)", E);
  if (k > 16) return fail(MOE_ERR_UNSUPPORTED, "top_k > 16 is not supported (got %d)", k);
  if ((long long)T * k > (1LL << 30)) return fail(MOE_ERR_UNSUPPORTED, "T * top_k too large");
  if (S > (1 << 20)) return fail(MOE_ERR_UNSUPPORTED, "n_seq > 2^20 is not supported (got %d)", S);
  return MOE_OK;
}

template <int L, int NJ>
moe_status launch_bal_tokens(const BalArgs& a, int grid, hipStream_t st) {
  hipLaunchKernelGGL((k_bal_tokens<L, NJ>), dim3(grid), dim3(256), 5 * L * NJ * 4 * 4, st, a);
  HIP_TRY(hipGetLastError());
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_layer_norm(int32_t T, int32_t H, int32_t in_dtype, int32_t out_dtype, int32_t scale_mode,
                          const void* x, const float* gamma, const float* beta, float eps, void* y, float* y_scales,
                          float* mean, float* rstd, moe_stream_t stream) {
  TRY(check_norm_shape(T, H));
  if (in_dtype != MOE_DTYPE_BF16 && in_dtype != MOE_DTYPE_F32)
    return fail(MOE_ERR_UNSUPPORTED, "in_dtype must be MOE_DTYPE_BF16 or MOE_DTYPE_F32 (got %d)", in_dtype);
  if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_FP8_E4M3)
    return fail(MOE_ERR_UNSUPPORTED, "out_dtype must be MOE_DTYPE_BF16, MOE_DTYPE_F32 or MOE_DTYPE_FP8_E4M3 (got %d)",
                out_dtype);
  const bool fp8 = out_dtype == MOE_DTYPE_FP8_E4M3;
  if (fp8 && scale_mode != MOE_INTER_SCALE_F32 && scale_mode != MOE_INTER_SCALE_POW2)
    return fail(MOE_ERR_INVALID_ARGUMENT, "unknown scale_mode %d", scale_mode);
  if (!(eps >= 0.f)) return fail(MOE_ERR_INVALID_ARGUMENT, "eps must not be negative (got %g)", (double)eps);
  TRY(check_ptr(x, "x"));
  TRY(check_ptr(gamma, "gamma"));
  TRY(check_ptr(beta, "beta", false));
  TRY(check_ptr(y, "y"));
  TRY(check_ptr(y_scales, "y_scales", fp8));
  if (!fp8 && y_scales) return fail(MOE_ERR_INVALID_ARGUMENT, "y_scales must be NULL unless the output is FP8");
  TRY(check_ptr(mean, "mean", rstd != nullptr));
  TRY(check_ptr(rstd, "rstd", mean != nullptr));
  DevInfo di;
  TRY(device_info(&di));
  const LnArgs a{x, gamma, beta, y, y_scales, mean, rstd, T, H, eps, fp8 && scale_mode == MOE_INTER_SCALE_POW2};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return in_dtype == MOE_DTYPE_BF16 ? launch_norm<LN_BF16>(a, out_dtype, di.cus, st)
                                    : launch_norm<LN_F32>(a, out_dtype, di.cus, st);
}

size_t moe_layer_norm_backward_workspace_size(int32_t T, int32_t H) {
  if (check_norm_shape(T, H) != MOE_OK) return 0;
  return align256((size_t)std::min((long)T, (long)kNormBwdMaxGroups) * 2 * H * 4);
}

moe_status moe_layer_norm_backward(int32_t T, int32_t H, int32_t x_dtype, int32_t dy_dtype, const void* x,
                                   const float* gamma, const float* mean, const float* rstd, const void* dy,
                                   float* dx, float* dgamma, float* dbeta, void* workspace, size_t workspace_bytes,
                                   moe_stream_t stream) {
  TRY(check_norm_shape(T, H));
  if (x_dtype != MOE_DTYPE_BF16 && x_dtype != MOE_DTYPE_F32)
    return fail(MOE_ERR_UNSUPPORTED, "x_dtype must be MOE_DTYPE_BF16 or MOE_DTYPE_F32 (got %d)", x_dtype);
  if (dy_dtype != MOE_DTYPE_BF16 && dy_dtype != MOE_DTYPE_F32)
    return fail(MOE_ERR_UNSUPPORTED, "dy_dtype must be MOE_DTYPE_BF16 or MOE_DTYPE_F32 (got %d)", dy_dtype);
  TRY(check_ptr(x, "x"));
  TRY(check_ptr(gamma, "gamma"));
  TRY(check_ptr(mean, "mean"));
  TRY(check_ptr(rstd, "rstd"));
  TRY(check_ptr(dy, "dy"));
  TRY(check_ptr(dx, "dx"));
  TRY(check_ptr(dgamma, "dgamma", false));
  TRY(check_ptr(dbeta, "dbeta", false));
  if (dx == dy && dy_dtype != MOE_DTYPE_F32)
    return fail(MOE_ERR_INVALID_ARGUMENT, "dx can be dy only where dy is fp32");
  const bool weights = dgamma || dbeta;
  TRY(check_ptr(workspace, "workspace", weights));
  const size_t need = weights ? moe_layer_norm_backward_workspace_size(T, H) : 0;
  if (workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  DevInfo di;
  TRY(device_info(&di));
  const int groups = std::min(norm_bwd_groups(T, H, di.cus), kNormBwdMaxGroups);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const LnBwdArgs a{x, gamma, mean, rstd, dy, dx, weights ? static_cast<float*>(workspace) : nullptr, T, H};
  if (x_dtype == MOE_DTYPE_BF16)
    TRY((dy_dtype == MOE_DTYPE_BF16 ? launch_norm_bwd<LN_BF16, LN_BF16>(a, groups, st)
                                    : launch_norm_bwd<LN_BF16, LN_F32>(a, groups, st)));
  else
    TRY((dy_dtype == MOE_DTYPE_BF16 ? launch_norm_bwd<LN_F32, LN_BF16>(a, groups, st)
                                    : launch_norm_bwd<LN_F32, LN_F32>(a, groups, st)));
  if (weights) {
    hipLaunchKernelGGL(k_ln_weight_grad, dim3(H / kLnSumCols, 2), dim3(256), 0, st, a.part, groups, H, dgamma, dbeta);
    HIP_TRY(hipGetLastError());
  }
  return MOE_OK;
}

size_t moe_balance_loss_workspace_size(int32_t T, int32_t E, int32_t top_k, int32_t n_seq) {
  if (check_balance(T, E, top_k, n_seq) != MOE_OK) return 0;
  return bal_layout(T, E, top_k, n_seq).total;
}

moe_status moe_balance_loss(int32_t T, int32_t E, int32_t top_k, int32_t n_seq, const float* logits,
                            const int32_t* topk_ids, const int32_t* seq_offsets, const uint8_t* token_mask,
                            float alpha, int32_t* counts, float* probs, float* loss, float* dlogits, void* workspace,
                            size_t workspace_bytes, moe_stream_t stream) {
  TRY(check_balance(T, E, top_k, n_seq));
  if (!seq_offsets && n_seq != 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n_seq must be 1 without seq_offsets (got %d)", n_seq);
  TRY(check_ptr(logits, "logits"));
  TRY(check_ptr(topk_ids, "topk_ids"));
  TRY(check_ptr(seq_offsets, "seq_offsets", false));
  TRY(check_ptr(token_mask, "token_mask", false));
  TRY(check_ptr(counts, "counts"));
  TRY(check_ptr(probs, "probs"));
  TRY(check_ptr(loss, "loss"));
  TRY(check_ptr(dlogits, "dlogits", false));
  if (dlogits == logits) return fail(MOE_ERR_INVALID_ARGUMENT, "dlogits is logits");
  TRY(check_ptr(workspace, "workspace"));
  const BalLayout L = bal_layout(T, E, top_k, n_seq);
  if (workspace_bytes < L.total)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", workspace_bytes, L.total);
  DevInfo di;
  TRY(device_info(&di));
  char* ws = static_cast<char*>(workspace);
  BalArgs a{};
  a.logits = logits; a.ids = topk_ids; a.off = seq_offsets; a.mask = token_mask;
  a.counts = counts; a.probs = probs; a.loss = loss; a.dlogits = dlogits;
  a.T = T; a.E = E; a.k = top_k; a.S = n_seq; a.alpha = alpha; a.cb = L.cb; a.tb = L.tb;
  a.rowcnt = reinterpret_cast<int32_t*>(ws + L.rowcnt);
  a.rown = reinterpret_cast<int32_t*>(ws + L.rown);
  a.rowp = reinterpret_cast<float*>(ws + L.rowp);
  a.lpart = reinterpret_cast<double*>(ws + L.lpart);
  a.done = reinterpret_cast<int32_t*>(ws + L.done);
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(k_bal_count, dim3(L.nc), dim3(kBalCountThreads), E * 4, st, a);
  HIP_TRY(hipGetLastError());
  if (E <= 64) TRY((launch_bal_tokens<16, 1>(a, L.nt, st)));
  else if (E <= 128) TRY((launch_bal_tokens<16, 2>(a, L.nt, st)));
  else if (E <= 256) TRY((launch_bal_tokens<16, 4>(a, L.nt, st)));
  else if (E <= 512) TRY((launch_bal_tokens<64, 2>(a, L.nt, st)));
  else TRY((launch_bal_tokens<64, 4>(a, L.nt, st)));
  hipLaunchKernelGGL(k_bal_final, dim3(L.gx, L.gy), dim3(256), 0, st, a);
  HIP_TRY(hipGetLastError());
  return MOE_OK;
}

}  // extern "C"
