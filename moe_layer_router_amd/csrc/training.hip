// The operators around the layer in a training step, as C entry points:
// layer norm in front of it (norm.h), the load-balance loss of its router
// (balance.h) and the orthogonalised update of its weights
// (orthogonalize.h).
#include "host.h"
#include "balance.h"
#include "norm.h"
#include "orthogonalize.h"

#include <algorithm>
#include <atomic>
#include <cmath>

using namespace moe;

namespace {

// ----------------------------------------------------------------- layer norm
size_t float_bytes(int32_t dtype) { return dtype == MOE_DTYPE_F32 ? 4 : dtype == MOE_DTYPE_BF16 ? 2 : 1; }

moe_status check_norm_shape(int32_t T, int32_t H) {
  if (T < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "T must be >= 1 (got %d)", T);
  if (H < 128 || H % 128) return fail(MOE_ERR_INVALID_ARGUMENT, "H must be a positive multiple of 128 (got %d)", H);
  if (H > 16384) return fail(MOE_ERR_UNSUPPORTED, "H > 16384 is not supported (got %d)", H);
  return MOE_OK;
}

// Threads of a row and chunks of 8 channels per thread: a wave per row while
// the row fits its registers (no barrier in the sums), more waves above.
template <int IN, int OUT, int TPR, int R>
moe_status launch_norm(const LnArgs& a, int cus, hipStream_t st) {
  constexpr int RPW = ln_threads(TPR) / TPR;
  // 16 waves per CU, each going through rows with gamma and beta read once
  // (T H = 59 M, BF16, H = 512 / 4096 / 7168: 44 / 46 / 48 us; with a quarter
  // of them 84 / 87 / -, with twice as many 48 / 49 / 50)
  const long rows = (a.T + RPW - 1) / RPW;
  const unsigned grid = (unsigned)std::min(rows, (long)cus * (1024 / ln_threads(TPR)));
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
  if (a.H <= 8192) return launch_norm<IN, OUT, 512, 2>(a, cus, st);
  return launch_norm<IN, OUT, 1024, 2>(a, cus, st);
}
template <int IN>
moe_status launch_norm(const LnArgs& a, int out_dtype, int cus, hipStream_t st) {
  if (out_dtype == MOE_DTYPE_BF16) return launch_norm<IN, LN_BF16>(a, cus, st);
  if (out_dtype == MOE_DTYPE_F32) return launch_norm<IN, LN_F32>(a, cus, st);
  return launch_norm<IN, LN_FP8>(a, cus, st);
}

// Workgroups of the backward kernel: each writes one partial row of dgamma
// and dbeta, so not more than one per CU (T H = 59 M, H = 4096 / 7168: 106 / 114
// us, with two per CU 113 / 123).
int norm_bwd_groups(long T, int H, int cus) {
  const int rows_per_wg = H <= 1024 ? 4 : 1;        // (rows of one wave: launch_norm_bwd)
  return (int)std::min((T + rows_per_wg - 1) / rows_per_wg, (long)cus);
}
constexpr int kNormBwdMaxGroups = 1024;             // (workspace: on any device)

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
  return launch_norm_bwd<XD, DYD, 512, 4>(a, groups, st);
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
  L.done = o; o = align256(o + 8);          // and S'
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

template <int L, int NJ, int VEC, int GRAD>
moe_status launch_bal(const BalArgs& a, const BalLayout& G, hipStream_t st) {
  // one workgroup while it does the tokens in at most 8 passes and 2^16 logits, else three
  // kernels.  On the GPU alone the border is at 2^15 (one against three: E = 64, T = 512
  // 15 us and 16, T = 768 20 and 16; E = 128, T = 256 14 and 16, T = 512 21 and 17; E = 256,
  // T = 128 14 and 17, T = 256 20 and 17; E = 1024, T = 16 10 and 19, T = 64 20 and 19), but
  // a call that allocates its outputs takes the host 21 us with three launches (T = 512: E
  // = 64 16 and 21, E = 128 21 and 21, E = 256 31 and 21; T = 64, E = 1024 20 and 21).
  constexpr int NT = L == 16 ? 1024 : 512;
  using One = BalTokens<L, NJ, VEC, GRAD, NT>;
  if (a.S <= kBalSegs && a.T <= 8 * One::G && a.T * a.E <= 1 << 16) {
    hipLaunchKernelGGL((k_bal_one<L, NJ, VEC, GRAD, NT>), dim3(1), dim3(NT), One::kLds + kBalSegs * a.E * 4, st, a);
    HIP_TRY(hipGetLastError());
    return MOE_OK;
  }
  hipLaunchKernelGGL(k_bal_count, dim3(G.nc), dim3(kBalCountThreads), kBalSegs * a.E * 4, st, a);
  HIP_TRY(hipGetLastError());
  hipLaunchKernelGGL((k_bal_tokens<L, NJ, VEC, GRAD>), dim3(G.nt), dim3(256),
                     (BalTokens<L, NJ, VEC, GRAD, 256>::kLds), st, a);
  HIP_TRY(hipGetLastError());
  hipLaunchKernelGGL(k_bal_final, dim3(G.gx, G.gy), dim3(kBalFinalThreads), 0, st, a);
  HIP_TRY(hipGetLastError());
  return MOE_OK;
}
template <int L, int NJ>
moe_status launch_bal(const BalArgs& a, const BalLayout& G, hipStream_t st) {
  if (a.E % 4 == 0) return a.dlogits ? launch_bal<L, NJ, 1, 1>(a, G, st) : launch_bal<L, NJ, 1, 0>(a, G, st);
  return a.dlogits ? launch_bal<L, NJ, 0, 1>(a, G, st) : launch_bal<L, NJ, 0, 0>(a, G, st);
}

// -------------------------------------------------------- orthogonalisation
// set_lds_limit, once per kernel and device (a call launches up to two dozen
// kernels, and the attribute costs as much as half a launch).
template <auto K>
moe_status set_lds_limit_once(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  HIP_TRY(hipGetDevice(&dev));
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit && (done.load(std::memory_order_relaxed) & bit)) return MOE_OK;
  TRY(set_lds_limit(K, bytes));
  done.fetch_or(bit, std::memory_order_relaxed);
  return MOE_OK;
}

constexpr float kOrthCoeffs[3] = {3.4445f, -4.7750f, 2.0315f};
constexpr int kOrthMaxSteps = 32;
constexpr size_t kOrthChunkBytes = (size_t)8 << 30;
// Tile shapes: 256 x 256 (eight waves of 64 x 128, one workgroup per CU), and
// smaller ones where there are too few of those to fill the GPU or they would
// cover too much that is not there.
using OrthBig = OrthTile<4, 2, 8, 2>;
using OrthMid = OrthTile<2, 2, 4, 2>;
using OrthMidDeep = OrthTile<2, 2, 4, 3>;
using OrthSmall = OrthTile<1, 2, 2, 3>;
constexpr int kOrthParts = 512;      // parts of tiles in one launch (at most 128 MiB of sums)

// Bytes for the sums of tiles worked on in parts, whichever tile shape is
// taken (that depends on the device): GRAM has the larger K.
template <class TL>
size_t orth_part_bytes(int batch, int mp, int np) {
  const size_t tj = (mp + TL::kSide - 1) / TL::kSide, tiles = tj * (tj + 1) / 2 * batch;
  const size_t split = np / 256;
  return split < 2 ? 0 : std::min((size_t)kOrthParts, tiles * split) * TL::kPart * 4;
}

struct OrthLayout {
  int m, n, mp, np, chunk;           // short and long side, padded; matrices worked on together
  size_t part, hi0, hi1, lo, a, b, sums, total;
  int sq, slabs;                     // narrow matrices: padded side, partial Gram matrices
  size_t q;
};

OrthLayout orth_layout(int batch, int M, int N) {
  OrthLayout L{};
  L.m = std::min(M, N);
  L.n = std::max(M, N);
  L.mp = (L.m + kOrthPad - 1) / kOrthPad * kOrthPad;
  L.np = (L.n + kOrthPad - 1) / kOrthPad * kOrthPad;
  if (L.m <= kOrthNarrow) {
    L.sq = L.m <= 16 ? 16 : L.m <= 32 ? 32 : 64;
    L.slabs = std::min(kOrthSlabs, (L.n + 63) / 64);
    L.chunk = batch;
    const size_t e = (size_t)L.sq * L.sq * batch;
    L.q = align256(L.slabs * e * 8);
    L.total = L.q + align256(e * 8);
    return L;
  }
  const size_t x = (size_t)L.mp * L.np * 2, q = (size_t)L.mp * L.mp * 2;
  // a large batch goes through in parts of at most 8 GiB, each of which
  // fills the GPU
  const size_t sums = std::max({orth_part_bytes<OrthBig>(batch, L.mp, L.np), orth_part_bytes<OrthMid>(batch, L.mp, L.np),
                                orth_part_bytes<OrthSmall>(batch, L.mp, L.np)});
  L.chunk = (int)std::min((size_t)batch, std::max((size_t)1, (kOrthChunkBytes - sums) / (3 * x + 2 * q)));
  const size_t c = L.chunk;
  size_t o = 0;
  L.part = o; o = align256(o + c * kOrthNormParts * 8);
  L.hi0 = o; o = align256(o + c * x);
  L.hi1 = o; o = align256(o + c * x);
  L.lo = o; o = align256(o + c * x);
  L.a = o; o = align256(o + c * q);
  L.b = o; o = align256(o + c * q);
  L.sums = o; o = align256(o + sums);
  L.total = o;
  return L;
}

moe_status check_orth(int32_t batch, int32_t M, int32_t N) {
  if (batch < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "batch must be >= 1 (got %d)", batch);
  if (M < 1 || N < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "M and N must be >= 1 (got %d, %d)", M, N);
  // 32-bit offsets within a matrix's FP16 buffers
  if (M > 32768 || N > 32768 || std::min(M, N) > 16384)
    return fail(MOE_ERR_UNSUPPORTED, "matrices up to 16384 x 32768 are supported (got %d x %d)", M, N);
  if (batch > 65535) return fail(MOE_ERR_UNSUPPORTED, "batch > 65535 is not supported (got %d)", batch);
  return MOE_OK;
}

// Whether X and A stay within the range of their FP16 parts over the
// steps: the singular values start in [0, 1], and a step takes [0, s] to its
// image under the polynomial.
bool orth_in_range(int steps, const float* co) {
  double top = 1;
  for (int k = 0; k < steps; ++k) {
    const double a = co[3 * k], b = co[3 * k + 1], c = co[3 * k + 2];
    double next = 0;
    for (int i = 0; i <= 1024; ++i) {
      const double s = top * i / 1024, s2 = s * s, bv = b * s2 + c * s2 * s2, to = std::fabs(s * (a + bv));
      if (!(std::fabs(a) + std::fabs(bv) < 1000) || !(to < 3.8)) return false;      // (NaN: false too)
      next = std::max(next, to);
    }
    top = 1.01 * next;                    // (rounding, and the grid's gaps)
  }
  return true;
}

// Tiles of a product, and how many of them are worked on in parts.
template <class TL, int MODE>
moe_status launch_orth_gemm(OrthGemm g, int batch, int cus, hipStream_t st) {
  const int ti = (g.rows + TL::kSide - 1) / TL::kSide;
  g.tj = (g.cols + TL::kSide - 1) / TL::kSide;
  g.tiles = orth_sym(MODE) ? ti * (ti + 1) / 2 : ti * g.tj;
  const int total = g.tiles * batch, slots = cus * (160 * 1024 / TL::kLds);
  g.full = total;
  g.split = 1;
  if (orth_sym(MODE)) {
    // what does not fill a whole round of the GPU is split along K, as far as
    // the slots and 256-K parts go
    const int rest = total % slots;
    const int split = rest ? std::min({slots / rest, g.K / 256, kOrthParts / rest}) : 1;
    if (split >= 2) {
      g.full = total - rest;
      g.split = split;
      g.rest = rest;
    }
  }
  TRY((set_lds_limit_once<k_orth_gemm<TL, MODE>>(TL::kLds)));
  const unsigned grid = (unsigned)((g.full + 7) / 8 * 8 + g.rest * g.split);
  hipLaunchKernelGGL((k_orth_gemm<TL, MODE>), dim3(grid), dim3(TL::kThreads), TL::kLds, st, g);
  HIP_TRY(hipGetLastError());
  if (g.rest) {
    hipLaunchKernelGGL((k_orth_join<TL, MODE>), dim3(g.rest * TL::NW * (TL::NJ / 2)), dim3(256), 0, st, g);
    HIP_TRY(hipGetLastError());
  }
  return MOE_OK;
}
template <int MODE>
moe_status launch_orth_gemm(const OrthGemm& g, int batch, int cus, hipStream_t st) {
  const long big = (long)((g.rows + 255) / 256) * ((g.cols + 255) / 256) * batch;
  const long ti = (g.rows + 127) / 128, tj = (g.cols + 127) / 128, mid = ti * tj * batch;
  // the large tiles unless they cover a quarter more than the middle ones do
  // (16 x 640 x 1400, a third more: 429 us, with the middle ones 363; 64 x 300 x 700
  // 441 and 317; 8 x 2048 x 7168, the same: 4.62 ms, with the middle ones 5.15)
  if (big >= cus && 16 * big <= 5 * mid) return launch_orth_gemm<OrthBig, MODE>(g, batch, cus, st);
  if (mid >= cus) {
    // up to one workgroup per CU: a third stage in place of the second workgroup
    // (4 x 1024 x 1024 337 -> 241 us, 20 x 450 x 900 379 -> 270; with more tiles 796 ->
    // 946 for 2048 x 7168), unless a product is one matrix's, would leave a third of the CUs
    // idle and has a K long enough for parts (whole tiles against three parts each, 136
    // tiles of 2048 rows: K = 4160 614 us and 590, 7168 860 and 797, 14336 1386 and
    // 1244).  The parts of a batch's matrices share less in the L2s (4 x 1024 x 8192
    // 935 and 996), and with fewer CUs idle they gain nothing (2700 x 8192 1331 and
    // 1352, 25 x 450 x 9000 1994 and 2262).
    const long tiles = orth_sym(MODE) ? ti * (ti + 1) / 2 * batch : mid;
    const bool parts = orth_sym(MODE) && batch == 1 && 3 * tiles <= 2 * cus && g.K > 4096;
    if (tiles <= cus && !parts) return launch_orth_gemm<OrthMidDeep, MODE>(g, batch, cus, st);
    return launch_orth_gemm<OrthMid, MODE>(g, batch, cus, st);
  }
  return launch_orth_gemm<OrthSmall, MODE>(g, batch, cus, st);
}

template <int BF, int MP>
moe_status launch_orth_narrow(OrthNarrow a, int batch, int cus, hipStream_t st) {
  hipLaunchKernelGGL((k_orth_gram64<BF, MP>), dim3(a.slabs, batch), dim3(OrthF64<MP>::kThreads), 0, st, a);
  HIP_TRY(hipGetLastError());
  TRY((set_lds_limit_once<k_orth_iter64<MP>>(OrthSq<MP>::kLds)));
  hipLaunchKernelGGL(k_orth_iter64<MP>, dim3(batch), dim3(OrthF64<MP>::kThreads), OrthSq<MP>::kLds, st, a);
  HIP_TRY(hipGetLastError());
  // a wave's tiles share its reads of Q, as far as there are four workgroups per CU
  constexpr int kCols = 16 * 4 / (MP / 16);       // columns of the workgroup's waves side by side
  const long passes = (a.n + kCols - 1) / kCols;
  a.tiles = (int)std::max(1L, std::min(8L, passes * batch / (4L * cus)));
  const dim3 grid((unsigned)((passes + a.tiles - 1) / a.tiles), batch);
  if (a.tall) hipLaunchKernelGGL((k_orth_apply<BF, MP, 1>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((k_orth_apply<BF, MP, 0>), grid, dim3(256), 0, st, a);
  HIP_TRY(hipGetLastError());
  return MOE_OK;
}
template <int BF>
moe_status launch_orth_narrow(const OrthNarrow& a, int sq, int batch, int cus, hipStream_t st) {
  if (sq == 16) return launch_orth_narrow<BF, 16>(a, batch, cus, st);
  if (sq == 32) return launch_orth_narrow<BF, 32>(a, batch, cus, st);
  return launch_orth_narrow<BF, 64>(a, batch, cus, st);
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
  const size_t n = (size_t)T * H;
  if (overlap(x, n * float_bytes(in_dtype), y, n * float_bytes(out_dtype)))
    return fail(MOE_ERR_INVALID_ARGUMENT, "y overlaps x");
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
  const size_t n = (size_t)T * H;
  if (overlap(dx, n * 4, dy, n * float_bytes(dy_dtype)) && !(dx == dy && dy_dtype == MOE_DTYPE_F32))
    return fail(MOE_ERR_INVALID_ARGUMENT, "dx overlaps dy (it may only be an fp32 dy itself)");
  if (overlap(dx, n * 4, x, n * float_bytes(x_dtype))) return fail(MOE_ERR_INVALID_ARGUMENT, "dx overlaps x");
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
  if (overlap(dlogits, (size_t)T * E * 4, logits, (size_t)T * E * 4))
    return fail(MOE_ERR_INVALID_ARGUMENT, "dlogits overlaps logits");
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
  a.used = a.done + 1;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (E <= 64) return launch_bal<16, 1>(a, L, st);
  if (E <= 128) return launch_bal<16, 2>(a, L, st);
  if (E <= 256) return launch_bal<16, 4>(a, L, st);
  if (E <= 512) return launch_bal<64, 2>(a, L, st);
  return launch_bal<64, 4>(a, L, st);
}

size_t moe_orthogonalize_workspace_size(int32_t batch, int32_t M, int32_t N) {
  if (check_orth(batch, M, N) != MOE_OK) return 0;
  return orth_layout(batch, M, N).total;
}

moe_status moe_orthogonalize(int32_t batch, int32_t M, int32_t N, int32_t in_dtype, const void* u, int32_t steps,
                             const float* coeffs, float eps, void* y, void* workspace, size_t workspace_bytes,
                             moe_stream_t stream) {
  TRY(check_orth(batch, M, N));
  if (in_dtype != MOE_DTYPE_BF16 && in_dtype != MOE_DTYPE_F32)
    return fail(MOE_ERR_UNSUPPORTED, "in_dtype must be MOE_DTYPE_BF16 or MOE_DTYPE_F32 (got %d)", in_dtype);
  if (steps < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "steps must be >= 1 (got %d)", steps);
  if (steps > kOrthMaxSteps) return fail(MOE_ERR_UNSUPPORTED, "steps > %d is not supported (got %d)", kOrthMaxSteps, steps);
  if (!(eps > 0.f)) return fail(MOE_ERR_INVALID_ARGUMENT, "eps must be positive (got %g)", (double)eps);
  if (coeffs && !orth_in_range(steps, coeffs))
    return fail(MOE_ERR_UNSUPPORTED, "coeffs let the iteration leave the range of its FP16 products");
  TRY(check_ptr(u, "u"));
  TRY(check_ptr(y, "y"));
  TRY(check_ptr(workspace, "workspace"));
  const size_t elems = (size_t)M * N, isz = in_dtype == MOE_DTYPE_BF16 ? 2 : 4;
  if (overlap(y, batch * elems * 2, u, batch * elems * isz))
    return fail(MOE_ERR_INVALID_ARGUMENT, "y overlaps u");
  const OrthLayout L = orth_layout(batch, M, N);
  if (workspace_bytes < L.total)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", workspace_bytes, L.total);
  DevInfo di;
  TRY(device_info(&di));
  char* ws = static_cast<char*>(workspace);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool bf = in_dtype == MOE_DTYPE_BF16;
  if (L.sq) {
    OrthNarrow a{};
    a.u = u; a.m = L.m; a.n = L.n; a.tall = M > N; a.slabs = L.slabs; a.steps = steps; a.eps = eps;
    for (int k = 0; k < steps; ++k)
      for (int i = 0; i < 3; ++i) a.co[k][i] = coeffs ? coeffs[3 * k + i] : kOrthCoeffs[i];
    a.part = reinterpret_cast<double*>(ws);
    a.q = reinterpret_cast<double*>(ws + L.q);
    a.y = static_cast<uint16_t*>(y);
    return bf ? launch_orth_narrow<1>(a, L.sq, batch, di.cus, st) : launch_orth_narrow<0>(a, L.sq, batch, di.cus, st);
  }
  for (int b0 = 0; b0 < batch; b0 += L.chunk) {
    const int nb = std::min(L.chunk, batch - b0);
    OrthArgs a{};
    a.u = static_cast<const char*>(u) + (size_t)b0 * elems * isz;
    a.M = M; a.N = N; a.m = L.m; a.n = L.n; a.mp = L.mp; a.np = L.np;
    a.tall = M > N;
    a.eps = eps;
    a.part = reinterpret_cast<double*>(ws + L.part);
    uint16_t* hi[2] = {reinterpret_cast<uint16_t*>(ws + L.hi0), reinterpret_cast<uint16_t*>(ws + L.hi1)};
    a.hi = hi[0];
    a.lo = reinterpret_cast<uint16_t*>(ws + L.lo);
    const dim3 norm_grid(kOrthNormParts, nb);
    const dim3 load_grid((a.tall ? L.mp : L.np) / 64, (a.tall ? L.np : L.mp) / 64, nb);
    if (bf) hipLaunchKernelGGL(k_orth_norm<1>, norm_grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL(k_orth_norm<0>, norm_grid, dim3(256), 0, st, a);
    HIP_TRY(hipGetLastError());
    if (bf) hipLaunchKernelGGL(k_orth_load<1>, load_grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL(k_orth_load<0>, load_grid, dim3(256), 0, st, a);
    HIP_TRY(hipGetLastError());
    uint16_t* A = reinterpret_cast<uint16_t*>(ws + L.a);
    uint16_t* B = reinterpret_cast<uint16_t*>(ws + L.b);
    const size_t xs = (size_t)L.mp * L.np, qs = (size_t)L.mp * L.mp;
    for (int k = 0; k < steps; ++k) {
      const float* co = coeffs ? coeffs + 3 * k : kOrthCoeffs;
      OrthGemm g{};
      g.part = reinterpret_cast<float*>(ws + L.sums);
      g.lo = a.lo; g.m = L.m; g.n = L.n; g.tall = a.tall;
      // A = X X^T: 2^24 times it in the accumulators, 2^12 in A
      g.p = g.q = hi[k & 1];
      g.p_stride = g.q_stride = xs;
      g.p_bytes = g.q_bytes = (uint32_t)(xs * 2);
      g.ldp = g.ldq = L.mp;
      g.rows = g.cols = L.mp;
      g.K = L.np;
      g.s = 1.0f / kOrthScale;
      g.c = A;
      TRY((launch_orth_gemm<ORTH_GRAM>(g, nb, di.cus, st)));
      // B' = a I + b A + c A A
      g.p = g.q = A;
      g.p_stride = g.q_stride = qs;
      g.p_bytes = g.q_bytes = (uint32_t)(qs * 2);
      g.K = L.mp;
      g.a = A;
      g.c = B;
      g.c0 = co[0];
      g.c1 = co[1] / kOrthScale;
      g.s = co[2] / (kOrthScale * kOrthScale);
      TRY((launch_orth_gemm<ORTH_POLY>(g, nb, di.cus, st)));
      // X'^T = hi B' + a lo
      g.p = hi[k & 1];
      g.q = B;
      g.p_stride = xs;
      g.p_bytes = (uint32_t)(xs * 2);
      g.rows = L.np;
      g.hi = hi[(k + 1) & 1];
      g.y = static_cast<uint16_t*>(y) + (size_t)b0 * elems;
      if (k + 1 < steps) TRY((launch_orth_gemm<ORTH_STEP>(g, nb, di.cus, st)));
      else TRY((launch_orth_gemm<ORTH_LAST>(g, nb, di.cus, st)));
    }
  }
  return MOE_OK;
}

}  // extern "C"
