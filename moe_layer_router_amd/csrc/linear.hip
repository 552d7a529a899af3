// Linear layers with an epilogue and their gradients (linear.h), as C entry points.
#include "host.h"
#include "linear.h"

#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

using namespace moe;

namespace {

using LinBig = LinTile<4, 2, 8, 2>;        // 256 columns, eight waves, one workgroup per CU
using LinMid = LinTile<2, 2, 4, 2>;        // 128 columns, two workgroups per CU
using LinMidDeep = LinTile<2, 2, 4, 4>;    // the same with four steps in LDS, one workgroup per CU
using LinSmall = LinTile<1, 2, 2, 4>;      // 64 columns
using LinSmallParts = LinTile<2, 2, 2, 4>; // the same, and as many rows of P in parts
constexpr int kLinMaxDim = 1 << 17;        // (offsets in a tile's 256 rows of three parts fit 32 bits)

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

size_t lin_bytes_of(int32_t dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }
bool lin_float(int32_t dtype) { return dtype == MOE_DTYPE_F32 || dtype == MOE_DTYPE_BF16; }

moe_status check_linear(int32_t T, int32_t K, int32_t N, int32_t act) {
  if (T < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "T must be >= 1 (got %d)", T);
  if (K < 8 || K % 8) return fail(MOE_ERR_INVALID_ARGUMENT, "K must be a positive multiple of 8 (got %d)", K);
  if (N < 8 || N % 8) return fail(MOE_ERR_INVALID_ARGUMENT, "N must be a positive multiple of 8 (got %d)", N);
  if (act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU) return fail(MOE_ERR_INVALID_ARGUMENT, "unknown act %d", act);
  if (K > kLinMaxDim || (act == MOE_ACT_SWIGLU ? 2 * (long)N : N) > kLinMaxDim)
    return fail(MOE_ERR_UNSUPPORTED, "K and the rows of W up to %d are supported (got %d, N = %d)", kLinMaxDim, K, N);
  return MOE_OK;
}
int lin_rows(int N, int act) { return act == MOE_ACT_SWIGLU ? 2 * N : N; }

// Bytes for the sums of tiles worked on in parts, whichever tiles are taken (that depends on the device).
template <class TL>
size_t lin_part_bytes(long rows, int cols, long K, int parts, bool gated) {
  const long mt = TL::rows(parts), nt = gated ? TL::kCols / 2 : TL::kCols;
  const long tiles = ((rows + mt - 1) / mt) * ((cols + nt - 1) / nt), split = K / 256;
  return split < 2 ? 0 : (size_t)std::min((long)kLinParts, tiles * split) * TL::sums(parts) * 4;
}
size_t lin_parts(long rows, int cols, long K, int parts, bool gated) {
  return std::max({lin_part_bytes<LinBig>(rows, cols, K, parts, gated), lin_part_bytes<LinMid>(rows, cols, K, parts, gated),
                   parts == 1 ? lin_part_bytes<LinSmall>(rows, cols, K, parts, gated)
                              : lin_part_bytes<LinSmallParts>(rows, cols, K, parts, gated)});
}

// What work on the tiles takes, in ns (measured with every slot of the GPU at work): a 64-k step with both operands along k, 1.15
// times that with one across it, 1.35 times with P in three parts; what a round's first loads and last stores leave uncovered.
template <class TL>
constexpr long kLinStep = std::is_same_v<TL, LinBig> ? 1650 : std::is_same_v<TL, LinMid> ? 1050 : std::is_same_v<TL, LinMidDeep> ? 580 : 480;
template <class TL>
constexpr long kLinRound = std::is_same_v<TL, LinBig> ? 8000 : std::is_same_v<TL, LinMid> ? 4000 : std::is_same_v<TL, LinMidDeep> ? 7000 : 2500;
template <class TL, int QT, int PARTS>
constexpr long lin_step() { return kLinStep<TL> * (QT ? PARTS == 3 ? 27 : 23 : 20) / 20; }
// Tiles in parts take a second launch (3 us on the GPU, 4 of the host's) and their sums' way through the caches (8 bytes each at 10 TB/s).
template <class TL, int PARTS>
constexpr long lin_join_ns(long parts) { return 5000 + parts * (long)TL::sums(PARTS) / 1250; }

// How a product's tiles are worked on; the workgroups.
template <class TL, int QT, int PARTS, int GATED>
moe_status plan_tiles(LinGemm& g, int cus, unsigned* grid) {
  constexpr int MT = TL::rows(PARTS), NT = GATED ? TL::kCols / 2 : TL::kCols;
  g.tj = (g.cols + NT - 1) / NT;
  const long total = (g.rows + MT - 1) / MT * g.tj, slots = (long)cus * (160 * 1024 / TL::lds(PARTS));
  if ((total + 16 + kLinParts) * TL::kThreads > UINT32_MAX)       // (threads of a grid)
    return fail(MOE_ERR_UNSUPPORTED, "the output has too many tiles");
  g.full = total;
  g.split = 1;
  g.rest = 0;
  // what does not fill a whole round of the GPU is split along k, as far as the slots and 256-k parts go and the second launch
  // leaves a gain
  const long rest = total % slots, steps = (g.K + 63) / 64;
  const long most = rest ? std::min({slots / rest, g.K / 256, (long)kLinParts / rest}) : 1;
  long least = steps * lin_step<TL, QT, PARTS>();
  for (long split = most; split >= 2; split /= 2) {
    const long ns = (steps + split - 1) / split * lin_step<TL, QT, PARTS>() + lin_join_ns<TL, PARTS>(rest * split);
    if (ns >= least) continue;
    least = ns;
    g.full = total - rest;
    g.split = (int)split;
    g.rest = (int)rest;
  }
  *grid = (unsigned)((g.full + 7) / 8 * 8 + (long)g.rest * g.split);
  return MOE_OK;
}
template <class TL, int PARTS, int GATED>
constexpr long lin_join_groups(const LinGemm& g) {
  return (long)g.rest * TL::rows(PARTS) * (GATED ? TL::kCols / 2 : TL::kCols) / 8 / 256;
}
template <class TL, int PARTS, int GATED>
moe_status launch_join(const LinGemm& g, hipStream_t st) {
  if (!g.rest) return MOE_OK;
  hipLaunchKernelGGL((k_linear_join<TL, PARTS, GATED>), dim3((unsigned)lin_join_groups<TL, PARTS, GATED>(g)), dim3(256), 0, st, g);
  HIP_TRY(hipGetLastError());
  return MOE_OK;
}
template <class TL, int PT, int QT, int PARTS, int GATED>
moe_status launch_tiles(LinGemm g, int cus, hipStream_t st) {
  constexpr auto kernel = k_linear<TL, PT, QT, PARTS, GATED>;
  unsigned grid;
  TRY((plan_tiles<TL, QT, PARTS, GATED>(g, cus, &grid)));
  TRY(set_lds_limit_once<kernel>(TL::lds(PARTS)));
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(TL::kThreads), TL::lds(PARTS), st, g);
  HIP_TRY(hipGetLastError());
  return launch_join<TL, PARTS, GATED>(g, st);
}

enum { LIN_BIG, LIN_MID, LIN_DEEP, LIN_SMALL };
template <int PARTS>
using LinLeast = std::conditional_t<PARTS == 1, LinSmall, LinSmallParts>;
// The tiles are chosen by the time that a product takes with each.  Measured, T x K x N:
//   4096 x 2048 x 7168  big 117 us, mid 153, deep 180, small 258        700 x 2048 x 7168  big 43.5, mid 34.9, deep 43.9, small 55.8
//   4096 x 1024 x 1024  big 35.7, mid 26.2, deep 18.3, small 21.6       700 x 2048 x 2048  big 36.0, mid 23.5, deep 23.6, small 18.8
template <class TL, int QT, int PARTS, int GATED>
long lin_cost(const LinGemm& g, int cus) {
  LinGemm p = g;
  unsigned grid;
  if (plan_tiles<TL, QT, PARTS, GATED>(p, cus, &grid) != MOE_OK) return LONG_MAX / 4;
  const long slots = (long)cus * (160 * 1024 / TL::lds(PARTS)), steps = (g.K + 63) / 64, full = (p.full + slots - 1) / slots;
  long ns = full * (steps * lin_step<TL, QT, PARTS>() + kLinRound<TL>);
  if (p.rest)
    ns += (steps + p.split - 1) / p.split * lin_step<TL, QT, PARTS>() + kLinRound<TL> + lin_join_ns<TL, PARTS>((long)p.rest * p.split);
  return ns;
}
struct LinChoice {
  int kind;
  long ns, small;                          // the kind's and the smallest tiles' time
};
template <int QT, int PARTS, int GATED>
LinChoice lin_choose(const LinGemm& g, int cus) {
  const long ns[4] = {lin_cost<LinBig, QT, PARTS, GATED>(g, cus), lin_cost<LinMid, QT, PARTS, GATED>(g, cus),
                      lin_cost<LinMidDeep, QT, PARTS, GATED>(g, cus), lin_cost<LinLeast<PARTS>, QT, PARTS, GATED>(g, cus)};
  int best = LIN_SMALL;
  for (int k = LIN_DEEP; k >= LIN_BIG; --k)
    if (ns[k] < ns[best]) best = k;
  return {best, ns[best], ns[LIN_SMALL]};
}
template <int PT, int QT, int PARTS, int GATED>
moe_status launch_product(const LinGemm& g, int cus, hipStream_t st) {
  switch (lin_choose<QT, PARTS, GATED>(g, cus).kind) {
    case LIN_BIG: return launch_tiles<LinBig, PT, QT, PARTS, GATED>(g, cus, st);
    case LIN_MID: return launch_tiles<LinMid, PT, QT, PARTS, GATED>(g, cus, st);
    case LIN_DEEP: return launch_tiles<LinMidDeep, PT, QT, PARTS, GATED>(g, cus, st);
    default: return launch_tiles<LinLeast<PARTS>, PT, QT, PARTS, GATED>(g, cus, st);
  }
}

// dx, dw and (b.db) dbias: together with small tiles where that takes no longer than one after another with each its own: two
// launches fewer.
constexpr long kLinJointNs = 6000;
template <int PX, int PW>
moe_status launch_grads(LinGemm x, LinGemm w, const LinDbias& b, int cus, hipStream_t st) {
  using TL = LinLeast<PW>;
  const unsigned nb = b.db ? (unsigned)(b.R + 63) / 64 : 0;
  const LinChoice cx = lin_choose<1, PX, 0>(x, cus), cw = lin_choose<1, PW, 0>(w, cus);
  if (cx.small + cw.small <= cx.ns + cw.ns + kLinJointNs) {
    constexpr auto kernel = k_linear_grads<TL, PX, PW>;
    constexpr int kLds = TL::lds(PX) > TL::lds(PW) ? TL::lds(PX) : TL::lds(PW);
    unsigned nx, nw;
    TRY((plan_tiles<TL, 1, PX, 0>(x, cus, &nx)));
    TRY((plan_tiles<TL, 1, PW, 0>(w, cus, &nw)));
    // (each has sums of its own)
    w.part = x.part + (size_t)x.rest * x.split * TL::sums(PX);
    TRY(set_lds_limit_once<kernel>(kLds));
    hipLaunchKernelGGL(kernel, dim3(nx + nw + nb), dim3(TL::kThreads), kLds, st, x, w, b, (int)nx, (int)nw);
    HIP_TRY(hipGetLastError());
    const long jx = lin_join_groups<TL, PX, 0>(x), jw = lin_join_groups<TL, PW, 0>(w);
    if (jx + jw == 0) return MOE_OK;
    hipLaunchKernelGGL((k_linear_joins<TL, PX, PW>), dim3((unsigned)(jx + jw)), dim3(256), 0, st, x, w, (int)jx);
    HIP_TRY(hipGetLastError());
    return MOE_OK;
  }
  if (nb) {
    hipLaunchKernelGGL(k_linear_dbias, dim3(nb), dim3(256), 0, st, b);
    HIP_TRY(hipGetLastError());
  }
  TRY((launch_product<0, 1, PX, 0>(x, cus, st)));
  return launch_product<1, 1, PW, 0>(w, cus, st);
}

// Few rows of x: W is read once by kernels that need no tile of rows.  They read x once per 16 rows of W, so that the tiles win with many
// rows and a long k.  Both in us, of a captured run of calls:
//   N = 2048:  K = 2048   T = 1 5.5 (tiles 9.5), T = 16 6.8 (9.6), T = 32 8.4 (10.3)
//              K = 7168   T = 1 11.8 (16.4), T = 4 13.5 (16.6), T = 16 17.4 (16.8), T = 32 23.9 (17.0)
//              K = 16384  T = 1 20.5 (21.5), T = 16 30.7 (21.9)
//   N = 7168:  K = 2048   T = 1 8.6 (16.3), T = 16 10.5 (14.3), T = 32 14.0 (17.0)
//              K = 4096   T = 16 17.6 (18.1), T = 17 19.1 (17.5), T = 32 24.0 (18.0)
//              K = 7168   T = 1 23.7 (25.7), T = 4 26.0 (24.8), T = 16 33.7 (25.5)
// (The rule does not know N: it takes the slower side at K = 7168 with N = 7168 and T = 4 to 16, and at K = 4096 with N = 2048 and T = 17 to 32,
// where these kernels take 11.2 to 13.8 for 15.5.)
bool lin_few(long T, long K) { return T <= 16 ? (T + 16) * K <= 1 << 18 : T <= 32 && K <= 2048; }
template <int GATED>
moe_status launch_rows(const LinGemm& g, hipStream_t st) {
  const dim3 grid((g.cols + (GATED ? 7 : 15)) / (GATED ? 8 : 16));
  if (g.rows <= 16) hipLaunchKernelGGL((k_linear_rows<1, GATED>), grid, dim3(512), 0, st, g);
  else hipLaunchKernelGGL((k_linear_rows<2, GATED>), grid, dim3(512), 0, st, g);
  HIP_TRY(hipGetLastError());
  return MOE_OK;
}

// Slabs of rows for the sums over the tokens.
constexpr int kLinSlabs = 256;
int lin_slab(long T) { return (int)std::max(4l, ((T + kLinSlabs - 1) / kLinSlabs + 3) / 4 * 4); }

struct LinBwdLayout {
  size_t dz, part, sums, total;
};
LinBwdLayout lin_bwd_layout(long T, int K, int N, int act) {
  const int R = lin_rows(N, act);
  LinBwdLayout L{};
  size_t o = 0;
  L.dz = o; o = align256(o + (size_t)T * ((R + 63) / 64 * 64) * 6);
  L.part = o; o = align256(o + (size_t)((T + lin_slab(T) - 1) / lin_slab(T)) * R * 4);
  L.sums = o;
  size_t sums = 0;
  for (int parts = 1; parts <= 3; ++parts)
    sums = std::max({sums, lin_parts(T, K, R, parts, false), lin_parts(R, K, T, parts, false)});
  // dx's and dw's side by side with small tiles
  const size_t both = lin_part_bytes<LinSmallParts>(T, K, R, 3, false) + lin_part_bytes<LinSmallParts>(R, K, T, 3, false);
  const size_t both1 = lin_part_bytes<LinSmall>(T, K, R, 1, false) + lin_part_bytes<LinSmall>(R, K, T, 1, false);
  L.total = align256(o + std::max({sums, both, both1}));
  return L;
}

}  // namespace

extern "C" {

size_t moe_linear_workspace_size(int32_t T, int32_t K, int32_t N, int32_t act) {
  if (check_linear(T, K, N, act) != MOE_OK) return 0;
  return lin_few(T, K) ? 256 : std::max((size_t)256, lin_parts(T, N, K, 1, act == MOE_ACT_SWIGLU));
}

moe_status moe_linear(int32_t T, int32_t K, int32_t N, int32_t act, const void* x, const void* w, const float* bias,
                      const void* residual, int32_t residual_dtype, void* y, int32_t y_dtype, void* pre,
                      int32_t pre_dtype, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  TRY(check_linear(T, K, N, act));
  if (!lin_float(y_dtype) || (residual && !lin_float(residual_dtype)) || (pre && !lin_float(pre_dtype)))
    return fail(MOE_ERR_UNSUPPORTED, "y, residual and pre must be MOE_DTYPE_BF16 or MOE_DTYPE_F32");
  TRY(check_ptr(x, "x"));
  TRY(check_ptr(w, "w"));
  TRY(check_ptr(bias, "bias", false));
  TRY(check_ptr(residual, "residual", false));
  TRY(check_ptr(y, "y"));
  TRY(check_ptr(pre, "pre", false));
  TRY(check_ptr(workspace, "workspace"));
  const int R = lin_rows(N, act);
  const size_t need = moe_linear_workspace_size(T, K, N, act);
  if (workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  const size_t nx = (size_t)T * K * 2, nw = (size_t)R * K * 2, nb = (size_t)R * 4;
  const size_t nr = (size_t)T * N * lin_bytes_of(residual_dtype), ny = (size_t)T * N * lin_bytes_of(y_dtype);
  const size_t np = (size_t)T * R * lin_bytes_of(pre_dtype);
  const struct { const void* p; size_t n; } in[] = {{x, nx}, {w, nw}, {bias, nb}, {residual, nr}}, out[] = {{y, ny}, {pre, np}, {workspace, need}};
  for (int i = 0; i < 3; ++i) {
    for (const auto& v : in) {
      // (an element of the residual is read where its y is written, by the same thread)
      if (i == 0 && v.p == residual && residual == y && residual_dtype == y_dtype) continue;
      if (overlap(out[i].p, out[i].n, v.p, v.n)) return fail(MOE_ERR_INVALID_ARGUMENT, "an output or the workspace overlaps an input");
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n))
        return fail(MOE_ERR_INVALID_ARGUMENT, "y, pre and the workspace must not overlap");
  }
  DevInfo di;
  TRY(device_info(&di));
  LinGemm g{};
  g.p = static_cast<const uint16_t*>(x);
  g.q = static_cast<const uint16_t*>(w);
  g.ldp = g.ldq = K;
  g.pch = 1;
  g.rows = T; g.cols = N; g.K = K;
  g.part = static_cast<float*>(workspace);
  g.e.bias = bias; g.e.res = residual; g.e.y = y; g.e.pre = pre;
  g.e.act = act; g.e.n = N;
  g.e.y_f32 = y_dtype == MOE_DTYPE_F32; g.e.res_f32 = residual_dtype == MOE_DTYPE_F32; g.e.pre_f32 = pre_dtype == MOE_DTYPE_F32;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (lin_few(T, K)) return act == MOE_ACT_SWIGLU ? launch_rows<1>(g, st) : launch_rows<0>(g, st);
  return act == MOE_ACT_SWIGLU ? launch_product<0, 0, 1, 1>(g, di.cus, st) : launch_product<0, 0, 1, 0>(g, di.cus, st);
}

size_t moe_linear_backward_workspace_size(int32_t T, int32_t K, int32_t N, int32_t act) {
  if (check_linear(T, K, N, act) != MOE_OK) return 0;
  return lin_bwd_layout(T, K, N, act).total;
}

moe_status moe_linear_backward(int32_t T, int32_t K, int32_t N, int32_t act, const void* x, const void* w,
                               const void* pre, int32_t pre_dtype, const void* dy, int32_t dy_dtype, void* dx,
                               int32_t dx_dtype, float* dw, float* dbias, void* workspace, size_t workspace_bytes,
                               moe_stream_t stream) {
  TRY(check_linear(T, K, N, act));
  if (!lin_float(dy_dtype) || (dx && !lin_float(dx_dtype)) || (act != MOE_ACT_NONE && !lin_float(pre_dtype)))
    return fail(MOE_ERR_UNSUPPORTED, "dy, dx and pre must be MOE_DTYPE_BF16 or MOE_DTYPE_F32");
  if (!dx && !dw && !dbias) return fail(MOE_ERR_INVALID_ARGUMENT, "no gradient is asked for");
  TRY(check_ptr(x, "x", dw != nullptr));
  TRY(check_ptr(w, "w", dx != nullptr));
  TRY(check_ptr(pre, "pre", act != MOE_ACT_NONE));
  TRY(check_ptr(dy, "dy"));
  TRY(check_ptr(dx, "dx", false));
  TRY(check_ptr(dw, "dw", false));
  TRY(check_ptr(dbias, "dbias", false));
  TRY(check_ptr(workspace, "workspace"));
  const int R = lin_rows(N, act);
  const LinBwdLayout L = lin_bwd_layout(T, K, N, act);
  if (workspace_bytes < L.total)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", workspace_bytes, L.total);
  const struct { const void* p; size_t n; } in[] = {{dw ? x : nullptr, (size_t)T * K * 2}, {dx ? w : nullptr, (size_t)R * K * 2},
      {act != MOE_ACT_NONE ? pre : nullptr, (size_t)T * R * lin_bytes_of(pre_dtype)}, {dy, (size_t)T * N * lin_bytes_of(dy_dtype)}},
      out[] = {{dx, (size_t)T * K * lin_bytes_of(dx_dtype)}, {dw, (size_t)R * K * 4}, {dbias, (size_t)R * 4}, {workspace, L.total}};
  for (int i = 0; i < 4; ++i) {
    for (const auto& v : in)
      if (overlap(out[i].p, out[i].n, v.p, v.n)) return fail(MOE_ERR_INVALID_ARGUMENT, "an output or the workspace overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n))
        return fail(MOE_ERR_INVALID_ARGUMENT, "the outputs and the workspace must not overlap");
  }
  DevInfo di;
  TRY(device_info(&di));
  hipStream_t st = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  uint16_t* dz = reinterpret_cast<uint16_t*>(ws + L.dz);
  float* sums = reinterpret_cast<float*>(ws + L.part);
  const bool whole = act == MOE_ACT_NONE && dy_dtype == MOE_DTYPE_BF16;      // dz is dy: one part
  const bool want_dz = !whole && (dx || dw);
  // parts of dz in memory: three for fp32 results, two for BF16 ones
  const int parts = whole ? 1 : dw || (dx && dx_dtype == MOE_DTYPE_F32) ? 3 : 2;
  LinDbias b{};
  if (want_dz || dbias) {
    LinDz a{};
    a.dy = dy; a.pre = act == MOE_ACT_NONE ? nullptr : pre;
    a.dz = want_dz ? dz : nullptr; a.part = dbias ? sums : nullptr;
    a.T = T; a.n = N; a.act = act; a.dy_f32 = dy_dtype == MOE_DTYPE_F32; a.pre_f32 = pre_dtype == MOE_DTYPE_F32;
    a.slab = lin_slab(T);
    a.parts = parts;
    const int slabs = (int)((T + a.slab - 1) / a.slab);
    const dim3 grid((N / 8 + 63) / 64, slabs);
    if (act == MOE_ACT_SWIGLU) hipLaunchKernelGGL(k_linear_dz<1>, grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL(k_linear_dz<0>, grid, dim3(256), 0, st, a);
    HIP_TRY(hipGetLastError());
    b = LinDbias{sums, dbias, slabs, R};
  }
  LinGemm g{};
  g.p = whole ? static_cast<const uint16_t*>(dy) : dz;
  g.ldp = whole ? R : (long)parts * ((R + 63) / 64 * 64);
  g.pch = parts;
  g.ldq = K;
  g.cols = K;
  g.e.n = K;
  g.part = reinterpret_cast<float*>(ws + L.sums);
  LinGemm gx = g, gw = g;
  gx.q = static_cast<const uint16_t*>(w);
  gx.rows = T; gx.K = R;
  gx.e.y = dx; gx.e.y_f32 = dx_dtype == MOE_DTYPE_F32;
  gw.q = static_cast<const uint16_t*>(x);
  gw.rows = R; gw.K = T;
  gw.e.y = dw; gw.e.y_f32 = 1;
  const bool two = !whole && dx_dtype == MOE_DTYPE_BF16;       // parts of dz in dx's product
  if (dx && dw) {
    if (whole) return launch_grads<1, 1>(gx, gw, b, di.cus, st);
    return two ? launch_grads<2, 3>(gx, gw, b, di.cus, st) : launch_grads<3, 3>(gx, gw, b, di.cus, st);
  }
  if (dbias) {
    hipLaunchKernelGGL(k_linear_dbias, dim3((R + 63) / 64), dim3(256), 0, st, b);
    HIP_TRY(hipGetLastError());
  }
  if (dx) {
    if (whole) return launch_product<0, 1, 1, 0>(gx, di.cus, st);
    return two ? launch_product<0, 1, 2, 0>(gx, di.cus, st) : launch_product<0, 1, 3, 0>(gx, di.cus, st);
  }
  if (dw) return whole ? launch_product<1, 1, 1, 0>(gw, di.cus, st) : launch_product<1, 1, 3, 0>(gw, di.cus, st);
  return MOE_OK;
}

}  // extern "C"
