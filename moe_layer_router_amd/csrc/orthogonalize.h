// Newton-Schulz orthogonalisation of the updates of weight matrices.
//
// For each matrix U (M x N), taken on its short side (transposed if M > N),
// X of m rows and n >= m columns:
//   X_0 = U / (|U|_F + eps)
//   A = X X^T,  B = b A + c A^2,  X' = a X + B X          (per step)
// i.e. every singular value s of X_0 goes through a s + b s^3 + c s^5 and
// the singular vectors stay.  A and B are symmetric: their products are
// formed on and above the diagonal and mirrored.
//
// Precision.  X is held as two FP16 parts (hi + lo, 22 bits) of 2^12 X, A and
// B as FP16 of 2^12 times their values (|X|, |A|, |B| stay below 3, and FP16
// reaches 2^16; a normal FP16 number goes down to 2^-26 of the scale), the
// products use the hi parts with fp32 accumulation, and a X is added from
// both parts in fp32.  One FP16 product has 2^-11 relative rounding per
// operand, eight times less than BF16: over spectra from flat to 1/r^2 the
// result is within 1e-3 of fp64 beside the output's own BF16 rounding
// (1.7e-3), where BF16 products are 1e-2 and, with X held in BF16 alone, up to
// 1.6e-1 off (small singular values are lost in the rounding of the large
// ones, which is why the lo part is kept).
//
// Layout.  Rows and columns are padded with zeros to multiples of 64: hi, lo
// [mp][np], A, B [mp][mp], and the transposed hi part ht [np][mp] (two, read
// and written in turn), so that each of the three products has both operands
// with contiguous K: X X^T from hi and hi, A A from A and A, B X from B and
// ht.
//
// Narrow matrices (m <= 64) go another way.  With G = X X^T and P = a + b G + c
// G^2 a step is X' = P X, G' = P G P: the whole iteration runs on m x m
// matrices, and y = Q X_0 with Q the product of the P.  G squares the
// spread of the singular values, which fp64 carries (its products are cheap
// at this size, 17 of m x m); the matrix itself is read twice and written
// once, in three launches.  It is also the accurate way for them: a matrix of
// few rows does not average the roundings of FP16 products (up to 1e-2 at m
// <= 8, below 2.3e-3 from m = 64 on).
#pragma once
#include "device_common.h"

namespace moe {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));

constexpr float kOrthScale = 4096.0f;
constexpr int kOrthPad = 64;
constexpr int kOrthNormParts = 64;       // partial sums of squares per matrix

struct OrthArgs {
  const void* u;             // [batch][M][N] fp32 or BF16
  int M, N, m, n, mp, np;
  int tall;                  // M > N: X is the transpose
  float eps;
  double* part;              // [batch][kOrthNormParts]
  uint16_t* hi;              // [batch][mp][np]
  uint16_t* lo;
  uint16_t* ht;              // [batch][np][mp]
};

template <int BF>
DEV float orth_ld(const void* u, size_t i) {
  return BF ? bf16_to_f32(static_cast<const uint16_t*>(u)[i]) : static_cast<const float*>(u)[i];
}

// Sum of squares in fp64 (fp32 squares of small gradients would underflow):
// workgroup (p, b) sums part p of matrix b.
template <int BF>
__global__ void __launch_bounds__(256) k_orth_norm(OrthArgs a) {
  __shared__ double red[256];
  const size_t total = (size_t)a.M * a.N, per = (total + kOrthNormParts - 1) / kOrthNormParts;
  const size_t i0 = blockIdx.x * per, i1 = i0 + per < total ? i0 + per : total;
  const size_t base = (size_t)blockIdx.y * total;
  double s = 0;
#pragma unroll 4
  for (size_t i = i0 + threadIdx.x; i < i1; i += 256) {
    const double v = orth_ld<BF>(a.u, base + i);
    s += v * v;
  }
  red[threadIdx.x] = s;
  __syncthreads();
  for (int h = 128; h > 0; h >>= 1) {
    if ((int)threadIdx.x < h) red[threadIdx.x] += red[threadIdx.x + h];
    __syncthreads();
  }
  if (threadIdx.x == 0) a.part[(size_t)blockIdx.y * kOrthNormParts + blockIdx.x] = red[0];
}

// X_0 as hi, lo and ht, zeros in the padding: workgroup (x, y, b) does the
// 64 x 64 tile (y, x) of U's padded matrix b.
template <int BF>
__global__ void __launch_bounds__(256) k_orth_load(OrthArgs a) {
  __shared__ float tile[64][65];
  __shared__ float s_scale;
  if (threadIdx.x == 0) {
    double s = 0;
    for (int i = 0; i < kOrthNormParts; ++i) s += a.part[(size_t)blockIdx.z * kOrthNormParts + i];
    // (a zero matrix stays zero: the scale is finite)
    const double sc = (double)kOrthScale / (sqrt(s) + (double)a.eps);
    s_scale = sc < 3e38 ? (float)sc : sc == sc ? 3e38f : (float)sc;
  }
  __syncthreads();
  const float sc = s_scale;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64, tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  const size_t ub = (size_t)blockIdx.z * a.M * a.N;
  const int ldd = a.tall ? a.mp : a.np;      // U's padded row length
  const size_t xb = (size_t)blockIdx.z * a.mp * a.np;
  uint16_t* direct = a.tall ? a.ht : a.hi;   // in U's own orientation
#pragma unroll 4
  for (int i = ty; i < 64; i += 4) {
    const int r = r0 + i, c = c0 + tx;
    const float v = r < a.M && c < a.N ? orth_ld<BF>(a.u, ub + (size_t)r * a.N + c) * sc : 0.f;
    tile[i][tx] = v;
    const _Float16 h = (_Float16)v;
    const size_t o = xb + (size_t)r * ldd + c;
    direct[o] = __builtin_bit_cast(uint16_t, h);
    if (!a.tall) a.lo[o] = __builtin_bit_cast(uint16_t, (_Float16)(v - (float)h));
  }
  __syncthreads();
  const int ldt = a.tall ? a.np : a.mp;
#pragma unroll 4
  for (int i = ty; i < 64; i += 4) {
    const int r = r0 + tx, c = c0 + i;       // element (r, c) of U at row c of the transpose
    const float v = tile[tx][i];
    const _Float16 h = (_Float16)v;
    const size_t o = xb + (size_t)c * ldt + r;
    (a.tall ? a.hi : a.ht)[o] = __builtin_bit_cast(uint16_t, h);
    if (a.tall) a.lo[o] = __builtin_bit_cast(uint16_t, (_Float16)(v - (float)h));
  }
}

// ------------------------------------------------------------------ products
enum { ORTH_GRAM = 0, ORTH_POLY = 1, ORTH_STEP = 2, ORTH_LAST = 3 };

// C[i][j] = sum_k P[i][k] Q[j][k] for each matrix of a batch, P [rows][ld], Q
// [cols][ld] FP16, K a multiple of 64, and what follows it:
//   GRAM   A = s C                             (symmetric)
//   POLY   B = c1 A + s C                      (symmetric)
//   STEP   X' = c1 X + s C as hi, lo, ht_out
//   LAST   the result: (c1 X + s C) / 2^12 as BF16 in U's orientation
struct OrthGemm {
  const uint16_t* p;
  const uint16_t* q;
  size_t p_stride, q_stride;           // elements between matrices
  uint32_t p_bytes, q_bytes;           // of one matrix
  int ldp, ldq;
  int rows, cols, K;                   // padded sizes
  int ti, tj, tiles;                   // tiles of rows and columns, tiles per matrix
  int total;                           // tiles of all matrices
  float c1, s;
  uint16_t* c;                         // GRAM: A; POLY: B
  const uint16_t* a;                   // POLY: A
  uint16_t* hi;
  uint16_t* lo;
  uint16_t* ht;
  uint16_t* y;                         // LAST: [batch][M][N]
  int m, n, tall;
};

DEV v4f mfma_f16(const v8h& a, const v8h& b, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
DEV uint32_t h_bits(float v) { return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v); }
DEV float h_val(uint32_t b) { return (float)__builtin_bit_cast(_Float16, (uint16_t)b); }

// Tile t of the n x n tiles on and above the diagonal: (i, j), i <= j, ordered
// by j.
DEV void orth_tri(int t, int* i, int* j) {
  int c = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
  while (c * (c + 1) / 2 > t) --c;
  while ((c + 1) * (c + 2) / 2 <= t) ++c;
  *j = c;
  *i = t - c * (c + 1) / 2;
}

// WM x WN waves, each MI x NJ subtiles of 16 x 16: a tile of 16 MI WM rows and
// 16 NJ WN columns, in steps of 64 K.
template <int WM, int WN, int MI, int NJ>
struct OrthTile {
  static constexpr int kRows = 16 * MI * WM, kCols = 16 * NJ * WN, kThreads = 64 * WM * WN;
  static constexpr int kStage = (kRows + kCols) * 128;        // bytes of a 64-K step
  static constexpr int kLds = 2 * kStage;
};

// Both operands' tiles of a step go straight to LDS (16-byte buffer loads,
// rows past the end read as zero), two stages: the next step's loads are in
// flight during a step's products, one barrier per step.  LDS rows are 128
// bytes, chunk c (16 bytes, K 8c .. 8c+7) of row r at chunk c ^ ((r ^ r/8) % 8),
// so that the 16 rows of an operand read fall in distinct banks.
template <int WM, int WN, int MI, int NJ, int MODE>
__global__ void __launch_bounds__(64 * WM * WN) k_orth_gemm(OrthGemm g) {
  using TL = OrthTile<WM, WN, MI, NJ>;
  constexpr int NW = WM * WN, PP = TL::kRows / 8 / NW, QP = TL::kCols / 8 / NW;   // 1 KB pieces per wave
  static_assert(TL::kRows % (8 * NW) == 0 && TL::kCols % (8 * NW) == 0, "whole pieces per wave");
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, gq = lane >> 4, wm = w / WN, wn = w % WN;

  // XCD x (workgroup ids go round-robin) takes a contiguous range of tiles
  const int per = (g.total + 7) / 8;
  const int t = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
  if (t >= g.total || (int)(blockIdx.x / 8) >= per) return;
  const int mat = t / g.tiles;
  int i0, j0;
  if (MODE == ORTH_GRAM || MODE == ORTH_POLY) {
    orth_tri(t % g.tiles, &i0, &j0);
  } else {
    i0 = t % g.tiles % g.ti;
    j0 = t % g.tiles / g.ti;
  }
  const bool mirror = (MODE == ORTH_GRAM || MODE == ORTH_POLY) && i0 != j0;
  i0 *= TL::kRows;
  j0 *= TL::kCols;
  const rsrc_t pr = make_rsrc(g.p + mat * g.p_stride, g.p_bytes), qr = make_rsrc(g.q + mat * g.q_stride, g.q_bytes);

  uint32_t poff[PP], qoff[QP];
#pragma unroll
  for (int q = 0; q < PP; ++q) {
    const int r = 8 * (q * NW + w) + (lane >> 3), c = (lane & 7) ^ ((r ^ (r >> 3)) & 7);
    poff[q] = (uint32_t)(i0 + r) * (uint32_t)g.ldp * 2 + 16 * c;
  }
#pragma unroll
  for (int q = 0; q < QP; ++q) {
    const int r = 8 * (q * NW + w) + (lane >> 3), c = (lane & 7) ^ ((r ^ (r >> 3)) & 7);
    qoff[q] = (uint32_t)(j0 + r) * (uint32_t)g.ldq * 2 + 16 * c;
  }
  const int steps = g.K / 64;
  auto load = [&](int s) {
    char* st = lds + (s & 1) * TL::kStage;
#pragma unroll
    for (int q = 0; q < PP; ++q) buf_ld16_lds(pr, st + (q * NW + w) * 1024, poff[q], (uint32_t)s * 128);
#pragma unroll
    for (int q = 0; q < QP; ++q)
      buf_ld16_lds(qr, st + TL::kRows * 128 + (q * NW + w) * 1024, qoff[q], (uint32_t)s * 128);
  };
  // operand reads: row r's chunk 4 kh + gq
  auto off = [&](int r, int kh) { return r * 128 + (((4 * kh + gq) ^ ((r ^ (r >> 3)) & 7)) << 4); };

  v4f acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  load(0);
  for (int s = 0; s < steps; ++s) {
    barrier_vmcnt<0>();                            // step s has landed, and every wave is past step s - 1
    if (s + 1 < steps) load(s + 1);
    const char* pt = lds + (s & 1) * TL::kStage;
    const char* qt = pt + TL::kRows * 128;
#pragma unroll
    for (int kh = 0; kh < 2; ++kh) {
      v8h qf[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        qf[j] = __builtin_bit_cast(v8h, ld16(qt + off(16 * NJ * wn + 16 * j + c16, kh)));
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const v8h pf = __builtin_bit_cast(v8h, ld16(pt + off(16 * MI * wm + 16 * i + c16, kh)));
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = mfma_f16(qf[j], pf, acc[i][j]);
      }
    }
  }

  // lane: row i0 + 16 MI wm + 16 i + c16, columns j0 + 16 NJ wn + 16 j + 4 gq + v
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int r = i0 + 16 * MI * wm + 16 * i + c16, c = j0 + 16 * NJ * wn + 16 * j + 4 * gq;
      if (r >= g.rows || c >= g.cols) continue;    // (c is a multiple of 4, cols of 64)
      if (MODE == ORTH_GRAM || MODE == ORTH_POLY) {
        const size_t o = mat * (size_t)g.rows * g.rows + (size_t)r * g.rows + c;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = g.s * acc[i][j][e];
        if (MODE == ORTH_POLY) {
          const v2u q = *reinterpret_cast<const v2u*>(g.a + o);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(g.c1, h_val(q[e >> 1] >> (16 * (e & 1))), v[e]);
        }
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = h_bits(v[e]);
        *reinterpret_cast<v2u*>(g.c + o) = v2u{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
        if (mirror) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            g.c[mat * (size_t)g.rows * g.rows + (size_t)(c + e) * g.rows + r] = (uint16_t)h[e];
        }
      } else {
        const size_t o = mat * (size_t)g.rows * g.cols + (size_t)r * g.cols + c;
        const v2u xh = *reinterpret_cast<const v2u*>(g.hi + o), xl = *reinterpret_cast<const v2u*>(g.lo + o);
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int sh = 16 * (e & 1);
          v[e] = __builtin_fmaf(g.c1, h_val(xh[e >> 1] >> sh) + h_val(xl[e >> 1] >> sh), g.s * acc[i][j][e]);
        }
        if (MODE == ORTH_STEP) {
          uint32_t h[4], l[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            h[e] = h_bits(v[e]);
            l[e] = h_bits(v[e] - h_val(h[e]));
          }
          *reinterpret_cast<v2u*>(g.hi + o) = v2u{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
          *reinterpret_cast<v2u*>(g.lo + o) = v2u{l[0] | (l[1] << 16), l[2] | (l[3] << 16)};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            g.ht[mat * (size_t)g.rows * g.cols + (size_t)(c + e) * g.rows + r] = (uint16_t)h[e];
        } else if (r < g.m) {
          const size_t yb = mat * (size_t)g.m * g.n;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < g.n)
              g.y[yb + (g.tall ? (size_t)(c + e) * g.m + r : (size_t)r * g.n + c + e)] =
                  (uint16_t)f32_to_bf16_rne(v[e] * (1.0f / kOrthScale));
        }
      }
    }
}

// ------------------------------------------------------------------- narrow
constexpr int kOrthNarrow = 64;          // largest m of the narrow kernels
constexpr int kOrthSlabs = 16;           // partial Gram matrices per matrix
constexpr int kOrthSlabCols = 32;        // columns of X per pass of a slab
constexpr int kOrthApply = 128;          // columns of X per workgroup of the last kernel

struct OrthNarrow {
  const void* u;             // [batch][M][N]
  int m, n, tall, slabs, steps;
  float eps;
  float co[32][3];
  double* part;              // [batch][slabs][MP][MP]
  float* q;                  // [batch][MP][MP]: Q / (|U|_F + eps)
  uint16_t* y;
};

// Element (i, j) of X's matrix b, before it is normalised.
template <int BF>
DEV float orth_x(const OrthNarrow& a, size_t base, int i, int j) {
  return orth_ld<BF>(a.u, base + (a.tall ? (size_t)j * a.m + i : (size_t)i * a.n + j));
}

// Workgroup (slab, b): the slab's share of U U^T (U^T U if tall) in fp64; 16 x
// 16 threads, R x R elements each.
template <int BF, int MP>
__global__ void __launch_bounds__(256) k_orth_gram64(OrthNarrow a) {
  constexpr int R = MP / 16, KC = kOrthSlabCols;
  __shared__ double xs[KC][MP + 1];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int per = (a.n + a.slabs - 1) / a.slabs, j0 = blockIdx.x * per, j1 = min(a.n, j0 + per);
  const size_t base = (size_t)blockIdx.y * a.m * a.n;
  double acc[R][R];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < R; ++c) acc[r][c] = 0;
  for (int jb = j0; jb < j1; jb += KC) {
    for (int e = threadIdx.x; e < KC * MP; e += 256) {        // (memory order: along i if tall, else along j)
      const int i = a.tall ? e % MP : e / KC, c = a.tall ? e / MP : e % KC;
      xs[c][i] = i < a.m && jb + c < j1 ? (double)orth_x<BF>(a, base, i, jb + c) : 0.0;
    }
    __syncthreads();
#pragma unroll 4
    for (int c = 0; c < KC; ++c) {
      double p[R], q[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        p[r] = xs[c][ty * R + r];
        q[r] = xs[c][tx + 16 * r];
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int s = 0; s < R; ++s) acc[r][s] = __builtin_fma(p[r], q[s], acc[r][s]);
    }
    __syncthreads();
  }
  double* out = a.part + ((size_t)blockIdx.y * a.slabs + blockIdx.x) * MP * MP;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int s = 0; s < R; ++s) out[(ty * R + r) * MP + tx + 16 * s] = acc[r][s];
}

// LDS matrices of the iteration: [MP][MP + 1] doubles.
template <int MP>
struct OrthSq {
  static constexpr int kLd = MP + 1, kSize = MP * kLd;
  static constexpr int kLds = 4 * kSize * 8;
};
// This thread's R x R elements of p q.
template <int MP, int R>
DEV void orth_mul64(const double* p, const double* q, int tx, int ty, double (&acc)[R][R]) {
  constexpr int LD = OrthSq<MP>::kLd;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < R; ++c) acc[r][c] = 0;
#pragma unroll 4
  for (int k = 0; k < MP; ++k) {
    double pv[R], qv[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      pv[r] = p[(ty * R + r) * LD + k];
      qv[r] = q[k * LD + tx + 16 * r];
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < R; ++c) acc[r][c] = __builtin_fma(pv[r], qv[c], acc[r][c]);
  }
}

// One workgroup per matrix: G from its slabs, the norm from G's trace, the
// steps, and Q.
template <int MP>
__global__ void __launch_bounds__(256) k_orth_iter64(OrthNarrow a) {
  constexpr int R = MP / 16, LD = OrthSq<MP>::kLd;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  double* G = reinterpret_cast<double*>(lds);
  double* P = G + OrthSq<MP>::kSize;
  double* Q = P + OrthSq<MP>::kSize;
  double* T = Q + OrthSq<MP>::kSize;
  __shared__ double s_inv;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const double* part = a.part + (size_t)blockIdx.x * a.slabs * MP * MP;
  for (int e = threadIdx.x; e < MP * MP; e += 256) {
    double s = 0;
    for (int p = 0; p < a.slabs; ++p) s += part[(size_t)p * MP * MP + e];
    G[e / MP * LD + e % MP] = s;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double tr = 0;
    for (int i = 0; i < MP; ++i) tr += G[i * LD + i];
    s_inv = 1.0 / (sqrt(tr) + (double)a.eps);
  }
  __syncthreads();
  const double inv = s_inv, inv2 = inv * inv;
  for (int e = threadIdx.x; e < MP * MP; e += 256) G[e / MP * LD + e % MP] *= inv2;
  __syncthreads();
  double acc[R][R];
  auto put = [&](double* dst) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < R; ++c) dst[(ty * R + r) * LD + tx + 16 * c] = acc[r][c];
  };
  for (int k = 0; k < a.steps; ++k) {
    const double ca = a.co[k][0], cb = a.co[k][1], cc = a.co[k][2];
    orth_mul64<MP, R>(G, G, tx, ty, acc);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < R; ++c) {
        const int i = ty * R + r, j = tx + 16 * c;
        acc[r][c] = cc * acc[r][c] + cb * G[i * LD + j] + (i == j ? ca : 0.0);
      }
    put(P);
    if (k == 0) put(Q);
    __syncthreads();
    if (k > 0) {
      orth_mul64<MP, R>(P, Q, tx, ty, acc);
      __syncthreads();
      put(Q);
    }
    if (k + 1 < a.steps) {
      orth_mul64<MP, R>(P, G, tx, ty, acc);
      put(T);
      __syncthreads();
      orth_mul64<MP, R>(T, P, tx, ty, acc);
      put(G);
    }
    __syncthreads();
  }
  float* out = a.q + (size_t)blockIdx.x * MP * MP;
  for (int e = threadIdx.x; e < MP * MP; e += 256) {
    const double v = Q[e / MP * LD + e % MP] * inv;
    // (a tiny norm's scale past fp32: a zero matrix still gives zero)
    out[e] = v > 3e38 ? 3e38f : v < -3e38 ? -3e38f : (float)v;
  }
}

// y = Q U: one column of X per thread, its m elements in registers, Q through
// the scalar cache (every thread of the grid's matrix reads the same
// element).  A tall matrix's columns are rows in memory: a workgroup's are one
// contiguous run, staged through LDS both ways.
template <int BF, int MP, int TALL>
__global__ void __launch_bounds__(kOrthApply) k_orth_apply(OrthNarrow a) {
  __shared__ float st[TALL ? kOrthApply * (MP + 1) : 1];
  typedef const __attribute__((address_space(4))) float KFloat;
  KFloat* q = (KFloat*)(uintptr_t)(a.q + (size_t)blockIdx.y * MP * MP);
  const int j0 = blockIdx.x * kOrthApply, j = j0 + (int)threadIdx.x;
  const size_t base = (size_t)blockIdx.y * a.m * a.n;
  const int cols = min(kOrthApply, a.n - j0);
  float x[MP];
  if (TALL) {
    for (int e = threadIdx.x; e < cols * a.m; e += kOrthApply)
      st[e / a.m * (MP + 1) + e % a.m] = orth_ld<BF>(a.u, base + (size_t)j0 * a.m + e);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MP; ++i) x[i] = i < a.m && j < a.n ? st[threadIdx.x * (MP + 1) + i] : 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < MP; ++i) x[i] = i < a.m && j < a.n ? orth_ld<BF>(a.u, base + (size_t)i * a.n + j) : 0.f;
  }
  for (int i = 0; i < a.m; ++i) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < MP; ++k) s[k & 3] = __builtin_fmaf(q[i * MP + k], x[k], s[k & 3]);
    const float v = (s[0] + s[1]) + (s[2] + s[3]);
    if (TALL) st[threadIdx.x * (MP + 1) + i] = v;             // (this thread's own row: x is in registers)
    else if (j < a.n) a.y[base + (size_t)i * a.n + j] = (uint16_t)f32_to_bf16_rne(v);
  }
  if (TALL) {
    __syncthreads();
    for (int e = threadIdx.x; e < cols * a.m; e += kOrthApply)
      a.y[base + (size_t)j0 * a.m + e] = (uint16_t)f32_to_bf16_rne(st[e / a.m * (MP + 1) + e % a.m]);
  }
}

}  // namespace moe
