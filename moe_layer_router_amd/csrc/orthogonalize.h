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
// Precision.  The products are FP16 matrix-core products with fp32
// accumulation, on 2^12 times the values of X and A (below 4 and 15, and FP16
// reaches 2^16) and on a I + B itself (its small elements are subnormal FP16
// numbers, which the matrix cores take: 3e-8 beside a), so that the
// accumulators of (a I + B) X hold 2^12 X'.
// X is held as an FP16 part hi and the FP16 rounding lo of what is left, 22 bits:
// the step is X' = (a I + B) hi + a lo, the first term one product, the second
// added in fp32.  One FP16 product has 2^-11 relative rounding per operand, eight
// times less than BF16.  Its roundings in A and B' move singular vectors and
// values a little; those of X would have full rank, and each step lifts what they put
// into directions that U lacks by a, 485-fold in 5 steps: hence lo.  Simulated in
// fp64 with these roundings, 5 steps, the result is within 2.6e-3 of the exact
// iteration for sides from 65 to 2048, spectra from flat to 1/r^2 and exact ranks from 1 on
// (within 1.1e-2 for matrices of one magnitude, whose elements all round alike),
// beside the output's own BF16 rounding (1.7e-3).  With an 8-bit E4M3 lo it is up
// to 6.8e-3 off after 5 steps and 1.5e-1 after 8 (2048 x 7168 of rank 1), for 1 to 4%
// less time; without lo up to 2e-2, with BF16 products 1e-2 to 1.6e-1.
//
// Layout.  Rows and columns are padded with zeros to multiples of 64.  X is kept
// transposed, hi (two, read and written in turn) and lo [np][mp], beside A and
// B' = a I + B [mp][mp]: then A A from A and A and the step, X'^T = X^T B', from hi
// and B' have both operands with contiguous K, and only X X^T has its K along the
// columns, whose tiles are transposed as they are read from LDS.  (With a second
// copy of X in the other orientation no product needs that, but a step then
// stores it, 110 of its 600 us at 8 x 2048 x 7168.)
//
// Narrow matrices (m <= 64) go another way.  With G = X X^T and P = a + b G + c
// G^2 a step is X' = P X, G' = P G P: the whole iteration runs on m x m
// matrices, and y = Q X_0 with Q the product of the P.  G squares the
// spread of the singular values, which fp64 carries (its products are cheap
// at this size, 17 of m x m on the fp64 matrix cores); the matrix itself is read
// twice and written once, in three launches.  It is also the accurate way for them: a matrix of
// few rows does not average the roundings of FP16 products (up to 1e-2 at m
// <= 8, below 2.3e-3 from m = 64 on).
// Where U lacks a direction, G holds rounding of either sign there, and a step
// multiplies it by a^2.  A negative one would grow past 1 after 16 default steps, and P
// with it, without end.  So G starts with 2^-44 on its diagonal: above its
// rounding (about 1e-15) and that of each P G P (2^-53 |P|^2, while the shift has grown as much), it
// stays positive and ends near 1 like any other value.  To the singular values that
// is sqrt(s^2 + 2^-44): those below 2^-22 of the norm, rounding in an fp32 U, are lifted
// 2^22-fold at most, and no other is off by more than 2^-45 / s.
//
// Measured (5 steps).  Large matrices are bound by the matrix cores: 8 x 2048 x
// 7168 takes 4.5 to 4.8 ms, by card, 820 to 875 TFLOP/s, where one large FP16 library
// product reaches 1390: norm 96 us (4.9 TB/s), load 220 (4.3), then per step X X^T 248 + 13
// (its parts), the polynomial 89 + 15, the step 547 (the last 491).  A step's products
// alone take 380 us; its tile ends, where the one workgroup of a CU stores and
// multiplies nothing, the rest.  Small ones are bound by their 17 to 22 dependent
// launches of 4 to 6 us: 8 x 256 x 256 76 us, 256 x 7168 135 us.  Narrow: 16 x 64 x
// 7168 23 + 53 + 32 us, bound by fp64 (its 17 products on one CU each take 2 us at
// the peak rate, 3 here; the last kernel's product 12 of its 32).
#pragma once
#include "device_common.h"
#include "norm.h"

namespace moe {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr float kOrthScale = 4096.0f;
constexpr int kOrthPad = 64;
constexpr int kOrthNormParts = 64;       // partial sums of squares per matrix

struct OrthArgs {
  const void* u;             // [batch][M][N] fp32 or BF16
  int M, N, m, n, mp, np;
  int tall;                  // M > N: X is the transpose
  float eps;
  double* part;              // [batch][kOrthNormParts]
  uint16_t* hi;              // [batch][np][mp]
  uint16_t* lo;
};

DEV uint32_t h_bits(float v) { return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v); }
DEV float h_val(uint32_t b) { return (float)__builtin_bit_cast(_Float16, (uint16_t)b); }
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
// Two values as packed FP16 (one conversion instruction, to nearest even).
DEV uint32_t h_pack(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{lo, hi}), v2h));
}

template <int BF>
DEV float orth_ld(const void* u, size_t i) {
  return BF ? bf16_to_f32(static_cast<const uint16_t*>(u)[i]) : static_cast<const float*>(u)[i];
}

// Sum of squares in fp64 (fp32 squares of small gradients would underflow):
// workgroup (p, b) sums part p of matrix b, 8 elements per thread and load
// where rows of 8 line up.
template <int BF>
__global__ void __launch_bounds__(256) k_orth_norm(OrthArgs a) {
  __shared__ double red[256];
  const size_t total = (size_t)a.M * a.N, per = ((total + kOrthNormParts - 1) / kOrthNormParts + 7) / 8 * 8;
  const size_t i0 = min(blockIdx.x * per, total), i1 = min(i0 + per, total);
  const size_t base = (size_t)blockIdx.y * total;
  double s = 0;
  size_t tail = i0;
  if (total % 8 == 0) {                    // (each matrix, and so each part, starts on 16 bytes)
    tail = i1;
#pragma unroll 4
    for (size_t i = i0 + 8 * threadIdx.x; i < i1; i += 8 * 256) {
      float v[8];
      ln_unpack<BF ? LN_BF16 : LN_F32>(ln_load<BF ? LN_BF16 : LN_F32>(a.u, base + i), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = __builtin_fma((double)v[e], (double)v[e], s);
    }
  }
  for (size_t i = tail + threadIdx.x; i < i1; i += 256) {
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

// X_0 as hi and lo, zeros in the padding: workgroup (x, y, b) does the 64 x 64
// tile (y, x) of U's padded matrix b.
template <int BF>
__global__ void __launch_bounds__(256) k_orth_load(OrthArgs a) {
  static_assert(kOrthNormParts == 64, "one part per lane");
  __shared__ float tile[64][65];
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  double ss = a.part[(size_t)blockIdx.z * kOrthNormParts + tx];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) ss += __shfl_xor(ss, d);
  // (in two factors, as the norm's reciprocal may leave fp32; a zero matrix stays
  // zero, eps being positive)
  int se;
  const float sc = (float)frexp((double)kOrthScale / (sqrt(ss) + (double)a.eps), &se);
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  const size_t ub = (size_t)blockIdx.z * a.M * a.N, xb = (size_t)blockIdx.z * a.mp * a.np;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float v[8];                              // eight rows' loads together
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + ty + 4 * (8 * q + i), c = c0 + tx;
      v[i] = r < a.M && c < a.N ? orth_ld<BF>(a.u, ub + (size_t)r * a.N + c) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[ty + 4 * (8 * q + i)][tx] = ldexpf(v[i], se) * sc;
  }
  __syncthreads();
  // 8 consecutive elements of a row of X^T at a time: column k of the tile, or a row if tall
  const size_t o0 = xb + (a.tall ? (size_t)r0 * a.mp + c0 : (size_t)c0 * a.mp + r0);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int k = (threadIdx.x >> 3) + 32 * q, e0 = 8 * (threadIdx.x & 7);
    v4i h, l;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float x0 = a.tall ? tile[k][e0 + e] : tile[e0 + e][k], x1 = a.tall ? tile[k][e0 + e + 1] : tile[e0 + e + 1][k];
      const uint32_t w = h_pack(x0, x1);
      h[e / 2] = (int)w;
      l[e / 2] = (int)h_pack(x0 - h_val(w & 0xFFFFu), x1 - h_val(w >> 16));
    }
    st16(a.hi + o0 + (size_t)k * a.mp + e0, h);
    st16(a.lo + o0 + (size_t)k * a.mp + e0, l);
  }
}

// ------------------------------------------------------------------ products
enum { ORTH_GRAM = 0, ORTH_POLY = 1, ORTH_STEP = 2, ORTH_LAST = 3 };
constexpr bool orth_sym(int mode) { return mode == ORTH_GRAM || mode == ORTH_POLY; }

// C[i][j] = sum_k P[i][k] Q[j][k] for each matrix of a batch, P [rows][ld], Q
// [cols][ld] FP16 (GRAM: P = Q [K][ld], C[i][j] = sum_k P[k][i] Q[k][j]), K a
// multiple of 64, and what follows it:
//   GRAM   A = s C                                  (symmetric)
//   POLY   B' = c0 I + c1 A + s C                   (symmetric)
//   STEP   X'^T = C + c0 lo as hi and lo
//   LAST   the result: (C + c0 lo) / 2^12 as BF16 in U's orientation
struct OrthGemm {
  const uint16_t* p;
  const uint16_t* q;
  size_t p_stride, q_stride;           // elements between matrices
  uint32_t p_bytes, q_bytes;           // of one matrix
  int ldp, ldq;
  int rows, cols, K;                   // padded sizes
  int tj, tiles;                       // tiles of columns, tiles per matrix
  int full;                            // tiles (of the batch) worked on whole
  int split, rest;                     // the other `rest` tiles: parts along K of each
  float* part;                         // [rest][split][tile] sums of the parts
  float c0, c1, s;
  uint16_t* c;                         // GRAM: A; POLY: B'
  const uint16_t* a;                   // POLY: A
  uint16_t* hi;                        // STEP: of X'
  uint16_t* lo;
  uint16_t* y;                         // LAST: [batch][M][N]
  int m, n, tall;
};

DEV v4f mfma_f16(const v8h& a, const v8h& b, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// WM x WN waves, each 4 x NJ subtiles of 16 x 16: a tile of 64 WM rows and as
// many columns, in steps of 64 K, ST steps in LDS.
template <int WM_, int WN_, int NJ_, int ST_>
struct OrthTile {
  static constexpr int WM = WM_, WN = WN_, NJ = NJ_, ST = ST_, NW = WM * WN, kThreads = 64 * NW, kSide = 64 * WM;
  static constexpr int kStage = 2 * kSide * 128;                        // bytes of a step's operands
  static constexpr int kLds = ST * kStage;
  static constexpr size_t kPart = (size_t)kSide * kSide;                // fp32 sums of one part
  static_assert(16 * NJ * WN == kSide && NJ % 2 == 0, "square tiles");
};

// Tile t of the tiles on and above the diagonal: (i, j), i <= j, by j.
DEV void orth_tri(int t, int* i, int* j) {
  int c = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
  while (c * (c + 1) / 2 > t) --c;
  while ((c + 1) * (c + 2) / 2 <= t) ++c;
  *j = c;
  *i = t - c * (c + 1) / 2;
}

// Tile t of the batch: its matrix and its first row and column; whether its
// mirror image is stored too.
template <class TL, int MODE>
DEV bool orth_tile(const OrthGemm& g, int t, int* mat, int* i0, int* j0) {
  *mat = t / g.tiles;
  const int l = t % g.tiles;
  int i, j;
  if (orth_sym(MODE)) {
    orth_tri(l, &i, &j);
  } else {
    i = l / g.tj;
    j = l % g.tj;
  }
  *i0 = i * TL::kSide;
  *j0 = j * TL::kSide;
  return orth_sym(MODE) && i < j;
}

// X's tile in memory, by 32-bit offsets into a matrix's buffer (half the
// registers of addresses): element offset of this lane's 4 rows x 8 columns, but
// for i rows and 32 p columns.  What a wave has past the end of the matrix is
// never stored, and read at the matrix's last rows and columns.
template <class TL>
DEV uint32_t orth_at(const OrthGemm& g, int i0, int j0, int w, int lane, int p) {
  const int r0 = min(i0 + 64 * (w / TL::WN), g.rows - 64);
  const int c0 = min(j0 + 16 * TL::NJ * (w % TL::WN) + 32 * p, g.cols - 32) - 32 * p;
  return (uint32_t)(r0 + 4 * (lane & 15)) * (uint32_t)g.cols + (uint32_t)(c0 + 8 * (lane >> 4));
}
DEV uint32_t orth_row(const OrthGemm& g, int i, int p) { return (uint32_t)(i * g.cols + 32 * p); }
template <typename T>
DEV rsrc_t orth_rsrc(const OrthGemm& g, T* x, int mat) {
  const size_t n = (size_t)g.rows * g.cols;
  return make_rsrc(x + mat * n, (uint32_t)(n * sizeof(T)));
}

// The lo parts of the elements that orth_store finishes, read ahead of it.
template <class TL, int MODE>
DEV void orth_lo(const OrthGemm& g, int mat, int i0, int j0, int w, int lane, int p, v4i (&lq)[4]) {
  if (orth_sym(MODE)) return;
  const uint32_t o = orth_at<TL>(g, i0, j0, w, lane, p);
  const rsrc_t lo = orth_rsrc(g, g.lo, mat);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    lq[i] = buf_ld16(lo, 2 * o, 2 * orth_row(g, i, p));
}

// GRAM: a wave's sums acc[i][j][v] are row 64 wm + 16 i + c16 and column 16 NJ wn +
// 16 j + 4 gq + v of its tile.  Rows are stored in 8-byte pieces; for the mirror
// image four lanes exchange their rows 16 i + (4 lanes) for four consecutive ones
// each, and columns are stored in 8-byte pieces, 128 bytes at a time.
DEV uint32_t quad_swap1(uint32_t v) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true); }
DEV uint32_t quad_swap2(uint32_t v) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true); }
template <class TL>
DEV void orth_store_gram(const OrthGemm& g, int mat, int i0, int j0, bool mirror, int w, int lane, int p,
                         const v4f (&acc)[4][2]) {
  const int c16 = lane & 15, gq = lane >> 4;
  const int r0 = i0 + 64 * (w / TL::WN), c0 = j0 + 16 * TL::NJ * (w % TL::WN) + 32 * p;
  if (r0 >= g.rows || c0 >= g.cols) return;        // (as in orth_store)
  uint16_t* a = g.c + (size_t)mat * g.rows * g.cols;
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    const int c = c0 + 16 * d + 4 * gq;
    uint32_t x[4][2];                              // rows 16 i + c16, columns c + 2 h and c + 2 h + 1
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) x[i][h] = h_pack(g.s * acc[i][d][2 * h], g.s * acc[i][d][2 * h + 1]);
      *reinterpret_cast<v2u*>(a + (size_t)(r0 + 16 * i + c16) * g.cols + c) = v2u{x[i][0], x[i][1]};
    }
    if (!mirror) continue;
    const bool b0 = lane & 1, b1 = lane & 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // 4 x 4 transpose of (i, lane % 4): by bit 0, then by bit 1 of both
      uint32_t y[4] = {x[0][h], x[1][h], x[2][h], x[3][h]};
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const uint32_t t = quad_swap1(b0 ? y[i] : y[i + 1]);
        if (b0) y[i] = t; else y[i + 1] = t;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t t = quad_swap2(b1 ? y[i] : y[i + 2]);
        if (b1) y[i] = t; else y[i + 2] = t;
      }
      // now rows 16 (lane % 4) + 4 (c16 / 4) + i
      const int r = r0 + 16 * (lane & 3) + (c16 & 12);
      *reinterpret_cast<v2u*>(a + (size_t)(c + 2 * h) * g.rows + r) =
          v2u{__builtin_amdgcn_perm(y[1], y[0], 0x05040100), __builtin_amdgcn_perm(y[3], y[2], 0x05040100)};
      *reinterpret_cast<v2u*>(a + (size_t)(c + 2 * h + 1) * g.rows + r) =
          v2u{__builtin_amdgcn_perm(y[1], y[0], 0x07060302), __builtin_amdgcn_perm(y[3], y[2], 0x07060302)};
    }
  }
}

// Else acc[i][j][v] is row 64 wm + 4 c16 + i and column 16 NJ wn + 32 (j / 2) + 8 gq +
// 4 (j % 2) + v of the tile (the operands are brought to LDS in that order).  A
// lane then holds 8 consecutive columns of a row and 4 consecutive rows of a
// column, and both orientations are stored straight from registers: rows in
// 16-byte pieces, 64 bytes at a time, columns (the mirror image, and a result
// whose orientation is the other) in 8-byte pieces, 128 bytes at a time.  This
// stores the columns of j = 2 p and 2 p + 1.  (With 64 columns alternating in the
// same way a row has 128 bytes in two stores: slower, 4555 -> 4640 us for 8 x 2048
// x 7168, measured with a lo of 8 bits.)
template <class TL, int MODE>
DEV void orth_store(const OrthGemm& g, int mat, int i0, int j0, bool mirror, int w, int lane, int p,
                    const v4f (&acc)[4][2], const v4i (&lq)[4]) {
  if (MODE == ORTH_GRAM) return orth_store_gram<TL>(g, mat, i0, j0, mirror, w, lane, p, acc);
  const int c16 = lane & 15, gq = lane >> 4;
  const int r0 = i0 + 64 * (w / TL::WN), c0 = j0 + 16 * TL::NJ * (w % TL::WN) + 32 * p;
  if (r0 >= g.rows || c0 >= g.cols) return;        // (whole waves: rows and cols are multiples of 64)
  const int rb = r0 + 4 * c16, c = c0 + 8 * gq;
  const uint32_t x = orth_at<TL>(g, i0, j0, w, lane, p);
  const rsrc_t hi_r = orth_rsrc(g, g.hi, mat), lo_r = orth_rsrc(g, g.lo, mat);
  const size_t sq = (size_t)mat * g.rows * g.cols, yb = (size_t)mat * g.m * g.n;
  float v[4][8];                                   // this lane's 4 rows x 8 columns
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const size_t o = sq + (size_t)(rb + i) * g.cols + c;
    const float scale = MODE == ORTH_LAST ? 1.0f / kOrthScale : orth_sym(MODE) ? g.s : 1.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = scale * acc[i][e >> 2][e & 3];
    if (MODE == ORTH_POLY) {
      const v4i q = ld16(g.a + o);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[i][e] = __builtin_fmaf(g.c1, h_val((uint32_t)q[e >> 1] >> (16 * (e & 1))), v[i][e]);
        if (c + e == rb + i) v[i][e] += g.c0;
      }
    }
    if (!orth_sym(MODE)) {
      const float c0 = g.c0 * scale;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int word = lq[i][e >> 1];            // (a bit cast of the vector's element itself reads element 0)
        v[i][e] = __builtin_fmaf(c0, (float)__builtin_bit_cast(v2h, word)[e & 1], v[i][e]);
      }
    }
    if (MODE == ORTH_LAST) {
      if (g.tall && rb + i < g.n) {
        uint16_t* y = g.y + yb + (size_t)(rb + i) * g.m + c;
        if (c + 8 <= g.m && g.m % 8 == 0) {        // (rows of y start on 16 bytes)
          st16(y, v4i{(int)bf16x2_rne(v[i][0], v[i][1]), (int)bf16x2_rne(v[i][2], v[i][3]),
                      (int)bf16x2_rne(v[i][4], v[i][5]), (int)bf16x2_rne(v[i][6], v[i][7])});
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < g.m) y[e] = (uint16_t)f32_to_bf16_rne(v[i][e]);
        }
      }
      continue;
    }
    const v4i hw = v4i{(int)h_pack(v[i][0], v[i][1]), (int)h_pack(v[i][2], v[i][3]), (int)h_pack(v[i][4], v[i][5]),
                       (int)h_pack(v[i][6], v[i][7])};
    if (orth_sym(MODE)) st16(g.c + o, hw);
    if (MODE == ORTH_STEP) {
      float l[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int word = hw[e >> 1];
        l[e] = v[i][e] - (float)__builtin_bit_cast(v2h, word)[e & 1];
      }
      const v4i lw = v4i{(int)h_pack(l[0], l[1]), (int)h_pack(l[2], l[3]), (int)h_pack(l[4], l[5]),
                         (int)h_pack(l[6], l[7])};
      // past the caches where there is more of X' than they hold (the large
      // tiles), so that it leaves the operands of the running products in the L2
      constexpr int kAux = TL::kSide >= 256 ? 2 : 0;
      __builtin_amdgcn_raw_buffer_store_b128(hw, hi_r, (int)(2 * x), (int)(2 * orth_row(g, i, p)), kAux);
      __builtin_amdgcn_raw_buffer_store_b128(lw, lo_r, (int)(2 * x), (int)(2 * orth_row(g, i, p)), kAux);
    }
  }
  if (mirror || (MODE == ORTH_LAST && !g.tall)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (MODE == ORTH_LAST) {
        if (c + e >= g.m) continue;
        uint16_t* y = g.y + yb + (size_t)(c + e) * g.n + rb;
        if (rb + 4 <= g.n && g.n % 4 == 0) {
          *reinterpret_cast<v2u*>(y) = v2u{bf16x2_rne(v[0][e], v[1][e]), bf16x2_rne(v[2][e], v[3][e])};
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (rb + i < g.n) y[i] = (uint16_t)f32_to_bf16_rne(v[i][e]);
        }
      } else {
        *reinterpret_cast<v2u*>(g.c + sq + (size_t)(c + e) * g.rows + rb) =
            v2u{h_pack(v[0][e], v[1][e]), h_pack(v[2][e], v[3][e])};
      }
    }
  }
}

// The operands' tiles of a step go straight to LDS (16-byte buffer loads, rows
// past the end read as zero), ST stages, one barrier per step.  An LDS row is
// 128 bytes (64 K), its 16-byte chunk c at c ^ ((row ^ row / 8) % 8), so that the
// 16 rows of an operand read fall in distinct banks.
DEV int orth_swz(int r) { return (r ^ (r >> 3)) & 7; }

// GRAM's tiles: an LDS row is one K of the tile's kSide columns.  An operand is
// read with the transposing load: lane l of 16 hands in the address of 8 bytes,
// columns 4 (l % 4) .. + 3 of row l / 4, and gets the 4 rows of column l.  Its 32-byte
// chunk c is at c ^ orth_swz_t(row), so that the rows of 32 lanes, 0 .. 3 and 8 .. 11
// (or 4 more, 16 more), fall in distinct banks.
typedef short v4s __attribute__((ext_vector_type(4)));
template <class TL>
DEV int orth_swz_t(int r) {
  if (TL::kSide == 64) return ((r >> 1) & 1) | ((r >> 2) & 2);      // (two rows in the banks' 256 bytes)
  return (r & 3) | ((r >> 1) & 4);
}
// (restrict: the compiler does not see which loads into LDS the barriers have
// waited for, and would wait for all of them before each read)
DEV v4s lds_tr16(const char* __restrict__ p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) v4s*)(__attribute__((address_space(3))) char*)const_cast<char*>(p));
}

template <class TL, int MODE>
__global__ void __launch_bounds__(TL::kThreads, 2) k_orth_gemm(OrthGemm g) {
  constexpr int NJ = TL::NJ, NW = TL::NW, PP = TL::kSide / 8 / NW;      // 1 KB pieces per wave and operand
  static_assert(TL::kSide % (8 * NW) == 0, "whole pieces per wave");
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, gq = lane >> 4, wm = w / TL::WN, wn = w % TL::WN;

  // XCD x (workgroup ids go round-robin) takes a contiguous range of the whole
  // tiles; the parts of the others follow
  const int per = (g.full + 7) / 8;
  int t, part = -1;
  if (!orth_sym(MODE) || (int)blockIdx.x < 8 * per) {
    t = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
    if (t >= g.full) return;
  } else {
    part = (int)blockIdx.x - 8 * per;
    t = g.full + part / g.split;
  }
  int mat, i0, j0;
  const bool mirror = orth_tile<TL, MODE>(g, t, &mat, &i0, &j0);
  int s0 = 0, s1 = g.K / 64;
  if (orth_sym(MODE) && part >= 0) {
    const int ks = part % g.split, n = s1;
    s0 = (int)((long)ks * n / g.split);
    s1 = (int)((long)(ks + 1) * n / g.split);
  }
  const rsrc_t pr = make_rsrc(g.p + mat * g.p_stride, g.p_bytes), qr = make_rsrc(g.q + mat * g.q_stride, g.q_bytes);

  constexpr bool TR = MODE == ORTH_GRAM;
  // (not GRAM:) LDS row r of the P tile is row 64 (r / 64) + 4 (r % 16) + r / 16 % 4, of the
  // Q tile column NC (r / NC) + 32 (j / 2) + 8 (x / 4) + 4 (j % 2) + x % 4 with NC
  // = 16 NJ, j = r % NC / 16, x = r % 16 (see orth_store)
  uint32_t poff[PP], qoff[PP];
#pragma unroll
  for (int q = 0; q < PP; ++q) {
    const int r = 8 * (q * NW + w) + (lane >> 3), c = (lane & 7) ^ orth_swz(r);
    if (TR) {
      constexpr int kRow = TL::kSide * 2;          // bytes of a K
      const int o = (q * NW + w) * 1024 + lane * 16, k = o / kRow;
      const int col = 8 * ((o % kRow / 16) ^ (orth_swz_t<TL>(k) << 1));
      // (columns past the end are never stored: the last ones again)
      poff[q] = ((uint32_t)k * g.ldp + min(i0 + col, g.rows - 8)) * 2;
      qoff[q] = ((uint32_t)k * g.ldq + min(j0 + col, g.cols - 8)) * 2;
      continue;
    }
    poff[q] = (uint32_t)(i0 + (r & ~63) + 4 * (r & 15) + ((r >> 4) & 3)) * (uint32_t)g.ldp * 2 + 16 * c;
    const int x = r & 15, j = r % (16 * NJ) / 16;
    const int col = r / (16 * NJ) * (16 * NJ) + 32 * (j >> 1) + 8 * (x >> 2) + 4 * (j & 1) + (x & 3);
    qoff[q] = (uint32_t)(j0 + col) * (uint32_t)g.ldq * 2 + 16 * c;
  }
  auto load = [&](int s, int stage) {
    char* st = lds + stage * TL::kStage;
    // (past the end: the last step again, never read)
    const uint32_t k = (uint32_t)min(s, s1 - 1) * 128 * (TR ? (uint32_t)g.ldp : 1u);
#pragma unroll
    for (int q = 0; q < PP; ++q) {
      buf_ld16_lds(pr, st + (q * NW + w) * 1024, poff[q], k);
      buf_ld16_lds(qr, st + TL::kSide * 128 + (q * NW + w) * 1024, qoff[q], k);
    }
  };

  v4f acc[4][NJ];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  // operand reads: chunk 4 kh + gq of row r0 + 16 i + c16 (r0: the wave's first)
  const int pr0 = 64 * wm, qr0 = 16 * NJ * wn;
  auto frag = [&](const char* op, int r0, int i, int kh) {
    if (TR) {                                      // K 32 kh + 8 gq + 0 .. 7 of column r0 + 16 i + c16
      const int k = 32 * kh + 8 * gq + (c16 >> 2), c = (r0 >> 4) + i;
      const char* a = op + k * (TL::kSide * 2) + ((c ^ orth_swz_t<TL>(k)) << 5) + 8 * (lane & 3);
      const v4s x0 = lds_tr16(a), x1 = lds_tr16(a + 4 * TL::kSide * 2);
      return __builtin_bit_cast(v8h, __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    return lds_ld<v8h>(op, (uint32_t)(r0 + 16 * i + c16) * 128 + (((4 * kh + gq) ^ orth_swz(r0 + 16 * i + c16)) << 4));
  };
  // Every step's first operands are read during the last products of the step
  // before (the last two of its NJ columns' subtiles), behind the barrier: their
  // LDS latency is covered by products.
  constexpr int NL = NJ >= 4 ? 2 : 1;              // column subtiles left behind the barrier, and read ahead
  v8h pf[4], qf[NJ];
  auto read_first = [&](const char* st) {
#pragma unroll
    for (int i = 0; i < 4; ++i) pf[i] = frag(st, pr0, i, 0);
#pragma unroll
    for (int j = 0; j < NL; ++j) qf[j] = frag(st + TL::kSide * 128, qr0, j, 0);
  };
  auto mul = [&](int j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i][j] = mfma_f16(qf[j], pf[i], acc[i][j]);
  };
#pragma unroll
  for (int s = 0; s < TL::ST; ++s) load(s0 + s, s);
  barrier_vmcnt<(TL::ST - 1) * 2 * PP>();          // the first step has landed
  read_first(lds);
  int stage = 0;
  auto halves = [&](const char* st) {              // the step but for the last NL column subtiles
#pragma unroll
    for (int j = NL; j < NJ; ++j) qf[j] = frag(st + TL::kSide * 128, qr0, j, 0);
#pragma unroll
    for (int j = 0; j < NJ; ++j) mul(j);
#pragma unroll
    for (int i = 0; i < 4; ++i) pf[i] = frag(st, pr0, i, 1);
#pragma unroll
    for (int j = 0; j < NJ; ++j) qf[j] = frag(st + TL::kSide * 128, qr0, j, 1);
#pragma unroll
    for (int j = 0; j < NJ - NL; ++j) mul(j);
  };
  for (int s = s0; s < s1 - 1; ++s) {
    halves(lds + stage * TL::kStage);
    const int cur = stage;
    stage = stage == TL::ST - 1 ? 0 : stage + 1;
    // this wave's loads of the next step have landed and its reads of this one
    // are done, and so are every wave's: this stage is free
    barrier_vmcnt<(TL::ST - 2) * 2 * PP>();
    load(s + TL::ST, cur);
    v8h pl[4], ql[NL];
#pragma unroll
    for (int i = 0; i < 4; ++i) pl[i] = pf[i];
#pragma unroll
    for (int j = 0; j < NL; ++j) ql[j] = qf[NJ - NL + j];
    read_first(lds + stage * TL::kStage);
    __builtin_amdgcn_sched_barrier(0);             // (these reads are issued before the products below)
#pragma unroll
    for (int j = 0; j < NL; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i][NJ - NL + j] = mfma_f16(ql[j], pl[i], acc[i][NJ - NL + j]);
    // (and stay in this step: the compiler would move them to the next one's start)
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(pf[i]));
#pragma unroll
    for (int j = 0; j < NL; ++j) asm volatile("" : "+v"(qf[j]));
  }
  // (the first lo parts are read during the last step, as many as the registers
  // beside the operands hold; the others as these are used)
  constexpr int NP = NJ / 2, NA = NP < 2 ? NP : 2;
  v4i lq[NP][4] = {};
#pragma unroll
  for (int p = 0; p < NA; ++p) orth_lo<TL, MODE>(g, mat, i0, j0, w, lane, p, lq[p]);
  halves(lds + stage * TL::kStage);
#pragma unroll
  for (int j = NJ - NL; j < NJ; ++j) mul(j);
  __builtin_amdgcn_sched_barrier(0);               // (the operands' registers are free below)
  // no load into LDS outlives the workgroup (they are older than those of lo)
  wait_vmcnt<orth_sym(MODE) ? 0 : 4 * NA>();
  if (orth_sym(MODE) && part >= 0) {
    v4f* dst = reinterpret_cast<v4f*>(g.part + (size_t)part * TL::kPart) + (size_t)w * 4 * NJ * 64 + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) dst[(i * NJ + j) * 64] = acc[i][j];
    return;
  }
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const v4f a[4][2] = {{acc[0][2 * p], acc[0][2 * p + 1]},
                         {acc[1][2 * p], acc[1][2 * p + 1]},
                         {acc[2][2 * p], acc[2][2 * p + 1]},
                         {acc[3][2 * p], acc[3][2 * p + 1]}};
    orth_store<TL, MODE>(g, mat, i0, j0, mirror, w, lane, p, a, lq[p]);
    if (p + NA < NP) orth_lo<TL, MODE>(g, mat, i0, j0, w, lane, p + NA, lq[p + NA]);
  }
}

// The tiles worked on in parts: a workgroup adds up the parts of 32 columns of
// what one wave of the tile holds (each of its four waves every fourth part,
// then the four sums in order) and finishes them.
template <class TL, int MODE>
__global__ void __launch_bounds__(256) k_orth_join(OrthGemm g) {
  constexpr int NJ = TL::NJ, NP = NJ / 2;
  __shared__ v4f sum[4][8][64];
  const int p = blockIdx.x % NP, w = blockIdx.x / NP % TL::NW, r = blockIdx.x / NP / TL::NW;
  const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
  int mat, i0, j0;
  const bool mirror = orth_tile<TL, MODE>(g, g.full + r, &mat, &i0, &j0);
  v4f acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int k = q; k < g.split; k += 4) {
    const v4f* src =
        reinterpret_cast<const v4f*>(g.part + ((size_t)r * g.split + k) * TL::kPart) + (size_t)w * 4 * NJ * 64 + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[i][0] += src[(i * NJ + 2 * p) * 64];
      acc[i][1] += src[(i * NJ + 2 * p + 1) * 64];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum[q][2 * i][lane] = acc[i][0];
    sum[q][2 * i + 1][lane] = acc[i][1];
  }
  __syncthreads();
  if (q) return;
#pragma unroll
  for (int k = 1; k < 4; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[i][0] += sum[k][2 * i][lane];
      acc[i][1] += sum[k][2 * i + 1][lane];
    }
  v4i lq[4];
  orth_lo<TL, MODE>(g, mat, i0, j0, w, lane, p, lq);
  orth_store<TL, MODE>(g, mat, i0, j0, mirror, w, lane, p, acc, lq);
}

// ------------------------------------------------------------------- narrow
constexpr int kOrthNarrow = 64;          // largest m of the narrow kernels
constexpr int kOrthSlabs = 16;           // partial Gram matrices per matrix
constexpr int kOrthSlabCols = 32;        // columns of X per pass of a slab

struct OrthNarrow {
  const void* u;             // [batch][M][N]
  int m, n, tall, slabs, steps;
  int tiles;                 // of 16 columns, for each wave of the last kernel
  float eps;
  float co[32][3];
  double* part;              // [batch][slabs][MP][MP]
  double* q;                 // [batch][MP][MP]: Q / (|U|_F + eps)
  uint16_t* y;
};

// Element (i, j) of X's matrix b, before it is normalised.
template <int BF>
DEV float orth_x(const OrthNarrow& a, size_t base, int i, int j) {
  return orth_ld<BF>(a.u, base + (a.tall ? (size_t)j * a.m + i : (size_t)i * a.n + j));
}

// Products of the narrow path, by fp64 matrix instructions (16 x 16 x 4): the
// MP x MP result in 16 x 16 tiles, 1 x kB of them per wave, of the workgroup's
// kThreads / 64 waves the first kWi x kWj.
typedef double v4d __attribute__((ext_vector_type(4)));
template <int MP>
struct OrthF64 {
  static constexpr int kB = MP == 64 ? 2 : 1, kWi = MP / 16, kWj = MP / 16 / kB;
  static constexpr int kThreads = kWi * kWj < 4 ? 256 : 64 * kWi * kWj;
  v4d acc[kB];
  int i0, j0, r, kk;                   // the wave's first row and column; this lane's row or column of a tile, and its K
  bool on;
  DEV void init() {
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    on = w < kWi * kWj;
    i0 = 16 * (w / kWj);
    j0 = 16 * kB * (w % kWj);
    r = lane & 15;
    kk = lane >> 4;
    zero();
  }
  DEV void zero() {
#pragma unroll
    for (int b = 0; b < kB; ++b) acc[b] = v4d{0, 0, 0, 0};
  }
  // acc += p q^T over four K: element (i, k) of p at p[i * si + k * sk], and so q
  DEV void mul4(const double* p, const double* q, int si, int sk) {
    const double pv = p[(i0 + r) * si + kk * sk];
    double qv[kB];
#pragma unroll
    for (int b = 0; b < kB; ++b) qv[b] = q[(j0 + 16 * b + r) * si + kk * sk];
#pragma unroll
    for (int b = 0; b < kB; ++b) acc[b] = __builtin_amdgcn_mfma_f64_16x16x4f64(pv, qv[b], acc[b], 0, 0, 0);
  }
  // f(row, column, element) for each element of this lane
  template <class F>
  DEV void each(F&& f) {
    if (!on) return;
#pragma unroll
    for (int b = 0; b < kB; ++b)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        double x = acc[b][v];
        f(i0 + kk + 4 * v, j0 + 16 * b + r, x);
        acc[b][v] = x;
      }
  }
};

// Workgroup (slab, b): the slab's share of U U^T (U^T U if tall) in fp64, in
// passes of kOrthSlabCols columns, the next of which is read during a pass.
// (Rows of a pass in LDS are 17 doubles past a multiple of the 32 that the
// banks hold: neither the writes along a column nor the reads along a row
// collide, but for one.)
template <int BF, int MP>
__global__ void __launch_bounds__(OrthF64<MP>::kThreads) k_orth_gram64(OrthNarrow a) {
  constexpr int NT = OrthF64<MP>::kThreads;
  constexpr int KC = kOrthSlabCols, LD = MP == 16 ? 17 : MP + 17, NE = KC * MP / NT;
  __shared__ double xs[KC * LD];
  const int per = (a.n + a.slabs - 1) / a.slabs, j0 = blockIdx.x * per, j1 = min(a.n, j0 + per);
  const size_t base = (size_t)blockIdx.y * a.m * a.n;
  OrthF64<MP> t;
  t.init();
  float next[NE];
  auto at = [&](int e, int* i, int* c) {           // (memory order: along i if tall, else along j)
    *i = a.tall ? e % MP : e / KC;
    *c = a.tall ? e / MP : e % KC;
  };
  auto load = [&](int jb) {
#pragma unroll
    for (int x = 0; x < NE; ++x) {
      int i, c;
      at(threadIdx.x + NT * x, &i, &c);
      next[x] = i < a.m && jb + c < j1 ? orth_x<BF>(a, base, i, jb + c) : 0.f;
    }
  };
  load(j0);
  for (int jb = j0; jb < j1; jb += KC) {
#pragma unroll
    for (int x = 0; x < NE; ++x) {
      int i, c;
      at(threadIdx.x + NT * x, &i, &c);
      xs[c * LD + i] = (double)next[x];
    }
    __syncthreads();
    load(jb + KC);
    if (t.on) {
#pragma unroll
      for (int c = 0; c < KC; c += 4) t.mul4(xs + c * LD, xs + c * LD, 1, LD);
    }
    __syncthreads();
  }
  double* out = a.part + ((size_t)blockIdx.y * a.slabs + blockIdx.x) * MP * MP;
  t.each([&](int i, int j, double& v) { out[i * MP + j] = v; });
}

// LDS matrices of the iteration: [MP][MP + 2] doubles (a wave's reads down 16
// rows fall in distinct banks).
template <int MP>
struct OrthSq {
  static constexpr int kLd = MP + 2, kSize = MP * kLd;
  static constexpr int kLds = 4 * kSize * 8;
};

// One workgroup per matrix: G from its slabs, the norm from G's trace, the
// steps, and Q.  G, P and Q are polynomials of the first G, so symmetric, and
// they commute: every product is formed as p q^T.  G is kept exactly symmetric: an
// antisymmetric part would grow with G's smallest values (9e-5 of y after 16 steps).
template <int MP>
__global__ void __launch_bounds__(OrthF64<MP>::kThreads) k_orth_iter64(OrthNarrow a) {
  constexpr int LD = OrthSq<MP>::kLd, NT = OrthF64<MP>::kThreads;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  double* G = reinterpret_cast<double*>(lds);
  double* P = G + OrthSq<MP>::kSize;
  double* Q = P + OrthSq<MP>::kSize;
  double* T = Q + OrthSq<MP>::kSize;
  __shared__ double s_inv;
  const double* part = a.part + (size_t)blockIdx.x * a.slabs * MP * MP;
  for (int e = threadIdx.x; e < MP * MP; e += NT) {
    double s = 0;
#pragma unroll 8
    for (int p = 0; p < a.slabs; ++p) s += part[(size_t)p * MP * MP + e];
    G[e / MP * LD + e % MP] = s;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    double tr = (int)threadIdx.x < MP ? G[threadIdx.x * (LD + 1)] : 0.0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) tr += __shfl_xor(tr, d);
    if (threadIdx.x == 0) s_inv = 1.0 / (sqrt(tr) + (double)a.eps);
  }
  __syncthreads();
  const double inv = s_inv, inv2 = inv * inv;
  constexpr double kShift = 1.0 / (1ull << 44);
  for (int e = threadIdx.x; e < MP * MP; e += NT) {
    double& v = G[e / MP * LD + e % MP];
    v = v * inv2 + (e / MP == e % MP ? kShift : 0.0);
  }
  __syncthreads();
  OrthF64<MP> t;
  t.init();
  auto mul = [&](const double* p, const double* q) {
    t.zero();
    if (!t.on) return;
#pragma unroll 4
    for (int k = 0; k < MP; k += 4) t.mul4(p + k, q + k, LD, 1);
  };
  auto put = [&](double* dst) {
    t.each([&](int i, int j, double& v) { dst[i * LD + j] = v; });
  };
  for (int k = 0; k < a.steps; ++k) {
    const double ca = a.co[k][0], cb = a.co[k][1], cc = a.co[k][2];
    mul(G, G);
    t.each([&](int i, int j, double& v) { v = cc * v + cb * G[i * LD + j] + (i == j ? ca : 0.0); });
    put(P);
    if (k == 0) put(Q);
    __syncthreads();
    if (k > 0) {
      mul(P, Q);
      __syncthreads();
      put(Q);
    }
    if (k + 1 < a.steps) {
      mul(P, G);
      put(T);
      __syncthreads();
      mul(T, P);
      t.each([&](int i, int j, double& v) {        // (exactly symmetric: one triangle, mirrored)
        if (i <= j) G[i * LD + j] = G[j * LD + i] = v;
      });
    }
    __syncthreads();
  }
  double* out = a.q + (size_t)blockIdx.x * MP * MP;
  for (int e = threadIdx.x; e < MP * MP; e += NT) out[e] = Q[e / MP * LD + e % MP] * inv;
}

// y = Q U in fp64 (where U lacks a direction Q holds up to 2^22, of which nothing may be
// left in y), by fp64 matrix instructions: a wave keeps 16 rows of Q in registers
// (lane r + 16 kk: row r, K from KS kk on) and goes through tiles of 16 columns of
// X, the next one's loads in flight; waves side by side have the other rows of Q or
// the next columns.  A tall matrix's columns are rows in memory: its product is
// formed transposed, so that 16 lanes store consecutive elements either way.
// (A call on 16 x 64 x 7168 105 us, with vector fp64 and Q through the scalar cache 147.)
template <int BF, int MP, int TALL>
__global__ void __launch_bounds__(256) k_orth_apply(OrthNarrow a) {
  constexpr int NI = MP / 16, CW = 4 / NI, KS = MP / 4;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, kk = lane >> 4;
  const int i0 = 16 * (w % NI), m = a.m, n = a.n;
  const size_t base = (size_t)blockIdx.y * m * n;
  const double* q = a.q + (size_t)blockIdx.y * MP * MP + (i0 + r) * MP + KS * kk;
  double qv[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) qv[s] = q[s];
  float x[KS];
  auto load = [&](int j0) {
    const int j = j0 + r;
    // (this lane's elements line up in 16-byte pieces: 16 x 7168 x 64 115 us a call, one by one 151)
    if (TALL && KS >= 8 && m == MP) {
#pragma unroll
      for (int s = 0; s + 8 <= KS; s += 8) {
        float v[8];
        ln_unpack<BF ? LN_BF16 : LN_F32>(
            ln_load<BF ? LN_BF16 : LN_F32>(a.u, base + (size_t)min(j, n - 1) * m + KS * kk + s), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[s + e] = v[e];
      }
      return;
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int k = KS * kk + s;
      x[s] = k < m && j < n ? orth_ld<BF>(a.u, base + (TALL ? (size_t)j * m + k : (size_t)k * n + j)) : 0.f;
    }
  };
  int j0 = 16 * (blockIdx.x * a.tiles * CW + w / NI);
  const int j1 = min(n, 16 * (int)((blockIdx.x + 1) * a.tiles * CW));
  if (j0 < j1) load(j0);
  for (; j0 < j1; j0 += 16 * CW) {
    double xv[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) xv[s] = (double)x[s];
    if (j0 + 16 * CW < j1) load(j0 + 16 * CW);
    v4d acc = v4d{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < KS; ++s)
      acc = TALL ? __builtin_amdgcn_mfma_f64_16x16x4f64(xv[s], qv[s], acc, 0, 0, 0)
                 : __builtin_amdgcn_mfma_f64_16x16x4f64(qv[s], xv[s], acc, 0, 0, 0);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int i = i0 + (TALL ? r : kk + 4 * v), j = j0 + (TALL ? kk + 4 * v : r);
      if (i < m && j < n)
        a.y[base + (TALL ? (size_t)j * m + i : (size_t)i * n + j)] = (uint16_t)f32_to_bf16_rne((float)acc[v]);
    }
  }
}

}  // namespace moe
