// Linear layers with what follows the product, and their gradients.
//
//   z = x W^T + b,  y = act(z) + residual            (SwiGLU: W's rows are gate and up, y = SiLU(g) u + residual)
//   dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum_t dz
//
// All three products are C[i][j] = sum_k P(i, k) Q(j, k) of BF16 operands on the matrix cores with
// fp32 sums; they differ in which operands lie along k in memory: x and W do in z, dz does and W does not in
// dx, neither does in dW.  An operand along k is read from LDS 8 k at a time, one across it by the transposing load.
// dz is an fp32 value: it enters as BF16 parts (bf16(dz), bf16 of what is left, and so on), each with a
// product of its own into the same sum.  Three hold all 24 bits, for fp32 results; two (within 2^-17) do for a BF16 dx, whose
// own rounding is 2^-8.  (An infinity of the other operand times the later parts, zeros or of the other sign, is NaN.)  (Two parts for fp32 results take two thirds of the time and leave an error of 2.5e-6 in
// the Frobenius norm where the fp32 sums alone leave 4e-7 to 1.6e-6.)  Where dz is the BF16 dy itself (no activation) there is one.
#pragma once
#include "elements.h"

namespace moe {

constexpr int kLinParts = 512;             // tiles' parts along k in one launch

enum { LIN_NONE = 0, LIN_RELU = 1, LIN_GELU = 2, LIN_GELU_TANH = 3, LIN_SILU = 4, LIN_SWIGLU = 5 };

// WM x WN waves with NJ subtiles of 16 columns each, 64 k at a time, ST steps in LDS.  A wave has 4 subtiles of 16 rows in LDS; with P in
// parts 2 subtiles of rows, times the parts.
// Bound by the matrix cores and what feeds them in large products: 8192 x 7168 x 2 x 2048 with SwiGLU and z
// kept takes 390 us (1230 TFLOP/s; a plain product of these sizes by the library 307 us, 1410), its gradients of three parts 1060 (dx) and 1020 us
// (dW), 1390 TFLOP/s of the parts' products.  Four waves of 128 x 128 each, half the reads of LDS, took 405 us in place of 395: one wave
// per SIMD has nothing to multiply at the barriers.
template <int WM_, int WN_, int NJ_, int ST_>
struct LinTile {
  static constexpr int WM = WM_, WN = WN_, NJ = NJ_, ST = ST_, NW = WM * WN, kThreads = 64 * NW;
  static constexpr int kCols = 16 * NJ * WN;
  static constexpr int kPitch = kCols + 4;                              // floats between rows of sums in LDS
  static constexpr int subs(int parts) { return parts == 1 ? 4 : 2 * parts; }
  static constexpr int prows(int parts) { return 16 * subs(parts) * WM; }          // rows of P in LDS
  static constexpr int rows(int parts) { return (parts == 1 ? 64 : 32) * WM; }     // of the output's tile
  static constexpr int stage(int parts) { return (prows(parts) + kCols) * 128; }   // bytes of a step's operands
  static constexpr int lds(int parts) {
    return ST * stage(parts) > 16 * WM * kPitch * 4 ? ST * stage(parts) : 16 * WM * kPitch * 4;
  }
  static constexpr size_t sums(int parts) { return (size_t)rows(parts) * kCols; }  // of one part along k
};

struct LinEpi {
  const float* bias;                       // [R]
  const void* res;                         // [rows][n]
  void* y;                                 // [rows][n]
  void* pre;                               // [rows][R]
  int act, y_f32, res_f32, pre_f32;
  int n;                                   // columns of y
};

struct LinGemm {
  const uint16_t* p;                       // along k: [rows][ldp], across: [K][ldp]
  const uint16_t* q;
  long ldp, ldq;                           // elements
  int pch;                                 // parts of P in memory: 64 elements of each in turn
  long rows;
  int cols;                                // of the output
  long K;
  int tj;                                  // tiles of columns
  long full;                               // tiles worked on whole
  int rest, split;                         // the other `rest` tiles: `split` parts along k of each
  float* part;                             // [rest][split][tile]
  LinEpi e;
};

// exp(v) by the instruction for 2^v: within 2 units, and the argument's rounding; what is below 2^-126 is zero.
DEV float lin_exp(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504f); }
DEV float lin_sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + lin_exp(-z)); }

// act(z), elementwise.
DEV void lin_act(int act, float (&v)[8]) {
  switch (act) {
    case LIN_RELU:
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] < 0.f ? 0.f : v[e];
      break;
    case LIN_GELU:
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.5f * v[e] * (1.0f + erff(v[e] * 0.70710678f));
      break;
    case LIN_GELU_TANH:                    // (1 + tanh a) / 2 = sigmoid(2 a)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] *= lin_sigmoid(1.5957691216f * (v[e] + 0.044715f * v[e] * v[e] * v[e]));
      break;
    case LIN_SILU:
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= lin_sigmoid(v[e]);
      break;
    default: break;
  }
}
// dy act'(z), elementwise.
DEV void lin_act_grad(int act, const float (&z)[8], float (&d)[8]) {
  switch (act) {
    case LIN_RELU:
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = z[e] > 0.f ? d[e] : z[e] <= 0.f ? 0.f : z[e];
      break;
    case LIN_GELU:
#pragma unroll
      for (int e = 0; e < 8; ++e)
        d[e] *= 0.5f * (1.0f + erff(z[e] * 0.70710678f)) + z[e] * 0.39894228f * lin_exp(-0.5f * z[e] * z[e]);
      break;
    case LIN_GELU_TANH:
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float s = lin_sigmoid(1.5957691216f * (z[e] + 0.044715f * z[e] * z[e] * z[e]));
        const float n = __builtin_amdgcn_fmed3f(z[e], -1024.0f, 1024.0f);      // (s (1 - s) is zero beyond, and z^2 may be infinite)
        d[e] *= s + n * s * (1.0f - s) * 1.5957691216f * (1.0f + 0.134145f * n * n);
      }
      break;
    case LIN_SILU:
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float s = lin_sigmoid(z[e]);
        d[e] *= s * (1.0f + z[e] * (1.0f - s));
      }
      break;
    default: break;
  }
}

DEV void lin_load8(const void* p, int f32, size_t at, float (&v)[8]) {
  if (f32) ln_load_f32(static_cast<const float*>(p), at, v);
  else ln_unpack<LN_BF16>(ln_load<LN_BF16>(p, at), v);
}
DEV void lin_store8(void* p, int f32, size_t at, const float (&v)[8]) {
  if (f32) {
    ln_store_f32(static_cast<float*>(p), at, v);
  } else {
    st16(static_cast<uint16_t*>(p) + at, v4i{(int)bf16x2_rne(v[0], v[1]), (int)bf16x2_rne(v[2], v[3]),
                                             (int)bf16x2_rne(v[4], v[5]), (int)bf16x2_rne(v[6], v[7])});
  }
}

// What follows the product, for 8 columns of a row: v z's sums (SwiGLU: of the gate, u of up).
template <bool GATED>
DEV void lin_finish(const LinEpi& e, long row, int col, float (&v)[8], float (&u)[8]) {
  const int R = GATED ? 2 * e.n : e.n;
  if (e.bias) {
    float b[8];
    ln_load_f32(e.bias, col, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
    if (GATED) {
      ln_load_f32(e.bias, e.n + col, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] += b[i];
    }
  }
  if (e.pre) {
    lin_store8(e.pre, e.pre_f32, (size_t)row * R + col, v);
    if (GATED) lin_store8(e.pre, e.pre_f32, (size_t)row * R + e.n + col, u);
  }
  if (GATED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * lin_sigmoid(v[i]) * u[i];
  } else {
    lin_act(e.act, v);
  }
  const size_t at = (size_t)row * e.n + col;
  if (e.res) {
    float r[8];
    lin_load8(e.res, e.res_f32, at, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  lin_store8(e.y, e.y_f32, at, v);
}

// An operand's tile goes straight to LDS (16-byte buffer loads, out of range reads as zero).  The swizzles leave no conflicts between
// the lanes that LDS serves together (lanes 0-3, 12-15 and 20-27, and so on): 411 -> 388 us in the product above.
// Along k an LDS row is 64 k of one row, its 16-byte chunk c at c ^ lin_swz(row), so that the 16 rows of an operand read
// fall in distinct banks.  Across k it is one k of the tile's columns, its 32-byte chunk c at c ^ lin_swz_t(k), so that the 8 k
// of 32 lanes do.
DEV int lin_swz(int r) { return (r & 2) | ((r >> 1) & 4); }
template <int COLS>
DEV int lin_swz_t(int r) {
  static_assert(COLS % 64 == 0, "whole groups of 4 chunks");
  if (COLS % 128) return ((r >> 1) & 1) | ((r >> 2) & 2);      // (every second k starts in the middle of the banks' 256 bytes)
  return (r & 3) | ((r >> 1) & 4);
}
typedef short v4s __attribute__((ext_vector_type(4)));
// Lane l of 16 hands in the address of 8 bytes, columns 4 (l % 4) .. + 3 of row l / 4, and gets the 4 rows of
// column l.  (restrict: the compiler does not see which loads into LDS the barriers have waited for)
DEV v4s lin_tr16(const char* __restrict__ p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) v4s*)(__attribute__((address_space(3))) char*)const_cast<char*>(p));
}
// Operand read from a tile in LDS: k 32 kh + 8 (lane / 16) .. + 7 of row r0 + 16 i + lane % 16.
template <int COLS, bool TR>
DEV v8bf lin_frag(const char* op, int r0, int i, int kh, int lane) {
  const int c16 = lane & 15, gq = lane >> 4;
  if (TR) {
    const int k = 32 * kh + 8 * gq + (c16 >> 2), c = (r0 >> 4) + i;
    const char* a = op + k * (2 * COLS) + ((c ^ lin_swz_t<COLS>(k)) << 5) + 8 * (lane & 3);
    const v4s x0 = lin_tr16(a), x1 = lin_tr16(a + 4 * 2 * COLS);
    return __builtin_bit_cast(v8bf, __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  const int r = r0 + 16 * i + c16;
  return lds_ld<v8bf>(op, (uint32_t)r * 128 + (((4 * kh + gq) ^ lin_swz(r)) << 4));
}
DEV uint32_t lin_bytes(long n) { return (uint32_t)(n < 0x7FFFFF00l ? n : 0x7FFFFF00l); }
constexpr uint32_t kLinNowhere = 0x7FFFFFF0u;                  // past every buffer's end

// PT, QT: the operand lies across k.  PARTS: P's, in memory 64 elements of each in turn; in LDS a wave's rows are its
// two subtiles of the first part, then of the next.
// GATED: the tile's columns are kCols / 2 of the gate and the same of up, q [2 cols][ldq].
template <class TL, int PT, int QT, int PARTS, int GATED>
DEV void lin_tile(const LinGemm& g, long block, char* lds) {
  constexpr int NJ = TL::NJ, NW = TL::NW, S = TL::kCols, SP = TL::prows(PARTS), IP = TL::subs(PARTS);
  constexpr int NI = PARTS == 1 ? 4 : 2, PP = SP / 8 / NW, QP = S / 8 / NW, kStage = TL::stage(PARTS);
  constexpr int MT = TL::rows(PARTS), NT = GATED ? S / 2 : S;  // rows and columns of the output's tile
  static_assert(SP % (8 * NW) == 0 && S % (8 * NW) == 0, "whole 1 KB pieces per wave");
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, gq = lane >> 4, wm = w / TL::WN, wn = w % TL::WN;

  // XCD x (workgroup ids go round-robin) takes a contiguous range of the whole tiles; the parts of the others follow
  const long per = (g.full + 7) / 8;
  long t;
  int part = -1;
  if (block < 8 * per) {
    t = block % 8 * per + block / 8;
    if (t >= g.full) return;
  } else {
    part = (int)(block - 8 * per);
    t = g.full + part / g.split;
  }
  const long i0 = t / g.tj * MT;
  const int j0 = (int)(t % g.tj) * NT;
  const int steps = (int)((g.K + 63) / 64);
  int s0 = 0, s1 = steps;
  if (part >= 0) {
    const int ks = part % g.split;
    s0 = (int)((long)ks * steps / g.split);
    s1 = (int)((long)(ks + 1) * steps / g.split);
  }

  // byte offsets of this lane's 16 bytes of each 1 KB piece, from the step's first byte of the operand
  uint32_t poff[PP], qoff[QP];
  int pk[PP], qk[QP];                              // along k: the chunk's first k in the step
#pragma unroll
  for (int n = 0; n < PP; ++n) {
    const int o = (n * NW + w) * 1024 + lane * 16;
    if (!PT) {
      const int r = o / 128, c = (lane & 7) ^ lin_swz(r), sub = r % (16 * IP) / 16;
      const int row = PARTS == 1 ? r : r / (16 * IP) * 32 + 16 * (sub & 1) + (r & 15);
      pk[n] = 8 * c;
      poff[n] = (uint32_t)row * (uint32_t)g.ldp * 2 + 16 * c + (PARTS == 1 ? 0 : 128 * (sub >> 1));
    } else {
      // (columns past the end are never stored: the last ones again)
      const int k = o / (2 * SP), cc = (o % (2 * SP) / 16) ^ (lin_swz_t<SP>(k) << 1), sub = cc % (2 * IP) / 2;
      const int col = PARTS == 1 ? 8 * cc : cc / (2 * IP) * 32 + 16 * (sub & 1) + 8 * (cc & 1);
      const uint32_t at = (uint32_t)min(i0 + col, g.rows - 8);
      pk[n] = 0;
      poff[n] = (uint32_t)k * (uint32_t)g.ldp * 2 + (PARTS == 1 ? 2 * at : 128 * ((at >> 6) * g.pch + (sub >> 1)) + 2 * (at & 63));
    }
  }
#pragma unroll
  for (int n = 0; n < QP; ++n) {
    const int o = (n * NW + w) * 1024 + lane * 16;
    if (!QT) {
      const int r = o / 128, c = (lane & 7) ^ lin_swz(r);
      qk[n] = 8 * c;
      qoff[n] = (uint32_t)(GATED ? r % NT : r) * (uint32_t)g.ldq * 2 + 16 * c;
    } else {
      const int k = o / (2 * S), cc = (o % (2 * S) / 16) ^ (lin_swz_t<S>(k) << 1);
      qk[n] = 0;
      qoff[n] = (uint32_t)k * (uint32_t)g.ldq * 2 + 2 * (uint32_t)min(j0 + 8 * cc, g.cols - 8);
    }
  }
  const uint16_t* pb = PT ? g.p : g.p + i0 * g.ldp;
  const uint16_t* qb = QT ? g.q : g.q + (long)j0 * g.ldq;
  const uint32_t pn = lin_bytes((g.rows - i0) * g.ldp * 2), qn = lin_bytes((long)(g.cols - j0) * g.ldq * 2);
  auto load = [&](int step, int stage) {
    char* ps = lds + stage * kStage;
    char* qs = ps + SP * 128;
    const int s = min(step, s1 - 1);               // (past the end: the last step again, never read)
    const long left = g.K - 64l * s;               // k from this step on
    const rsrc_t pr = PT ? make_rsrc(pb + 64l * s * g.ldp, lin_bytes(min(left, 64l) * g.ldp * 2))
                         : make_rsrc(pb, pn);
    const rsrc_t qr = QT ? make_rsrc(qb + 64l * s * g.ldq, lin_bytes(min(left, 64l) * g.ldq * 2))
                         : make_rsrc(qb, qn);
    const rsrc_t ur = make_rsrc(GATED ? qb + (long)g.cols * g.ldq : qb, qn);
    const uint32_t pa = PT ? 0 : (uint32_t)s * 128 * g.pch, qa = QT ? 0 : (uint32_t)s * 128;
    if ((PT && QT) || left >= 64) {
#pragma unroll
      for (int n = 0; n < PP; ++n) buf_ld16_lds(pr, ps + (n * NW + w) * 1024, poff[n], pa);
#pragma unroll
      for (int n = 0; n < QP; ++n)
        buf_ld16_lds(GATED && 8 * (n * NW + w) >= NT ? ur : qr, qs + (n * NW + w) * 1024, qoff[n], qa);
    } else {                                       // k past the end are zeros
#pragma unroll
      for (int n = 0; n < PP; ++n)
        buf_ld16_lds(pr, ps + (n * NW + w) * 1024, PT || pk[n] < left ? poff[n] + pa : kLinNowhere, 0);
#pragma unroll
      for (int n = 0; n < QP; ++n)
        buf_ld16_lds(GATED && 8 * (n * NW + w) >= NT ? ur : qr, qs + (n * NW + w) * 1024,
                     QT || qk[n] < left ? qoff[n] + qa : kLinNowhere, 0);
    }
  };

  v4f acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  const int pr0 = 16 * IP * wm, qr0 = 16 * NJ * wn;
  auto pfrag = [&](const char* st, int i, int kh) { return lin_frag<SP, PT != 0>(st, pr0, i, kh, lane); };
  auto qfrag = [&](const char* st, int j, int kh) { return lin_frag<S, QT != 0>(st + SP * 128, qr0, j, kh, lane); };
  // A step's first operands are read during the last products of the step before, behind the barrier: their
  // LDS latency is covered by products.
  constexpr int NL = NJ >= 4 ? 2 : 1;              // column subtiles left behind the barrier, and read ahead
  v8bf pf[IP], qf[NJ];
  auto read_first = [&](const char* st) {
#pragma unroll
    for (int i = 0; i < IP; ++i) pf[i] = pfrag(st, i, 0);
#pragma unroll
    for (int j = 0; j < NL; ++j) qf[j] = qfrag(st, j, 0);
  };
  auto mul = [&](int j) {
#pragma unroll
    for (int i = 0; i < IP; ++i) acc[i % NI][j] = mfma_bf16(qf[j], pf[i], acc[i % NI][j]);
  };
#pragma unroll
  for (int s = 0; s < TL::ST; ++s) load(s0 + s, s);
  barrier_vmcnt<(TL::ST - 1) * (PP + QP)>();          // the first step has landed
  read_first(lds);
  int stage = 0;
  auto halves = [&](const char* st) {              // the step but for the last NL column subtiles
#pragma unroll
    for (int j = NL; j < NJ; ++j) qf[j] = qfrag(st, j, 0);
#pragma unroll
    for (int j = 0; j < NJ; ++j) mul(j);
#pragma unroll
    for (int i = 0; i < IP; ++i) pf[i] = pfrag(st, i, 1);
#pragma unroll
    for (int j = 0; j < NJ; ++j) qf[j] = qfrag(st, j, 1);
#pragma unroll
    for (int j = 0; j < NJ - NL; ++j) mul(j);
  };
  for (int s = s0; s < s1 - 1; ++s) {
    halves(lds + stage * kStage);
    const int cur = stage;
    stage = stage == TL::ST - 1 ? 0 : stage + 1;
    // this wave's loads of the next step have landed and its reads of this one are done, and so are every
    // wave's: this stage is free
    barrier_vmcnt<(TL::ST - 2) * (PP + QP)>();
    load(s + TL::ST, cur);
    v8bf pl[IP], ql[NL];
#pragma unroll
    for (int i = 0; i < IP; ++i) pl[i] = pf[i];
#pragma unroll
    for (int j = 0; j < NL; ++j) ql[j] = qf[NJ - NL + j];
    read_first(lds + stage * kStage);
    __builtin_amdgcn_sched_barrier(0);             // (these reads are issued before the products below)
#pragma unroll
    for (int j = 0; j < NL; ++j)
#pragma unroll
      for (int i = 0; i < IP; ++i) acc[i % NI][NJ - NL + j] = mfma_bf16(ql[j], pl[i], acc[i % NI][NJ - NL + j]);
    // (and stay in this step: the compiler would move them to the next one's start)
#pragma unroll
    for (int i = 0; i < IP; ++i) asm volatile("" : "+v"(pf[i]));
#pragma unroll
    for (int j = 0; j < NL; ++j) asm volatile("" : "+v"(qf[j]));
  }
  halves(lds + stage * kStage);
#pragma unroll
  for (int j = NJ - NL; j < NJ; ++j) mul(j);
  wait_vmcnt<0>();                                 // no load into LDS is in flight below

  // The sums go through LDS, 16 rows of every wave at a time, so that whole rows of the tile are read, finished and
  // written 8 columns per thread: acc[i][j][v] is row 16 i + c16 and column 16 j + 4 gq + v of the wave's.
  float* sums = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      *reinterpret_cast<v4f*>(sums + (16 * wm + c16) * TL::kPitch + qr0 + 16 * j + 4 * gq) = acc[i][j];
    __syncthreads();
    for (int n = tid; n < 16 * TL::WM * (NT / 8); n += TL::kThreads) {
      const int lr = n / (NT / 8), col = 8 * (n % (NT / 8));
      const int tr = (lr >> 4) * (16 * NI) + 16 * i + (lr & 15);        // row of the tile
      float v[8], u[8];
      ln_load_f32(sums, (size_t)lr * TL::kPitch + col, v);
      if (GATED) ln_load_f32(sums, (size_t)lr * TL::kPitch + NT + col, u);
      if (part >= 0) {
        float* dst = g.part + (size_t)part * TL::sums(PARTS);
        ln_store_f32(dst, (size_t)tr * S + col, v);
        if (GATED) ln_store_f32(dst, (size_t)tr * S + NT + col, u);
        continue;
      }
      if (i0 + tr < g.rows && j0 + col < g.cols) lin_finish<GATED>(g.e, i0 + tr, j0 + col, v, u);
    }
  }
}

template <class TL, int PT, int QT, int PARTS, int GATED>
__global__ void __launch_bounds__(TL::kThreads, 2) k_linear(LinGemm g) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  lin_tile<TL, PT, QT, PARTS, GATED>(g, blockIdx.x, lds);
}

// The tiles worked on in parts: 8 columns of a row per thread, the parts added in order (128 tiles of 128 x 256 in two parts: 10 us).
template <class TL, int PARTS, int GATED>
DEV void lin_join(const LinGemm& g, int block) {
  constexpr int S = TL::kCols, MT = TL::rows(PARTS), NT = GATED ? S / 2 : S;
  const int n = block * 256 + threadIdx.x;         // (MT NT / 8 of a tile: whole workgroups)
  const int r = n / (MT * (NT / 8)), l = n % (MT * (NT / 8)), tr = l / (NT / 8), col = 8 * (l % (NT / 8));
  const long t = g.full + r, row = t / g.tj * MT + tr;
  const int c = (int)(t % g.tj) * NT + col;
  if (row >= g.rows || c >= g.cols) return;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0}, u[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int k = 0; k < g.split; ++k) {
    const float* src = g.part + ((size_t)r * g.split + k) * TL::sums(PARTS) + (size_t)tr * S + col;
    float x[8];
    ln_load_f32(src, 0, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += x[i];
    if (GATED) {
      ln_load_f32(src, NT, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] += x[i];
    }
  }
  lin_finish<GATED>(g.e, row, c, v, u);
}
template <class TL, int PARTS, int GATED>
__global__ void __launch_bounds__(256) k_linear_join(LinGemm g) { lin_join<TL, PARTS, GATED>(g, blockIdx.x); }
// Of dx and dW: nx workgroups for dx.
template <class TL, int PX, int PW>
__global__ void __launch_bounds__(256) k_linear_joins(LinGemm x, LinGemm w, int nx) {
  const int block = blockIdx.x;
  if (block < nx) lin_join<TL, PX, 0>(x, block);
  else lin_join<TL, PW, 0>(w, block - nx);
}

// ------------------------------------------------------------------ few rows
// z for up to 16 TT rows of x (a decoded token, a small batch): bound by reading W once.  A workgroup does 16 rows of W (SwiGLU: 8
// of the gate and the same 8 of up), its eight waves every eighth 64 k each; W and x go from memory to
// the matrix cores' operands, four steps of a wave in flight (with eight, K = 2048 takes 7.6 us for 5.4: a wave has four).  Lane l holds row l % 16 and k 16 (l / 16) .. + 15 of a step, in both operands, so
// that a row's 128 bytes are read together; the waves' sums meet in LDS.
template <int TT, int GATED>
__global__ void __launch_bounds__(512, 2) k_linear_rows(LinGemm g) {
  constexpr int NT = GATED ? 8 : 16, U = 4, kPitch = 20;
  __shared__ __attribute__((aligned(16))) float sums[8][16 * TT][kPitch];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, gq = lane >> 4, j0 = blockIdx.x * NT;
  const int wr = GATED ? (c16 < 8 ? j0 + c16 : g.cols + j0 + c16 - 8) : min(j0 + c16, g.cols - 1);
  const uint16_t* wp = g.q + (long)wr * g.ldq + 16 * gq;
  const uint16_t* xp[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) xp[t] = g.p + min((long)(16 * t + c16), g.rows - 1) * g.ldp + 16 * gq;   // (rows past the end: the last, never stored)
  v4f acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
  const int steps = (int)(g.K / 64), mine = (steps - w + 7) / 8;      // whole steps w, w + 8, ...
  v4i wf[U][2], xf[U][TT][2];
  auto load = [&](int i, int n) {
    const long k = 64l * (w + 8 * min(n, mine - 1));                  // (past the end: the last step again, never used)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      wf[i][h] = ld16(wp + k + 8 * h);
#pragma unroll
      for (int t = 0; t < TT; ++t) xf[i][t][h] = ld16(xp[t] + k + 8 * h);
    }
  };
  auto mul = [&](const v4i (&a)[2], const v4i (&b)[TT][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[t] = mfma_bf16(as_v8bf(a[h]), as_v8bf(b[t][h]), acc[t]);
  };
  if (mine > 0) {
#pragma unroll
    for (int i = 0; i < U; ++i) load(i, i);
    for (int n = 0; n < mine; n += U) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (n + i < mine) mul(wf[i], xf[i]);
        if (n + U < mine) load(i, n + U + i);
      }
    }
  }
  if (g.K % 64 && w == steps % 8) {                // what is left of k: zeros past the end
    const long k = 64l * steps;
    const v4i zero = v4i{0, 0, 0, 0};
    v4i a[2], b[TT][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = k + 16 * gq + 8 * h < g.K;
      const long at = in ? k + 8 * h : -16 * gq;   // (else the row's first elements)
      a[h] = ld16(wp + at);
      if (!in) a[h] = zero;
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        b[t][h] = ld16(xp[t] + at);
        if (!in) b[t][h] = zero;
      }
    }
    mul(a, b);
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) *reinterpret_cast<v4f*>(&sums[w][16 * t + c16][4 * gq]) = acc[t];
  __syncthreads();
  // 8 columns of a row per thread
  const int row = GATED ? tid : tid >> 1, c = GATED ? 0 : 8 * (tid & 1);
  if (row >= 16 * TT || row >= g.rows || j0 + c >= g.cols) return;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0}, u[8] = {0, 0, 0, 0, 0, 0, 0, 0}, x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    ln_load_f32(&sums[i][row][c], 0, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += x[e];
    if (GATED) {
      ln_load_f32(&sums[i][row][8], 0, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] += x[e];
    }
  }
  lin_finish<GATED>(g.e, row, j0 + c, v, u);
}

// ---------------------------------------------------------------- dz and db
struct LinDz {
  const void* dy;                          // [T][n]
  const void* pre;                         // [T][R]
  uint16_t* dz;                            // [T][ceil(R / 64)][parts][64], or NULL
  float* part;                             // [slabs][R] sums of dz over a slab's rows, or NULL
  long T;
  int n, act, dy_f32, pre_f32;
  int slab;                                // rows of a slab
  int parts;                               // of dz: 2 or 3
};

DEV void lin_split_store(const LinDz& a, long t, int R, int col, float (&v)[8]) {
  uint16_t* at = a.dz + ((size_t)t * ((R + 63) / 64) + col / 64) * 64 * a.parts + (col & 63);
  for (int p = 0; p < a.parts; ++p) {
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[e] = f32_to_bf16_rne(v[e]);
      // (what rounds up to infinity is cut instead; infinity and NaN leave nothing for the other parts)
      const bool over = (h[e] & 0x7F80) == 0x7F80, inf = over && !(fabsf(v[e]) <= 3.4028234e38f);
      if (over && !inf) h[e] = __builtin_bit_cast(uint32_t, v[e]) >> 16;
      v[e] = inf ? 0.f : v[e] - bf16_to_f32(h[e]);
    }
    st16(at + 64 * p, v4i{(int)(h[0] | h[1] << 16), (int)(h[2] | h[3] << 16), (int)(h[4] | h[5] << 16), (int)(h[6] | h[7] << 16)});
  }
}

// Workgroup (x, y): 512 columns of y (8 per lane), slab y's rows (wave w every fourth).  Bound by memory: 8192 x 2048 SwiGLU, 302 MB
// with three parts, in 59 us (5.1 TB/s).
template <int GATED>
__global__ void __launch_bounds__(256) k_linear_dz(LinDz a) {
  __shared__ float red[4][GATED ? 2 : 1][64][8];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, col = (blockIdx.x * 64 + lane) * 8;
  const int R = GATED ? 2 * a.n : a.n;
  const bool live = col < a.n;
  float sg[8] = {0, 0, 0, 0, 0, 0, 0, 0}, su[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  const long t1 = min((long)(blockIdx.y + 1) * a.slab, a.T);
  if (live) {
#pragma unroll 2
    for (long t = (long)blockIdx.y * a.slab + w; t < t1; t += 4) {
      float d[8], z[8], u[8];
      lin_load8(a.dy, a.dy_f32, (size_t)t * a.n + col, d);
      if (a.pre) lin_load8(a.pre, a.pre_f32, (size_t)t * R + col, z);
      if (GATED) {
        lin_load8(a.pre, a.pre_f32, (size_t)t * R + a.n + col, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float s = lin_sigmoid(z[e]), dy = d[e];
          d[e] = dy * (u[e] * (s * (1.0f + z[e] * (1.0f - s))));      // (what is at most 1.1 first: no infinity where s is zero)
          u[e] = dy * (z[e] * s);
          su[e] += u[e];
        }
        if (a.dz) lin_split_store(a, t, R, a.n + col, u);
      } else if (a.pre) {
        lin_act_grad(a.act, z, d);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sg[e] += d[e];
      if (a.dz) lin_split_store(a, t, R, col, d);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    red[w][0][lane][e] = sg[e];
    if (GATED) red[w][GATED ? 1 : 0][lane][e] = su[e];
  }
  __syncthreads();
  if (w >= 1 + GATED || !live) return;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (red[0][w][lane][e] + red[1][w][lane][e]) + (red[2][w][lane][e] + red[3][w][lane][e]);
  ln_store_f32(a.part, (size_t)blockIdx.y * R + (w ? a.n : 0) + col, v);
}

// db: the slabs' sums, 64 columns per workgroup of NW waves, each of them every NW-th slab.
struct LinDbias {
  const float* part;
  float* db;
  int slabs, R;
};
template <int NW>
DEV void lin_dbias(const LinDbias& a, int block, float* red) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = block * 64 + lane;
  float s = 0.f;
  if (c < a.R) {
#pragma unroll 8
    for (int i = w; i < a.slabs; i += NW) s += a.part[(size_t)i * a.R + c];
  }
  red[threadIdx.x] = s;
  __syncthreads();
  if (w || c >= a.R) return;
#pragma unroll
  for (int i = 1; i < NW; ++i) s += red[64 * i + lane];
  a.db[c] = s;
}
__global__ void __launch_bounds__(256) k_linear_dbias(LinDbias a) {
  __shared__ float red[256];
  lin_dbias<4>(a, blockIdx.x, red);
}

// dx, dW and db together, where one of them does not fill the GPU: nx workgroups for dx, nw for dW, the others for db.  Bound by the
// latency of a few steps: 333 x 1000 x 488 in 10.4 us, where the three apart took 26.
template <class TL, int PX, int PW>
__global__ void __launch_bounds__(TL::kThreads, 2) k_linear_grads(LinGemm x, LinGemm w, LinDbias b, int nx, int nw) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int block = blockIdx.x;
  if (block < nx) lin_tile<TL, 0, 1, PX, 0>(x, block, lds);
  else if (block < nx + nw) lin_tile<TL, 1, 1, PW, 0>(w, block - nx, lds);
  else lin_dbias<TL::NW>(b, block - nx - nw, reinterpret_cast<float*>(lds));
}

}  // namespace moe
