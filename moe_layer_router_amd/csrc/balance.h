// Load-balance loss of the router, the experts' token counts, and the
// gradient of the loss in the logits.
//
// For the tokens t of sequence s (N_s of them count), p[t] = softmax(l[t])
// over all E experts, c_s[e] = the entries of topk_ids equal to e:
//   P_s[e] = sum_t p[t][e] / N_s,  f_s[e] = E c_s[e] / (k N_s)
//   loss = alpha / S' sum_s sum_e f_s[e] P_s[e]    (S' sequences with N_s > 0)
// The counts are constants of the gradient:
//   dl[t][e] = kappa_s p[t][e] (c_s[e] - sum_i p[t][i] c_s[i]),
//   kappa_s = alpha E / (S' k N_s^2)
// which is evaluated as kappa p_e (h_e - sum_i p_i h_i) with h_e = c_s[e] -
// c_s[top], top being the token's likeliest expert: the differences of
// counts are exact integers, the sum leaves p_top out, and so neither a
// saturated token (p_top near 1) nor even counts cancel.
//
// Three kernels, bound by HBM on large batches (logits read once, dlogits
// written once) and by their launches on small ones (k_bal_one does the
// smallest in one):
//   k_bal_count   blocks of tokens: histogram in LDS, one row of counts for
//                 each (block, sequence) pair that meets
//   k_bal_tokens  softmax, the gradient, and sums of p, one row of partial
//                 sums for each (block, sequence) pair
//   k_bal_final   counts, P and the loss from the rows
// Row of (block b, sequence s): b + s.  Blocks and sequences both ascend
// with the tokens, so the pairs that meet form a staircase on which b + s
// grows by one each step: no two share a row, the rows of one sequence are
// consecutive, and blocks + sequences rows are enough.  Everything is summed
// in a fixed order (the only atomics count finished workgroups and add
// integers in LDS).
//
// Measured: T = 16384, E = 1024, k = 16, 13 sequences, masked (134 MB): 10.5 + 32 +
// 9.2 us, the middle kernel at 4.2 TB/s; T = 8192, E = 256, k = 8 (17 MB): 6.8 +
// 9.5 + 6.0 us, of which 3.3 is the traffic and the rest launches and the chains
// of dependent loads in them; T = 64, E = 8: 8 us in one launch.
//
// Sequence offsets are device data: each is clamped to [0, T], and a
// sequence that ends before it begins is empty.  With offsets that descend
// the results are unspecified, but every access stays in range.
#pragma once
#include "device_common.h"
#include "permute.h"

namespace moe {

typedef float v4fu __attribute__((ext_vector_type(4), aligned(4)));   // rows of E floats: 4-byte aligned

struct BalArgs {
  const float* logits;       // [T][E]
  const int32_t* ids;        // [T][k]
  const int32_t* off;        // [S+1], or NULL (one sequence of all T tokens)
  const uint8_t* mask;       // [T], or NULL (every token counts)
  int32_t* counts;           // [S][E]
  float* probs;              // [S][E]
  float* loss;               // [1]
  float* dlogits;            // [T][E], or NULL
  int T, E, k, S;
  float alpha;
  int cb, tb;                // tokens per block of k_bal_count and of k_bal_tokens
  int32_t* rowcnt;           // [count blocks + S][E]
  int32_t* rown;             // [count blocks + S] tokens that count
  float* rowp;               // [token blocks + S][E] sums of p
  double* lpart;             // [workgroups of k_bal_final]
  int32_t* used;             // S', at least 1
  int32_t* done;             // workgroups of k_bal_final that have finished
};

// The sequence offsets, clamped: in LDS where they fit (a search through global
// memory is a chain of round trips), else where they are.
constexpr int kBalOff = 256;
struct BalOff {
  const int* lds;                                             // NULL: global memory
  const BalArgs* a;
  DEV int operator()(int s) const {
    if (lds) return lds[s];
    return a->off ? min(max(a->off[s], 0), a->T) : (s ? a->T : 0);
  }
};
// By the whole workgroup, with a barrier; buf: kBalOff ints.
DEV BalOff bal_offsets(const BalArgs& a, int* buf) {
  const BalOff global{nullptr, &a};
  if (a.S >= kBalOff) return global;
  for (int s = threadIdx.x; s <= a.S; s += blockDim.x) buf[s] = global(s);
  __syncthreads();
  return BalOff{buf, &a};
}

// The first sequence that ends behind token t (S if none does).
DEV int bal_seq_of(const BalArgs& a, const BalOff& off, int t) {
  int lo = 0, hi = a.S;
  while (lo < hi) {
    const int m = (lo + hi) / 2;
    if (off(m + 1) > t) hi = m; else lo = m + 1;
  }
  return lo;
}

// Rows [*r0, *r1) of sequence s over blocks of `bt` tokens (none if empty).
DEV void bal_rows(const BalOff& off, int s, int bt, int* r0, int* r1) {
  const int t0 = off(s), t1 = off(s + 1);
  *r0 = t0 / bt + s;
  *r1 = t1 > t0 ? (t1 - 1) / bt + s + 1 : *r0;
}

// Counts of the tokens [lo, hi), which belong to up to kBalSegs sequences ending
// at end[]: a histogram each (together: short sequences would otherwise cost a
// round of memory and barriers each), in hist [kBalSegs][E], and the entries
// that count in s_n. nq: how many of them are in use. By a workgroup of NT
// threads, which may read the results when it returns.
constexpr int kBalCountThreads = 1024, kBalSegs = 4;
template <int NT>
DEV void bal_count_group(const BalArgs& a, int lo, int hi, const int (&end)[kBalSegs], int nq, int* hist, int* s_n) {
  // all loads of a pass before any of its counts (and the first pass's before
  // the histograms are cleared); -1: an entry that does not count
  constexpr int kU = 8;
  const int n = (hi - lo) * a.k;
  int mine[kBalSegs] = {0, 0, 0, 0};
  for (int p0 = 0; p0 < n; p0 += kU * NT) {
    int ev[kU], sv[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = p0 + u * NT + (int)threadIdx.x, j = min(i, n - 1), t = lo + j / a.k;
      const int e = min(max(a.ids[(size_t)lo * a.k + j], 0), a.E - 1);
      const bool in = i < n && (!a.mask || a.mask[t]);
      sv[u] = (t >= end[0]) + (t >= end[1]) + (t >= end[2]);
      ev[u] = in ? sv[u] * a.E + e : -1;
    }
    if (p0 == 0) {
      for (int e = threadIdx.x; e < nq * a.E; e += NT) hist[e] = 0;
      if (threadIdx.x < kBalSegs) s_n[threadIdx.x] = 0;
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (ev[u] >= 0) {
        atomicAdd(&hist[ev[u]], 1);
#pragma unroll
        for (int q = 0; q < kBalSegs; ++q) mine[q] += sv[u] == q;
      }
  }
#pragma unroll
  for (int q = 0; q < kBalSegs; ++q) {
    if (q >= nq) break;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) mine[q] += __shfl_xor(mine[q], d);
    if ((threadIdx.x & 63) == 0 && mine[q]) atomicAdd(&s_n[q], mine[q]);
  }
  __syncthreads();
}
// Histograms in use for tokens that end at hi.
DEV int bal_segs(int hi, const int (&end)[kBalSegs]) { return 1 + (hi > end[0]) + (hi > end[1]) + (hi > end[2]); }

__global__ void __launch_bounds__(kBalCountThreads) k_bal_count(BalArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int* hist = reinterpret_cast<int*>(lds);                    // [kBalSegs][E]
  __shared__ int s_n[kBalSegs];
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;
  __shared__ int s_off[kBalOff];
  const BalOff off = bal_offsets(a, s_off);
  const int t0 = blockIdx.x * a.cb, t1 = min(a.T, t0 + a.cb);
  for (int s = bal_seq_of(a, off, t0); s < a.S && off(s) < t1; s += kBalSegs) {
    int end[kBalSegs];                                        // where the sequences end
#pragma unroll
    for (int q = 0; q < kBalSegs; ++q) end[q] = off(min(s + q + 1, a.S));
    const int lo = max(t0, off(s)), hi = min(t1, end[kBalSegs - 1]);
    if (lo >= hi) continue;                                   // (uniform)
    const int nq = bal_segs(hi, end);
    bal_count_group<kBalCountThreads>(a, lo, hi, end, nq, hist, s_n);
#pragma unroll
    for (int q = 0; q < kBalSegs; ++q) {
      // (a sequence that does not meet the block has no row: the others' are taken)
      if (q >= nq || s + q >= a.S || max(t0, off(s + q)) >= min(t1, end[q])) continue;
      int32_t* row = a.rowcnt + (size_t)(blockIdx.x + s + q) * a.E;
      for (int e = threadIdx.x; e < a.E; e += kBalCountThreads) row[e] = hist[q * a.E + e];
      if (threadIdx.x == 0) a.rown[blockIdx.x + s + q] = s_n[q] / a.k;    // (k entries for each token that counts)
    }
    __syncthreads();
  }
}

// Tokens of sequence s that count, by one thread.
DEV int bal_tokens_of(const BalArgs& a, const BalOff& off, int s) {
  int r0, r1, n = 0;
  bal_rows(off, s, a.cb, &r0, &r1);
#pragma unroll 8
  for (int r = r0; r < r1; ++r) n += a.rown[r];
  return n;
}

// S' (at least 1) for the whole workgroup; `red`: one int per wave.
DEV int bal_used(const BalArgs& a, const BalOff& off, int* red) {
  int u = 0;
  for (int s = threadIdx.x; s < a.S; s += blockDim.x) u += bal_tokens_of(a, off, s) > 0;
  int tot;
  block_inclusive_scan(u, red, &tot);
  return max(tot, 1);
}

// Maximum over the L lanes of a token (counts: not negative).
template <int CTRL>
DEV int dpp_mov_i(int x) { return __builtin_amdgcn_mov_dpp(x, CTRL, 0xF, 0xF, false); }
template <int L>
DEV int bal_max(int v) {
  v = max(v, dpp_mov_i<0xB1>(v));
  v = max(v, dpp_mov_i<0x4E>(v));
  v = max(v, dpp_mov_i<0x141>(v));
  v = max(v, dpp_mov_i<0x140>(v));
  if (L == 64) {
    const auto r16 = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
    v = max((int)r16[0], (int)r16[1]);
    const auto r32 = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
    v = max((int)r32[0], (int)r32[1]);
  }
  return v;
}

// exp(x) for x <= 0 (NaN: NaN): 2^t of the rounded t = x log2 e times the 1 + e ln 2
// of what the rounding left, log2 e in two parts: within 2 units in the last
// place, without the range steps of a general exponential (a result below
// the normal range, -infinity's among them, is zero).
DEV float bal_exp(float x) {
  x = x < -200.f ? -200.f : x;
  constexpr float kHi = 1.44269504f, kLo = (float)(1.4426950408889634 - (double)1.44269504f);
  const float t = x * kHi;
  const float e = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -t));
  const float p = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(p, e * 0.693147181f, p);
}

// One token per L lanes (16 for E <= 256, else 64), NJ chunks of 4
// consecutive experts per lane, NT threads. Loads and stores are buffer
// accesses without branches: what lies outside the row, or belongs to a token
// that does not count, gets an offset past the buffer's end, which reads zero and
// drops a store (a condition on each would be a branch with a wait: 41 us
// instead of 36 at T = 16384, E = 1024). VEC: E is a multiple of 4, 16-byte
// accesses; otherwise a chunk may reach into the next row, and each element is
// its own access.
constexpr uint32_t kBalSkip = 0xFFFFFFF0u;
template <int L, int NJ, int VEC, int GRAD, int NT>
struct BalTokens {
  static constexpr int G = NT / L;                            // tokens in flight per workgroup
  static constexpr int kCols = L * NJ * 4;                    // experts the lanes of a token cover
  static constexpr int kLds = (NT / 64 + 1) * kCols * 4;      // psum and cnt
  float* psum;                                                // [NT / 64][kCols] sums of p by wave
  int* cnt;                                                   // [kCols] counts of the sequence
  const BalArgs& a;
  int t0, t1, li, gi, w;
  rsrc_t lr, dr;                                              // rows t0 .. t1 - 1

  DEV BalTokens(const BalArgs& args, char* lds, int b0, int b1) : a(args), t0(b0), t1(b1) {
    psum = reinterpret_cast<float*>(lds);
    cnt = reinterpret_cast<int*>(psum + NT / 64 * kCols);
    li = threadIdx.x % L;
    gi = threadIdx.x / L;
    w = threadIdx.x >> 6;
    const uint32_t bytes = (uint32_t)(t1 - t0) * (uint32_t)a.E * 4u;
    lr = make_rsrc(a.logits + (size_t)t0 * a.E, bytes);
    dr = make_rsrc(GRAD ? a.dlogits + (size_t)t0 * a.E : nullptr, GRAD ? bytes : 0u);
  }
  static DEV float row_max(float v) { v = row_max16(v); return L == 64 ? max_row_groups(v) : v; }
  static DEV float row_sum(float v) { return L == 64 ? wave_sum(v) : row_sum16(v); }
  DEV uint32_t place(int t, int j, int i, bool on) const {    // of expert 4 (li + L j) + i of token t
    const int e = 4 * (li + L * j) + i;
    return on && e < a.E ? ((uint32_t)(t - t0) * (uint32_t)a.E + (uint32_t)e) * 4u : kBalSkip;
  }
  DEV void load(int t, bool on, float (&v)[NJ][4]) const {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (VEC) {
        const v4i q = buf_ld16(lr, place(t, j, 0, on), 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = __int_as_float(q[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = buf_ldf(lr, place(t, j, i, on), 0);
      }
    }
  }
  DEV void store(int t, bool on, const float (&d)[NJ][4]) const {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (VEC) {
        buf_st16(dr, place(t, j, 0, on), v4i{__float_as_int(d[j][0]), __float_as_int(d[j][1]),
                                             __float_as_int(d[j][2]), __float_as_int(d[j][3])});
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) buf_stf(dr, place(t, j, i, on), d[j][i]);
      }
    }
  }
  // Zero gradients of the tokens [lo, hi).
  DEV void zero(int lo, int hi) const {
    float z[NJ][4];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) z[j][i] = 0.f;
    if (GRAD)
      for (int t = lo + gi; t < hi; t += G) store(t, true, z);
  }

  // The tokens [lo, hi) of one sequence: their gradients, and the sums of p over
  // them in psum, a row per wave (readable when it returns). prepare() is called
  // with the first loads under way, by the whole workgroup: it fills cnt, with a
  // barrier, and returns kappa. The next token's logits are loaded while the
  // current one is worked on.
  template <typename Prepare>
  DEV void segment(int lo, int hi, const Prepare& prepare) const {
    const float ninf = -__builtin_inff();
    auto counts_of = [&](int t) { return t < hi && (!a.mask || a.mask[t]); };
    float nx[NJ][4];
    bool nv = counts_of(lo + gi);                             // the loaded token counts
    load(lo + gi, nv, nx);
    const float kappa = GRAD ? prepare() : 0.f;
    float ps[NJ][4];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) ps[j][i] = 0.f;
    for (int tw = lo; tw < hi; tw += G) {                     // (the same passes for every lane)
      const int t = tw + gi;
      float v[NJ][4];
      const bool valid = nv;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = 4 * (li + L * j) + i < a.E ? nx[j][i] : ninf;
      nv = counts_of(t + G);
      load(t + G, nv, nx);
      float m = ninf;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaxf(m, v[j][i]);
      m = fmaxf(row_max(m), -__FLT_MAX__);                    // (finite also where every logit is -inf)
      // h: counts relative to the likeliest expert's (of equal ones the most frequent)
      float h[NJ][4];
      if (GRAD) {
        int top = 0, c[NJ][4];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const v4i q = *reinterpret_cast<const v4i*>(cnt + 4 * (li + L * j));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            c[j][i] = q[i];
            top = v[j][i] == m ? max(top, c[j][i]) : top;
          }
        }
        top = bal_max<L>(top);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) h[j][i] = (float)(c[j][i] - top);
      }
      float sum = 0.f, dot = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[j][i] = bal_exp(v[j][i] - m);
          sum += v[j][i];
          if (GRAD) dot = __builtin_fmaf(v[j][i], h[j][i], dot);
        }
      sum = row_sum(sum);
      // every logit -inf: no probability anywhere; a token that does not count: none
      const float inv = !valid || sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[j][i] *= inv;
          ps[j][i] += v[j][i];
        }
      if (GRAD) {
        dot = row_sum(dot) * inv;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[j][i] = kappa * v[j][i] * (h[j][i] - dot);
        store(t, t < hi, v);
      }
    }
    // the wave's sums: its groups of lanes joined
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      v4f x4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x = ps[j][i];
        if (L == 16) {
          const uint32_t u = __float_as_uint(x);
          const auto r16 = __builtin_amdgcn_permlane16_swap(u, u, false, false);
          x = __uint_as_float(r16[0]) + __uint_as_float(r16[1]);
          const uint32_t q = __float_as_uint(x);
          const auto r32 = __builtin_amdgcn_permlane32_swap(q, q, false, false);
          x = __uint_as_float(r32[0]) + __uint_as_float(r32[1]);
        }
        x4[i] = x;
      }
      if ((threadIdx.x & 63) < L) *reinterpret_cast<v4f*>(psum + w * kCols + 4 * (li + L * j)) = x4;
    }
    __syncthreads();
  }
  // Sum over the waves of column e.
  DEV float wave_total(int e) const {
    float v = psum[e];
#pragma unroll
    for (int i = 1; i < NT / 64; ++i) v += psum[i * kCols + e];
    return v;
  }
};

DEV float bal_kappa(const BalArgs& a, int used, int tokens) {
  const double n = (double)max(tokens, 1);
  return (float)((double)a.alpha * a.E / ((double)used * a.k * n * n));
}

template <int L, int NJ, int VEC, int GRAD>
__global__ void __launch_bounds__(256, 4) k_bal_tokens(BalArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  using BT = BalTokens<L, NJ, VEC, GRAD, 256>;
  __shared__ int red[4], s_off[kBalOff];
  const BalOff off = bal_offsets(a, s_off);
  const int t0 = blockIdx.x * a.tb, t1 = min(a.T, t0 + a.tb), E = a.E;
  const BT bt(a, lds, t0, t1);
  int used = 0;                                               // S', once it is needed
  if (blockIdx.x == 0) {
    used = bal_used(a, off, red);
    if (threadIdx.x == 0) *a.used = used;                     // (for k_bal_final)
  }
  int next = t0;                                              // tokens before it are done
  for (int s = bal_seq_of(a, off, t0); s < a.S && off(s) < t1; ++s) {
    const int lo = max(t0, off(s)), hi = min(t1, off(s + 1));
    if (lo >= hi) continue;
    bt.zero(next, lo);                                        // tokens of no sequence
    next = hi;
    bt.segment(lo, hi, [&]() {
      if (!used) used = bal_used(a, off, red);
      int r0, r1;
      bal_rows(off, s, a.cb, &r0, &r1);
      for (int e = threadIdx.x; e < BT::kCols; e += 256) {
        int c = 0;
        if (e < E) {
#pragma unroll 8
          for (int r = r0; r < r1; ++r) c += a.rowcnt[(size_t)r * E + e];
        }
        bt.cnt[e] = c;
      }
      const float kappa = bal_kappa(a, used, bal_tokens_of(a, off, s));
      __syncthreads();
      return kappa;
    });
    float* row = a.rowp + (size_t)(blockIdx.x + s) * E;
    for (int e = threadIdx.x; e < E; e += 256) row[e] = bt.wave_total(e);
    __syncthreads();
  }
  bt.zero(next, t1);                                          // tokens behind the last sequence
}

// Everything by one workgroup, for batches of a few passes of it and at most
// kBalSegs sequences: one launch instead of three (T = 64, E = 8: 22 -> 17 us a
// call, launches and host included).
template <int L, int NJ, int VEC, int GRAD, int NT>
__global__ void __launch_bounds__(NT) k_bal_one(BalArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  using BT = BalTokens<L, NJ, VEC, GRAD, NT>;
  int* hist = reinterpret_cast<int*>(lds + BT::kLds);         // [kBalSegs][E]
  __shared__ int s_n[kBalSegs], s_off[kBalOff];
  __shared__ double s_part[NT / 64];
  const BalOff off = bal_offsets(a, s_off);
  const BT bt(a, lds, 0, a.T);
  int end[kBalSegs];
#pragma unroll
  for (int q = 0; q < kBalSegs; ++q) end[q] = off(min(q + 1, a.S));
  const int first = off(0), last = end[kBalSegs - 1], nq = first < last ? bal_segs(last, end) : 0;
  if (nq) bal_count_group<NT>(a, first, last, end, nq, hist, s_n);
  int used = 0;
  for (int q = 0; q < nq; ++q) used += s_n[q] > 0;
  used = max(used, 1);
  int next = 0;
  double part = 0;
  for (int s = 0; s < a.S; ++s) {
    const int lo = off(s), hi = off(s + 1), n = s < nq && lo < hi ? s_n[s] / a.k : 0;
    if (lo < hi) {
      bt.zero(next, lo);
      next = hi;
      bt.segment(lo, hi, [&]() {
        for (int e = threadIdx.x; e < BT::kCols; e += NT) bt.cnt[e] = e < a.E ? hist[s * a.E + e] : 0;
        __syncthreads();
        return bal_kappa(a, used, n);
      });
    }
    for (int e = threadIdx.x; e < a.E; e += NT) {
      const int c = n > 0 ? hist[s * a.E + e] : 0;
      const float pm = n > 0 ? bt.wave_total(e) / (float)n : 0.f;
      a.counts[(size_t)s * a.E + e] = c;
      a.probs[(size_t)s * a.E + e] = pm;
      if (n > 0) part += (double)c * a.E / ((double)a.k * n) * pm;
    }
    __syncthreads();
  }
  bt.zero(next, a.T);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) part += __shfl_xor(part, d);
  if ((threadIdx.x & 63) == 0) s_part[threadIdx.x >> 6] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0;
    for (int i = 0; i < NT / 64; ++i) v += s_part[i];
    *a.loss = (float)((double)a.alpha / used * v);
  }
}

// Workgroup (x, s): experts [64x, 64x + 64) of sequence s (s, s + gridDim.y,
// ...): 64 groups of 16 lanes, each summing every 64th row, 4 experts per
// lane. The last workgroup to finish adds the loss.
constexpr int kBalFinalThreads = 1024;
__global__ void __launch_bounds__(kBalFinalThreads) k_bal_final(BalArgs a) {
  constexpr int NG = kBalFinalThreads / 16;
  __shared__ float redp[NG][64];
  __shared__ int redc[NG][64];
  __shared__ float redp2[16][64];
  __shared__ int redc2[16][64];
  __shared__ int s_last;
  __shared__ int s_off[kBalOff];
  const BalOff off = bal_offsets(a, s_off);
  const int tid = threadIdx.x, cl = tid & 15, grp = tid >> 4, E = a.E;
  double part = 0;
  for (int s = blockIdx.y; s < a.S; s += gridDim.y) {
    int c0, c1, p0, p1;
    bal_rows(off, s, a.cb, &c0, &c1);
    bal_rows(off, s, a.tb, &p0, &p1);
    v4f ps = v4f{0.f, 0.f, 0.f, 0.f};
    int cs[4] = {0, 0, 0, 0};
    const int e0 = blockIdx.x * 64 + 4 * cl;
    if (e0 + 4 <= E) {
#pragma unroll 8
      for (int r = p0 + grp; r < p1; r += NG) ps += *reinterpret_cast<const v4fu*>(a.rowp + (size_t)r * E + e0);
    } else {
      for (int r = p0 + grp; r < p1; r += NG)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e0 + i < E) ps[i] += a.rowp[(size_t)r * E + e0 + i];
    }
    for (int r = c0 + grp; r < c1; r += NG)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + i < E) cs[i] += a.rowcnt[(size_t)r * E + e0 + i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      redp[grp][4 * cl + i] = ps[i];
      redc[grp][4 * cl + i] = cs[i];
    }
    const int n = bal_tokens_of(a, off, s);
    __syncthreads();
    {                                                         // 64 groups to 16 sums of 4, then those
      const int col = tid & 63, q = tid >> 6;
      float p = redp[4 * q][col];
      int c = redc[4 * q][col];
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        p += redp[4 * q + i][col];
        c += redc[4 * q + i][col];
      }
      redp2[q][col] = p;
      redc2[q][col] = c;
    }
    __syncthreads();
    const int e = blockIdx.x * 64 + tid;
    if (tid < 64 && e < E) {
      float p = redp2[0][tid];
      int c = redc2[0][tid];
#pragma unroll
      for (int i = 1; i < 16; ++i) {
        p += redp2[i][tid];
        c += redc2[i][tid];
      }
      const float pm = n > 0 ? p / (float)n : 0.f;
      a.counts[(size_t)s * E + e] = c;
      a.probs[(size_t)s * E + e] = pm;
      if (n > 0) part += (double)c * E / ((double)a.k * n) * pm;
    }
  }
  // the workgroup's loss: the first wave holds it
  const int wg = blockIdx.y * gridDim.x + blockIdx.x, nwg = gridDim.x * gridDim.y;
  if (tid < 64) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) part += __shfl_xor(part, d);
    if (tid == 0) {
      st_coh(a.lpart + wg, part);
      wait_stores();                                          // the partial is in memory before it is counted
      s_last = __hip_atomic_fetch_add(a.done, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == nwg - 1;
    }
  }
  __syncthreads();
  if (!s_last || tid >= 64) return;
  double v = 0;
#pragma unroll 4
  for (int i = tid; i < nwg; i += 64) v += ld_coh(a.lpart + i);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  if (tid == 0) *a.loss = (float)((double)a.alpha / *a.used * v);
}

}  // namespace moe
