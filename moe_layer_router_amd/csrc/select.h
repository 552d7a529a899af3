// Selection of experts from router logits, and its gradient.
//
//   s = sigmoid(l) or softmax(l),  c = s + bias
//   group score = sum of the group's one or two largest c; the best groups stay
//   ids = the k experts by c (without a bias: by l) among them, ties to the lower index
//   w_j = scale s_j / sum_i s_i   (or scale s_j)
// Two experts' c may differ by less than fp32 resolves, and a wrong order there sends
// a token elsewhere: the order is that of fp64.  fp32 decides where its error cannot matter, in all but
// about one in a hundred tokens; the others are done again in fp64.
//
#pragma once
#include "device_common.h"
#include "select_host.h"

namespace moe {

// Monotone map of fp64 onto uint64 above 0 (NaN counts as -infinity, -0 as +0).
DEV uint64_t f64_order_key(double v) {
  if (!(v == v)) v = -__builtin_inf();
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}
template <int CTRL>
DEV uint64_t dpp_mov64(uint64_t x) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)x, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(x >> 32), CTRL, 0xF, 0xF, false);
  return (uint64_t)hi << 32 | lo;
}
DEV uint64_t sel_larger(uint64_t a, uint64_t b) { return a > b ? a : b; }
DEV uint64_t sel_max64(uint64_t v) {
  v = sel_larger(v, dpp_mov64<0xB1>(v));
  v = sel_larger(v, dpp_mov64<0x4E>(v));
  v = sel_larger(v, dpp_mov64<0x141>(v));
  v = sel_larger(v, dpp_mov64<0x140>(v));
  const auto l16 = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
  const auto h16 = __builtin_amdgcn_permlane16_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false);
  v = sel_larger((uint64_t)h16[0] << 32 | l16[0], (uint64_t)h16[1] << 32 | l16[1]);
  const auto l32 = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
  const auto h32 = __builtin_amdgcn_permlane32_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false);
  return sel_larger((uint64_t)h32[0] << 32 | l32[0], (uint64_t)h32[1] << 32 | l32[1]);
}
DEV float sel_readlane(float v, int lane) { return __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(v), lane)); }
DEV uint64_t sel_readlane64(uint64_t v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
  return (uint64_t)hi << 32 | lo;
}
DEV float sel_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
DEV double sel_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// Lane l holds experts 256 (i / 4) + 4 l + i % 4: four in a row, so that a load takes 16 bytes, and a
// group's lie in neighbouring lanes.
DEV int sel_expert(int lane, int i) { return 256 * (i >> 2) + 4 * lane + (i & 3); }
// (buffer loads: a uniform base and 32-bit offsets; zeros past the row's end)
template <int NV>
DEV void sel_load(const float* row, int E, int lane, float (&l)[NV]) {
  const rsrc_t r = make_rsrc(row, (uint32_t)E * 4);
  if (E % 4 == 0) {
#pragma unroll
    for (int q = 0; q < NV / 4; ++q) {
      const v4i v = buf_ld16(r, 16 * lane, 1024 * q);
#pragma unroll
      for (int j = 0; j < 4; ++j) l[4 * q + j] = __int_as_float(v[j]);
    }
  } else {                                         // (rows start on 4 bytes)
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = buf_ldf(r, 16 * lane + 4 * (i & 3), 1024 * (i >> 2));
  }
}

// What the fp64 functions take of a call.
struct SelRule {
  const float* bias;
  int E, k, sigmoid, groups, keep, top;
};
// fp64 scores of a row.  softmax: its largest logit and the sum of the exponentials (a row of -infinity: zero, no score at all; with a NaN: NaN, in every score).
struct SelRow {
  const float* l;
  float mx;
  double sum;
};
template <int UNROLL>
DEV SelRow sel_row64(const SelRule& a, const float* row) {
  SelRow r{row, -__builtin_inff(), 1.0};
  if (a.sigmoid) return r;
  const int lane = threadIdx.x & 63;
#pragma unroll 4
  for (int e = lane; e < a.E; e += 64) r.mx = fmaxf(r.mx, row[e]);
  r.mx = sel_max(r.mx);
  r.sum = 0;
#pragma unroll UNROLL
  for (int e = lane; e < a.E; e += 64) r.sum += row[e] == -__builtin_inff() ? 0.0 : exp((double)row[e] - (double)r.mx);
  r.sum = sel_sum(r.sum);
  return r;
}
DEV double sel_choice64(const SelRule& a, const SelRow& r, int e) {
  const float l = r.l[e];
  double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : r.sum == 0.0 || (l == -__builtin_inff() && r.sum == r.sum) ? 0.0 : exp((double)l - (double)r.mx) / r.sum;
  return a.bias ? s + (double)a.bias[e] : s;
}

// A token's k experts in fp64 for whatever there is in its row, expert j of them in lane j.  Few tokens get here, but a launch lasts
// until the last of them.  `buf`: E doubles of LDS of this wave's own.
__device__ __noinline__ int sel_exact(SelRule a, const float* row, double* buf) {
  const int lane = threadIdx.x & 63, n = a.E / a.groups;
  uint64_t kept = ~0ull;
  if (a.bias || a.groups > 1) {                    // (else the logits' order is the scores')
    const SelRow r = sel_row64<2>(a, row);
#pragma unroll 2
    for (int e = lane; e < a.E; e += 64) buf[e] = sel_choice64(a, r, e);
  }
  __builtin_amdgcn_wave_barrier();
  if (a.groups > 1) {
    int lg = 0;                                    // lanes of a group
    while (a.groups << (lg + 1) <= 64) ++lg;
    const int g = lane >> lg, L = 1 << lg;
    double m1 = -__builtin_inf(), m2 = m1;
    if (g < a.groups) {
      for (int e = lane & (L - 1); e < n; e += L) {
        const double v = buf[g * n + e];           // (NaN: never larger)
        if (v > m1) { m2 = m1; m1 = v; }
        else if (v > m2) m2 = v;
      }
    }
    for (int d = 1; d < L; d <<= 1) {
      const double o1 = __shfl_xor(m1, d), o2 = __shfl_xor(m2, d);
      m2 = o1 > m1 ? (m1 > o2 ? m1 : o2) : (o1 > m2 ? o1 : m2);
      m1 = o1 > m1 ? o1 : m1;
    }
    const uint64_t score = g < a.groups ? f64_order_key(a.top == 2 ? m1 + m2 : m1) : 0;
    int rank = 0;
    for (int h = 0; h < a.groups; ++h) {
      const uint64_t o = sel_readlane64(score, h << lg);
      rank += o > score || (o == score && h < g);
    }
    kept = __ballot(g < a.groups && rank < a.keep && (lane & (L - 1)) == 0);
    __builtin_amdgcn_wave_barrier();
    uint64_t* key = reinterpret_cast<uint64_t*>(buf);
    for (int e = lane; e < a.E; e += 64)
      key[e] = !(kept >> (e / n << lg) & 1) ? 0 : f64_order_key(a.bias ? buf[e] : (double)row[e]);
  } else {
    uint64_t* key = reinterpret_cast<uint64_t*>(buf);
    for (int e = lane; e < a.E; e += 64) key[e] = f64_order_key(a.bias ? buf[e] : (double)row[e]);
  }
  uint64_t* key = reinterpret_cast<uint64_t*>(buf);
  int mine = 0;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = 0;
    int at = 1 << 30;                              // the lowest index of that key
#pragma unroll 4
    for (int e = lane; e < a.E; e += 64) {
      const uint64_t v = key[e];
      if (v > best) { best = v; at = e; }
    }
    const uint64_t top = sel_max64(best), who = __ballot(best == top && at < 1 << 30);
    int id = __builtin_amdgcn_readlane(at, __builtin_ctzll(who));
    if (who & (who - 1)) {                         // (several lanes have it)
      int lowest = best == top ? at : 1 << 30;
      for (int d = 1; d < 64; d <<= 1) lowest = min(lowest, __shfl_xor(lowest, d));
      id = lowest;
    }
    if (lane == j) mine = id;
    if ((id & 63) == lane) key[id] = 0;
  }
  __builtin_amdgcn_wave_barrier();
  return mine;
}

// exp(v) by the instruction for 2^v: within 2 units, and the argument's rounding; what is below 2^-126 is zero.
DEV float sel_exp(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504f); }

// exp(v - m), m common to a row: its product's rounding is one factor of the whole row, which the sum divides out again, up to 2^(1/16)
// with |m| = kSelNear. From 1.5 10^9 on it could leave fp32's range: beyond kSelNear the difference is formed first (it is exact where it
// matters, within a factor of two of m), and an expert at -infinity has no part in the sum, also where m is.
constexpr float kSelNear = 0x1p20f;
DEV float sel_exp_from(float v, float m) { return __builtin_amdgcn_exp2f(__builtin_fmaf(v, 1.44269504f, -(m * 1.44269504f))); }
DEV float sel_exp_far(float v, float m) { return v == -__builtin_inff() ? 0.f : sel_exp(v - m); }
// Of a row with the largest logit m (in each half its own, or the wave's), and this lane's sum of them.
template <int NV>
DEV float sel_row_exps(const float (&v)[NV], float m, float (&e)[NV]) {
  const bool far = !(fabsf(m) <= kSelNear);
  float sum = 0.f;
  if (__ballot(far)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) sum += e[i] = far ? sel_exp_far(v[i], m) : sel_exp_from(v[i], m);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) sum += e[i] = sel_exp_from(v[i], m);
  }
  return sum;
}

// The same in fp32, where its rounding cannot change the result; false where it might.
//   - with u = 2^-24: the exponential's argument d (|l|, or softmax's distance to the largest logit) is off by 1.2 d u, which is s's
//     relative error, its function by 2 u, the sum, the reciprocal and the bias by 4 u, softmax's sum, common to all, by 16 u.  With S = |c| +
//     the bias's largest >= s, and d <= ln(1 / s), all of it is below S (8 + log2(1 / S)) u, softmax's below S (32 + log2(1 / S)) u.  Two c
//     (or group scores) are told apart only if they differ by more than that of both.
//   - A value that k to k + 4 of the 64 lanes' largest c reach is found by bisection.  The k best are among the experts that reach it,
//     some 1.3 k of up to 1024 (those of lanes with two of them).  They go to LDS, one to a lane, and are ranked by counting.
//   - A NaN reaches no value.  It counts as -infinity, so that it may be among the k best only where that is the value.
// Candidates too near to each other are ranked again by fp64 scores of their own.  A NaN that may matter, group scores too near to each
// other or too many candidates (few lanes with experts left) leave it all to sel_exact.
struct SelCand {
  float c[68];
  int e[64];
  float sc[20];              // by rank
  int se[20];
};
DEV float sel_wave_max(float v) { return max_row_groups(row_max16(v)); }
DEV float sel_wave_min(float v) { return -sel_wave_max(-v); }
// The two largest of a set, from those of its halves.
DEV void sel_top2(float& m1, float& m2, float o1, float o2) {
  m2 = fmaxf(fmaxf(m2, o2), fminf(m1, o1));
  m1 = fmaxf(m1, o1);
}
// The two largest over L lanes in a row (up to 32: two groups at least), from those of each.
DEV void sel_lanes_top2(float& m1, float& m2, int L) {
  if (L > 1) sel_top2(m1, m2, dpp_mov<0xB1>(m1), dpp_mov<0xB1>(m2));
  if (L > 2) sel_top2(m1, m2, dpp_mov<0x4E>(m1), dpp_mov<0x4E>(m2));
  if (L > 4) sel_top2(m1, m2, dpp_mov<0x141>(m1), dpp_mov<0x141>(m2));
  if (L > 8) sel_top2(m1, m2, dpp_mov<0x140>(m1), dpp_mov<0x140>(m2));
  if (L > 16) sel_top2(m1, m2, __shfl_xor(m1, 16), __shfl_xor(m2, 16));
}

// The m candidates `ce` of a token ranked again by their fp64 scores (without bias or groups: by the logits), through `se`.
// mx and sum: softmax's in fp32.  The sum's error (32 u, and what the largest logit's product was rounded by) moves all scores by one
// factor, so that it matters for two c only as far as their s differ: E exponentials in fp64 are formed only where that may decide.
// The factor is (1 + 32 u) e^(|mx| u) at most, which 1 + (40 + 1.1 |mx|) u covers up to |mx| = kSelNear; beyond, the sum has no such factor.
template <int UNROLL>
__device__ __noinline__ int sel_near(SelRule a, const float* row, const int* ce, int* se, int m, float mx, float sum) {
  const int lane = threadIdx.x & 63;
  const int mine = lane < m ? ce[lane] : 0;
  double c = row[mine];
  if (a.bias) c = sel_choice64(a, SelRow{row, mx, a.sigmoid ? 1.0 : (double)sum}, mine);
  const auto place = [&]() {
    const uint64_t key = lane < m ? f64_order_key(c) : 0;
    int rank = 0;
    for (int j = 0; j < m; ++j) {
      const uint64_t o = sel_readlane64(key, j);
      rank += o > key || (o == key && __builtin_amdgcn_readlane(mine, j) < mine);
    }
    return rank;
  };
  int rank = place();
  if (a.bias && !a.sigmoid) {
    const double s = c - (double)a.bias[mine], eps = 0x1p-24 * (40.0 + 1.1 * fabs((double)mx));
    bool doubt = false;
    for (int j = 0; j < m; ++j) {                  // all that are behind: one further back may differ by more in s
      const double cj = __builtin_bit_cast(double, sel_readlane64(__builtin_bit_cast(uint64_t, c), j));
      const double sj = __builtin_bit_cast(double, sel_readlane64(__builtin_bit_cast(uint64_t, s), j));
      doubt |= __builtin_amdgcn_readlane(rank, j) > rank && !(c - cj > eps * fabs(s - sj) + 0x1p-48 * (fabs(c) + fabs(cj)));
    }
    if (__ballot(lane < m && rank < a.k && doubt)) {
      c = sel_choice64(a, sel_row64<UNROLL>(a, row), mine);
      rank = place();
    }
  }
  if (lane < m && rank < a.k) se[rank] = mine;
  __builtin_amdgcn_wave_barrier();
  const int id = se[min(lane, 15)];
  __builtin_amdgcn_wave_barrier();
  return id;
}

// What scores of size S are off by, relative to it (infinite for zero: underflowed scores are told apart by none).
DEV float sel_tol(const SelArgs& a, float size) { return a.tol + 0x1p-24f * fmaxf(0.f, -__builtin_amdgcn_logf(size)); }

enum { SEL_CLEAR = 0, SEL_NEAR = 1, SEL_ALL = 2 };   // done; candidates too near; all in fp64
template <int NV, int GROUPED>
DEV int sel_fast(const SelArgs& a, int lane, float (&c)[NV], float bmax, float* buf, SelCand& q, int* count, int* id) {
  const float nan = __builtin_nanf("");            // (an expert that is out: no comparison holds)
  if (a.E != 64 * NV) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (sel_expert(lane, i) >= a.E) c[i] = nan;
  }
  if (GROUPED) {
    const int n = a.per, lg = a.lanes_log2, L = 1 << lg, g = lane >> lg;
    int fine = 0;                                  // (minima and maxima pass over a NaN)
#pragma unroll
    for (int i = 0; i < NV; ++i) fine += __popcll(__ballot(c[i] < __builtin_inff()));
    if (fine != a.E) return SEL_ALL;
    float m1 = -__builtin_inff(), m2 = m1;         // the two largest
    if (a.E % 4 == 0) {
#pragma unroll
      for (int i = 0; i < NV; i += 4)
        if (sel_expert(lane, i) < a.E) *reinterpret_cast<v4f*>(buf + sel_expert(lane, i)) = v4f{c[i], c[i + 1], c[i + 2], c[i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (sel_expert(lane, i) < a.E) buf[sel_expert(lane, i)] = c[i];
    }
    __builtin_amdgcn_wave_barrier();
    if (g < a.groups) {
      for (int e = lane & (L - 1); e < n; e += L) {
        const float v = buf[g * n + e];
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
    }
    __builtin_amdgcn_wave_barrier();
    sel_lanes_top2(m1, m2, L);
    const float score = g < a.groups ? (a.top == 2 ? m1 + m2 : m1) : nan;
    int rank = 0;
    for (int h = 0; h < a.groups; ++h)
      rank += __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(score), h << lg)) > score;
    const bool in = g < a.groups && rank < a.keep;
    const uint64_t kept = __ballot(in), last = __ballot(rank == a.keep - 1 && g < a.groups), next = __ballot(rank == a.keep && g < a.groups);
    // (equal scores share a rank, and the one behind it is missing)
    if (!last || !next) return SEL_ALL;
    const float lo = __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(score), __builtin_ctzll(last)));
    const float hi = __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(score), __builtin_ctzll(next)));
    if (!(lo - hi > sel_tol(a, fabsf(hi) + 2.0f * bmax) * (fabsf(lo) + fabsf(hi) + 4.0f * bmax))) return SEL_ALL;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      // (e / n: the quotient is at least 1 / 2048 away from the next whole number)
      const int of = (int)(((float)sel_expert(lane, i) + 0.5f) * a.per_inv);
      if (!(kept >> (of << lg & 63) & 1)) c[i] = nan;
    }
  }
  float t = c[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) t = fmaxf(t, c[i]);
  // Bisection of the lanes' largest, between what one lane of each of 16 sets at least reaches and the largest of all.
  if (!(t == t)) t = -__builtin_inff();
  float lo = max_row_groups(t), hi = row_max16(lo);
  lo = -row_max16(-lo);
  float from = -__builtin_inff();
  if (lo == from && __popcll(__ballot(t > from)) >= a.k)       // (a set without experts: the least of the lanes that have some)
    lo = sel_wave_min(t > from ? t : __builtin_inff());
  if (lo > from) {
    for (int i = 0; i < 16; ++i) {
      const float mid = 0.5f * lo + 0.5f * hi;
      const int in = __popcll(__ballot(t >= mid));
      if (in >= a.k) lo = mid; else hi = mid;
      if (in >= a.k && in <= a.k + 4) break;
    }
    from = lo - 4.0f * sel_tol(a, fabsf(lo) + bmax) * (fabsf(lo) + bmax);
  }
  int m = 0;
  int* be = reinterpret_cast<int*>(buf) + 64 * NV;             // candidates: c, and their experts
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = c[i] >= from;
    const uint64_t who = __ballot(in);
    const int at = m + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
    if (in) {
      buf[at] = c[i];
      be[at] = sel_expert(lane, i);
    }
    m += __popcll(who);
  }
  *count = m;
  if (m > 64 || m < a.k) return SEL_ALL;
  if (!GROUPED && lo == -__builtin_inff() && m != a.E) return SEL_ALL;
  __builtin_amdgcn_wave_barrier();
  const float mine = lane < m ? buf[lane] : nan;
  const int me = be[lane];
  q.c[lane] = mine;
  if (lane < 4) q.c[64 + lane] = nan;
  q.e[lane] = me;
  if (lane < 20) q.sc[lane] = nan;
  __builtin_amdgcn_wave_barrier();
  int rank = 0;
  for (int j = 0; j < m; j += 4) {
    const v4f o = *reinterpret_cast<const v4f*>(q.c + j);
    rank += (o[0] > mine) + (o[1] > mine) + (o[2] > mine) + (o[3] > mine);
  }
  if (lane < m && rank <= a.k) {
    q.sc[rank] = mine;
    q.se[rank] = me;
  }
  __builtin_amdgcn_wave_barrier();
  const int r = min(lane, 16);
  const float x = q.sc[r], y = q.sc[r + 1];        // (equal ones share a place: the next stays NaN)
  *id = q.se[r];
  __builtin_amdgcn_wave_barrier();
  const bool exact = !a.bias && !GROUPED;          // (logits themselves)
  const bool clear = x - y > (exact ? 0.f : sel_tol(a, fabsf(y) + bmax) * (fabsf(x) + fabsf(y) + 2.0f * bmax)) || (r == a.k - 1 && m == a.k);
  return __ballot(lane < a.k && !clear) ? SEL_NEAR : SEL_CLEAR;
}

// The scores of the selected experts (lane j < k: expert j, its logit lj), but for a factor
// that all of them share where `renorm` divides it out again:
//   sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)), times exp(-m), m the largest min(l, 0)
//   softmax(l): exp(l - m), m the largest of them
// so that no sum underflows however low the logits are.  Every selected expert at -infinity: zeros.
DEV float sel_scores16(bool sigmoid, bool live, float lj) {
  const float b = sigmoid ? fminf(lj, 0.f) : lj;
  const float m = row_max16(live ? b : -__builtin_inff());
  const float e = m == -__builtin_inff() && b == m ? 0.f : sel_exp(b - m);
  return !live ? 0.f : sigmoid ? e * __builtin_amdgcn_rcpf(1.0f + sel_exp(-fabsf(lj))) : e;
}

// One token per wave; GROUPED: some groups are left out.  Bound by the vector unit: 16384 tokens of 1024 experts with softmax
// scores and a bias, some 420 instructions each, take 23.0 us, 3.0 TB/s (27 us where every near-tie forms E exponentials in fp64).
template <int NV, int SIGMOID, int GROUPED>
__global__ void __launch_bounds__(64 * kSelWaves, 4) k_select(SelArgs a) {
  __shared__ __attribute__((aligned(16))) double buf[kSelWaves][64 * NV];
  __shared__ __attribute__((aligned(16))) SelCand cand[kSelWaves];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float bmax = 0.f;                                // of the finite ones
  if (a.bias) {
    float b[NV];
    sel_load<NV>(a.bias, a.E, threadIdx.x & 63, b);
#pragma unroll
    for (int i = 0; i < NV; ++i) bmax = fmaxf(bmax, fabsf(b[i]) < __builtin_inff() ? fabsf(b[i]) : 0.f);
    bmax = sel_wave_max(bmax);
  }
  const SelRule rule{a.bias, a.E, a.k, SIGMOID, a.groups, a.keep, a.top};
  const bool scored = a.bias || GROUPED;      // (else the logits' order is the scores')
  const bool dense = !SIGMOID && (!a.renorm || scored);      // softmax over all experts
  for (long t = (long)blockIdx.x * kSelWaves + w; t < a.T; t += (long)gridDim.x * kSelWaves) {
    // (opaque: what depends on the lane alone is formed again for each token, cheaper than the registers to keep it)
    const int lane = (int)opaque(threadIdx.x & 63);
    const float* row = a.logits + t * a.E;
    float c[NV], mx = 0.f, inv = 0.f, total = 1.f;   // logits, then scores, then c
    sel_load<NV>(row, a.E, lane, c);
    float b[NV];
    if (a.bias) sel_load<NV>(a.bias, a.E, lane, b);
    if (dense) {
      if (a.E != 64 * NV) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (sel_expert(lane, i) >= a.E) c[i] = -__builtin_inff();
      }
      mx = c[0];
#pragma unroll
      for (int i = 1; i < NV; ++i) mx = fmaxf(mx, c[i]);
      mx = sel_wave_max(mx);
      float e[NV];
      total = wave_sum(sel_row_exps<NV>(c, mx, e));
      inv = __builtin_amdgcn_rcpf(total);
      if (a.bias) {
#pragma unroll
        for (int i = 0; i < NV; ++i) c[i] = __builtin_fmaf(e[i], inv, b[i]);
      } else if (scored) {
#pragma unroll
        for (int i = 0; i < NV; ++i) c[i] = e[i] * inv;
      }
    } else if (scored) {
#pragma unroll
      for (int i = 0; i < NV; ++i) c[i] = __builtin_amdgcn_rcpf(1.0f + sel_exp(-c[i]));
      if (a.bias) {
#pragma unroll
        for (int i = 0; i < NV; ++i) c[i] += b[i];
      }
    }
    int e, m;
    const bool live = lane < a.k;
    const int state = sel_fast<NV, GROUPED>(a, lane, c, bmax, reinterpret_cast<float*>(buf[w]), cand[w], &m, &e);
    if (state != SEL_CLEAR) e = state == SEL_NEAR ? sel_near<NV / 4>(rule, row, cand[w].e, cand[w].se, m, mx, total) : sel_exact(rule, row, buf[w]);
    const float lj = row[live ? e : 0];
    float s;
    if (a.renorm) {
      s = sel_scores16(SIGMOID, live, lj);
      const float z = row_sum16(s);
      s = z == 0.f ? 0.f : s * __builtin_amdgcn_rcpf(z);
    } else if (SIGMOID) {
      s = __builtin_amdgcn_rcpf(1.0f + sel_exp(-lj));
    } else {
      s = total == 0.f ? 0.f : (fabsf(mx) <= kSelNear ? sel_exp_from(lj, mx) : sel_exp_far(lj, mx)) * inv;
    }
    if (live) {
      a.ids[t * a.k + lane] = e;
      a.w[t * a.k + lane] = a.scale * s;
    }
  }
}

// ------------------------------------------------------------------ up to 256 experts
// Two tokens per wave, 32 lanes each: what a token costs beside its experts (the bisection, the ranks, the weights' exponentials) is
// done for both by the same instructions.  V experts in a row per lane, twice: 32 V (i / V) + V l + i % V.
// Bound by the vector unit's instructions: 271 per token of 256 experts in 8 groups.  8192 such tokens take 7.8 us (one token per
// wave: 492 instructions, 10.4 us), one token 4.0 us.
struct SelHalf {
  float c[36];               // candidates
  int e[32];
  float sc[20];              // by rank
  int se[20];
  float g[64], gr[68];       // groups' scores, and by rank
};
template <int V>
DEV int sel_expert2(int l, int i) { return 32 * V * (i / V) + V * l + i % V; }
// Of the half's 32 lanes: from the two 16s, and over all of them.
DEV float sel_max16s(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
DEV float sel_half_max(float v) { return row_max16(sel_max16s(v)); }
DEV float sel_half_sum(float v) {
  v = row_sum16(v);
  const uint32_t u = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// A ballot's bits of this lane's half.
DEV uint32_t sel_half_bits(bool upper, uint64_t who) { return upper ? (uint32_t)(who >> 32) : (uint32_t)who; }
// A lane mask of both halves' conditions, which are the scalar unit's.
DEV uint64_t sel_halves(bool lower, bool upper) { return (lower ? 0xFFFFFFFFull : 0) | (upper ? 0xFFFFFFFFull << 32 : 0); }
DEV bool sel_lane_bit(uint64_t mask) { return __builtin_amdgcn_inverse_ballot_w64(mask); }
// Inclusive sum over the half's lanes up to this one.
DEV int sel_half_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);     // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
  return v + __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, true);   // the last lane of rows 0 and 2, in rows 1 and 3
}
// Rows of E floats at r's start, each half its own.  (What a lane without experts reads is another row's, or zeros past the last.)
template <int V>
DEV void sel_load2(rsrc_t r, int E, int l, int at, float (&c)[2 * V]) {
  if (E % V == 0) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if constexpr (V == 4) {
        const v4i v = buf_ld16(r, at + 16 * l, 512 * q);
#pragma unroll
        for (int j = 0; j < 4; ++j) c[4 * q + j] = __int_as_float(v[j]);
      } else {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, at + 8 * l, 256 * q, 0);
        c[2 * q] = __uint_as_float(v[0]);
        c[2 * q + 1] = __uint_as_float(v[1]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) c[i] = buf_ldf(r, at + 4 * V * l + 4 * (i % V), 128 * V * (i / V));
  }
}
// The groups that a token keeps: NaN for the experts of the others.  The lanes of tokens that fp32 can tell it for.
template <int V>
DEV uint64_t sel_groups2(const SelArgs& a, int l, bool upper, float (&c)[2 * V], float bmax, float* buf, SelHalf& q) {
  constexpr int NV = 2 * V;
  const float nan = __builtin_nanf("");
  const int n = a.per, lg = a.lanes_log2, L = 1 << lg;
  bool fine = true;                                // (minima and maxima pass over a NaN)
#pragma unroll
  for (int i = 0; i < NV; ++i) fine = fine && (c[i] < __builtin_inff() || sel_expert2<V>(l, i) >= a.E);
  const uint64_t bad = __ballot(!fine);
  q.g[l] = nan;
  q.g[32 + l] = nan;
  q.gr[l] = nan;
  q.gr[32 + l] = nan;
  if (l < 4) q.gr[64 + l] = nan;
  __builtin_amdgcn_wave_barrier();
  if (a.direct) {                                  // a group is V experts of each of L lanes
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float m1 = c[V * h], m2 = -__builtin_inff();
#pragma unroll
      for (int i = 1; i < V; ++i) {
        m2 = fmaxf(m2, fminf(m1, c[V * h + i]));
        m1 = fmaxf(m1, c[V * h + i]);
      }
      sel_lanes_top2(m1, m2, L);
      const int g = (32 * h + l) >> lg;
      if ((l & (L - 1)) == 0 && g < a.groups) q.g[g] = a.top == 2 ? m1 + m2 : m1;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (sel_expert2<V>(l, i) < a.E) buf[sel_expert2<V>(l, i)] = c[i];
    __builtin_amdgcn_wave_barrier();
    for (int g = l >> lg; __ballot(g < a.groups); g += 32 >> lg) {         // (all lanes: those of a group share what they found)
      float m1 = -__builtin_inff(), m2 = m1;
      if (g < a.groups) {
        for (int e = l & (L - 1); e < n; e += L) {
          const float v = buf[g * n + e];
          m2 = fmaxf(m2, fminf(m1, v));
          m1 = fmaxf(m1, v);
        }
      }
      sel_lanes_top2(m1, m2, L);
      if ((l & (L - 1)) == 0 && g < a.groups) q.g[g] = a.top == 2 ? m1 + m2 : m1;
    }
  }
  __builtin_amdgcn_wave_barrier();
  uint32_t kept[2] = {0, 0};
  for (int h = 0; 32 * h < a.groups; ++h) {        // lane l: group 32 h + l
    const float mine = q.g[32 * h + l];
    int rank = 0;
    for (int j = 0; j < a.groups; j += 4) {
      const v4f o = *reinterpret_cast<const v4f*>(q.g + j);
      rank += (o[0] > mine) + (o[1] > mine) + (o[2] > mine) + (o[3] > mine);
    }
    const bool in = 32 * h + l < a.groups;
    if (in) q.gr[rank] = mine;                     // (equal scores share a rank, and the one behind it stays NaN)
    kept[h] = sel_half_bits(upper, __ballot(in && rank < a.keep));
  }
  __builtin_amdgcn_wave_barrier();
  const float lo = q.gr[a.keep - 1], hi = q.gr[a.keep];
  __builtin_amdgcn_wave_barrier();
  if (a.direct) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int g = (32 * h + l) >> lg;
      const bool in = (g < 32 ? kept[0] >> g : kept[1] >> (g & 31)) & 1;
#pragma unroll
      for (int i = 0; i < V; ++i) c[V * h + i] = in ? c[V * h + i] : nan;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      // (e / n: the quotient is at least 1 / 512 away from the next whole number)
      const int g = (int)(((float)sel_expert2<V>(l, i) + 0.5f) * a.per_inv);
      if (!((g < 32 ? kept[0] >> g : kept[1] >> (g & 31)) & 1)) c[i] = nan;
    }
  }
  return __ballot(lo - hi > sel_tol(a, fabsf(hi) + 2.0f * bmax) * (fabsf(lo) + fabsf(hi) + 4.0f * bmax)) & sel_halves(!(uint32_t)bad, !(uint32_t)(bad >> 32));
}
// The k experts of both tokens (lane j of a half: expert j); per token SEL_*, and how many candidates.  there: of the upper half.
template <int V, int GROUPED>
DEV int sel_fast2(const SelArgs& a, int l, bool upper, bool there, float (&c)[2 * V], float bmax, float* buf, SelHalf& q,
                  int (&count)[2], int (&state)[2]) {
  constexpr int NV = 2 * V;
  const float nan = __builtin_nanf(""), none = -__builtin_inff();
  uint64_t fine = ~0ull;
  if (GROUPED) fine = sel_groups2<V>(a, l, upper, c, bmax, buf, q);
  if (a.E != 32 * NV) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (sel_expert2<V>(l, i) >= a.E) c[i] = nan;
  }
  float t = c[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) t = fmaxf(t, c[i]);
  // Bisection of the lanes' largest, between what one lane of each of 16 pairs at least reaches and the largest of all.
  if (!(t == t)) t = none;
  float lo = sel_max16s(t), hi = row_max16(lo);
  lo = -row_max16(-lo);
  uint64_t empty = __ballot(lo == none);
  if (empty) {                                     // (a pair without experts: the least of the lanes that have some)
    const uint64_t some = __ballot(t > none);
    const float least = -sel_half_max(t > none ? -t : none);
    empty &= ~sel_halves(__popc((uint32_t)some) >= a.k, __popc((uint32_t)(some >> 32)) >= a.k);
    lo = lo == none && !sel_lane_bit(empty) ? least : lo;
  }
  bool go0 = !(uint32_t)empty, go1 = there && !(uint32_t)(empty >> 32);
  for (int i = 0; i < 16 && (go0 || go1); ++i) {
    const float mid = 0.5f * lo + 0.5f * hi;
    const uint64_t in = __ballot(t >= mid);
    const int in0 = __popc((uint32_t)in), in1 = __popc((uint32_t)(in >> 32));
    const bool enough = sel_lane_bit(sel_halves(in0 >= a.k, in1 >= a.k));
    lo = enough ? mid : lo;
    hi = enough ? hi : mid;
    go0 = go0 && !(in0 >= a.k && in0 <= a.k + 4);
    go1 = go1 && !(in1 >= a.k && in1 <= a.k + 4);
  }
  const float from = lo == none ? none : lo - 4.0f * sel_tol(a, fabsf(lo) + bmax) * (fabsf(lo) + bmax);
  int mine_n = 0;                                  // a lane's candidates
#pragma unroll
  for (int i = 0; i < NV; ++i) mine_n += c[i] >= from;
  const int upto = sel_half_scan(mine_n);
  int m0 = __builtin_amdgcn_readlane(upto, 31), m1 = __builtin_amdgcn_readlane(upto, 63);
  fine &= sel_halves(m0 >= a.k && m0 <= 32, m1 >= a.k && m1 <= 32);
  if (!GROUPED) {                                  // (a NaN where experts at -infinity are needed)
    const uint64_t last = __ballot(lo == none);
    fine &= ~sel_halves((uint32_t)last && m0 != a.E, (uint32_t)(last >> 32) && m1 != a.E);
  }
  m0 = min(m0, 32);
  m1 = min(m1, 32);
  const int m = upper ? m1 : m0;
  int at = upto - mine_n;
  if (upto <= 32) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (c[i] >= from) {
        q.c[at] = c[i];
        q.e[at++] = sel_expert2<V>(l, i);
      }
    }
  }
  __builtin_amdgcn_wave_barrier();
  const float mine = l < m ? q.c[l] : nan;
  const int me = q.e[l];
  if (l >= m) q.c[l] = nan;
  if (l < 20) q.sc[l] = nan;
  __builtin_amdgcn_wave_barrier();
  int rank = 0;
  for (int j = 0; j < max(m0, m1); j += 4) {
    const v4f o = *reinterpret_cast<const v4f*>(q.c + j);
    rank += (o[0] > mine) + (o[1] > mine) + (o[2] > mine) + (o[3] > mine);
  }
  if (l < m && rank <= a.k) {
    q.sc[rank] = mine;
    q.se[rank] = me;
  }
  __builtin_amdgcn_wave_barrier();
  const int r = min(l, 16);
  const float x = q.sc[r], y = q.sc[r + 1];        // (equal ones share a place: the next stays NaN)
  const int id = q.se[r];
  __builtin_amdgcn_wave_barrier();
  const bool exact = !a.bias && !GROUPED;          // (logits themselves)
  const bool clear = x - y > (exact ? 0.f : sel_tol(a, fabsf(y) + bmax) * (fabsf(x) + fabsf(y) + 2.0f * bmax)) || (r == a.k - 1 && m == a.k);
  const uint64_t near = __ballot(l < a.k && !clear);
  count[0] = m0;
  count[1] = m1;
  state[0] = !(uint32_t)fine ? SEL_ALL : (uint32_t)near ? SEL_NEAR : SEL_CLEAR;
  state[1] = !there ? SEL_CLEAR : !(uint32_t)(fine >> 32) ? SEL_ALL : (uint32_t)(near >> 32) ? SEL_NEAR : SEL_CLEAR;
  return id;
}

template <int V, int SIGMOID, int GROUPED>
__global__ void __launch_bounds__(64 * kSelWaves, 4) k_select_pair(SelArgs a) {
  constexpr int NV = 2 * V;
  __shared__ __attribute__((aligned(16))) double buf[kSelWaves][32 * NV];
  __shared__ __attribute__((aligned(16))) SelHalf half[kSelWaves][2];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, l = lane & 31;
  const bool upper = lane >= 32;
  const long t0 = 2 * ((long)blockIdx.x * kSelWaves + w);
  if (t0 >= a.T) return;
  const SelRule rule{a.bias, a.E, a.k, SIGMOID, a.groups, a.keep, a.top};
  const bool scored = a.bias || GROUPED;      // (else the logits' order is the scores')
  const bool dense = !SIGMOID && (!a.renorm || scored);      // softmax over all experts
  float b[NV], bmax = 0.f;                         // of the finite ones
  if (a.bias) {
    sel_load2<V>(make_rsrc(a.bias, (uint32_t)a.E * 4), a.E, l, 0, b);
#pragma unroll
    for (int i = 0; i < NV; ++i) bmax = fmaxf(bmax, fabsf(b[i]) < __builtin_inff() ? fabsf(b[i]) : 0.f);
    bmax = sel_half_max(bmax);
  }
  const bool two = uni(t0 + 1 < a.T);
  const float* row = a.logits + t0 * a.E;
  float c[NV], mx = 0.f, inv = 0.f, total = 1.f;   // logits, then scores, then c
  sel_load2<V>(make_rsrc(row, (two ? 8 : 4) * (uint32_t)a.E), a.E, l, upper ? 4 * a.E : 0, c);
  if (dense) {
    if (a.E != 32 * NV) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (sel_expert2<V>(l, i) >= a.E) c[i] = -__builtin_inff();
    }
    mx = c[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) mx = fmaxf(mx, c[i]);
    mx = sel_half_max(mx);
    float e[NV];
    total = sel_half_sum(sel_row_exps<NV>(c, mx, e));
    inv = __builtin_amdgcn_rcpf(total);
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < NV; ++i) c[i] = __builtin_fmaf(e[i], inv, b[i]);
    } else if (scored) {
#pragma unroll
      for (int i = 0; i < NV; ++i) c[i] = e[i] * inv;
    }
  } else if (scored) {
#pragma unroll
    for (int i = 0; i < NV; ++i) c[i] = __builtin_amdgcn_rcpf(1.0f + sel_exp(-c[i]));
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < NV; ++i) c[i] += b[i];
    }
  }
  SelHalf& q = half[w][upper];
  int m[2], state[2];
  int e = sel_fast2<V, GROUPED>(a, l, upper, two, c, bmax, reinterpret_cast<float*>(buf[w]) + (upper ? 32 * NV : 0), q, m, state);
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {                  // the tokens that fp32 does not settle, the whole wave at each
    const int st = h ? state[1] : state[0];
    if (st == SEL_CLEAR) continue;
    const float* r = row + (long)h * a.E;
    const int id = st == SEL_NEAR ? sel_near<NV / 4>(rule, r, half[w][h].e, half[w][h].se, h ? m[1] : m[0],
                                                      sel_readlane(mx, 32 * h), sel_readlane(total, 32 * h))
                                  : sel_exact(rule, r, buf[w]);
    const int mine = __shfl(id, l & 15);
    if (upper == (h == 1)) e = mine;
  }
  const bool live = l < a.k && (two || !upper);
  const float lj = row[live ? (upper ? a.E : 0) + e : 0];
  float s;
  if (a.renorm) {
    s = sel_scores16(SIGMOID, live, lj);
    const float z = row_sum16(s);
    s = z == 0.f ? 0.f : s * __builtin_amdgcn_rcpf(z);
  } else if (SIGMOID) {
    s = __builtin_amdgcn_rcpf(1.0f + sel_exp(-lj));
  } else {
    s = total == 0.f ? 0.f : (fabsf(mx) <= kSelNear ? sel_exp_from(lj, mx) : sel_exp_far(lj, mx)) * inv;
  }
  if (live) {
    const size_t at = (size_t)(t0 + upper) * a.k + l;
    a.ids[at] = e;
    a.w[at] = a.scale * s;
  }
}

// ------------------------------------------------------------------ gradient
// d_j = scale dw_j, with renorm d_j = (scale dw_j - sum_i q_i scale dw_i) / sum_i s_i, q = s / sum s;
//   sigmoid: dl_j = d_j s_j (1 - s_j), zero elsewhere
//   softmax: dl_e = s_e ([e selected] d_e - sum_i s_i d_i); with renorm the sum is zero: dl_j = q_j (...)
// The differences cancel (1 - s of a sure expert, dw against its mean): they are formed in
// fp64, which only the k selected experts need.  Softmax's sum over all experts is fp32's: s, and 1 - s with it, are off by some 16 2^-24.
// An expert that stands twice among a token's ids has the sum of both entries.
//
// A wave does four tokens at a time: their selected experts in the four rows of 16 lanes, their rows of E one after another.
// Bound by the rows' way through memory with many experts (16384 tokens of 1024, dense: 27 us, 5 TB/s), by latency with
// few (8192 tokens of 256, sparse: 5.4 us).
template <int CTRL>
DEV double dpp_movd(double v) { return __builtin_bit_cast(double, dpp_mov64<CTRL>(__builtin_bit_cast(uint64_t, v))); }
DEV double sel_row_sum16(double v) {
  v += dpp_movd<0xB1>(v);
  v += dpp_movd<0x4E>(v);
  v += dpp_movd<0x141>(v);
  return v + dpp_movd<0x140>(v);
}
DEV double sel_row_max16(double v) {
  v = fmax(v, dpp_movd<0xB1>(v));
  v = fmax(v, dpp_movd<0x4E>(v));
  v = fmax(v, dpp_movd<0x141>(v));
  return fmax(v, dpp_movd<0x140>(v));
}

// Lane j of a row: the id (-1: none, or an earlier slot has it) and the gradient of its logit lj, d = scale dw.  Softmax without renorm: d_j s_j
// alone, s = exp(lj - mx) / sum, and *inner the sum of them over the token, which every expert's has to lose times its s.
DEV void sel_grad16(const SelArgs& a, bool live, double d, double lj, double mx, double sum, int* id, double* g, double* inner) {
  double v = 0;
  *inner = 0;
  if (a.renorm) {
    const double b = a.sigmoid ? fmin(lj, 0.0) : lj, m = sel_row_max16(live ? b : -__builtin_inf());
    double s = m == -__builtin_inf() && b == m ? 0.0 : exp(b - m);
    const double f = a.sigmoid ? exp(-fabs(lj)) : 0.0;         // s (1 - s) = f / (1 + f)^2
    if (a.sigmoid) s /= 1.0 + f;
    if (!live) s = 0;
    const double z = sel_row_sum16(s), q = z == 0.0 ? 0.0 : s / z;
    v = q * (d - sel_row_sum16(live ? q * d : 0.0));
    if (a.sigmoid) v *= lj > 0.0 ? f / (1.0 + f) : 1.0 / (1.0 + f);
  } else if (a.sigmoid) {
    const double f = exp(-fabs(lj));
    v = d * (f / ((1.0 + f) * (1.0 + f)));
  } else {
    const double s = sum == 0.0 ? 0.0 : exp(lj - mx) / sum;
    v = s * d;
    *inner = sel_row_sum16(live ? v : 0.0);
  }
  // the first of equal ids takes the others' share
  const int lane = threadIdx.x & 63, j = lane & 15;
  if (!live) *id = -1 - j;                         // (no two of them alike)
  bool twice = false;
#define SEL_ROR(N) twice |= __builtin_amdgcn_mov_dpp(*id, 0x120 + N, 0xF, 0xF, false) == *id
  SEL_ROR(1); SEL_ROR(2); SEL_ROR(3); SEL_ROR(4); SEL_ROR(5); SEL_ROR(6); SEL_ROR(7); SEL_ROR(8);
#undef SEL_ROR
  if (__ballot(twice)) {
    double total = 0;
    bool first = true;
    for (int i = 0; i < 16; ++i) {
      const int o = __shfl(*id, (lane & 48) + i);
      const double ov = __shfl(v, (lane & 48) + i);
      if (o == *id) {
        total += ov;
        first = first && i >= j;
      }
    }
    v = total;
    if (!first) *id = -1;
  }
  *g = v;
}

// DENSE: softmax scores without renorm: every expert of a token has a gradient.
template <int NV, int SPLIT, int DENSE>
__global__ void __launch_bounds__(64 * kSelWaves) k_select_bwd(SelArgs a) {
  __shared__ __attribute__((aligned(16))) float buf[kSelWaves][64 * NV];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, j = lane & 15;
  for (long t0 = ((long)blockIdx.x * kSelWaves + w) * 4; t0 < a.T; t0 += (long)gridDim.x * kSelWaves * 4) {
    const long t = min(t0 + (lane >> 4), a.T - 1);
    const bool live = j < a.k;
    const size_t f = (size_t)t * a.k + (live ? j : 0);
    int id = min(max(a.ids_in[f], 0), a.E - 1);
    const double d = live ? (double)a.scale * a.dw[f] : 0.0;
    const float lj = a.logits[t * a.E + id];
    float mx = 0.f, sum = 0.f;
    float l[DENSE ? 4 : 1][NV];                    // logits, then their exponentials
    if (DENSE) {
#pragma unroll
      for (int r = 0; r < 4; ++r) sel_load<NV>(a.logits + min(t0 + r, a.T - 1) * a.E, a.E, lane, l[DENSE * r]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float(&e)[NV] = l[DENSE * r];
        if (a.E != 64 * NV) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (sel_expert(lane, i) >= a.E) e[i] = -__builtin_inff();
        }
        float m = e[0], s = 0.f;
#pragma unroll
        for (int i = 1; i < NV; ++i) m = fmaxf(m, e[i]);
        m = sel_wave_max(m);
#pragma unroll
        for (int i = 0; i < NV; ++i) s += e[i] = sel_exp_far(e[i], m);
        s = wave_sum(s);
        if (lane >> 4 == r) { mx = m; sum = s; }
      }
    }
    double g, inner;
    sel_grad16(a, live, d, lj, mx, sum, &id, &g, &inner);
    const double s = DENSE && sum != 0.f ? exp((double)lj - (double)mx) / sum : 0.0;
    const float at_id = (float)(g - s * inner), scale = sum == 0.f ? 0.f : (float)(-inner / sum);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (t0 + r >= a.T) break;
      float v[NV];
      const float c = __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(scale), 16 * r));
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = DENSE ? c * l[DENSE * r][i] : 0.f;
#pragma unroll
      for (int q = 0; q < NV / 4; ++q)
        *reinterpret_cast<v4f*>(buf[w] + sel_expert(lane, 4 * q)) = v4f{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      __builtin_amdgcn_wave_barrier();
      if (lane >> 4 == r && id >= 0) buf[w][id] = at_id;
      __builtin_amdgcn_wave_barrier();
      const size_t o0 = (size_t)(t0 + r) * a.E;
      if (SPLIT) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = lane + 64 * i;
          if (e >= a.E) continue;
          float x = buf[w][e];
          if (a.aux) x += a.aux[o0 + e];
          const uint32_t h = f32_to_bf16_rne(x);
          a.hi[o0 + e] = (uint16_t)h;
          a.lo[o0 + e] = (uint16_t)f32_to_bf16_rne(x - bf16_to_f32(h));
        }
      } else if (a.E % 4 == 0) {
#pragma unroll
        for (int q = 0; q < NV / 4; ++q)
          if (sel_expert(lane, 4 * q) < a.E)
            *reinterpret_cast<v4f*>(a.dl + o0 + sel_expert(lane, 4 * q)) = *reinterpret_cast<const v4f*>(buf[w] + sel_expert(lane, 4 * q));
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (lane + 64 * i < a.E) a.dl[o0 + lane + 64 * i] = buf[w][lane + 64 * i];
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

}  // namespace moe
