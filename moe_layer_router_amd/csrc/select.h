// Selection of experts from router logits, and its gradient.
//
//   s = sigmoid(l) or softmax(l),  c = s + bias
//   group score = sum of the group's one or two largest c; the best groups stay
//   ids = the k experts by c (without a bias: by l) among them, ties to the lower index
//   w_j = scale s_j / sum_i s_i   (or scale s_j)
// Two experts' c may differ by less than fp32 resolves, and a wrong order there sends
// a token elsewhere: c, group scores and their comparisons are fp64.
//
// One wave per token.
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
DEV double sel_shfl_xor(double v, int d) { return __shfl_xor(v, d); }
DEV uint64_t sel_max64(uint64_t v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t o = (uint64_t)__shfl_xor((unsigned long long)v, d);
    v = o > v ? o : v;
  }
  return v;
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

// A token's k experts in fp64, expert j of them in lane j.  Lane l holds experts
// l + 64 i; `buf`: E doubles of LDS of this wave's own.
template <int NV>
DEV int sel_exact(const SelArgs& a, const float (&l)[NV], double* buf) {
  const int lane = threadIdx.x & 63;
  const bool need = a.bias || a.groups > 1;        // (the logits' order is the scores')
  uint64_t alive = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (lane + 64 * i < a.E) alive |= 1ull << i;
  double c[NV];
  if (need) {
    float mx = -__builtin_inff();
    double sum = 0;
    if (!a.sigmoid) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (alive >> i & 1) mx = fmaxf(mx, l[i]);
      mx = sel_max(mx);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      // (a row of -infinity: no score at all)
      if (a.sigmoid) c[i] = 1.0 / (1.0 + exp(-(double)l[i]));
      else c[i] = mx == -__builtin_inff() && l[i] == mx ? 0.0 : exp((double)l[i] - (double)mx);
      if (alive >> i & 1) sum += c[i];
    }
    if (!a.sigmoid) {
      sum = sel_sum(sum);
#pragma unroll
      for (int i = 0; i < NV; ++i) c[i] = sum == 0.0 ? 0.0 : c[i] / sum;
    }
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < NV; ++i) c[i] += (double)a.bias[min(lane + 64 * i, a.E - 1)];
    }
  }
  if (a.groups > 1) {
    const int n = a.E / a.groups;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (alive >> i & 1) buf[lane + 64 * i] = c[i];
    __builtin_amdgcn_wave_barrier();
    double m1 = -__builtin_inf(), m2 = m1;
    if (lane < a.groups) {
      for (int e = 0; e < n; ++e) {
        const double v = buf[lane * n + e];        // (NaN: never larger)
        if (v > m1) { m2 = m1; m1 = v; }
        else if (v > m2) m2 = v;
      }
    }
    __builtin_amdgcn_wave_barrier();
    const uint64_t score = lane < a.groups ? f64_order_key(a.top == 2 ? m1 + m2 : m1) : 0;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const uint64_t o = (uint64_t)__shfl((unsigned long long)score, g);
      rank += o > score || (o == score && g < lane);
    }
    const uint64_t kept = __ballot(lane < a.groups && rank < a.keep);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (!(kept >> (min(lane + 64 * i, a.E - 1) / n) & 1)) alive &= ~(1ull << i);
  }
  uint64_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) key[i] = alive >> i & 1 ? f64_order_key(a.bias ? c[i] : (double)l[i]) : 0;
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) best = key[i] > best ? key[i] : best;
    best = sel_max64(best);
    int e = 1 << 30;                               // the lowest index of that key
#pragma unroll
    for (int i = NV - 1; i >= 0; --i)
      if (key[i] == best) e = lane + 64 * i;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) e = min(e, __shfl_xor(e, d));
    if (lane == j) mine = e;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 64 * i == e) key[i] = 0;
  }
  return mine;
}

// The scores of the selected experts (lane j < k: expert j, its logit lj), but for a factor
// that all of them share where `renorm` divides it out again:
//   sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)), times exp(-m), m the largest min(l, 0)
//   softmax(l): exp(l - m), m the largest of them
// so that no sum underflows however low the logits are.  Every selected expert at -infinity: zeros.
DEV float sel_scores16(bool sigmoid, bool live, float lj) {
  const float b = sigmoid ? fminf(lj, 0.f) : lj;
  const float m = row_max16(live ? b : -__builtin_inff());
  const float e = m == -__builtin_inff() && b == m ? 0.f : expf(b - m);
  return !live ? 0.f : sigmoid ? e / (1.0f + expf(-fabsf(lj))) : e;
}

template <int NV>
__global__ void __launch_bounds__(64 * kSelWaves) k_select(SelArgs a) {
  __shared__ double buf[kSelWaves][64 * NV];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (long t = (long)blockIdx.x * kSelWaves + w; t < a.T; t += (long)gridDim.x * kSelWaves) {
    const float* row = a.logits + t * a.E;
    float l[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = row[min(lane + 64 * i, a.E - 1)];
    const int e = sel_exact<NV>(a, l, buf[w]);
    const bool live = lane < a.k;
    const float lj = row[live ? e : 0];
    float s;
    if (a.renorm) {
      s = sel_scores16(a.sigmoid, live, lj);
      const float sum = row_sum16(s);
      s = sum == 0.f ? 0.f : s / sum;
    } else if (a.sigmoid) {
      s = 1.0f / (1.0f + expf(-lj));
    } else {
      float mx = l[0], sum = 0.f;
#pragma unroll
      for (int i = 1; i < NV; ++i) mx = fmaxf(mx, l[i]);
      mx = sel_max(mx);
#pragma unroll
      for (int i = 0; i < NV; ++i) sum += lane + 64 * i < a.E ? expf(l[i] - mx) : 0.f;
      sum = wave_sum(sum);
      s = mx == -__builtin_inff() ? 0.f : expf(lj - mx) / sum;
    }
    if (live) {
      a.ids[t * a.k + lane] = e;
      a.w[t * a.k + lane] = a.scale * s;
    }
  }
}

// ------------------------------------------------------------------ gradient
// d_j = scale dw_j, with renorm d_j = (scale dw_j - sum_i q_i scale dw_i) / sum_i s_i, q = s / sum s;
//   sigmoid: dl_j = d_j s_j (1 - s_j), zero elsewhere
//   softmax: dl_e = s_e ([e selected] d_e - sum_i s_i d_i); with renorm the sum is zero: dl_j = q_j (...)
// The differences cancel (1 - s of a sure expert, dw against its mean): they are formed in
// fp64, which only the k selected experts need.
// An expert that stands twice among a token's ids has the sum of both entries.
DEV double sel_row_sum16(double v) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// Lane j < k: the id and the gradient of its logit (softmax without renorm: d_j s_j alone, and
// *inner the sum of them over the token, which every expert's has to lose times its s).
DEV void sel_grad16(const SelArgs& a, long t, const float* row, float mx, double sum, int* id, double* g, double* inner) {
  const int lane = threadIdx.x & 63;
  const bool live = lane < a.k;
  const size_t f = (size_t)t * a.k + (live ? lane : 0);
  *id = min(max(a.ids_in[f], 0), a.E - 1);
  const double d = live ? (double)a.scale * a.dw[f] : 0.0;
  const double lj = row[*id];
  double v = 0;
  *inner = 0;
  if (a.renorm) {
    double b = a.sigmoid ? fmin(lj, 0.0) : lj, m = live ? b : -__builtin_inf();
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) m = fmax(m, __shfl_xor(m, x));
    double s = m == -__builtin_inf() && b == m ? 0.0 : exp(b - m);
    if (a.sigmoid) s /= 1.0 + exp(-fabs(lj));
    if (!live) s = 0;
    const double z = sel_row_sum16(s), q = z == 0.0 ? 0.0 : s / z;
    v = q * (d - sel_row_sum16(q * d));
    if (a.sigmoid) v *= 1.0 / (1.0 + exp(lj));     // 1 - s
  } else if (a.sigmoid) {
    const double e = exp(-fabs(lj));               // s (1 - s)
    v = d * (e / ((1.0 + e) * (1.0 + e)));
  } else {
    const double s = sum == 0.0 ? 0.0 : exp(lj - (double)mx) / sum;
    v = s * d;
    *inner = sel_row_sum16(live ? v : 0.0);
  }
  // the first of equal ids takes the others' share
  double total = 0;
  bool first = live;
  for (int j = 0; j < a.k; ++j) {
    const int o = __shfl(*id, j);
    const double ov = __shfl(v, j);
    if (o == *id) {
      total += ov;
      if (j < lane) first = false;
    }
  }
  if (!first) *id = -1;
  *g = total;
  *inner = __shfl(*inner, 0);
}

template <int NV, int SPLIT>
__global__ void __launch_bounds__(64 * kSelWaves) k_select_bwd(SelArgs a) {
  __shared__ float buf[kSelWaves][64 * NV];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const bool dense = !a.sigmoid && !a.renorm;
  for (long t = (long)blockIdx.x * kSelWaves + w; t < a.T; t += (long)gridDim.x * kSelWaves) {
    const float* row = a.logits + t * a.E;
    float l[NV], mx = 0.f;
    double sum = 0;
    if (dense) {
#pragma unroll
      for (int i = 0; i < NV; ++i) l[i] = row[min(lane + 64 * i, a.E - 1)];
      mx = l[0];
#pragma unroll
      for (int i = 1; i < NV; ++i) mx = fmaxf(mx, l[i]);
      mx = sel_max(mx);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        l[i] = mx == -__builtin_inff() ? 0.f : expf(l[i] - mx);
        if (lane + 64 * i < a.E) sum += l[i];
      }
      sum = sel_sum(sum);
    }
    int id;
    double g, inner;
    sel_grad16(a, t, row, mx, sum, &id, &g, &inner);
    const float scale = dense && sum != 0.0 ? (float)(-inner / sum) : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) buf[w][lane + 64 * i] = dense ? scale * l[i] : 0.f;
    __builtin_amdgcn_wave_barrier();
    if (id >= 0) {
      const double s = dense ? (sum == 0.0 ? 0.0 : exp((double)row[id] - (double)mx) / sum) : 0.0;
      buf[w][id] = (float)(g - s * inner);
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      if (e >= a.E) continue;
      const size_t o = (size_t)t * a.E + e;
      float v = buf[w][e];
      if (!SPLIT) {
        a.dl[o] = v;
        continue;
      }
      if (a.aux) v += a.aux[o];
      const uint32_t h = f32_to_bf16_rne(v);
      a.hi[o] = (uint16_t)h;
      a.lo[o] = (uint16_t)f32_to_bf16_rne(v - bf16_to_f32(h));
    }
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace moe
