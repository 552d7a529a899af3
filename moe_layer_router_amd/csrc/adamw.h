// An AdamW step over many tensors in one launch.
//
//   g = grad_scale * grad
//   m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2
//   w' = w - lr decay w - (lr / c1) m' / (sqrt(v') / sqrt(c2) + eps),  c_i = 1 - b_i^t
// in fp32.  States of 8 bits: m and sqrt(v) as E4M3 codes, a scale per 128 elements
// (largest magnitude / 448).  The root, since it spans half the range of v in powers
// of two; it is what the update needs.
//
// Rounding to 8 bits, and of BF16 weights without fp32 master weights, is stochastic: up with the
// probability that the dropped part has.  To nearest, what a step changes by less than half
// a code's distance would never change: v moves by 1 - b2 = 1/1000 of itself, E4M3's
// codes lie 1/8 to 1/16 apart, and v would stand still until g^2 is some 90 times it.  The 16 random
// bits are a hash of (seed, step, tensor, element), so that the same call gives the same bits.
// A nonzero root is never stored as zero: its element's next update would be divided by
// the root of (1 - b2) g^2 alone.
//
// Bound by HBM with fp32 states: 352 M BF16 weights with masters 1.97 ms, 5.4 TB/s.  With 8-bit states and stochastic BF16 weights by vector
// instructions too (some 90 an element, a seventh of them the hash): 40 M weights 96 us, 5.1 TB/s.  A thread does 8 elements and
// ends: with 32 (a workgroup's 8192) these take 1.99 ms and 117 us.  Five small tensors: 7 us, a launch and one round trip to memory.
#pragma once
#include "elements.h"

namespace moe {

// kernel arguments hold 4 KB: 48 tensors a launch
constexpr int kAdamTensors = 48, kAdamThreads = 256, kAdamChunk = 8 * kAdamThreads;

struct AdamTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;                 // scales of 8-bit states
  float* vs;
  float* master;             // fp32 weights, or NULL
  int64_t n;
  float decay;
  int32_t index;             // the tensor's place in the call
};

struct AdamArgs {
  AdamTensor t[kAdamTensors];
  uint32_t first[kAdamTensors + 1];      // first chunk of each tensor
  int count;
  float b1, a1, b2, a2, eps;             // a = 1 - b
  float lr, step, rs;                    // lr, lr / c1, 1 / sqrt(c2)
  uint32_t seed, t_lo;                   // t_lo: the step's low 32 bits
  const float* grad_scale;               // device scalars, or NULL
  const float* lr_dev;
  const int64_t* t_dev;
  double log_b1, log_b2;
};
static_assert(sizeof(AdamArgs) <= 4096, "kernel arguments");

enum { ADAM_F32 = 0, ADAM_BF16 = 1, ADAM_MASTER = 2 };   // weights: fp32, BF16 alone, BF16 with fp32 master weights

// A 32-bit mixing function: xor-shifts and products with odd constants (the binary
// digits of sqrt(2) and sqrt(3)).
DEV uint32_t adam_mix(uint32_t x) {
  x ^= x >> 15;
  x *= 0x6A09E667u;
  x ^= x >> 13;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// E4M3 code of the magnitude a (at most 448 but for rounding), rounded up with probability (dropped part) by the 16 bits r.
DEV uint32_t adam_e4m3(float a, uint32_t r) {
  a = fminf(a, 448.0f);
  // from 2^-6 on 20 bits of the fraction are dropped; below, codes are multiples of 2^-9
  const uint32_t normal = ((__float_as_uint(a) + (r << 4)) >> 20) - (120u << 3);
  const uint32_t small = ((uint32_t)(a * 0x1p25f) + r) >> 16;
  return a < 0x1p-6f ? small : normal;
}
// fp32 to BF16 in the same way; infinities and (quiet) NaN as they are.
DEV uint32_t adam_bf16(float x, uint32_t r) {
  const uint32_t u = __float_as_uint(x);
  return (u + (__builtin_isfpclass(x, 0x207) ? 0 : r)) >> 16;      // (NaN, infinities: their classes)
}
// The square root of x >= 2^-96 (or zero), correctly rounded: the instruction's result s, at most a unit off, or one of its neighbours, by
// Tuckerman's test.  The root lies below s - ulp / 2, half way to the neighbour below, where x < (s - ulp / 2)^2 = s (s - ulp) + ulp^2 / 4;
// x and s (s - ulp) are multiples of ulp^2, so that this is x <= s (s - ulp), and above half way up likewise x > s (s + ulp).
// A fused residue has the exact difference's sign.
DEV float adam_sqrt(float x) {
  const float s = __builtin_amdgcn_sqrtf(x);
  const float down = __uint_as_float(__float_as_uint(s) - 1), up = __uint_as_float(__float_as_uint(s) + 1);
  float y = __builtin_fmaf(-down, s, x) <= 0.f ? down : s;
  return __builtin_fmaf(-up, s, x) > 0.f ? up : y;
}

DEV uint32_t row_max16_u32(uint32_t v) {
  uint32_t o;
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false); v = max(v, o);
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false); v = max(v, o);
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false); v = max(v, o);
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false); v = max(v, o);
  return v;
}

// b x + a y with every operation rounded on its own, as the formulas are read one operation at a time: a sum
// fused with a product may differ in the last bit, which can decide a stochastic rounding.
DEV float adam_mean(float b, float x, float a, float y) {
#pragma clang fp contract(off)
  const float p = b * x, q = a * y;
  return p + q;
}

// 8 elements from i on (those at n and past it zero).
template <int BF>
DEV void adam_load(const void* p, int64_t i, int64_t n, float (&v)[8]) {
  if (i + 8 <= n) {
    ln_unpack<BF ? LN_BF16 : LN_F32>(ln_load<BF ? LN_BF16 : LN_F32>(p, i), v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = i + e >= n ? 0.f : BF ? bf16_to_f32(static_cast<const uint16_t*>(p)[i + e]) : static_cast<const float*>(p)[i + e];
}
DEV void adam_store_f32(float* p, int64_t i, int64_t n, const float (&v)[8]) {
  if (i + 8 <= n) return ln_store_f32(p, i, v);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < n) p[i + e] = v[e];
}
DEV void adam_load_fp8(const void* p, int64_t i, int64_t n, float s, float (&v)[8]) {
  const uint8_t* q = static_cast<const uint8_t*>(p) + i;
  uint32_t w[2] = {0, 0};
  if (i + 8 <= n) {
    const v2u b = *reinterpret_cast<const v2u*>(q);
    w[0] = b[0]; w[1] = b[1];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i + e < n) w[e >> 2] |= (uint32_t)q[e] << (8 * (e & 3));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
    v[4 * h] = lo[0] * s; v[4 * h + 1] = lo[1] * s;
    v[4 * h + 2] = hi[0] * s; v[4 * h + 3] = hi[1] * s;
  }
}
// 8 elements of a block whose 16 lanes are a DPP row: codes, and the block's scale.  A block with
// something not finite gets a NaN scale, one below 2^-100 zeros.
template <int ROOT>
DEV void adam_store_fp8(void* p, float* scales, int64_t i, int64_t n, const float (&v)[8], const uint32_t (&r)[8]) {
  uint32_t mx = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) mx = max(mx, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  mx = row_max16_u32(mx);
  const float amax = __uint_as_float(mx);
  const bool tiny = mx < 0x0D800000u;              // 2^-100
  const float s = mx >= 0x7F800000u ? __builtin_nanf("") : tiny ? 1.0f : amax * (1.0f / 448.0f);
  const float inv = tiny ? 0.0f : 1.0f / s;
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint32_t c = adam_e4m3(ROOT ? v[e] * inv : fabsf(v[e] * inv), r[e]);
    if (ROOT) c = max(c, min(__float_as_uint(v[e]), 1u));
    else c |= __float_as_uint(v[e]) >> 24 & 0x80u;
    w[e >> 2] |= c << (8 * (e & 3));
  }
  uint8_t* q = static_cast<uint8_t*>(p) + i;
  if (i + 8 <= n) {
    *reinterpret_cast<v2u*>(q) = v2u{w[0], w[1]};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i + e < n) q[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
  }
  if ((threadIdx.x & 15) == 0 && i < n) scales[i / 128] = s;
}

// Workgroup b does chunk b of the tensors one after another, 8 elements per thread.
template <int W, int GBF, int S8>
__global__ void __launch_bounds__(kAdamThreads) k_adamw(const AdamArgs a) {
  float gs = 1.0f;
  if (a.grad_scale) {
    gs = *a.grad_scale;
    if (!(fabsf(gs) < __builtin_inff())) return;   // the step is left out
  }
  int lo = 0, hi = a.count;                        // the last tensor whose first chunk is not behind this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.first[mid] <= blockIdx.x) lo = mid; else hi = mid;
  }
  const AdamTensor& t = a.t[lo];
  const int64_t n = t.n, i = (int64_t)(blockIdx.x - a.first[lo]) * kAdamChunk + 8 * threadIdx.x;
  float lr = a.lr, step = a.step, rs = a.rs;
  uint32_t now = a.t_lo;
  if (a.lr_dev) lr = *a.lr_dev;
  if (a.t_dev) {                                   // (one wave forms the bias corrections)
    __shared__ float corr[2];
    const double k = (double)*a.t_dev;
    now = (uint32_t)*a.t_dev;
    if (threadIdx.x < 64) {
      corr[0] = (float)((double)lr / -expm1(k * a.log_b1));
      corr[1] = (float)(1.0 / sqrt(-expm1(k * a.log_b2)));
    }
    __syncthreads();
    step = corr[0];
    rs = corr[1];
  } else if (a.lr_dev) {
    step = lr * a.step;                            // (1 / c1)
  }
  const float shrink = -lr * t.decay;
  const uint32_t key = adam_mix(adam_mix(a.seed ^ (now * 0x9E3779B9u)) + (uint32_t)t.index * 0xA54FF53Bu);
  if (i >= ((n + 127) & ~(int64_t)127)) return;    // (whole blocks of 128: 16 lanes)
  float w[8], g[8], m[8], v[8];
  adam_load<GBF>(t.g, i, n, g);
  if (W == ADAM_F32) adam_load<0>(t.p, i, n, w);
  else if (W == ADAM_BF16) adam_load<1>(t.p, i, n, w);
  else adam_load<0>(t.master, i, n, w);
  if (S8) {
    adam_load_fp8(t.m, i, n, t.ms[i / 128], m);
    adam_load_fp8(t.v, i, n, t.vs[i / 128], v);
  } else {
    adam_load<0>(t.m, i, n, m);
    adam_load<0>(t.v, i, n, v);
  }
  float root[8];
  uint32_t rm[8], rv[8], rw[8], least = ~0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = g[e] * gs;
    if (S8) v[e] *= v[e];
    m[e] = adam_mean(a.b1, m[e], a.a1, x);
    v[e] = adam_mean(a.b2, v[e], a.a2, x * x);
    least = min(least, __float_as_uint(v[e]) - 1);     // (zero is not small)
  }
  if (__ballot(least < 0x0F800000u)) {             // 2^-96
#pragma unroll
    for (int e = 0; e < 8; ++e) root[e] = sqrtf(v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) root[e] = adam_sqrt(v[e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float u = m[e] * __builtin_amdgcn_rcpf(__builtin_fmaf(root[e], rs, a.eps));
    w[e] = __builtin_fmaf(-step, u, __builtin_fmaf(shrink, w[e], w[e]));
    if (S8 || W == ADAM_BF16) {
      const uint32_t h = adam_mix(((uint32_t)i + e) * 0x9E3779B1u + key);
      rm[e] = h & 0xFFFFu;
      rv[e] = h >> 16;
      rw[e] = (h * 0x3C6EF373u) >> 16;
    }
  }
  if (S8) {
    adam_store_fp8<0>(t.m, t.ms, i, n, m, rm);
    adam_store_fp8<1>(t.v, t.vs, i, n, root, rv);
  } else {
    adam_store_f32(static_cast<float*>(t.m), i, n, m);
    adam_store_f32(static_cast<float*>(t.v), i, n, v);
  }
  if (W == ADAM_F32) adam_store_f32(static_cast<float*>(t.p), i, n, w);
  if (W == ADAM_MASTER) adam_store_f32(t.master, i, n, w);
  if (W != ADAM_F32) {
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = W == ADAM_BF16 ? adam_bf16(w[e], rw[e]) : f32_to_bf16_rne(w[e]);
    uint16_t* p = static_cast<uint16_t*>(t.p) + i;
    if (i + 8 <= n) {
      st16(p, v4i{(int)(b[0] | b[1] << 16), (int)(b[2] | b[3] << 16), (int)(b[4] | b[5] << 16), (int)(b[6] | b[7] << 16)});
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i + e < n) p[e] = (uint16_t)b[e];
    }
  }
}

}  // namespace moe
