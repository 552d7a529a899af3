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
// written once) and by their launches on small ones:
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
// Sequence offsets are device data: each is clamped to [0, T], and a
// sequence that ends before it begins is empty.  With offsets that descend
// the results are unspecified, but every access stays in range.
#pragma once
#include "device_common.h"
#include "permute.h"

namespace moe {

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
  int32_t* done;             // workgroups of k_bal_final that have finished
};

DEV int bal_off(const BalArgs& a, int s) { return a.off ? min(max(a.off[s], 0), a.T) : (s ? a.T : 0); }

// The first sequence that ends behind token t (S if none does).
DEV int bal_seq_of(const BalArgs& a, int t) {
  if (!a.off) return 0;
  int lo = 0, hi = a.S;
  while (lo < hi) {
    const int m = (lo + hi) / 2;
    if (bal_off(a, m + 1) > t) hi = m; else lo = m + 1;
  }
  return lo;
}

// Rows [*r0, *r1) of sequence s over blocks of `bt` tokens (none if empty).
DEV void bal_rows(const BalArgs& a, int s, int bt, int* r0, int* r1) {
  const int t0 = bal_off(a, s), t1 = bal_off(a, s + 1);
  *r0 = t0 / bt + s;
  *r1 = t1 > t0 ? (t1 - 1) / bt + s + 1 : *r0;
}

constexpr int kBalCountThreads = 1024;
__global__ void __launch_bounds__(kBalCountThreads) k_bal_count(BalArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int* hist = reinterpret_cast<int*>(lds);
  __shared__ int s_n;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;
  const int t0 = blockIdx.x * a.cb, t1 = min(a.T, t0 + a.cb);
  for (int s = bal_seq_of(a, t0); s < a.S && bal_off(a, s) < t1; ++s) {
    const int lo = max(t0, bal_off(a, s)), hi = min(t1, bal_off(a, s + 1));
    if (lo >= hi) continue;                                   // (uniform)
    for (int e = threadIdx.x; e < a.E; e += kBalCountThreads) hist[e] = 0;
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    if (!a.mask) {
      count_experts(a.ids, (size_t)lo * a.k, (hi - lo) * a.k, a.E, hist);
    } else {
      for (int t = lo + threadIdx.x; t < hi; t += kBalCountThreads)
        if (a.mask[t]) {
          atomicAdd(&s_n, 1);
          for (int j = 0; j < a.k; ++j) atomicAdd(&hist[min(max(a.ids[(size_t)t * a.k + j], 0), a.E - 1)], 1);
        }
    }
    __syncthreads();
    int32_t* row = a.rowcnt + (size_t)(blockIdx.x + s) * a.E;
    for (int e = threadIdx.x; e < a.E; e += kBalCountThreads) row[e] = hist[e];
    if (threadIdx.x == 0) a.rown[blockIdx.x + s] = a.mask ? s_n : hi - lo;
    __syncthreads();
  }
}

// Tokens of sequence s that count, by one thread.
DEV int bal_tokens_of(const BalArgs& a, int s) {
  int r0, r1, n = 0;
  bal_rows(a, s, a.cb, &r0, &r1);
  for (int r = r0; r < r1; ++r) n += a.rown[r];
  return n;
}

// S' (at least 1) for the whole workgroup; `red`: one int per wave.
DEV int bal_used(const BalArgs& a, int* red) {
  int u = 0;
  for (int s = threadIdx.x; s < a.S; s += blockDim.x) u += bal_tokens_of(a, s) > 0;
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

// One token per L lanes (16 for E <= 256, else 64), NJ chunks of 4
// consecutive experts per lane; four waves.  The next token's logits are
// loaded while the current one is worked on.
typedef float v4fu __attribute__((ext_vector_type(4), aligned(4)));   // rows of E floats: 4-byte aligned
template <int L, int NJ>
__global__ void __launch_bounds__(256) k_bal_tokens(BalArgs a) {
  constexpr int G = 256 / L;                                  // tokens in flight per workgroup
  extern __shared__ __attribute__((aligned(16))) char lds[];
  float* psum = reinterpret_cast<float*>(lds);                // [4][L * NJ * 4]
  int* cnt = reinterpret_cast<int*>(psum + 4 * L * NJ * 4);   // [L * NJ * 4] counts of the sequence
  __shared__ int red[4];
  const int li = threadIdx.x % L, gi = threadIdx.x / L, w = threadIdx.x >> 6, E = a.E;
  const int t0 = blockIdx.x * a.tb, t1 = min(a.T, t0 + a.tb);
  const float ninf = -__builtin_inff();
  const bool grad = a.dlogits != nullptr;
  auto row_max = [&](float v) { v = row_max16(v); return L == 64 ? max_row_groups(v) : v; };
  auto row_sum = [&](float v) { return L == 64 ? wave_sum(v) : row_sum16(v); };
  auto load = [&](int t, float (&v)[NJ][4]) {
    const float* p = a.logits + (size_t)t * E;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = 4 * (li + L * j);
      if (e + 4 <= E) {
        const v4fu q = *reinterpret_cast<const v4fu*>(p + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = q[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = e + i < E ? p[e + i] : ninf;
      }
    }
  };
  auto store = [&](int t, const float (&d)[NJ][4]) {
    float* p = a.dlogits + (size_t)t * E;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = 4 * (li + L * j);
      if (e + 4 <= E) {
        *reinterpret_cast<v4fu*>(p + e) = v4fu{d[j][0], d[j][1], d[j][2], d[j][3]};
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e + i < E) p[e + i] = d[j][i];
      }
    }
  };
  float zero[NJ][4];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) zero[j][i] = 0.f;
  const int used = grad ? bal_used(a, red) : 1;

  int next = t0;                                              // tokens before it are done
  for (int s = bal_seq_of(a, t0); s < a.S && bal_off(a, s) < t1; ++s) {
    const int lo = max(t0, bal_off(a, s)), hi = min(t1, bal_off(a, s + 1));
    if (lo >= hi) continue;
    if (grad)
      for (int t = next + gi; t < lo; t += G) store(t, zero); // tokens of no sequence
    next = hi;
    float kappa = 0.f;
    if (grad) {
      int r0, r1;
      bal_rows(a, s, a.cb, &r0, &r1);
      for (int e = threadIdx.x; e < L * NJ * 4; e += 256) {
        int c = 0;
        if (e < E) {
#pragma unroll 8
          for (int r = r0; r < r1; ++r) c += a.rowcnt[(size_t)r * E + e];
        }
        cnt[e] = c;
      }
      const double n = (double)max(bal_tokens_of(a, s), 1);
      kappa = (float)((double)a.alpha * E / ((double)used * a.k * n * n));
      __syncthreads();
    }
    float ps[NJ][4];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) ps[j][i] = 0.f;
    float nx[NJ][4];
    bool nv = false;                                          // the loaded token counts
    if (lo + gi < hi) {
      nv = !a.mask || a.mask[lo + gi];
      if (nv) load(lo + gi, nx);
    }
    for (int t = lo + gi; t < hi; t += G) {
      float v[NJ][4];
      const bool valid = nv;
      if (valid) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[j][i] = nx[j][i];
      }
      if (t + G < hi) {
        nv = !a.mask || a.mask[t + G];
        if (nv) load(t + G, nx);
      }
      if (!valid) {
        if (grad) store(t, zero);
        continue;                                             // (lanes of one token stay together)
      }
      float m = ninf;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaxf(m, v[j][i]);
      m = row_max(m);
      // the count of the likeliest expert (of equal ones the most frequent)
      int top = 0;
      if (grad) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (v[j][i] == m) top = max(top, cnt[4 * (li + L * j) + i]);
        top = bal_max<L>(top);
      }
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[j][i] = v[j][i] == ninf ? 0.f : expf(v[j][i] - m);
          sum += v[j][i];
        }
      sum = row_sum(sum);
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;        // every logit -inf: no probability anywhere
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[j][i] *= inv;
          ps[j][i] += v[j][i];
          if (grad) dot = __builtin_fmaf(v[j][i], (float)(cnt[4 * (li + L * j) + i] - top), dot);
        }
      if (grad) {
        dot = row_sum(dot);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[j][i] = kappa * v[j][i] * ((float)(cnt[4 * (li + L * j) + i] - top) - dot);
        store(t, v);
      }
    }
    // the row of sums: the groups of a wave, then the waves
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x = ps[j][i];
        if (L == 16) {
          const uint32_t u = __float_as_uint(x);
          const auto r16 = __builtin_amdgcn_permlane16_swap(u, u, false, false);
          x = __uint_as_float(r16[0]) + __uint_as_float(r16[1]);
          const uint32_t h = __float_as_uint(x);
          const auto r32 = __builtin_amdgcn_permlane32_swap(h, h, false, false);
          x = __uint_as_float(r32[0]) + __uint_as_float(r32[1]);
        }
        if ((threadIdx.x & 63) < L) psum[w * L * NJ * 4 + 4 * (li + L * j) + i] = x;
      }
    __syncthreads();
    float* row = a.rowp + (size_t)(blockIdx.x + s) * E;
    for (int e = threadIdx.x; e < E; e += 256)
      row[e] = ((psum[e] + psum[L * NJ * 4 + e]) + psum[2 * L * NJ * 4 + e]) + psum[3 * L * NJ * 4 + e];
    __syncthreads();
  }
  if (grad)
    for (int t = next + gi; t < t1; t += G) store(t, zero);   // tokens behind the last sequence
}

// Workgroup (x, s): experts [64x, 64x + 64) of sequence s (s, s + gridDim.y,
// ...): 16 groups of 16 lanes, each summing every 16th row, 4 experts per
// lane.  The last workgroup to finish adds the loss.
__global__ void __launch_bounds__(256) k_bal_final(BalArgs a) {
  __shared__ float redp[16][64];
  __shared__ int redc[16][64];
  __shared__ int red[4], s_last;
  __shared__ double s_part[64];
  const int cl = threadIdx.x & 15, grp = threadIdx.x >> 4, E = a.E;
  const int used = bal_used(a, red);
  double part = 0;
  for (int s = blockIdx.y; s < a.S; s += gridDim.y) {
    int c0, c1, p0, p1;
    bal_rows(a, s, a.cb, &c0, &c1);
    bal_rows(a, s, a.tb, &p0, &p1);
    float ps[4] = {0.f, 0.f, 0.f, 0.f};
    int cs[4] = {0, 0, 0, 0};
    const int e0 = blockIdx.x * 64 + 4 * cl;
    if (e0 + 4 <= E) {
#pragma unroll 8
      for (int r = p0 + grp; r < p1; r += 16) {
        const v4fu q = *reinterpret_cast<const v4fu*>(a.rowp + (size_t)r * E + e0);
#pragma unroll
        for (int i = 0; i < 4; ++i) ps[i] += q[i];
      }
    } else {
      for (int r = p0 + grp; r < p1; r += 16)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e0 + i < E) ps[i] += a.rowp[(size_t)r * E + e0 + i];
    }
    for (int r = c0 + grp; r < c1; r += 16)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + i < E) cs[i] += a.rowcnt[(size_t)r * E + e0 + i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      redp[grp][4 * cl + i] = ps[i];
      redc[grp][4 * cl + i] = cs[i];
    }
    const int n = bal_tokens_of(a, s);
    __syncthreads();
    const int e = blockIdx.x * 64 + (int)threadIdx.x;
    if (threadIdx.x < 64 && e < E) {
      float p = redp[0][threadIdx.x];
      int c = redc[0][threadIdx.x];
#pragma unroll
      for (int i = 1; i < 16; ++i) {
        p += redp[i][threadIdx.x];
        c += redc[i][threadIdx.x];
      }
      const float pm = n > 0 ? p / (float)n : 0.f;
      a.counts[(size_t)s * E + e] = c;
      a.probs[(size_t)s * E + e] = pm;
      if (n > 0) part += (double)c * E / ((double)a.k * n) * pm;
    }
    __syncthreads();
  }
  if (threadIdx.x < 64) s_part[threadIdx.x] = part;
  __syncthreads();
  const int wg = blockIdx.y * gridDim.x + blockIdx.x, nwg = gridDim.x * gridDim.y;
  if (threadIdx.x == 0) {
    double v = 0;
    for (int i = 0; i < 64; ++i) v += s_part[i];
    st_coh(a.lpart + wg, v);
    wait_stores();                                            // the partial is in memory before it is counted
    s_last = __hip_atomic_fetch_add(a.done, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == nwg - 1;
  }
  __syncthreads();
  if (!s_last) return;
  double v = 0;
  for (int i = threadIdx.x; i < nwg; i += 256) v += ld_coh(a.lpart + i);
  __shared__ double s_sum[256];
  s_sum[threadIdx.x] = v;
  __syncthreads();
  for (int h = 128; h > 0; h >>= 1) {
    if ((int)threadIdx.x < h) s_sum[threadIdx.x] += s_sum[threadIdx.x + h];
    __syncthreads();
  }
  if (threadIdx.x == 0) *a.loss = (float)((double)a.alpha / used * s_sum[0]);
}

}  // namespace moe
