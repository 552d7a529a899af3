// Layer norm over the H channels of each token, in front of the router, and
// its backward pass.
//
//   mean = sum_h x / H, var = sum_h (x - mean)^2 / H, rstd = 1 / sqrt(var + eps)
//   z = (x - mean) rstd,  y = z gamma + beta
// With g = dy gamma (dy the gradient of y):
//   dx = rstd (g - sum_h g / H - z sum_h (g z) / H)
//   dgamma = sum_t dy z,  dbeta = sum_t dy
//
// Both are bound by HBM: forward 2 (or 4) bytes read and 2, 4 or 1 + 1/32
// written per element, backward x and dy read and 4 bytes written.  A row
// lives in the registers of TPR threads (8 consecutive channels per thread
// and chunk, R chunks), so it is read once and the variance is the sum of
// squared differences from the row's own mean, not a difference of sums.
// Every sum is fp32.
//
// Measured (T = 8192, H = 7168): forward BF16 -> BF16 41 to 45 us (5.2 to 5.7 TB/s; a
// large copy reaches 5.2), to FP8 52 to 55 us (3.2 TB/s; with as many elements at H =
// 4096 39 to 42: its vector instructions, 1.7 times those of BF16 output, take 0.7 of
// the SIMDs' time by the counters), backward of BF16 x and fp32 dy with the weight
// gradients 112 + 5 us (5.2 TB/s).  One token: 3.6 us, a launch.
#pragma once
#include "device_common.h"
#include "quant.h"

namespace moe {

enum { LN_BF16 = 0, LN_F32 = 1, LN_FP8 = 2 };

// The bytes of 8 consecutive elements.
template <int DT>
struct LnRaw {
  v4i q[DT == LN_F32 ? 2 : 1];
};
template <int DT>
DEV LnRaw<DT> ln_load(const void* p, size_t e0) {
  LnRaw<DT> r;
  if (DT == LN_F32) {
    r.q[0] = ld16(static_cast<const float*>(p) + e0);
    r.q[DT == LN_F32 ? 1 : 0] = ld16(static_cast<const float*>(p) + e0 + 4);
  } else {
    r.q[0] = ld16(static_cast<const uint16_t*>(p) + e0);
  }
  return r;
}
template <int DT>
DEV void ln_unpack(const LnRaw<DT>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (DT == LN_F32) {
      v[i] = __int_as_float(r.q[0][i]);
      v[4 + i] = __int_as_float(r.q[DT == LN_F32 ? 1 : 0][i]);
    } else {
      v[2 * i] = bf16_to_f32((uint32_t)r.q[0][i] & 0xFFFFu);
      v[2 * i + 1] = bf16_to_f32((uint32_t)r.q[0][i] >> 16);
    }
  }
}
DEV void ln_load_f32(const float* p, size_t e0, float (&v)[8]) { ln_unpack<LN_F32>(ln_load<LN_F32>(p, e0), v); }
DEV void ln_store_f32(float* p, size_t e0, const float (&v)[8]) {
  *reinterpret_cast<v4f*>(p + e0) = v4f{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<v4f*>(p + e0 + 4) = v4f{v[4], v[5], v[6], v[7]};
}

// Sums of N values per thread over the TPR threads of a row.  `red` holds
// two slots of [N][TPR / 64] floats; the slots alternate (`slot`, flipped
// here), so that one barrier per sum is enough: a wave writes a slot again
// only behind the barrier of the sum in between, which every wave passes
// after it has read the slot.
template <int TPR, int N>
DEV void ln_row_sum(float (&v)[N], float* red, int& slot) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
  if (TPR == 64) return;
  constexpr int NW = TPR / 64;
  float* s = red + slot * (N * NW);
  slot ^= 1;
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) s[n * NW + w] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float t = s[n * NW];
#pragma unroll
    for (int i = 1; i < NW; ++i) t += s[n * NW + i];
    v[n] = t;
  }
}

constexpr int ln_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

struct LnArgs {
  const void* x;
  const float* gamma;
  const float* beta;         // or NULL
  void* y;
  float* y_scales;           // FP8 output: [T][H/128]
  float* mean;               // or NULL
  float* rstd;               // or NULL
  long T;
  int H;
  float eps;
  int pow2;
};

// A workgroup holds 1 row (TPR >= 256) or 4 (TPR = 64: one per wave) at a
// time and goes through rows in steps of the grid, with gamma and beta in
// registers (reading them for every row would move more through the L2 than
// the row itself) and the next row's loads in flight.
template <int IN, int OUT, int TPR, int R>
__global__ void __launch_bounds__(ln_threads(TPR)) k_layer_norm(LnArgs a) {
  constexpr int RPW = ln_threads(TPR) / TPR;
  __shared__ float red[2 * (TPR / 64)];
  int slot = 0;
  const int rt = threadIdx.x % TPR, H = a.H, nch = H / 8;
  const long step = (long)gridDim.x * RPW;
  long t = (long)blockIdx.x * RPW + threadIdx.x / TPR;
  float ga[R][8], be[R][8];
  float bad[R];              // FP8: NaN where gamma or beta of the block is not finite, else 0
  LnRaw<IN> raw[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = rt + r * TPR;
    if (c < nch && t < a.T) raw[r] = ln_load<IN>(a.x, (size_t)t * H + 8 * c);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = rt + r * TPR;
    if (c < nch) {
      ln_load_f32(a.gamma, 8 * c, ga[r]);
      if (a.beta) ln_load_f32(a.beta, 8 * c, be[r]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (c >= nch) ga[r][i] = 0.f;
      if (c >= nch || !a.beta) be[r][i] = 0.f;
    }
    bad[r] = 0.f;
    if (OUT == LN_FP8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) bad[r] += ga[r][i] * 0.f + be[r][i] * 0.f;
      bad[r] = row_sum16(bad[r]);
    }
  }
  const float inv_h = 1.0f / (float)H;
  // (rows of one wave sum without a barrier, and a row of the whole workgroup
  // is the same for all its threads: every barrier is met by all of them)
  for (; t < a.T; t += step) {
    float v[R][8];
    float s[1] = {0.f};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (rt + r * TPR < nch) {
        ln_unpack<IN>(raw[r], v[r]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[r][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += v[r][i];
    }
    if (t + step < a.T) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int c = rt + r * TPR;
        if (c < nch) raw[r] = ln_load<IN>(a.x, (size_t)(t + step) * H + 8 * c);
      }
    }
    ln_row_sum<TPR, 1>(s, red, slot);
    const float mean = s[0] * inv_h;
    s[0] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (rt + r * TPR < nch) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[r][i] -= mean;
          s[0] = __builtin_fmaf(v[r][i], v[r][i], s[0]);
        }
      }
    ln_row_sum<TPR, 1>(s, red, slot);
    const float rstd = 1.0f / sqrtf(s[0] * inv_h + a.eps);
    if (rt == 0 && a.mean) {
      a.mean[t] = mean;
      a.rstd[t] = rstd;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = rt + r * TPR;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = __builtin_fmaf(v[r][i] * rstd, ga[r][i], be[r][i]);
      const size_t e0 = (size_t)t * H + 8 * c;
      if (OUT == LN_FP8) {
        // the 16 lanes of a DPP row hold one 128-channel block (quant.h)
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(o[i]));
        mx = row_max16(mx);
        float sc, inv;
        block_scale(mx, a.pow2 != 0, &sc, &inv);
        // (the maximum and E4M3's clamp drop NaN: it goes into the scale; rstd is
        // NaN where the row holds NaN or infinity, infinite where 0 / 0 follows)
        sc += bad[r] + (rstd - rstd);
        if (c < nch) {
          *reinterpret_cast<v2u*>(static_cast<uint8_t*>(a.y) + e0) =
              v2u{f32x4_to_e4m3x4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv),
                  f32x4_to_e4m3x4(o[4] * inv, o[5] * inv, o[6] * inv, o[7] * inv)};
          if ((rt & 15) == 0) a.y_scales[e0 / 128] = sc;
        }
      } else if (c < nch) {
        if (OUT == LN_F32) {
          ln_store_f32(static_cast<float*>(a.y), e0, o);
        } else {
          st16(static_cast<uint16_t*>(a.y) + e0,
               v4i{(int)bf16x2_rne(o[0], o[1]), (int)bf16x2_rne(o[2], o[3]), (int)bf16x2_rne(o[4], o[5]),
                   (int)bf16x2_rne(o[6], o[7])});
        }
      }
    }
  }
}

struct LnBwdArgs {
  const void* x;
  const float* gamma;
  const float* mean;
  const float* rstd;
  const void* dy;
  float* dx;
  float* part;               // [workgroups][2][H] partial dgamma, dbeta, or NULL
  long T;
  int H;
};

// dx of a row as the forward kernel holds it, and this workgroup's share of
// dgamma and dbeta (its rows, in ascending order, summed in registers; the
// rows of a workgroup of four waves joined in wave order) as one row of
// `part`, which k_ln_weight_grad sums.  dx may be dy: a row is read whole
// before it is written.
template <int XD, int DYD, int TPR, int R>
__global__ void __launch_bounds__(ln_threads(TPR)) k_layer_norm_bwd(LnBwdArgs a) {
  constexpr int RPW = ln_threads(TPR) / TPR;
  __shared__ float red[2 * 2 * (TPR / 64)];
  __shared__ float join[RPW == 1 ? 1 : RPW * TPR * R * 8];
  int slot = 0;
  const int rt = threadIdx.x % TPR, row = threadIdx.x / TPR, H = a.H, nch = H / 8;
  const long step = (long)gridDim.x * RPW;
  long t = (long)blockIdx.x * RPW + row;
  float ga[R][8], dg[R][8], db[R][8];
  LnRaw<XD> rx[R];
  LnRaw<DYD> ry[R];
  float mean = 0.f, rstd = 0.f;
  auto load = [&](long tt) {
    mean = a.mean[tt];
    rstd = a.rstd[tt];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = rt + r * TPR;
      if (c < nch) {
        rx[r] = ln_load<XD>(a.x, (size_t)tt * H + 8 * c);
        ry[r] = ln_load<DYD>(a.dy, (size_t)tt * H + 8 * c);
      }
    }
  };
  if (t < a.T) load(t);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = rt + r * TPR;
    if (c < nch) ln_load_f32(a.gamma, 8 * c, ga[r]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (c >= nch) ga[r][i] = 0.f;
      dg[r][i] = db[r][i] = 0.f;
    }
  }
  const float inv_h = 1.0f / (float)H;
  for (; t < a.T; t += step) {
    float z[R][8], g[R][8], s[2] = {0.f, 0.f};
    const float rs = rstd;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float dy[8];
      if (rt + r * TPR < nch) {
        ln_unpack<XD>(rx[r], z[r]);
        ln_unpack<DYD>(ry[r], dy);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[r][i] = mean, dy[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z[r][i] = (z[r][i] - mean) * rs;
        g[r][i] = dy[i] * ga[r][i];
        dg[r][i] = __builtin_fmaf(dy[i], z[r][i], dg[r][i]);
        db[r][i] += dy[i];
        s[0] += g[r][i];
        s[1] = __builtin_fmaf(g[r][i], z[r][i], s[1]);
      }
    }
    if (t + step < a.T) load(t + step);
    ln_row_sum<TPR, 2>(s, red, slot);
    const float m1 = s[0] * inv_h, m2 = s[1] * inv_h;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = rt + r * TPR;
      if (c < nch) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = rs * (g[r][i] - m1 - z[r][i] * m2);
        ln_store_f32(a.dx, (size_t)t * H + 8 * c, o);
      }
    }
  }
  if (!a.part) return;
  float* dst = a.part + (size_t)blockIdx.x * 2 * H;
  if (RPW == 1) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = rt + r * TPR;
      if (c < nch) {
        ln_store_f32(dst, 8 * c, dg[r]);
        ln_store_f32(dst + H, 8 * c, db[r]);
      }
    }
    return;
  }
  for (int q = 0; q < 2; ++q) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i) join[(row * R + r) * TPR * 8 + 8 * rt + i] = q ? db[r][i] : dg[r][i];
    __syncthreads();
    for (int i = threadIdx.x; i < H; i += ln_threads(TPR)) {
      float v = join[i];                                     // element i = 8 (TPR r + rt) + ...: chunk order
#pragma unroll
      for (int w = 1; w < RPW; ++w) v += join[w * R * TPR * 8 + i];
      dst[q * H + i] = v;
    }
    __syncthreads();
  }
}

// dgamma (blockIdx.y = 0) or dbeta (1) = the sum of the n partial rows, for
// 64 columns: 16 groups of threads each sum every 16th row, then the groups
// are joined in order.
constexpr int kLnSumCols = 64;
__global__ void __launch_bounds__(256) k_ln_weight_grad(const float* part, int n, int H, float* dgamma, float* dbeta) {
  __shared__ v4f red[16][16];
  float* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  const int cl = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int c = blockIdx.x * kLnSumCols + 4 * cl;               // (H is a multiple of 64)
  v4f s = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int r = grp; r < n; r += 16) s += *reinterpret_cast<const v4f*>(part + ((size_t)r * 2 + blockIdx.y) * H + c);
  red[grp][cl] = s;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += red[i][cl];
    *reinterpret_cast<v4f*>(out + c) = s;
  }
}

}  // namespace moe
