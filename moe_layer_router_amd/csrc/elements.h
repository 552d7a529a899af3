// Eight consecutive BF16 or fp32 elements of a tensor at a time, as fp32 values.
#pragma once
#include "device_common.h"

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

}  // namespace moe
