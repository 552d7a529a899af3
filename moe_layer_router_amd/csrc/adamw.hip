// The AdamW step over many tensors (adamw.h), as a C entry point.
#include "host.h"
#include "adamw.h"

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

using namespace moe;

namespace {

constexpr int64_t kAdamChunks = (1 << 24) - 1;     // of a launch (a grid has less than 2^32 threads)

struct Span {
  uintptr_t at, end;
  bool written;
};

size_t adam_bytes(int32_t dtype) { return dtype == MOE_DTYPE_F32 ? 4 : dtype == MOE_DTYPE_BF16 ? 2 : 1; }
int64_t adam_blocks(int64_t n) { return (n + 127) / 128; }

moe_status check_tensors(int32_t count, const moe_adamw_tensor* ts, int32_t state_dtype) {
  const bool f8 = state_dtype == MOE_DTYPE_FP8_E4M3;
  const size_t ssz = adam_bytes(state_dtype);
  std::unique_ptr<Span[]> spans(new (std::nothrow) Span[(size_t)count * 7]);
  if (!spans) return fail(MOE_ERR_HIP, "out of host memory");
  size_t ns = 0;
  for (int32_t i = 0; i < count; ++i) {
    const moe_adamw_tensor& t = ts[i];
    if (t.n < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "tensor %d: n must not be negative (got %lld)", i, (long long)t.n);
    if (t.n > (int64_t)1 << 34) return fail(MOE_ERR_UNSUPPORTED, "tensor %d: n > 2^34 is not supported", i);
    if (t.param_dtype != MOE_DTYPE_F32 && t.param_dtype != MOE_DTYPE_BF16)
      return fail(MOE_ERR_UNSUPPORTED, "tensor %d: param_dtype must be MOE_DTYPE_F32 or MOE_DTYPE_BF16 (got %d)", i, t.param_dtype);
    if (t.grad_dtype != MOE_DTYPE_F32 && t.grad_dtype != MOE_DTYPE_BF16)
      return fail(MOE_ERR_UNSUPPORTED, "tensor %d: grad_dtype must be MOE_DTYPE_F32 or MOE_DTYPE_BF16 (got %d)", i, t.grad_dtype);
    if (!std::isfinite(t.weight_decay)) return fail(MOE_ERR_INVALID_ARGUMENT, "tensor %d: weight_decay must be finite", i);
    if (t.reserved != 0) return fail(MOE_ERR_INVALID_ARGUMENT, "tensor %d: reserved must be 0 (got %d)", i, t.reserved);
    if (t.master && t.param_dtype == MOE_DTYPE_F32)
      return fail(MOE_ERR_INVALID_ARGUMENT, "tensor %d: fp32 weights have no master weights", i);
    if (!f8 && (t.m_scales || t.v_scales))
      return fail(MOE_ERR_INVALID_ARGUMENT, "tensor %d: fp32 states have no scales", i);
    const bool some = t.n > 0;
    TRY(check_ptr(t.param, "param", some));
    TRY(check_ptr(t.grad, "grad", some));
    TRY(check_ptr(t.m, "m", some));
    TRY(check_ptr(t.v, "v", some));
    if (some && f8 && (!t.m_scales || !t.v_scales || (uintptr_t)t.m_scales % 4 || (uintptr_t)t.v_scales % 4))
      return fail(MOE_ERR_INVALID_ARGUMENT, "tensor %d: m_scales and v_scales must be there, 4-byte aligned", i);
    TRY(check_ptr(t.master, "master", false));
    if (!some) continue;
    const auto add = [&](const void* p, size_t bytes, bool written) {
      if (p) spans[ns++] = Span{(uintptr_t)p, (uintptr_t)p + bytes, written};
    };
    add(t.param, t.n * adam_bytes(t.param_dtype), true);
    add(t.grad, t.n * adam_bytes(t.grad_dtype), false);
    add(t.m, t.n * ssz, true);
    add(t.v, t.n * ssz, true);
    add(t.m_scales, adam_blocks(t.n) * 4, true);
    add(t.v_scales, adam_blocks(t.n) * 4, true);
    add(t.master, t.n * 4, true);
  }
  std::sort(spans.get(), spans.get() + ns, [](const Span& x, const Span& y) { return x.at < y.at; });
  uintptr_t end = 0, wend = 0;              // ends so far: of any buffer, of what is written
  for (size_t i = 0; i < ns; ++i) {
    if (spans[i].at < (spans[i].written ? end : wend))
      return fail(MOE_ERR_INVALID_ARGUMENT, "a tensor that the step writes overlaps another one");
    end = std::max(end, spans[i].end);
    if (spans[i].written) wend = std::max(wend, spans[i].end);
  }
  return MOE_OK;
}

template <int W, int GBF, int S8>
moe_status launch_adamw(const AdamArgs& a, int64_t chunks, hipStream_t st) {
  hipLaunchKernelGGL((k_adamw<W, GBF, S8>), dim3((unsigned)chunks), dim3(kAdamThreads), 0, st, a);
  HIP_TRY(hipGetLastError());
  return MOE_OK;
}
template <int W, int GBF>
moe_status launch_adamw(const AdamArgs& a, int64_t chunks, bool f8, hipStream_t st) {
  return f8 ? launch_adamw<W, GBF, 1>(a, chunks, st) : launch_adamw<W, GBF, 0>(a, chunks, st);
}
template <int W>
moe_status launch_adamw(const AdamArgs& a, int64_t chunks, bool f8, bool gbf, hipStream_t st) {
  return gbf ? launch_adamw<W, 1>(a, chunks, f8, st) : launch_adamw<W, 0>(a, chunks, f8, st);
}

}  // namespace

extern "C" {

moe_status moe_adamw(int32_t n_tensors, const moe_adamw_tensor* tensors, const moe_adamw_options* o,
                     moe_stream_t stream) {
  if (n_tensors < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "n_tensors must not be negative (got %d)", n_tensors);
  if (n_tensors > (1 << 24)) return fail(MOE_ERR_UNSUPPORTED, "n_tensors > 2^24 is not supported (got %d)", n_tensors);
  if (n_tensors && !tensors) return fail(MOE_ERR_INVALID_ARGUMENT, "tensors is NULL");
  if (!o) return fail(MOE_ERR_INVALID_ARGUMENT, "options is NULL");
  if (!(o->beta1 >= 0 && o->beta1 < 1) || !(o->beta2 >= 0 && o->beta2 < 1))
    return fail(MOE_ERR_INVALID_ARGUMENT, "beta1 and beta2 must be in [0, 1) (got %g, %g)", o->beta1, o->beta2);
  if (!(o->eps >= 0x1p-100 && o->eps < 0x1p100))
    return fail(MOE_ERR_INVALID_ARGUMENT, "eps must be positive (got %g)", o->eps);
  if (!o->lr_dev && !std::isfinite(o->lr)) return fail(MOE_ERR_INVALID_ARGUMENT, "lr must be finite");
  if (!o->step_dev && o->step < 1)
    return fail(MOE_ERR_INVALID_ARGUMENT, "step must be >= 1 (got %lld)", (long long)o->step);
  if (o->state_dtype != MOE_DTYPE_F32 && o->state_dtype != MOE_DTYPE_FP8_E4M3)
    return fail(MOE_ERR_UNSUPPORTED, "state_dtype must be MOE_DTYPE_F32 or MOE_DTYPE_FP8_E4M3 (got %d)", o->state_dtype);
  const auto aligned = [](const void* p, size_t to) { return (uintptr_t)p % to == 0; };
  if (!aligned(o->grad_scale, 4) || !aligned(o->lr_dev, 4) || !aligned(o->step_dev, 8))
    return fail(MOE_ERR_INVALID_ARGUMENT, "a device scalar is not aligned to its size");
  TRY(check_tensors(n_tensors, tensors, o->state_dtype));
  DevInfo di;
  TRY(device_info(&di));
  const bool f8 = o->state_dtype == MOE_DTYPE_FP8_E4M3;
  hipStream_t st = static_cast<hipStream_t>(stream);
  AdamArgs a{};
  a.b1 = (float)o->beta1; a.a1 = (float)(1 - o->beta1);
  a.b2 = (float)o->beta2; a.a2 = (float)(1 - o->beta2);
  a.log_b1 = std::log(o->beta1); a.log_b2 = std::log(o->beta2);
  a.eps = (float)o->eps;
  a.lr = (float)o->lr;
  a.grad_scale = o->grad_scale; a.lr_dev = o->lr_dev; a.t_dev = o->step_dev;
  a.seed = o->seed;
  if (!o->step_dev) {
    const double t = (double)o->step;
    const double c1 = -std::expm1(t * a.log_b1), c2 = -std::expm1(t * a.log_b2);
    a.step = (float)((o->lr_dev ? 1.0 : o->lr) / c1);
    a.rs = (float)(1 / std::sqrt(c2));
    a.t_lo = (uint32_t)o->step;
  }
  // tensors of one kind of weights and gradients go together, as many as one launch takes
  for (int kind = 0; kind < 6; ++kind) {
    const int w = kind >> 1;
    const bool gbf = kind & 1;
    int64_t chunks = 0;
    const auto flush = [&]() -> moe_status {
      if (!a.count) return MOE_OK;
      a.first[a.count] = (uint32_t)chunks;
      if (w == ADAM_F32) TRY(launch_adamw<ADAM_F32>(a, chunks, f8, gbf, st));
      else if (w == ADAM_BF16) TRY(launch_adamw<ADAM_BF16>(a, chunks, f8, gbf, st));
      else TRY(launch_adamw<ADAM_MASTER>(a, chunks, f8, gbf, st));
      a.count = 0;
      chunks = 0;
      return MOE_OK;
    };
    for (int32_t i = 0; i < n_tensors; ++i) {
      const moe_adamw_tensor& t = tensors[i];
      const int tw = t.param_dtype == MOE_DTYPE_F32 ? ADAM_F32 : t.master ? ADAM_MASTER : ADAM_BF16;
      if (!t.n || tw != w || (t.grad_dtype == MOE_DTYPE_BF16) != gbf) continue;
      const int64_t mine = (t.n + kAdamChunk - 1) / kAdamChunk;
      if (a.count == kAdamTensors || chunks + mine > kAdamChunks) TRY(flush());
      a.t[a.count] = AdamTensor{t.param, t.grad, t.m, t.v, t.m_scales, t.v_scales, t.master, t.n, t.weight_decay, i};
      a.first[a.count++] = (uint32_t)chunks;
      chunks += mine;
    }
    TRY(flush());
  }
  return MOE_OK;
}

}  // extern "C"
