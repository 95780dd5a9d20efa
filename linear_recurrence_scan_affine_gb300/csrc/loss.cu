// Losses of a policy's logits and their gradients (rlcs_loss.h): the clipped
// policy loss and distillation from a teacher's top logits.
//
// With m the row's largest logit, s = 1 / T and, in base 2,
//   y_i = (x_i - m) s log2 e,   e_i = 2^y_i,   z = sum e_i,
// a row's distribution is p_i = e_i / z with log p_i = y_i ln 2 - log z, and
// both gradients are e_i (A + B y_i) plus terms at a few named elements.
#include "rlcs_loss.h"
#include "seq_common.cuh"

namespace rlcs {
namespace loss {
namespace {

using seq::aligned;
using seq::esize;
using seq::known;
using seq::launched;
using seq::meet;
using seq::outputs_overlap;
using seq::product_fits;
using seq::range;
using seq::Range;
using bf = __nv_bfloat16;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxTop = 1024;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float value(const float *p) { return *p; }
__device__ __forceinline__ float value(const bf *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(bf *p, float v) { *p = __float2bfloat16_rn(v); }

// A row's statistics: z and sum e y over its elements, relative to m.
struct Stats {
  float m, z, t;
};
// What m is subtracted as: a row (or part of one) with nothing above -infinity
// has e = 0 everywhere, not exp(NaN).
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ float shifted(float x, float base, float c) { return (x - base) * c; }
// y where it multiplies e: -infinity and what underflows far below 2^-149
// add nothing
__device__ __forceinline__ float bounded(float y) { return fmaxf(y, -200.0f); }

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}

// ---------------------------------------------------------------------------
// The two losses: what a row needs besides its statistics, its scalars, and
// the coefficients of its gradient
// ---------------------------------------------------------------------------
struct Coefficients {
  float a, b;  // dx_i = e_i (a + b y_i)
};

struct PolicyArgs {
  const void *logits;
  int64_t row_stride;
  const int32_t *actions;
  const float *old_logp, *advantages, *ref_logp;
  const uint8_t *mask;
  const float *dloss;
  void *dlogits;
  float *loss, *logp, *entropy, *kl;
  int64_t tokens, V;
  float low, high, kl_coef, entropy_coef;  // the ratio's bounds
};

// exp(d) - d - 1 without cancellation
__device__ __forceinline__ float exp_above_tangent(float d) {
  if (fabsf(d) < 0.5f) {
    float s = 1.0f / 362880.0f;
    const float f[7] = {1.0f / 40320.0f, 1.0f / 5040.0f, 1.0f / 720.0f, 1.0f / 120.0f,
                        1.0f / 24.0f,    1.0f / 6.0f,    0.5f};
#pragma unroll
    for (int i = 0; i < 7; ++i) s = fmaf(s, d, f[i]);
    return d * d * s;
  }
  return expm1f(d) - d;
}

struct PolicyRow {
  int action;
  float xa;    // its logit
  bool there;  // an action of the set
  float gain;  // what the gradient has at the action beyond e (a + b y)
};
__device__ __forceinline__ void zero_scalars(const PolicyArgs &p, int64_t row) {
  if (p.loss) p.loss[row] = 0.0f;
  if (p.logp) p.logp[row] = 0.0f;
  if (p.entropy) p.entropy[row] = 0.0f;
  if (p.kl) p.kl[row] = 0.0f;
}
// The row's scalars, written by the thread that `writes`, and its gradient.
// l carries a rounding of the size that old_logp and ref_logp have themselves.
__device__ __forceinline__ Coefficients finish(const PolicyArgs &p, int64_t row, PolicyRow &r,
                                               const Stats &s, bool writes) {
  const float logz = logf(s.z);
  const float H = logz - s.t / s.z * kLn2;
  const float l = r.there ? (r.xa - s.m) - logz : NAN;
  const float ratio = expf(l - p.old_logp[row]), A = p.advantages[row];
  const float free = ratio * A, held = fminf(fmaxf(ratio, p.low), p.high) * A;
  // (a NaN ratio goes through fminf and fmaxf: take it from `free`)
  const bool open = !(free > held);
  float loss = -(open ? free : held), g = open ? -free : 0.0f;
  if (p.ref_logp) {
    const float d = p.ref_logp[row] - l, kl = exp_above_tangent(d);
    if (p.kl && writes) p.kl[row] = kl;
    if (p.kl_coef != 0.0f) {
      loss += p.kl_coef * kl;
      g -= p.kl_coef * expm1f(d);
    }
  }
  if (p.entropy_coef != 0.0f) loss -= p.entropy_coef * H;
  if (writes) {
    if (p.loss) p.loss[row] = loss;
    if (p.logp) p.logp[row] = l;
    if (p.entropy) p.entropy[row] = H;
  }
  const float w = p.dloss ? p.dloss[row] : 0.0f, u = w / s.z;
  r.gain = w * g;
  return {u * (p.entropy_coef * (H - logz) - g), u * p.entropy_coef * kLn2};
}

struct DistillArgs {
  const void *logits;
  int64_t row_stride;
  const int32_t *ids;
  const float *top, *teacher_lse;
  const uint8_t *mask;
  const float *dloss;
  void *dlogits;
  float *loss;
  int64_t tokens, V;
  int K;
  float inv_t;
};

// ---------------------------------------------------------------------------
// Rows of any length, a block to a row, read twice
// ---------------------------------------------------------------------------
constexpr int kThreads = 512;

__device__ __forceinline__ float block_sum(float x, float *part) {
  x = warp_sum(x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < kThreads / 32 ? part[threadIdx.x & 31] : 0.0f);
}
__device__ __forceinline__ float block_max(float x, float *part) {
  x = warp_max(x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  return warp_max((threadIdx.x & 31) < kThreads / 32 ? part[threadIdx.x & 31] : -INFINITY);
}

template <class T, bool ENTROPY>
__device__ __forceinline__ Stats row_stats(const T *x, int64_t V, float c, float *part) {
  float m = -INFINITY, z = 0.0f, t = 0.0f;
  for (int64_t i = threadIdx.x; i < V; i += kThreads) {
    const float v = value(x + i);
    if (v > m) {  // rescale what was summed so far
      const float f = ex2(shifted(m, v, c));  // (0 from the start, m = -infinity)
      if (ENTROPY) t = z > 0.0f ? f * (t + z * shifted(m, v, c)) : 0.0f;
      z *= f;
      m = v;
    }
    const float y = shifted(v, base_of(m), c), e = ex2(y);
    z += e;
    if (ENTROPY) t = fmaf(e, bounded(y), t);
  }
  const float top = block_max(m, part), base = base_of(top);
  const float y = shifted(m, base, c), f = ex2(y);
  if (ENTROPY) t = f * (t + z * bounded(y));
  z *= f;
  return {top, block_sum(z, part), ENTROPY ? block_sum(t, part) : 0.0f};
}

template <class T, bool GRAD>
__global__ void __launch_bounds__(kThreads) policy_rows_kernel(const PolicyArgs p) {
  __shared__ float part[32];
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t row = blockIdx.x; row < p.tokens; row += gridDim.x) {
    const T *x = static_cast<const T *>(p.logits) + row * p.row_stride;
    T *dx = GRAD ? static_cast<T *>(p.dlogits) + row * p.V : nullptr;
    if (p.mask && !p.mask[row]) {
      if (threadIdx.x == 0) zero_scalars(p, row);
      if (GRAD)
        for (int64_t i = threadIdx.x; i < p.V; i += kThreads) put(dx + i, 0.0f);
      continue;
    }
    PolicyRow r;
    r.action = p.actions[row];
    r.there = r.action >= 0 && r.action < p.V;
    r.xa = r.there ? value(x + r.action) : 0.0f;
    const Stats s = row_stats<T, true>(x, p.V, kLog2e, part);
    const Coefficients k = finish(p, row, r, s, threadIdx.x == 0);
    if (GRAD)
      for (int64_t i = threadIdx.x; i < p.V; i += kThreads) {
        const float y = shifted(value(x + i), base_of(s.m), kLog2e);
        float d = ex2(y) * fmaf(k.b, bounded(y), k.a);
        if (i == r.action) d += r.gain;
        put(dx + i, d);
      }
  }
}

template <class T, bool GRAD>
__global__ void __launch_bounds__(kThreads) distill_rows_kernel(const DistillArgs p) {
  __shared__ float part[32], q[kMaxTop], logq[kMaxTop], at[kMaxTop];
  __shared__ int id[kMaxTop];
  pdl_wait();
  pdl_launch_dependents();
  const float c = p.inv_t * kLog2e;
  for (int64_t row = blockIdx.x; row < p.tokens; row += gridDim.x) {
    const T *x = static_cast<const T *>(p.logits) + row * p.row_stride;
    T *dx = GRAD ? static_cast<T *>(p.dlogits) + row * p.V : nullptr;
    bool on = !p.mask || p.mask[row];
    float top = -INFINITY;
    __syncthreads();
    if (on)
      for (int j = threadIdx.x; j < p.K; j += kThreads) {
        const int i = p.ids[row * p.K + j];
        const float v = p.top[row * p.K + j];
        const bool there = i >= 0 && i < p.V && !(v == -INFINITY);
        id[j] = there ? i : -1;
        logq[j] = v * p.inv_t;
        at[j] = there ? value(x + i) : 0.0f;
        if (there) top = fmaxf(top, v != v ? INFINITY : logq[j]);
      }
    top = block_max(top, part);
    on = on && top > -INFINITY;
    if (!on) {
      if (threadIdx.x == 0 && p.loss) p.loss[row] = 0.0f;
      if (GRAD)
        for (int64_t i = threadIdx.x; i < p.V; i += kThreads) put(dx + i, 0.0f);
      continue;
    }
    float lse;
    if (p.teacher_lse) {
      lse = p.teacher_lse[row];
    } else {
      float sum = 0.0f;
      for (int j = threadIdx.x; j < p.K; j += kThreads)
        if (id[j] >= 0) sum += expf(logq[j] - top);
      lse = top + logf(block_sum(sum, part));
    }
    const Stats s = row_stats<T, false>(x, p.V, c, part);
    const float logz = logf(s.z);
    float mass = 0.0f, loss = 0.0f;
    for (int j = threadIdx.x; j < p.K; j += kThreads) {
      q[j] = 0.0f;
      if (id[j] < 0) continue;
      const float lq = logq[j] - lse, e = expf(lq);
      q[j] = e;
      mass += e;
      if (e > 0.0f || e != e) loss += e * (lq - ((at[j] - s.m) * p.inv_t - logz));
    }
    mass = block_sum(mass, part);
    loss = block_sum(loss, part);
    if (threadIdx.x == 0 && p.loss) p.loss[row] = loss;
    if (!GRAD) continue;
    const float w = p.dloss[row] * p.inv_t, a = w * mass / s.z, base = base_of(s.m);
    for (int64_t i = threadIdx.x; i < p.V; i += kThreads)
      put(dx + i, ex2(shifted(value(x + i), base, c)) * a);
    __syncthreads();  // then the few elements with a target, again
    for (int j = threadIdx.x; j < p.K; j += kThreads) {
      if (id[j] < 0) continue;
      float target = 0.0f;
      for (int i = 0; i < p.K; ++i)
        if (id[i] == id[j]) target += q[i];
      put(dx + id[j], fmaf(ex2(shifted(at[j], base, c)), a, -w * target));
    }
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
template <class Args>
rlcs_status check_rows(const Args &p, bool grad, rlcs_dtype dtype) {
  if (p.tokens < 0 || p.V < 1 || p.V > INT32_MAX || !known(dtype) ||
      !product_fits(p.tokens, p.V, 1) || (p.tokens > 1 && p.row_stride < p.V) ||
      (p.tokens > 1 && !product_fits(p.tokens, p.row_stride, 1)))
    return RLCS_ERR_INVALID_ARG;
  if (p.tokens == 0) return RLCS_OK;
  const uintptr_t e = (uintptr_t)esize(dtype);
  if (!p.logits || (grad && (!p.dlogits || !p.dloss)) || (!grad && !p.loss))
    return RLCS_ERR_INVALID_ARG;
  if (!aligned(p.logits, e) || !aligned(p.dlogits, e)) return RLCS_ERR_MISALIGNED;
  return RLCS_OK;
}
// The logits as an input for the overlap check: left out where the gradient
// takes their place.
template <class Args>
Range logits_range(const Args &p, rlcs_dtype dtype) {
  if (p.dlogits == p.logits && (p.row_stride == p.V || p.tokens == 1)) return range(nullptr, 0);
  return range(p.logits, ((p.tokens - 1) * p.row_stride + p.V) * esize(dtype));
}

template <class K, class Args>
rlcs_status launch_rows(K kernel, const Args &p, cudaStream_t st) {
  const int64_t blocks = p.tokens < seq::kSms * 4 ? p.tokens : seq::kSms * 4;
  return launched(
      launch_ex(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, st, true, p));
}

rlcs_status run_policy(PolicyArgs p, bool grad, double clip_low, double clip_high, double kl_coef,
                       double entropy_coef, rlcs_dtype dtype, rlcs_stream_t stream) {
  const auto finite = [](double v) { return v >= -1e30 && v <= 1e30; };
  if (!(clip_low >= 0.0 && clip_low <= 1.0 && clip_high >= 0.0 && clip_high <= 1e30) ||
      !finite(kl_coef) || !finite(entropy_coef))
    return RLCS_ERR_INVALID_ARG;
  const rlcs_status st = check_rows(p, grad, dtype);
  if (st != RLCS_OK || p.tokens == 0) return st;
  if (!p.actions || !p.old_logp || !p.advantages || (!p.ref_logp && (kl_coef != 0.0 || p.kl)))
    return RLCS_ERR_INVALID_ARG;
  const int64_t n = p.tokens * 4;
  const Range outs[] = {range(p.dlogits, p.tokens * p.V * esize(dtype)), range(p.loss, n),
                        range(p.logp, n), range(p.entropy, n), range(p.kl, n)};
  const Range x = range(p.logits, ((p.tokens - 1) * p.row_stride + p.V) * esize(dtype));
  const Range ins[] = {logits_range(p, dtype), range(p.actions, n), range(p.old_logp, n),
                       range(p.advantages, n), range(p.ref_logp, n), range(p.mask, p.tokens),
                       range(p.dloss, n)};
  if (outputs_overlap(outs, ins)) return RLCS_ERR_INVALID_ARG;
  for (int i = 1; i < 5; ++i)
    if (meet(outs[i], x)) return RLCS_ERR_INVALID_ARG;
  p.low = (float)(1.0 - clip_low);
  p.high = (float)(1.0 + clip_high);
  p.kl_coef = (float)kl_coef;
  p.entropy_coef = (float)entropy_coef;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == RLCS_F32)
    return grad ? launch_rows(policy_rows_kernel<float, true>, p, s)
                : launch_rows(policy_rows_kernel<float, false>, p, s);
  return grad ? launch_rows(policy_rows_kernel<bf, true>, p, s)
              : launch_rows(policy_rows_kernel<bf, false>, p, s);
}

rlcs_status run_distill(DistillArgs p, int64_t K, bool grad, double temperature, rlcs_dtype dtype,
                        rlcs_stream_t stream) {
  if (K < 1 || K > kMaxTop || !(temperature >= 1e-6 && temperature <= 1e6))
    return RLCS_ERR_INVALID_ARG;
  const rlcs_status st = check_rows(p, grad, dtype);
  if (st != RLCS_OK || p.tokens == 0) return st;
  if (!p.ids || !p.top || !product_fits(p.tokens, K, 4)) return RLCS_ERR_INVALID_ARG;
  const int64_t n = p.tokens * 4;
  const Range outs[] = {range(p.dlogits, p.tokens * p.V * esize(dtype)), range(p.loss, n)};
  const Range x = range(p.logits, ((p.tokens - 1) * p.row_stride + p.V) * esize(dtype));
  const Range ins[] = {logits_range(p, dtype),  range(p.ids, n * K), range(p.top, n * K),
                       range(p.teacher_lse, n), range(p.mask, p.tokens), range(p.dloss, n)};
  if (outputs_overlap(outs, ins) || meet(outs[1], x)) return RLCS_ERR_INVALID_ARG;
  p.K = (int)K;
  p.inv_t = (float)(1.0 / temperature);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == RLCS_F32)
    return grad ? launch_rows(distill_rows_kernel<float, true>, p, s)
                : launch_rows(distill_rows_kernel<float, false>, p, s);
  return grad ? launch_rows(distill_rows_kernel<bf, true>, p, s)
              : launch_rows(distill_rows_kernel<bf, false>, p, s);
}

}  // namespace
}  // namespace loss
}  // namespace rlcs

using namespace rlcs;
using namespace rlcs::loss;

extern "C" {

rlcs_status rlcs_policy_loss(const void *logits, int64_t row_stride, const int32_t *actions,
                             const float *old_logp, const float *advantages,
                             const float *ref_logp, const uint8_t *mask, float *loss, float *logp,
                             float *entropy, float *kl, int64_t tokens, int64_t V,
                             double clip_low, double clip_high, double kl_coef,
                             double entropy_coef, rlcs_dtype dtype, rlcs_stream_t stream) {
  const PolicyArgs p = {logits, row_stride, actions, old_logp, advantages, ref_logp, mask, nullptr,
                        nullptr, loss, logp, entropy, kl, tokens, V, 0, 0, 0, 0};
  return run_policy(p, false, clip_low, clip_high, kl_coef, entropy_coef, dtype, stream);
}

rlcs_status rlcs_policy_loss_backward(
    const float *dloss, const void *logits, int64_t row_stride, const int32_t *actions,
    const float *old_logp, const float *advantages, const float *ref_logp, const uint8_t *mask,
    void *dlogits, float *loss, float *logp, float *entropy, float *kl, int64_t tokens, int64_t V,
    double clip_low, double clip_high, double kl_coef, double entropy_coef, rlcs_dtype dtype,
    rlcs_stream_t stream) {
  const PolicyArgs p = {logits, row_stride, actions, old_logp, advantages, ref_logp, mask, dloss,
                        dlogits, loss, logp, entropy, kl, tokens, V, 0, 0, 0, 0};
  return run_policy(p, true, clip_low, clip_high, kl_coef, entropy_coef, dtype, stream);
}

rlcs_status rlcs_distill_loss(const void *logits, int64_t row_stride, const int32_t *top_ids,
                              const float *top_logits, const float *teacher_lse,
                              const uint8_t *mask, float *loss, int64_t tokens, int64_t V,
                              int64_t K, double temperature, rlcs_dtype dtype,
                              rlcs_stream_t stream) {
  const DistillArgs p = {logits, row_stride, top_ids, top_logits, teacher_lse, mask, nullptr,
                         nullptr, loss, tokens, V, 0, 0};
  return run_distill(p, K, false, temperature, dtype, stream);
}

rlcs_status rlcs_distill_loss_backward(const float *dloss, const void *logits, int64_t row_stride,
                                       const int32_t *top_ids, const float *top_logits,
                                       const float *teacher_lse, const uint8_t *mask,
                                       void *dlogits, float *loss, int64_t tokens, int64_t V,
                                       int64_t K, double temperature, rlcs_dtype dtype,
                                       rlcs_stream_t stream) {
  const DistillArgs p = {logits, row_stride, top_ids, top_logits, teacher_lse, mask, dloss,
                         dlogits, loss, tokens, V, 0, 0};
  return run_distill(p, K, true, temperature, dtype, stream);
}

}  // extern "C"
