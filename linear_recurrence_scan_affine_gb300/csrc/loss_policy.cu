// The clipped policy loss and its gradient (rlcs_loss.h).
#include "loss_rows.cuh"

namespace rlcs {
namespace loss {
namespace {

// The highest code that a call has recorded on this device.
__device__ uint32_t device_status;

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

// What a token has besides its logits.
struct Token {
  int action;
  float old, adv, ref, w, xa;
  bool there;  // an action of the set
};
__device__ __forceinline__ Token token_of(const PolicyArgs &p, int64_t row) {
  Token a;
  a.action = p.actions[row];
  a.old = p.old_logp[row];
  a.adv = p.advantages[row];
  a.ref = p.ref_logp ? p.ref_logp[row] : 0.0f;
  a.w = p.dloss ? p.dloss[row] : 0.0f;
  a.there = a.action >= 0 && a.action < p.V;
  a.xa = 0.0f;
  return a;
}
template <class T>
__device__ __forceinline__ float logit_of(const PolicyArgs &p, int64_t row, const Token &a) {
  return a.there ? value(static_cast<const T *>(p.logits) + row * p.row_stride + a.action) : 0.0f;
}
__device__ __forceinline__ void zero_scalars(const PolicyArgs &p, int64_t row) {
  if (p.loss) p.loss[row] = 0.0f;
  if (p.logp) p.logp[row] = 0.0f;
  if (p.entropy) p.entropy[row] = 0.0f;
  if (p.kl) p.kl[row] = 0.0f;
}
// log z = k ln 2 + log f with f near 1.
struct LogZ {
  float k, f;
  __device__ __forceinline__ float whole() const { return fmaf(k, kLn2, f); }
};
__device__ __forceinline__ LogZ log_of(float z) {
  if (!(z >= 1e-30f && z < 1e30f)) return {0.0f, logf(z)};  // (a NaN, or no finite logit)
  const int bits = __float_as_int(z), k = (bits - 0x3f400000) >> 23;
  return {(float)k, logf(__int_as_float(bits - (k << 23)))};  // of 0.75 to 1.5
}
// log p of an element in two parts, so that its difference from another log
// probability keeps its digits: off by what z is, about 1e-7, not by roundings
// of l's own size. y is formed with its rounding's remainder; c stands for
// log2 e, off by kOff of it, which moves log z by the mean of y. A block's other
// warps wait for this: with a division and a logarithm more of its own it took 8
// us of 300 at 16384 x 32768 bf16.
struct LogProb {
  float high, low;
  __device__ __forceinline__ float above(float v) const { return (v - high) - low; }  // v - l
};
__device__ __forceinline__ LogProb log_prob(float x, const LogZ &z, float mean, float top) {
  constexpr double kExact = 0.693147180559945309417232, kLog2 = 1.442695040888963407359925;
  constexpr float kLow = (float)(kExact - (double)kLn2);
  constexpr float kOff = (float)(kLog2 / (double)kLog2e - 1.0);
  const Base base = base_of(top, kLog2e);
  if (__builtin_expect(base.c != kLog2e, false)) return {x - top, -z.whole()};
  // (each operation rounded by itself: none may be fused with the next)
  const float xc = __fmul_rn(x, base.c);
  const float xc_rest = fabsf(xc) < 1e30f ? fmaf(x, base.c, -xc) : 0.0f;
  const float d = __fsub_rn(xc, base.m), back = __fsub_rn(d, xc), y = __fadd_rn(d, xc_rest);
  const float y_rest = __fadd_rn(
      __fadd_rn(__fsub_rn(xc, __fsub_rn(d, back)), __fsub_rn(-base.m, back)),
      __fsub_rn(xc_rest, __fsub_rn(y, d)));
  const float a = __fsub_rn(y, z.k), a_back = __fsub_rn(a, y);
  const float a_rest =
      __fadd_rn(__fsub_rn(y, __fsub_rn(a, a_back)), __fsub_rn(-z.k, a_back));
  const float high = __fmul_rn(a, kLn2);
  float low = fmaf(a, kLow, fmaf(a, kLn2, -high));
  low = fmaf(a_rest + y_rest, kLn2, low);
  low = fmaf(kOff * kLn2, y - mean, low);
  return {high, (fabsf(y) < 1e30f ? low : 0.0f) - z.f};
}
// The row's scalars, written by the thread that `writes`, and its gradient:
// e (a + b y) and `gain` more at the action.
__device__ __forceinline__ Coefficients finish(const PolicyArgs &p, int64_t row, const Token &a,
                                               const Stats &s, bool writes, float &gain) {
  const LogZ z = log_of(s.z);
  const float logz = z.whole(), inv = 1.0f / s.z, mean = s.t * inv;
  float H = fmaf(-mean, kLn2, logz);
  if (H < 0.0f) H = 0.0f;  // (a certain action, by a rounding)
  LogProb l = {NAN, 0.0f};
  if (a.there) l = log_prob(a.xa, z, mean, s.top);
  if (l.high + l.low > 0.0f) l = {0.0f, 0.0f};
  const float ratio = expf(-l.above(a.old));
  const float free = ratio * a.adv, held = fminf(fmaxf(ratio, p.low), p.high) * a.adv;
  // (a NaN ratio goes through fminf and fmaxf: take it from `free`)
  const bool open = !(free > held);
  float loss = -(open ? free : held), g = open ? -free : 0.0f;
  if (p.ref_logp) {
    const float d = l.above(a.ref), kl = exp_above_tangent(d);
    if (p.kl && writes) p.kl[row] = kl;
    if (p.kl_coef != 0.0f) {
      loss += p.kl_coef * kl;
      g -= p.kl_coef * expm1f(d);
    }
  }
  if (p.entropy_coef != 0.0f) loss -= p.entropy_coef * H;
  if (writes) {
    if (p.loss) p.loss[row] = loss;
    if (p.logp) p.logp[row] = l.high + l.low;
    if (p.entropy) p.entropy[row] = H;
  }
  const float u = a.w * inv;
  gain = a.w * g;
  return {u * (p.entropy_coef * (H - logz) - g), u * p.entropy_coef * kLn2};
}

template <class T, bool GRAD, int TEAM, int NV>
__global__ void __launch_bounds__(kTeamBlock, team_blocks(NV))
    policy_team_kernel(const PolicyArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kTeams = kTeamBlock / TEAM;
  const int lane = threadIdx.x % TEAM;
  const int64_t step = (int64_t)gridDim.x * kTeams;
  int64_t row = (int64_t)blockIdx.x * kTeams + threadIdx.x / TEAM;
  // Lanes of one warp may belong to several teams: all go on while one has a
  // row, so that their shuffles meet.
  const auto any = [&](bool on) { return TEAM < 32 ? __any_sync(kFull, on) : on; };
  const auto live = [&](int64_t i) { return i < p.tokens && (!p.mask || p.mask[i]); };
  const auto see = [&](int64_t i) { return row_of<T>(p, i < p.tokens ? i : 0, lane, 0, 1); };
  bool on = live(row);
  Row<T> r = see(row);
  uint4 q[NV];
  load_row<T, TEAM, NV>(q, r, on);
  while (any(row < p.tokens)) {
    const int64_t next = row + step;
    const bool more = live(next);
    const Row<T> rn = see(next);
    Token a = {};
    Coefficients k = {0.0f, 0.0f};
    Base base = {0.0f, 0.0f};
    float gain = 0.0f;
    if (on) {
      a = token_of(p, row);
      a.xa = logit_of<T>(p, row, a);
      trim_row<T, TEAM, NV>(q, p, row, r);
    }
    const Stats s = lanes_stats<T, TEAM, NV, true>(q, kLog2e, NV);
    if (on) {
      k = finish(p, row, a, s, lane == 0, gain);
      base = base_of(s.top, kLog2e);
    }
    if (row < p.tokens) {
      T *dx = GRAD ? static_cast<T *>(p.dlogits) + row * p.V : nullptr;
      const int offset = a.there ? (a.action + r.skip) / kWord<T> - r.w0 : -1;
      const int element = (a.action + r.skip) % kWord<T>;
      const auto fix = [&](float2(&d)[kWord<T> / 2], int n) {
        if (n != offset) return;
#pragma unroll
        for (int i = 0; i < kWord<T>; ++i)
          if (i == element) (i % 2 ? d[i / 2].y : d[i / 2].x) += gain;
      };
      if (on) {
        use_row<T, GRAD, TEAM, NV, true, true>(q, r, base, k, rn, more, dx, p.V, fix);
      } else {
        if (lane == 0) zero_scalars(p, row);
        use_row<T, GRAD, TEAM, NV, false, false>(q, r, base, k, rn, more, dx, p.V, fix);
      }
    }
    row = next;
    r = rn;
    on = more;
  }
}

template <class T, bool GRAD>
__global__ void __launch_bounds__(kFewBlock) policy_few_kernel(const PolicyArgs p) {
  extern __shared__ float x[];
  __shared__ uint8_t live[kFewBlock];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row0 = (int64_t)blockIdx.x * kFewBlock, row = row0 + threadIdx.x;
  const int rows = p.tokens - row0 < kFewBlock ? (int)(p.tokens - row0) : kFewBlock;
  const int V = (int)p.V, pitch = V | 1;
  const bool held = row < p.tokens, on = held && (!p.mask || p.mask[row]);
  live[threadIdx.x] = on;
  Token a = {};
  if (on) a = token_of(p, row);
  if (p.mask) __syncthreads();
  few_copy<T, true>(p, static_cast<T *>(nullptr), x, rows, row0, pitch,
                    [&](int i) { return !p.mask || live[i]; });
  __syncthreads();
  float *mine = x + threadIdx.x * pitch;
  if (on) {
    if (a.there) a.xa = mine[a.action];
    const Stats s = few_stats<true>(mine, V, kLog2e);
    float gain;
    const Coefficients k = finish(p, row, a, s, true, gain);
    if (GRAD) {
      const Base base = base_of(s.top, kLog2e);
      for (int i = 0; i < V; ++i) {
        const float y = base.y(mine[i]);
        mine[i] = ex2(y) * fmaf(k.b, bounded(y), k.a);
      }
      if (a.there) mine[a.action] += gain;
    }
  } else if (held) {
    zero_scalars(p, row);
    if (GRAD)
      for (int i = 0; i < V; ++i) mine[i] = 0.0f;
  }
  if (!GRAD) return;
  __syncthreads();
  few_copy<T, false>(p, static_cast<T *>(p.dlogits), x, rows, row0, pitch,
                     [](int) { return true; });
}

template <class T>
struct PolicyLeader {
  static constexpr bool kTeacher = false;
  const PolicyArgs &p;
  Token a, soon;
  __device__ __forceinline__ void ahead(int64_t row, bool on) {
    if (on) soon = token_of(p, row);
  }
  __device__ __forceinline__ void before(int64_t row, bool on) {
    if (!on) return;
    a = soon;
    a.xa = logit_of<T>(p, row, a);
  }
  // (a number that is sent has been read)
  __device__ __forceinline__ float held() const { return a.xa; }
  __device__ __forceinline__ void plan(int64_t row, const Stats &s, bool on, int rank,
                                       LongSmem &sm) {
    const int lane = threadIdx.x & 31;
    if (!on) {
      if (rank == 0 && lane == 0) zero_scalars(p, row);
      return;
    }
    float gain;
    const Coefficients k = finish(p, row, a, s, rank == 0 && lane == 0, gain);
    if (lane != 0) return;
    const uintptr_t x =
        reinterpret_cast<uintptr_t>(static_cast<const T *>(p.logits) + row * p.row_stride);
    const int place = a.action + (int)(x % 16) / (int)sizeof(T);
    sm.k = k;
    sm.gain = gain;
    sm.word = a.there ? place / kWord<T> : -1;
    sm.element = place % kWord<T>;
    sm.on = 1;
  }
  __device__ __forceinline__ void teach(int64_t, bool, int, int, LongSmem &) {}
};

template <class T, bool GRAD, int NV>
__global__ void __launch_bounds__(kLongBlock, long_blocks(NV))
    policy_long_kernel(const PolicyArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  PolicyLeader<T> leader = {p, {}, {}};
  long_rows<T, GRAD, NV, true>(p, kLog2e, &device_status, leader);
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
    Token a = token_of(p, row);
    a.xa = logit_of<T>(p, row, a);
    const Stats s = row_stats<T, true>(x, p.V, kLog2e, part);
    float gain;
    const Coefficients k = finish(p, row, a, s, threadIdx.x == 0, gain);
    const Base base = base_of(s.top, kLog2e);
    if (GRAD)
      for (int64_t i = threadIdx.x; i < p.V; i += kThreads) {
        const float y = base.y(value(x + i));
        float d = ex2(y) * fmaf(k.b, bounded(y), k.a);
        if (i == a.action) d += gain;
        put(dx + i, d);
      }
  }
}

template <class T, bool GRAD>
struct Policy {
  static rlcs_status few(const PolicyArgs &p, cudaStream_t st) {
    return launch_few<policy_few_kernel<T, GRAD>>(p, st);
  }
  template <int TEAM, int NV>
  static rlcs_status team(const PolicyArgs &p, size_t, cudaStream_t st) {
    return launch_team<policy_team_kernel<T, GRAD, TEAM, NV>, TEAM>(p, team_blocks(NV), 0, st);
  }
  template <int NV>
  static rlcs_status block(const PolicyArgs &p, int ranks, size_t, cudaStream_t st) {
    return launch_long<policy_long_kernel<T, GRAD, NV>, NV>(p, kLongBlock, ranks, 0, st);
  }
  static rlcs_status any(const PolicyArgs &p, cudaStream_t st) {
    return launch_any(policy_rows_kernel<T, GRAD>, p, st);
  }
};

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
    return grad ? spread<float, Policy<float, true>>(p, 0, s)
                : spread<float, Policy<float, false>>(p, 0, s);
  return grad ? spread<bf, Policy<bf, true>>(p, 0, s) : spread<bf, Policy<bf, false>>(p, 0, s);
}

}  // namespace
}  // namespace loss
}  // namespace rlcs

using namespace rlcs;
using namespace rlcs::loss;

extern "C" {

rlcs_status rlcs_loss_status(void) {
  const rlcs_status a = take_status(&device_status), b = distill_status();
  return a > b ? a : b;
}

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

}  // extern "C"
