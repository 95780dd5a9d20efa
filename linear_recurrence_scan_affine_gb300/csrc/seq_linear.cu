// Linear attention with a decay for each head (rlcs_seq.h): forward, gradient
// and single steps.
//
// One walk serves all of them. A state S [D x D] per sequence and head takes
// in y_t z_t^T each step, and each x_t reads it:
//   forward    S = a S + y z^T, out = x S      (x, y, z) = (q, k, v):      out
//                                              (dout, v, k), state^T:      dq
//   backward   S = S + y z^T, out = x S, S = a S, from the last token:
//                                              (k, q, dout), dlast:        dv
//                                              (v, dout, q), dlast^T:      dk
// A state is shared by the query heads of its group: they are several x
// forwards, several y and z backwards.
#include "seq_common.cuh"

namespace rlcs {
namespace seq {
namespace {

using bf = __nv_bfloat16;

struct View {  // [tokens, heads, D]
  const bf *p;
  int64_t token, head;
};
struct WalkArgs {
  View x, y, z;
  const float *log_decay;
  const int32_t *cu;
  const float *init;  // [sequences, Hk, D, D] or null
  float *last;        // the same
  bf *out;            // [tokens, Hk * nx, D]
  int64_t sequences, tokens;
  int Hk, nx, ny, D;
  bool backward, transposed;  // walk from the end; init is [z's dimension, y's]
  float in_scale, out_scale;  // of y z^T, and of x S
};

// One column of the state to a thread.
template <int DP>
__global__ void __launch_bounds__(DP) linear_walk_kernel(const WalkArgs p) {
  __shared__ float x[DP], y[DP];
  pdl_wait();
  pdl_launch_dependents();
  const int e = threadIdx.x, h = blockIdx.x % p.Hk, D = p.D;
  const int64_t s = blockIdx.x / p.Hk, tokens = p.tokens;
  const auto bound = [&](int64_t i) {
    const int64_t b = p.cu[i];
    return b < 0 ? 0 : (b < tokens ? b : tokens);
  };
  if (s == p.sequences) {  // tokens that no sequence holds
    const int64_t lo = bound(0), hi = bound(p.sequences);
    for (int64_t t = 0; t < tokens; ++t)
      if ((t < lo || t >= hi) && e < D)
        for (int i = 0; i < p.nx; ++i)
          p.out[((t * p.Hk + h) * p.nx + i) * D + e] = __float2bfloat16_rn(0.0f);
    return;
  }
  const int64_t lo = bound(s), hi = bound(s + 1), n = hi > lo ? hi - lo : 0;
  const float a = expf(p.log_decay[h]);
  const int64_t base = (s * p.Hk + h) * D * D;
  float S[DP];
#pragma unroll
  for (int d = 0; d < DP; ++d)
    S[d] = p.init && d < D && e < D ? p.init[base + (p.transposed ? e * D + d : d * D + e)] : 0.0f;
  for (int64_t i = 0; i < n; ++i) {
    const int64_t t = p.backward ? hi - 1 - i : lo + i;
    if (!p.backward)
#pragma unroll
      for (int d = 0; d < DP; ++d) S[d] = a == 0.0f ? 0.0f : S[d] * a;
    for (int j = 0; j < p.ny; ++j) {
      __syncthreads();
      y[e] = e < D ? __bfloat162float(p.y.p[t * p.y.token + (h * p.ny + j) * p.y.head + e]) : 0.0f;
      __syncthreads();
      const float z = e < D ? p.in_scale * __bfloat162float(
                                  p.z.p[t * p.z.token + (h * p.ny + j) * p.z.head + e]) : 0.0f;
#pragma unroll
      for (int d = 0; d < DP; ++d) S[d] = fmaf(y[d], z, S[d]);
    }
    for (int j = 0; j < p.nx; ++j) {
      __syncthreads();
      x[e] = e < D ? __bfloat162float(p.x.p[t * p.x.token + (h * p.nx + j) * p.x.head + e]) : 0.0f;
      __syncthreads();
      float o = 0.0f;
#pragma unroll
      for (int d = 0; d < DP; ++d) o = fmaf(x[d], S[d], o);
      if (e < D)
        p.out[((t * p.Hk + h) * p.nx + j) * D + e] = __float2bfloat16_rn(o * p.out_scale);
    }
    if (p.backward)
#pragma unroll
      for (int d = 0; d < DP; ++d) S[d] = a == 0.0f ? 0.0f : S[d] * a;
  }
  if (p.last && e < D)
#pragma unroll
    for (int d = 0; d < DP; ++d)
      if (d < D) p.last[base + (p.transposed ? e * D + d : d * D + e)] = S[d];
}

cudaError_t launch_walk(const WalkArgs &p, cudaStream_t st) {
  const dim3 grid((unsigned)((p.sequences + 1) * p.Hk));
  return p.D <= 64 ? launch_ex(linear_walk_kernel<64>, grid, dim3(64), 0, st, true, p)
                   : launch_ex(linear_walk_kernel<128>, grid, dim3(128), 0, st, true, p);
}

// ---------------------------------------------------------------------------
// One step: the state's rows are spread over a warp each
// ---------------------------------------------------------------------------
struct StepArgs {
  View q, k, v;
  const float *log_decay;
  const uint8_t *reset;
  const float *state;
  float *next;
  bf *out;
  int64_t B;
  int Hk, group, D;
  float scale;
};

__global__ void __launch_bounds__(128) linear_step_kernel(const StepArgs p) {
  __shared__ float q[128], k[128];
  pdl_wait();
  pdl_launch_dependents();
  const int e = threadIdx.x, D = p.D;
  for (int64_t unit = blockIdx.x; unit < p.B * p.Hk; unit += gridDim.x) {
    const int64_t b = unit / p.Hk;
    const int h = (int)(unit % p.Hk);
    const float a = p.reset && p.reset[b] ? 0.0f : expf(p.log_decay[h]);
    const bool on = e < D;
    __syncthreads();
    k[e] = on ? __bfloat162float(p.k.p[b * p.k.token + h * p.k.head + e]) : 0.0f;
    __syncthreads();
    const float v = on ? __bfloat162float(p.v.p[b * p.v.token + h * p.v.head + e]) : 0.0f;
    for (int d = 0; on && d < D; ++d) {
      const int64_t at = (unit * D + d) * D + e;
      const float kept = a == 0.0f ? 0.0f : a * p.state[at];
      p.next[at] = fmaf(k[d], v, kept);
    }
    for (int g = 0; g < p.group; ++g) {
      __syncthreads();
      const int head = h * p.group + g;
      q[e] = on ? __bfloat162float(p.q.p[b * p.q.token + head * p.q.head + e]) : 0.0f;
      __syncthreads();
      float o = 0.0f;
      for (int d = 0; on && d < D; ++d) o = fmaf(q[d], p.next[(unit * D + d) * D + e], o);
      if (on) p.out[(unit * p.group + g) * D + e] = __float2bfloat16_rn(o * p.scale);
    }
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// Token and head strides that 16-byte loads can use.
rlcs_status strides_usable(const void *p, int64_t ts, int64_t hs, int64_t tokens, int64_t heads) {
  if (ts < 0 || hs < 0 || !product_fits(tokens, ts, 1) || !product_fits(heads, hs, 1))
    return RLCS_ERR_INVALID_ARG;
  return ts % 8 == 0 && hs % 8 == 0 && aligned(p, 16) ? RLCS_OK : RLCS_ERR_MISALIGNED;
}

bool linear_sizes(int64_t sequences, int64_t tokens, int64_t Hq, int64_t Hk, int64_t D,
                  double scale, rlcs_dtype t) {
  return sequences >= 0 && tokens >= 0 && tokens <= INT32_MAX && Hq > 0 && Hk > 0 &&
         Hq % Hk == 0 && D > 0 && D <= 128 && D % 8 == 0 && t == RLCS_BF16 && scale >= 1e-30 &&
         scale <= 1e30 && product_fits(tokens, Hq, D) && sequences < INT32_MAX - 1024 &&
         Hq < INT32_MAX && (sequences + tokens / 64 + 1) * Hq < (int64_t)INT32_MAX;
}

}  // namespace
}  // namespace seq
}  // namespace rlcs

using namespace rlcs;
using namespace rlcs::seq;

extern "C" {

size_t rlcs_linear_attention_scratch_bytes(int64_t sequences, int64_t tokens, int64_t Hq,
                                           int64_t Hk, int64_t D) {
  if (!linear_sizes(sequences, tokens, Hq, Hk, D, 1.0, RLCS_BF16)) return 0;
  return 64;
}

rlcs_status rlcs_linear_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                  const void *k, int64_t k_token_stride, int64_t k_head_stride,
                                  const void *v, int64_t v_token_stride, int64_t v_head_stride,
                                  const float *log_decay, const int32_t *cu_seqlens,
                                  const float *state, void *out, float *last_state,
                                  int64_t sequences, int64_t tokens, int64_t Hq, int64_t Hk,
                                  int64_t D, double scale, rlcs_dtype dtype, void *scratch,
                                  size_t scratch_bytes, rlcs_stream_t stream) {
  if (!linear_sizes(sequences, tokens, Hq, Hk, D, scale, dtype)) return RLCS_ERR_INVALID_ARG;
  if (sequences == 0) return RLCS_OK;
  if (!log_decay || !cu_seqlens || (tokens > 0 && (!q || !k || !v || !out)))
    return RLCS_ERR_INVALID_ARG;
  if (tokens > 0) {
    const rlcs_status su[] = {strides_usable(q, q_token_stride, q_head_stride, tokens, Hq),
                              strides_usable(k, k_token_stride, k_head_stride, tokens, Hk),
                              strides_usable(v, v_token_stride, v_head_stride, tokens, Hk)};
    for (rlcs_status s : su)
      if (s != RLCS_OK) return s;
  }
  if (!aligned(out, 16) || !aligned(state, 16) || !aligned(last_state, 16))
    return RLCS_ERR_MISALIGNED;
  const int64_t states = sequences * Hk * D * D * 4;
  const Range none = range(nullptr, 0);
  const Range outs[] = {range(out, tokens * Hq * D * 2), range(last_state, states),
                        range(scratch, (int64_t)scratch_bytes)};
  const Range ins[] = {
      tokens ? strided(q, tokens, q_token_stride, Hq, q_head_stride, D, 2) : none,
      tokens ? strided(k, tokens, k_token_stride, Hk, k_head_stride, D, 2) : none,
      tokens ? strided(v, tokens, v_token_stride, Hk, v_head_stride, D, 2) : none,
      range(log_decay, Hk * 4), range(cu_seqlens, (sequences + 1) * 4), range(state, states)};
  if (outputs_overlap(outs, ins)) return RLCS_ERR_INVALID_ARG;
  if (!scratch || !aligned(scratch, 16) ||
      scratch_bytes < rlcs_linear_attention_scratch_bytes(sequences, tokens, Hq, Hk, D))
    return RLCS_ERR_WORKSPACE;
  WalkArgs a = {};
  a.x = {static_cast<const bf *>(q), q_token_stride, q_head_stride};
  a.y = {static_cast<const bf *>(k), k_token_stride, k_head_stride};
  a.z = {static_cast<const bf *>(v), v_token_stride, v_head_stride};
  a.log_decay = log_decay;
  a.cu = cu_seqlens;
  a.init = state;
  a.last = last_state;
  a.out = static_cast<bf *>(out);
  a.sequences = sequences;
  a.tokens = tokens;
  a.Hk = (int)Hk;
  a.nx = (int)(Hq / Hk);
  a.ny = 1;
  a.D = (int)D;
  a.in_scale = 1.0f;
  a.out_scale = (float)scale;
  return launched(launch_walk(a, reinterpret_cast<cudaStream_t>(stream)));
}

rlcs_status rlcs_linear_attention_backward(
    const void *dout, const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
    int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
    int64_t v_head_stride, const float *log_decay, const int32_t *cu_seqlens, const float *state,
    const float *dlast, void *dq, void *dk, void *dv, float *dstate, int64_t sequences,
    int64_t tokens, int64_t Hq, int64_t Hk, int64_t D, double scale, rlcs_dtype dtype,
    void *scratch, size_t scratch_bytes, rlcs_stream_t stream) {
  if (!linear_sizes(sequences, tokens, Hq, Hk, D, scale, dtype)) return RLCS_ERR_INVALID_ARG;
  if (sequences == 0) return RLCS_OK;
  if (!log_decay || !cu_seqlens || (tokens > 0 && (!dout || !q || !k || !v || !dq || !dk || !dv)))
    return RLCS_ERR_INVALID_ARG;
  if (tokens > 0) {
    const rlcs_status su[] = {strides_usable(q, q_token_stride, q_head_stride, tokens, Hq),
                              strides_usable(k, k_token_stride, k_head_stride, tokens, Hk),
                              strides_usable(v, v_token_stride, v_head_stride, tokens, Hk)};
    for (rlcs_status s : su)
      if (s != RLCS_OK) return s;
  }
  if (!aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) ||
      !aligned(state, 16) || !aligned(dlast, 16) || !aligned(dstate, 16))
    return RLCS_ERR_MISALIGNED;
  const int64_t states = sequences * Hk * D * D * 4, nq = tokens * Hq * D * 2,
                nk = tokens * Hk * D * 2;
  const Range none = range(nullptr, 0);
  const Range outs[] = {range(dq, nq), range(dk, nk), range(dv, nk), range(dstate, states),
                        range(scratch, (int64_t)scratch_bytes)};
  const Range ins[] = {
      tokens ? strided(q, tokens, q_token_stride, Hq, q_head_stride, D, 2) : none,
      tokens ? strided(k, tokens, k_token_stride, Hk, k_head_stride, D, 2) : none,
      tokens ? strided(v, tokens, v_token_stride, Hk, v_head_stride, D, 2) : none,
      range(dout, nq), range(log_decay, Hk * 4), range(cu_seqlens, (sequences + 1) * 4),
      range(state, states), range(dlast, states)};
  if (outputs_overlap(outs, ins)) return RLCS_ERR_INVALID_ARG;
  if (!scratch || !aligned(scratch, 16) ||
      scratch_bytes < rlcs_linear_attention_scratch_bytes(sequences, tokens, Hq, Hk, D))
    return RLCS_ERR_WORKSPACE;
  const View vq = {static_cast<const bf *>(q), q_token_stride, q_head_stride},
             vk = {static_cast<const bf *>(k), k_token_stride, k_head_stride},
             vv = {static_cast<const bf *>(v), v_token_stride, v_head_stride},
             vd = {static_cast<const bf *>(dout), Hq * D, D};
  WalkArgs a = {};
  a.log_decay = log_decay;
  a.cu = cu_seqlens;
  a.sequences = sequences;
  a.tokens = tokens;
  a.Hk = (int)Hk;
  a.D = (int)D;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // dq
  a.x = vd, a.y = vv, a.z = vk;
  a.nx = (int)(Hq / Hk), a.ny = 1;
  a.in_scale = 1.0f, a.out_scale = (float)scale;
  a.init = state, a.last = nullptr, a.transposed = true, a.backward = false;
  a.out = static_cast<bf *>(dq);
  cudaError_t e = launch_walk(a, st);
  if (e != cudaSuccess) return launched(e);
  // dv
  a.x = vk, a.y = vq, a.z = vd;
  a.nx = 1, a.ny = (int)(Hq / Hk);
  a.in_scale = (float)scale, a.out_scale = 1.0f;
  a.init = dlast, a.last = dstate, a.transposed = false, a.backward = true;
  a.out = static_cast<bf *>(dv);
  e = launch_walk(a, st);
  if (e != cudaSuccess) return launched(e);
  // dk
  a.x = vv, a.y = vd, a.z = vq;
  a.last = nullptr, a.transposed = true;
  a.out = static_cast<bf *>(dk);
  return launched(launch_walk(a, st));
}

rlcs_status rlcs_linear_attention_step(const void *q, int64_t q_batch_stride,
                                       int64_t q_head_stride, const void *k,
                                       int64_t k_batch_stride, int64_t k_head_stride,
                                       const void *v, int64_t v_batch_stride,
                                       int64_t v_head_stride, const float *log_decay,
                                       const uint8_t *reset, const float *state, float *new_state,
                                       void *out, int64_t B, int64_t Hq, int64_t Hk, int64_t D,
                                       double scale, rlcs_dtype dtype, rlcs_stream_t stream) {
  if (!linear_sizes(0, B, Hq, Hk, D, scale, dtype) || !product_fits(B, Hk, D, D) ||
      q_batch_stride < 0 || q_head_stride < 0 || k_batch_stride < 0 || k_head_stride < 0 ||
      v_batch_stride < 0 || v_head_stride < 0 || !product_fits(B, q_batch_stride, 1) ||
      !product_fits(B, k_batch_stride, 1) || !product_fits(B, v_batch_stride, 1) ||
      !product_fits(Hq, q_head_stride, 1) || !product_fits(Hk, k_head_stride, 1) ||
      !product_fits(Hk, v_head_stride, 1))
    return RLCS_ERR_INVALID_ARG;
  if (B == 0) return RLCS_OK;
  if (!q || !k || !v || !log_decay || !state || !new_state || !out) return RLCS_ERR_INVALID_ARG;
  if (!aligned(q, 2) || !aligned(k, 2) || !aligned(v, 2) || !aligned(out, 16) ||
      !aligned(state, 16) || !aligned(new_state, 16))
    return RLCS_ERR_MISALIGNED;
  const int64_t states = B * Hk * D * D * 4;
  const Range outs[] = {range(new_state, states), range(out, B * Hq * D * 2)};
  const Range ins[] = {strided(q, B, q_batch_stride, Hq, q_head_stride, D, 2),
                       strided(k, B, k_batch_stride, Hk, k_head_stride, D, 2),
                       strided(v, B, v_batch_stride, Hk, v_head_stride, D, 2),
                       range(log_decay, Hk * 4),
                       range(reset, B),
                       state == new_state ? range(nullptr, 0) : range(state, states)};
  if (outputs_overlap(outs, ins) || meet(outs[1], range(state, states)))
    return RLCS_ERR_INVALID_ARG;
  const StepArgs a = {{static_cast<const bf *>(q), q_batch_stride, q_head_stride},
                      {static_cast<const bf *>(k), k_batch_stride, k_head_stride},
                      {static_cast<const bf *>(v), v_batch_stride, v_head_stride},
                      log_decay,
                      reset,
                      state,
                      new_state,
                      static_cast<bf *>(out),
                      B,
                      (int)Hk,
                      (int)(Hq / Hk),
                      (int)D,
                      (float)scale};
  const int64_t units = B * Hk;
  return launched(launch_ex(linear_step_kernel,
                            dim3((unsigned)(units < kSms * 8 ? units : kSms * 8)), dim3(128), 0,
                            reinterpret_cast<cudaStream_t>(stream), true, a));
}

}  // extern "C"
