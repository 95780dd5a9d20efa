// Causal attention over packed episodes with grouped heads (rlcs_seq.h):
// forward, gradient, and one new token over a cache.
//
// The softmax runs over the keys in one pass with a running maximum and sum;
// scores are kept in base 2 (scale * log2 e folded into one factor).
#include "seq_common.cuh"

namespace rlcs {
namespace seq {
namespace {

using bf = __nv_bfloat16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnArgs {
  const bf *q, *k, *v, *dout, *out;
  int64_t qt, qh, kt, kh, vt, vh;  // token and head strides
  const int32_t *cu;
  float *lse;    // [Hq, tokens]
  float *delta;  // [Hq, tokens]
  bf *o, *dq, *dk, *dv;
  int64_t sequences, tokens, Hq, Hk;
  int D, group;
  float scale;
};

// The sequence that holds token i: [lo, hi), empty if none does.
__device__ __forceinline__ void sequence_of(const AttnArgs &p, int64_t i, int64_t &lo, int64_t &hi) {
  int64_t a = 0, b = p.sequences;  // the last s with cu[s] <= i
  while (b - a > 1) {
    const int64_t m = (a + b) / 2;
    if (p.cu[m] <= i) a = m;
    else b = m;
  }
  lo = p.cu[a] < 0 ? 0 : p.cu[a];
  hi = p.cu[a + 1] < p.tokens ? p.cu[a + 1] : p.tokens;
  if (i < lo || i >= hi) lo = hi = i;
}

__device__ __forceinline__ float dot_row(const float *s, const bf *r, int D) {
  float t = 0.0f;
  for (int d = 0; d < D; d += 8) {
    const uint4 w = *reinterpret_cast<const uint4 *>(r + d);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      t = fmaf(s[d + 2 * j], __uint_as_float(u[j] << 16), t);
      t = fmaf(s[d + 2 * j + 1], __uint_as_float(u[j] & 0xffff0000u), t);
    }
  }
  return t;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
// acc[e] += w * r[lane + 32 e]
__device__ __forceinline__ void add_row(float (&acc)[4], float w, const bf *r, int lane, int D) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (lane + 32 * e < D) acc[e] = fmaf(w, __bfloat162float(r[lane + 32 * e]), acc[e]);
}
__device__ __forceinline__ void stage(float *s, const bf *r, int lane, int D) {
  for (int d = lane; d < D; d += 32) s[d] = __bfloat162float(r[d]);
}

// One warp per query row: keys in steps of 32, a key per lane for the scores.
__device__ __forceinline__ void attend(const float *qs, const bf *k, int64_t kt, const bf *v,
                                       int64_t vt, int64_t n, int D, float scale2, int lane,
                                       float (&acc)[4], float &m, float &l) {
  m = -INFINITY;
  l = 0.0f;
  for (int64_t j0 = 0; j0 < n; j0 += 32) {
    const bool in = j0 + lane < n;
    const float s = in ? dot_row(qs, k + (j0 + lane) * kt, D) * scale2 : -INFINITY;
    const float mn = fmaxf(m, warp_max(s)), ms = mn == -INFINITY ? 0.0f : mn;
    const float pj = exp2f(s - ms), f = exp2f(m - ms);
    l = l * f + warp_sum(pj);
    m = mn;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] *= f;
    for (int j = 0; j < 32 && j0 + j < n; ++j)
      add_row(acc, __shfl_sync(kFull, pj, j), v + (j0 + j) * vt, lane, D);
  }
}

__global__ void __launch_bounds__(128) attention_kernel(const AttnArgs p) {
  __shared__ float qs[4][128];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * 4 + warp, i = row / p.Hq, h = row % p.Hq;
  if (i >= p.tokens) return;
  int64_t lo, hi;
  sequence_of(p, i, lo, hi);
  if (lo == hi) return;
  stage(qs[warp], p.q + i * p.qt + h * p.qh, lane, p.D);
  __syncwarp();
  const int64_t g = h / p.group;
  float acc[4] = {}, m, l;
  attend(qs[warp], p.k + lo * p.kt + g * p.kh, p.kt, p.v + lo * p.vt + g * p.vh, p.vt, i - lo + 1,
         p.D, p.scale * kLog2e, lane, acc, m, l);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (lane + 32 * e < p.D)
      p.o[(i * p.Hq + h) * p.D + lane + 32 * e] = __float2bfloat16_rn(acc[e] / l);
  if (p.lse && lane == 0) p.lse[h * p.tokens + i] = (m + log2f(l)) * kLn2;
}

// delta_i = sum_d dout_id out_id
__global__ void __launch_bounds__(128) attention_delta_kernel(const AttnArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5), i = row / p.Hq, h = row % p.Hq;
  if (i >= p.tokens) return;
  float t = 0.0f;
  for (int d = lane; d < p.D; d += 32)
    t = fmaf(__bfloat162float(p.dout[row * p.D + d]), __bfloat162float(p.out[row * p.D + d]), t);
  t = warp_sum(t);
  if (lane == 0) p.delta[h * p.tokens + i] = t;
}

__global__ void __launch_bounds__(128) attention_dq_kernel(const AttnArgs p) {
  __shared__ float qs[4][128], ds[4][128];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * 4 + warp, i = row / p.Hq, h = row % p.Hq;
  if (i >= p.tokens) return;
  int64_t lo, hi;
  sequence_of(p, i, lo, hi);
  if (lo == hi) return;
  stage(qs[warp], p.q + i * p.qt + h * p.qh, lane, p.D);
  stage(ds[warp], p.dout + row * p.D, lane, p.D);
  __syncwarp();
  const int64_t g = h / p.group;
  const float lse = p.lse[h * p.tokens + i] * kLog2e, delta = p.delta[h * p.tokens + i];
  float acc[4] = {};
  for (int64_t j0 = lo; j0 <= i; j0 += 32) {
    const int64_t j = j0 + lane;
    float t = 0.0f;
    if (j <= i) {
      const float pj = exp2f(dot_row(qs[warp], p.k + j * p.kt + g * p.kh, p.D) * p.scale * kLog2e -
                             lse);
      t = pj * (dot_row(ds[warp], p.v + j * p.vt + g * p.vh, p.D) - delta);
    }
    for (int e = 0; e < 32 && j0 + e <= i; ++e)
      add_row(acc, __shfl_sync(kFull, t, e), p.k + (j0 + e) * p.kt + g * p.kh, lane, p.D);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (lane + 32 * e < p.D)
      p.dq[row * p.D + lane + 32 * e] = __float2bfloat16_rn(acc[e] * p.scale);
}

__global__ void __launch_bounds__(128) attention_dkv_kernel(const AttnArgs p) {
  __shared__ float ks[4][128], vs[4][128];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * 4 + warp, j = row / p.Hk, g = row % p.Hk;
  if (j >= p.tokens) return;
  int64_t lo, hi;
  sequence_of(p, j, lo, hi);
  if (lo == hi) return;
  stage(ks[warp], p.k + j * p.kt + g * p.kh, lane, p.D);
  stage(vs[warp], p.v + j * p.vt + g * p.vh, lane, p.D);
  __syncwarp();
  float dk[4] = {}, dv[4] = {};
  for (int64_t h = g * p.group; h < (g + 1) * p.group; ++h)
    for (int64_t i0 = j; i0 < hi; i0 += 32) {
      const int64_t i = i0 + lane;
      float pj = 0.0f, t = 0.0f;
      if (i < hi) {
        pj = exp2f((dot_row(ks[warp], p.q + i * p.qt + h * p.qh, p.D) * p.scale -
                    p.lse[h * p.tokens + i]) * kLog2e);
        t = pj * (dot_row(vs[warp], p.dout + (i * p.Hq + h) * p.D, p.D) - p.delta[h * p.tokens + i]);
      }
      for (int e = 0; e < 32 && i0 + e < hi; ++e) {
        add_row(dv, __shfl_sync(kFull, pj, e), p.dout + ((i0 + e) * p.Hq + h) * p.D, lane, p.D);
        add_row(dk, __shfl_sync(kFull, t, e), p.q + (i0 + e) * p.qt + h * p.qh, lane, p.D);
      }
    }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (lane + 32 * e < p.D) {
      p.dk[row * p.D + lane + 32 * e] = __float2bfloat16_rn(dk[e] * p.scale);
      p.dv[row * p.D + lane + 32 * e] = __float2bfloat16_rn(dv[e]);
    }
}

struct StepArgs {
  const bf *q, *k, *v;
  int64_t kb, kt, kh, vb, vt, vh;
  const int32_t *lengths;
  bf *o;
  int64_t B, S, Hq, Hk;
  int D, group;
  float scale;
};

__global__ void __launch_bounds__(128) attention_step_kernel(const StepArgs p) {
  __shared__ float qs[4][128];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * 4 + warp, b = row / p.Hq, h = row % p.Hq;
  if (b >= p.B) return;
  int64_t n = p.lengths[b];
  n = n < 0 ? 0 : (n > p.S ? p.S : n);
  stage(qs[warp], p.q + row * p.D, lane, p.D);
  __syncwarp();
  const int64_t g = h / p.group;
  float acc[4] = {}, m, l;
  attend(qs[warp], p.k + b * p.kb + g * p.kh, p.kt, p.v + b * p.vb + g * p.vh, p.vt, n, p.D,
         p.scale * kLog2e, lane, acc, m, l);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (lane + 32 * e < p.D)
      p.o[row * p.D + lane + 32 * e] = __float2bfloat16_rn(n > 0 ? acc[e] / l : 0.0f);
}

// Token and head strides that 16-byte loads can use.
rlcs_status strides_usable(const void *p, int64_t ts, int64_t hs, int64_t tokens, int64_t heads) {
  if (ts < 0 || hs < 0 || !product_fits(tokens, ts, 1) || !product_fits(heads, hs, 1))
    return RLCS_ERR_INVALID_ARG;
  return ts % 8 == 0 && hs % 8 == 0 && aligned(p, 16) ? RLCS_OK : RLCS_ERR_MISALIGNED;
}

bool attn_sizes(int64_t sequences, int64_t tokens, int64_t Hq, int64_t Hk, int64_t D, double scale,
                rlcs_dtype t) {
  return sequences >= 0 && tokens >= 0 && tokens <= INT32_MAX && sequences < INT32_MAX && Hq > 0 &&
         Hk > 0 && Hq % Hk == 0 && D > 0 && D <= 128 && D % 8 == 0 && t == RLCS_BF16 &&
         scale == scale && product_fits(tokens, Hq, D) && tokens * Hq < (int64_t)4 * INT32_MAX;
}

dim3 row_grid(int64_t rows) { return dim3((unsigned)ceil_div(rows, 4)); }

}  // namespace
}  // namespace seq
}  // namespace rlcs

using namespace rlcs;
using namespace rlcs::seq;

extern "C" {

size_t rlcs_attention_scratch_bytes(int64_t tokens, int64_t Hq) {
  if (tokens < 0 || Hq <= 0 || !product_fits(tokens, Hq, 4)) return 0;
  return 64 + (size_t)ceil_div(tokens * Hq * 4, 64) * 64;
}

rlcs_status rlcs_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                           const void *k, int64_t k_token_stride, int64_t k_head_stride,
                           const void *v, int64_t v_token_stride, int64_t v_head_stride,
                           const int32_t *cu_seqlens, void *out, float *lse, int64_t sequences,
                           int64_t tokens, int64_t Hq, int64_t Hk, int64_t D, double scale,
                           rlcs_dtype dtype, void *scratch, size_t scratch_bytes,
                           rlcs_stream_t stream) {
  if (!attn_sizes(sequences, tokens, Hq, Hk, D, scale, dtype)) return RLCS_ERR_INVALID_ARG;
  if (tokens == 0 || sequences == 0) return RLCS_OK;
  if (!q || !k || !v || !cu_seqlens || !out) return RLCS_ERR_INVALID_ARG;
  const rlcs_status su[] = {strides_usable(q, q_token_stride, q_head_stride, tokens, Hq),
                            strides_usable(k, k_token_stride, k_head_stride, tokens, Hk),
                            strides_usable(v, v_token_stride, v_head_stride, tokens, Hk)};
  for (rlcs_status s : su)
    if (s != RLCS_OK) return s;
  if (!aligned(out, 16)) return RLCS_ERR_MISALIGNED;
  const Range outs[] = {range(out, tokens * Hq * D * 2), range(lse, tokens * Hq * 4),
                        range(scratch, (int64_t)scratch_bytes)};
  const Range ins[] = {strided(q, tokens, q_token_stride, Hq, q_head_stride, D, 2),
                       strided(k, tokens, k_token_stride, Hk, k_head_stride, D, 2),
                       strided(v, tokens, v_token_stride, Hk, v_head_stride, D, 2),
                       range(cu_seqlens, (sequences + 1) * 4)};
  if (outputs_overlap(outs, ins)) return RLCS_ERR_INVALID_ARG;
  if (!scratch || scratch_bytes < rlcs_attention_scratch_bytes(tokens, Hq) || !aligned(scratch, 16))
    return RLCS_ERR_WORKSPACE;
  AttnArgs a = {};
  a.q = static_cast<const bf *>(q);
  a.k = static_cast<const bf *>(k);
  a.v = static_cast<const bf *>(v);
  a.qt = q_token_stride;
  a.qh = q_head_stride;
  a.kt = k_token_stride;
  a.kh = k_head_stride;
  a.vt = v_token_stride;
  a.vh = v_head_stride;
  a.cu = cu_seqlens;
  a.o = static_cast<bf *>(out);
  a.lse = lse;
  a.sequences = sequences;
  a.tokens = tokens;
  a.Hq = Hq;
  a.Hk = Hk;
  a.D = (int)D;
  a.group = (int)(Hq / Hk);
  a.scale = (float)scale;
  return launched(launch_ex(attention_kernel, row_grid(tokens * Hq), dim3(128), 0,
                            reinterpret_cast<cudaStream_t>(stream), true, a));
}

rlcs_status rlcs_attention_backward(
    const void *dout, const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
    int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
    int64_t v_head_stride, const void *out, const float *lse, const int32_t *cu_seqlens, void *dq,
    void *dk, void *dv, int64_t sequences, int64_t tokens, int64_t Hq, int64_t Hk, int64_t D,
    double scale, rlcs_dtype dtype, void *scratch, size_t scratch_bytes, rlcs_stream_t stream) {
  if (!attn_sizes(sequences, tokens, Hq, Hk, D, scale, dtype)) return RLCS_ERR_INVALID_ARG;
  if (tokens == 0 || sequences == 0) return RLCS_OK;
  if (!dout || !q || !k || !v || !out || !lse || !cu_seqlens || !dq || !dk || !dv)
    return RLCS_ERR_INVALID_ARG;
  const rlcs_status su[] = {strides_usable(q, q_token_stride, q_head_stride, tokens, Hq),
                            strides_usable(k, k_token_stride, k_head_stride, tokens, Hk),
                            strides_usable(v, v_token_stride, v_head_stride, tokens, Hk)};
  for (rlcs_status s : su)
    if (s != RLCS_OK) return s;
  if (!aligned(dout, 16) || !aligned(out, 16) || !aligned(dq, 16) || !aligned(dk, 16) ||
      !aligned(dv, 16))
    return RLCS_ERR_MISALIGNED;
  const int64_t nq = tokens * Hq * D * 2, nk = tokens * Hk * D * 2;
  const Range outs[] = {range(dq, nq), range(dk, nk), range(dv, nk),
                        range(scratch, (int64_t)scratch_bytes)};
  const Range ins[] = {strided(q, tokens, q_token_stride, Hq, q_head_stride, D, 2),
                       strided(k, tokens, k_token_stride, Hk, k_head_stride, D, 2),
                       strided(v, tokens, v_token_stride, Hk, v_head_stride, D, 2),
                       range(dout, nq),
                       range(out, nq),
                       range(lse, tokens * Hq * 4),
                       range(cu_seqlens, (sequences + 1) * 4)};
  if (outputs_overlap(outs, ins)) return RLCS_ERR_INVALID_ARG;
  if (!scratch || scratch_bytes < rlcs_attention_scratch_bytes(tokens, Hq) || !aligned(scratch, 16))
    return RLCS_ERR_WORKSPACE;
  AttnArgs a = {};
  a.dout = static_cast<const bf *>(dout);
  a.out = static_cast<const bf *>(out);
  a.q = static_cast<const bf *>(q);
  a.k = static_cast<const bf *>(k);
  a.v = static_cast<const bf *>(v);
  a.qt = q_token_stride;
  a.qh = q_head_stride;
  a.kt = k_token_stride;
  a.kh = k_head_stride;
  a.vt = v_token_stride;
  a.vh = v_head_stride;
  a.cu = cu_seqlens;
  a.lse = const_cast<float *>(lse);
  a.delta = reinterpret_cast<float *>(static_cast<char *>(scratch) + 64);
  a.dq = static_cast<bf *>(dq);
  a.dk = static_cast<bf *>(dk);
  a.dv = static_cast<bf *>(dv);
  a.sequences = sequences;
  a.tokens = tokens;
  a.Hq = Hq;
  a.Hk = Hk;
  a.D = (int)D;
  a.group = (int)(Hq / Hk);
  a.scale = (float)scale;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_ex(attention_delta_kernel, row_grid(tokens * Hq), dim3(128), 0, st, true, a);
  if (e == cudaSuccess)
    e = launch_ex(attention_dkv_kernel, row_grid(tokens * Hk), dim3(128), 0, st, true, a);
  if (e == cudaSuccess)
    e = launch_ex(attention_dq_kernel, row_grid(tokens * Hq), dim3(128), 0, st, true, a);
  return launched(e);
}

size_t rlcs_attention_step_scratch_bytes(int64_t B, int64_t S, int64_t Hq, int64_t Hk, int64_t D) {
  (void)S;
  (void)Hk;
  return B <= 0 || Hq <= 0 || D <= 0 ? 0 : 16;
}

rlcs_status rlcs_attention_step(const void *q, const void *k_cache, int64_t k_batch_stride,
                                int64_t k_position_stride, int64_t k_head_stride,
                                const void *v_cache, int64_t v_batch_stride,
                                int64_t v_position_stride, int64_t v_head_stride,
                                const int32_t *lengths, void *out, int64_t B, int64_t S,
                                int64_t Hq, int64_t Hk, int64_t D, double scale, rlcs_dtype dtype,
                                void *scratch, size_t scratch_bytes, rlcs_stream_t stream) {
  if (B < 0 || S < 0 || !attn_sizes(0, B, Hq, Hk, D, scale, dtype) ||
      !product_fits(B, k_batch_stride < 0 ? 0 : k_batch_stride, 1) ||
      !product_fits(B, v_batch_stride < 0 ? 0 : v_batch_stride, 1) || k_batch_stride < 0 ||
      v_batch_stride < 0)
    return RLCS_ERR_INVALID_ARG;
  if (B == 0) return RLCS_OK;
  if (!q || !lengths || !out || (S > 0 && (!k_cache || !v_cache))) return RLCS_ERR_INVALID_ARG;
  const rlcs_status su[] = {strides_usable(k_cache, k_position_stride, k_head_stride, S, Hk),
                            strides_usable(v_cache, v_position_stride, v_head_stride, S, Hk)};
  for (rlcs_status s : su)
    if (s != RLCS_OK) return s;
  if (k_batch_stride % 8 || v_batch_stride % 8 || !aligned(q, 16) || !aligned(out, 16))
    return RLCS_ERR_MISALIGNED;
  const Range none = range(nullptr, 0);
  const int64_t n = B * Hq * D * 2;
  const int64_t kl = (B - 1) * k_batch_stride + (S - 1) * k_position_stride +
                     (Hk - 1) * k_head_stride + D;
  const int64_t vl = (B - 1) * v_batch_stride + (S - 1) * v_position_stride +
                     (Hk - 1) * v_head_stride + D;
  const Range outs[] = {range(out, n), range(scratch, (int64_t)scratch_bytes)};
  const Range ins[] = {range(q, n), S > 0 ? range(k_cache, kl * 2) : none,
                       S > 0 ? range(v_cache, vl * 2) : none, range(lengths, B * 4)};
  if (outputs_overlap(outs, ins)) return RLCS_ERR_INVALID_ARG;
  if (!scratch || scratch_bytes < rlcs_attention_step_scratch_bytes(B, S, Hq, Hk, D) ||
      !aligned(scratch, 16))
    return RLCS_ERR_WORKSPACE;
  StepArgs a = {};
  a.q = static_cast<const bf *>(q);
  a.k = static_cast<const bf *>(k_cache);
  a.v = static_cast<const bf *>(v_cache);
  a.kb = k_batch_stride;
  a.kt = k_position_stride;
  a.kh = k_head_stride;
  a.vb = v_batch_stride;
  a.vt = v_position_stride;
  a.vh = v_head_stride;
  a.lengths = lengths;
  a.o = static_cast<bf *>(out);
  a.B = B;
  a.S = S;
  a.Hq = Hq;
  a.Hk = Hk;
  a.D = (int)D;
  a.group = (int)(Hq / Hk);
  a.scale = (float)scale;
  return launched(launch_ex(attention_step_kernel, row_grid(B * Hq), dim3(128), 0,
                            reinterpret_cast<cudaStream_t>(stream), true, a));
}

}  // extern "C"
