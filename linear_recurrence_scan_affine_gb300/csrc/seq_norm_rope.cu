// Head norm and rotary positions (rlcs_seq.h): the rotary tables, the norm
// with rotation of query and key heads in one pass, and its gradient.
#include "seq_common.cuh"

namespace rlcs {
namespace seq {
namespace {

// ---------------------------------------------------------------------------
// Tables
// ---------------------------------------------------------------------------
struct TableArgs {
  float *cos, *sin;
  int64_t rows, half;
  double base, factor, trained_len, slow, fast, scale;
  int scaling;
};

__global__ void __launch_bounds__(256) rope_table_kernel(const TableArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.rows * a.half) return;
  const int64_t pos = i / a.half, pair = i % a.half;
  double base = a.base;
  if (a.scaling == RLCS_ROPE_BASE) base *= pow(a.factor, (double)a.half / (double)(a.half - 1));
  double f = pow(base, -(double)pair / (double)a.half);
  if (a.scaling == RLCS_ROPE_LINEAR) f /= a.factor;
  if (a.scaling == RLCS_ROPE_PARTS) {
    const double turns = a.trained_len * f / 6.283185307179586476925;
    double keep = (turns - a.slow) / (a.fast - a.slow);
    keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
    f *= keep + (1.0 - keep) / a.factor;
  }
  double s, c;
  sincos((double)pos * f, &s, &c);
  a.cos[i] = (float)(a.scale * c);
  a.sin[i] = (float)(a.scale * s);
}

// ---------------------------------------------------------------------------
// Norm and rotation
// ---------------------------------------------------------------------------
struct HeadArgs {
  const void *x[2];       // q, k
  const void *dy[2];      // backward: gradients of the outputs
  void *y[2];             // outputs, or dq and dk
  int64_t ts[2], hs[2];   // token and head strides of x
  const float *w[2];
  const float *cos, *sin;
  const int32_t *positions;
  float *partial;         // backward: [blocks][2][D]
  int64_t tokens, heads, Hq, max_pos;
  int D, half, inter;
  float eps, inv_d;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Any head width: a warp per head, lanes over rotation pairs, then over the
// elements past the rotated ones.
template <class E, bool BACK>
__global__ void __launch_bounds__(256) head_any_kernel(const HeadArgs p) {
  extern __shared__ float sums[];  // backward: [8 warps][2][D]
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float *mine = sums + warp * 2 * p.D;
  if (BACK)
    for (int i = lane; i < 2 * p.D; i += 32) mine[i] = 0.0f;
  __syncwarp();
  const int R = 2 * p.half;
  for (int64_t row = (int64_t)blockIdx.x * 8 + warp; row < p.tokens * p.heads;
       row += (int64_t)gridDim.x * 8) {
    const int64_t tok = row / p.heads, head = row % p.heads;
    const int which = head < p.Hq ? 0 : 1;
    const int64_t hh = which ? head - p.Hq : head, Hn = which ? p.heads - p.Hq : p.Hq;
    const E *x = static_cast<const E *>(p.x[which]) + tok * p.ts[which] + hh * p.hs[which];
    const E *dy = BACK ? static_cast<const E *>(p.dy[which]) + (tok * Hn + hh) * p.D : nullptr;
    E *y = static_cast<E *>(p.y[which]) + (tok * Hn + hh) * p.D;
    const float *w = p.w[which];
    const int64_t pos = p.positions[tok];
    const bool known_pos = pos >= 0 && pos < p.max_pos;
    float ss = 0.0f;
    for (int i = lane; i < p.D; i += 32) {
      const float v = (float)x[i];
      ss = fmaf(v, v, ss);
    }
    const float r = rsqrtf(warp_sum(ss) * p.inv_d + p.eps);
    float dot = 0.0f;  // backward: sum of w du x
    for (int pass = BACK ? 0 : 1; pass < 2; ++pass) {
      const float k = BACK ? dot * r * r * p.inv_d : 0.0f;
      for (int j = lane; j < p.half + (p.D - R); j += 32) {
        const bool pair = j < p.half;
        const int i0 = pair ? (p.inter ? 2 * j : j) : R + (j - p.half);
        const int i1 = pair ? (p.inter ? 2 * j + 1 : j + p.half) : i0;
        float c = 1.0f, s = 0.0f;
        if (pair) {
          c = known_pos ? p.cos[pos * p.half + j] : __int_as_float(0x7fffffff);
          s = known_pos ? p.sin[pos * p.half + j] : c;
        }
        const float x0 = (float)x[i0], x1 = (float)x[i1];
        if (!BACK) {
          const float u0 = x0 * r * w[i0], u1 = x1 * r * w[i1];
          const float y0[1] = {pair ? u0 * c - u1 * s : u0}, y1[1] = {u1 * c + u0 * s};
          store(y + i0, y0);
          if (pair) store(y + i1, y1);
        } else {
          const float g0 = (float)dy[i0], g1 = (float)dy[i1];
          const float d0 = pair ? g0 * c + g1 * s : g0, d1 = g1 * c - g0 * s;
          const float t0 = d0 * w[i0], t1 = d1 * w[i1];
          if (pass == 0) {
            dot = fmaf(t0, x0, dot);
            mine[which * p.D + i0] += d0 * x0 * r;
            if (pair) {
              dot = fmaf(t1, x1, dot);
              mine[which * p.D + i1] += d1 * x1 * r;
            }
          } else {
            const float o0[1] = {r * (t0 - x0 * k)}, o1[1] = {r * (t1 - x1 * k)};
            store(y + i0, o0);
            if (pair) store(y + i1, o1);
          }
        }
      }
      if (BACK && pass == 0) dot = warp_sum(dot);
    }
  }
  if (BACK) {
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.D; i += 256) {
      float t = 0.0f;
      for (int w = 0; w < 8; ++w) t += sums[w * 2 * p.D + i];
      p.partial[(int64_t)blockIdx.x * 2 * p.D + i] = t;
    }
  }
}

// Sum the blocks' partial weight gradients, in block order.
__global__ void __launch_bounds__(1024)
    weight_sum_kernel(const float *partial, int blocks, int D, float *dq, float *dk) {
  __shared__ float part[1024];
  pdl_wait();
  pdl_launch_dependents();
  const int i = blockIdx.x * 32 + (threadIdx.x & 31), row = threadIdx.x >> 5;
  float t = 0.0f;
  if (i < 2 * D)
    for (int b = row; b < blocks; b += 32) t += partial[(int64_t)b * 2 * D + i];
  part[threadIdx.x] = t;
  __syncthreads();
  if (row == 0 && i < 2 * D) {
    for (int k = 1; k < 32; ++k) t += part[k * 32 + threadIdx.x];
    float *out = i < D ? dq : dk;
    if (out) out[i < D ? i : i - D] = t;
  }
}

constexpr int kBlocksMax = 152 * 8;  // blocks that leave partial weight gradients

bool head_sizes(int64_t tokens, int64_t Hq, int64_t Hk, int64_t D, int64_t R, int64_t max_pos,
                double eps, rlcs_dtype t) {
  return tokens >= 0 && Hq > 0 && Hk >= 0 && D > 0 && D <= 1024 && R >= 0 && R <= D && R % 2 == 0 &&
         max_pos >= 0 && eps >= 0.0 && known(t) && Hq <= INT32_MAX && Hk <= INT32_MAX &&
         product_fits(tokens, Hq + Hk, D) && product_fits(max_pos, D, 1);
}

template <class E, bool BACK>
cudaError_t launch_heads(const HeadArgs &a, int blocks, cudaStream_t st) {
  const size_t smem = BACK ? (size_t)8 * 2 * a.D * sizeof(float) : 0;
  if (smem > 48 * 1024) {
    const cudaError_t e = allow_dynamic_smem<head_any_kernel<E, BACK>>(64 * 1024);
    if (e != cudaSuccess) return e;
  }
  return launch_ex(head_any_kernel<E, BACK>, dim3((unsigned)blocks), dim3(256), smem, st, true, a);
}

HeadArgs head_args(const void *q, int64_t qts, int64_t qhs, const void *k, int64_t kts,
                   int64_t khs, const float *qw, const float *kw, const float *cos,
                   const float *sin, const int32_t *positions, int64_t tokens, int64_t Hq,
                   int64_t Hk, int64_t D, int64_t R, int64_t max_pos, int inter, double eps) {
  HeadArgs a = {};
  a.x[0] = q;
  a.x[1] = k;
  a.ts[0] = qts;
  a.ts[1] = kts;
  a.hs[0] = qhs;
  a.hs[1] = khs;
  a.w[0] = qw;
  a.w[1] = kw;
  a.cos = cos;
  a.sin = sin;
  a.positions = positions;
  a.tokens = tokens;
  a.heads = Hq + Hk;
  a.Hq = Hq;
  a.max_pos = max_pos;
  a.D = (int)D;
  a.half = (int)(R / 2);
  a.inter = inter ? 1 : 0;
  a.eps = (float)eps;
  a.inv_d = 1.0f / (float)D;
  return a;
}

// Whether every array of a call is there and its strides are usable.
bool head_arrays(const HeadArgs &a, int64_t Hk) {
  if (!a.x[0] || !a.w[0] || !a.positions || !a.y[0]) return false;
  if (Hk > 0 && (!a.x[1] || !a.w[1] || !a.y[1])) return false;
  if (a.half > 0 && (!a.cos || !a.sin)) return false;
  for (int i = 0; i < (Hk > 0 ? 2 : 1); ++i)
    if (a.ts[i] < 0 || a.hs[i] < 0 || !product_fits(a.tokens, a.ts[i], 1) ||
        !product_fits(a.heads, a.hs[i], 1))
      return false;
  return true;
}

int head_blocks(const HeadArgs &a) {
  const int64_t want = ceil_div(a.tokens * a.heads, 8);
  return (int)(want < kBlocksMax ? want : kBlocksMax);
}

}  // namespace
}  // namespace seq
}  // namespace rlcs

using namespace rlcs;
using namespace rlcs::seq;

extern "C" {

rlcs_status rlcs_rope_table(float *cos, float *sin, int64_t max_pos, int64_t rotary_dim,
                            double base, rlcs_rope_scaling scaling, double factor,
                            double trained_len, double slow, double fast, double scale,
                            rlcs_stream_t stream) {
  if (!cos || !sin || max_pos <= 0 || rotary_dim <= 0 || rotary_dim % 2 != 0 ||
      !product_fits(max_pos, rotary_dim, 1) || !(base > 0.0) || !(scale > 0.0))
    return RLCS_ERR_INVALID_ARG;
  if (scaling != RLCS_ROPE_PLAIN && scaling != RLCS_ROPE_LINEAR && scaling != RLCS_ROPE_BASE &&
      scaling != RLCS_ROPE_PARTS)
    return RLCS_ERR_INVALID_ARG;
  if (scaling != RLCS_ROPE_PLAIN && !(factor > 0.0)) return RLCS_ERR_INVALID_ARG;
  if (scaling == RLCS_ROPE_BASE && rotary_dim <= 2) return RLCS_ERR_INVALID_ARG;
  if (scaling == RLCS_ROPE_PARTS && !(trained_len > 0.0 && fast > slow))
    return RLCS_ERR_INVALID_ARG;
  TableArgs a = {cos,  sin,    max_pos,     rotary_dim / 2, base,
                 factor, trained_len, slow, fast, scale, (int)scaling};
  const int64_t n = a.rows * a.half;
  if (ceil_div(n, 256) >= (int64_t)INT32_MAX) return RLCS_ERR_INVALID_ARG;
  const Range outs[] = {range(cos, n * 4), range(sin, n * 4)};
  const Range none[] = {range(nullptr, 0)};
  if (outputs_overlap(outs, none)) return RLCS_ERR_INVALID_ARG;
  return launched(launch_ex(rope_table_kernel, dim3((unsigned)ceil_div(n, 256)), dim3(256), 0,
                            reinterpret_cast<cudaStream_t>(stream), true, a));
}

rlcs_status rlcs_qk_norm_rope(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                              const void *k, int64_t k_token_stride, int64_t k_head_stride,
                              const float *q_weight, const float *k_weight, const float *cos,
                              const float *sin, const int32_t *positions, void *q_out,
                              void *k_out, int64_t tokens, int64_t Hq, int64_t Hk, int64_t D,
                              int64_t rotary_dim, int64_t max_pos, int interleaved, double eps,
                              rlcs_dtype dtype, rlcs_stream_t stream) {
  if (!head_sizes(tokens, Hq, Hk, D, rotary_dim, max_pos, eps, dtype)) return RLCS_ERR_INVALID_ARG;
  if (tokens == 0) return RLCS_OK;
  HeadArgs a = head_args(q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride,
                         q_weight, k_weight, cos, sin, positions, tokens, Hq, Hk, D, rotary_dim,
                         max_pos, interleaved, eps);
  a.y[0] = q_out;
  a.y[1] = k_out;
  if (!head_arrays(a, Hk)) return RLCS_ERR_INVALID_ARG;
  const int64_t e = esize(dtype);
  const Range none = range(nullptr, 0);
  const Range outs[] = {range(q_out, tokens * Hq * D * e),
                        Hk ? range(k_out, tokens * Hk * D * e) : none};
  const Range ins[] = {
      strided(q, tokens, q_token_stride, Hq, q_head_stride, D, e),
      Hk ? strided(k, tokens, k_token_stride, Hk, k_head_stride, D, e) : none,
      range(q_weight, D * 4),
      Hk ? range(k_weight, D * 4) : none,
      a.half ? range(cos, max_pos * a.half * 4) : none,
      a.half ? range(sin, max_pos * a.half * 4) : none,
      range(positions, tokens * 4)};
  if (outputs_overlap(outs, ins)) return RLCS_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return launched(dtype == RLCS_F32 ? launch_heads<float, false>(a, head_blocks(a), st)
                                    : launch_heads<__nv_bfloat16, false>(a, head_blocks(a), st));
}

size_t rlcs_qk_norm_rope_scratch_bytes(int64_t D) {
  return D <= 0 || D > 1024 ? 0 : (size_t)kBlocksMax * 2 * (size_t)D * sizeof(float);
}

rlcs_status rlcs_qk_norm_rope_backward(
    const void *dq_out, const void *dk_out, const void *q, int64_t q_token_stride,
    int64_t q_head_stride, const void *k, int64_t k_token_stride, int64_t k_head_stride,
    const float *q_weight, const float *k_weight, const float *cos, const float *sin,
    const int32_t *positions, void *dq, void *dk, float *dq_weight, float *dk_weight,
    int64_t tokens, int64_t Hq, int64_t Hk, int64_t D, int64_t rotary_dim, int64_t max_pos,
    int interleaved, double eps, rlcs_dtype dtype, void *scratch, size_t scratch_bytes,
    rlcs_stream_t stream) {
  if (!head_sizes(tokens, Hq, Hk, D, rotary_dim, max_pos, eps, dtype) || !dq_weight ||
      (Hk > 0 && !dk_weight))
    return RLCS_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (tokens == 0) {  // no rows: the weights' gradients are zero
    cudaError_t e = cudaMemsetAsync(dq_weight, 0, (size_t)D * 4, st);
    if (e == cudaSuccess && Hk > 0) e = cudaMemsetAsync(dk_weight, 0, (size_t)D * 4, st);
    return launched(e);
  }
  HeadArgs a = head_args(q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride,
                         q_weight, k_weight, cos, sin, positions, tokens, Hq, Hk, D, rotary_dim,
                         max_pos, interleaved, eps);
  a.dy[0] = dq_out;
  a.dy[1] = dk_out;
  a.y[0] = dq;
  a.y[1] = dk;
  if (!head_arrays(a, Hk) || !dq_out || (Hk > 0 && !dk_out)) return RLCS_ERR_INVALID_ARG;
  const int64_t e = esize(dtype), nq = tokens * Hq * D * e, nk = tokens * Hk * D * e;
  const Range none = range(nullptr, 0);
  const Range work = range(scratch, (int64_t)scratch_bytes);
  const Range outs[] = {range(dq, nq), Hk ? range(dk, nk) : none, range(dq_weight, D * 4),
                        Hk ? range(dk_weight, D * 4) : none, work};
  const Range ins[] = {
      range(dq_out, nq),
      Hk ? range(dk_out, nk) : none,
      strided(q, tokens, q_token_stride, Hq, q_head_stride, D, e),
      Hk ? strided(k, tokens, k_token_stride, Hk, k_head_stride, D, e) : none,
      range(q_weight, D * 4),
      Hk ? range(k_weight, D * 4) : none,
      a.half ? range(cos, max_pos * a.half * 4) : none,
      a.half ? range(sin, max_pos * a.half * 4) : none,
      range(positions, tokens * 4)};
  if (outputs_overlap(outs, ins)) return RLCS_ERR_INVALID_ARG;
  if (!scratch || scratch_bytes < rlcs_qk_norm_rope_scratch_bytes(D) || !aligned(scratch, 16))
    return RLCS_ERR_WORKSPACE;
  a.partial = static_cast<float *>(scratch);
  const int blocks = head_blocks(a);
  const rlcs_status s =
      launched(dtype == RLCS_F32 ? launch_heads<float, true>(a, blocks, st)
                                 : launch_heads<__nv_bfloat16, true>(a, blocks, st));
  if (s != RLCS_OK) return s;
  return launched(launch_ex(weight_sum_kernel, dim3((unsigned)ceil_div(2 * D, 32)), dim3(1024), 0,
                            st, true, (const float *)a.partial, blocks, (int)D, dq_weight,
                            Hk > 0 ? dk_weight : (float *)nullptr));
}

}  // extern "C"
