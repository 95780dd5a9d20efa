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
  bool tables16;  // the tables' rows start on 16-byte boundaries
  int q_blocks;   // head_pairs_kernel: blocks that take queries
  float eps, inv_d;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Any head width, stride and alignment: a warp per head, lanes over rotation
// pairs, then over the elements past the rotated ones. Its loads are of single
// elements and the head is read twice: 32768 tokens, 16 + 4 heads of 128, bf16,
// forward and gradient took 643 us through a kernel of this shape, 147 through
// the paired lanes below.
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

// ---------------------------------------------------------------------------
// Heads of 8 n elements up to 256: a lane holds 8 of a head's elements as
// four rotation pairs, so nothing but the mean crosses lanes. A group of D/8
// lanes takes a few heads of one token at a time, whose cosines and sines it
// reads once; the first blocks take queries and the rest keys, so a block has
// one weight vector and, in the gradient, one set of sums. Bound by memory: one
// read and one write of every head; 32768 tokens, 16 + 4 heads of 128, bf16,
// forward and gradient 147 us for 840 MB, 5.7 TB/s (a copy reaches 6.7).
// ---------------------------------------------------------------------------
// Four elements of a head, loaded and stored together.
template <class E>
struct Four;
template <>
struct Four<float> {
  float4 w;
  __device__ __forceinline__ void load(const float *p) {
    w = __ldg(reinterpret_cast<const float4 *>(p));
  }
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
  }
  static __device__ __forceinline__ void put(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Four<__nv_bfloat16> {
  uint2 w;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    w = __ldg(reinterpret_cast<const uint2 *>(p));
  }
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xffff0000u);
  }
  static __device__ __forceinline__ void put(__nv_bfloat16 *p, const float (&v)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  }
};

// A lane's 8 elements: the four first and the four second members of its
// pairs, each as two two-wide values.
struct Pairs {
  float2 a[2], b[2];
};
template <bool INTER, class E>
__device__ __forceinline__ Pairs unpack(const Four<E> &x, const Four<E> &y) {
  float u[4], v[4];
  x.get(u);
  y.get(v);
  if (INTER)  // (u0, u1), (u2, u3), (v0, v1), (v2, v3)
    return {{make_float2(u[0], u[2]), make_float2(v[0], v[2])},
            {make_float2(u[1], u[3]), make_float2(v[1], v[3])}};
  return {{make_float2(u[0], u[1]), make_float2(u[2], u[3])},
          {make_float2(v[0], v[1]), make_float2(v[2], v[3])}};
}
template <bool INTER, class E>
__device__ __forceinline__ void write(E *first, E *second, const Pairs &p) {
  const float u[4] = {p.a[0].x, INTER ? p.b[0].x : p.a[0].y, INTER ? p.a[0].y : p.a[1].x,
                      INTER ? p.b[0].y : p.a[1].y};
  const float v[4] = {INTER ? p.a[1].x : p.b[0].x, INTER ? p.b[1].x : p.b[0].y,
                      INTER ? p.a[1].y : p.b[1].x, p.b[1].y};
  Four<E>::put(first, u);
  Four<E>::put(second, v);
}
__device__ __forceinline__ float2 neg(float2 x) { return make_float2(-x.x, -x.y); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Sum over the group of lanes that starts at `first`; every lane gets it.
// LANES: the group's size where it is a power of two, else 0 (`lanes`).
template <int LANES>
__device__ __forceinline__ float group_sum(float v, int lanes, int first, int at) {
  if constexpr (LANES != 0) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float q = __shfl_down_sync(kFull, v, o);
      if (at < o && at + o < lanes) v += q;
    }
    return __shfl_sync(kFull, v, first);
  }
}

// Heads a group takes at a time, and blocks per SM the registers are held to.
// Measured on 32768 tokens, 16 + 4 heads of 128, bf16 (f32: 16384 tokens), us
// against floors of 50 forward and 75 backward:
//   forward  4 heads, 4 blocks 56 (f32 63); 4, 3 60 (53); 2, 4 62 (54); 1, 8 82 (61)
//   gradient 4, 2 97 (82); 2, 3 106 (88); 1, 4 115 (83); 1, 6 214 (163)
template <class E, bool BACK>
constexpr int slab_heads() {
  return BACK || sizeof(E) == 2 ? 4 : 2;
}

template <class E, bool INTER, int LANES, bool BACK>
__global__ void __launch_bounds__(256, BACK ? 2 : 4) head_pairs_kernel(const HeadArgs p) {
  constexpr int kSlab = slab_heads<E, BACK>();
  extern __shared__ float sums[];  // backward: [groups of a block][D]
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = LANES ? LANES : p.D / 8, per_warp = 32 / lanes;
  const int gi = lane / lanes, j = lane % lanes, first = gi * lanes;
  const bool live = gi < per_warp;
  const int which = (int)blockIdx.x >= p.q_blocks;
  const int block = which ? (int)blockIdx.x - p.q_blocks : (int)blockIdx.x;
  const int blocks = which ? (int)gridDim.x - p.q_blocks : p.q_blocks;
  const int heads = which ? (int)(p.heads - p.Hq) : (int)p.Hq;
  const int R = 2 * p.half;
  // this lane's two runs of four elements; its first pair is 4 j
  const bool turns = 4 * j < p.half;  // (half layout: the whole lane turns or not)
  const int ea = INTER ? 8 * j : (turns ? 4 * j : R + 8 * (j - R / 8));
  const int eb = INTER || !turns ? ea + 4 : ea + p.half;
  Pairs w = {}, g = {};  // weights, and the sums of their gradients
  if (live) {
    Four<float> wa, wb;
    const float *pw = p.w[which];
    wa.w = make_float4(pw[ea], pw[ea + 1], pw[ea + 2], pw[ea + 3]);
    wb.w = make_float4(pw[eb], pw[eb + 1], pw[eb + 2], pw[eb + 3]);
    w = unpack<INTER>(wa, wb);
  }
  const int slabs = (heads + kSlab - 1) / kSlab, total = (int)p.tokens * slabs;
  const int64_t ts = p.ts[which], hs = p.hs[which];
  const E *px = static_cast<const E *>(p.x[which]);
  const E *pdy = static_cast<const E *>(p.dy[which]);
  E *py = static_cast<E *>(p.y[which]);
  for (int base = (block * 8 + warp) * per_warp; base < total; base += blocks * 8 * per_warp) {
    const bool on = live && base + gi < total;
    const int tok = on ? (base + gi) / slabs : 0, h0 = on ? (base + gi) % slabs * kSlab : 0;
    Four<E> xa[kSlab], xb[kSlab], da[BACK ? kSlab : 1], db[BACK ? kSlab : 1];
    const E *x0 = px + tok * ts + h0 * hs;
    const int64_t at = ((int64_t)tok * heads + h0) * p.D;  // in the contiguous arrays
#pragma unroll
    for (int u = 0; u < kSlab; ++u)
      if (on && h0 + u < heads) {
        xa[u].load(x0 + u * hs + ea);
        xb[u].load(x0 + u * hs + eb);
        if constexpr (BACK) {
          da[u].load(pdy + at + u * p.D + ea);
          db[u].load(pdy + at + u * p.D + eb);
        }
      }
    float c[4], sn[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = 1.0f, sn[e] = 0.0f;
    if (on && turns) {
      const int64_t pos = p.positions[tok];
      const bool known_pos = pos >= 0 && pos < p.max_pos;
      const float *ct = p.cos + pos * p.half + 4 * j, *st = p.sin + pos * p.half + 4 * j;
      if (known_pos && p.tables16) {
        Four<float> a, b;
        a.load(ct);
        b.load(st);
        a.get(c);
        b.get(sn);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * j + e < p.half) {
            c[e] = known_pos ? __ldg(ct + e) : __int_as_float(0x7fffffff);
            sn[e] = known_pos ? __ldg(st + e) : c[e];
          }
      }
    }
    const float2 c2[2] = {make_float2(c[0], c[1]), make_float2(c[2], c[3])};
    const float2 s2[2] = {make_float2(sn[0], sn[1]), make_float2(sn[2], sn[3])};
#pragma unroll
    for (int u = 0; u < kSlab; ++u) {
      const bool use = on && h0 + u < heads;  // (groups of a warp can be at different slabs)
      const Pairs x = unpack<INTER>(xa[u], xb[u]);
      float2 q = __fmul2_rn(x.a[0], x.a[0]);
      q = __ffma2_rn(x.a[1], x.a[1], q);
      q = __ffma2_rn(x.b[0], x.b[0], q);
      q = __ffma2_rn(x.b[1], x.b[1], q);
      const float ss = group_sum<LANES>(use ? q.x + q.y : 0.0f, lanes, first, j);
      const float r = rsqrtf(ss * p.inv_d + p.eps);
      Pairs y;
      if constexpr (!BACK) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 ua = __fmul2_rn(__fmul2_rn(x.a[e], both(r)), w.a[e]);
          const float2 ub = __fmul2_rn(__fmul2_rn(x.b[e], both(r)), w.b[e]);
          y.a[e] = __ffma2_rn(neg(ub), s2[e], __fmul2_rn(ua, c2[e]));
          y.b[e] = __ffma2_rn(ua, s2[e], __fmul2_rn(ub, c2[e]));
        }
      } else {
        const Pairs d = unpack<INTER>(da[u], db[u]);
        Pairs t;
        float2 dot = both(0.0f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 ua = __ffma2_rn(d.b[e], s2[e], __fmul2_rn(d.a[e], c2[e]));
          const float2 ub = __ffma2_rn(neg(d.a[e]), s2[e], __fmul2_rn(d.b[e], c2[e]));
          if (use) {
            g.a[e] = __ffma2_rn(ua, __fmul2_rn(x.a[e], both(r)), g.a[e]);
            g.b[e] = __ffma2_rn(ub, __fmul2_rn(x.b[e], both(r)), g.b[e]);
          }
          t.a[e] = __fmul2_rn(ua, w.a[e]);
          t.b[e] = __fmul2_rn(ub, w.b[e]);
          dot = __ffma2_rn(t.a[e], x.a[e], dot);
          dot = __ffma2_rn(t.b[e], x.b[e], dot);
        }
        const float sum = group_sum<LANES>(use ? dot.x + dot.y : 0.0f, lanes, first, j);
        const float k = sum * r * r * p.inv_d;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          y.a[e] = __fmul2_rn(both(r), __ffma2_rn(x.a[e], both(-k), t.a[e]));
          y.b[e] = __fmul2_rn(both(r), __ffma2_rn(x.b[e], both(-k), t.b[e]));
        }
      }
      if (use) write<INTER>(py + at + u * p.D + ea, py + at + u * p.D + eb, y);
    }
  }
  if constexpr (BACK) {
    if (live) {
      float *mine = sums + (warp * per_warp + gi) * p.D;
      write<INTER>(mine + ea, mine + eb, g);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.D; i += 256) {
      float t = 0.0f;
      for (int k = 0; k < 8 * per_warp; ++k) t += sums[k * p.D + i];
      p.partial[(int64_t)blockIdx.x * p.D + i] = t;
    }
  }
}

// Sum the blocks' partial weight gradients in one fixed order, for the same bits
// every time: 3 us for 304 blocks and D = 128. Rows [0, split)
// of `partial` belong to the queries' weight and the rest to the keys', or,
// with split = 0, the two halves of every 2 D wide row.
__global__ void __launch_bounds__(1024)
    weight_sum_kernel(const float *partial, int blocks, int split, int D, float *dq, float *dk) {
  __shared__ float part[1024];
  pdl_wait();
  pdl_launch_dependents();
  const int i = blockIdx.x * 32 + (threadIdx.x & 31), row = threadIdx.x >> 5;
  const int which = i >= D, d = which ? i - D : i;
  const int64_t width = split ? D : 2 * D, col = split ? d : i;
  const int from = split && which ? split : 0, to = split && !which ? split : blocks;
  float t = 0.0f;
  if (i < 2 * D)
    for (int b = from + row; b < to; b += 32) t += partial[b * width + col];
  part[threadIdx.x] = t;
  __syncthreads();
  if (row == 0 && i < 2 * D) {
    for (int k = 1; k < 32; ++k) t += part[k * 32 + threadIdx.x];
    float *out = which ? dk : dq;
    if (out) out[d] = t;
  }
}

// Blocks of a call: the gradient's each leave a row of partial sums, so they
// are no more than run at once.
template <bool BACK>
constexpr int blocks_max() {
  return kSms * (BACK ? 2 : 8);
}

bool head_sizes(int64_t tokens, int64_t Hq, int64_t Hk, int64_t D, int64_t R, int64_t max_pos,
                double eps, rlcs_dtype t) {
  return tokens >= 0 && Hq > 0 && Hk >= 0 && D > 0 && D <= 1024 && R >= 0 && R <= D && R % 2 == 0 &&
         max_pos >= 0 && eps >= 0.0 && known(t) && Hq <= INT32_MAX && Hk <= INT32_MAX &&
         product_fits(tokens, Hq + Hk, D) && product_fits(max_pos, D, 1);
}

// Whether a call can take the paired lanes: whole runs of four elements, each
// loaded together, that rotation pairs do not straddle.
template <class E>
bool pairs_fit(const HeadArgs &a, int Hk) {
  const int R = 2 * a.half;
  if (a.D % 8 || a.D > 256 || (!a.inter && R % 8) || a.tokens * a.heads >= (int64_t)INT32_MAX / 2)
    return false;
  const uintptr_t run = 4 * sizeof(E);
  for (int i = 0; i < (Hk > 0 ? 2 : 1); ++i)
    if (a.ts[i] % 4 || a.hs[i] % 4 || !aligned(a.x[i], run) || !aligned(a.y[i], run) ||
        !aligned(a.dy[i], run))
      return false;
  return true;
}

// Blocks of the queries' and the keys' heads, each leaving one row of partial
// weight gradients: as many as their slabs need, within `most` together.
template <class E, int LANES, bool BACK>
cudaError_t launch_pairs(HeadArgs &a, int &blocks, cudaStream_t st) {
  constexpr int kSlab = slab_heads<E, BACK>();
  const int per_block = 8 * (32 / (a.D / 8)), Hq = (int)a.Hq, Hk = (int)a.heads - Hq;
  const int64_t nq = ceil_div(a.tokens * ceil_div(Hq, kSlab), per_block);
  const int64_t nk = ceil_div(a.tokens * ceil_div(Hk, kSlab), per_block);
  constexpr int kMost = blocks_max<BACK>();
  if (nq + nk <= kMost) {
    a.q_blocks = (int)nq;
    blocks = (int)(nq + nk);
  } else {
    int64_t k = nk * kMost / (nq + nk);
    if (Hk > 0 && k == 0) k = 1;
    a.q_blocks = (int)(kMost - k);
    blocks = kMost;
  }
  a.tables16 = a.half % 4 == 0 && aligned(a.cos, 16) && aligned(a.sin, 16);
  const size_t smem = BACK ? (size_t)per_block * a.D * sizeof(float) : 0;  // 8 KB
  return a.inter ? launch_ex(head_pairs_kernel<E, true, LANES, BACK>, dim3((unsigned)blocks),
                             dim3(256), smem, st, true, a)
                 : launch_ex(head_pairs_kernel<E, false, LANES, BACK>, dim3((unsigned)blocks),
                             dim3(256), smem, st, true, a);
}

template <class E, bool BACK>
cudaError_t launch_heads(HeadArgs &a, int &blocks, cudaStream_t st) {
  a.q_blocks = 0;
  if (pairs_fit<E>(a, (int)(a.heads - a.Hq))) {
    if (a.D == 128) return launch_pairs<E, 16, BACK>(a, blocks, st);
    if (a.D == 64) return launch_pairs<E, 8, BACK>(a, blocks, st);
    return launch_pairs<E, 0, BACK>(a, blocks, st);
  }
  const int64_t want = ceil_div(a.tokens * a.heads, 8);
  blocks = (int)(want < blocks_max<BACK>() ? want : blocks_max<BACK>());
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
  int blocks;
  return launched(dtype == RLCS_F32 ? launch_heads<float, false>(a, blocks, st)
                                    : launch_heads<__nv_bfloat16, false>(a, blocks, st));
}

size_t rlcs_qk_norm_rope_scratch_bytes(int64_t D) {
  return D <= 0 || D > 1024 ? 0 : (size_t)blocks_max<true>() * 2 * (size_t)D * sizeof(float);
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
    if (e == cudaSuccess && dk_weight) e = cudaMemsetAsync(dk_weight, 0, (size_t)D * 4, st);
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
                        range(dk_weight, D * 4), work};
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
  int blocks = 0;
  const rlcs_status s =
      launched(dtype == RLCS_F32 ? launch_heads<float, true>(a, blocks, st)
                                 : launch_heads<__nv_bfloat16, true>(a, blocks, st));
  if (s != RLCS_OK) return s;
  return launched(launch_ex(weight_sum_kernel, dim3((unsigned)ceil_div(2 * D, 32)), dim3(1024), 0,
                            st, true, (const float *)a.partial, blocks, a.q_blocks, (int)D, dq_weight,
                            dk_weight));
}

}  // extern "C"
