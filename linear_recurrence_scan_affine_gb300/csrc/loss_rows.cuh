// Rows of logits (rlcs_loss.h): what the two losses share. A row's statistics,
// its words in registers, the teams and blocks that hold rows, and the checks
// of the arguments that both take.
//
// With m near c times the row's largest logit, c = log2(e) / T, and in base 2,
//   y_i = c x_i - m,   e_i = 2^y_i,   z = sum e_i,
// a row's distribution is p_i = e_i / z with log p_i = y_i ln 2 - log z, and
// both gradients are e_i (A + B y_i) plus terms at a few named elements. y is
// one fused multiply and add, rounded once at its own size: a common offset of
// the logits costs no digits. (What m is rounded by is in every y alike: 1/2 at
// most up to c top = 2^24, 32 at 2^30, where logits differ by half a power of
// two and more and an entropy is off by up to 2^-17. For rows yet further from 0
// see Base.)
#pragma once

#include <type_traits>

#include "rlcs_loss.h"
#include "seq_common.cuh"
#include "tensor_core.cuh"

namespace rlcs {
namespace loss {

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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float value(const float *p) { return *p; }
__device__ __forceinline__ float value(const bf *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(bf *p, float v) { *p = __float2bfloat16_rn(v); }

// What y is formed with. In a row with c top above 2^30 logits differ by nothing
// or by 64 powers of two and more, so that only its largest count, and c may be
// any larger number: a power of two, which rounds no product with top, or 1 where
// that would pass float32's range. A row (or part of one) with nothing above
// -infinity has e = 0.
struct Base {
  float c, m;
  __device__ __forceinline__ float y(float x) const { return fmaf(x, c, -m); }
};
constexpr float kFar = 1073741824.0f;
__device__ __forceinline__ Base base_of(float top, float c) {
  const float m = top * c;
  if (__builtin_expect(fabsf(m) <= kFar, true)) return {c, m};
  if (top == -INFINITY) return {c, 0.0f};
  const float power = __int_as_float((__float_as_int(c) + 0x7fffff) & 0x7f800000);
  const float other = fabsf(m) <= 1e38f ? power : 1.0f;
  return {other, top * other};
}
// A y of 1 in natural logarithms (base.c is c, or a power of two).
__device__ __forceinline__ float log_of_2(const Base &base, float c) {
  if (__builtin_expect(base.c == c, true)) return kLn2;
  return kLn2 * c * __int_as_float(0x7f000000 - __float_as_int(base.c));
}
// A row's statistics: its largest logit, z and sum e y.
struct Stats {
  float top, z, t;
};
// y where it multiplies e: -infinity and what underflows far below 2^-149
// add nothing
__device__ __forceinline__ float bounded(float y) { return fmaxf(y, -200.0f); }
// How far (in base 2) a part's base lies below the whole's.
__device__ __forceinline__ float below(float part, float whole, float c) {
  const float a = part * c, b = whole * c;
  if (__builtin_expect(fabsf(a) <= kFar && fabsf(b) <= kFar, true)) return a - b;
  if (part == whole) return 0.0f;
  // (a part whose e are all 0 is as far as can be)
  return fabsf(a) <= kFar ? fmaf(-whole, c, a)
                          : (fabsf(b) <= kFar ? fmaf(part, c, -b) : (part - whole) * c);
}

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

struct Coefficients {
  float a, b;  // dx_i = e_i (a + b y_i)
};

// ---------------------------------------------------------------------------
// Rows on chip: a team of threads holds a row in registers, as 16-byte words
// of the array. Lane l of the team has words l, l + TEAM, ... A row may start
// and end inside a word; what is not the row's is taken for -infinity, which
// adds nothing.
// ---------------------------------------------------------------------------
template <class T>
constexpr int kWord = 16 / sizeof(T);  // elements
template <class T>
constexpr uint32_t kNothing = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -infinity

__device__ __forceinline__ uint4 nothing(uint32_t w) { return make_uint4(w, w, w, w); }
// A word into its registers where `on`, -infinity otherwise. No branch and no
// other register stands between a load and its use, or each load would be
// waited for before the next is issued. Streamed: a row is read once.
__device__ __forceinline__ void load_word(uint4 &q, const void *p, bool on, uint32_t none) {
  q = nothing(none);
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "+r"(q.x), "+r"(q.y), "+r"(q.z), "+r"(q.w)
      : "l"(p), "r"((uint32_t)on)
      : "memory");
}

// Elements of a word in float32, as pairs.
__device__ __forceinline__ void unpack(const uint4 &q, float2 (&x)[2], const float *) {
  x[0] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
  x[1] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
}
__device__ __forceinline__ void unpack(const uint4 &q, float2 (&x)[4], const bf *) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack(const float2 (&x)[2], const float *) {
  return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                    __float_as_uint(x[1].y));
}
__device__ __forceinline__ uint4 pack(const float2 (&x)[4], const bf *) {
  return make_uint4(seq::pack_bf16(x[0].x, x[0].y), seq::pack_bf16(x[1].x, x[1].y),
                    seq::pack_bf16(x[2].x, x[2].y), seq::pack_bf16(x[3].x, x[3].y));
}
// (a NaN is left to the sums, which it enters)
__device__ __forceinline__ float word_max(const uint4 &q, const float *) {
  return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)),
               fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
}
__device__ __forceinline__ float word_max(const uint4 &q, const bf *) {
  const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&q);
  const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
  return fmaxf(__bfloat162float(m.x), __bfloat162float(m.y));
}

// A row as one thread of a team of TEAM sees it: word w0 + n TEAM is its word
// n. Counted in words from the one that the row starts in, its first `skip`
// elements another row's (or nothing's). Word n is the thread's where n TEAM <
// left, and lies inside the array where n TEAM < inside, but for the first.
template <class T>
struct Row {
  const char *at;  // the thread's first word
  int w0, skip;
  int left, inside;
  bool out;        // the thread's first word starts before the array
  __device__ __forceinline__ bool mine(int offset) const { return offset < left; }
  __device__ __forceinline__ bool loads(int offset) const {
    return offset < inside && (offset > 0 || !out);
  }
};
// `lane` of a team of blocks: rank of ranks, each with an equal run of words.
template <class T, class Args>
__device__ __forceinline__ Row<T> row_of(const Args &p, int64_t row, int lane, int rank,
                                         int ranks) {
  const T *x = static_cast<const T *>(p.logits) + row * p.row_stride;
  Row<T> r;
  r.skip = (int)(reinterpret_cast<uintptr_t>(x) % 16) / (int)sizeof(T);
  const int count = ((int)p.V + r.skip + kWord<T> - 1) / kWord<T>;
  const int run = ranks == 1 ? count : (count + ranks - 1) / ranks, from = rank * run;
  const int to = from + run < count ? from + run : count;
  r.w0 = from + lane;
  r.at = reinterpret_cast<const char *>(x - r.skip) + (int64_t)r.w0 * 16;
  r.left = to - r.w0;
  // words from the row's first to the array's end
  const int64_t after =
      ((p.tokens - 1 - row) * p.row_stride + p.V + r.skip) * (int64_t)sizeof(T) / 16;
  r.inside = (after < to ? (int)after : to) - r.w0;
  r.out = r.w0 == 0 && row * p.row_stride < r.skip;
  return r;
}
// A word that reaches out of the array, element by element.
template <class T>
__device__ __noinline__ uint4 load_edge(const T *x, int skip, int64_t V, int w) {
  uint4 q = nothing(kNothing<T>);
  T *e = reinterpret_cast<T *>(&q);
  for (int i = 0; i < kWord<T>; ++i) {
    const int64_t c = (int64_t)w * kWord<T> + i - skip;
    if (c >= 0 && c < V) e[i] = x[c];
  }
  return q;
}
// -infinity in place of what of word w is not the row's.
template <class T>
__device__ __forceinline__ void trim(uint4 &q, int w, int skip, int last) {
  const int lo = w == 0 ? skip : 0, hi = last - w * kWord<T>;
  uint32_t *r = reinterpret_cast<uint32_t *>(&q);
#pragma unroll
  for (int i = 0; i < kWord<T>; ++i)
    if (i < lo || i >= hi) {
      if (sizeof(T) == 4)
        r[i] = kNothing<T>;
      else
        r[i / 2] = i % 2 ? (r[i / 2] & 0xffffu) | 0xff800000u : (r[i / 2] & 0xffff0000u) | 0xff80u;
    }
}
// A word of the gradient that is not stored whole.
template <class T>
__device__ __noinline__ void store_edge(T *dx, int skip, int64_t V, int w, uint4 q) {
  const T *e = reinterpret_cast<const T *>(&q);
#pragma unroll
  for (int i = 0; i < kWord<T>; ++i) {
    const int64_t c = (int64_t)w * kWord<T> + i - skip;
    if (c >= 0 && c < V) dx[c] = e[i];
  }
}

// Sums over part of a row with the threads of a team or, where blocks are the
// teams, of one warp: the largest element first, then the sums relative to it.
template <int LANES>
__device__ __forceinline__ float lanes_max(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
  return x;
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}
// The statistics of a whole from those of LANES parts, one to a lane. Parts
// without anything above -infinity have z = 0.
template <int LANES, bool ENTROPY>
__device__ __forceinline__ Stats join(Stats s, float c) {
  const float top = lanes_max<LANES>(s.top);
  const float d = bounded(below(s.top, top, c)), f = ex2(d);
  if (ENTROPY) s.t = f * fmaf(s.z, d, s.t);
  return {top, lanes_sum<LANES>(f * s.z), ENTROPY ? lanes_sum<LANES>(s.t) : 0.0f};
}

// `used`: words that hold anything, the same for the whole warp.
template <class T, int TEAM, int NV, bool ENTROPY>
__device__ __forceinline__ Stats lanes_stats(const uint4 (&q)[NV], float c, int used) {
  constexpr int LANES = TEAM < 32 ? TEAM : 32, P = kWord<T> / 2;
  const T *type = nullptr;
  float m = word_max(q[0], type);
#pragma unroll
  for (int n = 1; n < NV; ++n) m = fmaxf(m, word_max(q[n], type));
  m = lanes_max<LANES>(m);
  const Base base = base_of(m, c);
  const float2 nb = make_float2(-base.m, -base.m), c2 = make_float2(base.c, base.c);
  // Sums of e y come without bounds on y first: only a logit of -infinity, and
  // a row that has no distribution, make them NaN.
  float z, t;
  const auto sums = [&](auto bound) {
    float2 z2 = make_float2(0.0f, 0.0f), t2 = z2;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      if (n >= used) break;
      float2 x[P];
      unpack(q[n], x, type);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float2 y = __ffma2_rn(x[i], c2, nb);
        const float2 e = make_float2(ex2(y.x), ex2(y.y));
        z2 = __fadd2_rn(z2, e);
        if (ENTROPY) {
          if (decltype(bound)::value) y = make_float2(bounded(y.x), bounded(y.y));
          t2 = __ffma2_rn(e, y, t2);
        }
      }
    }
    z = lanes_sum<LANES>(z2.x + z2.y);
    t = ENTROPY ? lanes_sum<LANES>(t2.x + t2.y) : 0.0f;
  };
  if (ENTROPY && TEAM > 32) {
    sums(std::false_type());
    if (t != t) sums(std::true_type());
  } else {
    sums(std::true_type());
  }
  return {m, z, t};
}

template <class T, int TEAM, int NV>
__device__ __forceinline__ void load_row(uint4 (&q)[NV], const Row<T> &r, bool on) {
#pragma unroll
  for (int n = 0; n < NV; ++n)
    load_word(q[n], r.at + n * TEAM * 16, on && r.loads(n * TEAM), kNothing<T>);
}
// The row's first and last word, where it shares them with something else.
template <class T, int TEAM, int NV, class Args>
__device__ __forceinline__ void trim_row(uint4 (&q)[NV], const Args &p, int64_t row,
                                         const Row<T> &r) {
  const int last = (int)p.V + r.skip;
  if (r.skip == 0 && last % kWord<T> == 0) return;
  const int to_last = (last - 1) / kWord<T> - r.w0;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    if (!r.mine(n * TEAM) || (r.w0 + n * TEAM != 0 && n * TEAM != to_last)) continue;
    const int w = r.w0 + n * TEAM;
    if (!r.loads(n * TEAM))
      q[n] = load_edge(static_cast<const T *>(p.logits) + row * p.row_stride, r.skip, p.V, w);
    trim<T>(q[n], w, r.skip, last);
  }
}

// dx = e (a + b y) of one word
template <class T, bool ENTROPY>
__device__ __forceinline__ void gradient(const uint4 &q, float2 (&d)[kWord<T> / 2], Base base,
                                         Coefficients k) {
  const T *type = nullptr;
  unpack(q, d, type);
  const float2 nb = make_float2(-base.m, -base.m), c2 = make_float2(base.c, base.c),
               a2 = make_float2(k.a, k.a);
#pragma unroll
  for (int i = 0; i < kWord<T> / 2; ++i) {
    float2 y = __ffma2_rn(d[i], c2, nb);
    const float2 e = make_float2(ex2(y.x), ex2(y.y));
    if (ENTROPY) {
      y = make_float2(bounded(y.x), bounded(y.y));
      d[i] = __fmul2_rn(e, __ffma2_rn(make_float2(k.b, k.b), y, a2));
    } else {
      d[i] = __fmul2_rn(e, a2);
    }
  }
}

// A row's gradient. Words are stored whole where its row starts as far into a
// word as that of the logits does. `then(n)` follows each word.
struct Nothing {
  __device__ __forceinline__ void operator()(int) const {}
};
template <class T, bool GRAD, int TEAM, int NV, bool ON, bool ENTROPY, class Fix,
          class Then = Nothing>
__device__ __forceinline__ void store_row(uint4 (&q)[NV], const Row<T> &r, Base base,
                                          Coefficients k, T *dx, int64_t V, Fix fix,
                                          Then then = Then()) {
  const bool alike = reinterpret_cast<uintptr_t>(dx) % 16 == (uintptr_t)(r.skip * sizeof(T));
  const int full = alike ? ((int)V + r.skip) / kWord<T> - r.w0 : 0;  // words stored whole
  const bool part = r.w0 == 0 && r.skip != 0;                        // but for the first
  char *to = reinterpret_cast<char *>(dx - r.skip) + (int64_t)r.w0 * 16;
  const T *type = nullptr;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    if (GRAD && r.mine(n * TEAM)) {
      uint4 o = make_uint4(0, 0, 0, 0);
      if (ON) {
        float2 d[kWord<T> / 2];
        gradient<T, ENTROPY>(q[n], d, base, k);
        fix(d, n * TEAM);
        o = pack(d, type);
      }
      if (n * TEAM < full && (n > 0 || !part))
        __stcs(reinterpret_cast<uint4 *>(to + n * TEAM * 16), o);
      else
        store_edge(dx, r.skip, V, r.w0 + n * TEAM, o);
    }
    then(n);
  }
}
// The same, and the next row's words are asked for as this row's are used up,
// so that copies in run beside copies out.
template <class T, bool GRAD, int TEAM, int NV, bool ON, bool ENTROPY, class Fix>
__device__ __forceinline__ void use_row(uint4 (&q)[NV], const Row<T> &r, Base base, Coefficients k,
                                        const Row<T> &next, bool more, T *dx, int64_t V, Fix fix) {
  store_row<T, GRAD, TEAM, NV, ON, ENTROPY>(q, r, base, k, dx, V, fix, [&](int n) {
    load_word(q[n], next.at + n * TEAM * 16, more && next.loads(n * TEAM), kNothing<T>);
  });
}

// ---------------------------------------------------------------------------
// Short rows: a warp, or eight lanes of one, to a row
// ---------------------------------------------------------------------------
constexpr int kTeamBlock = 128;
constexpr int team_blocks(int nv) { return nv >= 8 ? 5 : (nv == 4 ? 6 : 8); }  // to an SM

// ---------------------------------------------------------------------------
// The shortest rows: a thread to each, 256 rows of a block together in shared
// memory, so that what is copied in and out is whole. A row is `pitch` words
// apart, odd, so that a warp's threads meet no bank twice.
// ---------------------------------------------------------------------------
constexpr int kFew = 32, kFewBlock = 256;  // elements of a row at most; rows to a block

// Copies between the block's rows and shared memory, an element to a thread in
// the arrays' order; rows that are left out (of the copy in) are not read.
template <class T, bool IN, class Args, class On>
__device__ __forceinline__ void few_copy(const Args &p, T *dx, float *x, int rows, int64_t row0,
                                         int pitch, On on) {
  const int V = (int)p.V, n = rows * V;
  int row = threadIdx.x / V, col = threadIdx.x % V;
  const int drow = kFewBlock / V, dcol = kFewBlock % V;
  for (int i = threadIdx.x; i < n; i += kFewBlock) {
    if (IN) {
      if (on(row))
        x[row * pitch + col] =
            value(static_cast<const T *>(p.logits) + (row0 + row) * p.row_stride + col);
    } else {
      put(dx + row0 * V + i, x[row * pitch + col]);
    }
    row += drow;
    col += dcol;
    if (col >= V) col -= V, ++row;
  }
}
template <bool ENTROPY>
__device__ __forceinline__ Stats few_stats(const float *x, int V, float c) {
  float top = x[0];
  for (int i = 1; i < V; ++i) top = fmaxf(top, x[i]);
  const Base base = base_of(top, c);
  Stats s = {top, 0.0f, 0.0f};
  for (int i = 0; i < V; ++i) {
    const float y = base.y(x[i]), e = ex2(y);
    s.z += e;
    if (ENTROPY) s.t = fmaf(e, bounded(y), s.t);
  }
  return s;
}

// ---------------------------------------------------------------------------
// Long rows: blocks of 8 warps that hold a row's words, or of a cluster of
// blocks that share them, and one warp that leads. The leader takes what a
// token has besides its logits, joins the statistics, works out the
// coefficients of the gradient, and fetches the next row; the others wait for
// nothing but their words and those coefficients. What a teacher adds to a
// token takes as long as a row does: one more warp works on it, a row ahead.
//
// The grid has a block (or cluster) to each row, but one that is done takes a
// row whose block has not started yet, by cancelling that block: rows that the
// mask leaves out cost little, and a fixed assignment would leave some blocks
// with a fifth more work than others.
//
// The next row's words come into shared memory, by one bulk copy, while this
// row's are worked on in registers. Policy loss and gradient of 16384 x 32768
// bfloat16, a quarter masked: 307 us, 6.1 TB/s, 0.91 of the copy rate (326 with
// loads to registers as these were used up; 391 with fixed rows, 16 warps of half
// as many words and no leader, where every warp worked out every row's scalars).
// Distillation over 4096 x 131072 bfloat16, 64 entries, four blocks to a row: 390
// us, 5.5 TB/s (453 without the teacher's warp).
// ---------------------------------------------------------------------------
constexpr int kTeam = 256, kLongBlock = kTeam + 32, kMaxRanks = 8;
constexpr int long_blocks(int nv) { return nv >= 16 ? 2 : (nv == 8 ? 3 : 4); }  // to an SM

struct LongSmem {
  alignas(16) uint4 answer[2];      // of the requests for a row
  alignas(16) float4 ranks[2][kMaxRanks];  // top, z, t of each block of the cluster
  Stats warps[2][kTeam / 32];
  Coefficients k;
  float gain;      // added at element `element` of word `word`
  int word, element;
  Stats whole;
  int on;          // whether the row has a gradient
  // The next row, or past the last, and whether it has one. By turns: the
  // others read a row's when the leader may be at the row after.
  int64_t next[2];
  int more[2];
  uint64_t asked[2], told[2], full;  // barriers: an answer, the ranks' statistics, a row's words
  int abort;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Named barriers between the leader's warp and the others, or some of them.
template <int THREADS = kLongBlock>
__device__ __forceinline__ void meet_arrive(int id) {
  __syncwarp();
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}
template <int THREADS = kLongBlock>
__device__ __forceinline__ void meet_wait(int id) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}
// Rows take turns with the first three pairs: where no gradient is formed the
// leader and the others are up to a row apart, either way.
constexpr int kSummed = 1, kTaken = 3, kPlanned = 5, kStored = 7, kTaught = 8;

// Four numbers into another block's shared memory, counted on its barrier.
__device__ __forceinline__ void tell(const float4 *place, const uint64_t *bar, uint32_t rank,
                                     const float4 &v) {
  uint32_t there, mbar;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(there)
               : "r"(tc::smem_addr(place)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(mbar)
               : "r"(tc::smem_addr(bar)), "r"(rank));
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, "
      "[%5];" ::"r"(there),
      "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(mbar)
      : "memory");
}

// The end of a block one of whose waits ran out, by its leader's warp: copies under
// way arrive, and while other blocks of the cluster still write to its shared
// memory it stays. (A cluster's barrier opens when all threads that have not ended
// are there; what the others wait for before they end has limits.) Every other
// block has had all that is sent to it when it ends. (With __nanosleep in the loop,
// never run, 4096 x 131072 with a teacher took 405 us for 392.)
__device__ __forceinline__ void settle(int ranks) {
  const uint64_t until = globaltimer_ns() + 2000000;
  while (globaltimer_ns() < until) {
  }
  __syncwarp();
  if (ranks == 1) return;
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// What a loss adds, each call by a whole warp. The leader:
//   ahead(next, more)  ask for a token's own numbers, a row ahead
//   before(next, more) what of them does not need the row's statistics
//   held()             once all that this block reads of the row apart from its
//                      words has been read: a number that is sent with the
//                      statistics, after which others may write over the row
//   plan(...)          the gradient's coefficients, into shared memory
// With kTeacher one more warp runs teach(), from a row's plan to the next's.
template <class T, bool GRAD, int NV, bool ENTROPY, class Leader, class Args>
__device__ __forceinline__ void long_rows(const Args &p, float c, uint32_t *status,
                                          Leader &leader) {
  constexpr int kPlan = kLongBlock + (Leader::kTeacher ? 32 : 0);  // who meets at a plan
  // Without a gradient the others need to know the next row alone.
  constexpr bool kEarly = !GRAD && !Leader::kTeacher;
  extern __shared__ __align__(128) unsigned char dynamic[];
  uint4 *words = reinterpret_cast<uint4 *>(dynamic);  // of the next row
  __shared__ LongSmem sm;
  const int lane = threadIdx.x & 31, warp = __shfl_sync(kFull, threadIdx.x >> 5, 0);
  const int ranks = (int)cluster_size(), rank = (int)cluster_rank();
  if (threadIdx.x == 0) {
    for (uint64_t *b : {&sm.asked[0], &sm.asked[1], &sm.told[0], &sm.told[1], &sm.full})
      mbar_init(b, 1);
    sm.abort = 0;
    fence_mbar_init();
  }
  if (ranks > 1) {  // every block has started before another writes to it
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  int64_t row = (int)blockIdx.x / ranks;
  const auto live = [&](int64_t i) { return i < p.tokens && (!p.mask || p.mask[i]); };
  bool on = live(row);

  if (warp == kTeam / 32) {  // the leader
    volatile int *abort = &sm.abort;
    const auto request = [&](int i) {
      if (lane == 0) {
        fence_proxy_async_shared();
        mbar_arrive_expect_tx(&sm.asked[i & 1], 16);
        if (rank == 0) tc::ask(&sm.answer[i & 1], &sm.asked[i & 1], ranks > 1);
      }
      __syncwarp();
    };
    // a row's words into shared memory, those that lie inside the array
    const auto fetch = [&](int64_t i) {
      if (lane == 0) {
        const Row<T> r = row_of<T>(p, i, 0, rank, ranks);
        const int lo = r.out ? 1 : 0, n = r.inside - lo;
        fence_proxy_async_shared();
        mbar_arrive_expect_tx(&sm.full, n > 0 ? n * 16 : 0);
        if (n > 0) bulk_g2s(words + lo, r.at + lo * 16, n * 16, &sm.full);
      }
      __syncwarp();
    };
    request(0);
    if (on) fetch(row);
    leader.ahead(row, on);
    leader.before(row, on);
    for (int i = 0; row < p.tokens; ++i) {
      const int turn = i & 1;
      // the next row: asked for a row ago
      int64_t next = p.tokens;
      if (tc::warp_wait(&sm.asked[turn], (i >> 1) & 1, abort)) {
        const int64_t block = tc::granted(&sm.answer[turn]);
        if (block >= 0) next = block / ranks;
      }
      const bool more = live(next);
      if (lane == 0) sm.next[turn] = next, sm.more[turn] = more;
      if (kEarly) meet_arrive<kPlan>(kPlanned + turn);
      leader.ahead(next, more);
      if (on) meet_wait(kTaken + turn);  // the words of this row are in registers
      if (more) fetch(next);
      Stats s = {-INFINITY, 0.0f, 0.0f};
      meet_wait(kSummed + turn);
      if (on) s = join<kTeam / 32, ENTROPY>(sm.warps[turn][lane % (kTeam / 32)], c);
      const float held = leader.held();
      if (ranks > 1) {
        // A set is told again two rows later, which no block comes to before
        // all have told the row between, and so have read this one.
        if (lane == 0) mbar_arrive_expect_tx(&sm.told[turn], 16 * ranks);
        __syncwarp();
        if (lane < ranks)
          tell(&sm.ranks[turn][rank], &sm.told[turn], lane,
               make_float4(s.top, s.z, s.t, held));
        tc::warp_wait(&sm.told[turn], (i >> 1) & 1, abort);
        float4 v = sm.ranks[turn][lane & (ranks - 1)];
        if (lane % kMaxRanks >= ranks) v.y = v.z = 0.0f;  // (a part of nothing)
        s = join<kMaxRanks, ENTROPY>({v.x, v.y, v.z}, c);
      }
      // every block of the cluster has read the answer by now
      if (next < p.tokens) request(i + 1);
      leader.plan(row, s, on, rank, sm);
      if (lane == 0) sm.whole = s;
      if (!kEarly) meet_arrive<kPlan>(kPlanned + turn);
      leader.before(next, more);
      row = next;
      on = more;
    }
    if (*abort) {
      if (lane == 0) atomicMax(status, (uint32_t)RLCS_ERR_TIMEOUT);
      settle(ranks);
    }
    return;
  }

  if (Leader::kTeacher && warp == kTeam / 32 + 1) {
    leader.teach(row, on, rank, ranks, sm);
    return;
  }

  uint4 q[NV];
  Row<T> r = row_of<T>(p, row, threadIdx.x, rank, ranks);
  uint32_t phase = 0;
  for (int i = 0; row < p.tokens; ++i) {
    const int turn = i & 1;
    if (on) {
      tc::warp_wait(&sm.full, phase, &sm.abort);
      phase ^= 1;
#pragma unroll
      for (int n = 0; n < NV; ++n)
        q[n] = r.loads(n * kTeam) ? words[threadIdx.x + n * kTeam] : nothing(kNothing<T>);
      meet_arrive(kTaken + turn);
      trim_row<T, kTeam, NV>(q, p, row, r);
      const int mine = r.left + lane;  // words of the run from this warp's first on
      const int used = mine <= 0 ? 0 : (mine + kTeam - 1) / kTeam;
      const Stats s = lanes_stats<T, kTeam, NV, ENTROPY>(q, c, used);
      if (lane == 0) sm.warps[turn][warp] = s;
    }
    meet_arrive(kSummed + turn);
    meet_wait<kPlan>(kPlanned + turn);
    const int64_t next = sm.next[turn];
    const bool more = sm.more[turn];
    T *dx = GRAD ? static_cast<T *>(p.dlogits) + row * p.V : nullptr;
    if (!GRAD) {
    } else if (on && sm.on) {
      const Coefficients k = sm.k;
      const Base base = base_of(sm.whole.top, c);
      const int offset = sm.word - r.w0;
      const auto fix = [&](float2(&d)[kWord<T> / 2], int n) {
        if (n != offset) return;
        const int element = sm.element;
#pragma unroll
        for (int i = 0; i < kWord<T>; ++i)
          if (i == element) (i % 2 ? d[i / 2].y : d[i / 2].x) += sm.gain;
      };
      if (ENTROPY && k.b != 0.0f)
        store_row<T, GRAD, kTeam, NV, true, ENTROPY>(q, r, base, k, dx, p.V, fix);
      else
        store_row<T, GRAD, kTeam, NV, true, false>(q, r, base, k, dx, p.V, fix);
    } else {
      store_row<T, GRAD, kTeam, NV, false, false>(q, r, {0.0f, 0.0f}, {0.0f, 0.0f}, dx, p.V,
                                                  [](float2(&)[kWord<T> / 2], int) {});
    }
    if (Leader::kTeacher && GRAD) meet_arrive(kStored);
    row = next;
    r = row_of<T>(p, row < p.tokens ? row : 0, threadIdx.x, rank, ranks);
    on = more;
  }
}

// ---------------------------------------------------------------------------
// Rows longer than a cluster holds: a block to a row, read twice
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
  Stats s = {-INFINITY, 0.0f, 0.0f};
  Base base = base_of(s.top, c);
  for (int64_t i = threadIdx.x; i < V; i += kThreads) {
    const float v = value(x + i);
    if (v > s.top) {  // rescale what was summed so far
      const float d = bounded(below(s.top, v, c)), f = ex2(d);
      if (ENTROPY) s.t = f * fmaf(s.z, d, s.t);
      s.z *= f;
      s.top = v;
      base = base_of(v, c);
    }
    const float y = base.y(v), e = ex2(y);
    s.z += e;
    if (ENTROPY) s.t = fmaf(e, bounded(y), s.t);
  }
  const float top = block_max(s.top, part);
  const float d = bounded(below(s.top, top, c)), f = ex2(d);
  if (ENTROPY) s.t = f * fmaf(s.z, d, s.t);
  return {top, block_sum(f * s.z, part), ENTROPY ? block_sum(s.t, part) : 0.0f};
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

// What calls have recorded since this was last asked.
inline rlcs_status take_status(const void *symbol) {
  uint32_t code = 0;
  const uint32_t none = 0;
  if (cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpyFromSymbol(&code, symbol, sizeof(code)) != cudaSuccess ||
      (code && cudaMemcpyToSymbol(symbol, &none, sizeof(none)) != cudaSuccess)) {
    cudaGetLastError();
    return RLCS_ERR_CUDA;
  }
  return static_cast<rlcs_status>(code);
}
rlcs_status distill_status();

template <class K, class Args>
rlcs_status launch_any(K kernel, const Args &p, cudaStream_t st) {
  const int64_t blocks = p.tokens < seq::kSms * 4 ? p.tokens : seq::kSms * 4;
  return launched(launch_ex(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, st, true, p));
}
// `entries`: bytes of shared memory to a team, at most kTeamEntries.
constexpr size_t kTeamEntries = 49152 / (kTeamBlock / 32);
template <auto Kernel, int TEAM, class Args>
rlcs_status launch_team(const Args &p, int per_sm, size_t entries, cudaStream_t st) {
  constexpr int kTeams = kTeamBlock / TEAM;
  const size_t smem = entries * kTeams;
  if (smem > 0) {
    const cudaError_t e = allow_dynamic_smem<Kernel>(kTeamEntries * (kTeamBlock / 32));
    if (e != cudaSuccess) return launched(e);
  }
  const int64_t wanted = seq::ceil_div(p.tokens, kTeams), room = (int64_t)seq::kSms * per_sm;
  return launched(launch_ex(Kernel, dim3((unsigned)(wanted < room ? wanted : room)),
                            dim3(kTeamBlock), smem, st, true, p));
}
template <auto Kernel, class Args>
rlcs_status launch_few(const Args &p, cudaStream_t st) {
  const size_t smem = (size_t)kFewBlock * ((int)p.V | 1) * 4;
  return launched(launch_ex(Kernel, dim3((unsigned)seq::ceil_div(p.tokens, kFewBlock)),
                            dim3(kFewBlock), smem, st, true, p));
}
constexpr size_t kLongEntries = 65536;  // a block's, at most
template <auto Kernel, int NV, class Args>
rlcs_status launch_long(const Args &p, int threads, int ranks, size_t entries, cudaStream_t st) {
  constexpr size_t kWords = (size_t)NV * kTeam * 16;
  const cudaError_t e = allow_dynamic_smem<Kernel>(kWords + kLongEntries);
  if (e != cudaSuccess) return launched(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.tokens * ranks));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = kWords + entries;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  return launched(cudaLaunchKernelEx(&cfg, Kernel, p));
}

// How a call's rows are spread: the smallest team that holds a row. A row that
// starts inside a word may straddle one more than it fills. `On` has the
// kernels: few, team<TEAM, NV>, block<NV> and any. (In a graph, 524288 rows of 6
// float32: 79 us by teams of eight lanes, 14 by threads; 200000 of 32: 26 and 16.)
template <class T, class On, class Args>
rlcs_status spread(const Args &p, size_t entries, cudaStream_t st) {
  const bool whole = aligned(p.logits, 16) && (p.tokens == 1 || p.row_stride % kWord<T> == 0);
  const int64_t words = (p.V + kWord<T> - 1) / kWord<T> + (whole ? 0 : 1);
  if (p.V <= kFew && p.tokens > 2 * seq::kSms) return On::few(p, st);
  const bool narrow = entries * 4 <= kTeamEntries;  // four teams of 8 to a warp
  if (words <= 8 && narrow) return On::template team<8, 1>(p, entries, st);
  if (words <= 16 && narrow) return On::template team<8, 2>(p, entries, st);
  if (words <= 32 && narrow) return On::template team<8, 4>(p, entries, st);
  if (entries <= kTeamEntries) {
    if (words <= 64) return On::template team<32, 2>(p, entries, st);
    if (words <= 128) return On::template team<32, 4>(p, entries, st);
    if (words <= 256) return On::template team<32, 8>(p, entries, st);
  }
  // Few rows are spread over more blocks, as long as there are SMs without one.
  int ranks = 1;
  while (ranks < kMaxRanks && words > 16 * kTeam * ranks) ranks *= 2;
  while (ranks < kMaxRanks && p.tokens * ranks * 2 <= seq::kSms && words > 4 * kTeam * ranks)
    ranks *= 2;
  if (words > 16 * kTeam * ranks || p.tokens * ranks > INT32_MAX) return On::any(p, st);
  const int64_t each = seq::ceil_div(words, ranks);
  if (each <= 4 * kTeam) return On::template block<4>(p, ranks, entries, st);
  if (each <= 8 * kTeam) return On::template block<8>(p, ranks, entries, st);
  return On::template block<16>(p, ranks, entries, st);
}

}  // namespace loss
}  // namespace rlcs
