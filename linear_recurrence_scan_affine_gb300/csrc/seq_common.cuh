// Shared by the sequence operators (rlcs_seq.h): argument checks on the
// host, and typed loads and stores on the device.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch.cuh"
#include "rlcs_seq.h"
#include "scan_core.cuh"

namespace rlcs {
namespace seq {

constexpr int kSms = 152;  // GB300: what grids are sized for (a different count stays correct)
constexpr int64_t kMaxElems = (int64_t)1 << 60;  // element counts stay far below 2^63

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
inline int64_t esize(rlcs_dtype t) { return t == RLCS_F32 ? 4 : 2; }
inline bool known(rlcs_dtype t) { return t == RLCS_F32 || t == RLCS_BF16; }

// Whether a * b * c * d stays within kMaxElems (all >= 0).
inline bool product_fits(int64_t a, int64_t b, int64_t c, int64_t d = 1) {
  const int64_t f[4] = {a, b, c, d};
  int64_t p = 1;
  for (int64_t x : f) {
    if (x != 0 && p > kMaxElems / x) return false;
    p *= x;
  }
  return true;
}

// A byte range of device memory.
struct Range {
  uintptr_t lo, hi;
};
inline Range range(const void *p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, p ? a + (uintptr_t)bytes : a};
}
// A strided [tokens, heads, D] view (all sizes > 0, strides >= 0).
inline Range strided(const void *p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t D,
                     int64_t esz) {
  return range(p, ((n0 - 1) * s0 + (n1 - 1) * s1 + D) * esz);
}
inline bool meet(const Range &a, const Range &b) {
  return a.lo != a.hi && b.lo != b.hi && a.lo < b.hi && b.lo < a.hi;
}
// Outputs that overlap an input or one another.
template <int NO, int NI>
inline bool outputs_overlap(const Range (&outs)[NO], const Range (&ins)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (meet(outs[i], ins[j])) return true;
    for (int j = i + 1; j < NO; ++j)
      if (meet(outs[i], outs[j])) return true;
  }
  return false;
}

inline rlcs_status launched(cudaError_t e) {
  if (e == cudaSuccess) return RLCS_OK;
  cudaGetLastError();  // clear the non-sticky launch error
  return RLCS_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// V consecutive elements of a float32 or bfloat16 array, as raw words: what a
// load leaves in registers, and its values in float32.
// ---------------------------------------------------------------------------
template <class T, int V>
struct Raw;
template <>
struct Raw<float, 1> {
  float w;
  __device__ __forceinline__ void load(const float *p) { w = __ldg(p); }
  __device__ __forceinline__ float at(int) const { return w; }
  __device__ __forceinline__ void clear() { w = 0.0f; }
};
template <>
struct Raw<float, 2> {
  float2 w;
  __device__ __forceinline__ void load(const float *p) {
    w = __ldg(reinterpret_cast<const float2 *>(p));
  }
  __device__ __forceinline__ float at(int i) const { return i ? w.y : w.x; }
  __device__ __forceinline__ void clear() { w = make_float2(0.0f, 0.0f); }
};
template <>
struct Raw<__nv_bfloat16, 1> {
  unsigned short w;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    w = __ldg(reinterpret_cast<const unsigned short *>(p));
  }
  __device__ __forceinline__ float at(int) const { return __uint_as_float((uint32_t)w << 16); }
  __device__ __forceinline__ void clear() { w = 0; }
};
template <>
struct Raw<__nv_bfloat16, 2> {
  uint32_t w;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    w = __ldg(reinterpret_cast<const unsigned int *>(p));
  }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i ? (w & 0xffff0000u) : (w << 16));
  }
  __device__ __forceinline__ void clear() { w = 0u; }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ void store(float *p, const float (&v)[1]) { *p = v[0]; }
__device__ __forceinline__ void store(float *p, const float (&v)[2]) {
  *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
}
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[1]) {
  *p = __float2bfloat16_rn(v[0]);
}
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[2]) {
  *reinterpret_cast<uint32_t *>(p) = pack_bf16(v[0], v[1]);
}

// sigmoid(g) and 1 - sigmoid(g): both come from e = exp(-|g|) <= 1, so neither
// overflows nor cancels. The smaller one's relative error grows with |g|, as
// the exponent is rounded before its power is taken.
struct Gate {
  float a, om;
};
__device__ __forceinline__ Gate gate_of(float g) {
  const float e = __expf(-fabsf(g));
  const float big = __fdividef(1.0f, 1.0f + e), small = e * big;
  return g >= 0.0f ? Gate{big, small} : Gate{small, big};
}

}  // namespace seq
}  // namespace rlcs
