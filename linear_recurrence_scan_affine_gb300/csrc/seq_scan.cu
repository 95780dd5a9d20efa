// Gated linear recurrence (rlcs_seq.h): forward, gradient and single step.
//
//   h_t = k_t a_t h_{t-1} + (1 - a_t) x_t,  a_t = sigmoid(gate_t), k_t the
//   episode cut: one affine map per step and channel, (m, c) = (k a, (1-a) x).
// The gradient is the same recurrence backward in time. With mu_t what step t
// hands to step t-1,
//   mu_t = k_t a_t (dh_t + mu_{t+1}),   L_t = dh_t + mu_{t+1},   mu_T = dh_last
// so a step's map, (k a, k a dh), needs that step's inputs alone.
//
// A block owns CH channels of one batch row and walks the sequence in spans:
// each thread takes L consecutive steps of its channels into registers,
// composes their maps, the block joins its warps' maps through shared memory,
// and each thread replays its steps from the state that reaches them. Every
// input is read once. A cut's map has m = 0 and composes by selection, so a
// non-finite state of one episode does not reach the next.
#include "seq_common.cuh"

namespace rlcs {
namespace seq {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ FPair join(FPair outer, FPair inner) {  // inner applied first
  if (outer.m == 0.0f) return outer;
  return {outer.m * inner.m, fmaf(outer.m, inner.c, outer.c)};
}
__device__ __forceinline__ float reach(FPair p, float x) {
  return p.m == 0.0f ? p.c : fmaf(p.m, x, p.c);
}

struct ScanArgs {
  const void *x, *gate, *h, *dh;
  const uint8_t *reset;
  const float *first;  // state before the walk's first step: h0, or dh_last
  const float *h0;     // backward: the state before t = 0
  void *out, *out2;    // h, or dx and dgate
  float *last;         // state after the walk's last step: h_last, or dh0
  int64_t T, D, groups;
};

// BACK walks from t = T-1 to 0 (the gradient); step index s counts along the
// walk, so t = s forward and T-1-s backward.
template <class E, int V, int L, bool BACK>
__global__ void __launch_bounds__(kWarps * 32) gated_scan_kernel(const ScanArgs p) {
  constexpr int CH = 32 * V;
  constexpr int kSpan = kWarps * L;
  __shared__ FPair maps[2][kWarps][CH];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t b = blockIdx.x / p.groups, ch = (blockIdx.x % p.groups) * CH + lane * V;
  const bool on = ch < p.D;
  const int64_t base = b * p.T * p.D + ch;
  const E *x = static_cast<const E *>(p.x) + base, *gate = static_cast<const E *>(p.gate) + base;
  const E *hs = BACK ? static_cast<const E *>(p.h) + base : nullptr;
  const E *dh = BACK ? static_cast<const E *>(p.dh) + base : nullptr;
  E *out = static_cast<E *>(p.out) + base, *out2 = BACK ? static_cast<E *>(p.out2) + base : nullptr;

  float carry[V], start[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    carry[v] = p.first && on ? p.first[b * p.D + ch + v] : 0.0f;
    start[v] = BACK && p.h0 && on ? p.h0[b * p.D + ch + v] : 0.0f;
  }
  int buf = 0;
  for (int64_t s0 = 0; s0 < p.T; s0 += kSpan, buf ^= 1) {
    const int64_t s = s0 + warp * L;  // this thread's first step
    const int n = (int)(p.T - s < L ? (p.T - s > 0 ? p.T - s : 0) : L);
    Raw<E, V> rx[L], rg[L], rd[BACK ? L : 1], rh[BACK ? L : 1];
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int64_t t = BACK ? p.T - 1 - (s + i) : s + i;
      rx[i].clear();
      rg[i].clear();
      if (BACK) rd[i].clear(), rh[i].clear();
      if (i < n && on) {
        rx[i].load(x + t * p.D);
        rg[i].load(gate + t * p.D);
        if (BACK) {
          rd[i].load(dh + t * p.D);
          if (t > 0) rh[i].load(hs + (t - 1) * p.D);
        }
      }
    }
    uint32_t cut = 0;  // bit i: step i starts an episode
    if (p.reset) {
      bool c = false;
      if (lane < n) c = p.reset[b * p.T + (BACK ? p.T - 1 - (s + lane) : s + lane)] != 0;
      cut = __ballot_sync(kFull, c);
    }
    FPair own[V];
#pragma unroll
    for (int v = 0; v < V; ++v) own[v] = {1.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < L; ++i)
      if (i < n)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const Gate g = gate_of(rg[i].at(v));
          const float m = cut >> i & 1 ? 0.0f : g.a;
          const float c = BACK ? m * rd[i].at(v) : g.om * rx[i].at(v);
          own[v] = join({m, c}, own[v]);
        }
#pragma unroll
    for (int v = 0; v < V; ++v) maps[buf][warp][lane * V + v] = own[v];
    __syncthreads();
    float in[V], total[V];  // the state that reaches this thread's steps, and the span's end
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float st = carry[v];
      in[v] = st;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w == warp) in[v] = st;
        st = reach(maps[buf][w][lane * V + v], st);
      }
      total[v] = st;
    }
#pragma unroll
    for (int i = 0; i < L; ++i) {
      if (i < n && on) {
        const int64_t t = BACK ? p.T - 1 - (s + i) : s + i;
        float o[V], o2[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const Gate g = gate_of(rg[i].at(v));
          const bool kept = !(cut >> i & 1);
          if (BACK) {
            const float lam = rd[i].at(v) + in[v];
            const float before = kept ? (t > 0 ? rh[i].at(v) : start[v]) : 0.0f;
            o[v] = g.om * lam;
            o2[v] = g.a * o[v] * (before - rx[i].at(v));
            in[v] = kept ? g.a * lam : 0.0f;
          } else {
            const float add = g.om * rx[i].at(v);
            in[v] = kept ? fmaf(g.a, in[v], add) : add;
            o[v] = in[v];
          }
        }
        store(out + t * p.D, o);
        if (BACK) store(out2 + t * p.D, o2);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = total[v];
    if (p.last && on && n > 0 && s + n == p.T)
#pragma unroll
      for (int v = 0; v < V; ++v) p.last[b * p.D + ch + v] = in[v];
  }
}

template <class E, int V, bool BACK>
cudaError_t launch_scan(ScanArgs a, int64_t B, cudaStream_t st) {
  constexpr int L = 16;
  a.groups = ceil_div(a.D, 32 * V);
  return launch_ex(gated_scan_kernel<E, V, L, BACK>, dim3((unsigned)(B * a.groups)),
                   dim3(kWarps * 32), 0, st, true, a);
}

template <class E>
__global__ void __launch_bounds__(256)
    gated_step_kernel(const E *x, const E *gate, const uint8_t *reset, const float *state,
                      float *new_state, E *h, int64_t n, int64_t D) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  Raw<E, 1> rx, rg;
  rx.load(x + i);
  rg.load(gate + i);
  const Gate g = gate_of(rg.at(0));
  const bool kept = !(reset && reset[i / D]);
  const float add = g.om * rx.at(0);
  const float s[1] = {kept ? fmaf(g.a, state[i], add) : add};
  new_state[i] = s[0];
  store(h + i, s);
}

bool scan_sizes(int64_t B, int64_t T, int64_t D, rlcs_dtype t) {
  // a block per 32 channels at least: the grid's limit in x
  return B > 0 && T > 0 && D > 0 && known(t) && product_fits(B, T, D) &&
         product_fits(B, ceil_div(D, 32), 1) && B * ceil_div(D, 32) < (int64_t)INT32_MAX;
}

}  // namespace
}  // namespace seq
}  // namespace rlcs

using namespace rlcs;
using namespace rlcs::seq;

extern "C" {

rlcs_status rlcs_gated_scan(const void *x, const void *gate, const uint8_t *reset,
                            const float *h0, void *h, float *h_last, int64_t B, int64_t T,
                            int64_t D, rlcs_dtype dtype, rlcs_stream_t stream) {
  if (!scan_sizes(B, T, D, dtype) || !x || !gate || !h) return RLCS_ERR_INVALID_ARG;
  const int64_t full = B * T * D * esize(dtype);
  const Range outs[] = {range(h, full), range(h_last, B * D * 4)};
  const Range ins[] = {range(x, full), range(gate, full), range(reset, B * T),
                       range(h0, B * D * 4)};
  if (outputs_overlap(outs, ins)) return RLCS_ERR_INVALID_ARG;
  ScanArgs a = {};
  a.x = x;
  a.gate = gate;
  a.reset = reset;
  a.first = h0;
  a.out = h;
  a.last = h_last;
  a.T = T;
  a.D = D;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == RLCS_F32) return launched(launch_scan<float, 1, false>(a, B, st));
  const bool pairs = D % 2 == 0 && aligned(x, 4) && aligned(gate, 4) && aligned(h, 4);
  return launched(pairs ? launch_scan<__nv_bfloat16, 2, false>(a, B, st)
                        : launch_scan<__nv_bfloat16, 1, false>(a, B, st));
}

rlcs_status rlcs_gated_scan_backward(const void *dh, const void *x, const void *gate,
                                     const void *h, const uint8_t *reset, const float *h0,
                                     const float *dh_last, void *dx, void *dgate, float *dh0,
                                     int64_t B, int64_t T, int64_t D, rlcs_dtype dtype,
                                     rlcs_stream_t stream) {
  if (!scan_sizes(B, T, D, dtype) || !dh || !x || !gate || !h || !dx || !dgate)
    return RLCS_ERR_INVALID_ARG;
  const int64_t full = B * T * D * esize(dtype), row = B * D * 4;
  const Range outs[] = {range(dx, full), range(dgate, full), range(dh0, row)};
  const Range ins[] = {range(dh, full), range(x, full),    range(gate, full),   range(h, full),
                       range(reset, B * T), range(h0, row), range(dh_last, row)};
  if (outputs_overlap(outs, ins)) return RLCS_ERR_INVALID_ARG;
  ScanArgs a = {};
  a.x = x;
  a.gate = gate;
  a.h = h;
  a.dh = dh;
  a.reset = reset;
  a.first = dh_last;
  a.h0 = h0;
  a.out = dx;
  a.out2 = dgate;
  a.last = dh0;
  a.T = T;
  a.D = D;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == RLCS_F32) return launched(launch_scan<float, 1, true>(a, B, st));
  const bool pairs = D % 2 == 0 && aligned(x, 4) && aligned(gate, 4) && aligned(h, 4) &&
                     aligned(dh, 4) && aligned(dx, 4) && aligned(dgate, 4);
  return launched(pairs ? launch_scan<__nv_bfloat16, 2, true>(a, B, st)
                        : launch_scan<__nv_bfloat16, 1, true>(a, B, st));
}

rlcs_status rlcs_gated_step(const void *x, const void *gate, const uint8_t *reset,
                            const float *state, float *new_state, void *h, int64_t B, int64_t D,
                            rlcs_dtype dtype, rlcs_stream_t stream) {
  if (!scan_sizes(B, 1, D, dtype) || !x || !gate || !state || !new_state || !h ||
      ceil_div(B * D, 256) >= (int64_t)INT32_MAX)
    return RLCS_ERR_INVALID_ARG;
  const int64_t full = B * D * esize(dtype), row = B * D * 4;
  const Range outs[] = {range(new_state, row), range(h, full)};
  const Range ins[] = {range(x, full), range(gate, full), range(reset, B),
                       state == new_state ? range(nullptr, 0) : range(state, row)};
  if (outputs_overlap(outs, ins)) return RLCS_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)ceil_div(B * D, 256));
  if (dtype == RLCS_F32)
    return launched(launch_ex(gated_step_kernel<float>, grid, dim3(256), 0, st, true,
                              static_cast<const float *>(x), static_cast<const float *>(gate),
                              reset, state, new_state, static_cast<float *>(h), B * D, D));
  using bf = __nv_bfloat16;
  return launched(launch_ex(gated_step_kernel<bf>, grid, dim3(256), 0, st, true,
                            static_cast<const bf *>(x), static_cast<const bf *>(gate), reset,
                            state, new_state, static_cast<bf *>(h), B * D, D));
}

}  // extern "C"
