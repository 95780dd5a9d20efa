// Gated linear recurrence (rlcs_seq.h): forward, gradient and single step.
//
//   h_t = k_t a_t h_{t-1} + (1 - a_t) x_t,  a_t = sigmoid(gate_t), k_t the
//   episode cut: one affine map per step and channel, (m, c) = (k a, (1-a) x).
// The gradient is the same recurrence backward in time. With mu_t what step t
// hands to step t-1,
//   mu_t = k_t a_t (dh_t + mu_{t+1}),   L_t = dh_t + mu_{t+1},   mu_T = dh_last
// so a step's map, (k a, k a dh), needs that step's inputs alone.
//
// A warp walks the sequence for 32 or 64 channels (a row segment of 128 or
// 256 bytes), with its inputs copied asynchronously into a ring in shared
// memory a few chunks of steps ahead: each step costs a gate, one fma and a
// store, and every input is read once. Where a call has too few channels to
// fill the GPU that way, the warps of a cluster of blocks take consecutive
// segments of the steps instead: each composes its segment's map, the maps
// join through shared and distributed shared memory, and each replays its
// segment from the state that reaches it, its inputs still in the ring or in
// L2. Nothing passes through global memory and every sum has one fixed order.
//
// Measured, bfloat16. Warps alone, 64 x 512 x 1024: forward and gradient 124
// us for 605 MB, 4.9 TB/s (a copy reaches 6.7): bound by memory, the rest is
// the start and the end of the walks. Joined, 1 x 131072 x 512: 136 us for 403
// MB, 3.0 TB/s: the gates are worked out in both passes, on the 96 SMs that
// clusters of 12 can take, with 68% of the issue slots busy.
//
// A cut's map has m = -0, which no product of gates is, and composes by
// selection: a state that is not finite does not pass a cut, and passes
// everything else, however small the product of the gates on its way.
#include <atomic>
#include <type_traits>

#include "seq_common.cuh"

namespace rlcs {
namespace seq {
namespace {

// V channels in float32; pairs use the two-wide fp32 instructions.
template <int V>
struct Vf {
  float e[V];
};
template <int V>
__device__ __forceinline__ Vf<V> fma(Vf<V> a, Vf<V> b, Vf<V> c) {
  if constexpr (V == 2) {
    const float2 r = __ffma2_rn(make_float2(a.e[0], a.e[1]), make_float2(b.e[0], b.e[1]),
                                make_float2(c.e[0], c.e[1]));
    return {r.x, r.y};
  } else {
    return {fmaf(a.e[0], b.e[0], c.e[0])};
  }
}
template <int V>
__device__ __forceinline__ Vf<V> mul(Vf<V> a, Vf<V> b) {
  if constexpr (V == 2) {
    const float2 r = __fmul2_rn(make_float2(a.e[0], a.e[1]), make_float2(b.e[0], b.e[1]));
    return {r.x, r.y};
  } else {
    return {a.e[0] * b.e[0]};
  }
}
template <int V>
__device__ __forceinline__ Vf<V> add(Vf<V> a, Vf<V> b) {
  if constexpr (V == 2) {
    const float2 r = __fadd2_rn(make_float2(a.e[0], a.e[1]), make_float2(b.e[0], b.e[1]));
    return {r.x, r.y};
  } else {
    return {a.e[0] + b.e[0]};
  }
}
template <int V>
__device__ __forceinline__ Vf<V> all(float x) {
  Vf<V> r;
#pragma unroll
  for (int v = 0; v < V; ++v) r.e[v] = x;
  return r;
}
template <int V>
__device__ __forceinline__ Vf<V> one_less(Vf<V> x) {  // 1 - x
  return fma(x, all<V>(-1.0f), all<V>(1.0f));
}

// The map x -> c + m x of a run of steps, per channel.
template <int V>
struct alignas(8 * V) Map {
  Vf<V> m, c;
};
// The mark of a cut. Further gates, none below zero, keep its sign; a product
// of gates that has become too small for float32 is +0.
__device__ __forceinline__ float cut_mark() { return -0.0f; }
__device__ __forceinline__ bool is_cut(float m) { return __float_as_uint(m) == 0x80000000u; }
// A cut takes nothing of what came before, not even NaN * 0. A product of
// gates that has become +0 stands for a positive one: it leaves an infinity as
// it is, as the steps one by one would.
template <int V>
__device__ __forceinline__ Vf<V> reach(const Map<V> &p, Vf<V> x) {
  Vf<V> r;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float m = p.m.e[v] == 0.0f && fabsf(x.e[v]) == INFINITY ? 1.0f : p.m.e[v];
    r.e[v] = is_cut(p.m.e[v]) ? p.c.e[v] : fmaf(m, x.e[v], p.c.e[v]);
  }
  return r;
}
template <int V>
__device__ __forceinline__ Map<V> join(const Map<V> &outer, const Map<V> &inner) {  // inner first
  Map<V> r = {mul(outer.m, inner.m), reach(outer, inner.c)};
#pragma unroll
  for (int v = 0; v < V; ++v)  // (the product of two marks is +0)
    if (is_cut(outer.m.e[v])) r.m.e[v] = cut_mark();
  return r;
}
// a = sigmoid(g) and om = 1 - a = 1 / (1 + e^g), neither by cancellation: a =
// e^g om for a closed gate (g < 0), whose a is small, else 1 - om. Relative
// error up to (2 |g| + 8) 2^-24: the exponent g log2 e is rounded, to 2^-24 of
// itself, before its power is taken. An infinite e^g gives om = 0, a = 1.
template <int V>
struct Gates {
  Vf<V> a, om;
};
template <int V>
__device__ __forceinline__ Gates<V> gates_of(Vf<V> g) {
  Vf<V> e = mul(g, all<V>(1.4426950408889634f));
#pragma unroll
  for (int v = 0; v < V; ++v) asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.e[v]));
  Vf<V> om = add(e, all<V>(1.0f));
#pragma unroll
  for (int v = 0; v < V; ++v) asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(om.e[v]));
  Vf<V> a = one_less(om);
#pragma unroll
  // (a predicated product: 1 x 131072 x 512 136 us, 145 with a product and a selection)
  for (int v = 0; v < V; ++v)
    asm("{\n\t.reg .pred p;\n\tsetp.lt.f32 p, %1, 0f00000000;\n\t@p mul.f32 %0, %2, %3;\n\t}"
        : "+f"(a.e[v])
        : "f"(g.e[v]), "f"(e.e[v]), "f"(om.e[v]));
  return {a, om};
}

// This block's rank and the number of blocks in its cluster.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Write a map to the same shared-memory place of another block of the cluster.
template <int V>
__device__ __forceinline__ void put_remote(const Map<V> *place, uint32_t rank, const Map<V> &v) {
  uint32_t there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(there)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(place))), "r"(rank));
#pragma unroll
  for (int k = 0; k < V; ++k) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there + 4 * k), "f"(v.m.e[k]) : "memory");
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there + 4 * (V + k)), "f"(v.c.e[k])
                 : "memory");
  }
}

struct ScanArgs {
  const void *x, *gate, *h, *dh;
  const uint8_t *reset;
  const float *first;  // state before the walk's first step: h0, or dh_last
  const float *h0;     // backward: the state before t = 0
  void *out, *out2;    // h, or dx and dgate
  float *last;         // state after the walk's last step: h_last, or dh0
  int64_t T, D, groups;
  int segment;  // steps a warp takes at a time (joined walks)
};

constexpr int kChunkBytes = 4096;  // a chunk of steps, all inputs together
constexpr int kWarpsMax = 16;      // warps of a block that walk together

// Chunks in a warp's ring: a warp that walks alone keeps three copies in
// flight, one of 16 that share an SM two, and one that loads through
// registers writes the next chunk while it reads the last.
template <int CB, bool JOINED>
constexpr int ring_chunks() {
  return CB == 0 ? 2 : (JOINED ? 3 : 4);
}

template <int CB>
__device__ __forceinline__ void copy_async(uint32_t dst, uintptr_t src) {
  if constexpr (CB == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// BACK walks from t = T-1 to 0 (the gradient); step index s counts along the
// walk, so t = s forward and T-1-s backward. JOINED: the block's warps and
// the cluster's blocks share one group of channels; else every warp has its
// own. CB: bytes per asynchronous copy, or 0 for plain loads (bfloat16 rows
// that do not start on 4-byte boundaries).
template <class E, int V, int CB, bool BACK, bool JOINED>
__global__ void __launch_bounds__(JOINED ? kWarpsMax * 32 : 32)
    gated_scan_kernel(const ScanArgs p) {
  constexpr int CH = 32 * V, kRow = CH * (int)sizeof(E), ARRAYS = BACK ? 4 : 2;
  constexpr int kChunk = kChunkBytes / (ARRAYS * kRow);  // steps
  constexpr int kStages = ring_chunks<CB, JOINED>();
  constexpr int kArray = kChunk * kRow;                  // bytes
  constexpr int kBatch = kChunk < 16 / V ? kChunk : 16 / V;
  static_assert(kChunk <= 32 && (CB == 0 || kArray % ((CB ? CB : 1) * 32) == 0),
                "whole rounds of copies");
  extern __shared__ __align__(128) unsigned char ring_base[];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int warp = JOINED ? __shfl_sync(kFull, threadIdx.x >> 5, 0) : 0;
  const int warps = JOINED ? (int)blockDim.x >> 5 : 1;
  const int rank = JOINED ? (int)cluster_rank() : 0, blocks = JOINED ? (int)cluster_size() : 1;
  const int64_t group = JOINED ? blockIdx.x / blocks : blockIdx.x;
  const int64_t b = group / p.groups, ch = group % p.groups * CH + lane * V;
  const bool on = ch < p.D;
  unsigned char *ring = ring_base + warp * kStages * kChunkBytes;

  // this lane's share of a round of copies
  constexpr int kPer = CB ? kRow / CB : 1, kRows = CB ? 32 * CB / kRow : 1;
  const int crow = CB ? lane / kPer : 0;
  const int64_t cch = group % p.groups * CH + (CB ? lane % kPer * (CB / (int)sizeof(E)) : 0);
  const bool con = cch < p.D;
  const uint32_t cdst = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) +
                        (CB ? crow * kRow + lane % kPer * CB : 0);
  const void *const src[4] = {p.gate, BACK ? p.dh : p.x, BACK ? p.x : nullptr, p.h};
  // Copy steps [s, end) of arrays [0, arrays) into a stage: gate, then x
  // forward, or dh, x and the state before each step backward.
  auto copy = [&](int64_t s, int64_t end, int stage, int arrays) {
    if constexpr (CB != 0) {
      if (s < end && con) {
        const int64_t q = s + crow;
        const int64_t at = ((b * p.T + (BACK ? p.T - 1 - q : q)) * p.D + cch) * (int64_t)sizeof(E);
        const int64_t next = (BACK ? -p.D : p.D) * (int64_t)(kRows * sizeof(E));
        const bool whole = s + kChunk <= end && s + kChunk < p.T;  // and none reads before t = 0
#pragma unroll
        for (int a = 0; a < ARRAYS; ++a) {
          if (a >= arrays) break;
          uintptr_t from = reinterpret_cast<uintptr_t>(src[a]) +
                           (uintptr_t)(at - (a == 3 ? p.D * (int64_t)sizeof(E) : 0));
          const uint32_t to = cdst + stage * kChunkBytes + a * kArray;
#pragma unroll
          for (int k = 0; k < kChunk / kRows; ++k, from += (uintptr_t)next)
            if (whole || (q + k * kRows < end && (a != 3 || q + k * kRows < p.T - 1)))
              copy_async<CB>(to + k * kRows * kRow, from);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  auto place = [&](int stage, int a, int i) {
    return reinterpret_cast<Raw<E, V> *>(ring + stage * kChunkBytes + a * kArray + i * kRow +
                                         lane * V * (int)sizeof(E));
  };
  auto value = [&](int stage, int a, int i) { return *place(stage, a, i); };
  // The same through registers (CB = 0): each lane fetches its own column.
  Raw<E, V> held[CB == 0 ? ARRAYS : 1][CB == 0 ? kChunk : 1];
  auto fetch = [&](int64_t s, int64_t end, int arrays) {
    if constexpr (CB == 0) {
#pragma unroll
      for (int a = 0; a < ARRAYS; ++a) {
        if (a >= arrays) break;
        const int64_t t0 = (BACK ? p.T - 1 - s : s) - (a == 3 ? 1 : 0);
        const E *from = static_cast<const E *>(src[a]);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
          const int64_t t = BACK ? t0 - i : t0 + i;
          held[a][i].clear();
          if (on && s + i < end && t >= 0) held[a][i].load(from + (b * p.T + t) * p.D + ch);
        }
      }
    }
  };
  auto put = [&](int stage, int arrays) {
    if constexpr (CB == 0) {
#pragma unroll
      for (int a = 0; a < ARRAYS; ++a) {
        if (a >= arrays) break;
#pragma unroll
        for (int i = 0; i < kChunk; ++i) *place(stage, a, i) = held[a][i];
      }
    }
  };
  // Lane i reads step s + i's reset, a chunk ahead of its use (and compares
  // it only there, so that nothing waits for the load).
  auto read_cut = [&](int64_t s, int64_t end) -> uint32_t {
    const int64_t q = s + lane;
    uint32_t v = 0;
    if (p.reset && lane < kChunk && q < end)
      asm volatile("ld.global.nc.u8 %0, [%1];"
                   : "=r"(v)
                   : "l"(p.reset + b * p.T + (BACK ? p.T - 1 - q : q)));
    return v;
  };
  // Run `body` over the chunks of steps [from, end): body(s, n, cut, stage).
  // `copied`: the ring holds them already.
  auto walk = [&](int64_t from, int64_t end, int arrays, bool copied, auto body) {
    if (!copied) {
#pragma unroll
      for (int k = 0; k < kStages - 1; ++k) copy(from + k * kChunk, end, k, arrays);
      fetch(from, end, arrays);
      put(0, arrays);
    }
    uint32_t flag = read_cut(from, end);
    int stage = 0;
    for (int64_t s = from; s < end; s += kChunk) {
      if (CB != 0 && !copied) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncwarp();  // the chunk is here, and every lane is done with the stage refilled next
        copy(s + (kStages - 1) * kChunk, end, stage == 0 ? kStages - 1 : stage - 1, arrays);
      }
      const bool more = CB == 0 && !copied && s + kChunk < end;
      if (more) fetch(s + kChunk, end, arrays);
      const uint32_t cut = p.reset ? __ballot_sync(kFull, flag != 0) : 0u;
      flag = read_cut(s + kChunk, end);
      body(s, (int)(end - s < kChunk ? end - s : kChunk), cut, stage);
      stage = stage == kStages - 1 ? 0 : stage + 1;
      if (more) put(stage, arrays);
    }
    if (CB != 0 && !copied) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
    }
  };

  auto floats = [](const Raw<E, V> &r) {
    Vf<V> f;
#pragma unroll
    for (int v = 0; v < V; ++v) f.e[v] = r.at(v);
    return f;
  };

  Vf<V> state = all<V>(0.0f), start = all<V>(0.0f);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (p.first && on) state.e[v] = p.first[b * p.D + ch + v];
    if (BACK && p.h0 && on) start.e[v] = p.h0[b * p.D + ch + v];
  }

  // Replay steps from `state`, writing the results.
  auto replay = [&](int64_t s, int n, uint32_t cut, int stage) {
    const int64_t t0 = BACK ? p.T - 1 - s : s, step = BACK ? -p.D : p.D;
    E *out = static_cast<E *>(p.out) + (b * p.T + t0) * p.D + ch;
    E *out2 = BACK ? static_cast<E *>(p.out2) + (b * p.T + t0) * p.D + ch : nullptr;
    auto run = [&](auto plain) {
#pragma unroll
      for (int i0 = 0; i0 < kChunk; i0 += kBatch) {
        // a batch's inputs first, then its steps: the stores of one step
        // would otherwise hold back the next step's reads
        Vf<V> a[kBatch], y[kBatch];  // y: (1 - a) x, or dh
        // 1 - a, and a (keep h - x), which is dgate but for dx
        [[maybe_unused]] Vf<V> om[BACK ? kBatch : 1], slope[BACK ? kBatch : 1];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const Gates<V> g = gates_of(floats(value(stage, 0, i0 + i)));
          a[i] = g.a;
          y[i] = floats(value(stage, 1, i0 + i));
          if constexpr (BACK) {
            om[i] = g.om;
            Vf<V> prev = floats(value(stage, 3, i0 + i));
            if (!plain) {
              if (s + i0 + i == p.T - 1) prev = start;
              if (cut >> (i0 + i) & 1) prev = all<V>(0.0f);
            }
            slope[i] = mul(g.a, fma(floats(value(stage, 2, i0 + i)), all<V>(-1.0f), prev));
          } else {
            y[i] = mul(g.om, y[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i, out += step, out2 += BACK ? step : 0) {
          if (!plain && i0 + i >= n) break;
          const bool kept = plain || !(cut >> (i0 + i) & 1);
          if constexpr (BACK) {
            const Vf<V> lam = add(y[i], state), dx = mul(om[i], lam);
            const Vf<V> dg = mul(dx, slope[i]);
            state = mul(a[i], lam);
            if (!kept) state = all<V>(0.0f);
            if (on) {
              store(out, dx.e);
              store(out2, dg.e);
            }
          } else {
            state = kept ? fma(a[i], state, y[i]) : y[i];
            if (on) store(out, state.e);
          }
        }
      }
    };
    if (n == kChunk && cut == 0 && !(BACK && s + kChunk == p.T)) run(std::true_type{});
    else run(std::false_type{});
  };

  if constexpr (!JOINED) {
    walk(0, p.T, ARRAYS, false, replay);
    if (p.last && on)
#pragma unroll
      for (int v = 0; v < V; ++v) p.last[b * p.D + ch + v] = state.e[v];
  } else {
    Map<V>(*maps)[32] = reinterpret_cast<Map<V>(*)[32]>(
        ring_base + warps * kStages * kChunkBytes);  // [warps][32]
    Map<V>(*across)[32] = maps + warps;              // [blocks][32]
    const int64_t span = (int64_t)p.segment * warps * blocks;
    if (blocks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    for (int64_t w0 = 0; w0 < p.T; w0 += span) {
      const int64_t from = w0 + (int64_t)(rank * warps + warp) * p.segment;
      const int64_t end = from + p.segment < p.T ? from + p.segment : p.T;
      const bool fits = p.segment <= kStages * kChunk;  // the ring keeps the segment
      Map<V> own = {all<V>(1.0f), all<V>(0.0f)};
      walk(from, end, fits ? ARRAYS : 2, false, [&](int64_t s, int n, uint32_t cut, int stage) {
        auto run = [&](auto plain) {
#pragma unroll
          for (int i = 0; i < kChunk; ++i) {
            if (!plain && i >= n) break;
            const Gates<V> g = gates_of(floats(value(stage, 0, i)));
            const Vf<V> c = mul(BACK ? g.a : g.om, floats(value(stage, 1, i)));
            own.c = fma(g.a, own.c, c);
            own.m = mul(own.m, g.a);
            if (!plain && (cut >> i & 1)) {
              own.m = all<V>(cut_mark());
              own.c = BACK ? all<V>(0.0f) : c;
            }
          }
        };
        if (n == kChunk && cut == 0) run(std::true_type{});
        else run(std::false_type{});
      });
      maps[warp][lane] = own;
      __syncthreads();
      if (blocks > 1) {
        // the peers have started, and have read the last window's maps
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (warp == 0) {
          Map<V> all_of = maps[0][lane];
          for (int w = 1; w < warps; ++w) all_of = join(maps[w][lane], all_of);
          for (int r = 0; r < blocks; ++r) put_remote(&across[rank][lane], r, all_of);
        }
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      }
      Vf<V> after = state;
      if (blocks > 1) {
        for (int r = 0; r < blocks; ++r) {
          if (r == rank) state = after;
          after = reach(across[r][lane], after);
        }
        if (w0 + span < p.T) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      } else {
        for (int w = 0; w < warps; ++w) after = reach(maps[w][lane], after);
      }
      for (int w = 0; w < warp; ++w) state = reach(maps[w][lane], state);
      walk(from, end, ARRAYS, fits, replay);
      if (p.last && on && from < end && end == p.T)
#pragma unroll
        for (int v = 0; v < V; ++v) p.last[b * p.D + ch + v] = state.e[v];
      state = after;
      __syncthreads();  // every warp has read the block's maps
    }
  }
}

// How a call's steps are shared out. Measured on GB300, us forward / gradient:
//  - a warp walks alone from 5 channel groups per SM on, or where the walk is
//    short: 64 x 512 x 1024 bf16 35 / 70 against 58 / 83 joined, 128 x 40 x
//    2048 12 / 21 against 22 / 30; with 128 groups (8 x 4096 x 1024) alone
//    127 / 259 against 54 / 78 joined;
//  - joined, the blocks of a cluster are as many as let every group of channels
//    have its cluster at once, which depends on how many SMs each of the
//    device's processing clusters has: the runtime is asked. (8 clusters of 12
//    fit, 7 of 13 to 16: 1 x 131072 x 512 (8 groups) 136 / 196 with 12, 208 /
//    331 with 16, 171 / 239 with 8; 1 x 131072 x 832 (13) 185 / 266 with 10, 197
//    / 308 with 8; 1 x 65536 x 1088 (17) 145 / 208 with 6, 195 / 302 with 8; 2 x
//    16384 x 1024 (32) 55 / 81 with 4, 78 / 118 with 8 and 85 / 119 with 2.)
//    Sizes are not tried where a smaller one did as well: 26 groups take 4 (99 /
//    151) rather than 5 (117 / 140).
//  - segments of 256 steps, or, where most SMs work, 128 forward and 64 in the
//    gradient, which keep the second pass in L2: 8 x 4096 x 1024 54 / 78
//    against 54 / 87.
struct Share {
  int blocks, warps, steps;  // blocks = 0: every warp alone
};
// at_once(n): clusters of n blocks that the device runs at the same time.
template <class AtOnce>
Share share_out(int64_t groups, int64_t T, int chunk, bool back, AtOnce at_once) {
  if (T <= 128 || groups >= 5 * (int64_t)kSms) return {0, 1, 0};
  int blocks = 1;
  for (int wider : {2, 3, 4, 6, 8, 9, 10, 12, 16})
    if (groups * wider <= kSms && T >= (int64_t)wider * kWarpsMax * chunk &&
        groups <= at_once(wider))
      blocks = wider;
  const int64_t warps = ceil_div(T, 32) < kWarpsMax ? ceil_div(T, 32) : kWarpsMax;
  const int64_t most = groups * blocks <= 2 * kSms / 3 ? 256 : (back ? 64 : 128);
  const int64_t each = ceil_div(ceil_div(T, blocks * warps), chunk) * chunk;
  return {blocks, (int)warps, (int)(each < most ? each : most)};
}

// Clusters of `size` blocks of a kernel, each with an SM to itself, that the
// current device runs at once; asked once per device and size. The kernel may
// be launched with any size that was asked for.
template <auto Kernel>
int clusters_at_once(int size, size_t smem) {
  static std::atomic<int> known[64][17];  // the answer + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::atomic<int> *k = dev < 64 ? &known[dev][size] : nullptr;
  if (k && k->load(std::memory_order_relaxed)) return k->load(std::memory_order_relaxed) - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(size * kSms));
  cfg.blockDim = dim3(kWarpsMax * 32);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)size;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (allow_dynamic_smem<Kernel>(smem) != cudaSuccess ||
      cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (k) k->store(n + 1, std::memory_order_relaxed);
  return n;
}

template <class E, int V, int CB, bool BACK>
cudaError_t launch_scan(ScanArgs a, int64_t B, cudaStream_t st) {
  constexpr int kRow = 32 * V * (int)sizeof(E), kChunk = kChunkBytes / ((BACK ? 4 : 2) * kRow);
  a.groups = ceil_div(a.D, 32 * V);
  const int64_t groups = B * a.groups;
  constexpr auto kernel = gated_scan_kernel<E, V, CB, BACK, true>;
  constexpr size_t most =
      kWarpsMax * (ring_chunks<CB, true>() * kChunkBytes + 2 * sizeof(Map<V>) * 32);
  const Share share = share_out(groups, a.T, kChunk, BACK,
                                [](int size) { return clusters_at_once<kernel>(size, most); });
  if (share.blocks == 0)
    return launch_ex(gated_scan_kernel<E, V, CB, BACK, false>, dim3((unsigned)groups), dim3(32),
                     ring_chunks<CB, false>() * kChunkBytes, st, true, a);
  const cudaError_t e = allow_dynamic_smem<kernel>(most);
  if (e != cudaSuccess) return e;
  a.segment = share.steps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * share.blocks));
  cfg.blockDim = dim3((unsigned)share.warps * 32);
  cfg.dynamicSmemBytes = (size_t)share.warps * ring_chunks<CB, true>() * kChunkBytes +
                         sizeof(Map<V>) * 32 * (size_t)(share.warps + share.blocks);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)share.blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Two channels per lane where a pair of them can be loaded and stored
// together, copies of 16 bytes where every row starts on such a boundary.
template <bool BACK>
rlcs_status run_scan(const ScanArgs &a, int64_t B, rlcs_dtype dtype, rlcs_stream_t stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uintptr_t bits = (uintptr_t)(a.D * esize(dtype));
  for (const void *q : {a.x, a.gate, a.h, a.dh, (const void *)a.out, (const void *)a.out2})
    bits |= reinterpret_cast<uintptr_t>(q);
  using bf = __nv_bfloat16;
  if (dtype == RLCS_F32)
    return launched(bits % 16 == 0 ? launch_scan<float, 2, 16, BACK>(a, B, st)
                                   : launch_scan<float, 1, 4, BACK>(a, B, st));
  return launched(bits % 16 == 0  ? launch_scan<bf, 2, 16, BACK>(a, B, st)
                  : bits % 4 == 0 ? launch_scan<bf, 2, 4, BACK>(a, B, st)
                                  : launch_scan<bf, 1, 0, BACK>(a, B, st));
}

// One step, a thread to a channel: bound by the launch (1.3 us in a graph for
// 4 x 64), or by memory: 4096 x 512 bf16 moves 29 MB, 4.4 us.
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
         product_fits(B, ceil_div(D, 32), 1) && B * ceil_div(D, 32) * 16 < (int64_t)INT32_MAX;
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
  return run_scan<false>(a, B, dtype, stream);
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
  return run_scan<true>(a, B, dtype, stream);
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
