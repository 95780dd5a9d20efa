// Causal attention over packed episodes with grouped heads (rlcs_seq.h):
// forward, gradient, and one new token over a cache.
//
// The softmax runs over the keys in one pass with a running maximum and sum;
// scores are kept in base 2 (scale * log2 e folded into one factor).
#include "seq_common.cuh"
#include "tensor_core.cuh"

namespace rlcs {
namespace seq {

uint32_t *linear_status();  // where the linear attention kernels record on this device

namespace {

using bf = __nv_bfloat16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------------------
// Tiles of 128 tokens of one sequence
// ---------------------------------------------------------------------------
constexpr int kTile = 128;

// Rows of the tiles a block walks over: with heads up to 64 wide half as many,
// so that two or three blocks share an SM's tensor memory and hide each
// other's waits, which short sequences are made of (packed episodes of up to
// 1024 steps, 12 heads of 64 on 4, forward and gradient: 273 us against 304
// with 128). Wider heads keep 128 (one sequence of 16384, 8 heads of 128 on 1,
// forward: 414 us against 514 with 64).
template <int DP>
constexpr int inner() {
  return DP == 64 ? 64 : 128;
}

// Tile `index` in the order of sequences, longest rows first within each (its
// last tile first): the sequence's bounds and the tile's number. One warp
// looks, a slice of the sequences to a lane; past kWarpSearch sequences the
// whole block does, so that many short episodes cost a block one round of
// loads.
struct Tile {
  int lo, len, first;  // the sequence's first token and length; the tile's first row in it
};
struct TileSearch {
  unsigned upto[18];  // tiles of each warp's sequences
  Tile tile;
  int found;
};
constexpr int kWarpSearch = 128;

// The sequence between two bounds.
__device__ __forceinline__ Tile between(int a, int b, int tokens) {
  a = a < 0 ? 0 : a;
  b = b < tokens ? b : tokens;
  return {a, b > a ? b - a : 0, 0};
}
__device__ __forceinline__ unsigned tiles_of(const Tile &t) { return (t.len + kTile - 1) / kTile; }
// The whole block calls this; `searcher` is the warp that goes on with the
// result at once, the others read it after the block's next barrier. (Tiles of
// bounds that are not in order may be counted past 32 bits: what is found then
// is still a tile inside the arrays.)
__device__ __forceinline__ void find_tile(const int32_t *cu, int sequences, int tokens,
                                          unsigned index, int searcher, TileSearch &sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool few = sequences <= kWarpSearch;
  if (few && warp != searcher) return;
  const int slice = few ? (sequences + 31) / 32 : (int)((sequences + blockDim.x - 1) / blockDim.x);
  const int at = slice * (few ? lane : (int)threadIdx.x);
  const int end = at < sequences - slice ? at + slice : sequences;
  if (warp == searcher && lane == 0) sm.found = 0;
  constexpr int kOwn = kWarpSearch / 32;
  int bound[kOwn + 1];  // one round of loads
  unsigned own = 0;
  if (few) {
#pragma unroll
    for (int j = 0; j <= kOwn; ++j) bound[j] = cu[at + j < end ? at + j : end];
#pragma unroll
    for (int j = 0; j < kOwn; ++j) own += tiles_of(between(bound[j], bound[j + 1], tokens));
  } else {
    for (int s = at; s < end; ++s) own += tiles_of(between(cu[s], cu[s + 1], tokens));
  }
  unsigned upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned n = __shfl_up_sync(kFull, upto, o);
    if (lane >= o) upto += n;
  }
  if (!few) {
    if (lane == 31) sm.upto[warp] = upto;
    __syncthreads();
    for (int w = 0; w < warp; ++w) upto += sm.upto[w];
  } else {
    __syncwarp();
  }
  unsigned left = index - (upto - own);
  auto take = [&](const Tile &x) {  // whether the tile is this sequence's
    const unsigned tiles = tiles_of(x);
    if (left < tiles) {
      sm.tile = {x.lo, x.len, (int)(tiles - 1 - left) * kTile};
      sm.found = 1;
      return true;
    }
    left -= tiles;
    return false;
  };
  if (left < own) {
    if (few) {
      bool done = false;
#pragma unroll
      for (int j = 0; j < kOwn; ++j)
        if (!done) done = take(between(bound[j], bound[j + 1], tokens));
    } else {
      for (int s = at; s < end; ++s)
        if (take(between(cu[s], cu[s + 1], tokens))) break;
    }
  }
  if (few) __syncwarp();
  else __syncthreads();
}

// Tiles that well-formed bounds can need.
int64_t tile_bound(int64_t sequences, int64_t tokens) {
  return tokens / kTile + (sequences < tokens ? sequences : tokens);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float2 pair(const uint32_t *r) {
  return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Tokens that no sequence holds: those before the first bound and from the
// last on. Their rows of a result are zeros, each block of the grid taking a
// share of them, and their log sums are -inf (of nothing). The warps that wait
// for a block's first scores do it, so that the two loads cost a call without
// such tokens nothing.
struct Unheld {
  int lo, hi;  // [0, lo) and [hi, tokens)
};
__device__ __forceinline__ Unheld unheld(const int32_t *cu, int sequences, int tokens) {
  int lo = __ldg(cu), hi = __ldg(cu + sequences);
  lo = lo < 0 ? 0 : (lo < tokens ? lo : tokens);
  hi = hi < lo ? lo : (hi < tokens ? hi : tokens);
  return {lo, hi};
}
__device__ __noinline__ void zero_unheld(bf *x, int width, Unheld u, int tokens, int thread,
                                         int threads) {
  const int eights = width / 8;
  const int64_t n = (int64_t)(u.lo + tokens - u.hi) * eights;
  for (int64_t i = (int64_t)blockIdx.x * threads + thread; i < n;
       i += (int64_t)gridDim.x * threads) {
    const int64_t row = i / eights;
    reinterpret_cast<uint4 *>(x + (row < u.lo ? row : row - u.lo + u.hi) * width)[i % eights] =
        make_uint4(0, 0, 0, 0);
  }
}
__device__ __noinline__ void empty_unheld(float *lse, int heads, Unheld u, int tokens, int thread,
                                          int threads) {
  const int rows = u.lo + tokens - u.hi;
  for (int64_t i = (int64_t)blockIdx.x * threads + thread; i < (int64_t)rows * heads;
       i += (int64_t)gridDim.x * threads) {
    const int row = (int)(i % rows);
    lse[i / rows * tokens + (row < u.lo ? row : row - u.lo + u.hi)] = -INFINITY;
  }
}

// The highest code that any attention call has recorded on this device, for
// callers whose scratch does not outlive a call.
__device__ uint32_t device_status;

// Record what went wrong where rlcs_check_status and rlcs_attention_status
// look for it.
__device__ __forceinline__ void report(WsHeader *ws, rlcs_status code) {
  atomicMax(&ws->status, (uint32_t)code);
  atomicMax(&device_status, (uint32_t)code);
}

// A wait that ran out: let copies in flight land, then record it.
__device__ __forceinline__ void settle(int abort, WsHeader *ws) {
  if (!abort) return;
  for (int i = 0; i < 1000; ++i) __nanosleep(2000);
  if (threadIdx.x == 0) report(ws, RLCS_ERR_TIMEOUT);
}

// The two warps of a forward block that share 32 query rows.
__device__ __forceinline__ void pair_barrier(int quarter) {
  asm volatile("bar.sync %0, 64;" ::"r"(quarter + 1) : "memory");
}

// COLS columns of one row of an fp32 accumulator, times f, to bf16 in global
// memory; `left` of them exist.
template <int COLS>
__device__ __forceinline__ void write_row(uint32_t acc, bf *out, int left, float f, bool on) {
#pragma unroll
  for (int c = 0; c < COLS / 32; ++c) {
    uint32_t a[32];
    tc::ld32(acc + c * 32, a);
    tc::wait_ld();
    if (on)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c * 32 + i * 8 < left) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = pack_bf16(__uint_as_float(a[i * 8 + 2 * e]) * f,
                             __uint_as_float(a[i * 8 + 2 * e + 1]) * f);
          *reinterpret_cast<uint4 *>(out + c * 32 + i * 8) = make_uint4(w[0], w[1], w[2], w[3]);
        }
  }
}

// ---------------------------------------------------------------------------
// Forward: a block per query tile and head, two blocks per SM (three with heads
// up to 64 wide).
//
// Warps 0..7 turn scores into weights, two threads to a query row (the lower
// and the upper half of the key columns; they exchange maxima through shared
// memory): 16 such warps on an SM hide each other's latencies, where 8 that
// held whole rows spilled registers. Warp 8 copies tiles in; warp 9 issues the
// products. Per key tile, in tensor memory:
//   S = Q K^T (128 or 64 fp32 columns), P over S (bf16 pairs),
//   O += P V (DP fp32 columns).
// P is rounded to bf16, the type the product takes; its sum is of the unrounded
// weights in fp32.
// Products run in the order they are issued, so the next tile's S follows
// the product that reads P. While one block's weights are formed the other
// block's products keep the tensor cores busy. Key tiles run from the
// diagonal down, so only the first needs the mask. The running maximum is
// raised only when it grows by more than 2^8 (weights then stay within fp32
// and bf16 range, and the final division removes the common factor), so O is
// rarely rescaled.
//
// One sequence of 16384, 8 heads of 128 on 1: 420 us, 1.31 PFLOP/s (a library
// matrix product reaches 1.95), the tensor pipe busy 60% of the time. S takes
// 830 clocks where PV takes 510: both its operands come from shared memory, 128
// bytes a clock at full rate, which is all that an SM can read, while copies
// come in. The rest is the chain from a tile's scores to its weights (1100
// clocks) and on to the product, which two blocks cover only in part. 40 x 600,
// 12 heads of 64 on 4: 75 us, most of it starting and ending blocks of two to
// ten key tiles.
// ---------------------------------------------------------------------------
// The swizzle of tiles in shared memory counts from 1024-byte boundaries;
// `raw` is declared on one. A block that finds it elsewhere does nothing.
__device__ __forceinline__ bool aligned_tiles(const void *raw, WsHeader *ws) {
  if ((tc::smem_addr(raw) & 1023) == 0) return true;
  if (threadIdx.x == 0) report(ws, RLCS_ERR_CUDA);
  return false;
}

template <int DP>
struct ForwardSmem {
  static constexpr int kStages = DP == 64 ? 2 : 1;  // of keys and values
  alignas(1024) unsigned char q[DP * 256], k[kStages][DP * inner<DP>() * 2],
      v[kStages][DP * inner<DP>() * 2];
  float row[2][128];  // maxima, and at the end sums, of the two halves of each row
  uint64_t q_full, k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t s_full, p_ready, o_full;
  TileSearch search;
  uint32_t tmem;
  int abort;
  int special;  // an infinity or NaN among the diagonal's values
};

struct ForwardArgs {
  const int32_t *cu;
  const bf *v;
  int64_t v_token, v_head;  // strides
  bf *o;
  float *lse;
  WsHeader *ws;
  int64_t sequences, tokens;
  int Hq, group, D;
  float scale2;  // scale * log2 e
};

// Values that are not finite, on the diagonal: a weight of zero does not take
// them out of a product, so the product sees zeros in their place, and the
// rows whose mask lets them through get them here. One row of the tile, half
// of its columns; rare, and not made fast.
template <int DP>
__device__ __noinline__ void add_special(const ForwardArgs &p, const Tile &t, int h, int r,
                                         int half) {
  const int64_t first = (int64_t)t.lo + t.first;
  const bf *v = p.v + first * p.v_token + h / p.group * p.v_head;
  bf *o = p.o + ((first + r) * p.Hq + h) * p.D;
  for (int d = half * (DP / 2); d < (half + 1) * (DP / 2) && d < p.D; d += 8)
    for (int j = 0; j <= r; ++j) {
      const uint4 x = __ldg(reinterpret_cast<const uint4 *>(v + j * p.v_token + d));
      if (!tc::special(x)) continue;
      const bf *e = reinterpret_cast<const bf *>(&x);
      for (int i = 0; i < 8; ++i) {
        const float f = __bfloat162float(e[i]);
        if (!(fabsf(f) < INFINITY)) o[d + i] = __float2bfloat16_rn(__bfloat162float(o[d + i]) + f);
      }
    }
}

template <int DP>
__global__ void __launch_bounds__(320, DP == 64 ? 3 : 2)
    attention_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const ForwardArgs p) {
  extern __shared__ __align__(1024) unsigned char raw[];
  ForwardSmem<DP> &sm = *reinterpret_cast<ForwardSmem<DP> *>(raw);
  pdl_wait();  // before tensor memory is taken: an earlier grid's blocks may still need it
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = __shfl_sync(kFull, threadIdx.x >> 5, 0);
  const int h = blockIdx.x % p.Hq;
  constexpr int IT = inner<DP>(), kStages = ForwardSmem<DP>::kStages;
  if (!aligned_tiles(raw, p.ws)) return;
  // An SM starts its next block only when the last has taken its tensor memory
  // and given up the right to more: that comes before anything slow. (400
  // episodes of 60 steps, 12 heads on 4 of 64, with one warp looking for the
  // tile: forward 161 -> 84 us, dk and dv 76 -> 61, dq 147 -> 92. 40 of 600 are
  // 2% slower: their blocks now start together rather than in turn.)
  if (warp == 9) tc::tmem_alloc(&sm.tmem, IT + DP);
  find_tile(p.cu, (int)p.sequences, (int)p.tokens, blockIdx.x / p.Hq, 8, sm.search);
  Tile t;
  int rows, steps;  // steps: key tiles, the last one first
  auto take_tile = [&] {
    t = sm.search.tile;
    rows = t.len - t.first < kTile ? t.len - t.first : kTile;
    steps = (t.first + rows + IT - 1) / IT;
  };
  auto first_key = [&](int it) { return (steps - 1 - it) * IT; };
  auto diagonal = [&](int it) { return first_key(it) >= t.first; };  // at most kStages tiles
  auto load_k = [&](int it) {
    tc::load_tile<DP, IT>(sm.k[it % kStages], &mk, &sm.k_full[it % kStages], h / p.group,
                          t.lo + first_key(it));
  };
  auto load_v = [&](int it) {
    tc::load_tile<DP, IT>(sm.v[it % kStages], &mv, &sm.v_full[it % kStages], h / p.group,
                          t.lo + first_key(it));
  };
  // the copying lane sets the barriers up and starts the first copies at once
  if (warp == 8 && lane == 0 && sm.search.found) {
    take_tile();
    for (int i = 0; i < kStages; ++i)
      for (uint64_t *b : {&sm.k_full[i], &sm.k_empty[i], &sm.v_full[i], &sm.v_empty[i]})
        mbar_init(b, 1);
    for (uint64_t *b : {&sm.q_full, &sm.s_full, &sm.o_full}) mbar_init(b, 1);
    mbar_init(&sm.p_ready, 8);
    sm.abort = sm.special = 0;
    fence_mbar_init();
    tc::load_tile<DP, kTile>(sm.q, &mq, &sm.q_full, h, t.lo + t.first);
    load_k(0);
    load_v(0);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  auto clear_unheld = [&] {
    const Unheld u = unheld(p.cu, (int)p.sequences, (int)p.tokens);
    if (u.lo == 0 && u.hi == (int)p.tokens) return;
    zero_unheld(p.o, p.Hq * p.D, u, (int)p.tokens, threadIdx.x, 256);
    if (p.lse) empty_unheld(p.lse, p.Hq, u, (int)p.tokens, threadIdx.x, 256);
  };
  if (!sm.search.found) {
    if (warp < 8) clear_unheld();
    if (warp == 9) tc::tmem_dealloc(sm.tmem, IT + DP);
    return;
  }
  take_tile();
  const uint32_t tmem = __shfl_sync(kFull, sm.tmem, 0), tS = tmem, tO = tmem + IT;
  volatile int *abort = &sm.abort, *special = &sm.special;
  const uint32_t lead = lane == 0;  // the lane that issues products

  if (warp == 8) {
    if (lane == 0) {
      for (int it = 1; it < steps; ++it) {
        const int st = it % kStages, use = it / kStages;
        if (use > 0 && !tc::mbar_wait(&sm.k_empty[st], (use - 1) & 1, abort)) break;
        load_k(it);
        if (use > 0 && !tc::mbar_wait(&sm.v_empty[st], (use - 1) & 1, abort)) break;
        load_v(it);
      }
    }
  } else if (warp == 9) {
    bool ok = tc::warp_wait(&sm.q_full, 0, abort);
    for (int it = 0; it < steps && ok; ++it) {
      const int st = it % kStages, use = it / kStages;
      ok = tc::warp_wait(&sm.k_full[st], use & 1, abort);
      if (!ok) break;
      tc::product_nt<DP, IT>(lead, tS, tc::smem_addr(sm.q), tc::smem_addr(sm.k[st]));
      tc::commit(lead, &sm.k_empty[st]);
      tc::commit(lead, &sm.s_full);
      ok = tc::warp_wait(&sm.v_full[st], use & 1, abort);
      if (!ok) break;
      // values past the sequence's end meet weights of zero: they must be finite
      if (it == 0 && first_key(0) + IT > t.len)
        tc::clear_rows<DP, IT>(sm.v[st], t.len - first_key(0), lane);
      __syncwarp();
      ok = tc::warp_wait(&sm.p_ready, it & 1, abort);
      if (!ok) break;
      if (diagonal(it) && *special) tc::clear_special<DP, IT>(sm.v[st], lane);
      tc::fence_after_sync();
      tc::product_parts<DP, IT, 2>(lead, tO, tS, tc::smem_addr(sm.v[st]), it > 0);
      tc::commit(lead, &sm.v_empty[st]);
      if (it + 1 == steps) tc::commit(lead, &sm.o_full);
    }
  } else {
    constexpr int HC = IT / 2;  // key columns of a thread
    const int r = threadIdx.x & 127, half = warp >> 2;  // this thread's row and half of the keys
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t mine = tS + lanes + half * HC;
    const float2 k2 = make_float2(p.scale2, p.scale2);
    float m = -INFINITY, l = 0.0f;
    clear_unheld();
    // after a wait that ran out the loop goes on without waiting, so that
    // every warp meets its partner's barriers
    for (int it = 0; it < steps; ++it) {
      if (diagonal(it)) {  // look its values over while its scores are formed
        uint32_t found = 0;
        tc::warp_wait(&sm.v_full[it], 0, abort);
#pragma unroll
        for (int i = 0; i < DP * IT / 8; i += 256)
          found |= tc::special(reinterpret_cast<const uint4 *>(sm.v[it])[i + threadIdx.x]);
        if (found) *special = 1;
      }
      tc::warp_wait(&sm.s_full, it & 1, abort);
      tc::fence_after_sync();
      uint32_t s[HC];
#pragma unroll
      for (int c = 0; c < HC; c += 32)
        tc::ld32(mine + c, *reinterpret_cast<uint32_t(*)[32]>(s + c));
      tc::wait_ld();
      const int last = t.first + r - first_key(it) - half * HC;  // the last column this row sees
      if (diagonal(it)) {
#pragma unroll
        for (int c = 0; c < HC; ++c)
          if (c > last) s[c] = 0xff800000u;
      }
      float t4[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) t4[c] = __uint_as_float(s[c]);
#pragma unroll
      for (int c = 4; c < HC; ++c) t4[c % 4] = fmaxf(t4[c % 4], __uint_as_float(s[c]));
      const float own = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
      sm.row[half][r] = own;
      pair_barrier(warp & 3);
      const float top = fmaxf(own, sm.row[half ^ 1][r]) * p.scale2;
      const bool raise = top > m + 8.0f;  // from the start (m = -inf) too
      if (__any_sync(kFull, raise)) {
        const float f = raise ? ex2(m - top) : 1.0f;
        if (raise) m = top;
        l *= f;
        const uint32_t acc = tO + lanes + half * (DP / 2);
        if (it > 0)
#pragma unroll 1
          for (int c = 0; c < DP / 2; c += 16) {
            uint32_t o[16];
            tc::ld16(acc + c, o);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tc::st16(acc + c, o);
          }
      }
      const float zero = m == -INFINITY ? 0.0f : -m;  // (a row that has seen no key yet)
      const float2 m2 = make_float2(zero, zero);
      float2 sum[2] = {};
#pragma unroll
      for (int c = 0; c < HC / 32; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 a = __ffma2_rn(pair(s + c * 32 + 2 * i), k2, m2);
          a.x = ex2(a.x);
          a.y = ex2(a.y);
          sum[i & 1] = __fadd2_rn(sum[i & 1], a);
          w[i] = pack_bf16(a.x, a.y);
        }
        tc::st16(mine + c * 16, w);
      }
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      tc::wait_st();
      tc::fence_before_sync();
      tc::warp_arrive(&sm.p_ready, lead);
    }
    pair_barrier(warp & 3);  // the partner has read the last maximum
    sm.row[half][r] = l;
    pair_barrier(warp & 3);
    l += sm.row[half ^ 1][r];
    if (tc::warp_wait(&sm.o_full, 0, abort)) {
      tc::fence_after_sync();
      const int64_t row = (int64_t)t.lo + t.first + r;
      write_row<DP / 2>(tO + lanes + half * (DP / 2),
                        p.o + (row * p.Hq + h) * p.D + half * (DP / 2), p.D - half * (DP / 2),
                        1.0f / l, r < rows);
      if (p.lse && half == 0 && r < rows)
        p.lse[(int64_t)h * p.tokens + row] = (m + log2f(l)) * kLn2;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  settle(sm.abort, p.ws);
  if (*special && warp < 8 && (threadIdx.x & 127) < rows && !*abort)
    add_special<DP>(p, t, h, threadIdx.x & 127, warp >> 2);
  if (warp == 9) tc::tmem_dealloc(sm.tmem, IT + DP);
}

// ---------------------------------------------------------------------------
// Gradient. delta_i = sum_d dout_id out_id first, then two kernels that each
// form P and dS again from q, k, lse: dq by query tiles, dk and dv by key
// tiles. Recomputing costs two of seven products, and buys results without
// atomics: every sum has one fixed order. The output that delta is made from
// is rounded to bf16; rows short enough to have all their keys in one tile get
// it from P and dP instead, in the dq kernel (59 episodes of up to 3 steps: dq
// and dk within 1.7e-3 of 64 bits, the rounding of the result, 3.3e-3 before).
//
// Blocks of 576 threads, one per SM (all 512 columns of tensor memory); heads
// up to 64 wide, 320 threads, two per SM. Four warps to 32 columns of a tile
// work on the scores, a row and 32 columns to a thread; one more warp copies
// tiles and one issues products. A thread's bf16 piece goes over its own fp32
// columns, so the pieces of an operand start 32 columns apart. dS is rounded to
// bf16 for its product, as P is; on the diagonal tile, whose short rows carry
// most of the gradient, the rounding's remainder goes into the other half of
// those columns and is multiplied too.
//
// 2 x 4096, 16 heads of 128 on 4: delta 14 us (4.7 TB/s), dk and dv 198 us (1.39
// PFLOP/s with the recomputed product, the tensor pipe busy 68%), dq 167 us
// (1.24, 57%). Both are bound by the chain scores, weights, product within a
// step, of which products of the steps before and after cover part.
// ---------------------------------------------------------------------------
struct BackwardArgs {
  const int32_t *cu;
  const bf *dout, *out;
  const float *lse;  // [Hq, tokens]
  float *delta;      // the same
  bf *dq, *dk, *dv;
  WsHeader *ws;
  int64_t sequences, tokens;
  int Hq, Hk, group, D;
  int split;            // dk, dv: blocks (a cluster) that share a group's query heads
  float scale, scale2;  // scale2 = scale * log2 e
};

// Eight products of bf16, summed in fp32.
__device__ __forceinline__ float dot8(const uint4 &u, const uint4 &v) {
  const uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), t);
    t = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), t);
  }
  return t;
}

// delta: DP/8 lanes to a row, 8 elements to a lane, four rows at a time.
template <int DP>
__global__ void __launch_bounds__(256)
    attention_delta_kernel(const bf *dout, const bf *out, float *delta, int64_t tokens, int Hq,
                           int D) {
  constexpr int kLanes = DP / 8, kRows = 256 / kLanes;
  pdl_wait();
  pdl_launch_dependents();
  const int d = threadIdx.x % kLanes * 8;
  const int64_t first = (int64_t)blockIdx.x * 4 * kRows + threadIdx.x / kLanes, end = tokens * Hq;
  uint4 a[4], b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = first + i * kRows;
    a[i] = b[i] = make_uint4(0, 0, 0, 0);
    if (row < end && d < D) {
      a[i] = __ldg(reinterpret_cast<const uint4 *>(dout + row * D + d));
      b[i] = __ldg(reinterpret_cast<const uint4 *>(out + row * D + d));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = first + i * kRows;
    float t = dot8(a[i], b[i]);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) t += __shfl_xor_sync(kFull, t, o);
    if (row < end && d == 0) delta[row % Hq * tokens + row / Hq] = t;
  }
}

// 32 values as bf16 pairs over the first 16 of their columns and, where
// `rest`, what the rounding took away over the other 16.
__device__ __forceinline__ void store_bf16(uint32_t at, const uint32_t (&d)[32], bool rest) {
  uint32_t w[16];
#pragma unroll
  for (int c = 0; c < 16; ++c)
    w[c] = pack_bf16(__uint_as_float(d[2 * c]), __uint_as_float(d[2 * c + 1]));
  tc::st16(at, w);
  if (rest) {
#pragma unroll
    for (int c = 0; c < 16; ++c)
      w[c] = pack_bf16(__uint_as_float(d[2 * c]) - __uint_as_float(w[c] << 16),
                       __uint_as_float(d[2 * c + 1]) - __uint_as_float(w[c] & 0xffff0000u));
    tc::st16(at + 16, w);
  }
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Four words to the shared memory of another block of the cluster.
__device__ __forceinline__ void put_remote4(uint32_t place, uint32_t rank, const uint32_t *x) {
  uint32_t there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(place), "r"(rank));
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(there), "r"(x[0]),
               "r"(x[1]), "r"(x[2]), "r"(x[3])
               : "memory");
}

// Four score warps to 32 columns of the inner tile, one that copies and one
// that issues.
template <int DP>
constexpr int backward_threads() {
  return (4 * inner<DP>() / 32 + 2) * 32;
}

template <int DP>
__device__ __forceinline__ void compute_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(backward_threads<DP>() - 64) : "memory");
}

template <int DP>
struct KvSmem {
  alignas(1024) unsigned char k[DP * 256], v[DP * 256], q[3][DP * inner<DP>() * 2],
      dout[2][DP * inner<DP>() * 2];
  float lse[2][128], delta[2][128];
  uint64_t k_full, v_full, q_full[3], q_empty[3], do_full[2], do_empty[2];
  uint64_t s_full, dp_full, p_ready, ds_ready, done;
  TileSearch search;
  uint32_t tmem;
  int abort;
};

// dk, dv: a block per key tile and key/value head, over the query tiles at
// and after it of every query head of the group. In tensor memory:
//   S^T = K Q^T and dP^T = V dO^T (128 columns each), P^T and dS^T over them,
//   dV += P^T dO and dK += dS^T Q (DP columns each).
// Issue order dV(i), S(i+1), dK(i), dP(i+1): P(i+1) is formed while dK(i) and
// dP(i+1) run, dS(i+1) while dV(i+1) and S(i+2) run.
// Where key tiles and heads alone would leave SMs idle, a cluster of blocks
// shares the group's query heads and adds its sums up through distributed
// shared memory, in rank order, each block the columns of its own.
template <int DP>
__global__ void __launch_bounds__(backward_threads<DP>(), DP == 64 ? 2 : 1)
    attention_dkv_kernel(const __grid_constant__ CUtensorMap mq,
                         const __grid_constant__ CUtensorMap mk,
                         const __grid_constant__ CUtensorMap mv,
                         const __grid_constant__ CUtensorMap mdo, const BackwardArgs p) {
  extern __shared__ __align__(1024) unsigned char raw[];
  KvSmem<DP> &sm = *reinterpret_cast<KvSmem<DP> *>(raw);
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = __shfl_sync(kFull, threadIdx.x >> 5, 0);
  const int rank = blockIdx.x % p.split, g = blockIdx.x / p.split % p.Hk;
  const int heads = p.group / p.split, head0 = g * p.group + rank * heads;
  constexpr int IT = inner<DP>(), PARTS = IT / 32, kCopy = 4 * PARTS, kIssue = kCopy + 1;
  if (!aligned_tiles(raw, p.ws)) return;
  if (warp == kIssue) tc::tmem_alloc(&sm.tmem, 2 * IT + 2 * DP);
  find_tile(p.cu, (int)p.sequences, (int)p.tokens, blockIdx.x / p.split / p.Hk, kCopy, sm.search);
  constexpr int kSubs = kTile / IT;  // query tiles that meet the diagonal
  Tile t;
  int key0, per_head, steps, rows;
  int tail;  // rows of the sequence's last query tile
  auto take_tile = [&] {
    t = sm.search.tile;
    // the first key tile has the most query tiles: turn the order round
    key0 = ((t.len + kTile - 1) / kTile - 1) * kTile - t.first;
    const int tiles = (t.len + IT - 1) / IT;
    per_head = tiles - key0 / IT;
    steps = per_head * heads;
    rows = t.len - key0 < kTile ? t.len - key0 : kTile;
    tail = t.len - (tiles - 1) * IT;
  };
  // Step i is query tile `sub` of head `head`, counted up by each role.
  struct Step {
    int head, sub;
  };
  auto after = [&](Step x) {
    return x.sub + 1 < per_head ? Step{x.head, x.sub + 1} : Step{x.head + 1, 0};
  };
  const Step begin = {head0, 0};
  auto first_row = [&](Step x) { return key0 + x.sub * IT; };
  auto load_q = [&](int i, Step x) {
    tc::load_tile<DP, IT>(sm.q[i % 3], &mq, &sm.q_full[i % 3], x.head, t.lo + first_row(x));
  };
  auto load_dout = [&](int i, Step x) {
    tc::load_tile<DP, IT>(sm.dout[i & 1], &mdo, &sm.do_full[i & 1], x.head, t.lo + first_row(x));
  };
  if (warp == kCopy && lane == 0 && sm.search.found) {
    take_tile();
    for (int i = 0; i < 3; ++i) mbar_init(&sm.q_full[i], 1), mbar_init(&sm.q_empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sm.do_full[i], 1), mbar_init(&sm.do_empty[i], 1);
    for (uint64_t *b : {&sm.k_full, &sm.v_full, &sm.s_full, &sm.dp_full, &sm.done}) mbar_init(b, 1);
    mbar_init(&sm.p_ready, 4 * PARTS);
    mbar_init(&sm.ds_ready, 4 * PARTS);
    sm.abort = 0;
    fence_mbar_init();
    tc::load_tile<DP, kTile>(sm.k, &mk, &sm.k_full, g, t.lo + key0);
    load_q(0, begin);
    tc::load_tile<DP, kTile>(sm.v, &mv, &sm.v_full, g, t.lo + key0);
    load_dout(0, begin);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  auto clear_unheld = [&] {
    constexpr int kThreads = backward_threads<DP>() - 64;
    const Unheld u = unheld(p.cu, (int)p.sequences, (int)p.tokens);
    if (u.lo == 0 && u.hi == (int)p.tokens) return;
    zero_unheld(p.dk, p.Hk * p.D, u, (int)p.tokens, threadIdx.x, kThreads);
    zero_unheld(p.dv, p.Hk * p.D, u, (int)p.tokens, threadIdx.x, kThreads);
  };
  if (!sm.search.found) {
    if (warp < kCopy) clear_unheld();
    if (warp == kIssue) tc::tmem_dealloc(sm.tmem, 2 * IT + 2 * DP);
    return;
  }
  take_tile();
  const uint32_t tmem = __shfl_sync(kFull, sm.tmem, 0);
  const uint32_t tS = tmem, tP = tS + IT, tV = tP + IT, tK = tV + DP;
  volatile int *abort = &sm.abort;
  const uint32_t lead = lane == 0;  // the lane that issues products

  if (warp == kCopy) {
    if (lane == 0) {
      Step x = begin;
      for (int i = 1; i < steps; ++i) {
        x = after(x);
        if (i >= 3 && !tc::mbar_wait(&sm.q_empty[i % 3], (i / 3 - 1) & 1, abort)) break;
        load_q(i, x);
        if (i >= 2 && !tc::mbar_wait(&sm.do_empty[i & 1], (i / 2 - 1) & 1, abort)) break;
        load_dout(i, x);
      }
    }
  } else if (warp == kIssue) {
    const uint32_t k = tc::smem_addr(sm.k), v = tc::smem_addr(sm.v);
    // rows past the sequence's end are another sequence's: they meet weights
    // of zero as a second operand, so they must be finite
    auto scores = [&](int i, Step x) {
      const int a = i % 3;
      if (!tc::warp_wait(&sm.q_full[a], (i / 3) & 1, abort)) return false;
      if (x.sub == per_head - 1 && tail < IT) tc::clear_rows<DP, IT>(sm.q[a], tail, lane);
      __syncwarp();
      tc::product_nt<DP, IT>(lead, tS, k, tc::smem_addr(sm.q[a]));
      tc::commit(lead, &sm.s_full);
      return true;
    };
    auto grads = [&](int i, Step x) {
      const int b = i & 1;
      if (!tc::warp_wait(&sm.do_full[b], (i / 2) & 1, abort)) return false;
      if (x.sub == per_head - 1 && tail < IT) tc::clear_rows<DP, IT>(sm.dout[b], tail, lane);
      __syncwarp();
      tc::product_nt<DP, IT>(lead, tP, v, tc::smem_addr(sm.dout[b]));
      tc::commit(lead, &sm.dp_full);
      return true;
    };
    Step x = begin;
    bool ok = tc::warp_wait(&sm.k_full, 0, abort) && scores(0, x) &&
              tc::warp_wait(&sm.v_full, 0, abort) && grads(0, x);
    for (int i = 0; i < steps && ok; ++i) {
      const bool diagonal = x.sub < kSubs;
      x = after(x);
      ok = tc::warp_wait(&sm.p_ready, i & 1, abort);
      if (!ok) break;
      tc::fence_after_sync();
      tc::product_parts<DP, IT, PARTS>(lead, tV, tS, tc::smem_addr(sm.dout[i & 1]), i > 0);
      tc::commit(lead, &sm.do_empty[i & 1]);
      if (i + 1 < steps && !(ok = scores(i + 1, x))) break;
      ok = tc::warp_wait(&sm.ds_ready, i & 1, abort);
      if (!ok) break;
      tc::fence_after_sync();
      tc::product_parts<DP, IT, PARTS>(lead, tK, tP, tc::smem_addr(sm.q[i % 3]), i > 0);
      if (diagonal)
        tc::product_parts<DP, IT, PARTS>(lead, tK, tP + 16, tc::smem_addr(sm.q[i % 3]), true);
      tc::commit(lead, &sm.q_empty[i % 3]);
      if (i + 1 == steps) tc::commit(lead, &sm.done);
      if (i + 1 < steps) ok = grads(i + 1, x);
    }
  } else {
    const int r = threadIdx.x & 127, part = warp >> 2;  // this thread's key row, its columns
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, mine = lanes + part * 32;
    // Column statistics of step i, negated: one value per thread of parts 0
    // and 1, a step ahead.
    auto column = [&](Step y) {
      const int at = first_row(y) + r;
      if (part > 1 || r >= IT) return 0.0f;
      if (at >= t.len) return part ? 0.0f : -INFINITY;  // no row: weights of zero
      const float x = (part ? p.delta : p.lse)[(int64_t)y.head * p.tokens + t.lo + at];
      return part ? -x : -x * kLog2e;
    };
    Step x = begin;
    float next = column(x);
    clear_unheld();
    const float2 k2 = make_float2(p.scale2, p.scale2);
    // after a wait that ran out the loop goes on without waiting, so that
    // every warp meets the others' barriers
    for (int i = 0; i < steps; ++i) {
      if (part < 2 && r < IT) (part ? sm.delta : sm.lse)[i & 1][r] = next;
      compute_barrier<DP>();
      const int row0 = first_row(x);
      const bool diagonal = x.sub < kSubs;
      x = after(x);
      if (i + 1 < steps) next = column(x);
      const float *lse = &sm.lse[i & 1][part * 32], *delta = &sm.delta[i & 1][part * 32];
      const int own = key0 + r - row0 - part * 32;  // columns before this key's own row: masked
      uint32_t s[32], d[32];
      tc::warp_wait(&sm.s_full, i & 1, abort);
      tc::fence_after_sync();
      tc::ld32(tS + mine, s);
      tc::wait_ld();
#pragma unroll
      for (int c = 0; c < 32; c += 4) {
        const float4 m = *reinterpret_cast<const float4 *>(lse + c);
        const float2 a = __ffma2_rn(pair(s + c), k2, make_float2(m.x, m.y));
        const float2 b = __ffma2_rn(pair(s + c + 2), k2, make_float2(m.z, m.w));
        s[c] = __float_as_uint(ex2(a.x));
        s[c + 1] = __float_as_uint(ex2(a.y));
        s[c + 2] = __float_as_uint(ex2(b.x));
        s[c + 3] = __float_as_uint(ex2(b.y));
      }
      if (diagonal)
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c < own) s[c] = 0u;
      store_bf16(tS + mine, s, false);
      tc::wait_st();
      tc::fence_before_sync();
      tc::warp_arrive(&sm.p_ready, lead);

      tc::warp_wait(&sm.dp_full, i & 1, abort);
      tc::fence_after_sync();
      tc::ld32(tP + mine, d);
      tc::wait_ld();
#pragma unroll
      for (int c = 0; c < 32; c += 4) {
        const float4 m = *reinterpret_cast<const float4 *>(delta + c);
        const float2 a =
            __fmul2_rn(pair(s + c), __fadd2_rn(pair(d + c), make_float2(m.x, m.y)));
        const float2 b =
            __fmul2_rn(pair(s + c + 2), __fadd2_rn(pair(d + c + 2), make_float2(m.z, m.w)));
        d[c] = __float_as_uint(a.x);
        d[c + 1] = __float_as_uint(a.y);
        d[c + 2] = __float_as_uint(b.x);
        d[c + 3] = __float_as_uint(b.y);
      }
      if (diagonal)
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c < own) d[c] = 0u;
      store_bf16(tP + mine, d, diagonal);
      tc::wait_st();
      tc::fence_before_sync();
      tc::warp_arrive(&sm.ds_ready, lead);
    }
    if (tc::warp_wait(&sm.done, 0, abort) && p.split == 1) {
      tc::fence_after_sync();
      const int64_t row = (int64_t)t.lo + key0 + r;
      const int of = part * 64 / DP, from = part * 64 % DP;  // dv or dk, 64 columns
      write_row<64>((of ? tK : tV) + lanes + from,
                    (of ? p.dk : p.dv) + (row * p.Hk + g) * p.D + from, p.D - from,
                    of ? p.scale : 1.0f, r < rows);
    }
  }
  if (p.split > 1) {
    __syncwarp();
    tc::fence_before_sync();
    cluster_barrier();  // every block is done with its tiles: their memory takes the sums
    tc::fence_after_sync();
    const int r = threadIdx.x & 127, part = warp >> 2;
    const int fours = 2 * DP / 4 / p.split;  // of the 2 DP columns (dv, dk), a block's own
    // [source][own columns, by fours][row], 16 bytes each
    if (part < PARTS) {
      const uint32_t acc = (part * 64 < DP ? tV : tK) + ((uint32_t)((warp & 3) * 32) << 16) +
                           part * 64 % DP;
      const uint32_t here = tc::smem_addr(raw) + (rank * fours * 128 + r) * 16;
#pragma unroll
      for (int c = 0; c < 64; c += 16) {
        uint32_t x[16];
        tc::ld16(acc + c, x);
        tc::wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int four = (part * 64 + c) / 4 + k;
          put_remote4(here + four % fours * 2048, four / fours, x + 4 * k);
        }
      }
    }
    tc::fence_before_sync();
    cluster_barrier();
    tc::fence_after_sync();
    if (part < PARTS && r < rows) {
      const float4 *sums = reinterpret_cast<const float4 *>(raw);
      const int64_t row = ((int64_t)t.lo + key0 + r) * p.Hk + g;
      for (int four = part; four < fours; four += PARTS) {
        float4 x = sums[four * 128 + r];
        for (int k = 1; k < p.split; ++k) {
          const float4 y = sums[(k * fours + four) * 128 + r];
          x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        const int col = (rank * fours + four) * 4, of = col >= DP, d = col - of * DP;
        const float f = of ? p.scale : 1.0f;
        if (d < p.D)
          *reinterpret_cast<uint2 *>((of ? p.dk : p.dv) + row * p.D + d) =
              make_uint2(pack_bf16(x.x * f, x.y * f), pack_bf16(x.z * f, x.w * f));
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  settle(sm.abort, p.ws);
  if (warp == kIssue) tc::tmem_dealloc(sm.tmem, 2 * IT + 2 * DP);
}

template <int DP>
struct QSmem {
  alignas(1024) unsigned char q[DP * 256], dout[DP * 256], k[3][DP * inner<DP>() * 2],
      v[2][DP * inner<DP>() * 2];
  float sum[4][128];  // of weights times dP, by the threads of a row
  uint64_t q_full, do_full, k_full[3], k_empty[3], v_full[2], v_empty[2];
  uint64_t s_full[2], dp_full, ds_ready, done;
  TileSearch search;
  uint32_t tmem;
  int abort;
};

// The warps of a dq block that share 32 query rows.
template <int PARTS>
__device__ __forceinline__ void row_barrier(int quarter) {
  asm volatile("bar.sync %0, %1;" ::"r"(quarter + 1), "n"(PARTS * 32) : "memory");
}

// dq: a block per query tile and head, over the key tiles at and before it.
// In tensor memory: S = Q K^T twice (128 columns each, dS over the one it
// came from), dP = dO V^T (128), dQ += dS K (DP). Issue order dP(j+1), dQ(j),
// S(j+2): P(j+1) is formed while dP(j+1) runs, dS(j+1) while dQ(j) and S(j+2)
// do.
template <int DP>
__global__ void __launch_bounds__(backward_threads<DP>(), DP == 64 ? 2 : 1)
    attention_dq_kernel(const __grid_constant__ CUtensorMap mq,
                        const __grid_constant__ CUtensorMap mk,
                        const __grid_constant__ CUtensorMap mv,
                        const __grid_constant__ CUtensorMap mdo, const BackwardArgs p) {
  extern __shared__ __align__(1024) unsigned char raw[];
  QSmem<DP> &sm = *reinterpret_cast<QSmem<DP> *>(raw);
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = __shfl_sync(kFull, threadIdx.x >> 5, 0);
  const int h = blockIdx.x % p.Hq;
  constexpr int IT = inner<DP>(), PARTS = IT / 32, kCopy = 4 * PARTS, kIssue = kCopy + 1;
  if (!aligned_tiles(raw, p.ws)) return;
  if (warp == kIssue) tc::tmem_alloc(&sm.tmem, 3 * IT + DP);
  find_tile(p.cu, (int)p.sequences, (int)p.tokens, blockIdx.x / p.Hq, kCopy, sm.search);
  Tile t;
  int rows, steps;  // steps: key tiles, the last one first
  auto take_tile = [&] {
    t = sm.search.tile;
    rows = t.len - t.first < kTile ? t.len - t.first : kTile;
    steps = (t.first + rows + IT - 1) / IT;
  };
  auto first_key = [&](int j) { return (steps - 1 - j) * IT; };
  auto diagonal = [&](int j) { return first_key(j) + IT > t.first; };
  auto load_k = [&](int j) {
    tc::load_tile<DP, IT>(sm.k[j % 3], &mk, &sm.k_full[j % 3], h / p.group, t.lo + first_key(j));
  };
  auto load_v = [&](int j) {
    tc::load_tile<DP, IT>(sm.v[j & 1], &mv, &sm.v_full[j & 1], h / p.group, t.lo + first_key(j));
  };
  if (warp == kCopy && lane == 0 && sm.search.found) {
    take_tile();
    for (int i = 0; i < 3; ++i) mbar_init(&sm.k_full[i], 1), mbar_init(&sm.k_empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
    }
    for (uint64_t *b : {&sm.q_full, &sm.do_full, &sm.dp_full, &sm.done}) mbar_init(b, 1);
    mbar_init(&sm.ds_ready, 4 * PARTS);
    sm.abort = 0;
    fence_mbar_init();
    tc::load_tile<DP, kTile>(sm.q, &mq, &sm.q_full, h, t.lo + t.first);
    load_k(0);
    tc::load_tile<DP, kTile>(sm.dout, &mdo, &sm.do_full, h, t.lo + t.first);
    load_v(0);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  auto clear_unheld = [&] {
    const Unheld u = unheld(p.cu, (int)p.sequences, (int)p.tokens);
    if (u.lo == 0 && u.hi == (int)p.tokens) return;
    zero_unheld(p.dq, p.Hq * p.D, u, (int)p.tokens, threadIdx.x, backward_threads<DP>() - 64);
  };
  if (!sm.search.found) {
    if (warp < kCopy) clear_unheld();
    if (warp == kIssue) tc::tmem_dealloc(sm.tmem, 3 * IT + DP);
    return;
  }
  take_tile();
  const uint32_t tmem = __shfl_sync(kFull, sm.tmem, 0);
  const uint32_t tS0 = tmem, tP = tS0 + IT, tQ = tP + IT, tS1 = tQ + DP;
  volatile int *abort = &sm.abort;
  const uint32_t lead = lane == 0;  // the lane that issues products

  if (warp == kCopy) {
    if (lane == 0) {
      for (int j = 1; j < steps; ++j) {
        if (j >= 3 && !tc::mbar_wait(&sm.k_empty[j % 3], (j / 3 - 1) & 1, abort)) break;
        load_k(j);
        if (j >= 2 && !tc::mbar_wait(&sm.v_empty[j & 1], (j / 2 - 1) & 1, abort)) break;
        load_v(j);
      }
    }
  } else if (warp == kIssue) {
    const uint32_t q = tc::smem_addr(sm.q), dout = tc::smem_addr(sm.dout);
    auto scores = [&](int j) {
      const int a = j % 3;
      if (!tc::warp_wait(&sm.k_full[a], (j / 3) & 1, abort)) return false;
      // keys past the sequence's end meet a dS of zero: they must be finite
      if (j == 0 && first_key(0) + IT > t.len)
        tc::clear_rows<DP, IT>(sm.k[a], t.len - first_key(0), lane);
      __syncwarp();
      tc::product_nt<DP, IT>(lead, j & 1 ? tS1 : tS0, q, tc::smem_addr(sm.k[a]));
      tc::commit(lead, &sm.s_full[j & 1]);
      return true;
    };
    auto grads = [&](int j) {
      const int b = j & 1;
      if (!tc::warp_wait(&sm.v_full[b], (j / 2) & 1, abort)) return false;
      tc::product_nt<DP, IT>(lead, tP, dout, tc::smem_addr(sm.v[b]));
      tc::commit(lead, &sm.dp_full);
      tc::commit(lead, &sm.v_empty[b]);
      return true;
    };
    bool ok = tc::warp_wait(&sm.q_full, 0, abort) && scores(0) &&
              tc::warp_wait(&sm.do_full, 0, abort) && grads(0) && (steps < 2 || scores(1));
    for (int j = 0; j < steps && ok; ++j) {
      ok = tc::warp_wait(&sm.ds_ready, j & 1, abort);
      if (!ok) break;
      tc::fence_after_sync();
      if (j + 1 < steps && !(ok = grads(j + 1))) break;
      const uint32_t ds = j & 1 ? tS1 : tS0, k = tc::smem_addr(sm.k[j % 3]);
      tc::product_parts<DP, IT, PARTS>(lead, tQ, ds, k, j > 0);
      if (diagonal(j)) tc::product_parts<DP, IT, PARTS>(lead, tQ, ds + 16, k, true);
      tc::commit(lead, &sm.k_empty[j % 3]);
      if (j + 1 == steps) tc::commit(lead, &sm.done);
      if (j + 2 < steps) ok = scores(j + 2);
    }
  } else {
    const int r = threadIdx.x & 127, part = warp >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, mine = lanes + part * 32;
    const int64_t row = (int64_t)t.lo + t.first + r;
    float lse = 0.0f, delta = 0.0f;
    if (r < rows) {
      lse = p.lse[(int64_t)h * p.tokens + row] * kLog2e;
      delta = p.delta[(int64_t)h * p.tokens + row];
    }
    const float2 k2 = make_float2(p.scale2, p.scale2), l2 = make_float2(-lse, -lse);
    float2 d2 = make_float2(-delta, -delta);
    clear_unheld();
    // after a wait that ran out the loop goes on without waiting, so that
    // every warp meets the others' barriers
    for (int j = 0; j < steps; ++j) {
      const uint32_t at = (j & 1 ? tS1 : tS0) + mine;
      uint32_t s[32], d[32];
      tc::warp_wait(&sm.s_full[j & 1], (j / 2) & 1, abort);
      tc::fence_after_sync();
      tc::ld32(at, s);
      tc::wait_ld();
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const float2 a = __ffma2_rn(pair(s + c), k2, l2);
        s[c] = __float_as_uint(ex2(a.x));
        s[c + 1] = __float_as_uint(ex2(a.y));
      }
      tc::warp_wait(&sm.dp_full, j & 1, abort);
      tc::fence_after_sync();
      tc::ld32(tP + mine, d);
      tc::wait_ld();
      const int last = t.first + r - first_key(j) - part * 32;  // the last column this row sees
      if (t.first == 0 && first_key(j) == 0) {
        // rows whose keys all are in this tile: delta = sum_j P_ij dP_ij, without
        // the rounding of the output, which the few weights of a short row feel
        float own = 0.0f;
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c <= last) own = fmaf(__uint_as_float(s[c]), __uint_as_float(d[c]), own);
        sm.sum[part][r] = own;
        row_barrier<PARTS>(warp & 3);
        own = 0.0f;
#pragma unroll
        for (int c = 0; c < PARTS; ++c) own += sm.sum[c][r];
        if (r < IT && r < rows) {
          d2 = make_float2(-own, -own);
          if (part == 0) p.delta[(int64_t)h * p.tokens + row] = own;  // for dk
        }
      }
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const float2 a = __fmul2_rn(pair(s + c), __fadd2_rn(pair(d + c), d2));
        d[c] = __float_as_uint(a.x);
        d[c + 1] = __float_as_uint(a.y);
      }
      if (diagonal(j))
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c > last) d[c] = 0u;
      store_bf16(at, d, diagonal(j));
      tc::wait_st();
      tc::fence_before_sync();
      tc::warp_arrive(&sm.ds_ready, lead);
    }
    if (tc::warp_wait(&sm.done, 0, abort)) {
      tc::fence_after_sync();
      const int from = part * 32;  // (DP is 32 PARTS)
      write_row<32>(tQ + lanes + from, p.dq + (row * p.Hq + h) * p.D + from, p.D - from, p.scale,
                    r < rows);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  settle(sm.abort, p.ws);
  if (warp == kIssue) tc::tmem_dealloc(sm.tmem, 3 * IT + DP);
}

// ---------------------------------------------------------------------------
// One new token per sequence. Bound by reading the cache once.
//
// A unit of work is kUnit positions of one sequence's cache for one key/value
// head. All units stand in a row (sequence, head, position), which is cut into
// equal runs, one to each of the blocks that run at once: short and long
// caches share the GPU evenly, and a block leaves at most two heads
// unfinished, at its run's ends. A second kernel joins those, in run order.
// A warp takes 16 positions at a time, copied asynchronously into its own ring
// in shared memory, as the operands of two small products:
//   S^T[16 positions x 8 rows] = K Q^T,  O^T[16 elements x 8 rows] += V^T P^T
// (rows: the query heads that share the key/value head, 8 or 16 at a time).
// Loads straight from global memory into the operands' registers leave memory
// idle while a warp computes, and their values must be paired up: 115 us where
// this takes 106 (64 caches of up to 8192, 16 heads on 4 of 128, 5.9 TB/s).
// ---------------------------------------------------------------------------
// A head that starts in one block's run and ends in a later one's; kept by
// the block after the one it starts in.
struct Unfinished {
  int b, head, last;  // key/value head x row block; the block it ends in, 0 for none
};
struct StepArgs {
  const bf *q, *k, *v;
  int64_t kb, kt, kh, vb, vt, vh;
  const int32_t *lengths;
  bf *o;
  Unfinished *list;  // [blocks]
  float *partial;    // [blocks][2: first, last][rows][D + 2]: o, running maximum, sum
  int64_t B, S;
  int Hq, Hk, D, group, row_blocks, blocks;
  float scale2;
};
constexpr int kStepWarps = 4;
constexpr int kStepThreads = kStepWarps * 32;
constexpr int kUnit = kStepWarps * 32;
constexpr size_t kListBytes = 16384;  // of the scratch, for the list of unfinished heads
// Blocks per SM. Eight rows: 3 with rings of 16 KB (64 caches of 8192, 16 heads
// on 4 of 128: 91 us; 128 of 512, 8 on 8: 33) against 2 with 24 KB (91; 36).
// Sixteen: 2 (32 of 16384, 16 on 1: 37 us) against 3, whose sums spill (58).
constexpr int step_blocks(int eights) { return eights == 1 ? 3 : 2; }

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {  // an 8 x 8 matrix over the warp
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Four 8 x 8 matrices of shared memory, the row addresses of matrix i in lanes
// 8 i to 8 i + 7, as they are or transposed.
template <bool TRANS>
__device__ __forceinline__ void matrices(uint32_t at, uint32_t (&x)[4]) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(at)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(at)
                 : "memory");
}
// 16 bytes to shared memory, or zeros (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const bf *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ int64_t cache_length(const StepArgs &p, int64_t b) {
  const int64_t n = p.lengths[b];
  return n < 0 ? 0 : (n > p.S ? p.S : n);
}
__device__ __forceinline__ int units_of(int64_t n) { return (int)((n + kUnit - 1) / kUnit); }

constexpr int kRingBytes = 16384;  // of a warp

template <int DP, int NR>
__global__ void __launch_bounds__(kStepThreads, step_blocks(NR))
    attention_step_kernel(const StepArgs p) {
  constexpr int CH = DP / 8;            // 16-byte pieces of a row
  constexpr int kHalf = 16 * DP * 2;    // bytes of a stage's keys, or values
  constexpr int kStages = kRingBytes / (2 * kHalf);
  constexpr int MT = DP / 16;           // 16 columns at a time
  extern __shared__ __align__(128) unsigned char rings[];
  __shared__ float sm[kStepWarps][NR * 8], sl[kStepWarps][NR * 8];
  __shared__ int run[2], upto[kStepWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = lane >> 2, c = lane & 3;
  const int per = p.Hk * p.row_blocks;  // heads of a sequence
  // A lane's part in copies, and the rows and pieces it addresses for the
  // matrices. Piece x of row y is kept at place x ^ (y & 7) of its row, so that
  // neither meets bank conflicts.
  constexpr int kRows = 32 / CH;  // of a copy
  const int crow = lane / CH, cpiece = lane % CH;
  const uint32_t cswizzle = (cpiece ^ crow) * 16;
  const uint32_t krow = ((lane & 7) + (lane >> 3 & 1) * 8) * DP * 2;
  const uint32_t vrow = ((lane & 7) + (lane >> 4) * 8) * DP * 2 + kHalf;
  const uint32_t kpiece = ((lane >> 4) ^ (lane & 7)) * 16;
  const uint32_t vpiece = ((lane >> 3 & 1) ^ (lane & 7)) * 16;
  const uint32_t ring = tc::smem_addr(rings) + warp * kRingBytes;
  // a run's sums, in the ring once it is empty
  static_assert(NR * 8 * (DP + 4) * 4 <= kRingBytes, "the sums fit the ring");
  auto so = [&](int w, int row, int d) -> float & {
    return reinterpret_cast<float *>(rings + w * kRingBytes)[row * (DP + 4) + d];
  };
  // count the units, a slice of the sequences to a thread, and find the
  // sequence in which this block's run starts
  const int slice = (int)(p.B * threadIdx.x / kStepThreads);
  const int slice_end = (int)(p.B * (threadIdx.x + 1) / kStepThreads);
  int own = 0, sum_to;
  for (int x = slice; x < slice_end; ++x) own += units_of(cache_length(p, x)) * per;
  sum_to = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, sum_to, o);
    if (lane >= o) sum_to += y;
  }
  if (lane == 31) upto[warp] = sum_to;
  __syncthreads();
  int units = 0;
#pragma unroll
  for (int w = 0; w < kStepWarps; ++w) {
    if (w < warp) sum_to += upto[w];
    units += upto[w];
  }
  const int block = blockIdx.x, blocks = units < p.blocks ? units : p.blocks;  // that have a run
  auto run_start = [&](int i) { return (int)((int64_t)units * i / blocks); };
  const int start = block < blocks ? run_start(block) : units;
  if (start >= sum_to - own && start < sum_to) run[0] = slice, run[1] = sum_to - own;
  if (threadIdx.x == 0) p.list[block].last = 0;
  // nothing cached: zeros
  for (int64_t x = block; x < p.B; x += p.blocks)
    if (cache_length(p, x) == 0)
      for (int y = threadIdx.x; y < p.Hq * p.D; y += kStepThreads)
        p.o[x * p.Hq * p.D + y] = __float2bfloat16_rn(0.0f);
  __syncthreads();
  if (block >= blocks) return;
  const int end = run_start(block + 1);
  int b = run[0], before = run[1];  // the sequence a unit is in, units of those before it
  for (int unit = start; unit < end;) {
    const int64_t n = cache_length(p, b);
    const int of_head = units_of(n);
    if (unit >= before + of_head * per) {
      before += of_head * per;
      ++b;
      continue;
    }
    const int head = (unit - before) / of_head, t0 = (unit - before) % of_head;
    const int t1 = t0 + (end - unit) < of_head ? t0 + (end - unit) : of_head;
    unit += t1 - t0;
    const int g = head / p.row_blocks, r0 = head % p.row_blocks * (NR * 8);
    const int64_t from = (int64_t)t0 * kUnit;
    const int64_t to = (int64_t)t1 * kUnit < n ? (int64_t)t1 * kUnit : n;

    // queries: row e of each block of 8, as the second operand
    uint32_t q[NR][MT][2];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = r0 + r * 8 + e, col = m * 16 + i * 8 + c * 2;
          const bf *at = p.q + ((int64_t)b * p.Hq + g * p.group + row) * p.D + col;
          q[r][m][i] =
              row < p.group && col < p.D ? __ldg(reinterpret_cast<const uint32_t *>(at)) : 0u;
        }
    const bf *k = p.k + b * p.kb + g * p.kh, *v = p.v + b * p.vb + g * p.vh;
    // copy 16 positions; rows past the end and columns past D are zeros
    auto fetch = [&](int64_t pos, int stage) {
      if (pos < to) {
        const int left = cpiece * 8 < p.D ? (int)(to - pos < 16 ? to - pos : 16) - crow : 0;
        const bf *kp = k + (pos + crow) * p.kt + cpiece * 8;
        const bf *vp = v + (pos + crow) * p.vt + cpiece * 8;
        const uint32_t at = ring + stage * 2 * kHalf + crow * DP * 2;
#pragma unroll
        for (int j = 0; j < 16; j += kRows, kp += kRows * p.kt, vp += kRows * p.vt) {
          const uint32_t dst = at + j * DP * 2 + (cswizzle ^ ((j & 7) * 16));
          copy16(dst, j < left ? kp : k, j < left);
          copy16(dst + kHalf, j < left ? vp : v, j < left);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    float acc[NR][MT][4] = {};
    float top[NR][2], sum[NR][2];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int i = 0; i < 2; ++i) top[r][i] = -INFINITY, sum[r][i] = 0.0f;
    constexpr int kStride = kStepWarps * 16;
    int stage = 0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(from + warp * 16 + i * kStride, i);
    for (int64_t pos = from + warp * 16; pos < to; pos += kStride) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();  // these 16 are here, and every lane is done with the stage filled next
      fetch(pos + (kStages - 1) * kStride, stage == 0 ? kStages - 1 : stage - 1);
      const uint32_t keys = ring + stage * 2 * kHalf + krow;
      const uint32_t values = ring + stage * 2 * kHalf + vrow;
      stage = stage == kStages - 1 ? 0 : stage + 1;
      float s[NR][4] = {};
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint32_t x[4];
        matrices<false>(keys + (kpiece ^ (m * 32)), x);
#pragma unroll
        for (int r = 0; r < NR; ++r) mma16816(s[r], x[0], x[1], x[2], x[3], q[r][m][0], q[r][m][1]);
      }
      // weights: rows 2c and 2c + 1, positions e and e + 8. The maximum is
      // raised only when a score passes it by 2^8 (or is the first).
      uint32_t w[NR][2];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s[r][i] = pos + (i >> 1) * 8 + e < to ? s[r][i] * p.scale2 : -INFINITY;
        float hi[2] = {fmaxf(s[r][0], s[r][2]), fmaxf(s[r][1], s[r][3])};
        if (__any_sync(kFull, hi[0] > top[r][0] + 8.0f || hi[1] > top[r][1] + 8.0f)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) hi[i] = fmaxf(hi[i], __shfl_xor_sync(kFull, hi[i], o));
            hi[i] = fmaxf(hi[i], top[r][i]);
            const float f = hi[i] == -INFINITY ? 1.0f : ex2(top[r][i] - hi[i]);
            top[r][i] = hi[i];
            sum[r][i] *= f;
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[r][m][i] *= f, acc[r][m][2 + i] *= f;
          }
        }
        const float z[2] = {top[r][0] == -INFINITY ? 0.0f : top[r][0],
                            top[r][1] == -INFINITY ? 0.0f : top[r][1]};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x = ex2(s[r][2 * i] - z[0]), y = ex2(s[r][2 * i + 1] - z[1]);
          sum[r][0] += x;
          sum[r][1] += y;
          w[r][i] = transposed(pack_bf16(x, y));
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint32_t x[4];
        matrices<true>(values + (vpiece ^ (m * 32)), x);
#pragma unroll
        for (int r = 0; r < NR; ++r) mma16816(acc[r][m], x[0], x[1], x[2], x[3], w[r][0], w[r][1]);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    // join the warps: rows 2c and 2c + 1 of each block
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) sum[r][i] += __shfl_xor_sync(kFull, sum[r][i], o);
        if (e == 0) {
          sm[warp][r * 8 + 2 * c + i] = top[r][i];
          sl[warp][r * 8 + 2 * c + i] = sum[r][i];
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = m * 16 + (i >> 1) * 8 + e;
          so(warp, r * 8 + 2 * c + (i & 1), d) = acc[r][m][i];
        }
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == of_head;
    if (t0 > 0 && threadIdx.x == 0) {
      // t0 > 0 at the run's start alone; unit x is in run ((x + 1) * blocks - 1) / units
      const int head0 = before + head * of_head;
      if (run_start(block - 1) <= head0)
        p.list[block] = {b, head, (int)(((int64_t)(head0 + of_head) * blocks - 1) / units)};
    }
    for (int x = threadIdx.x; x < NR * 8 * DP; x += kStepThreads) {
      const int row = x / DP, d = x % DP;
      if (r0 + row >= p.group || d >= p.D) continue;
      float m = sm[0][row];
#pragma unroll
      for (int y = 1; y < kStepWarps; ++y) m = fmaxf(m, sm[y][row]);
      float l = 0.0f, o = 0.0f;
#pragma unroll
      for (int y = 0; y < kStepWarps; ++y) {
        const float f = sm[y][row] == -INFINITY ? 0.0f : ex2(sm[y][row] - m);
        l = fmaf(f, sl[y][row], l);
        if (f != 0.0f) o = fmaf(f, so(y, row, d), o);
      }
      const int64_t at = b * p.Hq + g * p.group + r0 + row;
      if (whole) {
        p.o[at * p.D + d] = __float2bfloat16_rn(o / l);
      } else {
        float *out = p.partial + ((int64_t)(2 * block + (t0 == 0)) * (NR * 8) + row) * (p.D + 2);
        out[d] = o;
        if (d == 0) out[p.D] = m, out[p.D + 1] = l;
      }
    }
    __syncthreads();
  }
}

// Join the heads that no block finished, blockIdx.x counting them in the list's
// order: that of block i starts in run i - 1 and goes on in run i. SPLIT warps
// share a row's runs; a lane has columns 2 lane, 2 lane + 1 and those + 64.
constexpr int kJoinWarps = 8;
template <int SPLIT>
__global__ void __launch_bounds__(kJoinWarps * 32)
    attention_step_join_kernel(const StepArgs p, int rows) {
  __shared__ int upto[kJoinWarps], entry;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // two entries of the list to a thread
  const int mine = 2 * threadIdx.x + 1;
  const bool a = mine < p.blocks && p.list[mine].last != 0;
  const bool b = mine + 1 < p.blocks && p.list[mine + 1].last != 0;
  const unsigned as = __ballot_sync(kFull, a), bs = __ballot_sync(kFull, b);
  if (lane == 0) upto[warp] = __popc(as) + __popc(bs);
  if (threadIdx.x == 0) entry = 0;
  __syncthreads();
  const unsigned below = (1u << lane) - 1;
  int before = __popc(as & below) + __popc(bs & below);
  for (int w = 0; w < warp; ++w) before += upto[w];
  if (a && before == (int)blockIdx.x) entry = mine;
  if (b && before + a == (int)blockIdx.x) entry = mine + 1;
  __syncthreads();
  const int i = entry;
  if (i == 0) return;
  const Unfinished u = p.list[i];
  const int runs = u.last - i + 2, g = u.head / p.row_blocks;
  const int row = blockIdx.y * (kJoinWarps / SPLIT) + warp / SPLIT;
  const int at = u.head % p.row_blocks * rows + row;  // of the group's query heads
  const bool on = at < p.group;
  float m = -INFINITY, l = 0.0f, o[4] = {};
  // 32 runs at a time: their weights, one to a lane, then their sums
  for (int k0 = warp % SPLIT; on && k0 < runs; k0 += 32 * SPLIT) {
    // the first run's last place, then the others' first
    auto place = [&](int k) {
      return p.partial + ((int64_t)(2 * (i - 1 + k) + (k == 0)) * rows + row) * (p.D + 2);
    };
    const int k = k0 + lane * SPLIT;
    const float2 own = k < runs ? *reinterpret_cast<const float2 *>(place(k) + p.D)
                                : make_float2(-INFINITY, 0.0f);
    float high = own.x;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) high = fmaxf(high, __shfl_xor_sync(kFull, high, x));
    high = fmaxf(high, m);
    const float z = high == -INFINITY ? 0.0f : high, f = ex2(m - z), w = ex2(own.x - z);
    m = high;
    float t = own.y * w;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) t += __shfl_xor_sync(kFull, t, x);
    l = fmaf(l, f, t);
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] *= f;
    const int n = (runs - k0 + SPLIT - 1) / SPLIT < 32 ? (runs - k0 + SPLIT - 1) / SPLIT : 32;
#pragma unroll 8
    for (int y = 0; y < n; ++y) {
      const float h = __shfl_sync(kFull, w, y);
      const float *in = place(k0 + y * SPLIT);
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (x * 64 + 2 * lane < p.D) {
          const float2 q = *reinterpret_cast<const float2 *>(in + x * 64 + 2 * lane);
          o[2 * x] = fmaf(h, q.x, o[2 * x]);
          o[2 * x + 1] = fmaf(h, q.y, o[2 * x + 1]);
        }
    }
  }
  if constexpr (SPLIT > 1) {  // the row's warps, in order
    static_assert(SPLIT == kJoinWarps, "a block has one row");
    __shared__ float parts[SPLIT][32][4], stats[SPLIT][2];
#pragma unroll
    for (int x = 0; x < 4; ++x) parts[warp][lane][x] = o[x];
    if (lane == 0) stats[warp][0] = m, stats[warp][1] = l;
    __syncthreads();
    if (warp > 0) return;
    for (int w = 1; w < SPLIT; ++w) m = fmaxf(m, stats[w][0]);
    const float z = m == -INFINITY ? 0.0f : m;
    l = o[0] = o[1] = o[2] = o[3] = 0.0f;
    for (int w = 0; w < SPLIT; ++w) {
      const float f = ex2(stats[w][0] - z);
      l = fmaf(f, stats[w][1], l);
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] = fmaf(f, parts[w][lane][x], o[x]);
    }
  }
  bf *out = p.o + ((int64_t)u.b * p.Hq + g * p.group + at) * p.D;
#pragma unroll
  for (int x = 0; x < 2; ++x)
    if (on && x * 64 + 2 * lane < p.D)
      *reinterpret_cast<uint32_t *>(out + x * 64 + 2 * lane) =
          pack_bf16(o[2 * x] / l, o[2 * x + 1] / l);
}

// Query heads to a row block, and blocks of a call: no more than run at once.
int step_rows(int64_t group) { return group <= 8 ? 8 : 16; }
int64_t step_heads(int64_t B, int64_t Hq, int64_t Hk) {
  const int64_t group = Hq / Hk;
  return B * Hk * ceil_div(group, step_rows(group));
}
bool step_fits(int64_t B, int64_t S, int64_t Hq, int64_t Hk) {  // units are counted in 32 bits
  return product_fits(B, Hq, S / kUnit + 1) &&
         step_heads(B, Hq, Hk) * ceil_div(S, kUnit) < (int64_t)INT32_MAX;
}
int step_grid(int64_t B, int64_t S, int64_t Hq, int64_t Hk) {
  const int64_t most = kSms * step_blocks(step_rows(Hq / Hk) / 8);
  const int64_t units = step_heads(B, Hq, Hk) * ceil_div(S, kUnit);
  return (int)(units < 1 ? 1 : units < most ? units : most);
}

template <int DP, int NR>
cudaError_t launch_step(const StepArgs &a, cudaStream_t st) {
  constexpr size_t smem = (size_t)kStepWarps * kRingBytes;
  cudaError_t e = allow_dynamic_smem<attention_step_kernel<DP, NR>>(smem);
  if (e == cudaSuccess)
    e = launch_ex(attention_step_kernel<DP, NR>, dim3((unsigned)a.blocks),
                  dim3(kStepThreads), smem, st,
                  true, a);
  if (e != cudaSuccess || a.blocks == 1) return e;
  // A warp to each of a head's rows, or, where a head is left in more than 8
  // runs, a block: with 4 caches of 65536, 16 heads on 1 (76 runs to a row) 11
  // us, and 22 by four warps; with 32 of 16384, 24 on 2 (5 runs) warps take 9
  // us and one block that goes over the rows 28.
  const int64_t heads = a.B * a.Hk * a.row_blocks, most = a.blocks - 1;
  const unsigned x = (unsigned)(heads < most ? heads : most);
  const dim3 threads(kJoinWarps * 32);
  return heads * 8 < a.blocks
             ? launch_ex(attention_step_join_kernel<kJoinWarps>, dim3(x, NR * 8), threads, 0, st,
                         true, a, NR * 8)
             : launch_ex(attention_step_join_kernel<1>, dim3(x, NR), threads, 0, st, true, a,
                         NR * 8);
}

// Token and head strides that 16-byte loads can use.
rlcs_status strides_usable(const void *p, int64_t ts, int64_t hs, int64_t tokens, int64_t heads) {
  if (ts < 0 || hs < 0 || !product_fits(tokens, ts, 1) || !product_fits(heads, hs, 1))
    return RLCS_ERR_INVALID_ARG;
  return ts % 8 == 0 && hs % 8 == 0 && aligned(p, 16) ? RLCS_OK : RLCS_ERR_MISALIGNED;
}

bool attn_sizes(int64_t sequences, int64_t tokens, int64_t Hq, int64_t Hk, int64_t D, double scale,
                rlcs_dtype t) {
  return sequences >= 0 && tokens >= 0 && tokens <= INT32_MAX &&
         sequences < INT32_MAX - 1024 && Hq > 0 && Hk > 0 && Hq % Hk == 0 && D > 0 && D <= 128 && D % 8 == 0 && t == RLCS_BF16 &&
         scale >= 1e-30 && scale <= 1e30 && product_fits(tokens, Hq, D) &&
         tile_bound(sequences, tokens) * Hq < (int64_t)INT32_MAX &&
         tokens * Hq < (int64_t)4 * INT32_MAX;
}

template <int DP>
cudaError_t launch_forward(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                           const ForwardArgs &a, int64_t grid, cudaStream_t st) {
  constexpr size_t smem = sizeof(ForwardSmem<DP>);
  const cudaError_t e = allow_dynamic_smem<attention_kernel<DP>>(smem);
  if (e != cudaSuccess) return e;
  return launch_ex(attention_kernel<DP>, dim3((unsigned)grid), dim3(320), smem, st, true, mq, mk,
                   mv, a);
}

// Blocks that share a group's query heads: the fewest, of the powers of two
// that divide the group, that make up a block per SM. (8192 tokens, 8 heads on 1
// of 128, 64 key tiles: 306 us with 4 to a tile, 1117 with one; 2 x 4096, 16 on
// 4, 256 tiles: 222 with one against 289 with 4.)
int group_split(int64_t blocks, int group) {
  int split = 1;
  while (split < 8 && group % (2 * split) == 0 && blocks * split < kSms) split *= 2;
  return split;
}

struct BackwardMaps {
  CUtensorMap q, k, v, dout;
};

template <int DP>
cudaError_t launch_backward(const BackwardMaps &stay, const BackwardMaps &walk,
                            const BackwardArgs &a, int64_t tiles, cudaStream_t st) {
  constexpr int kRows = 4 * 256 / (DP / 8);  // of delta, to a block
  cudaError_t e = launch_ex(attention_delta_kernel<DP>,
                            dim3((unsigned)ceil_div(a.tokens * a.Hq, kRows)), dim3(256), 0, st, true,
                            a.dout, a.out, a.delta, a.tokens, a.Hq, a.D);
  if (e != cudaSuccess) return e;
  constexpr size_t kv_smem = sizeof(KvSmem<DP>), q_smem = sizeof(QSmem<DP>);
  static_assert(kv_smem <= 232448 && q_smem <= 232448, "a block has 227 KB of shared memory");
  e = allow_dynamic_smem<attention_dkv_kernel<DP>>(kv_smem);
  if (e == cudaSuccess) e = allow_dynamic_smem<attention_dq_kernel<DP>>(q_smem);
  if (e != cudaSuccess) return e;
  // dq first: it leaves delta without the output's rounding for short rows
  e = launch_ex(attention_dq_kernel<DP>, dim3((unsigned)(tiles * a.Hq)),
                dim3(backward_threads<DP>()), q_smem, st, true, stay.q, walk.k, walk.v, stay.dout, a);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * a.Hk * a.split));
  cfg.blockDim = dim3(backward_threads<DP>());
  cfg.dynamicSmemBytes = kv_smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, attention_dkv_kernel<DP>, walk.q, stay.k, stay.v, walk.dout, a);
}

}  // namespace
}  // namespace seq
}  // namespace rlcs

using namespace rlcs;
using namespace rlcs::seq;

extern "C" {

rlcs_status rlcs_attention_status(void) {
  uint32_t code = 0, linear = 0;
  const uint32_t none = 0;
  uint32_t *other = linear_status();
  if (cudaDeviceSynchronize() != cudaSuccess || !other ||
      cudaMemcpyFromSymbol(&code, device_status, sizeof(code)) != cudaSuccess ||
      cudaMemcpy(&linear, other, sizeof(linear), cudaMemcpyDeviceToHost) != cudaSuccess ||
      (code && cudaMemcpyToSymbol(device_status, &none, sizeof(none)) != cudaSuccess) ||
      (linear && cudaMemset(other, 0, sizeof(linear)) != cudaSuccess)) {
    cudaGetLastError();
    return RLCS_ERR_CUDA;
  }
  return static_cast<rlcs_status>(code > linear ? code : linear);
}

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
  CUtensorMap mq, mk, mv;
  const int it = D <= 64 ? inner<64>() : inner<128>();
  if (!tc::make_map(&mq, q, tokens, Hq, D, q_token_stride, q_head_stride, kTile) ||
      !tc::make_map(&mk, k, tokens, Hk, D, k_token_stride, k_head_stride, it) ||
      !tc::make_map(&mv, v, tokens, Hk, D, v_token_stride, v_head_stride, it))
    return RLCS_ERR_CUDA;
  const ForwardArgs a = {cu_seqlens,
                         static_cast<const bf *>(v),
                         v_token_stride,
                         v_head_stride,
                         static_cast<bf *>(out),
                         lse,
                         static_cast<WsHeader *>(scratch),
                         sequences,
                         tokens,
                         (int)Hq,
                         (int)(Hq / Hk),
                         (int)D,
                         (float)(scale * 1.4426950408889634)};
  const int64_t grid = tile_bound(sequences, tokens) * Hq;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return launched(D <= 64 ? launch_forward<64>(mq, mk, mv, a, grid, st)
                          : launch_forward<128>(mq, mk, mv, a, grid, st));
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
  // tiles that stay (128 rows) and tiles a block walks over, of each array
  BackwardMaps stay, walk;
  for (int w = 0; w < 2; ++w) {
    BackwardMaps &m = w ? walk : stay;
    const int rows = w && D <= 64 ? inner<64>() : kTile;
    if (!tc::make_map(&m.q, q, tokens, Hq, D, q_token_stride, q_head_stride, rows) ||
        !tc::make_map(&m.k, k, tokens, Hk, D, k_token_stride, k_head_stride, rows) ||
        !tc::make_map(&m.v, v, tokens, Hk, D, v_token_stride, v_head_stride, rows) ||
        !tc::make_map(&m.dout, dout, tokens, Hq, D, Hq * D, D, rows))
      return RLCS_ERR_CUDA;
  }
  float *delta = reinterpret_cast<float *>(static_cast<char *>(scratch) + 64);
  const BackwardArgs a = {cu_seqlens,
                          static_cast<const bf *>(dout),
                          static_cast<const bf *>(out),
                          lse,
                          delta,
                          static_cast<bf *>(dq),
                          static_cast<bf *>(dk),
                          static_cast<bf *>(dv),
                          static_cast<WsHeader *>(scratch),
                          sequences,
                          tokens,
                          (int)Hq,
                          (int)Hk,
                          (int)(Hq / Hk),
                          (int)D,
                          group_split(tile_bound(sequences, tokens) * Hk, (int)(Hq / Hk)),
                          (float)scale,
                          (float)(scale * 1.4426950408889634)};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t tiles = tile_bound(sequences, tokens);
  return launched(D <= 64 ? launch_backward<64>(stay, walk, a, tiles, st)
                          : launch_backward<128>(stay, walk, a, tiles, st));
}

size_t rlcs_attention_step_scratch_bytes(int64_t B, int64_t S, int64_t Hq, int64_t Hk, int64_t D) {
  if (B <= 0 || S < 0 || Hq <= 0 || Hk <= 0 || Hk > Hq || D <= 0 || D > 128 ||
      !step_fits(B, S, Hq, Hk))
    return 16;
  const size_t rows = (size_t)step_grid(B, S, Hq, Hk) * 2 * step_rows(Hq / Hk);
  return kListBytes + rows * (size_t)(D + 2) * 4;
}

rlcs_status rlcs_attention_step(const void *q, const void *k_cache, int64_t k_batch_stride,
                                int64_t k_position_stride, int64_t k_head_stride,
                                const void *v_cache, int64_t v_batch_stride,
                                int64_t v_position_stride, int64_t v_head_stride,
                                const int32_t *lengths, void *out, int64_t B, int64_t S,
                                int64_t Hq, int64_t Hk, int64_t D, double scale, rlcs_dtype dtype,
                                void *scratch, size_t scratch_bytes, rlcs_stream_t stream) {
  if (B < 0 || S < 0 || !attn_sizes(0, B, Hq, Hk, D, scale, dtype) ||
      B * Hq >= (int64_t)INT32_MAX || !step_fits(B, S, Hq, Hk) ||
      !product_fits(B, k_batch_stride < 0 ? 0 : k_batch_stride, 1) ||
      !product_fits(B, v_batch_stride < 0 ? 0 : v_batch_stride, 1) || k_batch_stride < 0 ||
      v_batch_stride < 0)
    return RLCS_ERR_INVALID_ARG;
  static_assert(kSms * 3 <= 2 * kJoinWarps * 32 && kSms * 3 * sizeof(Unfinished) <= kListBytes,
                "an entry to each block, a thread of the join to two");
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
  a.Hq = (int)Hq;
  a.Hk = (int)Hk;
  a.D = (int)D;
  a.group = (int)(Hq / Hk);
  a.row_blocks = (int)ceil_div(a.group, step_rows(a.group));
  a.blocks = step_grid(B, S, Hq, Hk);
  a.list = static_cast<Unfinished *>(scratch);
  a.partial = reinterpret_cast<float *>(static_cast<char *>(scratch) + kListBytes);
  a.scale2 = (float)(scale * 1.4426950408889634);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a.group <= 8)
    return launched(D <= 64 ? launch_step<64, 1>(a, st) : launch_step<128, 1>(a, st));
  return launched(D <= 64 ? launch_step<64, 2>(a, st) : launch_step<128, 2>(a, st));
}

}  // extern "C"
