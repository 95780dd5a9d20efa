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
#include "tensor_core.cuh"

namespace rlcs {
namespace seq {
namespace {

using bf = __nv_bfloat16;

struct View {  // [tokens, heads, D]
  const bf *p;
  int64_t token, head;
};

// ---------------------------------------------------------------------------
// Where a block works: segments of `length` tokens (a multiple of 128) of each
// sequence. Segment j of sequence s has slot cu[s] / length + s + j: slots of
// different sequences do not meet, and no sums over the sequences are needed.
// ---------------------------------------------------------------------------
constexpr int kChunk = 128;  // tokens whose weights are formed together

struct Segment {
  int seq, lo, len;      // the sequence's first token and length
  int first, rows;       // the segment in it
  bool any;
};
__device__ __forceinline__ int bound(const int32_t *cu, int64_t i, int tokens) {
  const int b = __ldg(cu + i);
  return b < 0 ? 0 : (b < tokens ? b : tokens);
}
__device__ __forceinline__ int slot_of(int lo, int seq, int length) { return lo / length + seq; }
// One warp: the last sequence whose first slot is not past `slot`, by 32 probes
// a round.
__device__ __forceinline__ Segment find_segment(const int32_t *cu, int sequences, int tokens,
                                                int slot, int length) {
  const int lane = threadIdx.x & 31;
  int from = 0, count = sequences;  // the sequence is in [from, from + count)
  while (count > 1) {
    const int step = (count + 31) / 32, at = from + lane * step;
    const bool on = lane * step < count && slot_of(bound(cu, at, tokens), at, length) <= slot;
    const unsigned b = __ballot_sync(kFull, on);
    const int last = b ? 31 - __clz(b) : 0;
    from += last * step;
    count = count - last * step < step ? count - last * step : step;
  }
  Segment g;
  g.seq = from;
  g.lo = bound(cu, from, tokens);
  const int hi = bound(cu, from + 1, tokens);
  g.len = hi > g.lo ? hi - g.lo : 0;
  const int64_t first = (int64_t)(slot - slot_of(g.lo, from, length)) * length;
  g.any = first >= 0 && first < g.len;
  g.first = g.any ? (int)first : 0;
  g.rows = g.any ? (g.len - g.first < length ? g.len - g.first : length) : 0;
  return g;
}
// The whole of sequence `seq`.
__device__ __forceinline__ Segment whole_sequence(const int32_t *cu, int tokens, int seq) {
  Segment g;
  g.seq = seq;
  g.lo = bound(cu, seq, tokens);
  const int hi = bound(cu, seq + 1, tokens);
  g.len = hi > g.lo ? hi - g.lo : 0;
  g.first = 0;
  g.rows = g.len;
  g.any = g.len > 0;
  return g;
}
// Sequences that are not cut, the longest first, in shared memory: a block's
// threads count for each how many come before it. (Packed episodes of up to 1024,
// forward and gradient, against their own order: 48, 12 heads of 64 on 4: 45 and 124
// us, 59 and 165; 128, 16 heads of 128 on 4: 161 and 415, 211 and 523.) Of more than
// 128 the order does not fit beside the tiles, and a caller may sort them: 129 take
// 213 and 535 us as they come, 163 and 422 longest first; 256 take 366 and 945, 316
// and 808.
constexpr int kOrdered = 128;
__device__ __forceinline__ void order_sequences(const int32_t *cu, int sequences, int tokens,
                                                int *len, uint8_t *order) {
  const int t = threadIdx.x;
  int own = 0;
  if (t < sequences) {
    const int lo = bound(cu, t, tokens), hi = bound(cu, t + 1, tokens);
    len[t] = own = hi > lo ? hi - lo : 0;
  }
  __syncthreads();
  if (t < sequences) {
    int before = 0;
    for (int i = 0; i < sequences; ++i) before += len[i] > own || (len[i] == own && i < t);
    order[before] = (uint8_t)t;
  }
  __syncthreads();
}
int64_t slots(int64_t sequences, int64_t tokens, int64_t length) {
  return tokens / length + sequences;
}

// a^n for a = 2^l2; 1 for n = 0 whatever a is.
__device__ __forceinline__ float power(float l2, int n) {
  return n == 0 ? 1.0f : exp2f(l2 * (float)n);
}
constexpr float kLog2e = 1.4426950408889634f;

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
__device__ __forceinline__ float2 pair(const uint32_t *r) {
  return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The highest code that a call has recorded on this device.
__device__ uint32_t device_status;

// ---------------------------------------------------------------------------
// The walk in chunks of 128 tokens. A unit of work is a segment and one or more
// heads of x that read the same state, of one chunk at least: the warp that
// issues products looks a unit ahead, and no further, or it would wait for a
// place that it has to give up itself. The grid has a block to each; one that
// runs takes over units of blocks that have not started, and what it copies in
// runs ahead into the next unit.
//
// Per chunk, with rows r of x and c of y and z, d = r - c (c - r backwards),
//   P = X Y^T,  P' = P a^d for d >= 0 and 0 elsewhere,
//   O1 = P' Z,  O2 = X S,  out = O1 + a^into O2,  S = a^n S + (a^left Y)^T Z,
// into the steps from the state to a row, left those from a row to the state.
// Forwards a chunk has one Y and Z and `nx` X (an item each, with a result of
// its own); backwards one X and `ny` Y and Z (items that add up).
// Warps 0..7 turn P into P' and sums into results, two threads to a row; warps
// 8..15 scale Y in place, decay S and hand its rounding to bfloat16 to the next
// chunk. Warp 16 copies in, warp 18 out, warp 17 issues products. In tensor
// memory, float32: P (P' over it), O1, O2, S. Rounded to bfloat16, the type of
// the products' operands: P', the scaled Y and S as an operand; S itself is not.
// Results are within 2.7e-3 of 64 bits (2-norm) where rounding them alone makes
// 1.7e-3. With each of the three in two parts that is 1.7e-3, and 8 x 4096 training
// takes 693 us for 388, packed episodes of 64-wide heads 251 for 179: three products
// more, and parts that take turns in the shared memory that is left. (S alone in two
// parts: 2.3e-3; 497 and 196 us.)
//
// 8 x 4096, 16 heads of 128: 101 us, 5.3 TB/s, on the 128 SMs that have work; a
// chunk takes 3900 clocks when its tiles are there, and 5300 as they come. What
// a chunk spent its time on, by clocks stamped in the kernel: decays from a
// table for each element 1900 clocks (a product of two powers: 1100), results
// stored by rows 3500 (through a tile and the tensor copy: 1300), the state by
// way of registers 2900 (in tensor memory: 1000). The smallest time is that of
// shared memory, which gives 128 bytes a clock: products read 224 KB a chunk,
// copies and the scaling move 190 more, 3300 clocks. Fetching tiles to L2 some
// chunks ahead made it slower (394 -> 482 us, training).
// ---------------------------------------------------------------------------
struct WalkArgs {
  const float *log_decay;
  const int32_t *cu;
  const float *init;   // [slots or sequences, Hk, D, D] or null
  // Backwards dv and dk are two walks over the same queries, gradients and
  // states: the units of one segment stand side by side in the grid, so that
  // the second finds in L2 what the first has read, and the end of one walk
  // leaves no SM idle (gradient of 48 packed episodes 118 us, in two launches 141;
  // of 8 x 4096, 16 heads of 128, 292 and 303).
  int walks;           // 1, or 2
  bf *out[2];          // [tokens, heads of x, D]
  View x[2], y[2], z[2];
  bool transposed[2];  // init is [z's dimension, y's]
  int64_t sequences, tokens;
  int heads, group;    // heads of x; of x to a state
  int nx, ny;          // a block's heads of x; heads of y and z to a state
  int D, length;       // of a segment
  bool by_slot;        // init is by slot, else by sequence
  float in_scale, out_scale;  // of y z^T, and of x S
};
struct WalkMaps {
  CUtensorMap x, y, z, out;
};

struct Unit {
  Segment g;
  int slot, h0;             // the first head of x
  int walk;
  bool end;                 // no unit: the block is done
  // Powers of the decay, and what weights are multiplied by: decays d steps long
  // at 31 + d, zeros before them; and the columns' part of them in a block of 16.
  // A growing decay may be infinite at more steps than a segment of one chunk
  // has weights for, and there are zeros: backwards a row meets columns past the
  // segment's end, where P is 0, and without a state to begin with the last row
  // takes in nothing by one step more than its longest weight. (Where another
  // chunk follows, its weights are as long.)
  float power[kChunk + 1];
  float decay[31 + kChunk];
  alignas(16) float near[16];
};
template <int DP>
constexpr int stages() {  // of the rings of tiles
  return DP == 64 ? 4 : 2;
}
template <int DP>
struct WalkSmem {
  static constexpr int kStages = stages<DP>();
  // (z after y: with 64 columns a product reads past y, into rows of its result
  // that are not used)
  alignas(1024) unsigned char x[kStages][DP * 256], y[kStages][DP * 256], z[kStages][DP * 256],
      s[DP * DP * 2];
  Unit unit[2];
  alignas(16) uint4 answer[2];  // of the requests for a unit
  uint64_t asked[2], unit_full[2], unit_empty[2];
  uint64_t x_full[kStages], x_empty[kStages], y_full[kStages], y_empty[kStages];
  uint64_t result[kStages];  // a chunk's results are in the place of its x
  uint64_t odd[kStages][8];  // to a warp: columns of them without P' Z, see add_seen
  uint64_t p_full[2], p_ready[2], y_used[2], y_ready[2], o_full, o_free, u_full, s_ready, s_used;
  uint8_t order[kOrdered];
  uint32_t tmem;
  int abort;
};
constexpr int kWalkThreads = 19 * 32;

__device__ __forceinline__ void settle(int abort) {
  if (!abort) return;
  for (int i = 0; i < 1000; ++i) __nanosleep(2000);
  if (threadIdx.x == 0) atomicMax(&device_status, (uint32_t)RLCS_ERR_TIMEOUT);
}

// A = Y in shared memory, its columns the rows of the product.
template <int DP>
__device__ __forceinline__ void product_tn(uint32_t lead, uint32_t d, uint32_t y, uint32_t z,
                                           bool add) {
  const uint32_t a = tc::operand_n<kChunk>(y), b = tc::operand_n<kChunk>(z);
#pragma unroll
  for (int k = 0; k < kChunk / 16; ++k)
    tc::mma_ss(lead, d, a + k * (2048 >> 4), b + k * (2048 >> 4),
               tc::instr(DP, true) | (1u << 15), add || k > 0);
}
// X [128 x DP] S [DP x DP]
template <int DP>
__device__ __forceinline__ void product_state(uint32_t lead, uint32_t d, uint32_t x, uint32_t s) {
  const uint32_t a = tc::operand_k(x), b = tc::operand_n<DP>(s);
#pragma unroll
  for (int k = 0; k < DP / 16; ++k)
    tc::mma_ss(lead, d, a + (((k / 4) * 16384 + (k % 4) * 32) >> 4), b + k * (2048 >> 4),
               tc::instr(DP, true), k > 0);
}

// A factor as two bf16 parts, each twice: v f = v high + v low, rounded to
// bf16 once but for the rounding of v low, 2^-9 of the other.
struct Factor {
  __nv_bfloat162 high, low;
};
__device__ __forceinline__ Factor factor(float f) {
  const __nv_bfloat16 h = __float2bfloat16_rn(f), l = __float2bfloat16_rn(f - __bfloat162float(h));
  return {__bfloat162bfloat162(h), __bfloat162bfloat162(l)};
}
__device__ __forceinline__ uint4 scaled(uint4 v, const Factor &f) {
  __nv_bfloat162 *x = reinterpret_cast<__nv_bfloat162 *>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __hfma2(x[i], f.high, __hmul2(x[i], f.low));
  return v;
}

// A box of a tile of results to its place.
__device__ __forceinline__ void store_box(const void *from, const CUtensorMap *map, int col,
                                          int head, int token) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          map),
      "r"(tc::smem_addr(from)), "r"(col), "r"(head), "r"(token)
      : "memory");
}

// Rows of out that no sequence holds, [0, lo) and [hi, tokens): share number
// `share` of `shares`, by a warp.
__device__ __noinline__ void zero_unheld(bf *out, int width, int lo, int hi, int tokens,
                                         int64_t share, int64_t shares) {
  const int eights = width / 8;
  const int64_t n = ((int64_t)lo + tokens - hi) * eights;
  for (int64_t i = share * 32 + (threadIdx.x & 31); i < n; i += shares * 32) {
    const int64_t row = i / eights;
    reinterpret_cast<uint4 *>(out + (row < lo ? row : row - lo + hi) * width)[i % eights] =
        make_uint4(0, 0, 0, 0);
  }
}

// Of row r of a tile, where column col's word of 16 bytes lies.
__device__ __forceinline__ int place(int r, int col) {
  return col / 64 * 16384 + r * 128 + ((col % 64 / 8 ^ (r & 7)) * 16);
}
// A tile's product P' Z adds 0 times each token that a row does not see, and so a NaN
// for one that is not finite. A warp that finds such columns leaves P' Z out of them in
// its rows (bits of `odd`), and the warp that copies out adds it, from memory and to
// each row from the tokens that it sees alone. What the state gives is rounded to
// bfloat16 before: once more than elsewhere, in such columns alone.
template <int DP, bool BACK>
__device__ __forceinline__ void add_seen(const WalkArgs &p, const Unit *u, int j, int first, int n,
                                         uint64_t *odd, unsigned char *tile) {
  constexpr int kPairs = DP / 64;  // columns 2 lane + 64 m and the next to a lane
  const int lane = threadIdx.x & 31, ny = BACK ? p.ny : 1, head = u->h0 + (BACK ? 0 : j);
  const View x = p.x[u->walk], y = p.y[u->walk], z = p.z[u->walk];
  const int64_t token = (int64_t)u->g.lo + first, head0 = (int64_t)(u->h0 / p.group) * ny;
  const auto word = [&](const View &v, int c, int s, int col) {
    return *reinterpret_cast<const uint32_t *>(v.p + (token + c) * v.token +
                                               (head0 + s) * v.head + col);
  };
  // Tokens in the order seen (backwards from the last): how many a row may see before
  // one makes a column, or by its key all of them, not finite for good.
  const bool closed = u->g.rows > 1 && u->power[1] == 0.0f;
  int until[kPairs][2], all = kChunk;
#pragma unroll
  for (int m = 0; m < kPairs; ++m) until[m][0] = until[m][1] = kChunk;
  for (int s = 0; s < ny; ++s)
#pragma unroll 4
    for (int k = n - 1; k >= 0; --k)
#pragma unroll
      for (int m = 0; m < kPairs; ++m) {
        const int col = 2 * lane + 64 * m, c = BACK ? n - 1 - k : k;
        if (col >= p.D) continue;
        const uint32_t a = word(y, c, s, col), b = word(z, c, s, col);
        if (tc::special(a)) all = min(all, k);
        if (tc::special(b) & 0x8000u) until[m][0] = min(until[m][0], k);
        if (tc::special(b) & 0x80000000u) until[m][1] = min(until[m][1], k);
      }
  all = __reduce_min_sync(kFull, all);
#pragma unroll 1
  for (int r = 0; r < n; ++r) {
    // tokens (of a head that keeps nothing its own, and no other's place counts)
    const int sees = closed ? 1 : (BACK ? n - r : r + 1);
    const bf *xr = x.p + (token + r) * x.token + head * x.head;
    uint32_t own = 0;
#pragma unroll
    for (int m = 0; m < kPairs; ++m)
      if (2 * lane + 64 * m < p.D)
        own |= tc::special(*reinterpret_cast<const uint32_t *>(xr + 2 * lane + 64 * m));
    const int lasts = __any_sync(kFull, own != 0) ? 0 : all;
    bool fix[kPairs][2], wanted = false;    // columns to form, and those with a sum to form
    float sum[kPairs][2];
#pragma unroll
    for (int m = 0; m < kPairs; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = 2 * lane + 64 * m + e;
        fix[m][e] = odd[col / (DP / 2) * 4 + r / 32] >> col % (DP / 2) & 1;
        const bool lost = !closed && min(lasts, until[m][e]) < sees;
        sum[m][e] = lost ? NAN : 0.0f;
        wanted |= fix[m][e] && !lost;
      }
    if (__any_sync(kFull, wanted)) {
#pragma unroll 1
      for (int i0 = 0; i0 < ny * sees; i0 += 32) {
        float w = 0.0f;  // a term to a lane
        if (i0 + lane < ny * sees) {
          const int apart = (i0 + lane) % sees;
          const bf *yr = y.p + (token + (BACK ? r + apart : r - apart)) * y.token +
                         (head0 + (i0 + lane) / sees) * y.head;
#pragma unroll 1
          for (int d = 0; d < p.D; d += 8)
            w += dot8(*reinterpret_cast<const uint4 *>(xr + d),
                      *reinterpret_cast<const uint4 *>(yr + d));
          w *= u->decay[31 + apart];
        }
#pragma unroll 4
        for (int i = i0; i < min(i0 + 32, ny * sees); ++i) {
          const float f = __shfl_sync(kFull, w, i - i0);
#pragma unroll
          for (int m = 0; m < kPairs; ++m)
            if (2 * lane + 64 * m < p.D) {
              const uint32_t v = word(z, BACK ? r + i % sees : r - i % sees, i / sees,
                                      2 * lane + 64 * m);
              sum[m][0] = fmaf(f, __uint_as_float(v << 16), sum[m][0]);
              sum[m][1] = fmaf(f, __uint_as_float(v & 0xffff0000u), sum[m][1]);
            }
        }
      }
    }
#pragma unroll
    for (int m = 0; m < kPairs; ++m) {
      const int col = 2 * lane + 64 * m;
      if (col >= p.D || !(fix[m][0] || fix[m][1])) continue;
      uint32_t *at = reinterpret_cast<uint32_t *>(tile + place(r, col) + col % 8 * 2);
      *at = pack_bf16(__uint_as_float(*at << 16) + (fix[m][0] ? sum[m][0] : 0.0f),
                      __uint_as_float(*at & 0xffff0000u) + (fix[m][1] ? sum[m][1] : 0.0f));
    }
  }
  __syncwarp();
  if (lane < 8) odd[lane] = 0;
  fence_proxy_async_shared();
  __syncwarp();
}

template <int DP, bool BACK>
__global__ void __launch_bounds__(kWalkThreads, 1)
    linear_walk_kernel(const __grid_constant__ WalkMaps first,
                       const __grid_constant__ WalkMaps second, const WalkArgs p) {
  extern __shared__ __align__(1024) unsigned char raw[];
  WalkSmem<DP> &sm = *reinterpret_cast<WalkSmem<DP> *>(raw);
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = __shfl_sync(kFull, threadIdx.x >> 5, 0);
  const int blocks = p.heads / p.nx;  // units to a segment
  constexpr int kStages = stages<DP>();
  const int tokens = (int)p.tokens, sequences = (int)p.sequences;
  if (warp == 17) tc::tmem_alloc(&sm.tmem, 512);
  if (threadIdx.x == 0) {
    sm.abort = (tc::smem_addr(raw) & 1023) != 0;  // the swizzle counts from there
    for (int i = 0; i < kStages; ++i)
      for (uint64_t *b : {&sm.x_full[i], &sm.x_empty[i], &sm.y_full[i], &sm.y_empty[i]})
        mbar_init(b, 1);
    for (uint64_t *b : {&sm.p_full[0], &sm.p_full[1], &sm.y_used[0], &sm.y_used[1], &sm.o_full,
                        &sm.u_full, &sm.s_used, &sm.unit_full[0], &sm.unit_full[1],
                        &sm.asked[0], &sm.asked[1]})
      mbar_init(b, 1);
    for (uint64_t *b : {&sm.p_ready[0], &sm.p_ready[1], &sm.y_ready[0], &sm.y_ready[1], &sm.o_free,
                        &sm.s_ready})
      mbar_init(b, 8);
    for (int i = 0; i < kStages; ++i) mbar_init(&sm.result[i], 8);
    for (int i = 0; i < kStages * 8; ++i) sm.odd[0][i] = 0;
    for (uint64_t *b : {&sm.unit_empty[0], &sm.unit_empty[1]}) mbar_init(b, 18);
    fence_mbar_init();
  }
  const bool ordered = p.length >= tokens && sequences <= kOrdered;
  static_assert(sizeof(sm.unit[0].decay) >= kOrdered * sizeof(int), "room for the lengths");
  if (ordered)  // (the lengths lie where a unit's decays come later)
    order_sequences(p.cu, sequences, tokens, reinterpret_cast<int *>(sm.unit[0].decay), sm.order);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // Rows of results that no sequence holds are zeros: each unit has a share of
  // them, units without a segment too, and the warp that copies in writes it.
  const int lo = bound(p.cu, 0, tokens), hi = max(lo, bound(p.cu, sequences, tokens));
  const bool unheld = lo > 0 || hi < tokens;
  if (sm.abort) {
    if (warp == 17) tc::tmem_dealloc(sm.tmem, 512);
    if (threadIdx.x == 0) atomicMax(&device_status, (uint32_t)RLCS_ERR_CUDA);
    return;
  }
  const int nx = BACK ? 1 : p.nx, ny = BACK ? p.ny : 1, items = BACK ? ny : nx;  // to a chunk
  const uint32_t tmem = __shfl_sync(kFull, sm.tmem, 0);
  // P (two, where heads are up to 64 wide), O1, O2, S
  constexpr int kP = DP == 64 ? 2 : 1;
  const uint32_t tP = tmem, tO = tmem + kP * 128, tX = tO + DP, tU = tX + DP;
  volatile int *abort = &sm.abort;
  const uint32_t lead = lane == 0;
  // chunk number `c` of a segment in the order walked: its first row in the
  // sequence, and its rows
  const auto chunks_of = [](const Segment &g) {
    return (int)((unsigned)(g.rows + kChunk - 1) / (unsigned)kChunk);
  };
  const auto first_row = [&](const Segment &g, int c) {
    return g.first + (BACK ? chunks_of(g) - 1 - c : c) * kChunk;
  };
  const auto rows_of = [&](const Segment &g, int c) {
    const int left = g.first + g.rows - first_row(g, c);
    return left < kChunk ? left : kChunk;
  };
  // Units come to the other warps by turns; every count of tiles and barriers
  // goes on from one to the next.
  const auto next_unit = [&](int k) -> const Unit * {
    if (!tc::warp_wait(&sm.unit_full[k & 1], (k >> 1) & 1, abort)) return nullptr;
    const Unit *u = &sm.unit[k & 1];
    return u->end ? nullptr : u;
  };
  const auto unit_done = [&](int k) { tc::warp_arrive(&sm.unit_empty[k & 1], lead); };

  if (warp == 16) {
    int xi = 0, yi = 0;
    bool ok = true;
    const auto request = [&](int i) {
      if (lane == 0) {
        fence_proxy_async_shared();
        mbar_arrive_expect_tx(&sm.asked[i & 1], 16);
        tc::ask(&sm.answer[i & 1], &sm.asked[i & 1], false);
      }
      __syncwarp();
    };
    request(0);
    int64_t block = blockIdx.x;
    for (int i = 0, k = 0; ok; ++i) {
      const bool end = block < 0;
      const int walk = end ? 0 : (int)(block % p.walks);
      const int64_t at = end ? 0 : block / p.walks;
      const int slot = (int)(at / blocks), h0 = (int)(at % blocks) * p.nx;
      // the unit after this one, asked for a unit ago
      if (!end) {
        if (!(ok = tc::warp_wait(&sm.asked[i & 1], (i >> 1) & 1, abort))) break;
        block = tc::granted(&sm.answer[i & 1]);
        __syncwarp();
        if (block >= 0) request(i + 1);
      }
      Segment g = {};
      if (!end) {
        if (!ordered)
          g = find_segment(p.cu, sequences, tokens, slot, p.length);
        else if (slot < sequences)
          g = whole_sequence(p.cu, tokens, sm.order[slot]);
        if (unheld)
          zero_unheld(p.out[walk], p.heads * p.D, lo, hi, tokens, at, gridDim.x / p.walks);
        if (!g.any) continue;
      }
      if (k >= 2) ok = tc::warp_wait(&sm.unit_empty[k & 1], ((k >> 1) - 1) & 1, abort);
      if (!ok) break;
      Unit &u = sm.unit[k & 1];
      const int state_head = h0 / p.group;
      if (!end) {
        const float l2 = __ldg(p.log_decay + state_head) * kLog2e;
        const float scale = p.in_scale * p.out_scale;
        for (int i = lane; i < 31 + kChunk; i += 32) {
          const float f = i < 31 ? 0.0f : power(l2, i - 31);
          u.decay[i] = i - 31 < g.rows ? scale * f : 0.0f;
          if (i >= 31) u.power[i - 31] = i - 31 < g.rows || p.init ? f : 0.0f;
        }
        if (lane == 0) u.power[kChunk] = g.rows > kChunk || p.init ? power(l2, kChunk) : 0.0f;
        if (lane < 16) u.near[lane] = scale * power(l2, BACK ? lane : 15 - lane);
      }
      if (lane == 0) u.g = g, u.slot = slot, u.h0 = h0, u.walk = walk, u.end = end;
      tc::warp_arrive(&sm.unit_full[k & 1], lead);
      ++k;
      if (end) break;
      if (lane == 0) {
        const auto load = [&](unsigned char *to, const CUtensorMap *m, uint64_t *full, int head,
                              int token) {
#pragma unroll
          for (int i = 0; i < DP / 64; ++i)
            tc::load_box(to + i * 16384, m, full, i * 64, head, token);
        };
        const WalkMaps &m = walk ? second : first;
        const int chunks = chunks_of(g);
        for (int c = 0; c < chunks && ok; ++c) {
          const int token = g.lo + first_row(g, c);
          for (int j = 0; j < items; ++j) {
            if (!BACK || j == 0) {
              const int st = xi % kStages, use = xi / kStages;
              if (use > 0 && !(ok = tc::mbar_wait(&sm.x_empty[st], (use - 1) & 1, abort))) break;
              mbar_arrive_expect_tx(&sm.x_full[st], DP * 256);
              load(sm.x[st], &m.x, &sm.x_full[st], h0 + (BACK ? 0 : j), token);
              ++xi;
            }
            if (BACK || j == 0) {
              const int st = yi % kStages, use = yi / kStages;
              const int head = state_head * ny + (BACK ? j : 0);
              if (use > 0 && !(ok = tc::mbar_wait(&sm.y_empty[st], (use - 1) & 1, abort))) break;
              mbar_arrive_expect_tx(&sm.y_full[st], DP * 512);
              load(sm.y[st], &m.y, &sm.y_full[st], head, token);
              load(sm.z[st], &m.z, &sm.y_full[st], head, token);
              ++yi;
            }
          }
        }
      }
      ok = __shfl_sync(kFull, (int)ok, 0) != 0;
    }
  } else if (warp == 17) {
    // Items of all units in their order. P of an item is formed as soon as its
    // tiles are there and P's place is free; with two places an item ahead.
    struct Item {
      int k, c, j, chunks;  // unit, chunk and item of it; chunks of the unit
      int part, rows;       // the one chunk that may be short, and its rows
      bool any;
    };
    const auto enter = [&](Item &x) {  // the first item of unit k
      const Unit *unit = next_unit(x.k);
      x.any = unit != nullptr;
      if (!x.any) return;
      x.chunks = chunks_of(unit->g);
      x.c = x.j = 0;
      x.part = BACK ? 0 : x.chunks - 1;
      x.rows = rows_of(unit->g, x.part);
    };
    const auto advance = [&](Item &x) {
      if (++x.j < items) return;
      x.j = 0;
      if (++x.c < x.chunks) return;
      ++x.k;
      enter(x);
    };
    bool ok = true;
    int pi = 0, px = 0, py = 0;  // items, x tiles and y tiles that P has been formed from
    const auto weights = [&](const Item &x) {
      const bool new_x = !BACK || x.j == 0, new_y = BACK || x.j == 0, last = x.j + 1 == items;
      const int xi = new_x ? px++ : px - 1, yi = new_y ? py++ : py - 1;
      const int xs = xi % kStages, ys = yi % kStages;
      unsigned char *tx = sm.x[xs], *ty = sm.y[ys], *tz = sm.z[ys];
      if (new_x) ok = ok && tc::warp_wait(&sm.x_full[xs], (xi / kStages) & 1, abort);
      if (new_y) ok = ok && tc::warp_wait(&sm.y_full[ys], (yi / kStages) & 1, abort);
      if (!ok) return;
      if (x.c == x.part && x.rows < kChunk) {  // what follows is another's: it must be finite
        if (new_x) tc::clear_rows<DP, kChunk>(tx, x.rows, lane);
        if (new_y) tc::clear_rows<DP, kChunk>(ty, x.rows, lane);
        if (new_y) tc::clear_rows<DP, kChunk>(tz, x.rows, lane);
        __syncwarp();
      }
      tc::product_nt<DP, kChunk>(lead, tP + (kP > 1 ? (pi & 1) * 128 : 0), tc::smem_addr(tx),
                                 tc::smem_addr(ty));
      tc::commit(lead, &sm.p_full[pi & 1]);
      if (BACK || last) tc::commit(lead, &sm.y_used[yi & 1]);  // every product of the unscaled keys
      ++pi;
    };
    Item ahead = {}, now;
    enter(ahead);
    // x, y: tiles of each ring; it: items; o: results; sc: chunks
    int xi = 0, yi = 0, o = 0, sc = 0;
    if (ahead.any) weights(ahead);
    for (int it = 0; ahead.any && ok; ++it) {
      now = ahead;
      if (kP > 1) {
        advance(ahead);
        if (ahead.any) weights(ahead);
        if (!ok) break;
      }
      const int j = now.j;
      const bool new_x = !BACK || j == 0, last = j + 1 == items;
      const uint32_t x = tc::smem_addr(sm.x[xi % kStages]), y = tc::smem_addr(sm.y[yi % kStages]),
                     z = tc::smem_addr(sm.z[yi % kStages]);
      const auto state_product = [&] {
        if (!new_x) return true;
        if (o > 0 && !tc::warp_wait(&sm.o_free, (o - 1) & 1, abort)) return false;
        tc::fence_after_sync();
        product_state<DP>(lead, tX, x, tc::smem_addr(sm.s));
        // every product of the rounded state (with one place for P the sum comes
        // after them, and stands for them)
        if (kP > 1 && (BACK || last)) tc::commit(lead, &sm.s_used);
        return true;
      };
      const auto own_product = [&] {
        if (!tc::warp_wait(&sm.p_ready[it & 1], (it >> 1) & 1, abort)) return false;
        tc::fence_after_sync();
        tc::product_parts<DP, kChunk, 8>(lead, tO, tP + (kP > 1 ? (it & 1) * 128 : 0), z,
                                         BACK && j > 0);
        if (!BACK || last) tc::commit(lead, &sm.o_full);
        return true;
      };
      const auto sum_product = [&] {
        if (!BACK && !last) return true;
        if (!tc::warp_wait(&sm.y_ready[yi & 1], (yi >> 1) & 1, abort)) return false;
        tc::fence_after_sync();
        product_tn<DP>(lead, tU, y, z, true);
        if (last) tc::commit(lead, &sm.u_full);
        return true;
      };
      if (j == 0 && !(ok = tc::warp_wait(&sm.s_ready, sc++ & 1, abort))) break;
      // What the next state waits for comes first where its keys have long been
      // scaled, and last where they are scaled while the others run.
      if (kP > 1)
        ok = sum_product() && state_product() && own_product();
      else
        ok = state_product() && own_product() && sum_product();
      if (!ok) break;
      if (!BACK || last) ++o, ++xi;
      if (BACK || last) {
        tc::commit(lead, &sm.y_empty[yi % kStages]);
        ++yi;
      }
      const int k = now.k;
      const bool done = last && now.c + 1 == now.chunks;
      if (kP == 1) {
        if (done) unit_done(k);
        advance(ahead);
        if (ahead.any) weights(ahead);
      } else if (done) {
        unit_done(k);
      }
    }
  } else if (warp < 8) {
    // Blocks of 16 columns, every other one of a row to a thread. Where a block
    // lies wholly on the seen side its decays are products of two powers, one
    // of the thread and one of the column.
    const int r = threadIdx.x & 127, half = warp >> 2, row0 = (warp & 3) * 32;
    const uint32_t lanes = (uint32_t)row0 << 16;
    int it = 0, o = 0;
    for (int k = 0;; ++k) {
      const Unit *unit = next_unit(k);
      if (!unit) break;
      const Segment &g = unit->g;
      const int chunks = chunks_of(g), h0 = unit->h0;
      const bool one = BACK && g.rows < kChunk;
      for (int c = 0; c < chunks; ++c) {
        for (int j = 0; j < items; ++j, ++it) {
          tc::warp_wait(&sm.p_full[it & 1], (it >> 1) & 1, abort);
          const uint32_t scores = tP + (kP > 1 ? (it & 1) * 128 : 0) + lanes;
          tc::fence_after_sync();
#pragma unroll
          for (int i0 = 0; i0 < 4; i0 += 2) {
            // (two blocks are asked for together: a load takes some 300 clocks)
            uint32_t v[2][16];
#pragma unroll
            for (int i = 0; i < 2; ++i) tc::ld16(scores + (2 * (i0 + i) + half) * 16, v[i]);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int c0 = (2 * (i0 + i) + half) * 16;
              uint32_t w[8];
              // (the same for the whole warp; the row's own 32 columns are among these,
              // or it is a short segment backwards, see Unit::decay)
              if (i0 + i == (warp & 3) || (one && i0 + i > (warp & 3))) {
                const float *d = unit->decay + 31 + (BACK ? c0 - r : r - c0);
#pragma unroll
                for (int e = 0; e < 8; ++e)  // the type that the product takes
                  w[e] = pack_bf16(__uint_as_float(v[i][2 * e]) * d[BACK ? 2 * e : -2 * e],
                                   __uint_as_float(v[i][2 * e + 1]) *
                                       d[BACK ? 2 * e + 1 : -2 * e - 1]);
              } else if (BACK ? i0 + i < (warp & 3) : i0 + i > (warp & 3)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = 0;
              } else {
                const float f = unit->power[BACK ? c0 - r : r - c0 - 15];
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                  const float4 k = *reinterpret_cast<const float4 *>(unit->near + e);
                  const float2 a = __fmul2_rn(make_float2(k.x, k.y), make_float2(f, f)),
                               b = __fmul2_rn(make_float2(k.z, k.w), make_float2(f, f));
                  const float2 x = __fmul2_rn(pair(v[i] + e), a),
                               y = __fmul2_rn(pair(v[i] + e + 2), b);
                  w[e / 2] = pack_bf16(x.x, x.y);
                  w[e / 2 + 1] = pack_bf16(y.x, y.y);
                }
              }
              tc::st8(scores + c0, w);
            }
          }
          tc::wait_st();
          tc::fence_before_sync();
          tc::warp_arrive(&sm.p_ready[it & 1], lead);
          if (BACK && j + 1 < items) continue;
          const int n = rows_of(g, c), to_row = BACK ? n - 1 - r : r + 1;
          const float into = unit->power[to_row < 0 ? 0 : to_row] * p.out_scale;
          // Results take the place of their X and are copied out from there.
          unsigned char *tile = sm.x[o % kStages];
          tc::warp_wait(&sm.o_full, o & 1, abort);
          tc::fence_after_sync();
          const float2 f = make_float2(into, into);
#pragma unroll
          for (int i = 0; i < DP / 64; ++i) {
            uint32_t a[32], b[32];
            tc::ld32(tO + lanes + half * (DP / 2) + i * 32, a);
            tc::ld32(tX + lanes + half * (DP / 2) + i * 32, b);
            tc::wait_ld();
            // (a row that the state does not reach takes nothing of it, whatever it holds)
            if (into == 0.0f)
#pragma unroll
              for (int e = 0; e < 32; ++e) b[e] = 0;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              const int col = half * (DP / 2) + i * 32 + e;
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int q = e + 2 * k;
                const float2 t = __ffma2_rn(pair(b + q), f, pair(a + q));
                w[k] = pack_bf16(t.x, t.y);
              }
              const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4 *>(tile + place(r, col)) = v;
            }
          }
          // The row of these 32 that sees the fewest of them has all columns finite, or
          // something is looked at: see add_seen.
          __syncwarp();
          const int least = row0 + (BACK ? 31 : 0), pick = half * (DP / 2) + lane * (DP / 64);
          const unsigned char *at = tile + place(least, pick) + pick % 8 * 2;
          const uint32_t odd = DP == 128 ? tc::special(*reinterpret_cast<const uint32_t *>(at))
                                         : tc::special(*reinterpret_cast<const uint16_t *>(at));
          if (__any_sync(kFull, odd != 0) && row0 < n && !*abort) {
            uint64_t own = 0;  // columns of P' Z that have it (it may be the state's alone)
#pragma unroll 1
            for (int i = 0; i < DP / 2; i += 8) {
              uint32_t a[8];
              tc::ld8(tO + lanes + half * (DP / 2) + i, a);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const bool fine = fabsf(__uint_as_float(a[e])) < INFINITY;
                own |= (uint64_t)(__any_sync(kFull, r < n && !fine) != 0) << (i + e);
              }
            }
#pragma unroll 1
            for (int i = 0; i < DP / 2; i += 8) {
              if (!(own >> i & 255)) continue;
              uint32_t a[8], b[8], w[4];
              tc::ld8(tO + lanes + half * (DP / 2) + i, a);
              tc::ld8(tX + lanes + half * (DP / 2) + i, b);
              tc::wait_ld();
              float t[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                t[e] = into == 0.0f ? 0.0f : __uint_as_float(b[e]) * into;
                if (!(own >> (i + e) & 1)) t[e] += __uint_as_float(a[e]);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) w[k] = pack_bf16(t[2 * k], t[2 * k + 1]);
              *reinterpret_cast<uint4 *>(tile + place(r, half * (DP / 2) + i)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (lane == 0) sm.odd[o % kStages][warp] = own;
          }
          tc::fence_before_sync();
          tc::warp_arrive(&sm.o_free, lead);
          fence_proxy_async_shared();
          tc::warp_arrive(&sm.result[o % kStages], lead);
          ++o;
        }
      }
      unit_done(k);
    }
  } else if (warp == 18) {
    // results, from where X was; X is free when they have been read
    int o = 0;
    for (int k = 0;; ++k) {
      const Unit *unit = next_unit(k);
      if (!unit) break;
      const Segment &g = unit->g;
      const int chunks = chunks_of(g), h0 = unit->h0;
      for (int c = 0; c < chunks; ++c)
        for (int j = 0; j < nx; ++j, ++o) {
          const int st = o % kStages;
          const bool there = tc::warp_wait(&sm.result[st], (o / kStages) & 1, abort);
          const int n = rows_of(g, c);
          if (there && __any_sync(kFull, sm.odd[st][lane & 7] != 0) && !*abort)
            add_seen<DP, BACK>(p, unit, j, first_row(g, c), n, sm.odd[st], sm.x[st]);
          if (!there || *abort) {
          } else if (n < kChunk) {  // (what follows in memory is another's)
            bf *out = p.out[unit->walk] +
                      (((int64_t)g.lo + first_row(g, c)) * p.heads + h0 + j) * p.D;
            const int row = lane / (DP / 8), col = lane % (DP / 8) * 8;
            if (col < p.D)
#pragma unroll 4
              for (int r = row; r < n; r += 256 / DP)
                *reinterpret_cast<uint4 *>(out + (int64_t)r * p.heads * p.D + col) =
                    *reinterpret_cast<const uint4 *>(sm.x[st] + place(r, col));
          } else if (lane == 0) {
#pragma unroll
            for (int b = 0; b < DP / 64; ++b)
              if (b * 64 < p.D)
                store_box(sm.x[st] + b * 16384,
                          unit->walk ? &second.out : &first.out, b * 64,
                          h0 + j, g.lo + first_row(g, c));
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          }
          tc::warp_arrive(&sm.x_empty[st], lead);
        }
      unit_done(k);
    }
  } else {
    const int t = threadIdx.x - 256, r = t & 127, half = (warp - 8) >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    constexpr int HC = DP / 2;  // columns of the state to a thread, in row r of it
    float s[HC];
    // The state before a chunk: rounded, as the product's second operand (rows
    // in boxes of 64 columns), and times the chunk's decay back to where the
    // chunk's own part is added.
    int handed = 0;
    const auto hand_over = [&](float keep) {
      if (kP > 1 && handed++ > 0) tc::warp_wait(&sm.s_used, handed & 1, abort);
      if (r < DP)
#pragma unroll
        for (int c = 0; c < HC; c += 8) {
          const int col = half * HC + c, chunk = (col % 64) / 8;
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = pack_bf16(s[c + 2 * k], s[c + 2 * k + 1]);
          *reinterpret_cast<uint4 *>(sm.s + (col / 64) * DP * 128 + r * 128 +
                                     ((chunk ^ (r & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      if (keep == 0.0f)  // (nothing is kept, whatever the state holds)
#pragma unroll
        for (int c = 0; c < HC; ++c) s[c] = 0.0f;
#pragma unroll
      for (int c = 0; c < HC; c += 16) {
        uint32_t u[16];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float2 k = __fmul2_rn(make_float2(s[c + e], s[c + e + 1]), make_float2(keep, keep));
          u[e] = __float_as_uint(k.x);
          u[e + 1] = __float_as_uint(k.y);
        }
        tc::st16(tU + lanes + half * HC + c, u);
      }
      fence_proxy_async_shared();
      tc::wait_st();
      tc::fence_before_sync();
      tc::warp_arrive(&sm.s_ready, lead);
    };
    constexpr int kTimes = DP * 16 / 256;  // words of a tile to a thread, 32 rows apart
    int yi = 0, sc = 0;
    for (int k = 0;; ++k) {
      const Unit *unit = next_unit(k);
      if (!unit) break;
      const Segment &g = unit->g;
      const int chunks = chunks_of(g);
#pragma unroll
      for (int c = 0; c < HC; ++c) s[c] = 0.0f;
      if (p.init && r < p.D) {
        const float *from = p.init + ((p.by_slot ? (int64_t)unit->slot : (int64_t)g.seq) *
                                          (p.heads / p.group) + unit->h0 / p.group) * p.D * p.D;
        if (p.transposed[unit->walk]) {
#pragma unroll
          for (int c = 0; c < HC; ++c)
            if (half * HC + c < p.D) s[c] = __ldg(from + (int64_t)(half * HC + c) * p.D + r);
        } else {
#pragma unroll
          for (int c = 0; c < HC; c += 4)
            if (half * HC + c < p.D)
              *reinterpret_cast<float4 *>(s + c) =
                  __ldg(reinterpret_cast<const float4 *>(from + (int64_t)r * p.D + half * HC + c));
        }
      }
      // (asked for before the last unit's last product is waited for)
      if (sc > 0) tc::warp_wait(&sm.u_full, (sc - 1) & 1, abort);
      hand_over(unit->power[rows_of(g, 0)]);
      for (int c = 0; c < chunks; ++c, ++sc) {
        const int n = rows_of(g, c);
        for (int j = 0; j < ny; ++j, ++yi) {
          tc::warp_wait(&sm.y_used[yi & 1], (yi >> 1) & 1, abort);
          uint4 *y = reinterpret_cast<uint4 *>(sm.y[yi % kStages]) + t;
          Factor f[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = t / 8 + i * 32, left = BACK ? row + 1 : n - 1 - row;
            f[i] = factor(unit->power[left < 0 ? 0 : left] * p.in_scale);
          }
#pragma unroll
          for (int i0 = 0; i0 < kTimes; i0 += 4) {
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = y[(i0 + i) * 256];
#pragma unroll
            for (int i = 0; i < 4; ++i)  // (rows that are not the sequence's are zeros already)
              y[(i0 + i) * 256] = t / 8 + i * 32 < n ? scaled(v[i], f[i]) : make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_shared();
          tc::warp_arrive(&sm.y_ready[yi & 1], lead);
        }
        if (c + 1 == chunks) continue;
        tc::warp_wait(&sm.u_full, sc & 1, abort);
        tc::fence_after_sync();
#pragma unroll
        for (int i = 0; i < HC / 32; ++i)
          tc::ld32(tU + lanes + half * HC + i * 32, *reinterpret_cast<uint32_t(*)[32]>(s + i * 32));
        tc::wait_ld();
        // (a head that keeps nothing has no state, whatever has been added to it)
        if (unit->power[1] == 0.0f)
#pragma unroll
          for (int e = 0; e < HC; ++e) s[e] = 0.0f;
        hand_over(unit->power[rows_of(g, c + 1)]);
      }
      unit_done(k);
    }
    // no product is under way when tensor memory is given up
    if (sc > 0) tc::warp_wait(&sm.u_full, (sc - 1) & 1, abort);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  settle(sm.abort);
  if (warp == 17) tc::tmem_dealloc(sm.tmem, 512);
}

// ---------------------------------------------------------------------------
// What a segment adds to the state: sum a^left y z^T over its tokens, left the
// steps to its end. Float32 results come from here, so a decayed key is held in
// two bfloat16 parts, off by at most 2^-17 together: two products. Tokens that
// count the most are added last, as the sum is cut off to float32 at each addition:
// states are within 3e-6 of 64 bits (2-norm; first states' gradients 1.2e-5 in the
// other order). A third part made fast heads' 2e-7, left those of decays above 0.999
// at 2.5e-6, and took 27 us more of 301. 131072 tokens, 8 heads of 128, in 38
// segments: 99 us, 5.4 TB/s; joining them 18 us.
// ---------------------------------------------------------------------------
struct SumArgs {
  const float *log_decay;
  const int32_t *cu;
  const float *init;  // [sequences, Hk, D, D] or null, where the sums are final
  float *sums;        // [slots, Hk, D, D], or [sequences, Hk, D, D] where final
  int64_t sequences, tokens;
  int Hk, ny, D, length;
  bool final;         // one segment to a sequence: add what is left of init
  bool all;           // sums of every segment, not only of those that others follow
  // Launched behind the walk, whose results are not read here: blocks take the
  // SMs that the walk's end leaves idle. All blocks of the walk have waited for
  // what came before when the first of these starts, so the wait, which is for
  // the walk, stands at the end: what comes next may count on both.
  bool beside;
  float in_scale;
};
constexpr int kSumStages = 3;
template <int DP>
struct SumSmem {
  // (in this order: with 64 columns a product reads past y and rest, into rows
  // of its result that are not used)
  alignas(1024) unsigned char y[kSumStages][DP * 256], rest[DP * 256], z[kSumStages][DP * 256];
  uint64_t full[kSumStages], empty[kSumStages], ready, rest_free, done;
  Segment segment;
  int len[kOrdered];
  uint8_t order[kOrdered];
  uint32_t tmem;
  int abort;
};
constexpr int kSumThreads = 10 * 32;

template <int DP, bool BACK>
__global__ void __launch_bounds__(kSumThreads, 1)
    linear_sum_kernel(const __grid_constant__ CUtensorMap my,
                      const __grid_constant__ CUtensorMap mz, const SumArgs p) {
  extern __shared__ __align__(1024) unsigned char raw[];
  SumSmem<DP> &sm = *reinterpret_cast<SumSmem<DP> *>(raw);
  if (!p.beside) pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = __shfl_sync(kFull, threadIdx.x >> 5, 0);
  const int h = blockIdx.x % p.Hk, slot = blockIdx.x / p.Hk;
  const int tokens = (int)p.tokens, sequences = (int)p.sequences;
  if (warp == 9) tc::tmem_alloc(&sm.tmem, 128);
  const bool ordered = p.length >= tokens && sequences <= kOrdered;
  if (ordered) order_sequences(p.cu, sequences, tokens, sm.len, sm.order);
  if (warp == 8) {
    Segment g = {};
    if (!ordered)
      g = find_segment(p.cu, sequences, tokens, slot, p.length);
    else if (slot < sequences)
      g = whole_sequence(p.cu, tokens, sm.order[slot]);
    if (lane == 0) {
      sm.segment = g;
      sm.abort = (tc::smem_addr(raw) & 1023) != 0;
      for (int i = 0; i < kSumStages; ++i) mbar_init(&sm.full[i], 1), mbar_init(&sm.empty[i], 1);
      mbar_init(&sm.rest_free, 1);
      mbar_init(&sm.done, 1);
      mbar_init(&sm.ready, 8);
      fence_mbar_init();
    }
  }
  const float l2 = __ldg(p.log_decay + h) * kLog2e;
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  Segment g = sm.segment;
  // a segment that no other follows in the walk is summed for the last state alone
  const bool followed = BACK ? g.first > 0 : g.first + g.rows < g.len;
  const bool work = g.any && !sm.abort && (p.all || followed);
  if (!work) {
    if (warp == 9) tc::tmem_dealloc(sm.tmem, 128);
    if (sm.abort && threadIdx.x == 0) atomicMax(&device_status, (uint32_t)RLCS_ERR_CUDA);
    // an empty sequence's last state is its first
    if (p.final && !g.any && g.len == 0 &&
        (ordered ? slot < sequences : slot == slot_of(g.lo, g.seq, p.length))) {
      const int64_t at = ((int64_t)g.seq * p.Hk + h) * p.D * p.D;
      for (int i = threadIdx.x; i < p.D * p.D; i += kSumThreads)
        p.sums[at + i] = p.init ? p.init[at + i] : 0.0f;
    }
    if (p.beside) pdl_wait();
    return;
  }
  // A head that keeps nothing adds a segment's last token, or backwards nothing.
  const float kept = p.final ? power(l2, g.rows) : 0.0f;
  if (power(l2, 1) == 0.0f) {
    g.first += g.rows - 1;
    g.rows = BACK ? 0 : 1;
  }
  const int chunks = g.rows ? (g.rows + kChunk - 1) / kChunk : 1, items = chunks * p.ny;
  const uint32_t tmem = __shfl_sync(kFull, sm.tmem, 0);
  volatile int *abort = &sm.abort;
  const uint32_t lead = lane == 0;
  const auto first_of = [&](int it) {  // the first row, in the segment, of an item's tile
    return (BACK ? chunks - 1 - it / p.ny : it / p.ny) * kChunk;
  };
  if (warp == 8) {
    if (lane == 0)
      for (int it = 0; it < items; ++it) {
        const int st = it % kSumStages, use = it / kSumStages;
        const int token = g.lo + g.first + first_of(it), head = h * p.ny + it % p.ny;
        if (use > 0 && !tc::mbar_wait(&sm.empty[st], (use - 1) & 1, abort)) break;
        mbar_arrive_expect_tx(&sm.full[st], DP * 256 * 2);
#pragma unroll
        for (int b = 0; b < DP / 64; ++b) {
          tc::load_box(sm.y[st] + b * 16384, &my, &sm.full[st], b * 64, head, token);
          tc::load_box(sm.z[st] + b * 16384, &mz, &sm.full[st], b * 64, head, token);
        }
      }
  } else if (warp == 9) {
    for (int it = 0; it < items; ++it) {
      const int st = it % kSumStages, n = g.rows - first_of(it);
      if (!tc::warp_wait(&sm.full[st], (it / kSumStages) & 1, abort)) break;
      if (n < kChunk) {
        tc::clear_rows<DP, kChunk>(sm.z[st], n, lane);
        __syncwarp();
      }
      if (!tc::warp_wait(&sm.ready, it & 1, abort)) break;
      tc::fence_after_sync();
      const uint32_t z = tc::smem_addr(sm.z[st]);
      product_tn<DP>(lead, tmem, tc::smem_addr(sm.rest), z, it > 0);
      tc::commit(lead, &sm.rest_free);
      product_tn<DP>(lead, tmem, tc::smem_addr(sm.y[st]), z, true);
      tc::commit(lead, &sm.empty[st]);
    }
    tc::commit(lead, &sm.done);
  } else {
    for (int it = 0; it < items; ++it) {
      const int st = it % kSumStages, first = first_of(it);
      tc::warp_wait(&sm.full[st], (it / kSumStages) & 1, abort);
      if (it > 0) tc::warp_wait(&sm.rest_free, (it - 1) & 1, abort);
      uint4 *y = reinterpret_cast<uint4 *>(sm.y[st]), *rest = reinterpret_cast<uint4 *>(sm.rest);
      float f[4];  // of rows threadIdx.x / 8, + 32, + 64, + 96
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = first + threadIdx.x / 8 + i * 32, left = BACK ? row + 1 : g.rows - 1 - row;
        f[i] = row < g.rows ? power(l2, left) * p.in_scale : 0.0f;
      }
      y += threadIdx.x, rest += threadIdx.x;
#pragma unroll
      for (int i0 = 0; i0 < DP / 16; i0 += 4) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = y[(i0 + i) * 256];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // (rows that are not the sequence's may hold anything)
          if (first + (int)threadIdx.x / 8 + i * 32 >= g.rows) v[i] = make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          const float2 f2 = make_float2(f[i], f[i]);
          uint32_t a[4], b[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 t = __fmul2_rn(make_float2(__uint_as_float(w[k] << 16),
                                                    __uint_as_float(w[k] & 0xffff0000u)), f2);
            a[k] = pack_bf16(t.x, t.y);
            b[k] = pack_bf16(t.x - __uint_as_float(a[k] << 16),
                             t.y - __uint_as_float(a[k] & 0xffff0000u));
          }
          y[(i0 + i) * 256] = make_uint4(a[0], a[1], a[2], a[3]);
          rest[(i0 + i) * 256] = make_uint4(b[0], b[1], b[2], b[3]);
        }
      }
      fence_proxy_async_shared();
      tc::warp_arrive(&sm.ready, lead);
    }
    const int r = threadIdx.x & 127, half = warp >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const bool fine = tc::warp_wait(&sm.done, 0, abort);
    tc::fence_after_sync();
    const int64_t at = ((p.final ? (int64_t)g.seq : (int64_t)slot) * p.Hk + h) * p.D * p.D;
#pragma unroll
    for (int i = 0; i < DP / 64; ++i) {
      const int col = half * (DP / 2) + i * 32;
      uint32_t u[32];
      tc::ld32(tmem + lanes + col, u);
      tc::wait_ld();
      if (fine && r < p.D)
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          if (col + e < p.D) {
            const int64_t to = at + (int64_t)r * p.D + col + e;
            float4 v = make_float4(__uint_as_float(u[e]), __uint_as_float(u[e + 1]),
                                   __uint_as_float(u[e + 2]), __uint_as_float(u[e + 3]));
            if (p.init && kept != 0.0f) {
              const float4 o = __ldg(reinterpret_cast<const float4 *>(p.init + to));
              v.x = fmaf(kept, o.x, v.x);
              v.y = fmaf(kept, o.y, v.y);
              v.z = fmaf(kept, o.z, v.z);
              v.w = fmaf(kept, o.w, v.w);
            }
            *reinterpret_cast<float4 *>(p.sums + to) = v;
          }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  settle(sm.abort);
  if (warp == 9) tc::tmem_dealloc(sm.tmem, 128);
  if (p.beside) pdl_wait();
}

// The states before each segment from what the segments add, in place, and
// the state after the last: an element to a thread.
struct JoinArgs {
  const float *log_decay;
  const int32_t *cu;
  const float *init;
  float *sums, *last;
  int64_t sequences, tokens;
  int Hk, D, length;
  bool back, transposed;
};
__global__ void __launch_bounds__(256) linear_join_kernel(const JoinArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  const int size = p.D * p.D, i = blockIdx.x * 256 + threadIdx.x;
  const int64_t unit = blockIdx.y + (int64_t)blockIdx.z * 65535;
  if (i >= size || unit >= p.sequences * p.Hk) return;
  const int seq = (int)(unit / p.Hk), h = (int)(unit % p.Hk);
  const int lo = bound(p.cu, seq, (int)p.tokens), hi = bound(p.cu, seq + 1, (int)p.tokens);
  const int len = hi > lo ? hi - lo : 0, n = len / p.length + (len % p.length != 0);
  const float l2 = __ldg(p.log_decay + h) * kLog2e;
  const int64_t own = unit * size + (p.transposed ? i % p.D * p.D + i / p.D : i);
  float run = p.init ? __ldg(p.init + own) : 0.0f;
  float *at = p.sums + ((int64_t)slot_of(lo, seq, p.length) * p.Hk + h) * size + i;
  const int64_t step = (int64_t)p.Hk * size;
  constexpr int kAtOnce = 20;
  for (int j = 0; j < n; j += kAtOnce) {
    float add[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int seg = p.back ? n - 1 - j - k : j + k;
      // the last one walked is summed only if the last state is asked for
      add[k] = j + k < n - 1 || (j + k == n - 1 && p.last) ? at[seg * step] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (j + k >= n) break;
      const int seg = p.back ? n - 1 - j - k : j + k;
      const int rows = len - seg * p.length < p.length ? len - seg * p.length : p.length;
      const float keep = power(l2, rows);
      at[seg * step] = run;
      run = (keep == 0.0f ? 0.0f : keep * run) + add[k];
    }
  }
  if (p.last) p.last[own] = run;
}

// ---------------------------------------------------------------------------
// Host: one walk
// ---------------------------------------------------------------------------
struct Walk {
  View x[2], y[2], z[2];  // of one walk or two (see WalkArgs)
  bf *out[2];
  bool transposed[2];
  int walks;
  const float *log_decay;
  const int32_t *cu;
  const float *init;
  float *last;  // of the first walk
  int64_t sequences, tokens;
  int Hk, nx, ny, D;
  float in_scale, out_scale;
};

// How a walk is laid out. Heads of x that share a state go to one block, which
// then reads y and z and forms the state once, as far as a block to an SM is left.
// Where sequences and heads alone are fewer than 3/4 of the SMs, sequences are cut
// into segments: that costs a second reading of y and z and a pass over the states,
// and none is under 1024 tokens. Forward, heads of 128, one sequence, uncut and cut:
// 4 heads of 2048 tokens 39 us and 48 (so none of up to 2048 is cut), of 4096 71 and
// 49; 16 of 16384 300 and 122; 48 of 4096 87 and 105, of 16384 317 and 259; 96 of
// 16384 350 and 460. Of sequences that are alike more than about 56 are better left
// whole. But lengths are not known here: one long sequence among short ones, left
// whole, is a chain to a head, so the limit is higher; past it that is the case.
struct Layout {
  int64_t length;  // of a segment
  int nx;          // heads of x to a block
};
Layout layout_of(int64_t sequences, int64_t tokens, int64_t Hk, int64_t group) {
  Layout l = {(tokens + kChunk - 1) / kChunk * kChunk, 1};
  if (l.length == 0) l.length = kChunk;
  for (int64_t nx = group; nx > 1; --nx)
    if (group % nx == 0 && sequences * Hk * (group / nx) >= kSms) {
      l.nx = (int)nx;
      break;
    }
  const int64_t blocks = sequences * Hk * (group / l.nx);
  if (blocks * 4 >= kSms * 3 || tokens <= 2048) return l;
  const int64_t each = (tokens * Hk * group + 2 * kSms - 1) / (2 * kSms);
  l.length = (each + kChunk - 1) / kChunk * kChunk;
  if (l.length < 1024) l.length = 1024;
  return l;
}
size_t sums_bytes(int64_t sequences, int64_t tokens, int64_t group, int64_t Hk, int64_t D) {
  const int64_t length = layout_of(sequences, tokens, Hk, group).length;
  if (length >= tokens) return 0;
  return (size_t)(slots(sequences, tokens, length) * Hk * D * D) * 4;
}

bool map_of(CUtensorMap *m, const View &v, const Walk &w, int heads) {
  return tc::make_map(m, v.p, w.tokens, heads, w.D, v.token, v.head, kChunk);
}

template <int DP, bool BACK>
rlcs_status launch_walk(const Walk &w, float *sums, cudaStream_t st) {
  const Layout l = layout_of(w.sequences, w.tokens, w.Hk, w.nx);
  const int64_t length = l.length;
  const int64_t n = slots(w.sequences, w.tokens, length);
  const bool split = length < w.tokens;
  WalkMaps m[2] = {};
  for (int i = 0; w.tokens > 0 && i < w.walks; ++i)
    if (!map_of(&m[i].x, w.x[i], w, w.Hk * w.nx) || !map_of(&m[i].y, w.y[i], w, w.Hk * w.ny) ||
        !map_of(&m[i].z, w.z[i], w, w.Hk * w.ny) ||
        !map_of(&m[i].out, {w.out[i], (int64_t)w.Hk * w.nx * w.D, w.D}, w, w.Hk * w.nx))
      return RLCS_ERR_CUDA;
  cudaError_t e = cudaSuccess;
  const auto sum = [&](bool beside) {
    const SumArgs a = {w.log_decay, w.cu, split ? nullptr : w.init, split ? sums : w.last,
                       w.sequences, w.tokens, w.Hk, w.ny, w.D, (int)length, !split,
                       w.last != nullptr, beside, w.in_scale};
    constexpr size_t smem = sizeof(SumSmem<DP>);
    const cudaError_t e = allow_dynamic_smem<linear_sum_kernel<DP, BACK>>(smem);
    if (e != cudaSuccess) return e;
    return launch_ex(linear_sum_kernel<DP, BACK>, dim3((unsigned)(n * w.Hk)), dim3(kSumThreads),
                     smem, st, true, m[0].y, m[0].z, a);
  };
  if (split || (w.last && w.tokens == 0)) {
    e = sum(false);
    if (e != cudaSuccess) return launched(e);
  }
  if (split) {
    const JoinArgs a = {w.log_decay, w.cu, w.init, sums, w.last, w.sequences, w.tokens, w.Hk, w.D,
                        (int)length, BACK, w.transposed[0]};
    const int64_t units = w.sequences * w.Hk;
    const dim3 grid((unsigned)ceil_div(w.D * w.D, 256), (unsigned)(units < 65535 ? units : 65535),
                    (unsigned)ceil_div(units, 65535));
    e = launch_ex(linear_join_kernel, grid, dim3(256), 0, st, true, a);
    if (e != cudaSuccess) return launched(e);
  }
  if (w.tokens == 0) return RLCS_OK;
  // the sums of segments lie as the first walk has its state
  WalkArgs a = {};
  a.log_decay = w.log_decay;
  a.cu = w.cu;
  a.init = split ? sums : w.init;
  a.walks = w.walks;
  for (int i = 0; i < w.walks; ++i) {
    a.out[i] = w.out[i];
    a.x[i] = w.x[i];
    a.y[i] = w.y[i];
    a.z[i] = w.z[i];
    a.transposed[i] = split ? w.transposed[i] != w.transposed[0] : w.transposed[i];
  }
  a.sequences = w.sequences;
  a.tokens = w.tokens;
  a.heads = w.Hk * w.nx;
  a.group = w.nx;
  a.nx = l.nx;
  a.ny = w.ny;
  a.D = w.D;
  a.length = (int)length;
  a.by_slot = split;
  a.in_scale = w.in_scale;
  a.out_scale = w.out_scale;
  constexpr size_t smem = sizeof(WalkSmem<DP>);
  static_assert(smem <= 232448 && sizeof(SumSmem<DP>) <= 232448, "a block has 227 KB");
  e = allow_dynamic_smem<linear_walk_kernel<DP, BACK>>(smem);
  if (e != cudaSuccess) return launched(e);
  e = launch_ex(linear_walk_kernel<DP, BACK>,
                dim3((unsigned)(n * w.Hk * (w.nx / l.nx) * w.walks)), dim3(kWalkThreads), smem, st,
                true, m[0], m[1], a);
  if (e == cudaSuccess && w.last && !split) e = sum(true);
  return launched(e);
}
template <bool BACK>
rlcs_status launch(const Walk &w, float *sums, cudaStream_t st) {
  return w.D <= 64 ? launch_walk<64, BACK>(w, sums, st) : launch_walk<128, BACK>(w, sums, st);
}

// ---------------------------------------------------------------------------
// One step: a block to a state, four columns to a lane, DP / 4 lanes to a row.
// The state is read and written once, all of a thread's rows asked for before
// the first is used; it stays in registers for the query heads that share it.
// 256 states of 16 heads of 128: 86 us, 6.3 TB/s.
// ---------------------------------------------------------------------------
struct StepArgs {
  View q, k, v;
  const float *log_decay;
  const uint8_t *reset;
  const float *state;
  float *next;
  bf *out;
  int Hk, group, D;
  float scale;
};
constexpr int kStepWarps = 8, kStepHeads = 4;  // query heads summed up together

template <int DP>
__global__ void __launch_bounds__(kStepWarps * 32, 2) linear_step_kernel(const StepArgs p) {
  constexpr int kLanes = DP / 4, kAtOnce = kStepWarps * 32 / kLanes, kRows = DP / kAtOnce;
  __shared__ float k[DP], q[kStepHeads][DP], part[kStepHeads][kStepWarps][DP];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t unit = blockIdx.x, b = unit / p.Hk;
  const int h = (int)(unit % p.Hk), D = p.D, warp = threadIdx.x >> 5;
  const int col = threadIdx.x % kLanes * 4, first = threadIdx.x / kLanes;
  const float a = p.reset && p.reset[b] ? 0.0f : expf(p.log_decay[h]);
  const int64_t at = unit * D * D;
  float4 s[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = first + i * kAtOnce;
    s[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (a != 0.0f && row < D && col < D)  // (dropped whatever it holds)
      s[i] = *reinterpret_cast<const float4 *>(p.state + at + (int64_t)row * D + col);
  }
  if (threadIdx.x < DP)
    k[threadIdx.x] =
        threadIdx.x < D
            ? __bfloat162float(p.k.p[b * p.k.token + h * p.k.head + threadIdx.x])
            : 0.0f;
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    v[e] = col + e < D ? __bfloat162float(p.v.p[b * p.v.token + h * p.v.head + col + e]) : 0.0f;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = first + i * kAtOnce;
    const float x = k[row];
    s[i] = make_float4(fmaf(x, v[0], a * s[i].x), fmaf(x, v[1], a * s[i].y),
                       fmaf(x, v[2], a * s[i].z), fmaf(x, v[3], a * s[i].w));
    if (row < D && col < D)
      *reinterpret_cast<float4 *>(p.next + at + (int64_t)row * D + col) = s[i];
  }
  for (int g = 0; g < p.group; g += kStepHeads) {
    const int heads = p.group - g < kStepHeads ? p.group - g : kStepHeads;
    for (int i = threadIdx.x; i < heads * DP; i += kStepWarps * 32) {
      const int d = i % DP;
      q[i / DP][d] = d < D ? __bfloat162float(p.q.p[b * p.q.token +
                                                    (h * p.group + g + i / DP) * p.q.head + d])
                           : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kStepHeads; ++j) {
      if (j >= heads) break;
      float o[4] = {};
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float x = q[j][first + i * kAtOnce];
        o[0] = fmaf(x, s[i].x, o[0]);
        o[1] = fmaf(x, s[i].y, o[1]);
        o[2] = fmaf(x, s[i].z, o[2]);
        o[3] = fmaf(x, s[i].w, o[3]);
      }
#pragma unroll
      for (int w = kLanes; w < 32; w <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += __shfl_xor_sync(kFull, o[e], w);
      if ((threadIdx.x & 31) < kLanes)
        *reinterpret_cast<float4 *>(&part[j][warp][col]) = make_float4(o[0], o[1], o[2], o[3]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < heads * DP; i += kStepWarps * 32) {
      const int d = i % DP;
      float o = 0.0f;
#pragma unroll
      for (int w = 0; w < kStepWarps; ++w) o += part[i / DP][w][d];
      if (d < D)
        p.out[(unit * p.group + g + i / DP) * D + d] = __float2bfloat16_rn(o * p.scale);
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

// (rounded up to whole chunks, a segment's length is an int)
constexpr int64_t kMaxTokens = INT32_MAX / kChunk * kChunk;
bool linear_sizes(int64_t sequences, int64_t tokens, int64_t Hq, int64_t Hk, int64_t D,
                  double scale, rlcs_dtype t) {
  return sequences >= 0 && tokens >= 0 && tokens <= kMaxTokens && Hq > 0 && Hk > 0 &&
         Hq % Hk == 0 && D > 0 && D <= 128 && D % 8 == 0 && t == RLCS_BF16 && scale >= 1e-30 &&
         scale <= 1e30 && product_fits(tokens, Hq, D) && sequences < INT32_MAX - 1024 &&
         Hq < INT32_MAX && (sequences + tokens / 64 + 1) * Hq < (int64_t)INT32_MAX / 2;
}

}  // namespace

uint32_t *linear_status() {
  void *at = nullptr;
  return cudaGetSymbolAddress(&at, device_status) == cudaSuccess ? static_cast<uint32_t *>(at)
                                                                 : nullptr;
}

}  // namespace seq
}  // namespace rlcs

using namespace rlcs;
using namespace rlcs::seq;

extern "C" {

size_t rlcs_linear_attention_scratch_bytes(int64_t sequences, int64_t tokens, int64_t Hq,
                                           int64_t Hk, int64_t D) {
  if (!linear_sizes(sequences, tokens, Hq, Hk, D, 1.0, RLCS_BF16)) return 0;
  const size_t a = sums_bytes(sequences, tokens, Hq / Hk, Hk, D),
               b = sums_bytes(sequences, tokens, 1, Hk, D);
  return 64 + (a > b ? a : b);
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
  Walk w = {};
  w.x[0] = {static_cast<const bf *>(q), q_token_stride, q_head_stride};
  w.y[0] = {static_cast<const bf *>(k), k_token_stride, k_head_stride};
  w.z[0] = {static_cast<const bf *>(v), v_token_stride, v_head_stride};
  w.out[0] = static_cast<bf *>(out);
  w.walks = 1;
  w.log_decay = log_decay;
  w.cu = cu_seqlens;
  w.init = state;
  w.last = last_state;
  w.sequences = sequences;
  w.tokens = tokens;
  w.Hk = (int)Hk;
  w.nx = (int)(Hq / Hk);
  w.ny = 1;
  w.D = (int)D;
  w.in_scale = 1.0f;
  w.out_scale = (float)scale;
  return launch<false>(w, reinterpret_cast<float *>(static_cast<char *>(scratch) + 64),
                       reinterpret_cast<cudaStream_t>(stream));
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
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  float *sums = reinterpret_cast<float *>(static_cast<char *>(scratch) + 64);
  const int group = (int)(Hq / Hk);
  Walk w = {};
  w.log_decay = log_decay;
  w.cu = cu_seqlens;
  w.sequences = sequences;
  w.tokens = tokens;
  w.Hk = (int)Hk;
  w.D = (int)D;
  // dq
  w.x[0] = vd, w.y[0] = vv, w.z[0] = vk;
  w.out[0] = static_cast<bf *>(dq);
  w.transposed[0] = true;
  w.walks = 1;
  w.init = state;
  w.nx = group, w.ny = 1;
  w.in_scale = 1.0f, w.out_scale = (float)scale;
  const rlcs_status e = launch<false>(w, sums, st);
  if (e != RLCS_OK) return e;
  // dv and dk
  w.x[0] = vk, w.y[0] = vq, w.z[0] = vd;
  w.x[1] = vv, w.y[1] = vd, w.z[1] = vq;
  w.out[0] = static_cast<bf *>(dv);
  w.out[1] = static_cast<bf *>(dk);
  w.transposed[0] = false, w.transposed[1] = true;
  w.walks = 2;
  w.init = dlast, w.last = dstate;
  w.nx = 1, w.ny = group;
  w.in_scale = (float)scale, w.out_scale = 1.0f;
  return launch<true>(w, sums, st);
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
      B * Hk > INT32_MAX ||
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
                      (int)Hk,
                      (int)(Hq / Hk),
                      (int)D,
                      (float)scale};
  const dim3 grid((unsigned)(B * Hk)), block(kStepWarps * 32);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return launched(D <= 64 ? launch_ex(linear_step_kernel<64>, grid, block, 0, st, true, a)
                          : launch_ex(linear_step_kernel<128>, grid, block, 0, st, true, a));
}

}  // extern "C"
