// Distillation from a teacher's top logits and its gradient (rlcs_loss.h).
#include "loss_rows.cuh"

namespace rlcs {
namespace loss {
namespace {

// The highest code that a call has recorded on this device.
__device__ uint32_t device_status;
constexpr int kMaxTop = 1024;
static_assert(2 * (kMaxTop * 16 + 2 * kMaxTop * 8) <= kLongEntries,
              "a block holds a token's entries");

struct DistillArgs {
  const void *logits;
  int64_t row_stride;
  const int32_t *ids;
  const float *top, *teacher_lse;
  const uint8_t *mask;
  const float *dloss;
  void *dlogits;
  float *loss;
  int64_t tokens, V;
  int K, slots;  // slots: of the table of ids, a power of two
  float inv_t;
};


// ---------------------------------------------------------------------------
// A token's entries, by the lanes of a warp or of a part of one
// ---------------------------------------------------------------------------
// Shared memory of one team: K of each, and a table that finds ids which occur
// more than once.
struct Entries {
  int *id;    // -1 where absent
  float *q;   // the teacher's logit, then q
  float *lq;  // log q
  float *x;   // the student's logit
  int *table, *times;
  int K, slots;
};
inline int slots_of(int K) {
  int n = 2;
  while (n < 2 * K) n *= 2;
  return n;
}
inline size_t entry_bytes(int K) { return (size_t)K * 16 + (size_t)slots_of(K) * 8; }
__device__ __forceinline__ Entries entries_at(float *raw, int K, int slots) {
  Entries e;
  e.id = reinterpret_cast<int *>(raw);
  e.q = raw + K;
  e.lq = raw + 2 * K;
  e.x = raw + 3 * K;
  e.table = reinterpret_cast<int *>(raw + 4 * K);
  e.times = e.table + slots;
  e.K = K;
  e.slots = slots;
  return e;
}
__device__ __forceinline__ bool absent(const DistillArgs &p, int id, float t) {
  return id < 0 || id >= p.V || t == -INFINITY;
}
// Teachers' logits are taken from their largest before anything else: an offset
// that they have in common costs no digits, and one at the type's lowest value
// has no weight, whatever the temperature makes of it. z is the sum of
// exp((t - top) / T).
__device__ __forceinline__ void add_entry(const DistillArgs &p, float t, Stats &sum) {
  if (t > sum.top) sum.z *= expf((sum.top - t) * p.inv_t), sum.top = t;  // (0 at first)
  sum.z += expf((t - sum.top) * p.inv_t);
}
__device__ __forceinline__ float log_q(const DistillArgs &p, int64_t row, const Stats &sum,
                                       float log_sum, float t) {
  return p.teacher_lse ? fmaf(t, p.inv_t, -p.teacher_lse[row])
                       : (t - sum.top) * p.inv_t - log_sum;
}
// The sum of q, of entries that have any.
__device__ __forceinline__ float mass_of(const DistillArgs &p, int64_t row, const Stats &sum) {
  return p.teacher_lse ? sum.z * expf(fmaf(sum.top, p.inv_t, -p.teacher_lse[row])) : 1.0f;
}
template <int LANES>
__device__ __forceinline__ Stats join_entries(const DistillArgs &p, const Stats &sum) {
  const float top = lanes_max<LANES>(sum.top);
  const float f = sum.top == top ? 1.0f : expf((sum.top - top) * p.inv_t);
  return {top, lanes_sum<LANES>(f * sum.z), 0.0f};
}
// One entry, and the lane's sum over its entries.
__device__ __forceinline__ void enter(const DistillArgs &p, const Entries &en, int j, int id,
                                      float t, float x, Stats &sum) {
  if (absent(p, id, t)) id = -1;
  en.id[j] = id;
  en.q[j] = t;
  en.x[j] = x;
  if (id >= 0) add_entry(p, t, sum);
}
// After all have been entered: q, log q and their mass, and the table of ids to
// begin with. Only an id that occurs twice is looked for in all entries, in their
// order.
template <int LANES>
__device__ __forceinline__ float settle(const DistillArgs &p, const Entries &en, int64_t row,
                                        const Stats &sum, int lane, bool on, bool grad) {
  float mass = 1.0f;
  if (on) {
    const float log_sum = logf(sum.z);
    mass = mass_of(p, row, sum);
    for (int j = lane; j < en.K; j += LANES) {
      const float lq = log_q(p, row, sum, log_sum, en.q[j]);
      en.lq[j] = lq;
      en.q[j] = expf(lq);
    }
    if (grad)
      for (int i = lane; i < en.slots; i += LANES) en.table[i] = -1, en.times[i] = 0;
  }
  __syncwarp();
  return mass;
}
__device__ __forceinline__ int slot_of(const Entries &en, int id) {
  return (int)((unsigned)id * 2654435761u >> 7) & (en.slots - 1);
}
template <int LANES>
__device__ __forceinline__ void count(const Entries &en, int lane, bool on) {
  if (on)
    for (int j = lane; j < en.K; j += LANES) {
      const int id = en.id[j];
      if (id < 0) continue;
      // (half of the slots stay free)
      for (int s = slot_of(en, id);; s = (s + 1) & (en.slots - 1)) {
        const int was = atomicCAS(&en.table[s], -1, id);
        if (was == -1 || was == id) {
          atomicAdd(&en.times[s], 1);
          break;
        }
      }
    }
  __syncwarp();
}
__device__ __forceinline__ float target(const Entries &en, int j) {
  const int id = en.id[j];
  int s = slot_of(en, id);
  while (en.table[s] != id) s = (s + 1) & (en.slots - 1);
  if (en.times[s] == 1) return en.q[j];
  float sum = 0.0f;
  for (int i = 0; i < en.K; ++i)
    if (en.id[i] == id) sum += en.q[i];
  return sum;
}
// The lane's part of the loss.
template <int LANES>
__device__ __forceinline__ float loss_part(const Entries &en, const Base &base, float c,
                                           float logz, int lane) {
  const float ln2 = log_of_2(base, c);
  float loss = 0.0f;
  for (int j = lane; j < en.K; j += LANES) {
    const float e = en.q[j];
    if (en.id[j] >= 0 && (e > 0.0f || e != e))
      loss += e * (en.lq[j] - (base.y(en.x[j]) * ln2 - logz));
  }
  return loss;
}

template <class T, bool GRAD, int TEAM, int NV>
__global__ void __launch_bounds__(kTeamBlock, team_blocks(NV))
    distill_team_kernel(const DistillArgs p) {
  extern __shared__ float raw[];
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kTeams = kTeamBlock / TEAM;
  const int lane = threadIdx.x % TEAM;
  const Entries en = entries_at(raw + threadIdx.x / TEAM * (4 * p.K + 2 * p.slots), p.K, p.slots);
  const int64_t step = (int64_t)gridDim.x * kTeams;
  int64_t row = (int64_t)blockIdx.x * kTeams + threadIdx.x / TEAM;
  const auto any = [&](bool on) { return TEAM < 32 ? __any_sync(kFull, on) : on; };
  const auto live = [&](int64_t i) { return i < p.tokens && (!p.mask || p.mask[i]); };
  const auto see = [&](int64_t i) { return row_of<T>(p, i < p.tokens ? i : 0, lane, 0, 1); };
  const float c = p.inv_t * kLog2e;
  bool on = live(row);
  Row<T> r = see(row);
  uint4 q[NV];
  load_row<T, TEAM, NV>(q, r, on);
  while (any(row < p.tokens)) {
    const int64_t next = row + step;
    const bool more = live(next);
    const Row<T> rn = see(next);
    const T *x = static_cast<const T *>(p.logits) + row * p.row_stride;
    Stats te = {-INFINITY, 0.0f, 0.0f};
    if (on) {
      trim_row<T, TEAM, NV>(q, p, row, r);
      for (int j = lane; j < p.K; j += TEAM) {
        const int id = p.ids[row * p.K + j];
        const float t = p.top[row * p.K + j];
        enter(p, en, j, id, t, absent(p, id, t) ? 0.0f : value(x + id), te);
      }
    }
    te = join_entries<TEAM>(p, te);
    on = on && te.z != 0.0f;  // (a NaN is an entry)
    const float mass = settle<TEAM>(p, en, row, te, lane, on, GRAD);
    if (GRAD) count<TEAM>(en, lane, on);
    const Stats s = lanes_stats<T, TEAM, NV, false>(q, c, NV);
    const Base base = base_of(s.top, c);
    const float loss = lanes_sum<TEAM>(on ? loss_part<TEAM>(en, base, c, logf(s.z), lane) : 0.0f);
    if (row < p.tokens && lane == 0 && p.loss) p.loss[row] = loss;
    const float w = GRAD && on ? p.dloss[row] * p.inv_t : 0.0f;
    const Coefficients k = {w * mass / s.z, 0.0f};
    T *dx = GRAD ? static_cast<T *>(p.dlogits) + row * p.V : nullptr;
    if (row < p.tokens) {
      const auto none = [](float2(&)[kWord<T> / 2], int) {};
      if (on)
        use_row<T, GRAD, TEAM, NV, true, false>(q, r, base, k, rn, more, dx, p.V, none);
      else
        use_row<T, GRAD, TEAM, NV, false, false>(q, r, base, k, rn, more, dx, p.V, none);
    }
    __syncwarp();
    // then the few elements with a target, again
    if (GRAD && on)
      for (int j = lane; j < p.K; j += TEAM)
        if (en.id[j] >= 0)
          put(dx + en.id[j], fmaf(ex2(base.y(en.x[j])), k.a, -w * target(en, j)));
    __syncwarp();
    row = next;
    r = rn;
    on = more;
  }
}

// A token's entries are gone through by its thread, in their order.
template <class T, bool GRAD>
__global__ void __launch_bounds__(kFewBlock) distill_few_kernel(const DistillArgs p) {
  extern __shared__ float x[];
  __shared__ uint8_t live[kFewBlock];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row0 = (int64_t)blockIdx.x * kFewBlock, row = row0 + threadIdx.x;
  const int rows = p.tokens - row0 < kFewBlock ? (int)(p.tokens - row0) : kFewBlock;
  const int V = (int)p.V, pitch = V | 1;
  const bool held = row < p.tokens;
  bool on = held && (!p.mask || p.mask[row]);
  live[threadIdx.x] = on;
  const int32_t *ids = p.ids + row * p.K;
  const float *top = p.top + row * p.K;
  Stats te = {-INFINITY, 0.0f, 0.0f};
  if (on)
    for (int j = 0; j < p.K; ++j)
      if (!absent(p, ids[j], top[j])) add_entry(p, top[j], te);
  if (p.mask) __syncthreads();
  few_copy<T, true>(p, static_cast<T *>(nullptr), x, rows, row0, pitch,
                    [&](int i) { return !p.mask || live[i]; });
  __syncthreads();
  on = on && te.z != 0.0f;  // (a NaN is an entry)
  float *mine = x + threadIdx.x * pitch;
  float loss = 0.0f;
  if (on) {
    const float c = p.inv_t * kLog2e;
    const Stats s = few_stats<false>(mine, V, c);
    const Base base = base_of(s.top, c);
    const float logz = logf(s.z), ln2 = log_of_2(base, c);
    const float log_sum = logf(te.z);
    for (int j = 0; j < p.K; ++j) {
      if (absent(p, ids[j], top[j])) continue;
      const float lq = log_q(p, row, te, log_sum, top[j]), e = expf(lq);
      if (e > 0.0f || e != e) loss += e * (lq - (base.y(mine[ids[j]]) * ln2 - logz));
    }
    if (GRAD) {
      const float w = p.dloss[row] * p.inv_t, a = w * mass_of(p, row, te) / s.z;
      for (int i = 0; i < V; ++i) mine[i] = ex2(base.y(mine[i])) * a;
      for (int j = 0; j < p.K; ++j)
        if (!absent(p, ids[j], top[j]))
          mine[ids[j]] -= w * expf(log_q(p, row, te, log_sum, top[j]));
    }
  } else if (GRAD && held) {
    for (int i = 0; i < V; ++i) mine[i] = 0.0f;
  }
  if (held && p.loss) p.loss[row] = loss;
  if (!GRAD) return;
  __syncthreads();
  few_copy<T, false>(p, static_cast<T *>(p.dlogits), x, rows, row0, pitch,
                     [](int) { return true; });
}

// The teacher's warp: a lane's first kHeld entries are asked for together. Two
// sets of entries take turns: a row's are made ready while the row before is
// stored.
struct Taught {
  float mass, w;  // of the teacher's q; dloss / T
  int any;        // entries at all
};
template <class T, bool GRAD>
struct DistillLeader {
  static constexpr bool kTeacher = true;
  static constexpr int kHeld = 4;
  const DistillArgs &p;
  float *raw;
  Taught *taught;  // in shared memory, by turns
  int turn;
  __device__ __forceinline__ Entries set(int i) const {
    return entries_at(raw + i * (4 * p.K + 2 * p.slots), p.K, p.slots);
  }
  __device__ __forceinline__ void ahead(int64_t, bool) {}
  __device__ __forceinline__ void before(int64_t, bool) {}
  // The teacher's warp has put the student's logits of its entries into shared
  // memory: they have been read.
  __device__ __forceinline__ float held() const {
    meet_wait<64>(kTaught);
    return 0.0f;
  }
  __device__ __forceinline__ void plan(int64_t, const Stats &s, bool, int, LongSmem &sm) {
    if ((threadIdx.x & 31) == 0) {
      const Taught t = taught[turn];
      sm.k = {t.w * t.mass / s.z, 0.0f};
      sm.word = -1;
      sm.on = t.any;
    }
    turn ^= 1;
  }

  __device__ __forceinline__ void prepare(int64_t row, bool on, int turn) {
    const int lane = threadIdx.x & 31;
    const Entries en = set(turn);
    const T *x = static_cast<const T *>(p.logits) + row * p.row_stride;
    Stats te = {-INFINITY, 0.0f, 0.0f};
    float w = 0.0f;
    if (on) {
      if (GRAD) w = p.dloss[row] * p.inv_t;
      int id[kHeld];
      float t[kHeld], held[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (lane + 32 * i < p.K) {
          id[i] = p.ids[row * p.K + lane + 32 * i];
          t[i] = p.top[row * p.K + lane + 32 * i];
        }
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        held[i] = lane + 32 * i < p.K && !absent(p, id[i], t[i]) ? value(x + id[i]) : 0.0f;
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (lane + 32 * i < p.K) enter(p, en, lane + 32 * i, id[i], t[i], held[i], te);
      for (int j = lane + 32 * kHeld; j < p.K; j += 32) {
        const int i = p.ids[row * p.K + j];
        const float v = p.top[row * p.K + j];
        enter(p, en, j, i, v, absent(p, i, v) ? 0.0f : value(x + i), te);
      }
    }
    te = join_entries<32>(p, te);
    const bool any = on && te.z != 0.0f;  // (a NaN is an entry)
    const float mass = settle<32>(p, en, row, te, lane, any, GRAD);
    if (lane == 0) taught[turn] = {mass, any ? w : 0.0f, any};
    meet_arrive<64>(kTaught);
    if (GRAD) count<32>(en, lane, any);
  }
  __device__ __forceinline__ void teach(int64_t row, bool on, int rank, int ranks, LongSmem &sm) {
    const int lane = threadIdx.x & 31;
    prepare(row, on, 0);
    for (int turn = 0; row < p.tokens; turn ^= 1) {
      meet_wait<kLongBlock + 32>(kPlanned + turn);
      const int64_t next = sm.next[turn];
      const bool more = sm.more[turn];
      const Stats s = sm.whole;
      if (next < p.tokens) prepare(next, more, turn ^ 1);
      const Entries en = set(turn);
      const Taught t = taught[turn];
      const float c = p.inv_t * kLog2e;
      const Base base = base_of(s.top, c);
      if (rank == 0) {
        const float loss =
            lanes_sum<32>(t.any ? loss_part<32>(en, base, c, logf(s.z), lane) : 0.0f);
        if (lane == 0 && p.loss) p.loss[row] = loss;
      }
      if (GRAD) {
        const Row<T> r = row_of<T>(p, row, 0, rank, ranks);
        T *dx = static_cast<T *>(p.dlogits) + row * p.V;
        const float scale = t.w * t.mass / s.z;
        meet_wait(kStored);  // then the few elements with a target, again
        if (t.any)
          for (int j = lane; j < p.K; j += 32) {
            const int id = en.id[j], word = (id + r.skip) / kWord<T> - r.w0;
            if (id >= 0 && word >= 0 && word < r.left)
              put(dx + id, fmaf(ex2(base.y(en.x[j])), scale, -t.w * target(en, j)));
          }
        __syncwarp();
      }
      row = next;
    }
  }
};

template <class T, bool GRAD, int NV>
__global__ void __launch_bounds__(kLongBlock + 32, long_blocks(NV))
    distill_long_kernel(const DistillArgs p) {
  extern __shared__ __align__(128) unsigned char dynamic[];
  __shared__ Taught taught[2];
  pdl_wait();
  pdl_launch_dependents();
  float *raw = reinterpret_cast<float *>(dynamic + NV * kTeam * 16);  // behind a row's words
  DistillLeader<T, GRAD> leader = {p, raw, taught, 0};
  long_rows<T, GRAD, NV, false>(p, p.inv_t * kLog2e, &device_status, leader);
}

template <class T, bool GRAD>
__global__ void __launch_bounds__(kThreads) distill_rows_kernel(const DistillArgs p) {
  __shared__ float part[32], q[kMaxTop], logq[kMaxTop], at[kMaxTop];
  __shared__ int id[kMaxTop];
  pdl_wait();
  pdl_launch_dependents();
  const float c = p.inv_t * kLog2e;
  for (int64_t row = blockIdx.x; row < p.tokens; row += gridDim.x) {
    const T *x = static_cast<const T *>(p.logits) + row * p.row_stride;
    T *dx = GRAD ? static_cast<T *>(p.dlogits) + row * p.V : nullptr;
    bool on = !p.mask || p.mask[row];
    float top = -INFINITY;
    __syncthreads();
    if (on)
      for (int j = threadIdx.x; j < p.K; j += kThreads) {
        const int i = p.ids[row * p.K + j];
        const float v = p.top[row * p.K + j];
        const bool there = i >= 0 && i < p.V && !(v == -INFINITY);
        id[j] = there ? i : -1;
        logq[j] = v;
        at[j] = there ? value(x + i) : 0.0f;
        if (there) top = fmaxf(top, v != v ? INFINITY : v);
      }
    top = block_max(top, part);
    on = on && top > -INFINITY;
    if (!on) {
      if (threadIdx.x == 0 && p.loss) p.loss[row] = 0.0f;
      if (GRAD)
        for (int64_t i = threadIdx.x; i < p.V; i += kThreads) put(dx + i, 0.0f);
      continue;
    }
    Stats te = {top, 0.0f, 0.0f};
    if (!p.teacher_lse) {
      for (int j = threadIdx.x; j < p.K; j += kThreads)
        if (id[j] >= 0) te.z += expf((logq[j] - top) * p.inv_t);
      te.z = block_sum(te.z, part);
    }
    const float log_sum = logf(te.z);
    const Stats s = row_stats<T, false>(x, p.V, c, part);
    const Base base = base_of(s.top, c);
    const float logz = logf(s.z), ln2 = log_of_2(base, c);
    float mass = 0.0f, loss = 0.0f;
    for (int j = threadIdx.x; j < p.K; j += kThreads) {
      q[j] = 0.0f;
      if (id[j] < 0) continue;
      const float lq = log_q(p, row, te, log_sum, logq[j]), e = expf(lq);
      q[j] = e;
      mass += e;
      if (e > 0.0f || e != e) loss += e * (lq - (base.y(at[j]) * ln2 - logz));
    }
    mass = block_sum(mass, part);
    loss = block_sum(loss, part);
    if (threadIdx.x == 0 && p.loss) p.loss[row] = loss;
    if (!GRAD) continue;
    const float w = p.dloss[row] * p.inv_t, a = w * mass / s.z;
    for (int64_t i = threadIdx.x; i < p.V; i += kThreads)
      put(dx + i, ex2(base.y(value(x + i))) * a);
    __syncthreads();  // then the few elements with a target, again
    for (int j = threadIdx.x; j < p.K; j += kThreads) {
      if (id[j] < 0) continue;
      float target = 0.0f;
      for (int i = 0; i < p.K; ++i)
        if (id[i] == id[j]) target += q[i];
      put(dx + id[j], fmaf(ex2(base.y(at[j])), a, -w * target));
    }
  }
}

template <class T, bool GRAD>
struct Distill {
  static rlcs_status few(const DistillArgs &p, cudaStream_t st) {
    return launch_few<distill_few_kernel<T, GRAD>>(p, st);
  }
  template <int TEAM, int NV>
  static rlcs_status team(const DistillArgs &p, size_t entries, cudaStream_t st) {
    return launch_team<distill_team_kernel<T, GRAD, TEAM, NV>, TEAM>(p, team_blocks(NV), entries,
                                                                     st);
  }
  template <int NV>
  static rlcs_status block(const DistillArgs &p, int ranks, size_t entries, cudaStream_t st) {
    return launch_long<distill_long_kernel<T, GRAD, NV>, NV>(p, kLongBlock + 32, ranks, 2 * entries,
                                                              st);
  }
  static rlcs_status any(const DistillArgs &p, cudaStream_t st) {
    return launch_any(distill_rows_kernel<T, GRAD>, p, st);
  }
};

rlcs_status run_distill(DistillArgs p, int64_t K, bool grad, double temperature, rlcs_dtype dtype,
                        rlcs_stream_t stream) {
  if (K < 1 || K > kMaxTop || !(temperature >= 1e-6 && temperature <= 1e6))
    return RLCS_ERR_INVALID_ARG;
  const rlcs_status st = check_rows(p, grad, dtype);
  if (st != RLCS_OK || p.tokens == 0) return st;
  if (!p.ids || !p.top || !product_fits(p.tokens, K, 4)) return RLCS_ERR_INVALID_ARG;
  const int64_t n = p.tokens * 4;
  const Range outs[] = {range(p.dlogits, p.tokens * p.V * esize(dtype)), range(p.loss, n)};
  const Range x = range(p.logits, ((p.tokens - 1) * p.row_stride + p.V) * esize(dtype));
  const Range ins[] = {logits_range(p, dtype),  range(p.ids, n * K), range(p.top, n * K),
                       range(p.teacher_lse, n), range(p.mask, p.tokens), range(p.dloss, n)};
  if (outputs_overlap(outs, ins) || meet(outs[1], x)) return RLCS_ERR_INVALID_ARG;
  p.K = (int)K;
  p.inv_t = (float)(1.0 / temperature);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.slots = slots_of(p.K);
  const size_t entries = entry_bytes(p.K);
  if (dtype == RLCS_F32)
    return grad ? spread<float, Distill<float, true>>(p, entries, s)
                : spread<float, Distill<float, false>>(p, entries, s);
  return grad ? spread<bf, Distill<bf, true>>(p, entries, s)
              : spread<bf, Distill<bf, false>>(p, entries, s);
}

}  // namespace

rlcs_status distill_status() { return take_status(&device_status); }

}  // namespace loss
}  // namespace rlcs

using namespace rlcs;
using namespace rlcs::loss;

extern "C" {

rlcs_status rlcs_distill_loss(const void *logits, int64_t row_stride, const int32_t *top_ids,
                              const float *top_logits, const float *teacher_lse,
                              const uint8_t *mask, float *loss, int64_t tokens, int64_t V,
                              int64_t K, double temperature, rlcs_dtype dtype,
                              rlcs_stream_t stream) {
  const DistillArgs p = {logits, row_stride, top_ids, top_logits, teacher_lse, mask, nullptr,
                         nullptr, loss, tokens, V, 0, 0, 0};
  return run_distill(p, K, false, temperature, dtype, stream);
}

rlcs_status rlcs_distill_loss_backward(const float *dloss, const void *logits, int64_t row_stride,
                                       const int32_t *top_ids, const float *top_logits,
                                       const float *teacher_lse, const uint8_t *mask,
                                       void *dlogits, float *loss, int64_t tokens, int64_t V,
                                       int64_t K, double temperature, rlcs_dtype dtype,
                                       rlcs_stream_t stream) {
  const DistillArgs p = {logits, row_stride, top_ids, top_logits, teacher_lse, mask, dloss,
                         dlogits, loss, tokens, V, 0, 0, 0};
  return run_distill(p, K, true, temperature, dtype, stream);
}

}  // extern "C"
