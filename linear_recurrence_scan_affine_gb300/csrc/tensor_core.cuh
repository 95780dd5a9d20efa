// tcgen05, tensor memory, tensor-map copies and the taking over of blocks for
// sm_103a: the PTX wrappers that the attention kernels and the losses use, with
// the operand layouts they assume.
//
// Operand tiles in shared memory are boxes of 64 bf16 columns (128 bytes) by
// R rows, 128-byte swizzled as the tensor-map copy writes them; a tile of 128
// columns is two such boxes, one after the other. A box starts on a 1024-byte
// boundary.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "scan_core.cuh"

namespace rlcs {
namespace tc {

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---------------------------------------------------------------------------
// Bounded waits. A wait that runs out raises `abort` for the block; every
// later wait of the block then returns at once, so all warps reach the end,
// where the block records the timeout and releases its tensor memory.
// ---------------------------------------------------------------------------
constexpr uint64_t kWaitNs = 2000000000ull;  // far above any tile's time

__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  uint64_t until = 0;
  for (int i = 0; !mbar_try_wait(bar, parity); ++i) {
    if (*abort) return false;
    if (i == 64) until = globaltimer_ns() + kWaitNs;
    if (i > 64 && globaltimer_ns() > until) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
// The whole warp waits, and goes on or gives up together.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  return __all_sync(kFull, mbar_wait(bar, parity, abort));
}
// One arrival for the whole warp, after what its lanes have done.
__device__ __forceinline__ void warp_arrive(uint64_t *bar, uint32_t lead) {
  __syncwarp();
  if (lead)
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// ---------------------------------------------------------------------------
// Tensor memory
// ---------------------------------------------------------------------------
// One warp, converged. The column count is a power of two from 32 to 512.
__device__ __forceinline__ void tmem_alloc(uint32_t *out, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(out)),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t base, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns)
               : "memory");
}
__device__ __forceinline__ void fence_before_sync() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after_sync() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 consecutive columns of this thread's lane (address: lane in bits 16..31,
// the warp's own 32 lanes; column in bits 0..15).
__device__ __forceinline__ void ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void ld8(uint32_t addr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}

__device__ __forceinline__ void st8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr)
      : "memory");
}

// ---------------------------------------------------------------------------
// Matrix products: D[128 x N] (+)= A[128 x 16] B[16 x N], bf16 in, fp32 out
// ---------------------------------------------------------------------------
// Instruction descriptor: fp32 accumulator (bits 4-5 = 1), bf16 A and B (bits
// 7-9, 10-12 = 1), B stored with N contiguous (bit 16) or with K contiguous,
// N/8 in bits 17-22, M/16 in bits 24-28. A is K-contiguous.
constexpr uint32_t instr(int n, bool b_n_contiguous) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_n_contiguous ? 1u : 0u) << 16) |
         ((uint32_t)(n / 8) << 17) | ((128u / 16) << 24);
}
// Shared-memory descriptor of a 128-byte-swizzled operand. Low word: start
// address and leading byte offset, in 16-byte units; high word: stride byte
// offset in 16-byte units, version 1 (bits 46-47), swizzle code 2 (bits
// 61-63). With K contiguous the stride offset is the 1024 bytes between
// groups of 8 rows (leading offset unused). With N contiguous it is the 1024
// bytes between groups of 8 k-rows, and the leading offset is the distance
// between 64-column boxes.
constexpr uint32_t kOperandHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
// (In a cluster a shared-memory address carries the block's rank above its
// 18 bits of offset.)
__device__ __forceinline__ uint32_t operand_k(uint32_t addr) {
  return ((addr & 0x3ffff) >> 4) | (1u << 16);
}
template <int ROWS>
__device__ __forceinline__ uint32_t operand_n(uint32_t addr) {
  return ((addr & 0x3ffff) >> 4) | ((ROWS * 128u >> 4) << 16);
}
// Products are issued by one lane, but every lane of its warp runs the code
// and `lead` predicates the instruction alone: in a branch taken by one lane
// each descriptor would be built in that lane's registers and moved over, and
// issuing a tile's products would take longer than running them.
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint32_t a, uint32_t b,
                                       uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 x, {%1, %6};\n\tmov.b64 y, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead), "r"(kOperandHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b,
                                       uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 y, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead), "r"(kOperandHigh)
      : "memory");
}
// Arrive on `bar` when every product the lead lane has issued is complete.
__device__ __forceinline__ void commit(uint32_t lead, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_addr(bar)),
      "r"(lead)
      : "memory");
}

// C[128 x N] = A[128 x DP] B[N x DP]^T, both K-contiguous in shared memory.
template <int DP, int N>
__device__ __forceinline__ void product_nt(uint32_t lead, uint32_t d, uint32_t a, uint32_t b) {
  const uint32_t x = operand_k(a), y = operand_k(b);
#pragma unroll
  for (int k = 0; k < DP / 16; ++k)
    mma_ss(lead, d, x + (((k / 4) * 16384 + (k % 4) * 32) >> 4),
           y + (((k / 4) * N * 128 + (k % 4) * 32) >> 4), instr(N, false), k > 0);
}
// C[128 x DP] (+)= A[128 x K] B[K x DP], B's rows contiguous in shared memory
// and A in tensor memory as bf16 pairs (8 columns per 16 of A): its K columns
// in PARTS pieces, each written by its own warps over the start of the K /
// PARTS fp32 columns they had read.
template <int DP, int K, int PARTS>
__device__ __forceinline__ void product_parts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b,
                                              bool add) {
  constexpr int kSteps = K / 16 / PARTS;
  const uint32_t y = operand_n<K>(b);
#pragma unroll
  for (int k = 0; k < K / 16; ++k)
    mma_ts(lead, d, a + (k / kSteps) * (K / PARTS) + (k % kSteps) * 8, y + k * (2048 >> 4),
           instr(DP, true), add || k > 0);
}

// ---------------------------------------------------------------------------
// Tensor-map copies
// ---------------------------------------------------------------------------
__device__ __forceinline__ void load_box(void *dst, const CUtensorMap *map, uint64_t *bar, int col,
                                         int head, int token) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(col), "r"(head), "r"(token)
      : "memory");
}
// A tile of ROWS tokens by DP columns: DP/64 boxes; columns past the array's
// width and tokens past its end read as zero.
template <int DP, int ROWS>
__device__ __forceinline__ void load_tile(unsigned char *dst, const CUtensorMap *map, uint64_t *bar,
                                          int head, int token) {
  mbar_arrive_expect_tx(bar, DP * ROWS * 2);
#pragma unroll
  for (int c = 0; c < DP / 64; ++c) load_box(dst + c * ROWS * 128, map, bar, c * 64, head, token);
}
// Zero rows [from, ROWS) of a tile that a copy has filled, by one warp.
template <int DP, int ROWS>
__device__ __forceinline__ void clear_rows(unsigned char *tile, int from, int lane) {
#pragma unroll
  for (int c = 0; c < DP / 64; ++c)
    for (int i = from * 8 + lane; i < ROWS * 8; i += 32)
      reinterpret_cast<uint4 *>(tile + c * ROWS * 128)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_shared();
}
// The signs' places of two bf16 values, set where one is infinite or NaN: its
// exponent's eight ones carry there.
__device__ __forceinline__ uint32_t special(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
// The same of eight values together.
__device__ __forceinline__ uint32_t special(const uint4 &x) {
  auto carry = [](uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; };
  return (carry(x.x) | carry(x.y) | carry(x.z) | carry(x.w)) & 0x80008000u;
}
// Zeros in place of such values of a tile, by one warp.
template <int DP, int ROWS>
__device__ __noinline__ void clear_special(unsigned char *tile, int lane) {
  uint32_t *w = reinterpret_cast<uint32_t *>(tile);
  for (int i = lane; i < DP * ROWS / 2; i += 32) {
    const uint32_t s = ((w[i] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
    if (s) w[i] &= (s & 0x8000u ? 0u : 0xffffu) | (s & 0x80000000u ? 0u : 0xffff0000u);
  }
  __syncwarp();
  fence_proxy_async_shared();
}

// ---------------------------------------------------------------------------
// Work of blocks that have not started
// ---------------------------------------------------------------------------
// Ask for a block that has not started; the answer goes to every block of the
// cluster. One thread of the cluster.
__device__ __forceinline__ void ask(uint4 *answer, uint64_t *bar, bool cluster) {
  if (cluster)
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
        ".multicast::cluster::all.b128 [%0], [%1];" ::"r"(smem_addr(answer)),
        "r"(smem_addr(bar))
        : "memory");
  else
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
        ".b128 [%0], [%1];" ::"r"(smem_addr(answer)),
        "r"(smem_addr(bar))
        : "memory");
}
// The block whose place was given, or -1.
__device__ __forceinline__ int64_t granted(const uint4 *answer) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_addr(answer))
      : "memory");
  return ok ? (int64_t)x : -1;
}
// Host: the map of a [tokens, heads, D] bf16 view, in 64-column boxes of
// `rows` tokens of one head.
inline bool make_map(CUtensorMap *map, const void *base, int64_t tokens, int64_t heads, int64_t D,
                     int64_t token_stride, int64_t head_stride, int rows) {
  using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)token_stride * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows}, one[3] = {1, 1, 1};
  auto make = [&] {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
                  strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = make();
  int dev = 0;
  // A thread whose first CUDA call this is has no context yet, which the
  // runtime's calls would have given it.
  if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess &&
      cudaSetDevice(dev) == cudaSuccess)
    r = make();
  return r == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace rlcs
