// The fifth-generation tensor cores as the output layer's products use them:
// operand tiles brought into shared memory by tensor copies (TMA), tcgen05.mma
// issued by one thread, accumulators in tensor memory.  Thin wrappers over the
// PTX instructions, and the descriptors that they take.
#pragma once

#include <cuda.h>

#include "device.cuh"

namespace cgk {
namespace tc {

// ---- clusters --------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address, in the cluster's window, of what `local` (a shared address) is in block `rank`
__device__ __forceinline__ uint32_t in_block(uint32_t local, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  return a;
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_address) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_address) : "memory");
}
__device__ __forceinline__ void fence_barrier_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// whether a phase is over, without waiting
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok)
               : "r"(smem_addr(bar)), "r"(parity)
               : "memory");
  return ok != 0;
}

// ---- tensor copies ---------------------------------------------------------------------
// A box of a three-dimensional map into this block's shared memory.  With a pair of blocks
// the bytes are counted on a barrier of either block of the pair (cluster address).  The
// innermost coordinate is a multiple of 64 elements of 2 bytes at every call: on the
// 16-byte grid that the copies want.
template <int CTAS>
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  if (CTAS == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// A box from this block's shared memory, to be written or (floats) added to what is there
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t from, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x), "r"(y),
               "r"(z), "r"(from)
               : "memory");
}
__device__ __forceinline__ void add_box(const CUtensorMap* map, uint32_t from, int x, int y, int z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
               "r"(x), "r"(y), "r"(z), "r"(from)
               : "memory");
}
__device__ __forceinline__ void stores_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// all but the newest N groups have read their shared memory / are done
template <int N>
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- tensor memory ---------------------------------------------------------------------
constexpr uint32_t kTmemColumns = 512;

// by one whole warp; the address is written to shared memory
template <int CTAS>
__device__ __forceinline__ void tmem_alloc(uint32_t* where) {
  if (CTAS == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)),
                 "r"(kTmemColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)),
                 "r"(kTmemColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}
template <int CTAS>
__device__ __forceinline__ void tmem_free(uint32_t at) {
  if (CTAS == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(kTmemColumns));
  else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(kTmemColumns));
}
// 32 columns of the warp's 32 lanes, thread i gets lane i's; complete after tmem_wait
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]) : "r"(at));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---- matrix instructions ---------------------------------------------------------------

// Shared-memory operand descriptor, 128-byte swizzle (bits 61-63 = 2), version 1 (bit 46):
// address, leading and stride byte offsets in units of 16 bytes.
// K-major (k contiguous): rows of 64 k = 128 bytes, 8-row groups 1024 bytes apart; the
// leading offset is not used.  MN-major: boxes of 64 mn (128 bytes) x 64 k; 8-k groups
// 1024 bytes apart (stride), boxes 8192 bytes apart (leading).
template <bool MN>
__device__ __forceinline__ uint64_t operand(uint32_t address) {
  constexpr uint64_t fixed = (uint64_t(2) << 61) | (uint64_t(1) << 46) | (uint64_t(1024 >> 4) << 32) |
                             (uint64_t(MN ? 8192 >> 4 : 1) << 16);
  return fixed | ((address & 0x3FFFFu) >> 4);
}
// the next 16 k: 32 bytes along a K-major row, two 8-k groups of a MN-major box
template <bool MN>
constexpr uint64_t kStep16 = MN ? (2048 >> 4) : (32 >> 4);

// bf16 x bf16 with 32-bit sums: D format (bit 4), A and B formats (7, 10), A and B
// MN-major (15, 16), N / 8 (17), M / 16 (24)
template <bool A_MN, bool B_MN>
constexpr uint32_t instruction(uint32_t m, uint32_t n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(A_MN) << 15) | (uint32_t(B_MN) << 16) | ((n >> 3) << 17) |
         ((m >> 4) << 24);
}

template <int CTAS>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t instr, bool add) {
  if (CTAS == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(instr), "r"(uint32_t(add))
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(instr), "r"(uint32_t(add))
        : "memory");
}
// one arrival, at the barrier of this place in every block of the pair, once the matrix
// instructions issued so far are done
template <int CTAS>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if (CTAS == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(uint16_t(3))
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// ---- host: tensor maps -----------------------------------------------------------------

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiled encode_tiled() {
  static const EncodeTiled f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return f;
}

// [parts][rows][width] of bf16 (or float), rows `ld` elements apart, boxes of 128 bytes x
// box_rows with a 128-byte swizzle; what lies outside reads as zero and is not written, but for
// the rest of the 16 bytes that a row's last element lies in: a store writes those too.  The
// address and the row pitch are multiples of 16 bytes.
inline bool make_map(CUtensorMap* map, const void* at, uint64_t width, uint64_t rows, uint64_t parts, uint64_t ld,
                     uint64_t part_stride, uint32_t box_rows, bool f32 = false) {
  const EncodeTiled f = encode_tiled();
  if (!f) return false;
  const uint32_t size_of = f32 ? 4 : 2;
  const cuuint64_t size[3] = {width, rows, parts};
  const cuuint64_t pitch[2] = {ld * size_of, part_stride * size_of};
  const cuuint32_t box[3] = {128 / size_of, box_rows, 1}, step[3] = {1, 1, 1};
  return f(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(at), size,
           pitch, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace cgk
