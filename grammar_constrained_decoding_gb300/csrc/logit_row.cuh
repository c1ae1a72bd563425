// Rows of logits held on chip, the frame of the per-row operators
// (sample_rows, top_logprobs, and distill's gradient of short rows and small batches).
//
// A row belongs to a cluster of n <= 16 blocks of 256 threads.  Each block copies
// its part once into shared memory (bulk copies completing on mbarriers), and
// every pass an operator makes over the row reads it there, so the row is read
// from memory once.  A thread only ever reads the 16-byte groups (8 bf16 or 4
// floats) that are its own, so the passes need no barriers between them.
//
// An earlier form held the parts in registers: 32 of them a thread spilled in the
// longer passes, whose traffic (118 MB written for 66 MB of logits) cost more
// than the row, and its unrolled passes missed the instruction cache.
//
// Groups lie on the 16-byte grid of the memory, not of the row: a row that starts
// off the grid has a first group with some elements before the row, which its
// thread loads one by one, and every other group is copied whatever the row's
// alignment.
//
// The blocks exchange what they must (maxima, sums, bounds, entries) through one
// another's shared memory.  Short messages go as asynchronous stores that
// complete on the receiver's mbarrier: the sender neither fences nor waits (a
// cluster barrier with release semantics made every thread wait for its stores,
// the longest stall of an earlier form).
//
// A logit that is -inf or NaN, or whose bitmask bit is clear, is not allowed
// and reads as -inf; +inf reads as the largest finite value.
#pragma once

#include <cfloat>

#include "bf16_ops.cuh"
#include "device_answers.h"

namespace cgk {
namespace row {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kWarps = kThreads / 32;
constexpr uint32_t kMaxCluster = 16;   // more than 8 is not portable, but the one target has it
constexpr uint32_t kBinBits = 9;
constexpr uint32_t kBins = 1u << kBinBits;  // bins of one selection level
constexpr uint32_t kListCap = 1024;    // entries of a list
constexpr uint32_t kStage = 512;       // entries a block may send
constexpr uint32_t kPairCap = kThreads;  // lists ranked by comparing all pairs, an entry a thread
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMaxBf16 = 3.38953138925e38f;  // largest finite bf16
constexpr uint32_t kKeyInf = 0xFF800000u;      // fkey(+inf); NaN keys lie above
constexpr uint32_t kKeyLowest = 0x00800000u;   // fkey(-FLT_MAX); fkey(-inf) lies below

template <bool BF16>
struct Fmt {
  static constexpr uint32_t E = BF16 ? 8 : 4;         // elements per group
  static constexpr uint32_t kSize = BF16 ? 2 : 4;     // bytes per element
  static constexpr uint32_t kNegInf = BF16 ? 0xFF80FF80u : 0xFF800000u;
  // selection keys: the bits that tell two logits of the type apart
  static __device__ __forceinline__ uint32_t key(float x) { return BF16 ? fkey(x) >> 16 : fkey(x); }
};

// ---- clusters ---------------------------------------------------------------------

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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// address of the same shared variable in the block of rank r
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t r) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(r));
  return a;
}
__device__ __forceinline__ void st_remote(uint32_t a, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
// asynchronous stores that complete 4, 8 or 16 bytes on a barrier of the block
// that a lies in
__device__ __forceinline__ void send(uint32_t a, uint32_t v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(a), "r"(v),
               "r"(bar)
               : "memory");
}
__device__ __forceinline__ void send(uint32_t a, unsigned long long v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(a), "l"(v),
               "r"(bar)
               : "memory");
}
__device__ __forceinline__ void send(uint32_t a, uint4 v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a),
               "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(bar)
               : "memory");
}
// Asks for [from, to) of global memory to be brought to L2 (whole 16-byte pieces of it)
__device__ __forceinline__ void prefetch_l2(const void* from, const void* to) {
  const uintptr_t a = (reinterpret_cast<uintptr_t>(from) + 15) & ~uintptr_t(15);
  const uintptr_t b = reinterpret_cast<uintptr_t>(to) & ~uintptr_t(15);
  if (b > a) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a), "r"(uint32_t(b - a)) : "memory");
}
// bounded wait for what others have sent
__device__ __forceinline__ bool wait_sent(uint64_t* bar, uint32_t parity = 0) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  return false;
}
__device__ __forceinline__ uint32_t add_remote(uint32_t a, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(a), "r"(v) : "memory");
  return old;
}
__device__ __forceinline__ void ld_remote2(uint32_t a, unsigned long long& x, unsigned long long& y) {
  asm volatile("ld.shared::cluster.v2.u64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(a) : "memory");
}
// all blocks of the cluster (a cluster of one: the block)
__device__ __forceinline__ void cluster_sync(uint32_t n) {
  if (n == 1) {
    __syncthreads();
  } else {
    cluster_arrive();
    cluster_wait();
  }
}
// A block whose wait ran out does not leave before the others of its cluster, who may
// still send to its shared memory or read it.  Threads that have left count as arrived,
// so a round ends when the others meet once more or are gone; they meet less than kMeets
// times (a selection has five levels at most, and there are two of them).  The others'
// waits are bounded, so they come to their end.  For all threads of the block that have
// not left.
constexpr uint32_t kMeets = 32;
__device__ __forceinline__ void leave_last(uint32_t n) {
#pragma unroll 1
  for (uint32_t i = 0; n > 1 && i < kMeets; ++i) {
    cluster_arrive();
    cluster_wait();
  }
}

constexpr uint32_t kMaxRecords = kMaxCluster * kWarps;  // warps of a cluster
constexpr uint32_t kMaxBounds = 512;                     // group maxima a cluster exchanges

// Exponentials are taken as exp2((x - m) c): the difference to a maximum first, which
// is exact near it, so that no size of x or c costs precision or overflows.

// What a warp tells all blocks about its part of the row: its maximum and the sum of
// exp2((x - m) c) over its elements but one that is the maximum.  Without that 1 the sum
// is as good where the maximum has nearly all the mass: log p = -log(1 + rest) of such a
// token had errors of 4e-7 with the 1 inside, 1e-4 of a log p of 0.003, all of one of 5e-9.
struct __align__(8) Record {
  float m, rest;
};
// What a block tells about the entries it has sent.
struct __align__(8) Tally {
  float mass;
  uint32_t count;   // kTooMany: not sent
};
constexpr float kMassOne = 1099511627776.f;  // mass_q of the maximum
constexpr uint32_t kTooMany = 0xFFFFFFFFu;
constexpr uint32_t kChunk = 4;       // groups a thread takes at a time
constexpr uint32_t kMaxChunks = 8;
constexpr uint32_t kBars = 5 + kMaxChunks;
constexpr uint32_t kMaxGroups = kChunk * kMaxChunks;  // of a thread: a lane a copy

// What every operator's cluster meets in: barriers, records, reductions
struct __align__(16) Meet {
  uint64_t bar_rec, bar_tally, bar_list, bar_best, bar_mass;  // kBars barriers in a row ...
  uint64_t bar_part[kMaxChunks];                              // ... the last for the copies of this block's part
  float M, rest;                       // what the merging warp found
  uint32_t late;                       // a bounded wait ran out
  uint32_t n_list, n_local, n_stage;
  Record rec[kMaxRecords];
  unsigned long long red64[kWarps], red64b[kWarps];
  uint32_t red_max[kWarps];
  float red_f[kWarps];
};
// ... and those in which the tokens above a threshold are sought
struct __align__(16) Common : Meet {
  float cut, guess, floor_z;
  uint32_t mode;
  union {
    uint32_t bound[kMaxBounds];                     // keys of group maxima (rows with a count)
    __align__(16) float4 sample[kMaxRecords][2];    // sampled masses (rows without)
    unsigned long long few[kPairCap];               // the list's entries that matter (rank 0)
    unsigned long long top[kMaxRecords];            // the best token of each warp
  };
  Tally tally[kMaxCluster];
  unsigned long long best[kMaxCluster];
  unsigned long long sums[kMaxCluster];
  unsigned long long base;
  uint32_t bin;
  float best_x[kMaxCluster];           // the logits of best[]
  __align__(8) float2 mass[kMaxRecords];            // per warp: mass above the drawn token, mass at or above the cut
};
// ... with lists and histograms (the second histogram only where a cluster selects,
// which then has no use for a list)
struct Shared : Common {
  union {
    __align__(16) unsigned long long list[kListCap];     // entries as pack_best packs them: gathered (rank 0) or own
    __align__(16) unsigned long long hist1[kBins];       // odd selection levels of a cluster
  };
  union {
    __align__(16) unsigned long long hist0[kBins];       // the other selection levels
    __align__(16) unsigned long long stage[kStage];      // a block's entries on their way to rank 0
    struct {
      __align__(16) uint32_t keys[kPairCap];             // of the gathered entries
      uint32_t place[kPairCap];                          // entries above each
      unsigned long long masses[kPairCap];               // by place
    };
  };
};

// ---- block reductions that cost one barrier each --------------------------------------
// (the caller keeps a barrier between two uses of the same array)

template <typename T, typename Op>
__device__ __forceinline__ T block_fold(T v, Op op, T* red) {
  v = warp_reduce(v, op);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[threadIdx.x & (kWarps - 1)];  // kWarps is a power of two: a butterfly over as many lanes
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* red) { return block_fold(v, SumOp(), red); }
template <typename T>
__device__ __forceinline__ T block_max(T v, T* red) { return block_fold(v, MaxOp(), red); }
static_assert((kWarps & (kWarps - 1)) == 0 && kWarps <= 32, "the butterfly above");

// Inclusive sums over the block in thread order
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* red) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= uint32_t(o)) v += y;
  }
  if (lane == 31) red[warp] = v;
  __syncthreads();
  for (uint32_t i = 0; i < warp; ++i) v += red[i];
  return v;
}

// The block's barriers and counters; ends with a block barrier.
__device__ __forceinline__ void begin(Meet& s) {
  if (threadIdx.x < kBars) {
    mbar_init(&s.bar_rec + threadIdx.x, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x == 32) {  // not the warp that issues the copies: the fence would wait for them
    s.n_list = s.n_local = s.n_stage = s.late = 0;
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
  }
  __syncthreads();
}
// Tells the cluster that this block may be sent to; ready_others() waits until all
// blocks may.
__device__ __forceinline__ void may_send() { cluster_arrive_relaxed(); }
__device__ __forceinline__ void ready_others() { cluster_wait(); }

// scale of the exponent of exp((x - m) / T) as a power of two, finite for every T > 0
__device__ __forceinline__ float exp_scale(float T) { return fminf(__fdiv_rn(kLog2e, T), FLT_MAX); }

// ---- the row ----------------------------------------------------------------------------

// Where a row's groups lie.  Group g holds tokens g * E - a + (0 .. E-1).
template <bool BF16>
struct Row {
  using F = Fmt<BF16>;
  const char* base;      // the row's start rounded down to 16 bytes
  uint32_t a;            // elements between base and the row's start
  uint32_t V, W;
  const uint8_t* mask;   // the row's bitmask or null

  __device__ __forceinline__ Row(const void* logits, uint64_t ld, const uint32_t* bitmask, uint32_t W_, uint32_t V_,
                                 uint32_t b) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(logits) + size_t(b) * ld * F::kSize;
    base = reinterpret_cast<const char*>(p & ~uintptr_t(15));
    a = uint32_t(p & 15u) / F::kSize;
    V = V_;
    W = W_;
    mask = bitmask ? reinterpret_cast<const uint8_t*>(bitmask + size_t(b) * W_) : nullptr;
  }
  // Bit e: element e of group g is allowed by the bitmask.  t0 is the group's
  // first token; some token of the group is in the row.
  __device__ __forceinline__ uint32_t mask_bits(int t0) const {
    if (a == 0) return uint32_t(mask[t0 >> 3]) >> (BF16 ? 0 : t0 & 4);
    if (t0 < 0) return uint32_t(mask[0]) << -t0;
    const uint32_t sh = uint32_t(t0) & 7u;
    uint32_t w = mask[t0 >> 3];
    // the second byte exists: the last token of the group that is in the row lies in it or before
    if (sh + F::E > 8u && uint32_t(t0 | 7) + 1u < V) w |= uint32_t(mask[(t0 >> 3) + 1]) << 8;
    return w >> sh;
  }
  // whole groups, those that a bulk copy may bring: [first, end)
  __device__ __forceinline__ uint32_t first_whole() const { return a ? 1u : 0u; }
  __device__ __forceinline__ uint32_t end_whole() const { return (V + a) / F::E; }
  // a group that is not whole: element by element, -inf outside the row
  __device__ __forceinline__ uint4 edge(uint32_t g) const {
    const int t0 = int(g * F::E) - int(a);
    uint32_t w[4] = {F::kNegInf, F::kNegInf, F::kNegInf, F::kNegInf};
#pragma unroll
    for (uint32_t e = 0; e < F::E; ++e) {
      const int t = t0 + int(e);
      if (t < 0 || t >= int(V)) continue;
      const char* p = base + size_t(g) * 16 + e * F::kSize;
      if (BF16) {
        const uint32_t h = *reinterpret_cast<const volatile uint16_t*>(p);
        w[e >> 1] = (e & 1u) ? (w[e >> 1] & 0xFFFFu) | (h << 16) : (w[e >> 1] & 0xFFFF0000u) | h;
      } else {
        w[e] = *reinterpret_cast<const volatile uint32_t*>(p);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint4 masked(uint4 v, uint32_t bits) const {
    if (BF16) return apply_mask(v, pair_mask_of(bits & 0xFFu));
    if (!(bits & 1u)) v.x = F::kNegInf;
    if (!(bits & 2u)) v.y = F::kNegInf;
    if (!(bits & 4u)) v.z = F::kNegInf;
    if (!(bits & 8u)) v.w = F::kNegInf;
    return v;
  }
  __device__ __forceinline__ bool in_row(uint32_t g) const { return int(g * F::E) - int(a) < int(V); }
  // the logit of one token with every convention applied (a plain load)
  __device__ __forceinline__ float at(uint32_t t) const {
    if (mask && !((mask[t >> 3] >> (t & 7u)) & 1u)) return -INFINITY;
    return value(t);
  }
  // ... of any id, -inf where it is not in the row: the loads wait for no branch
  __device__ __forceinline__ float at_any(uint32_t t) const {
    const uint32_t at = t < V ? t : 0u, allowed = mask ? uint32_t(mask[at >> 3]) >> (at & 7u) : 1u;
    const float x = value(at);
    return t < V && (allowed & 1u) ? x : -INFINITY;
  }
  __device__ __forceinline__ float value(uint32_t t) const {
    const char* p = base + (size_t(t) + a) * F::kSize;
    const float x = BF16 ? bf16_bits_to_float(*reinterpret_cast<const volatile uint16_t*>(p))
                         : *reinterpret_cast<const volatile float*>(p);
    return x != x ? -INFINITY : fminf(x, BF16 ? kMaxBf16 : FLT_MAX);
  }
};

// f(token, logit) for every allowed token of the row, spread over one block,
// from memory: for rank 0 on its own, where a gathered list has overflowed
template <bool BF16, typename Fn>
__device__ __forceinline__ void each_of_row(const Row<BF16>& r, Fn f) {
#pragma unroll 1
  for (uint32_t t = threadIdx.x; t < r.V; t += kThreads) {
    const float x = r.at(t);
    if (x > -INFINITY) f(t, x);
  }
}

template <bool BF16>
__device__ __forceinline__ float elem(const uint4& v, uint32_t e) {
  if (BF16) return group_at(v, e);
  return __uint_as_float(e < 2 ? (e == 0 ? v.x : v.y) : (e == 2 ? v.z : v.w));
}
template <bool BF16>
__device__ __forceinline__ float2 pair(const uint4& v, uint32_t q) {  // elements 2q and 2q + 1
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (BF16) return make_float2(lo_f(w[q]), hi_f(w[q]));
  return make_float2(__uint_as_float(w[2 * q]), __uint_as_float(w[2 * q + 1]));
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// maximum of a group, a (positive) NaN when it holds one
template <bool BF16>
__device__ __forceinline__ float group_max_nan(const uint4& v) {
  if (BF16) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(w);
    const __nv_bfloat162 r = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&r);
    return max_nan(lo_f(u), hi_f(u));
  }
  return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                 max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
}
// maximum of kN groups, a (positive) NaN when one of them holds one
template <bool BF16, int kN>
__device__ __forceinline__ float groups_max_nan(const uint4* v) {
  if (BF16) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(v);
    __nv_bfloat162 r[4] = {h[0], h[1], h[2], h[3]};
#pragma unroll
    for (int i = 1; i < kN; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) r[q] = __hmax2_nan(r[q], h[4 * i + q]);
    r[0] = __hmax2_nan(__hmax2_nan(r[0], r[1]), __hmax2_nan(r[2], r[3]));
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&r[0]);
    return max_nan(lo_f(u), hi_f(u));
  }
  float t = group_max_nan<BF16>(v[0]);
#pragma unroll
  for (int i = 1; i < kN; ++i) t = max_nan(t, group_max_nan<BF16>(v[i]));
  return t;
}
// NaN -> -inf, +inf -> the largest finite value
template <bool BF16>
__device__ __forceinline__ uint32_t clean_word(uint32_t w) {
  if (!BF16) {
    const float x = __uint_as_float(w);
    return x != x ? 0xFF800000u : __float_as_uint(fminf(x, FLT_MAX));
  }
  uint32_t r = 0;
#pragma unroll
  for (uint32_t s = 0; s < 32; s += 16) {
    uint32_t h = (w >> s) & 0xFFFFu;
    if ((h & 0x7FFFu) > 0x7F80u) h = 0xFF80u;
    else if (h == 0x7F80u) h = 0x7F7Fu;
    r |= h << s;
  }
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint4 clean_group(uint4 v) {
  return make_uint4(clean_word<BF16>(v.x), clean_word<BF16>(v.y), clean_word<BF16>(v.z), clean_word<BF16>(v.w));
}

// bit e: element e >= cut (cut finite; for bf16 the least bf16 not below it in both halves of cut2)
template <bool BF16>
__device__ __forceinline__ uint32_t ge_bits(const uint4& v, float cut, uint32_t cut2) {
  if (BF16) return group_ge_bits(v, cut2);
  return (__uint_as_float(v.x) >= cut ? 1u : 0u) | (__uint_as_float(v.y) >= cut ? 2u : 0u) |
         (__uint_as_float(v.z) >= cut ? 4u : 0u) | (__uint_as_float(v.w) >= cut ? 8u : 0u);
}
__device__ __forceinline__ uint32_t bf16_pair_up(float cut) {
  const __nv_bfloat162 t = __bfloat162bfloat162(__float2bfloat16_ru(cut));
  return *reinterpret_cast<const uint32_t*>(&t);
}

// A key that at least k of s.bound[0 .. count) reach, by bisection, count <= 512.  For
// one warp.
__device__ __forceinline__ uint32_t bound_key(const Common& s, uint32_t count, uint32_t k) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t v[kMaxBounds / 32], lo = 0xFFFFFFFFu, hi = 0;
  const uint32_t each = (count + 31) / 32;
#pragma unroll
  for (uint32_t i = 0; i < kMaxBounds / 32; ++i) {
    v[i] = 0;
    if (i < each && i * 32 + lane < count) {
      v[i] = s.bound[i * 32 + lane];
      lo = min(lo, v[i]);
      hi = max(hi, v[i]);
    }
  }
  lo = __reduce_min_sync(0xFFFFFFFFu, lo);
  hi = __reduce_max_sync(0xFFFFFFFFu, hi) + 1u;  // fewer than k reach hi, all reach lo
#pragma unroll 1
  while (hi - lo > 0x10000u) {  // 1/128 of an octave; three pivots a round, counted in 10 bits each
    const uint32_t q = (hi - lo) / 4, p1 = lo + q, p2 = p1 + q, p3 = p2 + q;
    uint32_t reach = 0;
#pragma unroll
    for (uint32_t i = 0; i < kMaxBounds / 32; i += 4)
      if (i < each) {
#pragma unroll
        for (uint32_t w = 0; w < 4; ++w)
          reach += (v[i + w] >= p1 ? 1u : 0u) + (v[i + w] >= p2 ? 1u << 10 : 0u) + (v[i + w] >= p3 ? 1u << 20 : 0u);
      }
    reach = __reduce_add_sync(0xFFFFFFFFu, reach);
    if ((reach >> 20) >= k) lo = p3;
    else if (((reach >> 10) & 1023u) >= k) lo = p2, hi = p3;
    else if ((reach & 1023u) >= k) lo = p1, hi = p2;
    else hi = p1;
  }
  return lo;
}

// Takes kN groups whose maximum is t into a running maximum tm and the running sum
// acc.x + acc.y of exp2((x - tm) c), which is scaled on as the maximum rises
template <bool BF16, int kN>
__device__ __forceinline__ void add_groups(const uint4* v, float t, float c, float& tm, float2& acc) {
  if (t > tm) {
    const float f = ex2((tm - t) * c);  // 0 from the first -inf on
    acc = make_float2(acc.x * f, acc.y * f);
    tm = t;
  }
  if (!(tm > -INFINITY)) return;
  const float2 nm = make_float2(-tm, -tm), c2 = make_float2(c, c);
  float2 sum[2] = {};
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (uint32_t q = 0; q < Fmt<BF16>::E / 2; ++q)
      sum[q & 1u] = __fadd2_rn(sum[q & 1u], ex2_pair(__fmul2_rn(__fadd2_rn(pair<BF16>(v[i], q), nm), c2)));
  acc = __fadd2_rn(acc, __fadd2_rn(sum[0], sum[1]));
}

__device__ __forceinline__ unsigned long long record_bits(float m, float rest) {
  return (static_cast<unsigned long long>(__float_as_uint(rest)) << 32) | __float_as_uint(m);
}
// A lane's share of its warp's record: m the warp's maximum, who the lanes that have it.
// The shares of all lanes and the lanes of `who` but one make the rest.
__device__ __forceinline__ float share_of(float tm, float ts, float c, float& m, uint32_t& who) {
  m = fkey_inv(__reduce_max_sync(0xFFFFFFFFu, fkey(tm)));
  who = __ballot_sync(0xFFFFFFFFu, tm == m);
  if (!(tm > -INFINITY)) return 0.f;
  return tm == m ? ts - 1.f : ts * ex2((tm - m) * c);
}
__device__ __forceinline__ unsigned long long record_of(float share, float m, uint32_t who) {
  return record_bits(m, warp_reduce(share, SumOp()) + float(__popc(who) - 1));
}
// A warp's record from its lanes' maxima and sums
__device__ __forceinline__ unsigned long long warp_record(float tm, float ts, float c) {
  float m;
  uint32_t who;
  const float share = share_of(tm, ts, c, m, who);
  return record_of(share, m, who);
}

// The part of a row that a block holds
template <bool BF16>
struct Held {
  using F = Fmt<BF16>;
  Row<BF16> r;
  uint32_t n, rank;   // cluster size, this block
  uint32_t nv;        // groups of a thread
  uint4* part;        // group j of thread t at [j * kThreads + t]
  const uint8_t* bits;  // the part's mask, kMaskRun bytes a run, where it can be copied; else null
  float tm;           // this thread's maximum
  float ts;           // its sum of exp2((x - tm) c)

  static constexpr uint32_t kMaskRun = kThreads * F::E / 8;
  __device__ __forceinline__ Held(const Row<BF16>& row, uint32_t nv_, void* memory)
      : r(row), n(cluster_size()), rank(cluster_rank()), nv(nv_), part(static_cast<uint4*>(memory)) {
    // on the 16-byte grid, whole 16-byte pieces to a row, groups whole bytes or halves
    const bool copied = r.mask && r.a == 0 && ((reinterpret_cast<uintptr_t>(r.mask) | (r.W * 4u)) & 15u) == 0;
    bits = copied ? reinterpret_cast<const uint8_t*>(part + nv * kThreads) : nullptr;
  }
  // group j of this thread: consecutive threads hold consecutive groups, the
  // blocks take turns at runs of kThreads
  __device__ __forceinline__ uint32_t group(uint32_t j) const { return (j * n + rank) * kThreads + threadIdx.x; }
  __device__ __forceinline__ int first_token(uint32_t j) const { return int(group(j) * F::E) - int(r.a); }
  __device__ __forceinline__ uint4 at(uint32_t j) const { return part[j * kThreads + threadIdx.x]; }

  // Starts the copies, a lane a run of kThreads groups (kMaxGroups lanes, kChunk
  // neighbours a barrier); the groups that they do not bring are written by their
  // threads.  once: the row is not read or written again soon, so L2 need not keep it
  // (what else is read, the random numbers, then stays longer: 256 x 128256 rows
  // without a cut 53.6 -> 51.6 us; a gradient that is written meanwhile loses by it:
  // 222.5 -> 233.9 us of 2048 x 128256).
  __device__ __forceinline__ void start(Meet& s, bool once) const {
    const uint32_t lo = r.first_whole(), hi = r.end_whole();
    if (threadIdx.x < 32) {
      const uint32_t j = threadIdx.x, g0 = (j * n + rank) * kThreads, from = max(g0, lo), to = min(g0 + kThreads, hi);
      uint32_t bytes = j < nv && to > from ? (to - from) * 16u : 0u;
      void* to_part = part + j * kThreads + (from - g0);
      if (bytes && once)
        bulk_g2s_hint(to_part, r.base + size_t(from) * 16, bytes, s.bar_part + j / kChunk, evict_first_policy());
      else if (bytes)
        bulk_g2s(to_part, r.base + size_t(from) * 16, bytes, s.bar_part + j / kChunk);
      if (bits && j < nv) {
        const uint32_t off = (j * n + rank) * kMaskRun, end = r.W * 4u;
        const uint32_t k = off < end ? min(kMaskRun, end - off) : 0u;
        if (k) bulk_g2s(const_cast<uint8_t*>(bits) + j * kMaskRun, r.mask + off, k, s.bar_part + j / kChunk);
        bytes += k;
      }
      bytes += __shfl_xor_sync(0xFFFFFFFFu, bytes, 1);
      bytes += __shfl_xor_sync(0xFFFFFFFFu, bytes, 2);
      // what has arrived by now counts against this
      if (j % kChunk == 0 && j < nv) mbar_expect_tx(s.bar_part + j / kChunk, bytes);
    }
    // groups before lo or from hi on: at most one each side in the row
    const uint32_t run = group(0) - threadIdx.x;
    if (lo && run == 0 && threadIdx.x == 0) part[0] = r.edge(0);
    for (uint32_t j = nv; j-- > 0;) {
      const uint32_t g = group(j);
      if (g < hi) break;
      if (g >= lo) part[j * kThreads + threadIdx.x] = r.edge(g);
    }
  }
  // First pass, chunk by chunk as the copies land: applies the mask and the
  // replacements of NaN and +inf (writing back what they change), and finds this
  // thread's maximum and, with SUM, its sum of exp2((x - tm) c), scaled on as the
  // maximum rises.  False when a wait ran out.
  template <bool SUM>
  __device__ __forceinline__ bool take(Meet& s, float c) {
    bool ok = true;
    tm = -INFINITY;
    float2 acc = {};
#pragma unroll 1
    for (uint32_t j0 = 0; j0 < nv; j0 += kChunk) {
      uint32_t allowed[kChunk];
      if (r.mask && !bits) {
#pragma unroll
        for (uint32_t i = 0; i < kChunk; ++i)
          allowed[i] = j0 + i < nv && r.in_row(group(j0 + i)) ? r.mask_bits(first_token(j0 + i)) : 0u;
      }
      ok = mbar_wait(s.bar_part + j0 / kChunk, 0) && ok;
      uint4 v[kChunk];
#pragma unroll
      for (uint32_t i = 0; i < kChunk; ++i) {
        v[i] = make_uint4(F::kNegInf, F::kNegInf, F::kNegInf, F::kNegInf);
        if (j0 + i < nv) v[i] = at(j0 + i);
      }
      if (r.mask) {
        if (bits) {  // groups outside the row are -inf whatever their bits
          const uint8_t* p = bits + j0 * kMaskRun + (BF16 ? threadIdx.x : threadIdx.x / 2);
#pragma unroll
          for (uint32_t i = 0; i < kChunk; ++i)
            allowed[i] = j0 + i < nv ? uint32_t(p[i * kMaskRun]) >> (BF16 ? 0u : (threadIdx.x & 1u) * 4u) : 0u;
        }
#pragma unroll
        for (uint32_t i = 0; i < kChunk; ++i) {
          v[i] = r.masked(v[i], allowed[i]);
          if (j0 + i < nv) part[(j0 + i) * kThreads + threadIdx.x] = v[i];
        }
      }
      float t = groups_max_nan<BF16, kChunk>(v);
      if (fkey(t) >= kKeyInf) {
#pragma unroll
        for (uint32_t i = 0; i < kChunk; ++i) {
          v[i] = clean_group<BF16>(v[i]);
          if (j0 + i < nv) part[(j0 + i) * kThreads + threadIdx.x] = v[i];
        }
        t = groups_max_nan<BF16, kChunk>(v);
      }
      if (SUM) add_groups<BF16, kChunk>(v, t, c, tm, acc);
      else tm = fmaxf(tm, t);
    }
    ts = acc.x + acc.y;
    return ok;
  }
  // Tells every block of the cluster this warp's record, and, for a
  // bound on the k-th largest logit, the maxima of `per_warp` groups of its
  // lanes (a power of two, 0 for none), completing on bar_rec.  After
  // ready_others().
  __device__ __forceinline__ void publish(Meet& s, unsigned long long rec) const { publish_with(s, rec, 0u, nullptr); }
  __device__ __forceinline__ void publish(Common& s, unsigned long long rec, uint32_t per_warp) const {
    publish_with(s, rec, per_warp, s.bound);
  }
  __device__ __forceinline__ void publish_with(Meet& s, unsigned long long rec, uint32_t per_warp, uint32_t* bound) const {
    const uint32_t lane = threadIdx.x & 31, w = rank * kWarps + (threadIdx.x >> 5);
    if (threadIdx.x == 0) mbar_expect_tx(&s.bar_rec, n * kWarps * (8u + 4u * per_warp));
    if (lane < n) send(at_rank(&s.rec[w], lane), rec, at_rank(&s.bar_rec, lane));
    if (per_warp == 0) return;
    uint32_t key = fkey(tm);
    for (uint32_t o = 16; o >= per_warp; o >>= 1) key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, o));
    // every lane holds the maximum of the lanes equal to it modulo per_warp
    for (uint32_t i = lane; i < per_warp * n; i += 32)
      send(at_rank(&bound[w * per_warp + (i & (per_warp - 1))], i / per_warp), key,
           at_rank(&s.bar_rec, i / per_warp));
  }
  // This warp's record.  Where no share is large (the rest may be lost in the roundings of
  // 1 + rest) the sum of the lane with the maximum is added up again without it.
  __device__ __forceinline__ unsigned long long record(float c) const {
    float m;
    uint32_t who;
    float share = share_of(tm, ts, c, m, who);
    if (!__any_sync(0xFFFFFFFFu, share >= 0.25f) && __popc(who) == 1) share = again(share, __ffs(who) - 1, m, c);
    return record_of(share, m, who);
  }
  // The shares with the elements of lane `from` but one that is the maximum spread over
  // the warp, a word of the lane's groups each
  __device__ __forceinline__ float again(float share, uint32_t from, float m, float c) const {
    const uint32_t lane = threadIdx.x & 31, words = nv * 4;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(part + (threadIdx.x & ~31u) + from);
    if (lane == from) share = 0.f;
    bool left_out = false;
    __syncwarp();  // what the lane has written there
#pragma unroll 1
    for (uint32_t i0 = 0; i0 < words; i0 += 32) {
      const uint32_t i = i0 + lane, w = i < words ? p[(i >> 2) * (kThreads * 4) + (i & 3u)] : F::kNegInf;
      float2 x = BF16 ? make_float2(lo_f(w), hi_f(w)) : make_float2(__uint_as_float(w), -INFINITY);
      const uint32_t hits = __ballot_sync(0xFFFFFFFFu, x.x == m || x.y == m);
      if (hits && !left_out) {
        left_out = true;
        if (lane == __ffs(hits) - 1) (x.x == m ? x.x : x.y) = -INFINITY;
      }
      share += ex2((x.x - m) * c);
      if (BF16) share += ex2((x.y - m) * c);
    }
    return share;
  }
  // Tells rank 0 alone, and with BEST this warp's best token too
  template <bool BEST>
  __device__ __forceinline__ void report(Meet& s, unsigned long long rec, unsigned long long* top = nullptr) const {
    const uint32_t lane = threadIdx.x & 31, w = rank * kWarps + (threadIdx.x >> 5);
    if (rank == 0 && threadIdx.x == 0) mbar_expect_tx(&s.bar_rec, n * kWarps * (BEST ? 16u : 8u));
    if (BEST) {
      const float m = __uint_as_float(uint32_t(rec));
      uint32_t t = 0xFFFFFFFFu;
      if (tm == m && m > -INFINITY) {
#pragma unroll 1
        for (uint32_t j = 0; j < nv && t == 0xFFFFFFFFu; ++j) {  // tokens rise with j
          const uint32_t hits = ge_bits<BF16>(at(j), m, BF16 ? bf16_pair_up(m) : 0u);
          if (hits) t = uint32_t(first_token(j)) + __ffs(hits) - 1;
        }
      }
      t = __reduce_min_sync(0xFFFFFFFFu, t);
      if (lane == 0)
        send(at_rank(&top[w], 0), m > -INFINITY ? pack_best(m, t) : 0ull, at_rank(&s.bar_rec, 0));
    }
    if (lane == 0) send(at_rank(&s.rec[w], 0), rec, at_rank(&s.bar_rec, 0));
  }
  // f(token, logit) for every element of this thread's groups that is >= cut (finite)
  template <typename Fn>
  __device__ __forceinline__ void each(float cut, Fn f) const {
    if (!(tm >= cut)) return;
    const uint32_t cut2 = BF16 ? bf16_pair_up(cut) : 0u;
#pragma unroll 1
    for (uint32_t j = 0; j < nv; ++j) {
      const uint4 v = at(j);
      uint32_t hits = ge_bits<BF16>(v, cut, cut2);
      while (hits) {
        const uint32_t e = __ffs(hits) - 1;
        hits &= hits - 1;
        f(uint32_t(first_token(j)) + e, elem<BF16>(v, e));
      }
    }
  }
  // Appends (logit, token) of every element >= cut to a list of the block's own, in
  // any order; *count, zero before, goes on past the capacity, the entries do not.
  __device__ __forceinline__ void stage(float cut, unsigned long long* list, uint32_t cap, uint32_t* count) const {
    if (!(tm >= cut)) return;
    const uint32_t cut2 = BF16 ? bf16_pair_up(cut) : 0u;
#pragma unroll 1
    for (uint32_t j0 = 0; j0 < nv; j0 += kChunk) {
      uint32_t with = 0;  // groups of the chunk that hold some
#pragma unroll
      for (uint32_t i = 0; i < kChunk; ++i)
        if (j0 + i < nv && group_max_nan<BF16>(at(j0 + i)) >= cut) with |= 1u << i;
      while (with) {
        const uint32_t j = j0 + __ffs(with) - 1;
        with &= with - 1;
        const uint4 v = at(j);
        uint32_t hits = ge_bits<BF16>(v, cut, cut2);
        uint32_t place = atomicAdd(count, uint32_t(__popc(hits)));
        while (hits) {
          const uint32_t e = __ffs(hits) - 1;
          hits &= hits - 1;
          if (place < cap) list[place] = pack_best(elem<BF16>(v, e), uint32_t(first_token(j)) + e);
          ++place;
        }
      }
    }
  }
  // Sends (logit, token) of every element >= cut to rank 0's list, completing on
  // its bar_list, and then the block's count and (MASS) its elements' mass in units
  // of the maximum's to rank 0 or to every block (all), completing on bar_tally.
  // The list's count goes on past its capacity, the entries do not.  Their order is
  // arbitrary.  A block with more than kStage entries sends none.  The entries are
  // staged in the block's own memory: one warp sends them, with one reservation.
  template <bool MASS>
  __device__ __forceinline__ void gather(Shared& s, float cut, bool all, float M, float c) const {
    const uint32_t lane = threadIdx.x & 31;
    stage(cut, s.stage, kStage, &s.n_stage);
    __syncthreads();
    const uint32_t found = s.n_stage;
    const bool fits = found <= kStage;
    if (MASS && !fits) {
      const float mass = warp_reduce(masses_from(M, c, cut, cut).y, SumOp());
      if (lane == 0) s.red_f[threadIdx.x >> 5] = mass;
      __syncthreads();
    }
    if (threadIdx.x >= 32) return;
    float mass = 0.f;
    if (fits && found) {
      uint32_t place = 0;
      if (lane == 0) place = add_remote(at_rank(&s.n_list, 0), found);
      place = __shfl_sync(0xFFFFFFFFu, place, 0);
      const uint32_t list = at_rank(s.list, 0), bar = at_rank(&s.bar_list, 0);
      unsigned long long units = 0;  // in integers: the order is arbitrary
      for (uint32_t i = lane; i < found; i += 32) {
        const unsigned long long e = s.stage[i];
        if (place + i < kListCap) send(list + (place + i) * 8, e, bar);
        if (MASS) units += mass_q(fkey_inv(uint32_t(e >> 32)), M, c);
      }
      if (MASS) mass = float(warp_reduce(units, SumOp())) * (1.f / kMassOne);
    } else if (MASS && !fits) {
      for (uint32_t w = 0; w < kWarps; ++w) mass += s.red_f[w];
    }
    if (lane < (all ? n : 1u))
      send(at_rank(&s.tally[rank], lane),
           (static_cast<unsigned long long>(fits ? found : kTooMany) << 32) | __float_as_uint(mass),
           at_rank(&s.bar_tally, lane));
  }
  // this thread's sums of exp2((x - M) c) over its elements > x, and over those >= y
  __device__ __forceinline__ float2 masses_from(float M, float c, float x, float y) const {
    float2 above = {}, from = {};
    if (!(tm >= fminf(x, y))) return above;
    const float2 nm = make_float2(-M, -M), c2 = make_float2(c, c);
#pragma unroll 2
    for (uint32_t j = 0; j < nv; ++j) {
      const uint4 v = at(j);
#pragma unroll
      for (uint32_t q = 0; q < F::E / 2; ++q) {
        const float2 p = pair<BF16>(v, q);
        const float2 e = ex2_pair(__fmul2_rn(__fadd2_rn(p, nm), c2));
        above = __fadd2_rn(above, make_float2(p.x > x ? e.x : 0.f, p.y > x ? e.y : 0.f));
        from = __fadd2_rn(from, make_float2(p.x >= y ? e.x : 0.f, p.y >= y ? e.y : 0.f));
      }
    }
    return make_float2(above.x + above.y, from.x + from.y);
  }
  // stage() to this block's own list, between two barriers; whether it holds them all
  __device__ __forceinline__ bool compact(Shared& s, float cut) const {
    stage(cut, s.list, kListCap, &s.n_local);
    __syncthreads();
    return s.n_local <= kListCap;
  }
  // The gathered entries' count, whether every warp has sent its own, and the
  // mass, to every thread of a block that tallies go to; false to all of them when
  // a wait ran out.  The barrier's expectation is set here: early tallies wait in
  // its transaction count.
  __device__ __forceinline__ bool tallied(Shared& s, uint32_t& count, bool& whole, float& mass) const {
    if (threadIdx.x == 0) mbar_expect_tx(&s.bar_tally, n * uint32_t(sizeof(Tally)));
    const bool ok = __syncthreads_and(wait_sent(&s.bar_tally));
    mass = 0.f;
    count = 0;
    bool over = false;
    for (uint32_t i = 0; i < n; ++i) {
      mass += s.tally[i].mass;
      const uint32_t k = s.tally[i].count;
      over |= k == kTooMany;
      count += k == kTooMany ? 0u : k;
    }
    whole = !over;
    return ok;
  }
  // Rank 0, after tallied(): the list's entries are there; the same to every thread
  __device__ __forceinline__ bool listed(Shared& s, uint32_t count) const {
    if (threadIdx.x == 0) mbar_expect_tx(&s.bar_list, min(count, kListCap) * 8u);
    return __syncthreads_and(wait_sent(&s.bar_list));
  }
};

// The row's maximum, and the sum S = 1 + rest of exp2((x - M) c), from the warps'
// records, the same in every warp of the cluster (0 and 0 for an empty row).  For one
// warp of a block, after its wait.
__device__ __forceinline__ void merge(const Record* rec, uint32_t count, float c, float& M, float& S, float& rest) {
  constexpr uint32_t kEach = kMaxRecords / 32;
  Record r[kEach];
  uint32_t top = 0;
#pragma unroll
  for (uint32_t k = 0; k < kEach; ++k) {
    const uint32_t i = k * 32 + (threadIdx.x & 31);
    r[k].m = -INFINITY;
    r[k].rest = 0.f;
    if (i < count) r[k] = rec[i];
    top = max(top, fkey(r[k].m));
  }
  M = fkey_inv(__reduce_max_sync(0xFFFFFFFFu, top));
  float t = 0.f;
  uint32_t have = 0;  // records with the row's maximum: all but one of their 1s belong to the rest
#pragma unroll
  for (uint32_t k = 0; k < kEach; ++k) {
    const bool has = r[k].m == M;
    have += has ? 1u : 0u;
    t += has ? r[k].rest : (1.f + r[k].rest) * ex2((r[k].m - M) * c);
  }
  have = __reduce_add_sync(0xFFFFFFFFu, have);
  rest = warp_reduce(t, SumOp()) + float(have - 1);
  S = M > -INFINITY ? 1.f + rest : 0.f;
}

// Groups of lanes per warp whose maxima bound the k-th largest logit: the least power
// of two that gives the cluster a third more groups than k (with P groups of random
// logits about -P log(1 - k / P) tokens lie at or above the bound), else as many as
// there are when those are k at least (tight is false then), else 0.
__device__ __forceinline__ uint32_t bounds_per_warp(uint32_t k, uint32_t n, bool& tight) {
  const uint32_t warps = n * kWarps;
  uint32_t most = 0;
  tight = true;
  for (uint32_t g = 1; g <= 32u && warps * g <= kMaxBounds; g <<= 1) {
    if (4 * k <= 3 * warps * g) return g;
    most = g;
  }
  tight = false;
  return k <= warps * most ? most : 0u;
}

// Largest key k in [lo, hi] whose upper set {key >= k}, over the whole row,
// carries at least `target` of the weights that each(f) reports for this block's
// part through f(key, weight); lo when none does.  Radix selection: up to kBins
// equal bins of the key interval per level, the blocks' bins added up by every
// block, then the bin that the target falls into.  Integer weights: the result
// does not depend on the order of the atomics.  `above` receives the weight of
// the keys above the result's bin.  `level` counts the uses of the two
// histograms (start with 0, keep it).
template <typename Each>
__device__ uint32_t select_key(Shared& s, uint32_t n, Each each, uint32_t lo, uint32_t hi, unsigned long long target,
                               uint32_t& level, unsigned long long& above) {
  constexpr uint32_t kOwn = kBins / kThreads;
  static_assert(kOwn % 2 == 0, "two bins a load");
  const uint32_t tid = threadIdx.x;
  above = 0;
  for (;;) {
    const uint32_t range = hi - lo;
    const uint32_t shift = range < kBins ? 0u : 32u - kBinBits - __clz(range);
    // alone, the barriers of the scan separate a level's reads from the next
    // level's zeros; in a cluster the level two before, which used this histogram,
    // was read by every block before the cluster met in the level between
    unsigned long long* hist = n > 1 && (level & 1u) ? s.hist1 : s.hist0;
    ++level;
    for (uint32_t i = tid; i < kBins; i += kThreads) hist[i] = 0ull;
    if (tid == 0) s.bin = kBins;
    __syncthreads();
    each([&](uint32_t key, unsigned long long w) {
      if (key >= lo && key <= hi) atomicAdd(hist + ((hi - key) >> shift), w);
    });
    cluster_sync(n);
    // kOwn consecutive bins a thread
    unsigned long long own[kOwn] = {};
    for (uint32_t i = 0; i < n; ++i) {
      const uint32_t at = at_rank(hist + kOwn * tid, i);
#pragma unroll
      for (uint32_t q = 0; q < kOwn; q += 2) {
        unsigned long long x, y;
        ld_remote2(at + q * 8, x, y);
        own[q] += x;
        own[q + 1] += y;
      }
    }
    unsigned long long mine = 0;
#pragma unroll
    for (uint32_t q = 0; q < kOwn; ++q) mine += own[q];
    unsigned long long before = above + block_scan(mine, s.red64) - mine;
    if (before + mine >= target) {
      unsigned long long w = before;
      uint32_t q = 0;
#pragma unroll
      for (uint32_t i = 0; i + 1 < kOwn; ++i)
        if (q == i && w + own[i] < target) {
          w += own[i];
          ++q;
        }
      atomicMin(&s.bin, kOwn * tid + q);
    }
    __syncthreads();
    const uint32_t bin = s.bin;
    if (bin / kOwn == tid) {
      unsigned long long w = before;
#pragma unroll
      for (uint32_t i = 0; i + 1 < kOwn; ++i)
        if (i < bin % kOwn) w += own[i];
      s.base = w;
    }
    __syncthreads();
    if (bin == kBins) return lo;
    above = s.base;
    hi -= bin << shift;
    const uint32_t width = (1u << shift) - 1u;
    lo = hi - lo > width ? hi - width : lo;
    if (shift == 0) return hi;
    __syncthreads();  // s.bin is set again above
  }
}

// s.place[i] = the number of entries of list[0 .. c), c <= kPairCap, above entry i:
// by key alone, or by key and id.  The block's threads share the pairs out (parts
// of it compare with parts of the list).  Ends with a barrier.
template <bool IDS>
__device__ __forceinline__ void place_entries(Shared& s, const unsigned long long* list, uint32_t c) {
  uint32_t C = 32;
  while (C < c) C <<= 1;
  const uint32_t tid = threadIdx.x, i = tid & (C - 1), part = tid / C, parts = kThreads / C;
  if (!IDS) s.keys[tid] = tid < c ? uint32_t(list[tid] >> 32) : 0u;  // zeros are above nothing
  s.place[tid] = 0;
  __syncthreads();
  if (i < c) {
    uint32_t above = 0;
    if (IDS) {
      const unsigned long long e = list[i];
      for (uint32_t j = part; j < c; j += parts) above += list[j] > e;
    } else {
      const uint32_t key = s.keys[i];
#pragma unroll 4
      for (uint32_t j = 4 * part; j < c; j += 4 * parts) {
        const uint4 k = *reinterpret_cast<const uint4*>(s.keys + j);
        above += (k.x > key) + (k.y > key) + (k.z > key) + (k.w > key);
      }
    }
    if (above) atomicAdd(s.place + i, above);
  }
  __syncthreads();
}

// Copies the entries of s.list[0 .. c) whose key is at least `key` > 0 to s.few; returns
// their number (none are copied past kPairCap).  Ends with a barrier.
__device__ __forceinline__ uint32_t keep_few(Shared& s, uint32_t c, uint32_t key) {
  __syncthreads();
  if (threadIdx.x == 0) s.n_local = 0;
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < c; i += kThreads) {
    const unsigned long long e = s.list[i];
    if (uint32_t(e >> 32) < key) continue;
    const uint32_t at = atomicAdd(&s.n_local, 1u);
    if (at < kPairCap) s.few[at] = e;
  }
  __syncthreads();
  return s.n_local;
}
// A key that at least k of the entries of s.list[0 .. c), c <= kListCap, reach, and few
// more: by bisection, the block counting together.  1 when there are not more than k.
__device__ __forceinline__ uint32_t list_bound(Shared& s, uint32_t c, uint32_t k) {
  constexpr uint32_t kOwn = kListCap / kThreads;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (c <= k) return 1u;
  uint32_t v[kOwn], lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll
  for (uint32_t i = 0; i < kOwn; ++i) {
    const uint32_t at = i * kThreads + tid;
    v[i] = at < c ? uint32_t(s.list[at] >> 32) : 0u;
    if (at < c) {
      lo = min(lo, v[i]);
      hi = max(hi, v[i]);
    }
  }
  lo = ~block_max(~lo, s.red_max);
  __syncthreads();
  hi = block_max(hi, s.red_max) + 1u;
  for (uint32_t round = 0; hi - lo > 0x4000u; ++round) {  // three pivots and a barrier a round: two sets of counters
    const uint32_t q = (hi - lo) / 4, p1 = lo + q, p2 = p1 + q, p3 = p2 + q;
    uint32_t reach = 0;
#pragma unroll
    for (uint32_t i = 0; i < kOwn; ++i)
      reach += (v[i] >= p1 ? 1u : 0u) + (v[i] >= p2 ? 1u << 10 : 0u) + (v[i] >= p3 ? 1u << 20 : 0u);
    reach = __reduce_add_sync(0xFFFFFFFFu, reach);
    uint32_t* sum = reinterpret_cast<uint32_t*>(round & 1u ? s.red64 : s.red64b);
    if (lane == 0) sum[warp] = reach;
    __syncthreads();
    uint32_t r1 = 0, r2 = 0, r3 = 0;
#pragma unroll
    for (uint32_t w = 0; w < kWarps; ++w) {
      const uint32_t t = sum[w];
      r1 += t & 1023u;
      r2 += (t >> 10) & 1023u;
      r3 += t >> 20;
    }
    uint32_t got;
    if (r3 >= k) lo = p3, got = r3;
    else if (r2 >= k) lo = p2, hi = p3, got = r2;
    else if (r1 >= k) lo = p1, hi = p2, got = r1;
    else hi = p1, got = 0;
    if (got == k) break;
  }
  return lo;
}

// Descending sort of list[0 .. n) (bitonic network over the next power of two,
// padded with zeros, which sort last).  list: kListCap words of shared memory.
__device__ inline void sort_desc(unsigned long long* list, uint32_t n) {
  uint32_t N = 2;
  while (N < n) N <<= 1;
  for (uint32_t i = n + threadIdx.x; i < N; i += kThreads) list[i] = 0ull;
  __syncthreads();
  for (uint32_t k = 2; k <= N; k <<= 1)
    for (uint32_t j = k >> 1; j > 0; j >>= 1) {
      for (uint32_t i = threadIdx.x; i < N / 2; i += kThreads) {
        const uint32_t a = 2 * i - (i & (j - 1)), b = a + j;
        const unsigned long long x = list[a], y = list[b];
        if ((x < y) == ((a & k) == 0)) {
          list[a] = y;
          list[b] = x;
        }
      }
      __syncthreads();
    }
}

// ---- launching -----------------------------------------------------------------------

// Shared memory of a block's part: its groups and, with a bitmask, their bits
inline size_t part_bytes(bool bf16, uint32_t nv, bool mask) {
  return size_t(nv) * kThreads * 16 + (mask ? size_t(nv) * kThreads / (bf16 ? 1 : 2) : 0);
}

// The cluster size of a launch and the groups of a thread.  Few rows take the widest
// cluster whose blocks are all resident together, so that a row is split over more
// SMs; many rows take parts of `full` groups a thread.
struct Plan {
  uint32_t nv, n;
};
// Blocks up to which a row is split further, over 2, 4, 8 or 16 blocks (clusters of
// other sizes take longer to meet): two an SM, for 16 blocks one an SM and three
// groups a thread at least.  Microseconds, top-k 50 with top-p, then top-p alone:
//   64 x 32000    by blocks at one, two, four an SM   10.5   9.5  14.2
//   1 x 32000     8 blocks 7.5 and 8.9, 12 7.7 and 9.3, 16 8.1 and 9.5
//   1 x 128256    8 blocks 8.4 and 10.1, 12 8.6 and 10.3, 16 7.8 and 9.7
//   12 x 128256   8 blocks 9.0 and 12.3, 16 9.0 and 13.8
//   32 x 128256   8 blocks 11.2 and 16.0, 9 11.7 and 17.2
constexpr uint32_t kSlots = 2 * 152;
// A row always fits kMaxGroups: a context takes vocabularies whose bitmask its mask
// kernels hold in 48 KB, fewer than 393216 tokens.
static_assert(kMaxCluster * kMaxGroups * kThreads * 4 >= 393216 + 8, "rows of floats");
inline Plan plan_row(bool bf16, uint32_t V, uint32_t B, bool aligned, uint32_t full) {
  const uint32_t E = bf16 ? 8 : 4;
  const uint32_t runs = ((V + (aligned ? 0 : E - 1) + E - 1) / E + kThreads - 1) / kThreads;  // of kThreads groups
  uint32_t n = (runs + full - 1) / full;
  if (n > kMaxCluster) n = kMaxCluster;
  for (uint32_t k = 2; k <= kMaxCluster; k *= 2) {
    const bool wide = k == kMaxCluster;
    if (k > n && k <= runs && uint64_t(B) * k <= (wide ? kSlots / 2 : kSlots) && (!wide || runs >= 3 * k)) n = k;
  }
  return {(runs + n - 1) / n, n};
}

// A launch of clusters of n blocks
struct ClusterLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2] = {};
  ClusterLaunch(uint32_t clusters, uint32_t n, uint32_t threads, size_t smem, cudaStream_t stream) {
    cfg.gridDim = dim3(clusters * n);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = n;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
};
// The kernel's shared memory and cluster size limits are raised on its first launch on
// a device.
constexpr int kMaxSmem = 227 * 1024;
template <auto Kernel>
cudaError_t raise_limits(int device) {
  static DeviceAnswers raised;
  cudaError_t e = cudaSuccess;
  raised.get(device, [&] {
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e == cudaSuccess ? 1 : 0;
  });
  return e;
}
template <auto Kernel, typename... Args>
cudaError_t launch_clusters(int device, uint32_t clusters, uint32_t n, uint32_t threads, size_t smem,
                            cudaStream_t stream, Args&&... args) {
  const cudaError_t e = raise_limits<Kernel>(device);
  if (e != cudaSuccess) return e;
  ClusterLaunch l(clusters, n, threads, smem, stream);
  return cudaLaunchKernelEx(&l.cfg, Kernel, std::forward<Args>(args)...);
}

}  // namespace row

// Host checks shared by the per-row entry points: an aligned pointer of the
// logits' dtype, a row stride of at least V.
inline bool row_args_ok(const cg_ctx* c, const void* logits, int dtype, uint32_t B, uint32_t V, uint64_t ld,
                        const uint32_t* bitmask) {
  if (!c || (dtype != CG_F32 && dtype != CG_BF16)) return false;
  if (V != ctx_view(c).t.V || ld < V || ld > (uint64_t(1) << 40)) return false;
  if (B > 0x07FFFFFFu || (B && !logits)) return false;  // the grid: up to 16 blocks a row
  const uintptr_t size = dtype == CG_BF16 ? 2 : 4;
  return reinterpret_cast<uintptr_t>(logits) % size == 0 && reinterpret_cast<uintptr_t>(bitmask) % 4 == 0;
}
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool rows_on_grid(const void* logits, int dtype, uint64_t ld) {
  return ((reinterpret_cast<uintptr_t>(logits) | (ld * (dtype == CG_BF16 ? 2 : 4))) & 15u) == 0;
}

}  // namespace cgk
