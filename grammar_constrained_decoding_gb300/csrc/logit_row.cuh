// A row of logits as the per-row operators see it (sample_rows, top_logprobs,
// distill): a logit that is -inf or NaN, or whose bitmask bit is clear, is not
// allowed and reads as -inf; +inf reads as the largest finite value.
#pragma once

#include <cfloat>

#include "bf16_ops.cuh"

namespace cgk {
namespace row {

constexpr uint32_t kThreads = 512;
constexpr uint32_t kBins = 1024;       // bins of one selection level
constexpr uint32_t kSortCap = 2048;    // entries of the sorted list
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMaxBf16 = 3.38953138925e38f;  // largest finite bf16

template <bool BF16>
struct Row {
  const void* x;         // the row's first logit
  const uint32_t* mask;  // its bitmask or null
  uint32_t V;
  __device__ __forceinline__ bool bit(uint32_t t) const { return !mask || ((mask[t >> 5] >> (t & 31)) & 1u); }
  __device__ __forceinline__ float value(uint32_t t) const {
    const float v = BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(x)[t]) : static_cast<const float*>(x)[t];
    return v != v ? -INFINITY : fminf(v, BF16 ? kMaxBf16 : FLT_MAX);
  }
  __device__ __forceinline__ float at(uint32_t t) const { return bit(t) ? value(t) : -INFINITY; }
  // f(token, logit) for every allowed token, spread over the block
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (uint32_t t = threadIdx.x; t < V; t += blockDim.x) {
      const float v = at(t);
      if (v > -INFINITY) f(t, v);
    }
  }
};

// scale of the exponent of exp((x - m) / T) as a power of two, finite for every T > 0
__device__ __forceinline__ float exp_scale(float T) { return fminf(__fdiv_rn(kLog2e, T), FLT_MAX); }

// m = max and s = sum exp2((x - m) c) over the row, to every thread
template <bool BF16>
__device__ void max_and_sum(const Row<BF16>& r, float c, float& m, float& s) {
  __shared__ float red[33];
  float a = -INFINITY;
  r.each([&](uint32_t, float x) { a = fmaxf(a, x); });
  m = block_reduce(a, MaxOp(), -INFINITY, red);
  const float mm = m;
  float b = 0.f;
  r.each([&](uint32_t, float x) { b += ex2((x - mm) * c); });
  s = block_reduce(b, SumOp(), 0.f, red);
}

// Largest key k in [lo, hi] whose upper set {key >= k} carries at least
// `target` of the weights that each(f) reports through f(key, weight); lo when
// none does.  Radix selection: up to 1024 equal bins of the key interval per
// level, then the bin that the target falls into.  Integer weights: the result
// does not depend on the order of the atomics.  hist: kBins words of shared
// memory.  All threads take part and get the result.
template <typename Each>
__device__ uint32_t select_key(Each each, uint32_t lo, uint32_t hi, unsigned long long target,
                               unsigned long long* hist) {
  __shared__ unsigned long long s_part[33];
  __shared__ uint32_t s_bin;
  __shared__ unsigned long long s_base;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned long long base = 0;  // weight above hi
  for (;;) {
    const uint32_t range = hi - lo;
    const uint32_t shift = range < kBins ? 0u : 22u - __clz(range);
    __syncthreads();
    for (uint32_t i = tid; i < kBins; i += kThreads) hist[i] = 0ull;
    if (tid == 0) s_bin = kBins;
    __syncthreads();
    each([&](uint32_t key, unsigned long long w) {
      if (key >= lo && key <= hi) atomicAdd(hist + ((hi - key) >> shift), w);
    });
    __syncthreads();
    // two bins a thread, bins in order
    const unsigned long long h0 = hist[2 * tid], h1 = hist[2 * tid + 1];
    unsigned long long inc = h0 + h1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= uint32_t(o)) inc += y;
    }
    if (lane == 31) s_part[warp] = inc;
    __syncthreads();
    unsigned long long before = base;
    for (uint32_t i = 0; i < warp; ++i) before += s_part[i];
    before += inc - h0 - h1;
    if (before + h0 + h1 >= target) atomicMin(&s_bin, before + h0 >= target ? 2 * tid : 2 * tid + 1);
    __syncthreads();
    const uint32_t bin = s_bin;
    if (bin == kBins) return lo;
    if (bin >> 1 == tid) s_base = before + ((bin & 1u) ? h0 : 0ull);
    __syncthreads();
    base = s_base;
    hi -= bin << shift;
    const uint32_t width = (1u << shift) - 1u;
    lo = hi - lo > width ? hi - width : lo;
    if (shift == 0) return hi;
  }
}

// Descending sort of list[0 .. n) (bitonic network over the next power of two,
// padded with zeros, which sort last).  list: kSortCap words of shared memory.
__device__ inline void sort_desc(unsigned long long* list, uint32_t n) {
  uint32_t N = 2;
  while (N < n) N <<= 1;
  for (uint32_t i = n + threadIdx.x; i < N; i += blockDim.x) list[i] = 0ull;
  __syncthreads();
  for (uint32_t k = 2; k <= N; k <<= 1)
    for (uint32_t j = k >> 1; j > 0; j >>= 1) {
      for (uint32_t i = threadIdx.x; i < N / 2; i += blockDim.x) {
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

}  // namespace row

// Host checks shared by the per-row entry points: an aligned pointer of the
// logits' dtype, a row stride of at least V.
inline bool row_args_ok(const cg_ctx* c, const void* logits, int dtype, uint32_t B, uint32_t V, uint64_t ld,
                        const uint32_t* bitmask) {
  if (!c || (dtype != CG_F32 && dtype != CG_BF16)) return false;
  if (V != ctx_view(c).t.V || ld < V || ld > (uint64_t(1) << 40)) return false;
  if (B > 0x07FFFFFFu || (B && !logits)) return false;  // the grid: a few blocks a row
  const uintptr_t size = dtype == CG_BF16 ? 2 : 4;
  return reinterpret_cast<uintptr_t>(logits) % size == 0 && reinterpret_cast<uintptr_t>(bitmask) % 4 == 0;
}
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace cgk
