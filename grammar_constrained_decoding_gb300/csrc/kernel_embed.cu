// The embedding lookup with a scale, and its gradient over sorted tokens (cg_embed,
// cg_embed_grad).
//
//   out_i = scale * table[t_i],   grad_v = scale * sum over {i : t_i = v} of g_i
//
// Both move rows: memory bounds them.  The lookup is one launch of row copies.  The
// gradient first sorts the positions by token (stable, so that a token's rows are summed
// in the order of their positions and no result depends on the order of the blocks), then
// sums runs of equal tokens: chunks of positions side by side, runs that cross a chunk's
// border joined afterwards in the chunks' order.  Sums are held in 32 bits and rounded once.
#include <algorithm>

#include "logit_row.cuh"
#include "matrix_args.h"

namespace cgk {
namespace {

using namespace row;

constexpr uint32_t kEmbedSms = 152;

// ---- rows in vectors of BYTES bytes: the widest that every row's start and width allow ----
template <int BYTES> struct VecOf;
template <> struct VecOf<16> { using type = uint4; };
template <> struct VecOf<8> { using type = uint2; };
template <> struct VecOf<4> { using type = uint32_t; };
template <> struct VecOf<2> { using type = uint16_t; };

// a vector's elements as floats and back
template <bool BF16, int BYTES>
struct Elems {
  static constexpr int kN = BYTES / (BF16 ? 2 : 4);
  using Vec = typename VecOf<BYTES>::type;
  static __device__ __forceinline__ void get(const Vec& v, float (&x)[kN]) {
    if (BF16) {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(&v);
#pragma unroll
      for (int i = 0; i < kN; ++i) x[i] = __uint_as_float(uint32_t(h[i]) << 16);
    } else {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
      for (int i = 0; i < kN; ++i) x[i] = __uint_as_float(w[i]);
    }
  }
  static __device__ __forceinline__ Vec put(const float (&x)[kN]) {
    Vec v;
    if (BF16) {
      __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(&v);
#pragma unroll
      for (int i = 0; i < kN; ++i) h[i] = __float2bfloat16_rn(x[i]);
    } else {
      float* w = reinterpret_cast<float*>(&v);
#pragma unroll
      for (int i = 0; i < kN; ++i) w[i] = x[i];
    }
    return v;
  }
};

// ---- the lookup ----------------------------------------------------------------------------

constexpr uint32_t kLookThreads = 256;
constexpr uint32_t look_each(int bytes) { return bytes == 16 ? 4 : 8; }

// Vectors are numbered through all rows; a block takes 1024 (2048 narrow ones) that follow
// one another, all of a thread's loads under way together
template <bool BF16, int BYTES>
__global__ void __launch_bounds__(kLookThreads) look_kernel(const char* table, uint64_t pitch, const uint32_t* tokens,
                                                            uint32_t N, uint32_t V, uint32_t vecs, float scale, char* out,
                                                            uint64_t pitch_out, uint32_t* status) {
  using E = Elems<BF16, BYTES>;
  using Vec = typename E::Vec;
  constexpr uint32_t kLookEach = look_each(BYTES);
  griddep_launch_dependents();
  griddep_wait();
  const uint64_t base = uint64_t(blockIdx.x) * (kLookThreads * kLookEach);
  const uint32_t row0 = uint32_t(base / vecs), off = uint32_t(base - uint64_t(row0) * vecs);
  Vec v[kLookEach];
  uint32_t row[kLookEach], col[kLookEach];
#pragma unroll
  for (uint32_t k = 0; k < kLookEach; ++k) {
    const uint32_t at = off + k * kLookThreads + threadIdx.x;
    row[k] = row0 + at / vecs;
    col[k] = at % vecs;
    v[k] = Vec{};
    if (row[k] >= N) continue;
    const uint32_t t = tokens[row[k]];
    if (t < V) v[k] = *reinterpret_cast<const Vec*>(table + t * pitch + uint64_t(col[k]) * BYTES);
    else if (t != CG_NO_TOKEN && col[k] == 0) record_error(status, CG_DEV_BAD_TOKEN);
  }
#pragma unroll
  for (uint32_t k = 0; k < kLookEach; ++k) {
    if (row[k] >= N) continue;
    if (scale != 1.f) {
      float x[E::kN];
      E::get(v[k], x);
#pragma unroll
      for (int i = 0; i < E::kN; ++i) x[i] = tokens[row[k]] < V ? x[i] * scale : 0.f;
      v[k] = E::put(x);
    }
    *reinterpret_cast<Vec*>(out + row[k] * pitch_out + uint64_t(col[k]) * BYTES) = v[k];
  }
}

// ---- sorting the positions by token ----------------------------------------------------------

constexpr uint32_t kSortThreads = 1024, kSortWarps = 32, kSortBits = 9, kBins = 1u << kSortBits;
constexpr uint32_t kSortMost = 16;  // blocks of the cluster
constexpr uint32_t kSortKeep = 4;   // tiles whose keys a thread keeps between counting and moving

struct SortArgs {
  const uint32_t* tokens;
  uint32_t N, V, passes;
  uint32_t* key[2];        // tokens in the order so far (V for a row without one)
  uint32_t* pos[2];        // and their positions; the sorted ones are in key[0], pos[0]
  uint32_t* runs;          // the count of the runs to be joined, set to none
  uint32_t* status;
};
struct SortShared {
  uint32_t count[kBins];                    // this block's digits, read by the others
  uint32_t base[kBins];                     // where the next position of a digit goes
  uint32_t tile_base[kBins];                // ... as a tile begins
  uint32_t warp_sum[kSortWarps];
  alignas(16) uint16_t mine[kSortWarps][kBins];         // a tile's digits by warp, then where the warp's begin
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, uint32_t i, bool report) {
  const uint32_t t = a.tokens[i];
  if (t >= a.V && t != CG_NO_TOKEN && report) record_error(a.status, CG_DEV_BAD_TOKEN);
  return t < a.V ? t : a.V;
}
__device__ __forceinline__ uint32_t read_count(const uint32_t* count, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(count)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ void clear_tile(SortShared& s) {
  uint4* zero = reinterpret_cast<uint4*>(s.mine);
#pragma unroll
  for (uint32_t i = 0; i < sizeof(s.mine) / 16 / kSortThreads; ++i) zero[i * kSortThreads + threadIdx.x] = uint4{};
}

// A radix sort by one cluster, 9 bits a pass: each block counts the digits of its own
// stretch of positions, learns from the others where its digits begin, and moves its
// positions there tile by tile, in their order.
__device__ void sort_tokens(const SortArgs& a, SortShared& s) {
  const uint32_t n = cluster_size(), rank = cluster_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (rank == 0 && tid == 0) *a.runs = 0;
  const uint32_t each = (((a.N + n - 1) / n) + kSortThreads - 1) / kSortThreads * kSortThreads;
  const uint32_t from = min(a.N, rank * each), to = min(a.N, from + each);
  for (uint32_t pass = 0; pass < a.passes; ++pass) {
    const uint32_t shift = pass * kSortBits;
    const bool odd = (a.passes - pass) & 1u;   // the last pass writes key[0]
    const uint32_t* const key_in = odd ? a.key[1] : a.key[0];
    const uint32_t* const pos_in = odd ? a.pos[1] : a.pos[0];
    uint32_t* const key_out = odd ? a.key[0] : a.key[1];
    uint32_t* const pos_out = odd ? a.pos[0] : a.pos[1];
    uint32_t kept[kSortKeep], kept_pos[kSortKeep];
#pragma unroll
    for (uint32_t q = 0; q < kSortKeep; ++q) {
      const uint32_t i = from + q * kSortThreads + tid;
      kept[q] = 0;
      kept_pos[q] = i;
      if (i < to) {
        kept[q] = pass == 0 ? sort_key(a, i, true) : __ldcg(key_in + i);
        if (pass) kept_pos[q] = __ldcg(pos_in + i);
      }
    }
    if (tid < kBins) s.count[tid] = 0;
    clear_tile(s);
    __syncthreads();
#pragma unroll
    for (uint32_t q = 0; q < kSortKeep; ++q)
      if (from + q * kSortThreads + tid < to) atomicAdd(&s.count[(kept[q] >> shift) & (kBins - 1)], 1u);
    for (uint32_t i = from + kSortKeep * kSortThreads + tid; i < to; i += kSortThreads) {
      const uint32_t k = pass == 0 ? sort_key(a, i, true) : __ldcg(key_in + i);
      atomicAdd(&s.count[(k >> shift) & (kBins - 1)], 1u);
    }
    cluster_sync(n);
    // where this block's positions of digit d begin: all smaller digits, and d's in the blocks before
    uint32_t all = 0, before = 0;
    if (tid < kBins) {
#pragma unroll
      for (uint32_t r = 0; r < kSortMost; ++r) {
        const uint32_t x = r >= n ? 0u : n == 1 ? s.count[tid] : read_count(&s.count[tid], r);
        all += x;
        if (r < rank) before += x;
      }
    }
    uint32_t up = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, up, o);
      if (lane >= uint32_t(o)) up += x;
    }
    if (lane == 31) s.warp_sum[warp] = up;
    __syncthreads();
    if (tid < kBins) {
      const uint32_t w = lane < warp ? s.warp_sum[lane] : 0u;   // at most 16 warps of bins
      s.base[tid] = __reduce_add_sync(0xFFFFFFFFu, w) + up - all + before;
    }
#pragma unroll 1
    for (uint32_t tile = from, q = 0; tile < to; tile += kSortThreads, ++q) {
      const uint32_t i = tile + tid;
      const bool there = i < to;
      uint32_t k = kept[0], p = kept_pos[0];
#pragma unroll
      for (uint32_t u = 1; u < kSortKeep; ++u)
        if (q == u) k = kept[u], p = kept_pos[u];
      if (q >= kSortKeep && there) {
        k = pass == 0 ? sort_key(a, i, false) : __ldcg(key_in + i);
        p = pass ? __ldcg(pos_in + i) : i;
      }
      const uint32_t digit = there ? (k >> shift) & (kBins - 1) : kBins + lane;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, digit);
      const uint32_t nth = __popc(same & ((1u << lane) - 1u));
      if (q) {
        clear_tile(s);
        __syncthreads();
      }
      if (there && nth == 0) s.mine[warp][digit] = uint16_t(__popc(same));
      __syncthreads();
      if (tid < kBins) {
        uint32_t at = 0, x[kSortWarps];
#pragma unroll
        for (uint32_t w = 0; w < kSortWarps; ++w) x[w] = s.mine[w][tid];
#pragma unroll
        for (uint32_t w = 0; w < kSortWarps; ++w) {
          s.mine[w][tid] = uint16_t(at);
          at += x[w];
        }
        s.tile_base[tid] = s.base[tid];
        s.base[tid] += at;
      }
      __syncthreads();
      if (there) {
        const uint32_t to_at = s.tile_base[digit] + s.mine[warp][digit] + nth;
        if (to_at < a.N) {   // always, unless the tokens were written meanwhile
          __stcg(key_out + to_at, k);
          __stcg(pos_out + to_at, p);
        }
      }
      __syncthreads();
    }
    __threadfence();
    cluster_sync(n);
  }
}

constexpr uint32_t kZeroBytes = 32768;   // of zeros in shared memory, copied out again and again

__device__ __forceinline__ void bulk_s2g(void* to, const void* from, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(smem_addr(from)), "r"(bytes)
               : "memory");
}

// Zeros over the gradient by `blocks` blocks: rows without gaps by bulk copies of 32 KB from
// shared memory, other rows a warp each in 16-byte stores; what lies off the 16-byte grid at
// either end element by element.
template <uint32_t SIZE>
__device__ __forceinline__ void zero_edge(char* from, uint32_t bytes, uint32_t lane) {   // fewer than 16
  if (lane * SIZE < bytes) *reinterpret_cast<typename VecOf<SIZE>::type*>(from + lane * SIZE) = 0;
}
template <uint32_t SIZE>
__device__ void write_zeros(char* out, uint64_t pitch, uint32_t rows, uint64_t width, uint32_t block, uint32_t blocks,
                            unsigned char* smem) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (pitch == width) {
    for (uint32_t i = threadIdx.x; i < kZeroBytes / 16; i += kSortThreads) reinterpret_cast<uint4*>(smem)[i] = uint4{};
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    const uint64_t all = uint64_t(rows) * pitch, lead = min(all, uint64_t(-reinterpret_cast<uintptr_t>(out) & 15u));
    const uint64_t body = (all - lead) & ~uint64_t(15);
    if (threadIdx.x == 0) {
      for (uint64_t at = uint64_t(block) * kZeroBytes; at < body; at += uint64_t(blocks) * kZeroBytes)
        bulk_s2g(out + lead + at, smem, uint32_t(min(uint64_t(kZeroBytes), body - at)));
      asm volatile("cp.async.bulk.commit_group;\n cp.async.bulk.wait_group 0;" ::: "memory");
    }
    if (block == 0 && warp == 1) {
      zero_edge<SIZE>(out, uint32_t(lead), lane);
      zero_edge<SIZE>(out + lead + body, uint32_t(all - lead - body), lane);
    }
    return;
  }
  for (uint64_t row = uint64_t(block) * kSortWarps + warp; row < rows; row += uint64_t(blocks) * kSortWarps) {
    char* at = out + row * pitch;
    const uint64_t lead = min(width, uint64_t(-reinterpret_cast<uintptr_t>(at) & 15u)), body = (width - lead) & ~uint64_t(15);
    zero_edge<SIZE>(at, uint32_t(lead), lane);
#pragma unroll 4
    for (uint64_t i = lane * 16; i < body; i += 512) *reinterpret_cast<uint4*>(at + lead + i) = uint4{};
    zero_edge<SIZE>(at + lead + body, uint32_t(width - lead - body), lane);
  }
}

// The first cluster sorts; the others meanwhile write zeros over the gradient (all of it: rows
// of tokens that occur are written again afterwards, at most one a position)
template <uint32_t SIZE>
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const SortArgs a, char* out, uint64_t pitch, uint64_t width) {
  extern __shared__ __align__(128) unsigned char smem[];
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t n = cluster_size();
  if (blockIdx.x < n) sort_tokens(a, *reinterpret_cast<SortShared*>(smem));
  else if (out) write_zeros<SIZE>(out, pitch, a.V, width, blockIdx.x - n, gridDim.x - n, smem);
}
constexpr size_t kSortSmem = sizeof(SortShared) > kZeroBytes ? sizeof(SortShared) : kZeroBytes;

// ---- summing runs ------------------------------------------------------------------------------

constexpr uint32_t kSumThreads = 128, kMostChunk = 32, kMostShort = 2 * kMostChunk;

struct SumArgs {
  const uint32_t* key;     // sorted tokens, V at the end for rows without one
  const uint32_t* pos;
  uint32_t N, V, chunk, vecs, slabs;
  const char* grad;
  uint64_t pitch;
  float scale;
  bool add;
  char* out;
  uint64_t pitch_out;
  float* part;             // [chunks][2][ld_part]: what a chunk has of the run that began before it, and of the one that goes on
  uint32_t ld_part;
  uint32_t* runs;          // how many runs are to be joined, and the chunks they begin in (in any order)
};

template <bool BF16, int BYTES>
__device__ __forceinline__ void write_sum(const SumArgs& a, uint32_t token, uint32_t col,
                                          float (&x)[Elems<BF16, BYTES>::kN]) {
  using E = Elems<BF16, BYTES>;
  using Vec = typename E::Vec;
  Vec* at = reinterpret_cast<Vec*>(a.out + token * a.pitch_out + uint64_t(col) * BYTES);
  float old[E::kN] = {};
  if (a.add) E::get(*at, old);
#pragma unroll
  for (int i = 0; i < E::kN; ++i) x[i] = a.add ? old[i] + a.scale * x[i] : a.scale * x[i];
  *at = E::put(x);
}

// How many keys right before, or from, `at` on equal the token: up to 64
__device__ __forceinline__ uint32_t equal_before(const uint32_t* at, uint32_t token, uint32_t lane) {
  const uint32_t a = __ballot_sync(0xFFFFFFFFu, *(at - 1 - int(lane)) == token);
  if (a != 0xFFFFFFFFu) return __ffs(~a) - 1;
  const uint32_t b = __ballot_sync(0xFFFFFFFFu, *(at - 33 - int(lane)) == token);
  return 32 + (b != 0xFFFFFFFFu ? __ffs(~b) - 1 : 32);
}
__device__ __forceinline__ uint32_t equal_after(const uint32_t* at, uint32_t token, uint32_t lane) {
  const uint32_t a = __ballot_sync(0xFFFFFFFFu, at[lane] == token);
  if (a != 0xFFFFFFFFu) return __ffs(~a) - 1;
  const uint32_t b = __ballot_sync(0xFFFFFFFFu, at[32 + lane] == token);
  return 32 + (b != 0xFFFFFFFFu ? __ffs(~b) - 1 : 32);
}

// A block takes a chunk of the sorted positions and a slab of the columns: kCols vectors of a
// row to a thread, 128 vectors apart (two in rows of more than 128 narrow vectors)
template <bool BF16, int BYTES, uint32_t kCols>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const SumArgs a) {
  using E = Elems<BF16, BYTES>;
  using Vec = typename E::Vec;
  constexpr uint32_t kAhead = 8, kWindow = kMostChunk + 2 * kMostShort;
  __shared__ uint32_t key[kWindow];
  __shared__ uint64_t row[kMostChunk + kMostShort];   // where the positions' rows begin
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t chunk = blockIdx.x / a.slabs, lane = threadIdx.x & 31;
  const uint32_t col0 = (blockIdx.x - chunk * a.slabs) * kSumThreads * kCols + threadIdx.x;
  const uint32_t from = chunk * a.chunk, n = min(a.chunk, a.N - from);
  // key[i]: of position from + i - kMostShort; past either end a value that no token has
  for (uint32_t i = threadIdx.x; i < n + 2 * kMostShort; i += kSumThreads) {
    const uint32_t at = from + i - kMostShort;
    key[i] = from + i < kMostShort || at >= a.N ? CG_NO_TOKEN : a.key[at];
  }
  for (uint32_t i = threadIdx.x; i < n + kMostShort; i += kSumThreads) row[i] = from + i < a.N ? min(a.pos[from + i], a.N - 1) * a.pitch : 0u;
  __syncthreads();
  // a run of up to two chunks is summed by the chunk it begins in: [begin, end) of the positions
  // from `from` on
  const uint32_t* const k0 = key + kMostShort;
  const uint32_t most = 2 * a.chunk;
  const uint32_t head = k0[0], tail = k0[n - 1];
  const uint32_t before = equal_before(k0, head, lane), after = equal_after(k0 + n, tail, lane);
  uint32_t begin = 0, end = n;
  bool head_part = false, tail_part = false;   // longer ones in parts
  if (before) {
    const uint32_t here = equal_after(k0, head, lane);   // up to 64: enough to tell
    head_part = before + here > most;
    if (!head_part) begin = min(here, n);
  }
  if (after && begin < n) {
    const uint32_t here = min(equal_before(k0 + n, tail, lane), n);
    const bool whole = here == n && head == tail;           // the chunk is one run
    if (!(whole && before)) {
      tail_part = here + after > most;
      if (!tail_part) end = n + after;
    }
  }
  // a longer run is for the join: it begins here
  if (tail_part && tail < a.V && threadIdx.x == 0 && blockIdx.x == chunk * a.slabs) a.runs[1 + atomicAdd(a.runs, 1u)] = chunk;
  if (col0 >= a.vecs) return;
  // rows without a token come last
  while (end > begin && k0[end - 1] >= a.V) --end;
  const char* in = a.grad + uint64_t(col0) * BYTES;
  float acc[kCols][E::kN] = {};
  bool first = head_part;   // the run at hand began before the chunk
  for (uint32_t i0 = begin; i0 < end; i0 += kAhead) {
    Vec v[kAhead][kCols];
#pragma unroll
    for (uint32_t u = 0; u < kAhead; ++u)
#pragma unroll
      for (uint32_t q = 0; q < kCols; ++q)
        if (i0 + u < end && (q == 0 || col0 + q * kSumThreads < a.vecs))
          v[u][q] = *reinterpret_cast<const Vec*>(in + row[i0 + u] + q * (kSumThreads * BYTES));
#pragma unroll
    for (uint32_t u = 0; u < kAhead; ++u) {
      const uint32_t i = i0 + u;
      if (i >= end) break;
      const uint32_t token = k0[i];
#pragma unroll
      for (uint32_t q = 0; q < kCols; ++q) {
        float x[E::kN];
        E::get(v[u][q], x);
#pragma unroll
        for (int e = 0; e < E::kN; ++e) acc[q][e] += x[e];
      }
      if (i + 1 < end && k0[i + 1] == token) continue;
      const bool part = first || (tail_part && i + 1 == n);
#pragma unroll
      for (uint32_t q = 0; q < kCols; ++q) {
        const uint32_t col = col0 + q * kSumThreads;
        if (col < a.vecs && token < a.V) {   // the token is, unless the tokens were written meanwhile
          if (!part) {
            write_sum<BF16, BYTES>(a, token, col, acc[q]);
          } else {
            float* to = a.part + (size_t(chunk) * 2 + (first ? 0 : 1)) * a.ld_part + col * E::kN;
#pragma unroll
            for (int e = 0; e < E::kN; ++e) to[e] = acc[q][e];
          }
        }
#pragma unroll
        for (int e = 0; e < E::kN; ++e) acc[q][e] = 0.f;
      }
      first = false;
    }
  }
}

constexpr uint32_t kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinColumns = 128;

// A block takes 128 columns of a run in turn: the warps take the chunks' sums in turn, and the
// warps' sums are added in their order
template <bool BF16>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const SumArgs a, uint32_t D) {
  __shared__ float4 mine[kJoinWarps][32];
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, across = (D + kJoinColumns - 1) / kJoinColumns;
  const uint32_t items = a.runs[0] * across;
  for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
    const uint32_t run = item / across, base = (item - run * across) * kJoinColumns, chunk = a.runs[1 + run];
    const uint32_t token = a.key[(chunk + 1) * a.chunk];   // it goes on into the next chunk
    // the run's last chunk: the one after which the next does not begin with the token
    uint32_t last = chunk + 1;
    for (;;) {
      const uint64_t at = (uint64_t(last) + 1 + lane) * a.chunk;
      const uint32_t same = __ballot_sync(0xFFFFFFFFu, at < a.N && a.key[min(at, uint64_t(a.N - 1))] == token);
      last += __ffs(~same) ? __ffs(~same) - 1 : 32;
      if (same != 0xFFFFFFFFu) break;
    }
    const uint32_t col = base + 4 * lane;   // a part's rows are padded to whole groups of 4
    float4 s = {};
    if (col < D)
#pragma unroll 8
      for (uint32_t j = chunk + warp; j <= last; j += kJoinWarps) {
        const float4 x = *reinterpret_cast<const float4*>(a.part + (size_t(j) * 2 + (j == chunk ? 1 : 0)) * a.ld_part + col);
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
      }
    mine[warp][lane] = s;
    __syncthreads();
    if (threadIdx.x < kJoinColumns && base + threadIdx.x < D) {
      float x = 0.f;
#pragma unroll
      for (uint32_t w = 0; w < kJoinWarps; ++w) x += reinterpret_cast<const float*>(mine[w])[threadIdx.x];
      x *= a.scale;
      char* at = a.out + token * a.pitch_out + uint64_t(base + threadIdx.x) * (BF16 ? 2 : 4);
      if (BF16) {
        __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(at);
        *o = __float2bfloat16_rn(a.add ? __bfloat162float(*o) + x : x);
      } else {
        float* o = reinterpret_cast<float*>(at);
        *o = a.add ? *o + x : x;
      }
    }
    __syncthreads();
  }
}

// ---- host ----------------------------------------------------------------------------------------

// the widest vector that two matrices' rows allow
int vector_bytes(const void* x, uint64_t pitch_x, const void* y, uint64_t pitch_y, uint64_t width) {
  const uint64_t all = reinterpret_cast<uintptr_t>(x) | pitch_x | reinterpret_cast<uintptr_t>(y) | pitch_y | width;
  return all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : 2;
}

struct GradPlan {
  uint32_t chunk, chunks, ld_part;
  size_t at_key[2], at_pos[2], at_part, at_runs, bytes;
};
// Chunks of 32 positions, fewer where that leaves SMs without work.  Every width gets the same
// chunks whatever its alignment, so that results do not depend on it.
GradPlan plan_grad(uint32_t N, uint32_t D, int dtype) {
  GradPlan p = {};
  const uint32_t slabs = tiles_of(uint64_t(D) * dtype_size(dtype), kSumThreads * 16);
  p.chunk = kMostChunk;
  while (p.chunk > 4 && uint64_t(tiles_of(N, p.chunk)) * slabs < 4 * kEmbedSms) p.chunk /= 2;
  p.chunks = tiles_of(N, p.chunk);
  p.ld_part = uint32_t(up_to(D, 4));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up_to(bytes, 256);
    return here;
  };
  for (int i = 0; i < 2; ++i) {
    p.at_key[i] = take(size_t(N) * 4);
    p.at_pos[i] = take(size_t(N) * 4);
  }
  p.at_part = take(size_t(p.chunks) * 2 * p.ld_part * 4);
  p.at_runs = take((size_t(p.chunks) + 1) * 4);
  p.bytes = at;
  return p;
}

template <bool BF16, int BYTES>
cudaError_t launch_look(const void* table, uint64_t pitch, const uint32_t* tokens, uint32_t N, uint32_t V, uint32_t D,
                        float scale, void* out, uint64_t pitch_out, uint32_t* status, cudaStream_t stream) {
  const uint32_t vecs = uint32_t(uint64_t(D) * (BF16 ? 2 : 4) / BYTES);
  const uint32_t blocks = tiles_of(uint64_t(N) * vecs, kLookThreads * look_each(BYTES));
  return launch_dependent(look_kernel<BF16, BYTES>, dim3(blocks), dim3(kLookThreads), 0, stream,
                          static_cast<const char*>(table), pitch, tokens, N, V, vecs, scale, static_cast<char*>(out),
                          pitch_out, status);
}

template <bool BF16, int BYTES>
cudaError_t launch_grad(int device, const SortArgs& sort, SumArgs sum, uint32_t chunks, uint32_t D, cudaStream_t stream) {
  sum.vecs = uint32_t(uint64_t(D) * (BF16 ? 2 : 4) / BYTES);
  // (4-byte vectors of 20000 x 1001 floats: one a thread 55.1 us, two 49.7, four 53.3)
  constexpr uint32_t kMany = BYTES == 16 ? 1 : 2;
  const uint32_t cols = sum.vecs > kSumThreads ? kMany : 1;
  sum.slabs = tiles_of(sum.vecs, kSumThreads * cols);
  uint32_t n = 1;
  while (n < kSortMost && sort.N > n * kSortThreads) n *= 2;
  // without zeros to write the sorting cluster is alone
  const uint32_t clusters = sum.add ? 1 : kEmbedSms / n;
  cudaError_t e = launch_clusters<sort_kernel<BF16 ? 2 : 4>>(device, clusters, n, kSortThreads, kSortSmem, stream, sort,
                                                            sum.add ? static_cast<char*>(nullptr) : sum.out, sum.pitch_out,
                                                            uint64_t(D) * (BF16 ? 2 : 4));
  if (e != cudaSuccess) return e;
  e = launch_dependent(cols == 1 ? sum_kernel<BF16, BYTES, 1> : sum_kernel<BF16, BYTES, kMany>, dim3(chunks * sum.slabs), dim3(kSumThreads), 0, stream, sum);
  if (e != cudaSuccess || chunks < 2) return e;
  return launch_dependent(join_kernel<BF16>, dim3(std::min(chunks * tiles_of(D, kJoinColumns), 4 * kEmbedSms)),
                          dim3(kJoinThreads), 0, stream, sum, D);
}

template <typename F>
cudaError_t by_vector(int dtype, int bytes, const F& f) {
  if (dtype == CG_BF16)
    switch (bytes) {
      case 16: return f.template operator()<true, 16>();
      case 8: return f.template operator()<true, 8>();
      case 4: return f.template operator()<true, 4>();
      default: return f.template operator()<true, 2>();
    }
  switch (bytes) {
    case 16: return f.template operator()<false, 16>();
    case 8: return f.template operator()<false, 8>();
    default: return f.template operator()<false, 4>();
  }
}
struct Look {
  const void* table;
  uint64_t pitch;
  const uint32_t* tokens;
  uint32_t N, V, D;
  float scale;
  void* out;
  uint64_t pitch_out;
  uint32_t* status;
  cudaStream_t stream;
  template <bool BF16, int BYTES>
  cudaError_t operator()() const {
    return launch_look<BF16, BYTES>(table, pitch, tokens, N, V, D, scale, out, pitch_out, status, stream);
  }
};
struct Grad {
  int device;
  SortArgs sort;
  SumArgs sum;
  uint32_t chunks, D;
  cudaStream_t stream;
  template <bool BF16, int BYTES>
  cudaError_t operator()() const {
    return launch_grad<BF16, BYTES>(device, sort, sum, chunks, D, stream);
  }
};

int embed_args(const cg_ctx* c, int dtype, uint32_t N, uint32_t V, uint32_t D, const uint32_t* tokens, float scale) {
  if (!c || (dtype != CG_F32 && dtype != CG_BF16) || V != ctx_view(c).t.V || D == 0) return CG_E_ARG;
  if ((N && !tokens) || !aligned4(tokens) || !(fabsf(scale) <= FLT_MAX)) return CG_E_ARG;
  return N > kMaxMatrixRows || D > kMaxMatrixWidth ? CG_E_LIMIT : CG_OK;
}

}  // namespace
}  // namespace cgk

extern "C" int cg_embed(cg_ctx* c, const void* d_table, int dtype, uint32_t V, uint32_t D, uint64_t ld_table,
                        const uint32_t* d_tokens, uint32_t N, float scale, void* d_out, uint64_t ld_out) {
  using namespace cgk;
  const int rc = embed_args(c, dtype, N, V, D, d_tokens, scale);
  if (rc != CG_OK) return rc;
  if (!matrix_ok(d_table, dtype, V, D, ld_table) || !matrix_ok(d_out, dtype, N, D, ld_out)) return CG_E_ARG;
  const uint64_t size = dtype_size(dtype);
  if (matrices_meet(d_out, N, ld_out, d_table, V, ld_table, D, size)) return CG_E_ARG;
  if (N == 0) return CG_OK;
  DeviceGuard dg(ctx_device(c), "cg_embed");
  if (!dg.ok) return CG_E_CUDA;
  const CtxView v = ctx_view(c);
  const Look f{d_table, ld_table * size, d_tokens, N, V, D, scale, d_out, ld_out * size, v.t.status, v.stream};
  return by_vector(dtype, vector_bytes(d_table, ld_table * size, d_out, ld_out * size, D * size), f) == cudaSuccess
             ? CG_OK
             : CG_E_CUDA;
}

extern "C" int cg_embed_workspace(const cg_ctx* c, int dtype, uint32_t N, uint32_t D, size_t* bytes) {
  using namespace cgk;
  if (!c || !bytes || (dtype != CG_F32 && dtype != CG_BF16) || D == 0) return CG_E_ARG;
  if (N > kMaxMatrixRows || D > kMaxMatrixWidth) return CG_E_LIMIT;
  *bytes = N == 0 ? 0 : plan_grad(N, D, dtype).bytes;
  return CG_OK;
}

extern "C" int cg_embed_grad(cg_ctx* c, const void* d_grad, int dtype, uint32_t N, uint32_t V, uint32_t D, uint64_t ld_grad,
                             const uint32_t* d_tokens, float scale, int accumulate, void* d_out_grad, uint64_t ld_out,
                             void* d_workspace, size_t workspace_bytes) {
  using namespace cgk;
  const int rc = embed_args(c, dtype, N, V, D, d_tokens, scale);
  if (rc != CG_OK) return rc;
  if (!matrix_ok(d_grad, dtype, N, D, ld_grad) || !matrix_ok(d_out_grad, dtype, V, D, ld_out)) return CG_E_ARG;
  const uint64_t size = dtype_size(dtype);
  if (matrices_meet(d_out_grad, V, ld_out, d_grad, N, ld_grad, D, size)) return CG_E_ARG;
  const GradPlan p = plan_grad(std::max(N, 1u), D, dtype);
  if (N && (!d_workspace || reinterpret_cast<uintptr_t>(d_workspace) % 256)) return CG_E_ARG;
  if (N && workspace_bytes < p.bytes) return CG_E_NOMEM;
  DeviceGuard dg(ctx_device(c), "cg_embed_grad");
  if (!dg.ok) return CG_E_CUDA;
  const CtxView v = ctx_view(c);
  if (N == 0)  // no rows: zeros, or what is there
    return accumulate || cudaMemset2DAsync(d_out_grad, ld_out * size, 0, D * size, V, v.stream) == cudaSuccess ? CG_OK
                                                                                                                : CG_E_CUDA;
  unsigned char* ws = static_cast<unsigned char*>(d_workspace);
  SortArgs sort = {};
  sort.tokens = d_tokens;
  sort.N = N;
  sort.V = V;
  sort.passes = (32 - uint32_t(__builtin_clz(V)) + kSortBits - 1) / kSortBits;
  for (int i = 0; i < 2; ++i) {
    sort.key[i] = reinterpret_cast<uint32_t*>(ws + p.at_key[i]);
    sort.pos[i] = reinterpret_cast<uint32_t*>(ws + p.at_pos[i]);
  }
  sort.status = v.t.status;
  SumArgs sum = {};
  sum.key = sort.key[0];
  sum.pos = sort.pos[0];
  sum.N = N;
  sum.V = V;
  sum.chunk = p.chunk;
  sum.grad = static_cast<const char*>(d_grad);
  sum.pitch = ld_grad * size;
  sum.scale = scale;
  sum.add = accumulate != 0;
  sum.out = static_cast<char*>(d_out_grad);
  sum.pitch_out = ld_out * size;
  sum.part = reinterpret_cast<float*>(ws + p.at_part);
  sum.ld_part = p.ld_part;
  sum.runs = sort.runs = reinterpret_cast<uint32_t*>(ws + p.at_runs);
  const Grad f{ctx_device(c), sort, sum, p.chunks, D, v.stream};
  return by_vector(dtype, vector_bytes(d_grad, ld_grad * size, d_out_grad, ld_out * size, D * size), f) == cudaSuccess
             ? CG_OK
             : CG_E_CUDA;
}
