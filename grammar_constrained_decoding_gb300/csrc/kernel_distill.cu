// Distillation from a teacher's top logits, forward and backward
// (cg_distill_loss, cg_distill_grad).
//
//   loss = T^2 sum_k q_k (log q_k - log p[id_k]),  log p_v = (x_v - m) / T - log S,
//   dloss/dx_v = T (p_v - sum_{k: id_k = v} q_k),
// q the softmax of the teacher's listed logits / T, S = sum exp((x - m) / T).
//
// A cluster takes rows in turn, its blocks the row's chunks in turn, through a ring of
// chunks in shared memory that one warp of each block keeps filling across the rows'
// ends (bulk copies).  Eight warps take the chunks; the rest read the rows' lists
// meanwhile.  The logits are read from memory once and the gradient is written once.
// Short rows and small batches with a gradient are held instead (logit_row.cuh).
#include <algorithm>

#include "logit_row.cuh"

namespace cgk {
namespace {

using namespace row;

struct DistillArgs {
  const void* logits;
  uint64_t ld;
  const uint32_t* bitmask;
  uint32_t V, W;
  const uint32_t* ids;
  const float* teacher;
  uint32_t K;
  float temp;
  const float* lse_in;   // backward alone: the kept normaliser, one value a row
  const float* norm_in;  // ... or two, which is exact for every row; else null
  float* loss;
  float* lse_out;
  float* norm_out;
  const float* up;
  void* grad;
  uint64_t ld_grad;
  uint32_t* status;
};

// the teacher's logit by the rows' conventions
__device__ __forceinline__ float teacher_logit(float t) { return t != t ? -INFINITY : fminf(t, FLT_MAX); }
// q (log q - log p) of one listed token: dt, dx its logits below the teacher's and the
// row's maximum, ts the teacher's sum
__device__ __forceinline__ float loss_term(float dt, float ts, float log_ts, float dx, float log_s, float c, float T) {
  const float q = __fdiv_rn(ex2(dt * c), ts);
  return q > 0.f ? q * ((__fdiv_rn(dt, T) - log_ts) - (__fdiv_rn(dx, T) - log_s)) : 0.f;
}
__device__ __forceinline__ void store_loss(const DistillArgs& a, uint32_t b, float loss, float M, float S, float log_s) {
  a.loss[b] = loss;
  if (a.norm_out) {
    a.norm_out[2 * size_t(b)] = M;
    a.norm_out[2 * size_t(b) + 1] = S;
  }
  if (a.lse_out) a.lse_out[b] = M > -INFINITY ? __fdiv_rn(M, a.temp) + log_s : -INFINITY;
}
// The kept normaliser, p = exp2((x - M) c) / S.  From the one value M = lse T and S = 1: its
// rounding is an error of |lse| 2^-23 in every p, and where it overflows p is lost.
__device__ __forceinline__ void kept_norm(const DistillArgs& a, uint32_t b, float& M, float& S) {
  M = a.norm_in ? a.norm_in[2 * size_t(b)] : a.lse_in[b] * a.temp;
  S = a.norm_in ? a.norm_in[2 * size_t(b) + 1] : 1.f;
}

template <bool BF16>
__device__ __forceinline__ void store_grad(char* row, uint32_t t, float g) {
  if (BF16) reinterpret_cast<__nv_bfloat16*>(row)[t] = __float2bfloat16_rn(g);
  else reinterpret_cast<float*>(row)[t] = g;
}
__device__ __forceinline__ uint32_t bf16_pack(float2 g) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(g.x, g.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// one group's gradients: 16 bytes at once inside the row when the gradient's
// rows lie on the 16-byte grid like the logits', else one by one
template <bool BF16>
__device__ __forceinline__ void store_group(char* row, int t0, uint32_t V, bool wide, const float2* g) {
  constexpr uint32_t E = Fmt<BF16>::E;
  if (wide && t0 >= 0 && uint32_t(t0) + E <= V) {
    uint4 v;
    if (BF16) v = make_uint4(bf16_pack(g[0]), bf16_pack(g[1]), bf16_pack(g[2]), bf16_pack(g[3]));
    else v = make_uint4(__float_as_uint(g[0].x), __float_as_uint(g[0].y), __float_as_uint(g[1].x),
                        __float_as_uint(g[1].y));
    *reinterpret_cast<uint4*>(row + ptrdiff_t(t0) * ptrdiff_t(Fmt<BF16>::kSize)) = v;
    return;
  }
#pragma unroll
  for (uint32_t e = 0; e < E; ++e) {
    const int t = t0 + int(e);
    if (t >= 0 && t < int(V)) store_grad<BF16>(row, uint32_t(t), (e & 1u) ? g[e / 2].y : g[e / 2].x);
  }
}

// ---- the teacher's list -------------------------------------------------------------------

// in shared memory, K entries
struct List {
  uint32_t* id;     // listed ids that count, CG_NO_TOKEN for the others
  float* t;         // teacher logits
  float* x;         // the student's logits there
  __device__ List(void* at, uint32_t K)
      : id(static_cast<uint32_t*>(at)), t(reinterpret_cast<float*>(id + K)), x(t + K) {}
  // A thread reads its entries of row b: k, k + step and so on; the largest teacher's
  // logit that counts, else -inf.  Several at a time where there are more, so that their
  // loads are under way together.
  template <bool BF16>
  __device__ __forceinline__ float read(const DistillArgs& a, const Row<BF16>& r, uint32_t b, uint32_t k, uint32_t step,
                                        bool report) const {
    return a.K <= step ? read_by<BF16, 1>(a, r, b, k, step, report) : read_by<BF16, 4>(a, r, b, k, step, report);
  }
  template <bool BF16, uint32_t kBatch>
  __device__ __forceinline__ float read_by(const DistillArgs& a, const Row<BF16>& r, uint32_t b, uint32_t k,
                                           uint32_t step, bool report) const {
    float top = -INFINITY;
#pragma unroll 1
    for (; k < a.K; k += kBatch * step) {
      uint32_t i[kBatch];
      float tk[kBatch], xk[kBatch];
#pragma unroll
      for (uint32_t u = 0; u < kBatch; ++u) {
        const bool in = k + u * step < a.K;
        i[u] = in ? a.ids[size_t(b) * a.K + k + u * step] : CG_NO_TOKEN;
        tk[u] = in ? a.teacher[size_t(b) * a.K + k + u * step] : -INFINITY;
      }
#pragma unroll
      for (uint32_t u = 0; u < kBatch; ++u) xk[u] = r.at_any(i[u]);
#pragma unroll
      for (uint32_t u = 0; u < kBatch; ++u) {
        if (k + u * step >= a.K) break;
        if (i[u] >= a.V && i[u] != CG_NO_TOKEN && report) record_error(a.status, CG_DEV_BAD_TOKEN);
        tk[u] = teacher_logit(tk[u]);
        const bool counts = xk[u] > -INFINITY && tk[u] > -INFINITY;
        id[k + u * step] = counts ? i[u] : CG_NO_TOKEN;
        x[k + u * step] = xk[u];
        t[k + u * step] = tk[u];
        if (counts) top = fmaxf(top, tk[u]);
      }
    }
    return top;
  }
  // Writes the gradient of entry k's token: tm, ts the list's maximum and sum, M and S
  // the row's
  template <bool BF16>
  __device__ __forceinline__ void write(char* to, uint32_t k, uint32_t K, bool repeated, float tm, float ts, float M,
                                        float S, float c, float scale) const {
    float q = ex2((t[k] - tm) * c);
    if (repeated) {  // every entry of the id writes the same sum (K^2 steps: 1024 of 1024 x 128256 1611 us, without 245)
      q = 0.f;
      for (uint32_t j = 0; j < K; ++j)
        if (id[j] == id[k]) q += ex2((t[j] - tm) * c);
    }
    store_grad<BF16>(to, id[k], scale * (__fdiv_rn(ex2((x[k] - M) * c), S) - __fdiv_rn(q, ts)));
  }
};
// Repeated ids: every id claims a slot of the hash (more slots than ids, all CG_NO_TOKEN
// at first); the second of equal ones finds it taken by itself
__host__ __device__ inline uint32_t hash_slots(uint32_t K) {
  uint32_t s = 4;
  while (s < 2 * K) s <<= 1;
  return s;
}
__device__ __forceinline__ bool claimed_before(uint32_t* hash, uint32_t slots, uint32_t id) {
  for (uint32_t at = (id * 0x9E3779B1u) & (slots - 1);; at = (at + 1) & (slots - 1)) {
    const uint32_t old = atomicCAS(hash + at, CG_NO_TOKEN, id);
    if (old == CG_NO_TOKEN) return false;
    if (old == id) return true;
  }
}

// ---- the ring of chunks -------------------------------------------------------------------
//
// Chunk g of a row: WARPS * 32 * PER groups from group g on, group k * WARPS * 32 + t of
// them thread t's.  A block's chunks of all its rows follow one another through the
// slots; full: the chunk has landed, empty: every warp has taken it.

constexpr uint32_t kTakers = 8;  // warps that take chunks
template <bool BF16, uint32_t PER>
struct Ring {
  using F = Fmt<BF16>;
  static constexpr uint32_t kGroups = kTakers * 32 * PER, kBytes = kGroups * 16, kBits = kGroups * F::E / 8;
  uint64_t *full, *empty;
  unsigned char *data, *bits;  // the chunks, and their part of the bitmask
  uint32_t slots;
  uint32_t slot = 0, turn = 0;
  __device__ __forceinline__ Ring(uint64_t* f, uint64_t* e, unsigned char* memory, uint32_t count)
      : full(f), empty(e), data(memory), bits(memory + count * kBytes), slots(count) {}
  static size_t bytes(uint32_t count, bool mask) { return size_t(count) * (kBytes + (mask ? kBits : 0)); }
  __device__ __forceinline__ void init() const {
    for (uint32_t i = 0; i < slots; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, kTakers);
    }
  }
  __device__ __forceinline__ void next() {
    if (++slot == slots) slot = 0, ++turn;
  }
  // the chunks' bits come by copies too: on the 16-byte grid, groups whole bytes or halves
  static __device__ __forceinline__ bool copies_bits(const Row<BF16>& r) {
    return r.mask && r.a == 0 && ((reinterpret_cast<uintptr_t>(r.mask) | (r.W * 4u)) & 15u) == 0;
  }
  static __device__ __forceinline__ uint32_t end(const Row<BF16>& r) { return (r.V + r.a + F::E - 1) / F::E; }
  // One thread: this block's chunks of row r (of rank's, every n-th).  once: as Held::start.
  __device__ __forceinline__ bool fill(const Row<BF16>& r, uint32_t n, uint32_t rank, bool once) {
    const uint32_t lo = r.first_whole(), hi = r.end_whole();
    const bool with_bits = copies_bits(r);
    for (uint32_t g = rank * kGroups; g < end(r); g += n * kGroups, next()) {
      if (turn) {
        if (!mbar_wait(empty + slot, (turn - 1) & 1u)) return false;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the takers' reads come before the copy
      }
      const uint32_t from = max(g, lo), to = min(g + kGroups, hi), off = g * F::E / 8;
      const uint32_t size = to > from ? (to - from) * 16u : 0u, more = with_bits ? min(kBits, r.W * 4u - off) : 0u;
      mbar_expect_tx(full + slot, size + more);
      unsigned char* at = data + slot * kBytes + (from - g) * 16;
      if (size && once) bulk_g2s_hint(at, r.base + size_t(from) * 16, size, full + slot, evict_first_policy());
      else if (size) bulk_g2s(at, r.base + size_t(from) * 16, size, full + slot);
      if (more) bulk_g2s(bits + slot * kBits, r.mask + off, more, full + slot);
    }
    return true;
  }
  // after the last fill: all copies have landed, whatever the block's other warps do
  __device__ __forceinline__ bool landed() const {
    bool ok = true;
    for (uint32_t i = 0; i < slots; ++i)
      if (turn || i < slot) ok = mbar_wait(full + i, (i < slot ? turn : turn - 1) & 1u) && ok;
    return ok;
  }
  __device__ __forceinline__ uint4* part(uint32_t at) const {
    return reinterpret_cast<uint4*>(data + at * kBytes) + threadIdx.x;
  }
  // A taker: its groups of the chunk in the slot, by the rows' conventions, and their
  // maximum.  kept: the chunk stays in its slot, as taken (wrote: something of it was
  // written).  late: a wait ran out; none is begun any more.
  template <bool KEPT>
  __device__ __forceinline__ float take(const Row<BF16>& r, uint32_t g, uint4* v, bool& wrote, bool& late) const {
    const uint32_t lo = r.first_whole(), hi = r.end_whole(), own = g + threadIdx.x;
    const bool with_bits = copies_bits(r);
    uint32_t allowed[PER];
    if (r.mask && !with_bits) {
#pragma unroll
      for (uint32_t k = 0; k < PER; ++k) {
        const uint32_t at = own + k * kTakers * 32;
        allowed[k] = at < end(r) ? r.mask_bits(int(at * F::E) - int(r.a)) : 0u;
      }
    }
    if (!late) late = !__all_sync(0xFFFFFFFFu, mbar_wait(full + slot, turn & 1u));
    uint4* held = part(slot);
#pragma unroll
    for (uint32_t k = 0; k < PER; ++k) v[k] = held[k * kTakers * 32];
    if (with_bits) {
      const unsigned char* p = bits + slot * kBits + (BF16 ? threadIdx.x : threadIdx.x / 2);
#pragma unroll
      for (uint32_t k = 0; k < PER; ++k)
        allowed[k] = uint32_t(p[k * (kBits / PER)]) >> (BF16 ? 0u : (threadIdx.x & 1u) * 4u);
    }
    bool changed = r.mask != nullptr;
    if (g < lo || g + kGroups > hi) {  // groups that the copies do not bring
      changed = true;
#pragma unroll
      for (uint32_t k = 0; k < PER; ++k) {
        const uint32_t at = own + k * kTakers * 32;
        if (at < lo || at >= hi) v[k] = r.edge(at);
      }
    }
    if (r.mask) {
#pragma unroll
      for (uint32_t k = 0; k < PER; ++k) v[k] = r.masked(v[k], allowed[k]);
    }
    float t = groups_max_nan<BF16, PER>(v);
    if (fkey(t) >= kKeyInf) {
      changed = true;
#pragma unroll
      for (uint32_t k = 0; k < PER; ++k) v[k] = clean_group<BF16>(v[k]);
      t = groups_max_nan<BF16, PER>(v);
    }
    if (KEPT && changed) {
#pragma unroll
      for (uint32_t k = 0; k < PER; ++k) held[k * kTakers * 32] = v[k];
      wrote = true;
    }
    return t;
  }
  // This warp has taken the chunk in the slot.  An arrival may overtake loads that are
  // still queued behind stores, so it follows a vote on something that needs the values
  // of all loads of all lanes and is never true: every load has returned by then.  The
  // thread that fills the slot puts the proxy fence between the loads and the next copy
  // (of 512 x 128256 with a fence in every taker 29.8 us, in the filler 29.2).
  __device__ __forceinline__ void release(bool never) const {
    const bool none = __any_sync(0xFFFFFFFFu, never);
    if ((threadIdx.x & 31) == 0 && !none) mbar_arrive(empty + slot);
  }
  // a word of each of PER groups by the rows' conventions is a NaN
  static __device__ __forceinline__ bool holds_nan(const uint4* v) {
    uint32_t word = v[0].x;
#pragma unroll
    for (uint32_t k = 1; k < PER; ++k) word = max(word, v[k].x);
    return word == 0xFFFFFFFFu;
  }
};

// ---- the loss alone ---------------------------------------------------------------------
//
// Nothing of a row is needed twice.  The warps send their maxima and sums of the
// cluster's i-th row to block i mod n, where one more warp (of one or two) has read
// the row's list meanwhile and finishes the row.  2048 x 128256 bf16: 81.2 us, 6.5 TB/s, bound by the
// memory.
//
// Few barriers and many loads at once: 8 groups of a thread a chunk.  Of 2048 x 128256
// bf16, masked too: 16 warps x 2 groups x 6 chunks 93.7 and 108.8 us, 8 x 4 x 6 83.9 and
// 95.5, 8 x 8 x 3 83.6 and 86.2, three blocks of 8 x 4 x 4 an SM 86.8 and 90.8.
constexpr uint32_t kLossPer = 8;       // groups of a thread in a chunk
constexpr uint32_t kLossSlots = 3;     // chunks on their way or being taken, at most
constexpr uint32_t kLossBlocks = 2 * 152;  // resident
constexpr uint32_t kLossBatch = 8;     // list entries of a lane read at a time
// Longer lists and shorter rows (in bytes) take two warps, a row each, the others one:
//   2048 x 32000, 64 listed     one 37.5 us, two 29.2
//   2048 x 32000, 1024 listed   two 108, one reading an entry at a time 316
//   1024 x 128256, 256 listed   one 54.3, two 47.1; 64 listed 46.0 and 45.9
//   512 x 128256 masked, 64     one 28.7, two 30.9 (fewer registers for the takers)
constexpr uint32_t kLongList = 64, kShortLossRow = 128 << 10;
constexpr size_t kHalfSmem = 113 * 1024;   // of a block of two on an SM
// Few rows are split over clusters of 2, 4 or 8 blocks as long as all are resident
// together (36 clusters of 8, 74 of 4).  Microseconds of B x 128256 bf16 by cluster
// size, at 16 warps x 2 groups x 6 chunks:
//   B      1     2     4     8    16
//   512  30.3  31.4  30.8  37.1  66.5
//   128  16.0  11.4  12.1  13.6
//   64   13.1  10.4   8.2   9.1
//   32          8.1   7.1   6.0
//   4                 5.4   4.4   4.3
constexpr uint32_t kLossCluster = 8, kLossSplit = 288;

struct LossShared {
  uint64_t full[kLossSlots], empty[kLossSlots];
  uint64_t bar_rec[2];                // by turns of this block's rows
  uint64_t done[kLossCluster][2];     // ... of each block's: their records have been read
  __align__(16) Record rec[2][kLossCluster * kTakers];
};
// ... then the lists' logits, teacher's and student's, and the ring
__host__ __device__ constexpr size_t loss_fixed(uint32_t K, uint32_t lists) {
  return sizeof(LossShared) + ((size_t(K) * 8 * lists + 15) & ~size_t(15));
}

template <bool BF16, uint32_t LISTS>
__global__ void __launch_bounds__((kTakers + 1 + LISTS) * 32, 2) loss_kernel(const DistillArgs a, uint32_t B, uint32_t slots) {
  extern __shared__ __align__(16) unsigned char smem[];
  LossShared& s = *reinterpret_cast<LossShared*>(smem);
  static_assert(sizeof(LossShared) % 16 == 0, "the list and the ring lie behind it");
  using R = Ring<BF16, kLossPer>;
  R ring(s.full, s.empty, smem + loss_fixed(a.K, LISTS), slots);
  griddep_launch_dependents();
  const uint32_t n = cluster_size(), rank = cluster_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t first = blockIdx.x / n, step = gridDim.x / n, rows = (B - first + step - 1) / step;
  if (tid == 0) {
    ring.init();
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(s.bar_rec + i, 1);
      for (uint32_t r = 0; r < kLossCluster; ++r) mbar_init(&s.done[r][i], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  may_send();
  griddep_wait();
  const float T = a.temp, c = exp_scale(T);
  auto row = [&](uint32_t i) { return Row<BF16>(a.logits, a.ld, a.bitmask, a.W, a.V, first + i * step); };
  bool late = false;
  if (warp == kTakers) {  // fills the ring
    if (lane == 0) {
      for (uint32_t i = 0; i < rows && !late; ++i) late = !ring.fill(row(i), n, rank, true);
      late = !ring.landed() || late;
    }
    __syncwarp();
    ready_others();
  } else if (warp < kTakers) {
    for (uint32_t i = 0; i < rows; ++i) {
      const Row<BF16> r = row(i);
      float tm = -INFINITY;
      float2 acc = {};
      bool wrote;
#pragma unroll 1
      for (uint32_t g = rank * R::kGroups; g < R::end(r); g += n * R::kGroups, ring.next()) {
        uint4 v[kLossPer];
        const float t = ring.template take<false>(r, g, v, wrote, late);
        ring.release(t == INFINITY);  // replaced by the largest finite value
        add_groups<BF16, kLossPer>(v, t, c, tm, acc);
      }
      if (i == 0) ready_others();
      const unsigned long long rec = warp_record(tm, acc.x + acc.y, c);
      const uint32_t home = i % n, use = i / n;  // of the home's records, by turns in two buffers
      if (lane == 0) {
        if (use >= 2 && !late) late = !wait_sent(&s.done[home][use & 1u], (use / 2 - 1) & 1u);
        send(at_rank(&s.rec[use & 1u][rank * kTakers + warp], home), rec, at_rank(s.bar_rec + (use & 1u), home));
      }
      late = __any_sync(0xFFFFFFFFu, late);
    }
  } else {  // the lists' warps finish the rows that are this block's, in turn
    const uint32_t K = a.K, turn = warp - (kTakers + 1);
    float* list_t = reinterpret_cast<float*>(smem + sizeof(LossShared)) + size_t(turn) * 2 * K;  // -inf: does not count
    float* list_x = list_t + K;
    ready_others();
    for (uint32_t i = rank + turn * n; i < rows; i += LISTS * n) {
      const uint32_t b = first + i * step, use = i / n;
      const Row<BF16> r = row(i);
      if (lane == 0 && !late) mbar_expect_tx(s.bar_rec + (use & 1u), n * kTakers * uint32_t(sizeof(Record)));
      float tm = -INFINITY;
#pragma unroll 1
      for (uint32_t k0 = lane; k0 < K; k0 += 32 * kLossBatch) {  // the loads of a batch are under way together
        uint32_t id[kLossBatch];
        float t[kLossBatch], x[kLossBatch];
#pragma unroll
        for (uint32_t u = 0; u < kLossBatch; ++u) {
          const bool in = k0 + u * 32 < K;
          id[u] = in ? a.ids[size_t(b) * K + k0 + u * 32] : CG_NO_TOKEN;
          t[u] = in ? a.teacher[size_t(b) * K + k0 + u * 32] : -INFINITY;
        }
#pragma unroll
        for (uint32_t u = 0; u < kLossBatch; ++u) x[u] = r.at_any(id[u]);
#pragma unroll
        for (uint32_t u = 0; u < kLossBatch; ++u) {
          if (k0 + u * 32 >= K) break;
          if (id[u] >= a.V && id[u] != CG_NO_TOKEN) record_error(a.status, CG_DEV_BAD_TOKEN);
          const float tk = teacher_logit(t[u]);
          const bool counts = x[u] > -INFINITY && tk > -INFINITY;
          list_x[k0 + u * 32] = x[u];
          list_t[k0 + u * 32] = counts ? tk : -INFINITY;
          if (counts) tm = fmaxf(tm, tk);
        }
      }
      tm = warp_reduce(tm, MaxOp());
      const bool listed = tm > -INFINITY;
      float ts = 0.f;
      for (uint32_t k = lane; k < K; k += 32)
        if (list_t[k] > -INFINITY) ts += ex2((list_t[k] - tm) * c);
      ts = warp_reduce(ts, SumOp());
      if (!late) late = !__all_sync(0xFFFFFFFFu, wait_sent(s.bar_rec + (use & 1u), (use / 2) & 1u));
      float M, S, rest;
      merge(s.rec[use & 1u], n * kTakers, c, M, S, rest);
      __syncwarp();
      if (i + 2 * n < rows && lane < n) {  // the buffer is used again
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                         at_rank(&s.done[rank][use & 1u], lane))
                     : "memory");
      }
      const float log_ts = logf(ts), log_s = log1pf(rest);
      float part = 0.f;
      for (uint32_t k = lane; k < K; k += 32)
        if (list_t[k] > -INFINITY) part += loss_term(list_t[k] - tm, ts, log_ts, list_x[k] - M, log_s, c, T);
      part = warp_reduce(part, SumOp());
      if (lane == 0) store_loss(a, b, listed ? T * (T * part) : 0.f, M, S, log_s);
    }
  }
  if (late) record_error(a.status, CG_DEV_TIMEOUT);
  __syncwarp();
  cluster_sync(n);  // what others send arrives, and so do their signals
}

// ---- the gradient, and the loss with it ---------------------------------------------------
//
// A block's chunks of a row stay in the ring until their gradient is written.  With the
// loss the warps take them once for the row's maximum and sum, tell every block
// of the cluster, and take them again for the gradient; with the kept normaliser the
// second pass is the only one.  Every gradient is written as T w p_v first; the lists'
// warps write the listed tokens' over after the row.  They also tell the cluster when
// they have read the row's listed logits, before which nothing of it is written: the
// gradient may take the logits' place.  (That keeps a cluster's blocks side by side, too:
// without it the gradient alone of 512 x 151936 took 63.8 us, with it 57.2.)
//
// 2048 x 128256 bf16: loss and gradient 197.4 us, 5.3 TB/s of reads and writes; the
// gradient alone 162 to 171, 6.1 to 6.5 TB/s.  The memory bounds them, and with the loss the exchange
// of a row's sums, which the next row's copies cover only in part: of a block's six chunks
// two are ahead.  Fetching a chunk's values before the stores of the one before: 218 us.
// Clusters of 6 and 8 blocks with three or two chunks each are not all resident together:
// 397 and 472 us.
constexpr uint32_t kGradPer = 4;       // groups of a thread in a chunk
constexpr uint32_t kGradSlots = 12;    // at most
constexpr uint32_t kListWarps = 4;
constexpr uint32_t kListThreads = kListWarps * 32;
constexpr uint32_t kGradThreads = (kTakers + 1) * 32 + kListThreads;

struct GradShared {
  uint64_t full[kGradSlots], empty[kGradSlots];
  uint64_t bar_rec[2], bar_list[2], bar_done[2];   // by turns of the rows: the cluster's records and notes, this
                                                   // block's list, its takers' stores
  __align__(16) Record rec[2][kMaxCluster * kTakers];
  uint32_t note[2][kMaxCluster];
  float tm[2], ts[2];                              // the list's maximum (-inf: none listed) and sum
  uint32_t repeated[2];
  float red[kListWarps];
};
// ... then two lists, the hash and the ring
__host__ __device__ inline size_t grad_fixed(uint32_t K) {
  return (sizeof(GradShared) + size_t(K) * 24 + size_t(hash_slots(K)) * 4 + 15) & ~size_t(15);
}

__device__ __forceinline__ void list_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kListThreads) : "memory"); }
template <typename Op>
__device__ __forceinline__ float list_fold(float v, Op op, float* red) {
  v = warp_reduce(v, op);
  const uint32_t w = (threadIdx.x >> 5) - (kTakers + 1);
  if ((threadIdx.x & 31) == 0) red[w] = v;
  list_sync();
  v = op(op(red[0], red[1]), op(red[2], red[3]));
  list_sync();
  return v;
}
static_assert(kListWarps == 4, "the fold above");

template <bool BF16, bool LOSS>
__global__ void __launch_bounds__(kGradThreads, 2) grad_kernel(const DistillArgs a, uint32_t B, uint32_t slots) {
  extern __shared__ __align__(16) unsigned char smem[];
  GradShared& s = *reinterpret_cast<GradShared*>(smem);
  const uint32_t K = a.K;
  unsigned char* lists = smem + sizeof(GradShared);
  uint32_t* hash = reinterpret_cast<uint32_t*>(lists + size_t(K) * 24);
  using R = Ring<BF16, kGradPer>;
  R ring(s.full, s.empty, smem + grad_fixed(K), slots);
  griddep_launch_dependents();
  const uint32_t n = cluster_size(), rank = cluster_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t first = blockIdx.x / n, step = gridDim.x / n, rows = (B - first + step - 1) / step;
  // bytes of a row's records and notes
  const uint32_t told = n * (LOSS ? kTakers * uint32_t(sizeof(Record)) + 4u : 4u);
  if (tid == 0) {
    ring.init();
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(s.bar_rec + i, 1);
      mbar_init(s.bar_list + i, 1);
      mbar_init(s.bar_done + i, kTakers);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    // armed once a phase: the first two rows here, the others when the phase before is over
    mbar_expect_tx(s.bar_rec, told);
    mbar_expect_tx(s.bar_rec + 1, told);
  }
  __syncthreads();
  may_send();
  griddep_wait();
  const float T = a.temp, c = exp_scale(T);
  auto row = [&](uint32_t i) { return Row<BF16>(a.logits, a.ld, a.bitmask, a.W, a.V, first + i * step); };
  auto out = [&](uint32_t i) {
    return static_cast<char*>(a.grad) + size_t(first + i * step) * a.ld_grad * Fmt<BF16>::kSize;
  };
  bool late = false;
  if (warp == kTakers) {  // fills the ring
    if (lane == 0) {
      for (uint32_t i = 0; i < rows && !late; ++i) late = !ring.fill(row(i), n, rank, false);
      late = !ring.landed() || late;
    }
    __syncwarp();
    ready_others();
  } else if (warp < kTakers) {
    for (uint32_t i = 0; i < rows; ++i) {
      const Row<BF16> r = row(i);
      const uint32_t b = first + i * step, buf = i & 1u, parity = (i / 2) & 1u;
      const float up = a.up ? a.up[b] : 1.f;
      float M = 0.f, S = 1.f;  // p = exp2((x - M) c) / S
      if (!LOSS) kept_norm(a, b, M, S);
      bool wrote = false;
      if (LOSS) {
        R ahead = ring;
        float tm = -INFINITY;
        float2 acc = {};
#pragma unroll 1
        for (uint32_t g = rank * R::kGroups; g < R::end(r); g += n * R::kGroups, ahead.next()) {
          uint4 v[kGradPer];
          const float t = ahead.template take<true>(r, g, v, wrote, late);
          add_groups<BF16, kGradPer>(v, t, c, tm, acc);
        }
        if (i == 0) ready_others();
        const unsigned long long rec = warp_record(tm, acc.x + acc.y, c);
        if (lane < n) send(at_rank(&s.rec[buf][rank * kTakers + warp], lane), rec, at_rank(s.bar_rec + buf, lane));
      } else if (i == 0) {
        ready_others();
      }
      if (!late) late = !__all_sync(0xFFFFFFFFu, mbar_wait(s.bar_list + buf, parity) &&
                                                 wait_sent(s.bar_rec + buf, parity));
      float rest = 0.f;
      if (LOSS) merge(s.rec[buf], n * kTakers, c, M, S, rest);
      const bool listed = s.tm[buf] > -INFINITY;
      const float w = __fdiv_rn(listed ? T * up : 0.f, S);
      char* to = out(i);
      const bool wide = ((reinterpret_cast<uintptr_t>(to) / Fmt<BF16>::kSize - r.a) & (Fmt<BF16>::E - 1)) == 0;
      const float2 nm = make_float2(-M, -M), c2 = make_float2(c, c), w2 = make_float2(w, w);
#pragma unroll 1
      for (uint32_t g = rank * R::kGroups; g < R::end(r); g += n * R::kGroups, ring.next()) {
        uint4 v[kGradPer];
        if (LOSS) {
          const uint4* held = ring.part(ring.slot);
#pragma unroll
          for (uint32_t k = 0; k < kGradPer; ++k) v[k] = held[k * kTakers * 32];
          // what this thread wrote there comes before the next copy
          if (wrote) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          ring.release(R::holds_nan(v));
        } else {
          ring.release(ring.template take<false>(r, g, v, wrote, late) == INFINITY);
        }
#pragma unroll
        for (uint32_t k = 0; k < kGradPer; ++k) {
          const uint32_t at = g + k * kTakers * 32 + tid;
          float2 d[Fmt<BF16>::E / 2];
#pragma unroll
          for (uint32_t q = 0; q < Fmt<BF16>::E / 2; ++q) {
            d[q] = make_float2(0.f, 0.f);
            if (listed) d[q] = __fmul2_rn(ex2_pair(__fmul2_rn(__fadd2_rn(pair<BF16>(v[k], q), nm), c2)), w2);
          }
          if (at < R::end(r)) store_group<BF16>(to, int(at * Fmt<BF16>::E) - int(r.a), a.V, wide, d);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(s.bar_done + buf);
    }
  } else {  // the lists
    const uint32_t lt = tid - (kTakers + 1) * 32, size = hash_slots(K);
    auto read = [&](uint32_t i) {  // row i's, its maximum, sum and repeated ids
      const Row<BF16> r = row(i);
      const uint32_t b = first + i * step, buf = i & 1u;
      const List l(lists + buf * size_t(K) * 12, K);
      for (uint32_t k = lt; k < size; k += kListThreads) hash[k] = CG_NO_TOKEN;
      if (lt == 0) s.repeated[buf] = 0;
      const float tm = list_fold(l.read<BF16>(a, r, b, lt, kListThreads, rank == 0), MaxOp(), s.red);
      float ts = 0.f;
      for (uint32_t k = lt; k < K; k += kListThreads) {
        const uint32_t id = l.id[k];
        if (id == CG_NO_TOKEN) continue;
        ts += ex2((l.t[k] - tm) * c);
        if (claimed_before(hash, size, id)) s.repeated[buf] = 1;
      }
      ts = list_fold(ts, SumOp(), s.red);
      if (lt == 0) {
        s.tm[buf] = tm;
        s.ts[buf] = ts;
        mbar_arrive(s.bar_list + buf);
      }
    };
    auto tell = [&](uint32_t i) {  // after what of the buffer's former row has been read here
      if (lt < n) send(at_rank(&s.note[i & 1u][rank], lt), 1u, at_rank(s.bar_rec + (i & 1u), lt));
    };
    read(0);
    ready_others();
    tell(0);
    for (uint32_t i = 0; i < rows; ++i) {
      const uint32_t b = first + i * step, buf = i & 1u, parity = (i / 2) & 1u;
      if (i + 1 < rows) read(i + 1);
      if (!late) late = !__all_sync(0xFFFFFFFFu, wait_sent(s.bar_rec + buf, parity));
      float M = 0.f, S = 1.f, rest = 0.f;
      if (LOSS) merge(s.rec[buf], n * kTakers, c, M, S, rest);
      else kept_norm(a, b, M, S);
      list_sync();
      if (!late && lt == 0 && i + 2 < rows) mbar_expect_tx(s.bar_rec + buf, told);
      if (i + 1 < rows) tell(i + 1);
      const Row<BF16> r = row(i);
      const List l(lists + buf * size_t(K) * 12, K);
      const float tm = s.tm[buf], ts = s.ts[buf];
      const bool listed = tm > -INFINITY;
      if (LOSS && rank == 0) {
        float part = 0.f;
        const float log_ts = logf(ts), log_s = log1pf(rest);
        for (uint32_t k = lt; k < K; k += kListThreads)
          if (l.id[k] != CG_NO_TOKEN) part += loss_term(l.t[k] - tm, ts, log_ts, l.x[k] - M, log_s, c, T);
        part = list_fold(part, SumOp(), s.red);
        if (lt == 0) store_loss(a, b, listed ? T * (T * part) : 0.f, M, S, log_s);
      }
      if (!late) late = !__all_sync(0xFFFFFFFFu, mbar_wait(s.bar_done + buf, parity));
      if (listed) {
        const bool repeated = s.repeated[buf] != 0;
        const float scale = T * (a.up ? a.up[b] : 1.f);
        char* to = out(i);
        for (uint32_t k = lt; k < K; k += kListThreads) {
          const uint32_t id = l.id[k];
          if (id == CG_NO_TOKEN || ((id + r.a) / Fmt<BF16>::E / R::kGroups) % n != rank) continue;
          l.write<BF16>(to, k, K, repeated, tm, ts, M, S, c, scale);
        }
      }
      list_sync();  // the next list takes this one's place
    }
  }
  if (late) record_error(a.status, CG_DEV_TIMEOUT);
  __syncwarp();
  cluster_sync(n);
}

// ---- the gradient of short rows and small batches -------------------------------------------
//
// Where a cluster has one row, or rows of a chunk or two, there is nothing to stream: the
// blocks hold the row (logit_row.cuh) and more of them share an SM.
//
// Microseconds, held and streamed, loss and gradient, then the gradient alone (bf16):
//   4096 x 12000    78.2   79.5     52.1   60.4
//   4096 x 20000    94.8   93.2     66.3   68.9
//   1024 x 32000    37.3   35.5     32.0   29.4
//   64 x 64006       9.1    7.5      7.2    7.9
//   64 x 128256     13.4   10.5     10.4   10.8
//   128 x 128256    23.6   17.7     19.2   16.2
//   2048 x 128256  223.2  197.5    182.2  161.9
constexpr uint64_t kShortRow = 48 << 10, kSmallLoss = 6 << 20, kSmallGrad = 16 << 20;  // bytes
// Groups of a thread for many rows: 64 KB parts, three blocks an SM.
constexpr uint32_t kFull = 16;
constexpr size_t kThird = 75 * 1024;  // shared memory of a block of three on an SM

struct HeldShared : Meet {
  uint32_t repeated;
};
// ... then the list, the hash and the part
__host__ __device__ inline size_t held_fixed(uint32_t K) {
  return (sizeof(HeldShared) + size_t(K) * 12 + size_t(hash_slots(K)) * 4 + 15) & ~size_t(15);
}

template <bool BF16, bool LOSS>
__global__ void __launch_bounds__(kThreads, 3) held_kernel(const DistillArgs a, uint32_t nv) {
  extern __shared__ __align__(16) unsigned char smem[];
  HeldShared& s = *reinterpret_cast<HeldShared*>(smem);
  const List l(smem + sizeof(HeldShared), a.K);
  uint32_t* hash = reinterpret_cast<uint32_t*>(smem + sizeof(HeldShared) + size_t(a.K) * 12);
  griddep_launch_dependents();
  const uint32_t n = cluster_size(), rank = cluster_rank(), b = blockIdx.x / n, tid = threadIdx.x, K = a.K;
  begin(s);
  Held<BF16> h(Row<BF16>(a.logits, a.ld, a.bitmask, a.W, a.V, b), nv, smem + held_fixed(K));
  griddep_wait();
  h.start(s, false);
  may_send();
  const float T = a.temp, c = exp_scale(T);
  // the teacher's list
  const uint32_t slots = hash_slots(K);
  for (uint32_t i = tid; i < slots; i += kThreads) hash[i] = CG_NO_TOKEN;
  if (tid == 0) s.repeated = 0;
  const float tm = block_max(l.read<BF16>(a, h.r, b, tid, kThreads, rank == 0), s.red_f);
  const bool listed = tm > -INFINITY;
  float ts = 0.f;
  for (uint32_t k = tid; k < K; k += kThreads) {
    const uint32_t id = l.id[k];
    if (id == CG_NO_TOKEN) continue;
    ts += ex2((l.t[k] - tm) * c);
    if (claimed_before(hash, slots, id)) s.repeated = 1;
  }
  __syncthreads();
  ts = block_sum(ts, s.red_f);
  __syncthreads();

  float M = 0.f, S = 1.f;  // p = exp2((x - M) c) / S
  if (LOSS) {
    if (!h.template take<true>(s, c)) record_error(a.status, CG_DEV_TIMEOUT);
    const unsigned long long rec = h.record(c);
    ready_others();
    h.publish(s, rec);
    if (tid < 32) {
      const bool ok = wait_sent(&s.bar_rec);
      float m, sum, rest;
      merge(s.rec, n * kWarps, c, m, sum, rest);
      if (tid == 0) {
        s.M = m;
        s.rest = rest;
        if (!ok) {
          s.late = 1;
          record_error(a.status, CG_DEV_TIMEOUT);
        }
      }
    }
    __syncthreads();
    M = s.M;
    S = M > -INFINITY ? 1.f + s.rest : 0.f;
    if (rank == 0) {
      float part = 0.f;
      const float log_ts = logf(ts), log_s = log1pf(s.rest);
      for (uint32_t k = tid; k < K; k += kThreads)
        if (l.id[k] != CG_NO_TOKEN) part += loss_term(l.t[k] - tm, ts, log_ts, l.x[k] - M, log_s, c, T);
      __syncthreads();
      part = block_sum(part, s.red_f);
      if (tid == 0) store_loss(a, b, listed ? T * (T * part) : 0.f, M, S, log_s);
    }
  } else {
    kept_norm(a, b, M, S);
    if (!h.template take<false>(s, c)) record_error(a.status, CG_DEV_TIMEOUT);
    ready_others();
    if (a.grad == a.logits) cluster_sync(n);  // every block has read what it needs
  }

  const float scale = listed ? T * (a.up ? a.up[b] : 1.f) : 0.f;
  const float r = __fdiv_rn(scale, S);
  char* row = static_cast<char*>(a.grad) + size_t(b) * a.ld_grad * Fmt<BF16>::kSize;
  const bool wide = ((reinterpret_cast<uintptr_t>(row) / Fmt<BF16>::kSize - h.r.a) & (Fmt<BF16>::E - 1)) == 0;
  const float2 nm = make_float2(-M, -M), c2 = make_float2(c, c), r2 = make_float2(r, r);
#pragma unroll 4
  for (uint32_t j = 0; j < nv; ++j) {
    if (!h.r.in_row(h.group(j))) break;
    const uint4 v = h.at(j);
    float2 g[Fmt<BF16>::E / 2];
#pragma unroll
    for (uint32_t q = 0; q < Fmt<BF16>::E / 2; ++q) {
      g[q] = make_float2(0.f, 0.f);
      if (listed) g[q] = __fmul2_rn(ex2_pair(__fmul2_rn(__fadd2_rn(pair<BF16>(v, q), nm), c2)), r2);
    }
    store_group<BF16>(row, h.first_token(j), a.V, wide, g);
  }
  __syncthreads();
  const bool repeated = s.repeated != 0;
  for (uint32_t k = tid; listed && k < K; k += kThreads) {
    const uint32_t id = l.id[k];
    if (id == CG_NO_TOKEN) continue;
    const uint32_t g = (id + h.r.a) / Fmt<BF16>::E;
    if ((g / kThreads) % n != rank) continue;
    l.write<BF16>(row, k, K, repeated, tm, ts, M, S, c, scale);
  }
  if (LOSS && s.late) leave_last(n);
}

template <bool BF16, uint32_t LISTS>
cudaError_t launch_loss(int device, uint32_t B, const DistillArgs& a, cudaStream_t stream) {
  using R = Ring<BF16, kLossPer>;
  const uint32_t chunks = (a.V / Fmt<BF16>::E + R::kGroups) / R::kGroups;
  uint32_t n = 1;
  while (n < kLossCluster && 2 * n <= chunks && uint64_t(B) * 2 * n <= kLossSplit) n *= 2;
  const size_t fixed = loss_fixed(a.K, LISTS);
  uint32_t slots = kLossSlots;
  while (fixed + R::bytes(slots, a.bitmask) > kHalfSmem) --slots;
  return launch_clusters<loss_kernel<BF16, LISTS>>(device, n == 1 && B > kLossBlocks ? kLossBlocks : B, n,
                                                   (kTakers + 1 + LISTS) * 32, fixed + R::bytes(slots, a.bitmask), stream,
                                                   a, B, slots);
}

// Clusters of n = 1, 2, 4, 8, 16 blocks that are resident together, asked once per device, n
// and blocks an SM (which smem decides); 0 and an error where the device cannot tell
template <auto Kernel>
uint32_t resident(int device, uint32_t n, size_t smem, cudaError_t& e) {
  static DeviceAnswers known[2][5];
  e = cudaSuccess;
  return uint32_t(known[smem > kHalfSmem][__builtin_ctz(n)].get(device, [&] {
    int clusters = 0;
    e = raise_limits<Kernel>(device);
    const ClusterLaunch l(1, n, kGradThreads, smem > kHalfSmem ? kMaxSmem : kHalfSmem, nullptr);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&clusters, Kernel, &l.cfg);
    if (e == cudaSuccess && clusters <= 0) e = cudaErrorInvalidConfiguration;
    return e == cudaSuccess ? clusters : 0;
  }));
}

template <bool BF16, bool LOSS>
cudaError_t launch_grad(int device, uint32_t B, const DistillArgs& a, cudaStream_t stream) {
  using R = Ring<BF16, kGradPer>;
  constexpr uint32_t E = Fmt<BF16>::E;
  const uint32_t chunks = ((a.V + 2 * E - 2) / E + R::kGroups - 1) / R::kGroups;
  const size_t fixed = grad_fixed(a.K);
  uint32_t slots = 0, n = 1;
  // a row has to fit the cluster's rings (with the loss): the longest take one block an SM
  for (size_t limit : {kHalfSmem, size_t(kMaxSmem)}) {
    slots = std::min(kGradSlots, uint32_t((limit - fixed) / R::bytes(1, a.bitmask)));
    n = 1;
    while (n < kMaxCluster && n * slots < chunks) n *= 2;
    if (n * slots >= chunks) break;
  }
  while (n < kLossCluster && 2 * n <= chunks && uint64_t(B) * 2 * n <= kLossSplit) n *= 2;
  const size_t smem = fixed + R::bytes(slots, a.bitmask);
  cudaError_t e;
  const uint32_t at_once = resident<grad_kernel<BF16, LOSS>>(device, n, smem, e);
  if (e != cudaSuccess) return e;
  return launch_clusters<grad_kernel<BF16, LOSS>>(device, std::min(B, at_once), n, kGradThreads, smem, stream, a, B,
                                                       slots);
}

template <bool BF16>
cudaError_t launch_held(int device, uint32_t B, const DistillArgs& a, bool loss, cudaStream_t stream) {
  const size_t fixed = held_fixed(a.K);
  uint32_t full = kFull;
  while (full > 1 && fixed + part_bytes(BF16, full, a.bitmask) > kThird) --full;
  const Plan plan = plan_row(BF16, a.V, B, rows_on_grid(a.logits, BF16 ? CG_BF16 : CG_F32, a.ld), full);
  const size_t smem = fixed + part_bytes(BF16, plan.nv, a.bitmask);
  return loss ? launch_clusters<held_kernel<BF16, true>>(device, B, plan.n, kThreads, smem, stream, a, plan.nv)
              : launch_clusters<held_kernel<BF16, false>>(device, B, plan.n, kThreads, smem, stream, a, plan.nv);
}
// whether rows with a gradient stream
bool streams(bool bf16, uint32_t V, uint32_t B, bool loss) {
  const uint64_t row = uint64_t(V) * (bf16 ? 2 : 4);
  return row > kShortRow && row * B > (loss ? kSmallLoss : kSmallGrad);
}

template <bool BF16>
cudaError_t launch_distill(int device, uint32_t B, const DistillArgs& a, bool loss, cudaStream_t stream) {
  if (!a.grad)
    return a.K > kLongList || a.V * (BF16 ? 2u : 4u) <= kShortLossRow ? launch_loss<BF16, 2>(device, B, a, stream)
                                                                      : launch_loss<BF16, 1>(device, B, a, stream);
  if (!streams(BF16, a.V, B, loss)) return launch_held<BF16>(device, B, a, loss, stream);
  return loss ? launch_grad<BF16, true>(device, B, a, stream) : launch_grad<BF16, false>(device, B, a, stream);
}

int distill(cg_ctx* c, const char* call, const DistillArgs& base, int dtype, uint32_t B, bool loss) {
  if (B == 0) return CG_OK;
  DeviceGuard dg(ctx_device(c), call);
  if (!dg.ok) return CG_E_CUDA;
  const CtxView v = ctx_view(c);
  DistillArgs a = base;
  a.W = v.t.W;
  a.status = v.t.status;
  const int dev = ctx_device(c);
  const cudaError_t e = dtype == CG_BF16 ? launch_distill<true>(dev, B, a, loss, v.stream)
                                         : launch_distill<false>(dev, B, a, loss, v.stream);
  return e == cudaSuccess ? CG_OK : CG_E_CUDA;
}

// Whether the gradient overlaps the logits other than as the same rows: their
// byte ranges meet, and they are not columns of one buffer side by side.
bool overlaps(uintptr_t x, uint64_t ldx, uintptr_t g, uint64_t ldg, uint32_t B, uint32_t V, uintptr_t size) {
  if (x == g) return ldx != ldg && B > 1;
  const uint64_t nx = (uint64_t(B - 1) * ldx + V) * size, ng = (uint64_t(B - 1) * ldg + V) * size;
  if (x + nx <= g || g + ng <= x) return false;
  if (B == 1 || ldx != ldg) return true;
  const uint64_t pitch = ldx * size, off = (g > x ? g - x : pitch - (x - g) % pitch) % pitch;
  return off < V * size || pitch - off < V * size;
}

// host checks of what the two calls share; CG_OK or the error
int list_args(const cg_ctx* c, const void* logits, int dtype, uint32_t B, uint32_t V, uint64_t ld,
              const uint32_t* bitmask, const uint32_t* ids, const float* teacher, uint32_t K, float temp,
              const float* up, const void* grad, uint64_t ld_grad) {
  if (!row_args_ok(c, logits, dtype, B, V, ld, bitmask)) return CG_E_ARG;
  if (K == 0 || (B && (!ids || !teacher)) || !(temp > 0.f) || temp > FLT_MAX) return CG_E_ARG;
  if (!aligned4(ids) || !aligned4(teacher) || !aligned4(up)) return CG_E_ARG;
  if (grad) {
    const uintptr_t size = dtype == CG_BF16 ? 2 : 4;
    if (ld_grad < V || ld_grad > (uint64_t(1) << 40) || reinterpret_cast<uintptr_t>(grad) % size) return CG_E_ARG;
    if (B && overlaps(reinterpret_cast<uintptr_t>(logits), ld, reinterpret_cast<uintptr_t>(grad), ld_grad, B, V, size))
      return CG_E_ARG;
  }
  return K > CG_TOP_MAX ? CG_E_LIMIT : CG_OK;
}

}  // namespace
}  // namespace cgk

extern "C" int cg_distill_loss_norm(cg_ctx* c, const void* d_logits, int dtype, uint32_t B, uint32_t V, uint64_t ld,
                                    const uint32_t* d_bitmask, const uint32_t* d_ids, const float* d_teacher,
                                    uint32_t K, float temp, float* d_out_loss, float* d_out_lse, float* d_out_norm,
                                    const float* d_grad_loss, void* d_out_grad, uint64_t ld_grad) {
  using namespace cgk;
  const int rc = list_args(c, d_logits, dtype, B, V, ld, d_bitmask, d_ids, d_teacher, K, temp, d_grad_loss,
                           d_out_grad, ld_grad);
  if (rc != CG_OK) return rc;
  if ((B && !d_out_loss) || !aligned4(d_out_loss) || !aligned4(d_out_lse) || !aligned4(d_out_norm)) return CG_E_ARG;
  const DistillArgs a{d_logits, ld,      d_bitmask,  V,         0,          d_ids,       d_teacher,  K,       temp,
                      nullptr,  nullptr, d_out_loss, d_out_lse, d_out_norm, d_grad_loss, d_out_grad, ld_grad, nullptr};
  return distill(c, "cg_distill_loss", a, dtype, B, true);
}

extern "C" int cg_distill_loss(cg_ctx* c, const void* d_logits, int dtype, uint32_t B, uint32_t V, uint64_t ld,
                               const uint32_t* d_bitmask, const uint32_t* d_ids, const float* d_teacher, uint32_t K,
                               float temp, float* d_out_loss, float* d_out_lse, const float* d_grad_loss,
                               void* d_out_grad, uint64_t ld_grad) {
  return cg_distill_loss_norm(c, d_logits, dtype, B, V, ld, d_bitmask, d_ids, d_teacher, K, temp, d_out_loss,
                              d_out_lse, nullptr, d_grad_loss, d_out_grad, ld_grad);
}

// the backward pass from either form of the normaliser
static int distill_backward(cg_ctx* c, const void* d_logits, int dtype, uint32_t B, uint32_t V, uint64_t ld,
                            const uint32_t* d_bitmask, const uint32_t* d_ids, const float* d_teacher, uint32_t K,
                            float temp, const float* d_lse, const float* d_norm, const float* d_grad_loss,
                            void* d_out_grad, uint64_t ld_grad) {
  using namespace cgk;
  const int rc = list_args(c, d_logits, dtype, B, V, ld, d_bitmask, d_ids, d_teacher, K, temp, d_grad_loss,
                           d_out_grad, ld_grad);
  if (rc != CG_OK) return rc;
  if ((B && ((!d_lse && !d_norm) || !d_out_grad)) || !aligned4(d_lse) || !aligned4(d_norm)) return CG_E_ARG;
  const DistillArgs a{d_logits, ld,     d_bitmask, V,       0,       d_ids,       d_teacher,  K,       temp,
                      d_lse,    d_norm, nullptr,   nullptr, nullptr, d_grad_loss, d_out_grad, ld_grad, nullptr};
  return distill(c, "cg_distill_grad", a, dtype, B, false);
}

extern "C" int cg_distill_grad(cg_ctx* c, const void* d_logits, int dtype, uint32_t B, uint32_t V, uint64_t ld,
                               const uint32_t* d_bitmask, const uint32_t* d_ids, const float* d_teacher, uint32_t K,
                               float temp, const float* d_lse, const float* d_grad_loss, void* d_out_grad,
                               uint64_t ld_grad) {
  return distill_backward(c, d_logits, dtype, B, V, ld, d_bitmask, d_ids, d_teacher, K, temp, d_lse, nullptr,
                          d_grad_loss, d_out_grad, ld_grad);
}

extern "C" int cg_distill_grad_norm(cg_ctx* c, const void* d_logits, int dtype, uint32_t B, uint32_t V, uint64_t ld,
                                    const uint32_t* d_bitmask, const uint32_t* d_ids, const float* d_teacher,
                                    uint32_t K, float temp, const float* d_norm, const float* d_grad_loss,
                                    void* d_out_grad, uint64_t ld_grad) {
  return distill_backward(c, d_logits, dtype, B, V, ld, d_bitmask, d_ids, d_teacher, K, temp, nullptr, d_norm,
                          d_grad_loss, d_out_grad, ld_grad);
}
