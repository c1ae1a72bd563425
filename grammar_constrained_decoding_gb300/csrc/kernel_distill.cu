// Distillation from a teacher's top logits, forward and backward
// (cg_distill_loss, cg_distill_grad).
//
//   loss = T^2 sum_k q_k (log q_k - log p[id_k]),  log p_v = (x_v - m) / T - log S,
//   dloss/dx_v = T (p_v - sum_{k: id_k = v} q_k),
// q the softmax of the teacher's listed logits / T, S = sum exp((x - m) / T).
//
// With a gradient the row is held on chip by a cluster (logit_row.cuh): the logits are
// read from memory once and the gradient is written once from the registers.  Every
// gradient is written as T w p_v first; the block that wrote a listed token's
// writes it over after a block barrier.  All reads of the row's logits, the
// listed ones by every block included, come before the cluster meets, all
// writes after it, so the gradient may take the logits' place.  Without a gradient the
// rows stream (below).
//
// What bounds them, of 2048 x 128256 bf16: the loss alone 83.6 us, 6.3 TB/s, the memory;
// the gradient from the kept normaliser 178.9 us, 5.9 TB/s of reads and writes, nearly
// so; loss and gradient 221.5 us, 4.7 TB/s: a block waits for its part, then for the
// cluster's sums, then writes, and three of them on an SM do not always cover one
// another.
#include "logit_row.cuh"

namespace cgk {
namespace {

using namespace row;

// groups of a thread for many rows: 64 KB parts, three blocks an SM; fewer, longer
// parts cost fewer exchanges and list look-ups.  Loss and gradient of 2048 x 128256: 8
// groups 270.6 us, 12 237.9, 16 224.6, 24 274.0
constexpr uint32_t kFull = 16;
constexpr size_t kThird = 75 * 1024;  // shared memory of a block of three on an SM

// The teacher's list in shared memory, K entries
struct List {
  uint32_t* id;     // listed ids that count, CG_NO_TOKEN for the others
  float* t;         // teacher logits
  float* x;         // the student's logits there
  uint32_t* hash;   // slots of the repeated-id check, more than twice K
  uint32_t slots;
  __host__ __device__ static uint32_t slots_of(uint32_t K) {
    uint32_t s = 4;
    while (s < 2 * K) s <<= 1;
    return s;
  }
  __host__ __device__ static size_t bytes(uint32_t K) { return (size_t(K) * 12 + size_t(slots_of(K)) * 4 + 15) & ~size_t(15); }
  __device__ List(void* at, uint32_t K)
      : id(static_cast<uint32_t*>(at)), t(reinterpret_cast<float*>(id + K)), x(t + K),
        hash(reinterpret_cast<uint32_t*>(x + K)), slots(slots_of(K)) {}
};
struct DistillShared : Meet {
  uint32_t repeated;
};

struct DistillArgs {
  const void* logits;
  uint64_t ld;
  const uint32_t* bitmask;
  uint32_t V, W;
  const uint32_t* ids;
  const float* teacher;
  uint32_t K;
  float temp;
  const float* lse_in;   // backward alone: the kept normaliser
  float* loss;
  float* lse_out;
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
__device__ __forceinline__ void store_loss(const DistillArgs& a, uint32_t b, float loss, float M, float log_s) {
  a.loss[b] = loss;
  if (a.lse_out) a.lse_out[b] = M > -INFINITY ? __fdiv_rn(M, a.temp) + log_s : -INFINITY;
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

template <bool BF16, bool LOSS>
__global__ void __launch_bounds__(kThreads, 3) distill_kernel(const DistillArgs a, uint32_t nv) {
  extern __shared__ __align__(16) unsigned char smem[];
  DistillShared& s = *reinterpret_cast<DistillShared*>(smem);
  const List l(smem + sizeof(DistillShared), a.K);
  griddep_launch_dependents();
  const uint32_t n = cluster_size(), rank = cluster_rank(), b = blockIdx.x / n, tid = threadIdx.x, K = a.K;
  begin(s);
  Held<BF16> h(Row<BF16>(a.logits, a.ld, a.bitmask, a.W, a.V, b), nv, 
               smem + sizeof(DistillShared) + List::bytes(K));
  griddep_wait();
  h.start(s, false);
  may_send();
  const float T = a.temp, c = exp_scale(T);
  // the teacher's list
  const uint32_t slots = l.slots;
  for (uint32_t i = tid; i < slots; i += kThreads) l.hash[i] = CG_NO_TOKEN;
  if (tid == 0) s.repeated = 0;
  float tm = -INFINITY;
  for (uint32_t k = tid; k < K; k += kThreads) {
    uint32_t id = a.ids[size_t(b) * K + k];
    const float t = teacher_logit(a.teacher[size_t(b) * K + k]);
    float x = -INFINITY;
    if (id < a.V) x = h.r.at(id);
    else if (id != CG_NO_TOKEN && rank == 0) record_error(a.status, CG_DEV_BAD_TOKEN);
    if (!(x > -INFINITY) || !(t > -INFINITY)) id = CG_NO_TOKEN;
    l.id[k] = id;
    l.x[k] = x;
    l.t[k] = t;
    if (id != CG_NO_TOKEN) tm = fmaxf(tm, t);
  }
  tm = block_max(tm, s.red_f);
  const bool listed = tm > -INFINITY;
  float ts = 0.f;
  for (uint32_t k = tid; k < K; k += kThreads) {
    const uint32_t id = l.id[k];
    if (id == CG_NO_TOKEN) continue;
    ts += ex2((l.t[k] - tm) * c);
    // repeated ids: every id claims a slot (more slots than ids), the second
    // of equal ones finds it taken by itself
    for (uint32_t at = (id * 0x9E3779B1u) & (slots - 1);; at = (at + 1) & (slots - 1)) {
      const uint32_t old = atomicCAS(l.hash + at, CG_NO_TOKEN, id);
      if (old == CG_NO_TOKEN) break;
      if (old == id) {
        s.repeated = 1;
        break;
      }
    }
  }
  __syncthreads();
  ts = block_sum(ts, s.red_f);
  __syncthreads();

  float M = 0.f, S = 1.f;  // p = exp2((x - M) c) / S
  if (LOSS) {
    if (!h.template take<true>(s, c)) record_error(a.status, CG_DEV_TIMEOUT);
    ready_others();
    h.publish(s, c);
    if (tid < 32) {
      const bool ok = wait_sent(&s.bar_rec);
      float m, sum;
      merge(s.rec, n * kWarps, c, m, sum);
      if (tid == 0) {
        s.M = m;
        s.S = sum;
        if (!ok) record_error(a.status, CG_DEV_TIMEOUT);
      }
    }
    __syncthreads();
    M = s.M;
    S = s.S;
    if (rank == 0) {
      float part = 0.f;
      const float log_ts = logf(ts), log_s = logf(S);
      for (uint32_t k = tid; k < K; k += kThreads)
        if (l.id[k] != CG_NO_TOKEN) part += loss_term(l.t[k] - tm, ts, log_ts, l.x[k] - M, log_s, c, T);
      __syncthreads();
      part = block_sum(part, s.red_f);
      if (tid == 0) store_loss(a, b, listed ? T * T * part : 0.f, M, log_s);
    }
  } else {
    M = a.lse_in[b] * T;  // p = exp((x - lse T) / T)
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
  if (!listed) return;
  __syncthreads();
  const bool repeated = s.repeated != 0;
  for (uint32_t k = tid; k < K; k += kThreads) {
    const uint32_t id = l.id[k];
    if (id == CG_NO_TOKEN) continue;
    const uint32_t g = (id + h.r.a) / Fmt<BF16>::E;
    if ((g / kThreads) % n != rank) continue;
    float q = ex2((l.t[k] - tm) * c);
    if (repeated) {  // every entry of the id writes the same sum
      q = 0.f;
      for (uint32_t j = 0; j < K; ++j)
        if (l.id[j] == id) q += ex2((l.t[j] - tm) * c);
    }
    store_grad<BF16>(row, id, scale * (__fdiv_rn(ex2((l.x[k] - M) * c), S) - __fdiv_rn(q, ts)));
  }
}

// ---- the loss alone ---------------------------------------------------------------------
//
// Nothing of a row is needed twice, so it streams: a cluster takes rows in turn, its
// blocks the row's chunks in turn, through a ring of chunks that one warp keeps
// filling across the rows' ends.  The warps send their maxima and sums of row i to
// block i mod n, where one more warp has read the row's list meanwhile and finishes
// the row.
// Few barriers and many loads at once: 8 groups of a thread a chunk.  Of 2048 x 128256
// bf16, masked too: 16 warps x 2 groups x 6 chunks 93.7 and 108.8 us, 8 x 4 x 6 83.9 and
// 95.5, 8 x 8 x 3 83.6 and 86.2, three blocks of 8 x 4 x 4 an SM 86.8 and 90.8.
constexpr uint32_t kStreamWarps = 8;   // that take chunks
constexpr uint32_t kPer = 8;           // groups of a thread in a chunk
constexpr uint32_t kRing = 3;          // chunks on their way or being taken, at most
constexpr uint32_t kStreamBlocks = 2;  // an SM
constexpr uint32_t kStreamSlots = kStreamBlocks * 152;
constexpr size_t kStreamSmem = 113 * 1024;  // of a block
constexpr uint32_t kStreamThreads = (kStreamWarps + 2) * 32;
constexpr uint32_t kChunkGroups = kStreamWarps * 32 * kPer;
// Few rows are split over clusters of 2, 4 or 8 blocks as long as all are resident
// together (36 clusters of 8, 74 of 4).  Microseconds of B x 128256 bf16 by cluster
// size, at 16 warps x 2 groups x 6 chunks:
//   B      1     2     4     8    16
//   512  30.3  31.4  30.8  37.1  66.5
//   128  16.0  11.4  12.1  13.6
//   64   13.1  10.4   8.2   9.1
//   32          8.1   7.1   6.0
//   4                 5.4   4.4   4.3
constexpr uint32_t kStreamCluster = 8, kStreamSplit = 288;

struct StreamShared {
  uint64_t full[kRing], empty[kRing];
  uint64_t bar_rec[2];                  // by turns of this block's rows
  uint64_t done[kStreamCluster][2];        // ... of each block's: their records have been read
  Record rec[2][kStreamCluster * kStreamWarps];
};
// ... then the list's logits, teacher's and student's, and the ring: its chunks, their bits
size_t stream_smem(uint32_t K, uint32_t ring, uint32_t bits) {
  return sizeof(StreamShared) + ((size_t(K) * 8 + 15) & ~size_t(15)) + size_t(ring) * (kChunkGroups * 16 + bits);
}

template <bool BF16>
__global__ void __launch_bounds__(kStreamThreads, kStreamBlocks) stream_loss_kernel(const DistillArgs a, uint32_t B,
                                                                                       uint32_t chunks) {
  extern __shared__ __align__(16) unsigned char smem[];
  using F = Fmt<BF16>;
  constexpr uint32_t kBytes = kChunkGroups * 16, kBits = kChunkGroups * F::E / 8;
  StreamShared& s = *reinterpret_cast<StreamShared*>(smem);
  static_assert(sizeof(StreamShared) % 16 == 0, "the list and the ring lie behind it");
  float* list_t = reinterpret_cast<float*>(smem + sizeof(StreamShared));  // -inf where an entry does not count
  float* list_x = list_t + a.K;
  unsigned char* ring = smem + sizeof(StreamShared) + ((a.K * 8 + 15) & ~15u);
  unsigned char* ring_bits = ring + chunks * kBytes;
  griddep_launch_dependents();
  const uint32_t n = cluster_size(), rank = cluster_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t first = blockIdx.x / n, step = gridDim.x / n;
  if (tid == 0) {
    for (uint32_t i = 0; i < chunks; ++i) {
      mbar_init(s.full + i, 1);
      mbar_init(s.empty + i, kStreamWarps);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(s.bar_rec + i, 1);
      for (uint32_t r = 0; r < kStreamCluster; ++r) mbar_init(&s.done[r][i], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  may_send();
  griddep_wait();
  const float T = a.temp, c = exp_scale(T);
  auto row = [&](uint32_t b) { return Row<BF16>(a.logits, a.ld, a.bitmask, a.W, a.V, b); };
  auto groups = [&](const Row<BF16>& r) { return (a.V + r.a + F::E - 1) / F::E; };
  auto copied = [&](const Row<BF16>& r) {  // the chunks' bits come by copies
    return r.mask && r.a == 0 && ((reinterpret_cast<uintptr_t>(r.mask) | (a.W * 4u)) & 15u) == 0;
  };
  bool ok = true;
  if (warp == kStreamWarps) {  // fills the ring
    if (lane == 0) {
      const uint64_t policy = evict_first_policy();
      uint32_t slot = 0, turn = 0;
      for (uint32_t b = first; ok && b < B; b += step) {
        const Row<BF16> r = row(b);
        const uint32_t lo = r.first_whole(), hi = r.end_whole(), end = groups(r);
        const bool bits = copied(r);
        for (uint32_t g = rank * kChunkGroups; g < end; g += n * kChunkGroups) {
          if (turn && !(ok = mbar_wait(s.empty + slot, (turn - 1) & 1u))) break;
          const uint32_t from = max(g, lo), to = min(g + kChunkGroups, hi), off = g * F::E / 8;
          const uint32_t bytes = to > from ? (to - from) * 16u : 0u, more = bits ? min(kBits, a.W * 4u - off) : 0u;
          mbar_expect_tx(s.full + slot, bytes + more);
          if (bytes)
            bulk_g2s_hint(ring + slot * kBytes + (from - g) * 16, r.base + size_t(from) * 16, bytes, s.full + slot, policy);
          if (more) bulk_g2s(ring_bits + slot * kBits, r.mask + off, more, s.full + slot);
          if (++slot == chunks) slot = 0, ++turn;
        }
      }
      for (uint32_t i = 0; i < chunks; ++i)  // all have landed when the block ends, whatever its other warps did
        if (turn || i < slot) ok = mbar_wait(s.full + i, (i < slot ? turn : turn - 1) & 1u) && ok;
    }
    __syncwarp();
    ready_others();
  } else if (warp < kStreamWarps) {
    uint32_t slot = 0, turn = 0, i = 0;
    for (uint32_t b = first; ok && b < B; b += step, ++i) {
      const Row<BF16> r = row(b);
      const uint32_t lo = r.first_whole(), hi = r.end_whole(), end = groups(r);
      const bool bits = copied(r);
      float tm = -INFINITY;
      float2 acc = {};
#pragma unroll 1
      for (uint32_t g = rank * kChunkGroups; g < end; g += n * kChunkGroups) {
        uint32_t allowed[kPer];
        if (r.mask && !bits) {
#pragma unroll
          for (uint32_t k = 0; k < kPer; ++k) {
            const uint32_t own = g + k * kStreamWarps * 32 + tid;
            allowed[k] = own < end ? r.mask_bits(int(own * F::E) - int(r.a)) : 0u;
          }
        }
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(s.full + slot, turn & 1u));
        if (!ok) break;
        uint4 v[kPer];
        const uint4* part = reinterpret_cast<const uint4*>(ring + slot * kBytes) + tid;
#pragma unroll
        for (uint32_t k = 0; k < kPer; ++k) v[k] = part[k * kStreamWarps * 32];
        if (bits) {
          const unsigned char* p = ring_bits + slot * kBits + (BF16 ? tid : tid / 2);
#pragma unroll
          for (uint32_t k = 0; k < kPer; ++k)
            allowed[k] = uint32_t(p[k * (kBits / kPer)]) >> (BF16 ? 0u : (tid & 1u) * 4u);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(s.empty + slot);
        if (++slot == chunks) slot = 0, ++turn;
        if (g < lo || g + kChunkGroups > hi) {  // groups that the copies do not bring
#pragma unroll
          for (uint32_t k = 0; k < kPer; ++k) {
            const uint32_t own = g + k * kStreamWarps * 32 + tid;
            if (own < lo || own >= hi) v[k] = r.edge(own);
          }
        }
        if (r.mask) {
#pragma unroll
          for (uint32_t k = 0; k < kPer; ++k) v[k] = r.masked(v[k], allowed[k]);
        }
        float t = groups_max_nan<BF16, kPer>(v);
        if (fkey(t) >= kKeyInf) {
#pragma unroll
          for (uint32_t k = 0; k < kPer; ++k) v[k] = clean_group<BF16>(v[k]);
          t = groups_max_nan<BF16, kPer>(v);
        }
        add_groups<BF16, kPer>(v, t, c, tm, acc);
      }
      if (i == 0) ready_others();
      if (!ok) break;
      const unsigned long long rec = warp_record(tm, acc.x + acc.y, c);
      const uint32_t home = i % n, use = i / n;  // of the home's records, by turns in two buffers
      if (lane == 0) {
        if (use >= 2) ok = wait_sent(&s.done[home][use & 1u], (use / 2 - 1) & 1u);
        send(at_rank(&s.rec[use & 1u][rank * kStreamWarps + warp], home), rec, at_rank(s.bar_rec + (use & 1u), home));
      }
      ok = __all_sync(0xFFFFFFFFu, ok);
    }
  } else {  // finishes the rows that are this block's
    const uint32_t K = a.K, rows = (B - first + step - 1) / step;
    ready_others();
    for (uint32_t i = rank; i < rows; i += n) {
      const uint32_t b = first + i * step, use = i / n;
      const Row<BF16> r = row(b);
      if (lane == 0) mbar_expect_tx(s.bar_rec + (use & 1u), n * kStreamWarps * uint32_t(sizeof(Record)));
      float tm = -INFINITY;
#pragma unroll 4
      for (uint32_t k = lane; k < K; k += 32) {
        const uint32_t id = a.ids[size_t(b) * K + k];
        const float t = teacher_logit(a.teacher[size_t(b) * K + k]);
        const float x = id < a.V ? r.at(id) : -INFINITY;
        if (id >= a.V && id != CG_NO_TOKEN) record_error(a.status, CG_DEV_BAD_TOKEN);
        const bool counts = x > -INFINITY && t > -INFINITY;
        list_x[k] = x;
        list_t[k] = counts ? t : -INFINITY;
        if (counts) tm = fmaxf(tm, t);
      }
      tm = warp_reduce(tm, MaxOp());
      const bool listed = tm > -INFINITY;
      float ts = 0.f;
      for (uint32_t k = lane; k < K; k += 32)
        if (list_t[k] > -INFINITY) ts += ex2((list_t[k] - tm) * c);
      ts = warp_reduce(ts, SumOp());
      ok = __all_sync(0xFFFFFFFFu, wait_sent(s.bar_rec + (use & 1u), (use / 2) & 1u));
      if (!ok) break;
      float M, S;
      merge(s.rec[use & 1u], n * kStreamWarps, c, M, S);
      __syncwarp();
      if (i + 2 * n < rows && lane < n) {  // the buffer is used again
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                         at_rank(&s.done[rank][use & 1u], lane))
                     : "memory");
      }
      const float log_ts = logf(ts), log_s = logf(S);
      float part = 0.f;
      for (uint32_t k = lane; k < K; k += 32)
        if (list_t[k] > -INFINITY) part += loss_term(list_t[k] - tm, ts, log_ts, list_x[k] - M, log_s, c, T);
      part = warp_reduce(part, SumOp());
      if (lane == 0) store_loss(a, b, listed ? T * T * part : 0.f, M, log_s);
    }
  }
  if (!ok) record_error(a.status, CG_DEV_TIMEOUT);
  __syncwarp();
  cluster_sync(n);  // what others send arrives, and so do their signals
}

template <bool BF16>
cudaError_t launch_stream(int device, uint32_t B, const DistillArgs& a, cudaStream_t stream) {
  const uint32_t chunks = (a.V / Fmt<BF16>::E + kChunkGroups) / kChunkGroups;
  uint32_t n = 1;
  while (n < kStreamCluster && 2 * n <= chunks && uint64_t(B) * 2 * n <= kStreamSplit) n *= 2;
  const uint32_t bits = a.bitmask ? kChunkGroups * Fmt<BF16>::E / 8 : 0;
  uint32_t ring = kRing;
  while (stream_smem(a.K, ring, bits) > kStreamSmem) --ring;
  return launch_clusters<stream_loss_kernel<BF16>>(device, n == 1 && B > kStreamSlots ? kStreamSlots : B, n, kStreamThreads,
                                                  stream_smem(a.K, ring, bits), stream, a, B, ring);
}

template <bool BF16>
cudaError_t launch_distill(int device, uint32_t B, const DistillArgs& a, bool loss, cudaStream_t stream) {
  if (!a.grad) return launch_stream<BF16>(device, B, a, stream);
  const size_t fixed = sizeof(DistillShared) + List::bytes(a.K);
  uint32_t full = kFull;
  while (full > 1 && fixed + part_bytes(BF16, full, a.bitmask) > kThird) --full;
  const Plan plan = plan_row(BF16, a.V, B, rows_on_grid(a.logits, BF16 ? CG_BF16 : CG_F32, a.ld), full);
  const size_t smem = fixed + part_bytes(BF16, plan.nv, a.bitmask);
  return loss ? launch_clusters<distill_kernel<BF16, true>>(device, B, plan.n, kThreads, smem, stream, a, plan.nv)
              : launch_clusters<distill_kernel<BF16, false>>(device, B, plan.n, kThreads, smem, stream, a, plan.nv);
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

extern "C" int cg_distill_loss(cg_ctx* c, const void* d_logits, int dtype, uint32_t B, uint32_t V, uint64_t ld,
                               const uint32_t* d_bitmask, const uint32_t* d_ids, const float* d_teacher, uint32_t K,
                               float temp, float* d_out_loss, float* d_out_lse, const float* d_grad_loss,
                               void* d_out_grad, uint64_t ld_grad) {
  using namespace cgk;
  const int rc = list_args(c, d_logits, dtype, B, V, ld, d_bitmask, d_ids, d_teacher, K, temp, d_grad_loss,
                           d_out_grad, ld_grad);
  if (rc != CG_OK) return rc;
  if ((B && !d_out_loss) || !aligned4(d_out_loss) || !aligned4(d_out_lse)) return CG_E_ARG;
  const DistillArgs a{d_logits, ld, d_bitmask, V, 0, d_ids, d_teacher, K, temp, nullptr, d_out_loss, d_out_lse,
                      d_grad_loss, d_out_grad, ld_grad, nullptr};
  return distill(c, "cg_distill_loss", a, dtype, B, true);
}

extern "C" int cg_distill_grad(cg_ctx* c, const void* d_logits, int dtype, uint32_t B, uint32_t V, uint64_t ld,
                               const uint32_t* d_bitmask, const uint32_t* d_ids, const float* d_teacher, uint32_t K,
                               float temp, const float* d_lse, const float* d_grad_loss, void* d_out_grad,
                               uint64_t ld_grad) {
  using namespace cgk;
  const int rc = list_args(c, d_logits, dtype, B, V, ld, d_bitmask, d_ids, d_teacher, K, temp, d_grad_loss,
                           d_out_grad, ld_grad);
  if (rc != CG_OK) return rc;
  if ((B && (!d_lse || !d_out_grad)) || !aligned4(d_lse)) return CG_E_ARG;
  const DistillArgs a{d_logits, ld, d_bitmask, V, 0, d_ids, d_teacher, K, temp, d_lse, nullptr, nullptr,
                      d_grad_loss, d_out_grad, ld_grad, nullptr};
  return distill(c, "cg_distill_grad", a, dtype, B, false);
}
