// The n best allowed tokens of each row with their log-probabilities
// (cg_top_logprobs).
//
// The row is held on chip by a cluster (logit_row.cuh).  At least n tokens lie at or
// above the n-th largest of the maxima of any groups of tokens, and little more for
// many groups: the warps publish the maxima of groups of their lanes, the tokens at
// or above that bound are gathered by rank 0 and put in order by (logit, lower id),
// up to 256 of them by counting for each how many are above it, an entry a thread,
// more by a bitonic network.  Where ties make the gathered list overflow, rank 0
// reads the row again by itself: the n-th largest logit and the last ids among its
// ties by radix selection, then exactly n entries.
//
// What bounds it: the chain of a block, not the memory.  2048 x 32000 bf16, n = 64,
// takes 69.9 us (1.9 TB/s); the same rows read and summed alone take 27.  A block's
// part arrives, is summed, the bounds cross the cluster, the entries cross it again,
// and rank 0 ranks them while its three neighbours on the SM do their own: n = 5 52.8,
// n = 20 57.6 us, so the ordering of 64 costs 12.  Past about 200 entries the bound is
// loose and the network sorts: n = 256 148 us.  Near the list's capacity the ties of
// bf16 logits overflow it, and rank 0 reads the row again: n = 1024 4651 us.
#include "logit_row.cuh"

namespace cgk {
namespace {

using namespace row;

// groups of a thread for many rows.  2048 x 32000, n = 64: 6 groups (three blocks a
// row) 94.8 us, 8 (two) 69.4, 16 (one, fewer on an SM) 73.2
constexpr uint32_t kFull = 8;

struct TopArgs {
  const void* logits;
  uint64_t ld;
  const uint32_t* bitmask;
  uint32_t V, W, n;
  uint32_t* out_ids;
  float* out_lp;
  float* out_lse;
  uint32_t* status;
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 4) top_kernel(const TopArgs a, uint32_t nv) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  using F = Fmt<BF16>;
  griddep_launch_dependents();
  const uint32_t n = cluster_size(), rank = cluster_rank(), b = blockIdx.x / n, tid = threadIdx.x;
  begin(s);
  Held<BF16> h(Row<BF16>(a.logits, a.ld, a.bitmask, a.W, a.V, b), nv, smem + sizeof(Shared));
  griddep_wait();
  h.start(s, true);
  may_send();
  if (!h.template take<true>(s, kLog2e)) {
    s.late = 1;
    record_error(a.status, CG_DEV_TIMEOUT);
  }
  bool tight;
  const uint32_t per_warp = bounds_per_warp(a.n, n, tight);
  const unsigned long long rec = h.record(kLog2e);
  ready_others();
  h.publish(s, rec, per_warp);
  if (tid < 32) {
    const bool ok = wait_sent(&s.bar_rec);
    float m, sum, rest;
    merge(s.rec, n * kWarps, kLog2e, m, sum, rest);
    const uint32_t key = per_warp ? bound_key(s, n * kWarps * per_warp, a.n) : 0u;
    if (tid == 0) {
      s.M = m;
      s.rest = rest;
      s.cut = key >= kKeyLowest ? fkey_inv(key) : -FLT_MAX;
      if (!ok) s.late = 1;
    }
  }
  __syncthreads();
  const float M = s.M;
  uint32_t found = 0;
  bool late = s.late != 0;
  const unsigned long long* list = s.list;
  if (M > -INFINITY && !late) {
    float from = s.cut;
    if (!tight && h.r.V > kStage) {  // a bound too low: the n-th largest itself, and its ties
      uint32_t level = 0;
      unsigned long long above;
      const uint32_t key = select_key(
          s, n, [&](auto f) { h.each(from, [&](uint32_t, float x) { f(fkey(x), 1ull); }); }, fkey(from), fkey(M), a.n,
          level, above);
      from = fkey_inv(key);
      cluster_sync(n);  // everybody has read the histograms: the list and the stage take their place
    }
    h.template gather<false>(s, from, false, 0.f, 0.f);
    if (rank != 0) return;  // its entries are with rank 0
    float none;
    bool whole = true;
    late = !h.tallied(s, found, whole, none) || !h.listed(s, found);
    if (late) found = 0;
    if (found > kListCap || !whole) {
      uint32_t level = 0;
      unsigned long long above;
      // the n-th largest logit: a key whose upper set holds n tokens
      const uint32_t tau = select_key(
          s, 1, [&](auto f) { each_of_row(h.r, [&](uint32_t, float x) { f(F::key(x), 1ull); }); }, F::key(-FLT_MAX),
          F::key(M), a.n, level, above);
      // of the tokens with that key, the lowest ids (as many as are missing)
      unsigned long long skip;
      const uint32_t last = select_key(
          s, 1, [&](auto f) { each_of_row(h.r, [&](uint32_t t, float x) { if (F::key(x) == tau) f(~t, 1ull); }); },
          ~(a.V - 1u), ~0u, a.n - above, level, skip);
      if (tid == 0) s.n_list = 0;
      __syncthreads();
      each_of_row(h.r, [&](uint32_t t, float x) {
        const uint32_t key = F::key(x);
        if (key > tau || (key == tau && ~t >= last)) {
          const uint32_t at = atomicAdd(&s.n_list, 1u);
          if (at < kListCap) s.list[at] = pack_best(x, t);
        }
      });
      __syncthreads();
      found = min(s.n_list, kListCap);  // a.n, unless the row is written meanwhile
    } else if (found > kPairCap) {
      const uint32_t few = keep_few(s, found, list_bound(s, found, a.n));
      if (few <= kPairCap) {
        found = few;
        list = s.few;
      }
    }
  } else if (rank != 0) {
    if (late) leave_last(n);
    return;
  }
  if (late && tid == 0) record_error(a.status, CG_DEV_TIMEOUT);
  const float log_s = log1pf(s.rest);
  uint32_t* ids = a.out_ids + size_t(b) * a.n;
  float* lps = a.out_lp + size_t(b) * a.n;
  auto write = [&](uint32_t i, unsigned long long e) {
    ids[i] = best_id(e);
    lps[i] = (fkey_inv(uint32_t(e >> 32)) - M) - log_s;
  };
  if (found <= kPairCap) {
    place_entries<true>(s, list, found);
    if (tid < found && s.place[tid] < a.n) write(s.place[tid], list[tid]);
  } else {
    sort_desc(s.list, found);
    for (uint32_t i = tid; i < min(found, a.n); i += kThreads) write(i, s.list[i]);
  }
  for (uint32_t i = found + tid; i < a.n; i += kThreads) {
    ids[i] = CG_NO_TOKEN;
    lps[i] = -INFINITY;
  }
  if (a.out_lse && tid == 0) a.out_lse[b] = M > -INFINITY ? M + log_s : -INFINITY;
  if (late) leave_last(n);
}

// Self-test of leave_last: rank 0's wait runs out at once and it leaves last; the other
// blocks are kLag waits slower, meet once as a selection does, and send to rank 0's
// shared memory then.  out: how many of their messages and additions rank 0 saw.
constexpr uint32_t kTestCluster = 4, kLag = 2;
struct TestShared {
  uint64_t never, sent;
  unsigned long long slot[kTestCluster];
  uint32_t added;
};
__global__ void __launch_bounds__(64) leave_last_self_test_kernel(uint32_t* out, uint32_t* status) {
  extern __shared__ __align__(16) unsigned char smem[];
  TestShared& s = *reinterpret_cast<TestShared*>(smem);
  const uint32_t n = cluster_size(), rank = cluster_rank(), tid = threadIdx.x;
  griddep_wait();
  if (tid == 0) {
    mbar_init(&s.never, 1);
    mbar_init(&s.sent, 1);
    s.added = 0;
    for (uint32_t i = 0; i < kTestCluster; ++i) s.slot[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  cluster_sync(n);
  bool ok = true;
  for (uint32_t i = 0; i < (rank == 0 ? 1 : 1 + kLag); ++i) ok = __syncthreads_and(wait_sent(&s.never)) && ok;
  if (rank != 0) {
    cluster_sync(n);
    if (tid == 0) {
      add_remote(at_rank(&s.added, 0), 1u);
      send(at_rank(&s.slot[rank], 0), 1ull, at_rank(&s.sent, 0));
    }
    return;
  }
  if (!ok) leave_last(n);
  if (tid == 0) {
    mbar_expect_tx(&s.sent, (n - 1) * 8u);
    uint32_t seen = wait_sent(&s.sent) ? s.added : 0u;
    for (uint32_t i = 0; i < n; ++i) seen += uint32_t(s.slot[i]);
    *out = seen;
    if (!ok) record_error(status, CG_DEV_TIMEOUT);
  }
}

template <bool BF16>
cudaError_t launch_top(int device, uint32_t B, const TopArgs& a, cudaStream_t stream) {
  const Plan plan = plan_row(BF16, a.V, B, rows_on_grid(a.logits, BF16 ? CG_BF16 : CG_F32, a.ld), kFull);
  return launch_clusters<top_kernel<BF16>>(device, B, plan.n, kThreads,
                                           sizeof(Shared) + part_bytes(BF16, plan.nv, a.bitmask), stream, a, plan.nv);
}

}  // namespace
}  // namespace cgk

extern "C" int cg_top_logprobs(cg_ctx* c, const void* d_logits, int dtype, uint32_t B, uint32_t V, uint64_t ld,
                               const uint32_t* d_bitmask, uint32_t n, uint32_t* d_out_ids, float* d_out_logprobs,
                               float* d_out_lse) {
  using namespace cgk;
  if (!row_args_ok(c, d_logits, dtype, B, V, ld, d_bitmask)) return CG_E_ARG;
  if (n == 0 || (B && (!d_out_ids || !d_out_logprobs))) return CG_E_ARG;
  if (!aligned4(d_out_ids) || !aligned4(d_out_logprobs) || !aligned4(d_out_lse)) return CG_E_ARG;
  if (n > CG_TOP_MAX) return CG_E_LIMIT;
  if (B == 0) return CG_OK;
  DeviceGuard dg(ctx_device(c), "cg_top_logprobs");
  if (!dg.ok) return CG_E_CUDA;
  const CtxView v = ctx_view(c);
  const TopArgs a{d_logits, ld, d_bitmask, V, v.t.W, n, d_out_ids, d_out_logprobs, d_out_lse, v.t.status};
  const int dev = ctx_device(c);
  const cudaError_t e =
      dtype == CG_BF16 ? launch_top<true>(dev, B, a, v.stream) : launch_top<false>(dev, B, a, v.stream);
  return e == cudaSuccess ? CG_OK : CG_E_CUDA;
}

extern "C" int cg_self_test_cluster_timeout(cg_ctx* c, uint32_t* d_out) {
  using namespace cgk;
  if (!c || !d_out || !aligned4(d_out)) return CG_E_ARG;
  DeviceGuard dg(ctx_device(c), "cg_self_test_cluster_timeout");
  if (!dg.ok) return CG_E_CUDA;
  const CtxView v = ctx_view(c);
  const cudaError_t e = launch_clusters<leave_last_self_test_kernel>(ctx_device(c), 1, kTestCluster, 64,
                                                                     sizeof(TestShared), v.stream, d_out, v.t.status);
  return e == cudaSuccess ? CG_OK : CG_E_CUDA;
}
