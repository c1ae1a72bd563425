// The n best allowed tokens of each row with their log-probabilities
// (cg_top_logprobs).
//
// The row is held on chip by a cluster (logit_row.cuh).  With N blocks, each
// finds a bound that ceil(n / N) of its threads' maxima reach; at least n
// tokens lie at or above the least of these bounds, and little more (a thread
// rarely holds two of the best).  Those are gathered by rank 0 and put in order
// by (logit, lower id).  Where ties or small clusters make the gathered list
// overflow, the n-th largest logit comes from histograms over the cluster, the
// last ids among its ties from a second selection, and exactly n are gathered.
#include "logit_row.cuh"

namespace cgk {
namespace {

using namespace row;

struct TopArgs {
  const void* logits;
  uint64_t ld;
  const uint32_t* bitmask;
  uint32_t V, W, n;
  uint32_t* out_ids;
  float* out_lp;
  float* out_lse;
};

template <bool BF16, int NV>
__global__ void __launch_bounds__(kThreads, NV <= 8 ? 2 : 1) top_kernel(const TopArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  using F = Fmt<BF16>;
  griddep_launch_dependents();
  const uint32_t n = cluster_size(), rank = cluster_rank(), b = blockIdx.x / n, tid = threadIdx.x;
  if (tid == 0) s.n_list = s.n_local = 0;
  if (n > 1) cluster_arrive();  // this block's shared memory is ready for the others
  griddep_wait();
  Held<BF16, NV> h(Row<BF16>(a.logits, a.ld, a.bitmask, a.W, a.V, b));
  h.load();
  uint32_t low;
  h.find_max(s, low);
  const float sum = h.sum_exps(s, kLog2e);
  uint32_t cut_key = h.share_cut((a.n + n - 1) / n, low);
  if (n > 1) cluster_wait();
  exchange(s, n, rank, h.m, sum, cut_key);
  float M, S;
  merge(s, n, kLog2e, M, S, cut_key);
  uint32_t found = 0;
  bool waiting = false;
  if (M > -INFINITY) {
    const float cut = cut_key >= kKeyLowest ? fkey_inv(cut_key) : -FLT_MAX;
    h.collect(s, cut, true);
    cluster_sync(n);
    found = s.n_list;
    if (rank != 0) {
      if (tid == 0) s.total = ld_remote(at_rank(&s.n_list, 0));
      __syncthreads();
      found = s.total;
    }
    waiting = n > 1;
    if (waiting) {
      cluster_arrive();  // rank 0's count has been read
      if (rank != 0 || found > kListCap) {
        cluster_wait();
        waiting = false;
      }
    }
    if (found > kListCap) {
      h.collect(s, cut, false);
      __syncthreads();
      uint32_t level = 0;
      unsigned long long above;
      // the n-th largest logit: a key whose upper set holds n tokens
      const uint32_t tau = select_key(s, n, [&](auto f) { h.each(s, cut, [&](uint32_t, float x) { f(F::key(x), 1ull); }); },
                                      F::key(cut), F::key(M), a.n, level, above);
      // of the tokens with that key, the lowest ids (as many as are missing)
      const uint32_t first = ~(a.V - 1u);
      const uint32_t last = select_key(
          s, n, [&](auto f) { h.each(s, cut, [&](uint32_t t, float x) { if (F::key(x) == tau) f(~t, 1ull); }); }, first,
          ~0u, a.n - above, level, above);
      if (rank == 0 && tid == 0) s.n_list = 0;
      cluster_sync(n);
      const uint32_t count = at_rank(&s.n_list, 0), list = at_rank(s.list, 0);
      h.each(s, cut, [&](uint32_t t, float x) {
        const uint32_t key = F::key(x);
        if (key > tau || (key == tau && ~t >= last)) {
          const uint32_t at = add_remote(count, 1u);
          if (at < kListCap) st_remote(list + at * 8, pack_best(x, t));
        }
      });
      cluster_sync(n);
      found = s.n_list;
    }
    if (rank != 0) return;  // rank 0 reads nobody else's shared memory from here on
  } else if (rank != 0) {
    return;
  }
  const float log_s = logf(S);
  uint32_t* ids = a.out_ids + size_t(b) * a.n;
  float* lps = a.out_lp + size_t(b) * a.n;
  auto write = [&](uint32_t i, unsigned long long e) {
    ids[i] = best_id(e);
    lps[i] = (fkey_inv(uint32_t(e >> 32)) - M) - log_s;
  };
  if (found <= kPairCap) {
    // an entry's place is the number of entries above it; parts of the block
    // compare with parts of the list
    uint32_t C = 32;
    while (C < found) C <<= 1;
    const uint32_t i = tid & (C - 1), part = tid / C, parts = kThreads / C;
    uint32_t* place = reinterpret_cast<uint32_t*>(s.local);
    if (tid < C) place[tid] = 0;
    __syncthreads();
    const unsigned long long e = i < found ? s.list[i] : 0ull;
    if (i < found) {
      uint32_t before = 0;
      for (uint32_t j = part; j < found; j += parts) before += s.list[j] > e;
      if (before) atomicAdd(place + i, before);
    }
    __syncthreads();
    if (part == 0 && i < found && place[i] < a.n) write(place[i], e);
  } else {
    sort_desc(s.list, found);
    for (uint32_t i = tid; i < min(found, a.n); i += kThreads) write(i, s.list[i]);
  }
  for (uint32_t i = found + tid; i < a.n; i += kThreads) {
    ids[i] = CG_NO_TOKEN;
    lps[i] = -INFINITY;
  }
  if (a.out_lse && tid == 0) a.out_lse[b] = M > -INFINITY ? M + log_s : -INFINITY;
  if (waiting) cluster_wait();  // before this block's count goes away
}

template <bool BF16>
cudaError_t launch_top(int device, uint32_t B, const TopArgs& a, cudaStream_t stream) {
  const Plan plan = plan_row(BF16, a.V, B, rows_on_grid(a.logits, BF16 ? CG_BF16 : CG_F32, a.ld));
  return with_nv<BF16>(plan.nv, [&](auto nv) {
    return launch_clusters<top_kernel<BF16, decltype(nv)::value>>(device, B, plan.n, sizeof(Shared), stream, a);
  });
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
  const TopArgs a{d_logits, ld, d_bitmask, V, v.t.W, n, d_out_ids, d_out_logprobs, d_out_lse};
  const int dev = ctx_device(c);
  const cudaError_t e =
      dtype == CG_BF16 ? launch_top<true>(dev, B, a, v.stream) : launch_top<false>(dev, B, a, v.stream);
  return e == cudaSuccess ? CG_OK : CG_E_CUDA;
}
