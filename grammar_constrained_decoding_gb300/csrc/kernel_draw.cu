// Sampling with per-row temperature, top-k, top-p and min-p from given random
// numbers (cg_sample_rows).
//
// Per row, with d_t = x_t - max x and z_t = d_t / T: every cut keeps an upper
// set of the logits, so all of them together are one threshold on x -- the
// k-th largest logit (counted), the largest value whose upper set carries
// top_p of the kept mass (weighed), max x + T log(min_p) -- and the token is
// argmax z_t - log(-log u_t) over x_t >= threshold.
//
// The row is held on chip by a cluster (logit_row.cuh).  A lower bound of the
// threshold is known after one exchange between the blocks:
//   top-k  the k-th largest logit is at least the least of the blocks' bounds c,
//          each block having ceil(k / n) threads whose maximum is >= its c;
//   top-p  tokens more than D = log(V / ((1 - p) S)) nats below the maximum have
//          together less than (1 - p) S of the mass S, so the threshold lies
//          above them;
//   min-p  is the threshold itself.
// Only tokens at or above the bound matter from there on.  When they are few
// they are gathered by rank 0, which settles the cuts by comparing all pairs
// (the weight strictly above each token decides whether it stays); otherwise
// every block keeps its own list and the threshold comes from histograms over
// the cluster.
#include "logit_row.cuh"

namespace cgk {
namespace {

using namespace row;

constexpr float kULo = 2.3283064365386963e-10f;  // 2^-32
constexpr float kUHi = 0.999999940395355224609375f;  // 1 - 2^-24

struct DrawArgs {
  const void* logits;
  uint64_t ld;
  const uint32_t* bitmask;
  uint32_t V, W;
  const float* temp;
  const uint32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  uint64_t ld_u;
  uint32_t* out_tok;
  float* out_lp;
  uint32_t* status;
};

// top-k rows up to this k, and top-p rows whose nucleus holds at least this
// mass in units of the best token, are gathered; beyond it the list would
// overflow its kListCap entries as a rule
constexpr uint32_t kGatherK = 1024;
constexpr float kGatherMass = 256.f;

struct RowSettings {
  float T, Ts, p, floor_z;  // Ts: the softmax's temperature (1 for greedy rows)
  uint32_t k;               // 0: no top-k
  bool greedy;
};

// score of a kept token; false when min-p drops it
__device__ __forceinline__ bool score_of(const RowSettings& q, float d, const float* u, uint32_t t, float& score) {
  if (q.greedy) {
    score = 0.f;
    return true;
  }
  const float z = __fdiv_rn(d, q.T);
  if (!(z >= q.floor_z)) return false;
  score = z - logf(-logf(fminf(fmaxf(u[t], kULo), kUHi)));
  return true;
}

// Rank 0: the threshold key of list[0 .. c) under top-k and top-p.  kept_mass:
// the mass top-p is relative to when there is no top-k.
__device__ uint32_t list_threshold(Shared& s, uint32_t c, const RowSettings& q, float M, float scale, float S) {
  uint32_t tau = 0;
  if (c <= kPairCap) {
    // entry i against all: parts of the block take parts of the list
    uint32_t C = 32;
    while (C < c) C <<= 1;
    const uint32_t i = threadIdx.x & (C - 1), part = threadIdx.x / C, parts = kThreads / C;
    unsigned long long* above_n = s.hist[0];            // [C]
    unsigned long long* above_w = s.hist[0] + kPairCap; // [C]
    if (threadIdx.x < C) above_n[threadIdx.x] = above_w[threadIdx.x] = 0ull;
    __syncthreads();
    const uint32_t key = i < c ? uint32_t(s.list[i] >> 32) : 0u;
    const unsigned long long w = i < c ? mass_q(fkey_inv(key), M, scale) : 0ull;
    if (i < c) {
      unsigned long long nn = 0, ww = 0;
      for (uint32_t j = part; j < c; j += parts) {
        const uint32_t kj = uint32_t(s.list[j] >> 32);
        if (kj > key) {
          ++nn;
          ww += mass_q(fkey_inv(kj), M, scale);
        }
      }
      if (nn) atomicAdd(above_n + i, nn);
      if (ww) atomicAdd(above_w + i, ww);
    }
    __syncthreads();
    bool stays = i < c && (q.k == 0 || above_n[i] < q.k);
    if (q.p < 1.f) {
      unsigned long long kept = static_cast<unsigned long long>(double(S) * 1099511627776.0);
      if (q.k) kept = block_sum(stays && part == 0 ? w : 0ull, s.red64);
      unsigned long long target = static_cast<unsigned long long>(double(q.p) * double(kept));
      stays = stays && above_w[i] < (target ? target : 1ull);
    }
    // the least key that stays
    const uint32_t low = __reduce_min_sync(0xFFFFFFFFu, stays ? key : 0xFFFFFFFFu);
    if ((threadIdx.x & 31) == 0) s.red_min[threadIdx.x >> 5] = low;
    __syncthreads();
    return __reduce_min_sync(0xFFFFFFFFu, s.red_min[threadIdx.x & (kWarps - 1)]);
  }
  uint32_t level = 0;
  unsigned long long above;
  const uint32_t top = fkey(M);
  auto entries = [&](auto f) {
    for (uint32_t i = threadIdx.x; i < c; i += kThreads) f(uint32_t(s.list[i] >> 32));
  };
  if (q.k && q.k < c)
    tau = select_key(s, 1, [&](auto f) { entries([&](uint32_t key) { f(key, 1ull); }); }, kKeyLowest, top, q.k, level,
                     above);
  if (q.p < 1.f) {
    unsigned long long kept = static_cast<unsigned long long>(double(S) * 1099511627776.0);
    if (q.k) {
      unsigned long long w = 0;
      entries([&](uint32_t key) { w += key >= tau ? mass_q(fkey_inv(key), M, scale) : 0ull; });
      __syncthreads();
      kept = block_sum(w, s.red64);
      __syncthreads();
    }
    const unsigned long long target = static_cast<unsigned long long>(double(q.p) * double(kept));
    tau = select_key(s, 1, [&](auto f) { entries([&](uint32_t key) { f(key, mass_q(fkey_inv(key), M, scale)); }); },
                     max(tau, kKeyLowest), top, target ? target : 1ull, level, above);
  }
  return tau;
}

template <bool BF16, int NV>
__global__ void __launch_bounds__(kThreads, NV <= 8 ? 2 : 1) draw_kernel(const DrawArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  griddep_launch_dependents();
  const uint32_t n = cluster_size(), rank = cluster_rank(), b = blockIdx.x / n, tid = threadIdx.x;
  if (tid == 0) s.n_list = s.n_local = 0;
  if (n > 1) cluster_arrive();  // this block's shared memory is ready for the others
  griddep_wait();
  Held<BF16, NV> h(Row<BF16>(a.logits, a.ld, a.bitmask, a.W, a.V, b));
  h.load();
  RowSettings q;
  q.T = a.temp ? a.temp[b] : 1.f;
  q.k = a.top_k ? a.top_k[b] : 0u;
  const float p = a.top_p ? a.top_p[b] : 1.f, mp = a.min_p ? a.min_p[b] : 0.f;
  q.p = fmaxf(p, 0.f);
  q.greedy = q.T == 0.f;
  q.Ts = q.greedy ? 1.f : q.T;
  const bool bad = !(q.T >= 0.f && q.T <= FLT_MAX) || p != p || mp != mp || (!q.greedy && !a.u);
  if (q.k >= a.V) q.k = 0;
  q.floor_z = logf(fminf(fmaxf(mp, 0.f), 1.f));  // -inf for min_p = 0
  const float c = exp_scale(q.Ts);

  uint32_t low, cut_key = 0;
  h.find_max(s, low);
  const float sum = bad ? 0.f : h.sum_exps(s, c);
  if (q.k && !q.greedy) cut_key = h.share_cut((q.k + n - 1) / n, low);
  if (n > 1) cluster_wait();
  exchange(s, n, rank, h.m, sum, cut_key);
  float M, S;
  merge(s, n, c, M, S, cut_key);
  const float* u = a.u + size_t(b) * a.ld_u;

  if (bad || M == -INFINITY) {  // the same in every block
    if (rank == 0 && tid == 0) {
      if (bad) record_error(a.status, CG_DEV_BAD_PARAM);
      a.out_tok[b] = CG_NO_TOKEN;
      if (a.out_lp) a.out_lp[b] = -INFINITY;
    }
    return;  // nobody reads this block's shared memory after the exchange
  }

  // a lower bound of the threshold, and how to settle it
  float cut = -FLT_MAX;
  bool gather = false, select = false;
  if (q.greedy) {
    cut = M;
  } else if (q.k) {
    if (cut_key >= kKeyLowest) cut = fkey_inv(cut_key);
    gather = q.k <= kGatherK;
    select = !gather;
  } else if (q.p < 1.f) {
    // 1e-3 nats more than D, for the roundings
    const float D = logf(float(a.V) / ((1.f - q.p) * S)) + 1e-3f;
    cut = fmaxf(M - D * q.T, -FLT_MAX);
    gather = q.p * S <= kGatherMass;
    select = !gather;
  } else {
    // min-p alone: z >= floor_z decides, a little above its rounding
    cut = fmaxf(M + q.floor_z * q.T * (q.floor_z < 0.f ? 1.000001f : 1.f) - 1e-6f * fabsf(M), -FLT_MAX);
  }

  unsigned long long best = 0ull;
  if (gather) {
    h.collect(s, cut, true);
    cluster_sync(n);
    uint32_t total = s.n_list;
    if (rank != 0) {
      if (tid == 0) s.total = ld_remote(at_rank(&s.n_list, 0));
      __syncthreads();
      total = s.total;
    }
    if (n > 1) {
      cluster_arrive();  // rank 0's count has been read
      if (rank != 0 || total > kListCap) cluster_wait();
    }
    if (total <= kListCap) {
      if (rank != 0) return;  // rank 0 reads nobody else's shared memory
      const uint32_t tau = list_threshold(s, total, q, M, c, S);
      for (uint32_t i = tid; i < total; i += kThreads) {
        const unsigned long long e = s.list[i];
        const uint32_t key = uint32_t(e >> 32), t = best_id(e);
        float score;
        if (key >= tau && score_of(q, fkey_inv(key) - M, u, t, score)) best = max(best, pack_best(score, t));
      }
      __syncthreads();
      best = block_max(best, s.red64);
      if (n > 1) cluster_wait();  // before this block's count goes away
    } else {
      select = true;
    }
  }
  if (!gather || select) {
    h.collect(s, cut, false);
    __syncthreads();
    uint32_t tau = 0;
    if (select) {
      using F = Fmt<BF16>;
      const uint32_t lo = F::key(cut), hi = F::key(M);
      uint32_t level = 0;
      unsigned long long above, kept = static_cast<unsigned long long>(double(S) * 1099511627776.0);
      uint32_t tk = 0;
      if (q.k) {
        tk = select_key(s, n, [&](auto f) { h.each(s, cut, [&](uint32_t, float x) { f(F::key(x), 1ull); }); }, lo, hi,
                        q.k, level, above);
        if (q.p < 1.f) {  // the mass of what top-k keeps
          unsigned long long w = 0;
          h.each(s, cut, [&](uint32_t, float x) { w += F::key(x) >= tk ? mass_q(x, M, c) : 0ull; });
          __syncthreads();
          w = block_sum(w, s.red64);
          if (tid < n) st_remote(at_rank(&s.sums[rank], tid), w);
          cluster_sync(n);
          kept = 0;
          for (uint32_t i = 0; i < n; ++i) kept += s.sums[i];
        }
      }
      uint32_t tp = tk;
      if (q.p < 1.f) {
        const unsigned long long target = static_cast<unsigned long long>(double(q.p) * double(kept));
        tp = select_key(s, n, [&](auto f) { h.each(s, cut, [&](uint32_t, float x) { f(F::key(x), mass_q(x, M, c)); }); },
                        max(lo, tk), hi, target ? target : 1ull, level, above);
      }
      tau = BF16 ? tp << 16 : tp;  // a 16-bit key's tokens have fkey >= it shifted
    }
    h.each(s, cut, [&](uint32_t t, float x) {
      float score;
      if (fkey(x) >= tau && score_of(q, x - M, u, t, score)) best = max(best, pack_best(score, t));
    });
    __syncthreads();
    best = block_max(best, s.red64);
    if (tid == 0) st_remote(at_rank(&s.best[rank], 0), best);
    cluster_sync(n);
    if (rank != 0) return;
    for (uint32_t i = 0; i < n; ++i) best = max(best, s.best[i]);
  }
  if (tid == 0) {
    const uint32_t tok = best_id(best);
    a.out_tok[b] = tok;
    if (a.out_lp) a.out_lp[b] = __fdiv_rn(h.r.value(tok) - M, q.Ts) - logf(S);
  }
}

template <bool BF16>
cudaError_t launch_draw(int device, uint32_t B, const DrawArgs& a, cudaStream_t stream) {
  const Plan plan = plan_row(BF16, a.V, B, rows_on_grid(a.logits, BF16 ? CG_BF16 : CG_F32, a.ld));
  return with_nv<BF16>(plan.nv, [&](auto nv) {
    return launch_clusters<draw_kernel<BF16, decltype(nv)::value>>(device, B, plan.n, sizeof(Shared), stream, a);
  });
}

}  // namespace
}  // namespace cgk

extern "C" int cg_sample_rows(cg_ctx* c, const void* d_logits, int dtype, uint32_t B, uint32_t V, uint64_t ld,
                              const uint32_t* d_bitmask, const float* d_temp, const uint32_t* d_top_k,
                              const float* d_top_p, const float* d_min_p, const float* d_uniform,
                              uint64_t ld_uniform, uint32_t* d_out_tok, float* d_out_logprob) {
  using namespace cgk;
  if (!row_args_ok(c, d_logits, dtype, B, V, ld, d_bitmask)) return CG_E_ARG;
  if (B && (!d_out_tok || (!d_uniform && !d_temp))) return CG_E_ARG;
  if (d_uniform && ld_uniform != 0 && (ld_uniform < V || ld_uniform > (uint64_t(1) << 40))) return CG_E_ARG;
  for (const void* p : {static_cast<const void*>(d_temp), static_cast<const void*>(d_top_k),
                        static_cast<const void*>(d_top_p), static_cast<const void*>(d_min_p),
                        static_cast<const void*>(d_uniform), static_cast<const void*>(d_out_tok),
                        static_cast<const void*>(d_out_logprob)})
    if (!aligned4(p)) return CG_E_ARG;
  if (B == 0) return CG_OK;
  DeviceGuard dg(ctx_device(c), "cg_sample_rows");
  if (!dg.ok) return CG_E_CUDA;
  const CtxView v = ctx_view(c);
  const DrawArgs a{d_logits, ld, d_bitmask, V, v.t.W, d_temp, d_top_k, d_top_p, d_min_p, d_uniform, ld_uniform,
                   d_out_tok, d_out_logprob, v.t.status};
  const int dev = ctx_device(c);
  const cudaError_t e =
      dtype == CG_BF16 ? launch_draw<true>(dev, B, a, v.stream) : launch_draw<false>(dev, B, a, v.stream);
  return e == cudaSuccess ? CG_OK : CG_E_CUDA;
}
