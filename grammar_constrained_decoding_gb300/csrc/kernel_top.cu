// The n best allowed tokens of each row with their log-probabilities
// (cg_top_logprobs): the n-th largest logit by counting, then the tokens above
// it and the lowest ids among those equal to it, sorted by (logit, id).
//
// One block per row; each pass reads the row again.
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

template <bool BF16>
__global__ void __launch_bounds__(kThreads) top_kernel(const TopArgs a) {
  __shared__ unsigned long long list[kSortCap];
  __shared__ uint32_t s_n, s_ties;
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t b = blockIdx.x;
  const Row<BF16> r{static_cast<const char*>(a.logits) + size_t(b) * a.ld * (BF16 ? 2 : 4),
                    a.bitmask ? a.bitmask + size_t(b) * a.W : nullptr, a.V};
  float M, S;
  max_and_sum(r, kLog2e, M, S);
  uint32_t found = 0;
  if (M > -INFINITY) {
    const uint32_t tau = select_key([&](auto f) { r.each([&](uint32_t, float x) { f(fkey(x), 1ull); }); },
                                    fkey(-FLT_MAX), fkey(M), a.n, list);
    __syncthreads();
    if (threadIdx.x == 0) s_n = s_ties = 0;
    __syncthreads();
    uint32_t above = 0, ties = 0;
    r.each([&](uint32_t, float x) {
      above += fkey(x) > tau;
      ties += fkey(x) == tau;
    });
    if (above) atomicAdd(&s_n, above);
    if (ties) atomicAdd(&s_ties, ties);
    __syncthreads();
    // the lowest ids among the ties: ~id selected like a key
    const uint32_t want = a.n - s_n;
    uint32_t last = ~(a.V - 1u);
    if (s_ties > want)
      last = select_key([&](auto f) { r.each([&](uint32_t t, float x) { if (fkey(x) == tau) f(~t, 1ull); }); },
                        ~(a.V - 1u), ~0u, want, list);
    __syncthreads();
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    r.each([&](uint32_t t, float x) {
      if (fkey(x) > tau || (fkey(x) == tau && ~t >= last)) list[atomicAdd(&s_n, 1u)] = pack_best(x, t);
    });
    __syncthreads();
    found = s_n;
    sort_desc(list, found);
  }
  const float log_s = logf(S);
  for (uint32_t i = threadIdx.x; i < a.n; i += kThreads) {
    const bool there = i < found;
    a.out_ids[size_t(b) * a.n + i] = there ? best_id(list[i]) : CG_NO_TOKEN;
    a.out_lp[size_t(b) * a.n + i] = there ? (fkey_inv(uint32_t(list[i] >> 32)) - M) - log_s : -INFINITY;
  }
  if (a.out_lse && threadIdx.x == 0) a.out_lse[b] = M > -INFINITY ? M + log_s : -INFINITY;
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
  const cudaError_t e = dtype == CG_BF16 ? launch_dependent(top_kernel<true>, B, row::kThreads, 0, v.stream, a)
                                         : launch_dependent(top_kernel<false>, B, row::kThreads, 0, v.stream, a);
  return e == cudaSuccess ? CG_OK : CG_E_CUDA;
}
