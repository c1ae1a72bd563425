// Sampling with per-row temperature, top-k, top-p and min-p from given random
// numbers (cg_sample_rows).
//
// Per row, with d_t = x_t - max x and z_t = d_t / T: every cut keeps an upper
// set of the logits, so all of them together are one threshold on x -- the
// k-th largest logit (counted), the largest value whose upper set carries
// top_p of the kept mass (weighed), max x + T log(min_p) -- and the token is
// argmax z_t - log(-log u_t) over x_t >= threshold.
//
// One block per row; each pass reads the row again.
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

template <bool BF16>
__global__ void __launch_bounds__(kThreads) draw_kernel(const DrawArgs a) {
  __shared__ unsigned long long hist[kBins];
  __shared__ unsigned long long red[33];
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t b = blockIdx.x;
  const float T = a.temp ? a.temp[b] : 1.f;
  const uint32_t k = a.top_k ? a.top_k[b] : 0u;
  const float p = a.top_p ? a.top_p[b] : 1.f, mp = a.min_p ? a.min_p[b] : 0.f;
  const bool greedy = T == 0.f;
  if (!(T >= 0.f && T <= FLT_MAX) || p != p || mp != mp || (!greedy && !a.u)) {
    if (threadIdx.x == 0) {
      record_error(a.status, CG_DEV_BAD_PARAM);
      a.out_tok[b] = CG_NO_TOKEN;
      if (a.out_lp) a.out_lp[b] = -INFINITY;
    }
    return;
  }
  const Row<BF16> r{static_cast<const char*>(a.logits) + size_t(b) * a.ld * (BF16 ? 2 : 4),
                    a.bitmask ? a.bitmask + size_t(b) * a.W : nullptr, a.V};
  const float Ts = greedy ? 1.f : T, c = exp_scale(Ts);
  float M, S;
  max_and_sum(r, c, M, S);
  if (M == -INFINITY) {
    if (threadIdx.x == 0) {
      a.out_tok[b] = CG_NO_TOKEN;
      if (a.out_lp) a.out_lp[b] = -INFINITY;
    }
    return;
  }
  uint32_t tau = fkey(-FLT_MAX);
  if (greedy) {
    tau = fkey(M);
  } else {
    if (k != 0 && k < a.V)
      tau = select_key([&](auto f) { r.each([&](uint32_t, float x) { f(fkey(x), 1ull); }); }, tau, fkey(M), k, hist);
    if (p < 1.f) {
      auto masses = [&](auto f) { r.each([&](uint32_t, float x) { f(fkey(x), mass_q(x, M, c)); }); };
      unsigned long long kept = 0ull;
      masses([&](uint32_t key, unsigned long long w) { kept += key >= tau ? w : 0ull; });
      kept = block_reduce(kept, SumOp(), 0ull, red);
      const unsigned long long target = static_cast<unsigned long long>(double(fmaxf(p, 0.f)) * double(kept));
      tau = select_key(masses, tau, fkey(M), target ? target : 1ull, hist);
    }
  }
  const float floor_z = logf(fminf(fmaxf(mp, 0.f), 1.f));  // -inf for min_p = 0
  const float* u = a.u + size_t(b) * a.ld_u;
  unsigned long long best = 0ull;
  r.each([&](uint32_t t, float x) {
    if (fkey(x) < tau) return;
    float score = 0.f;
    if (!greedy) {
      const float z = __fdiv_rn(x - M, T);
      if (!(z >= floor_z)) return;
      const float v = fminf(fmaxf(u[t], kULo), kUHi);
      score = z - logf(-logf(v));
    }
    best = max(best, pack_best(score, t));
  });
  best = block_reduce(best, MaxOp(), 0ull, red);
  if (threadIdx.x == 0) {
    const uint32_t tok = best_id(best);
    a.out_tok[b] = tok;
    if (a.out_lp) a.out_lp[b] = __fdiv_rn(r.value(tok) - M, Ts) - logf(S);
  }
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
  const cudaError_t e = dtype == CG_BF16 ? launch_dependent(draw_kernel<true>, B, row::kThreads, 0, v.stream, a)
                                         : launch_dependent(draw_kernel<false>, B, row::kThreads, 0, v.stream, a);
  return e == cudaSuccess ? CG_OK : CG_E_CUDA;
}
