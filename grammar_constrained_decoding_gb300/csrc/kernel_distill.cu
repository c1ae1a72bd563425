// Distillation from a teacher's top logits, forward and backward
// (cg_distill_loss, cg_distill_grad).
//
//   loss = T^2 sum_k q_k (log q_k - log p[id_k]),  log p_v = (x_v - m) / T - log S,
//   dloss/dx_v = T (p_v - sum_{k: id_k = v} q_k),
// q the softmax of the teacher's listed logits / T, S = sum exp((x - m) / T).
//
// One block per row; each pass reads the row again.  The gradient is written
// for every token as T w p_v first; the listed ones are written over after a
// block barrier (same block, so in order).
#include "logit_row.cuh"

namespace cgk {
namespace {

using namespace row;

constexpr uint32_t kSlotsMax = 2 * CG_TOP_MAX;

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

template <bool BF16>
__device__ __forceinline__ void store_grad(void* row, uint32_t t, float g) {
  if (BF16) static_cast<__nv_bfloat16*>(row)[t] = __float2bfloat16_rn(g);
  else static_cast<float*>(row)[t] = g;
}

template <bool BF16, bool LOSS>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillArgs a) {
  __shared__ uint32_t s_id[CG_TOP_MAX];   // listed ids that count, CG_NO_TOKEN for the others
  __shared__ float s_t[CG_TOP_MAX];       // teacher logits, then weights q
  __shared__ float s_x[CG_TOP_MAX];       // the student's logits there
  __shared__ float red[33];
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t b = blockIdx.x, tid = threadIdx.x, K = a.K;
  const float T = a.temp, c = exp_scale(T);
  const Row<BF16> r{static_cast<const char*>(a.logits) + size_t(b) * a.ld * (BF16 ? 2 : 4),
                    a.bitmask ? a.bitmask + size_t(b) * a.W : nullptr, a.V};
  // the teacher's list
  float tm = -INFINITY;
  for (uint32_t k = tid; k < K; k += kThreads) {
    uint32_t id = a.ids[size_t(b) * K + k];
    const float t = fminf(a.teacher[size_t(b) * K + k], FLT_MAX);
    const bool nan = a.teacher[size_t(b) * K + k] != a.teacher[size_t(b) * K + k];
    float x = -INFINITY;
    if (id < a.V) x = r.at(id);
    else if (id != CG_NO_TOKEN) record_error(a.status, CG_DEV_BAD_TOKEN);
    if (!(x > -INFINITY) || nan || !(t > -INFINITY)) id = CG_NO_TOKEN;
    s_id[k] = id;
    s_x[k] = x;
    s_t[k] = t;
    if (id != CG_NO_TOKEN) tm = fmaxf(tm, t);
  }
  tm = block_reduce(tm, MaxOp(), -INFINITY, red);
  float ts = 0.f;
  for (uint32_t k = tid; k < K; k += kThreads)
    if (s_id[k] != CG_NO_TOKEN) ts += ex2((s_t[k] - tm) * c);
  ts = block_reduce(ts, SumOp(), 0.f, red);
  const bool listed = tm > -INFINITY;

  float M = 0.f, S = 1.f;  // p = exp2((x - M) c) / S
  if (LOSS) {
    max_and_sum(r, c, M, S);
    float l = 0.f;
    const float log_ts = logf(ts), log_s = logf(S);
    for (uint32_t k = tid; k < K; k += kThreads)
      if (s_id[k] != CG_NO_TOKEN) {
        const float lt = __fdiv_rn(s_t[k] - tm, T);
        const float q = __fdiv_rn(ex2((s_t[k] - tm) * c), ts);
        if (q > 0.f) l += q * ((lt - log_ts) - (__fdiv_rn(s_x[k] - M, T) - log_s));
      }
    l = block_reduce(l, SumOp(), 0.f, red);
    if (tid == 0) {
      a.loss[b] = listed ? T * T * l : 0.f;
      if (a.lse_out) a.lse_out[b] = M > -INFINITY ? __fdiv_rn(M, T) + log_s : -INFINITY;
    }
  }
  if (!a.grad) return;
  const float up = a.up ? a.up[b] : 1.f;
  const float scale = listed ? T * up : 0.f;
  char* grow = static_cast<char*>(a.grad) + size_t(b) * a.ld_grad * (BF16 ? 2 : 4);
  const float lse = LOSS ? 0.f : a.lse_in[b];
  auto prob = [&](float x) { return LOSS ? __fdiv_rn(ex2((x - M) * c), S) : ex2((__fdiv_rn(x, T) - lse) * kLog2e); };
  for (uint32_t k = tid; k < K; k += kThreads) s_t[k] = __fdiv_rn(ex2((s_t[k] - tm) * c), ts);
  for (uint32_t t = tid; t < a.V; t += kThreads) {
    const float x = r.at(t);
    store_grad<BF16>(grow, t, x > -INFINITY && listed ? scale * prob(x) : 0.f);
  }
  __syncthreads();
  for (uint32_t k = tid; k < K; k += kThreads) {
    const uint32_t id = s_id[k];
    if (id == CG_NO_TOKEN) continue;
    float q = 0.f;  // an id listed twice: every one of its entries writes the same sum
    for (uint32_t j = 0; j < K; ++j)
      if (s_id[j] == id) q += s_t[j];
    store_grad<BF16>(grow, id, scale * (prob(s_x[k]) - q));
  }
}

int distill(cg_ctx* c, const char* call, const DistillArgs& base, int dtype, uint32_t B, bool loss) {
  if (B == 0) return CG_OK;
  DeviceGuard dg(ctx_device(c), call);
  if (!dg.ok) return CG_E_CUDA;
  const CtxView v = ctx_view(c);
  DistillArgs a = base;
  a.W = v.t.W;
  a.status = v.t.status;
  auto* kernel = dtype == CG_BF16 ? (loss ? distill_kernel<true, true> : distill_kernel<true, false>)
                                  : (loss ? distill_kernel<false, true> : distill_kernel<false, false>);
  return launch_dependent(kernel, B, row::kThreads, 0, v.stream, a) == cudaSuccess ? CG_OK : CG_E_CUDA;
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
