// Distillation from a teacher's top logits, forward and backward
// (cg_distill_loss, cg_distill_grad).
//
//   loss = T^2 sum_k q_k (log q_k - log p[id_k]),  log p_v = (x_v - m) / T - log S,
//   dloss/dx_v = T (p_v - sum_{k: id_k = v} q_k),
// q the softmax of the teacher's listed logits / T, S = sum exp((x - m) / T).
//
// The row is held on chip by a cluster (logit_row.cuh): the logits are read from
// memory once and the gradient is written once from the registers.  Every
// gradient is written as T w p_v first; the block that wrote a listed token's
// writes it over after a block barrier.  All reads of the row's logits, the
// listed ones by every block included, come before the cluster meets, all
// writes after it, so the gradient may take the logits' place.
#include "logit_row.cuh"

namespace cgk {
namespace {

using namespace row;

// groups of a thread for many rows: 64 KB parts, three blocks an SM; fewer, longer
// parts cost fewer exchanges and list look-ups.  Loss and gradient of 2048 x 128256: 8
// groups 270.6 us, 12 237.9, 16 224.6, 24 274.0
constexpr uint32_t kFull = 16;

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
__global__ void __launch_bounds__(kThreads, 4) distill_kernel(const DistillArgs a, uint32_t nv) {
  extern __shared__ __align__(16) unsigned char smem[];
  DistillShared& s = *reinterpret_cast<DistillShared*>(smem);
  const List l(smem + sizeof(DistillShared), a.K);
  griddep_launch_dependents();
  const uint32_t n = cluster_size(), rank = cluster_rank(), b = blockIdx.x / n, tid = threadIdx.x, K = a.K;
  begin(s);
  Held<BF16> h(Row<BF16>(a.logits, a.ld, a.bitmask, a.W, a.V, b), nv, 
               smem + sizeof(DistillShared) + List::bytes(K));
  griddep_wait();
  h.start(s, !a.grad);
  may_send();
  const float T = a.temp, c = exp_scale(T);
  // the teacher's list (without a gradient only rank 0 has a use for it)
  if (LOSS && !a.grad && rank != 0) {
    if (!h.template take<true>(s, c)) record_error(a.status, CG_DEV_TIMEOUT);
    ready_others();
    h.template report<false>(s, c);
    return;
  }
  const uint32_t slots = l.slots;
  for (uint32_t i = tid; i < slots; i += kThreads) l.hash[i] = CG_NO_TOKEN;
  if (tid == 0) s.repeated = 0;
  float tm = -INFINITY;
  for (uint32_t k = tid; k < K; k += kThreads) {
    uint32_t id = a.ids[size_t(b) * K + k];
    const float raw = a.teacher[size_t(b) * K + k];
    const float t = raw != raw ? -INFINITY : fminf(raw, FLT_MAX);
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
    if (a.grad) {
      h.publish(s, c);
    } else {
      h.template report<false>(s, c);
    }
    if (tid < 32) {
      const bool ok = wait_sent(&s.bar_rec);
      float m, sum;
      merge(s, n, c, m, sum);
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
        if (l.id[k] != CG_NO_TOKEN) {
          const float q = __fdiv_rn(ex2((l.t[k] - tm) * c), ts);
          if (q > 0.f) part += q * ((__fdiv_rn(l.t[k] - tm, T) - log_ts) - (__fdiv_rn(l.x[k] - M, T) - log_s));
        }
      __syncthreads();
      part = block_sum(part, s.red_f);
      if (tid == 0) {
        a.loss[b] = listed ? T * T * part : 0.f;
        if (a.lse_out) a.lse_out[b] = M > -INFINITY ? __fdiv_rn(M, T) + log_s : -INFINITY;
      }
    }
    if (!a.grad) return;
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
#pragma unroll 2
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

template <bool BF16>
cudaError_t launch_distill(int device, uint32_t B, const DistillArgs& a, bool loss, cudaStream_t stream) {
  const Plan plan = plan_row(BF16, a.V, B, rows_on_grid(a.logits, BF16 ? CG_BF16 : CG_F32, a.ld), kFull);
  const size_t smem = sizeof(DistillShared) + List::bytes(a.K) + part_bytes(BF16, plan.nv, a.bitmask);
  return loss ? launch_clusters<distill_kernel<BF16, true>>(device, B, plan.n, smem, stream, a, plan.nv)
              : launch_clusters<distill_kernel<BF16, false>>(device, B, plan.n, smem, stream, a, plan.nv);
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
