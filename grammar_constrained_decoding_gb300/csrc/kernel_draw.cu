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
//   top-k  the k-th largest logit is at least the k-th largest of the maxima of
//          groups of lanes that the warps publish;
//   top-p  tokens more than D = log(V / ((1 - p) S)) nats below the maximum have
//          together less than (1 - p) S of the mass S, so the threshold lies
//          above them;
//   min-p  is the threshold itself.
// Only tokens at or above the bound matter from there on.  Where they are few rank
// 0 gathers and settles them alone.  D supposes all V tokens just below the bound,
// so a top-p row first gathers down to kGuess nats less, with the gathered mass
// added up: it is settled when that reaches the target, which every block sees.
//
// A top-p row with many tokens is drawn without finding its threshold: the best
// scored token w of those at or above the cut is the answer exactly when the mass
// strictly above x_w is less than the target (w then belongs to the kept set, and
// nothing in it scores better).  If it is not, nothing at or below x_w is kept,
// and the best of the rest is tried.  The first try succeeds with probability
// top_p; after kTries the threshold is found by radix selection.
//
// What bounds it: a block's chain of copy, passes and exchanges, with no copy of a later
// row behind it, and the instructions of the passes.  256 x 128256 bf16 (66 MB, 9.7 us to
// read), back to back: 23.1 us for greedy rows, which read, sum and report (2.8 TB/s);
// 37.2 with top-k 50 and top-p 0.9, which gather; 51.9 without a cut, which read 131 MB of
// random numbers too and take a logarithm a token (3.8 TB/s); 36.2 with min-p 0.05 alone;
// 60.0 with top-p 0.9 at T = 0.7 (peaked rows 40.3) and 84.0 with 0.95 at T = 1 (78.9),
// where thousands of tokens a row are scored and their masses added.  A single row of
// 32000 with top-k and top-p takes 7.4 us: a launch, a row's copy and two exchanges, one
// after the other.
#include "logit_row.cuh"

namespace cgk {
namespace {

using namespace row;

// groups of a thread for many rows: 32 KB parts, four blocks an SM.  Of 256 x 128256,
// greedy: 4 groups 33.3 us, 6 27.6, 8 23.1, 12 25.6, 16 27.3
constexpr uint32_t kFull = 8;

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

// min-p rows whose kept tokens cannot be more than this are gathered: the list
// then overflows only by ties
constexpr float kGatherCount = 768.f;
// The nats that a peaked top-p row's first gather stays above the certain bound.
// 256 x 128256 peaked rows, top-p 0.9 at T = 0.7 and 0.95 at T = 1: 2 nats 42.4 and 91.9
// us, 3 38.8 and 83.6, 4 37.0 and 87.8
constexpr float kGuess = 3.f;
// After a guess that fell short: the mass below a cut falls off by about this a nat
constexpr float kFallOff = 0.35f;
// Rows with less mass than this, in units of the maximum's, are peaked: they gather
// first, the others sample masses.  256 x 128256, peaked rows at 0.9 and T = 0.7, at 0.95
// and T = 1, flat rows at 0.9: 1.5 45.0, 80.3 and 59.3 us, 2 40.5, 81.2 and 59.6, 3 38.8,
// 83.6 and 61.3; none 51.6, 78.4 and 59.0, all 39.3, 87.6 and 76.5
constexpr float kFlat = 2.f;
// Tries before the radix selection, which is taken where the random numbers rank the
// tokens against their logits.  256 x 128256 peaked rows, 0.95 at T = 1: one try 174 us,
// 16 83.6
constexpr uint32_t kTries = 16;

enum Mode : uint32_t { kNothing, kGather, kGuessFirst, kSample, kSpread };

struct RowSettings {
  float T, Ts, p, floor_z;  // Ts: the softmax's temperature (1 for greedy rows)
  uint32_t k;               // 0: no top-k
  bool greedy;
};

__device__ __forceinline__ float clamp_u(float u) { return fminf(fmaxf(u, kULo), kUHi); }
// score of a kept token; false when min-p drops it
__device__ __forceinline__ float exact_score(float d, float T, float u) {
  return __fdiv_rn(d, T) - logf(-logf(clamp_u(u)));
}
__device__ __forceinline__ bool score_of(const RowSettings& q, float d, float u, float& score) {
  score = exact_score(d, q.T, u);
  return q.floor_z == -INFINITY || __fdiv_rn(d, q.T) >= q.floor_z;
}
__device__ __forceinline__ unsigned long long mass_target(float p, unsigned long long kept) {
  const unsigned long long t = static_cast<unsigned long long>(double(p) * double(kept));
  return t ? t : 1ull;
}
__device__ __forceinline__ unsigned long long mass_total(float S) {
  return static_cast<unsigned long long>(double(S) * double(kMassOne));
}

// The threshold's key (fkey) under top-k and top-p by radix selection over the
// weights that keys(f) reports through f(key), in one block or over the cluster
template <typename Keys>
__device__ uint32_t threshold_by_levels(Shared& s, uint32_t n, uint32_t rank, Keys keys, const RowSettings& q,
                                        float cut, float M, float scale, float S) {
  const uint32_t top = fkey(M);
  uint32_t tau = fkey(cut), level = 0;
  unsigned long long above;
  if (q.k)
    tau = select_key(s, n, [&](auto f) { keys([&](uint32_t key) { f(key, 1ull); }); }, tau, top, q.k, level, above);
  if (q.p >= 1.f) return tau;
  unsigned long long kept = mass_total(S);
  if (q.k) {  // the mass of what top-k keeps
    unsigned long long w = 0;
    keys([&](uint32_t key) { w += key >= tau ? mass_q(fkey_inv(key), M, scale) : 0ull; });
    __syncthreads();
    w = block_sum(w, s.red64);
    kept = w;
    if (n > 1) {
      if (threadIdx.x < n) st_remote(at_rank(&s.sums[rank], threadIdx.x), w);
      cluster_sync(n);
      kept = 0;
      for (uint32_t i = 0; i < n; ++i) kept += s.sums[i];
    }
  }
  return select_key(s, n, [&](auto f) { keys([&](uint32_t key) { f(key, mass_q(fkey_inv(key), M, scale)); }); }, tau, top,
                    mass_target(q.p, kept), level, above);
}

// ---- drawing ------------------------------------------------------------------------

// The best of a list and, carried along, its logit
struct Drawn {
  unsigned long long best = 0ull;
  float x = 0.f;
  __device__ __forceinline__ void offer(float score, uint32_t t, float logit) {
    const unsigned long long e = pack_best(score, t);
    if (e > best) {
      best = e;
      x = logit;
    }
  }
};

// Rank 0: draws from the gathered list[0 .. c), c <= kPairCap, an entry a thread.
// With the number of entries above each (its place) and the masses added up by
// place, an entry stays when fewer than k are above it and less than the target's
// mass; the random numbers are on their way meanwhile.
__device__ Drawn draw_pairs(Shared& s, const unsigned long long* list, uint32_t c, const RowSettings& q, float M,
                            float scale, float S, const float* u) {
  const uint32_t tid = threadIdx.x;
  const unsigned long long e = tid < c ? list[tid] : 0ull;
  const float x = fkey_inv(uint32_t(e >> 32)), ut = tid < c ? u[best_id(e)] : 0.5f;
  bool stays = tid < c;
  if (q.k || q.p < 1.f) {
    s.masses[tid] = 0ull;
    place_entries<false>(s, list, c);
    const uint32_t place = s.place[tid];
    if (q.k) stays = stays && place < q.k;
    if (q.p < 1.f) {
      const unsigned long long w = stays ? mass_q(x, M, scale) : 0ull;
      if (w) atomicAdd(s.masses + place, w);
      __syncthreads();
      const unsigned long long own = s.masses[tid], upto = block_scan(own, s.red64);
      s.masses[tid] = upto - own;  // mass above place tid
      if (tid == kThreads - 1) s.base = upto;
      __syncthreads();
      stays = stays && s.masses[place] < mass_target(q.p, q.k ? s.base : mass_total(S));
    }
  }
  Drawn d;
  float score;
  if (stays && score_of(q, x - M, ut, score)) d.offer(score, best_id(e), x);
  return d;
}

// The random numbers of a group's tokens: 16-byte loads where the group is inside
// the row and the numbers lie on the 16-byte grid with the logits
template <bool BF16>
struct Numbers {
  static constexpr uint32_t E = Fmt<BF16>::E;
  const float* u;
  bool wide;
  __device__ __forceinline__ Numbers(const Held<BF16>& h, const float* u_) : u(u_) {
    wide = ((reinterpret_cast<uintptr_t>(u) / 4 - h.r.a) & 3u) == 0;
  }
  __device__ __forceinline__ void load(const Held<BF16>& h, uint32_t j, float* out) const {
    const int t0 = h.first_token(j);
    if (wide && t0 >= 0 && uint32_t(t0) + E <= h.r.V) {
#pragma unroll
      for (uint32_t i = 0; i < E / 4; ++i) {
        const float4 w = __ldcs(reinterpret_cast<const float4*>(u + t0) + i);
        out[4 * i] = w.x;
        out[4 * i + 1] = w.y;
        out[4 * i + 2] = w.z;
        out[4 * i + 3] = w.w;
      }
    } else {
#pragma unroll
      for (uint32_t e = 0; e < E; ++e) out[e] = t0 + int(e) >= 0 && t0 + int(e) < int(h.r.V) ? u[t0 + int(e)] : 0.f;
    }
  }
};

// Draws from this block's part, tokens >= low, however many.  From -log u >= 1 - u,
// a score is at most z - log(1 - u), which costs one logarithm in the
// multi-function unit.  Every thread finds the group with its best bound and the
// next group's bound; the best token of that group is scored exactly, and a thread
// with another bound that reaches the block's best score goes over its part again.
template <bool BF16>
__device__ Drawn draw_screened(Shared& s, const Held<BF16>& h, const RowSettings& q, float low, float M, float c,
                               const float* u) {
  constexpr uint32_t E = Fmt<BF16>::E;
  const Numbers<BF16> numbers(h, u);
  const float2 nm = make_float2(-M, -M), c2 = make_float2(c, c);
  // upper bounds of a group's scores, in bits
  auto bounds = [&](const uint4& v, const float* un, float* ub) {
#pragma unroll
    for (uint32_t p = 0; p < E / 2; ++p) {
      const float2 x = pair<BF16>(v, p), z = __fmul2_rn(__fadd2_rn(x, nm), c2);
      float l0, l1;
      asm("lg2.approx.f32 %0, %1;" : "=f"(l0) : "f"(__saturatef(1.f - un[2 * p])));
      asm("lg2.approx.f32 %0, %1;" : "=f"(l1) : "f"(__saturatef(1.f - un[2 * p + 1])));
      ub[2 * p] = x.x >= low ? z.x - l0 : -INFINITY;
      ub[2 * p + 1] = x.y >= low ? z.y - l1 : -INFINITY;
    }
  };
  if (threadIdx.x < h.nv) {  // the random numbers of a run are one piece: all on their way to L2 at once
    const int t = int((threadIdx.x * h.n + h.rank) * kThreads * E) - int(h.r.a), V = int(h.r.V);
    if (t < V) prefetch_l2(u + max(t, 0), u + min(t + int(kThreads * E), V));
  }
  float first = -INFINITY, second = -INFINITY;
  uint32_t at = 0;
#pragma unroll 2
  for (uint32_t j = 0; j < h.nv; ++j) {
    const uint4 v = h.at(j);
    if (!(group_max_nan<BF16>(v) >= low)) continue;
    float un[E], ub[E];
    numbers.load(h, j, un);
    bounds(v, un, ub);
    float top = ub[0];
#pragma unroll
    for (uint32_t e = 1; e < E; ++e) top = fmaxf(top, ub[e]);
    second = fmaxf(second, fminf(first, top));
    if (top > first) {
      first = top;
      at = j;
    }
  }
  Drawn d;
  float score;
  if (first > -INFINITY) {
    const uint4 v = h.at(at);
    float un[E], ub[E], top = -INFINITY;
    numbers.load(h, at, un);
    bounds(v, un, ub);
    uint32_t best = 0;
    float ut = 0.f;
#pragma unroll
    for (uint32_t e = 0; e < E; ++e) {
      second = fmaxf(second, fminf(top, ub[e]));
      if (ub[e] > top) {
        top = ub[e];
        best = e;
        ut = un[e];
      }
    }
    const float x = elem<BF16>(v, best);
    if (score_of(q, x - M, ut, score)) d.offer(score, uint32_t(h.first_token(at)) + best, x);
  }
  const unsigned long long best = block_max(d.best, s.red64);
  // 1e-3 nats cover the roundings of the bounds
  if (second > -INFINITY && (best == 0ull || second >= (fkey_inv(uint32_t(best >> 32)) - 1e-3f) * kLog2e)) {
#pragma unroll 1
    for (uint32_t j = 0; j < h.nv; ++j) {
      const uint4 v = h.at(j);
#pragma unroll 1
      for (uint32_t e = 0; e < E; ++e) {
        const float x = elem<BF16>(v, e);
        const uint32_t t = uint32_t(h.first_token(j)) + e;
        if (x >= low && score_of(q, x - M, u[t], score)) d.offer(score, t, x);
      }
    }
  }
  return d;
}

// A top-p row over the whole cluster, by trial as described above.  Returns the
// drawn token to every block; near: a cut that is likely low enough, low: one that
// certainly is.  late: a wait of the block ran out.
template <bool BF16>
__device__ Drawn draw_by_trial(Shared& s, const Held<BF16>& h, const RowSettings& q, float near, float low, float M,
                               float c, float S, const float* u, bool& late) {
  const uint32_t tid = threadIdx.x, lane = tid & 31, n = h.n;
  const float target = fmaxf(q.p * S, 1e-30f);
  float cut = fmaxf(near, low);
  Drawn d;
  bool listed = false;
#pragma unroll 1
  for (uint32_t round = 0;; ++round) {
    const bool settled = round == kTries;  // the random numbers rank the tokens almost against their logits
    if (settled) {
      if (listed) {  // the histograms take the list's place
        listed = false;
        __syncthreads();
        if (tid == 0) s.n_local = 0;
      }
      cut = fkey_inv(threshold_by_levels(
          s, n, h.rank, [&](auto f) { h.each(low, [&](uint32_t, float y) { f(fkey(y)); }); }, q, low, M, c, S));
    }
    __syncthreads();
    if (!listed && !settled) {  // few enough: from a list, else from the part itself
      // the first groups tell about how many there are
      const uint32_t some = h.tm >= cut ? __popc(ge_bits<BF16>(h.at(0), cut, BF16 ? bf16_pair_up(cut) : 0u)) : 0u;
      if (block_sum(some, s.red_max) * h.nv <= kListCap) listed = h.compact(s, cut);
    }
    const uint32_t key = fkey(cut);
    if (listed) {
      d = Drawn();
      for (uint32_t i = tid; i < s.n_local; i += kThreads) {
        const unsigned long long e = s.list[i];
        const uint32_t k = uint32_t(e >> 32), t = best_id(e);
        float score;
        if (k >= key && score_of(q, fkey_inv(k) - M, u[t], score)) d.offer(score, t, fkey_inv(k));
      }
    } else {
      d = draw_screened<BF16>(s, h, q, cut, M, c, u);
    }
    const unsigned long long best = block_max(d.best, s.red64b);
    if (best ? d.best == best : tid == 0) {  // one thread
      for (uint32_t r = 0; r < n; ++r) {
        send(at_rank(&s.best[h.rank], r), best, at_rank(&s.bar_best, r));
        send(at_rank(&s.best_x[h.rank], r), __float_as_uint(d.x), at_rank(&s.bar_best, r));
      }
    }
    if (tid == 0) mbar_expect_tx(&s.bar_best, n * 12u);
    bool ok = __syncthreads_and(wait_sent(&s.bar_best, round & 1u));
    d = Drawn();
    for (uint32_t r = 0; r < n; ++r)
      if (s.best[r] > d.best) {
        d.best = s.best[r];
        d.x = s.best_x[r];
      }
    if (ok && (settled || !d.best)) return d;
    // the mass above the drawn token and, for the first cut, at or above it
    const bool check = round == 0 && cut > low;
    float2 w = make_float2(0.f, 0.f);
    if (listed) {  // in integers: the list's order is arbitrary
      const uint32_t x = fkey(d.x);
      unsigned long long above = 0, from = 0;
      for (uint32_t i = tid; i < s.n_local; i += kThreads) {
        const uint32_t k = uint32_t(s.list[i] >> 32);
        const unsigned long long m = mass_q(fkey_inv(k), M, c);
        above += k > x ? m : 0ull;
        from += k >= key ? m : 0ull;
      }
      __syncthreads();
      w.x = float(block_sum(above, s.red64)) * (1.f / kMassOne) * (1.f / kWarps);
      w.y = float(block_sum(from, s.red64b)) * (1.f / kMassOne) * (1.f / kWarps);
    } else if (__any_sync(0xFFFFFFFFu, h.tm >= cut)) {
      w = h.masses_from(M, c, d.x, check ? cut : INFINITY);
      w.x = warp_reduce(w.x, SumOp());
      w.y = warp_reduce(w.y, SumOp());
    }
    if (lane < n)
      send(at_rank(&s.mass[h.rank * kWarps + (tid >> 5)], lane),
           (static_cast<unsigned long long>(__float_as_uint(w.y)) << 32) | __float_as_uint(w.x),
           at_rank(&s.bar_mass, lane));
    if (tid == 0) mbar_expect_tx(&s.bar_mass, n * kWarps * 8u);
    late = !__syncthreads_and(wait_sent(&s.bar_mass, round & 1u) && ok);
    if (late) return Drawn();
    w = make_float2(0.f, 0.f);
    for (uint32_t i = lane; i < n * kWarps; i += 32) {
      w.x += s.mass[i].x;
      w.y += s.mass[i].y;
    }
    w.x = warp_reduce(w.x, SumOp());
    w.y = warp_reduce(w.y, SumOp());
    if (check && !(w.y >= target * 1.00001f)) {
      cut = low;  // kept tokens may lie below
      listed = false;
      __syncthreads();
      if (tid == 0) s.n_local = 0;  // a barrier opens the next round
      continue;
    }
    if (w.x < target) return d;
    if (!listed) {
      __syncthreads();
      if (tid == 0) s.n_local = 0;
    }
    // the next value of the type above the refused token's
    cut = BF16 ? fkey_inv(((fkey(d.x) >> 16) + 1u) << 16) : fkey_inv(fkey(d.x) + 1u);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 4) draw_kernel(const DrawArgs a, uint32_t nv) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  griddep_launch_dependents();
  const uint32_t n = cluster_size(), rank = cluster_rank(), b = blockIdx.x / n, tid = threadIdx.x;
  begin(s);
  Held<BF16> h(Row<BF16>(a.logits, a.ld, a.bitmask, a.W, a.V, b), nv, smem + sizeof(Shared));
  griddep_wait();
  h.start(s, true);
  may_send();
  RowSettings q;
  q.T = a.temp ? a.temp[b] : 1.f;
  q.k = a.top_k ? a.top_k[b] : 0u;
  const float p = a.top_p ? a.top_p[b] : 1.f, mp = a.min_p ? a.min_p[b] : 0.f;
  q.p = fmaxf(p, 0.f);
  q.greedy = q.T == 0.f;
  q.Ts = q.greedy ? 1.f : q.T;
  if (q.k >= a.V || q.greedy) q.k = 0;
  const float c = exp_scale(q.Ts);
  const bool bad = !(q.T >= 0.f && q.T <= FLT_MAX) || (!q.greedy && (p != p || mp != mp || !a.u));
  // Rows that need nothing of the others' parts before they send what may be drawn:
  // the maximum, or the best of all tokens.
  enum { kTogether, kBest, kAny } alone = kTogether;
  if (!bad) {
    if (q.greedy) alone = kBest;
    else if (!q.k && q.p >= 1.f && !(mp > 0.f)) alone = kAny;
  }
  bool tight = true;
  const uint32_t per_warp = q.k && !alone ? bounds_per_warp(q.k, n, tight) : 0u;
  const bool taken = h.template take<true>(s, c);
  if (!taken) {
    s.late = 1;
    record_error(a.status, CG_DEV_TIMEOUT);
  }
  ready_others();
  const unsigned long long rec = h.record(c);
  if (alone) {
    if (alone == kBest) {
      h.template report<true>(s, rec, s.top);
    } else {
      h.template report<false>(s, rec);
      // the block's best by scores relative to its own maximum: their order is that
      // of scores relative to the row's
      q.floor_z = -INFINITY;
      const float m = fkey_inv(block_max(fkey(h.tm), s.red_max));
      Drawn d;
      if (m > -INFINITY) d = draw_screened<BF16>(s, h, q, -FLT_MAX, m, c, a.u + size_t(b) * a.ld_u);
      const unsigned long long best = block_max(d.best, s.red64b);
      if (best ? d.best == best : tid == 0)  // one thread
        send(at_rank(&s.best[rank], 0), best ? pack_best(d.x, best_id(best)) : 0ull, at_rank(&s.bar_best, 0));
    }
    if (rank != 0) return;
  } else {
    h.publish(s, rec, per_warp);
  }
  if (tid < 32) {
    const bool ok = wait_sent(&s.bar_rec);
    float M, S, rest;  // S = 1 + rest
    merge(s.rec, n * kWarps, c, M, S, rest);
    // a lower bound of the threshold, and how to settle it.  Without top-k the
    // mass that top-p refers to is known, so min-p bounds what matters as well.
    const float floor_z = logf(fminf(fmaxf(mp, 0.f), 1.f));  // -inf for min_p = 0
    float cut = -FLT_MAX, guess = 0.f;
    Mode mode = kSpread;
    if (bad || !ok || M == -INFINITY) {
      mode = kNothing;
    } else if (q.k) {
      const uint32_t key = per_warp ? bound_key(s, n * kWarps * per_warp, q.k) : 0u;
      if (key >= kKeyLowest) cut = fkey_inv(key);
      if (tight) mode = kGather;
    } else if (!alone) {
      // a little below M + T log(min_p), for the roundings
      if (floor_z > -INFINITY) {
        cut = fmaxf(M + floor_z * q.T * 1.000001f - 1e-6f * fabsf(M), -FLT_MAX);
        if (S <= kGatherCount * mp) mode = kGather;  // every kept token has at least min_p of the maximum's mass
      }
      if (q.p < 1.f) {
        const float D = logf(float(a.V) / ((1.f - q.p) * S)) + 1e-3f;
        cut = fmaxf(cut, M - D * q.T);
        if (mode != kGather) {
          guess = fmaxf(D, 0.f);
          mode = S < kFlat ? kGuessFirst : kSample;
        }
      }
    }
    if (tid == 0) {
      s.M = M;
      s.rest = rest;
      s.cut = cut;
      s.guess = guess;
      s.floor_z = floor_z;
      s.mode = mode;
      if (!ok) s.late = 1;
    }
  }
  __syncthreads();
  const float M = s.M, S = 1.f + s.rest, cut = s.cut;
  uint32_t mode = s.mode;
  bool late = s.late != 0;
  if (mode == kNothing || late) {
    if (rank == 0 && tid == 0) {
      if (late) record_error(a.status, CG_DEV_TIMEOUT);
      else if (bad) record_error(a.status, CG_DEV_BAD_PARAM);
      a.out_tok[b] = CG_NO_TOKEN;
      if (a.out_lp) a.out_lp[b] = -INFINITY;
    }
    if (alone == kAny) {  // not before what the others send has arrived
      if (tid == 0) mbar_expect_tx(&s.bar_best, n * 8u);
      late = !__syncthreads_and(wait_sent(&s.bar_best)) || late;
    }
    if (late) leave_last(n);
    return;
  }
  q.floor_z = s.floor_z;
  const float* u = a.u + size_t(b) * a.ld_u;

  if (alone == kBest || alone == kAny) {  // rank 0, one warp
    if (tid >= 32) return;
    Drawn d;
    bool ok = true;
    if (alone == kBest) {
      for (uint32_t i = tid; i < n * kWarps; i += 32) d.best = max(d.best, s.top[i]);
      d.x = M;
    } else {
      if (tid == 0) mbar_expect_tx(&s.bar_best, n * 8u);
      ok = wait_sent(&s.bar_best);
      const unsigned long long e = tid < n ? s.best[tid] : 0ull;
      float score;
      if (e) {
        const float x = fkey_inv(uint32_t(e >> 32));
        if (score_of(q, x - M, u[best_id(e)], score)) d.offer(score, best_id(e), x);
      }
    }
    const unsigned long long best = warp_reduce(d.best, MaxOp());
    if (alone == kBest ? tid == 0 : d.best == best) {
      a.out_tok[b] = ok ? best_id(best) : CG_NO_TOKEN;
      if (a.out_lp) a.out_lp[b] = ok ? __fdiv_rn(d.x - M, q.Ts) - log1pf(s.rest) : -INFINITY;
      if (!ok) record_error(a.status, CG_DEV_TIMEOUT);
    }
    if (__any_sync(0xFFFFFFFFu, !ok)) leave_last(n);
    return;
  }

  Drawn d;
  float list_cut = cut, near = cut;
  uint32_t total = 0;
  bool left_out = false;  // a block had too many entries to send
  if (mode == kGather) {
    h.template gather<false>(s, cut, false, 0.f, 0.f);
    if (rank != 0) return;  // its entries are with rank 0
    float none;
    bool whole = true;
    if (!h.tallied(s, total, whole, none)) mode = kNothing;
    else if (!whole) left_out = true;
  } else if (mode == kGuessFirst) {
    list_cut = fmaxf(cut, M - fmaxf(s.guess - kGuess, 0.f) * q.T);
    h.template gather<true>(s, list_cut, true, M, c);
    float mass;
    bool whole;
    const bool ok = h.tallied(s, total, whole, mass);
    mode = !ok ? kNothing : whole && total <= kListCap && mass >= q.p * S * 1.00001f ? kGather : kSpread;
    if (rank != 0 && mode == kNothing) leave_last(n);
    if (rank != 0 && (mode == kGather || mode == kNothing)) return;
    // where the missing mass probably ends: the mass below a cut falls off by
    // about kFallOff a nat
    near = list_cut;
    if (mass < q.p * S * 1.00001f) {
      const float below = fmaxf(1.f - mass / S, 1e-6f);
      near -= __fdividef(logf(below / (1.f - q.p)) + 0.05f, kFallOff) * q.T;
    }
  }
  if (mode == kSample) {
    // the masses below eight cuts, estimated from the first group of every thread:
    // the first cut that leaves little enough below it is the one to try
    constexpr int kCuts = 8;
    constexpr float depth[kCuts] = {5.5f, 4.9f, 4.3f, 3.7f, 3.1f, 2.5f, 1.8f, 1.f};
    float w[kCuts] = {};
    const float D = s.guess;
    auto level = [&](int i) { return M - fmaxf(D - depth[i], 0.f) * q.T; };
    const uint4 v0 = h.at(0);
#pragma unroll
    for (uint32_t e = 0; e < Fmt<BF16>::E; ++e) {
      const float x = elem<BF16>(v0, e), m = ex2((x - M) * c);
#pragma unroll
      for (int i = 0; i < kCuts; ++i) w[i] += x < level(i) ? m : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kCuts; ++i) w[i] = warp_reduce(w[i], SumOp());
    const uint32_t lane = tid & 31;
    if (lane < n) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        send(at_rank(&s.sample[rank * kWarps + (tid >> 5)][i], lane),
             make_uint4(__float_as_uint(w[4 * i]), __float_as_uint(w[4 * i + 1]), __float_as_uint(w[4 * i + 2]),
                        __float_as_uint(w[4 * i + 3])),
             at_rank(&s.bar_tally, lane));
    }
    if (tid == 0) mbar_expect_tx(&s.bar_tally, n * kWarps * 32u);
    const bool ok = __syncthreads_and(wait_sent(&s.bar_tally));
#pragma unroll
    for (int i = 0; i < kCuts; ++i) w[i] = 0.f;
    for (uint32_t i = lane; i < n * kWarps; i += 32) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float4 t = s.sample[i][k];
        w[4 * k] += t.x;
        w[4 * k + 1] += t.y;
        w[4 * k + 2] += t.z;
        w[4 * k + 3] += t.w;
      }
    }
    const float share = fminf(1.f, float(n * kThreads * Fmt<BF16>::E) / float(a.V));
    const float most = (1.f - q.p) * S * share * 0.93f;
    near = cut;
#pragma unroll
    for (int i = kCuts - 1; i >= 0; --i)
      if (warp_reduce(w[i], SumOp()) <= most) near = level(i);
    if (!ok) {
      if (rank == 0 && tid == 0) {
        record_error(a.status, CG_DEV_TIMEOUT);
        a.out_tok[b] = CG_NO_TOKEN;
        if (a.out_lp) a.out_lp[b] = -INFINITY;
      }
      leave_last(n);
      return;
    }
    mode = kSpread;
  }
  // the entries are on their way to rank 0, which settles them or, after a wrong
  // guess, uses the list's memory again
  if ((s.mode == kGather || s.mode == kGuessFirst) && rank == 0 && (mode == kNothing || !h.listed(s, total))) {
    if (tid == 0) {
      record_error(a.status, CG_DEV_TIMEOUT);
      a.out_tok[b] = CG_NO_TOKEN;
      if (a.out_lp) a.out_lp[b] = -INFINITY;
    }
    leave_last(n);
    return;
  }
  const bool gather = mode == kGather;
  if (gather) {
    const unsigned long long* list = s.list;
    uint32_t few = total;
    if (left_out) {
      few = kListCap + 1;
    } else if (total > kPairCap && total <= kListCap && q.k) {
      few = keep_few(s, total, list_bound(s, total, q.k));
      list = s.few;
    }
    if (few <= kPairCap) {
      d = draw_pairs(s, list, few, q, M, c, S, u);
    } else {
      // from the list, or from the row when ties have made it overflow
      const bool fits = total <= kListCap && !left_out;
      auto entries = [&](auto f) {
        if (fits) {
          for (uint32_t i = tid; i < total; i += kThreads)
            f(best_id(s.list[i]), fkey_inv(uint32_t(s.list[i] >> 32)));
        } else {
          each_of_row(h.r, f);
        }
      };
      float tau = list_cut;
      if (q.k || q.p < 1.f) {
        tau = fkey_inv(threshold_by_levels(
            s, 1, 0, [&](auto f) { entries([&](uint32_t, float x) { f(fkey(x)); }); }, q, list_cut, M, c, S));
      }
      entries([&](uint32_t t, float x) {
        float score;
        if (x >= tau && score_of(q, x - M, u[t], score)) d.offer(score, t, x);
      });
    }
    __syncthreads();
    const unsigned long long best = block_max(d.best, s.red64);
    if (d.best == best && (best != 0ull || tid == 0)) {
      a.out_tok[b] = best_id(best);
      if (a.out_lp) a.out_lp[b] = __fdiv_rn(d.x - M, q.Ts) - log1pf(s.rest);
    }
    return;
  }

  if (!q.k && q.p < 1.f) {
    d = draw_by_trial<BF16>(s, h, q, near, cut, M, c, S, u, late);
    if (late && tid == 0) record_error(a.status, CG_DEV_TIMEOUT);
    if (rank == 0 && tid == 0) {
      a.out_tok[b] = d.best ? best_id(d.best) : CG_NO_TOKEN;
      if (a.out_lp) a.out_lp[b] = d.best ? __fdiv_rn(d.x - M, q.Ts) - log1pf(s.rest) : -INFINITY;
    }
    if (late) leave_last(n);
    return;
  }

  float tau = cut;
  if (q.k)
    tau = fkey_inv(threshold_by_levels(
        s, n, rank, [&](auto f) { h.each(cut, [&](uint32_t, float x) { f(fkey(x)); }); }, q, cut, M, c, S));
  d = draw_screened<BF16>(s, h, q, tau, M, c, u);
  unsigned long long best = block_max(d.best, s.red64b);
  if (best ? d.best == best : tid == 0) {  // one thread
    send(at_rank(&s.best[rank], 0), best, at_rank(&s.bar_best, 0));
    send(at_rank(&s.best_x[rank], 0), __float_as_uint(d.x), at_rank(&s.bar_best, 0));
  }
  if (q.k) {  // the others may still be reading this block's histograms
    cluster_arrive_relaxed();
    cluster_wait();
  }
  if (rank != 0) return;
  if (tid >= 32) return;
  if (tid == 0) mbar_expect_tx(&s.bar_best, n * 12u);
  const bool ok = wait_sent(&s.bar_best);
  d = Drawn();
  for (uint32_t r = 0; r < n; ++r)
    if (s.best[r] > d.best) {
      d.best = s.best[r];
      d.x = s.best_x[r];
    }
  if (tid == 0) {
    if (!ok) record_error(a.status, CG_DEV_TIMEOUT);
    const bool there = ok && d.best;
    a.out_tok[b] = there ? best_id(d.best) : CG_NO_TOKEN;
    if (a.out_lp) a.out_lp[b] = there ? __fdiv_rn(d.x - M, q.Ts) - log1pf(s.rest) : -INFINITY;
  }
  if (__any_sync(0xFFFFFFFFu, !ok)) leave_last(n);
}

template <bool BF16>
cudaError_t launch_draw(int device, uint32_t B, const DrawArgs& a, cudaStream_t stream) {
  const Plan plan = plan_row(BF16, a.V, B, rows_on_grid(a.logits, BF16 ? CG_BF16 : CG_F32, a.ld), kFull);
  return launch_clusters<draw_kernel<BF16>>(device, B, plan.n, kThreads,
                                            sizeof(Shared) + part_bytes(BF16, plan.nv, a.bitmask), stream, a, plan.nv);
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
