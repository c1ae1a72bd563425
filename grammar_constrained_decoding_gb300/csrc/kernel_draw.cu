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
// Otherwise, and for a large k, the blocks count the tokens at or above the bound
// by key, add up the counts, find the threshold and each draw from their own part.
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

// min-p rows whose kept tokens cannot be more than this are gathered: the list
// then overflows only by ties
constexpr float kGatherCount = 1536.f;
constexpr float kGuess = 3.f;
constexpr float kMassOne = 1099511627776.f;  // mass_q of the maximum

enum Mode : uint32_t { kNothing, kGather, kGuessFirst, kSpread };

struct RowSettings {
  float T, Ts, p, floor_z;  // Ts: the softmax's temperature (1 for greedy rows)
  uint32_t k;               // 0: no top-k
  bool greedy;
};

__device__ __forceinline__ float clamp_u(float u) { return fminf(fmaxf(u, kULo), kUHi); }
// score of a kept token; false when min-p drops it
__device__ __forceinline__ bool score_of(const RowSettings& q, float d, float u, float& score) {
  const float z = __fdiv_rn(d, q.T);
  score = z - logf(-logf(clamp_u(u)));
  return z >= q.floor_z;
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
  if (q.k) tau = select_key(s, n, [&](auto f) { keys([&](uint32_t key) { f(key, 1ull); }); }, tau, top, q.k, level, above);
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

// ---- counting bf16 keys -----------------------------------------------------------
// Tokens of one bf16 value have one mass, so counts per value give both the
// k-th largest and every upper set's mass.  Bins follow the values from M down to
// the cut: a signed magnitude index, magnitudes up to H0 sharing bin 0 (their
// tokens' mass is added up apart, should there be several values).  H0 is 0, or
// M's or the cut's magnitude when both have one sign, or, where the interval
// reaches over zero, the least that leaves kCounts bins: 2^-14 or so of the
// largest magnitude.
struct KeyBins {
  uint32_t H0;
  int top;       // signed index of M
  uint32_t n;    // bins
  bool one0;     // bin 0 holds a single value

  __device__ __forceinline__ int index(uint32_t h) const {
    const int q = int(max(h & 0x7FFFu, H0) - H0);
    return (h & 0x8000u) ? -q : q;
  }
  __device__ __forceinline__ KeyBins(float M, float cut) {
    uint32_t hm = __float_as_uint(M) >> 16, hc = bf16_pair_up(cut) & 0xFFFFu;
    hm = hm == 0x8000u ? 0u : hm;
    hc = hc == 0x8000u ? 0u : hc;
    const uint32_t a = hm & 0x7FFFu, b = hc & 0x7FFFu, big = max(a, b), most = kCounts - 2;
    const uint32_t low = big > most ? big - most : 0u;
    if ((hm ^ hc) & 0x8000u) {
      H0 = max(low, a + b > most ? (a + b - most + 1) / 2 : 0u);
      one0 = H0 == 0;
    } else {
      H0 = max(low, min(a, b));
      one0 = H0 == min(a, b);
    }
    top = index(hm);
    n = uint32_t(top - index(hc)) + 1u;
  }
  __device__ __forceinline__ uint32_t bin(uint32_t h) const { return min(uint32_t(top - index(h)), n - 1u); }
  __device__ __forceinline__ bool is_odd(uint32_t i) const { return !one0 && int(i) == top; }
  // the value of bin i (of the odd bin: zero)
  __device__ __forceinline__ float value(uint32_t i) const {
    const int q = top - int(i);
    if (q == 0 && !one0) return 0.f;
    const uint32_t h = H0 + uint32_t(q < 0 ? -q : q);
    // bin 0 with a single value other than zero is M or the cut, of the sign of both
    return bf16_bits_to_float(q < 0 || (q == 0 && negative0) ? h | 0x8000u : h);
  }
  bool negative0 = false;
};

// First bin at which the running sum of weight(i) reaches target, from bin 0 to
// n - 1; n when it never does.  before: the sum above it.
template <typename Weight>
__device__ uint32_t find_bin(Shared& s, uint32_t n, unsigned long long target, Weight weight,
                             unsigned long long& before) {
  const uint32_t tid = threadIdx.x;
  unsigned long long base = 0;
  for (uint32_t from = 0; from < n; from += 4 * kThreads) {
    __syncthreads();
    if (tid == 0) s.bin = n;
    unsigned long long w[4], mine = 0;
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) {
      const uint32_t i = from + 4 * tid + q;
      w[q] = i < n ? weight(i) : 0ull;
      mine += w[q];
    }
    const unsigned long long upto = base + block_scan(mine, s.red64);
    if (tid == kThreads - 1) s.base = upto;
    if (upto >= target && upto - mine < target) {
      unsigned long long b = upto - mine;
      uint32_t i = 0;
#pragma unroll
      for (uint32_t q = 0; q < 3; ++q)
        if (i == q && b + w[q] < target) {
          b += w[q];
          ++i;
        }
      s.bin = from + 4 * tid + i;
      s.sums[0] = b;
    }
    __syncthreads();
    if (s.bin < n) {
      before = s.sums[0];
      return s.bin;
    }
    base = s.base;
  }
  before = base;
  return n;
}

// The threshold (a value) under top-k and top-p from the counts of bf16 values;
// false when it falls among the several values of the odd bin.
__device__ bool threshold_in_counts(Shared& s, const KeyBins& bins, const uint32_t* counts, unsigned long long odd,
                                    const RowSettings& q, float M, float scale, float S, float& tau) {
  auto mass = [&](uint32_t i) {
    return bins.is_odd(i) ? odd : static_cast<unsigned long long>(counts[i]) * mass_q(bins.value(i), M, scale);
  };
  uint32_t last = bins.n - 1;
  unsigned long long before, kept = mass_total(S);
  if (q.k) {
    last = min(last, find_bin(s, bins.n, q.k, [&](uint32_t i) { return static_cast<unsigned long long>(counts[i]); }, before));
    if (q.p < 1.f) {
      unsigned long long w = 0;
      for (uint32_t i = threadIdx.x; i <= last; i += kThreads) w += mass(i);
      kept = block_sum(w, s.red64b);
    }
  }
  if (q.p < 1.f) last = min(last, find_bin(s, last + 1u, mass_target(q.p, kept), mass, before));
  tau = bins.value(last);
  return !bins.is_odd(last);
}

// ... of a row whose blocks count their parts
template <int NV>
__device__ bool threshold_by_counts(Shared& s, const Held<true, NV>& h, const RowSettings& q, float cut, float M,
                                    float scale, float S, float& tau) {
  const uint32_t tid = threadIdx.x;
  KeyBins bins(M, cut);
  bins.negative0 = M < 0.f;
  const uint32_t words = (bins.n + 3u) & ~3u;
  for (uint32_t i = tid; i < words; i += kThreads) s.counts[i] = 0u;
  if (tid == 0) s.odd_mass = 0ull;
  __syncthreads();
  const uint32_t cut2 = bf16_pair_up(cut);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint32_t hits = group_ge_bits(h.v[j], cut2);
    if (!hits) continue;
    const uint32_t w[4] = {h.v[j].x, h.v[j].y, h.v[j].z, h.v[j].w};
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e)
      if ((hits >> e) & 1u) {
        const uint32_t i = bins.bin((e & 1u) ? w[e / 2] >> 16 : w[e / 2] & 0xFFFFu);
        atomicAdd(s.counts + i, 1u);
        if (bins.is_odd(i)) atomicAdd(&s.odd_mass, mass_q(group_at(h.v[j], e), M, scale));
      }
  }
  cluster_sync(h.n);
  // the whole row's counts, four bins a load
  for (uint32_t i = 4 * tid; i < words; i += 4 * kThreads) {
    uint4 t = make_uint4(0u, 0u, 0u, 0u);
    for (uint32_t r = 0; r < h.n; ++r) {
      const uint4 x = ld_remote4(at_rank(s.counts + i, r));
      t.x += x.x;
      t.y += x.y;
      t.z += x.z;
      t.w += x.w;
    }
    *reinterpret_cast<uint4*>(s.merged + i) = t;
  }
  unsigned long long odd = 0;
  if (!bins.one0)
    for (uint32_t r = 0; r < h.n; ++r) odd += ld_remote64(at_rank(&s.odd_mass, r));
  __syncthreads();
  return threshold_in_counts(s, bins, s.merged, odd, q, M, scale, S, tau);
}

// The same from the gathered list[0 .. c)
__device__ bool threshold_in_list(Shared& s, uint32_t c, const RowSettings& q, float cut, float M, float scale, float S,
                                  float& tau) {
  const uint32_t tid = threadIdx.x;
  KeyBins bins(M, cut);
  bins.negative0 = M < 0.f;
  for (uint32_t i = tid; i < bins.n; i += kThreads) s.counts[i] = 0u;
  if (tid == 0) s.odd_mass = 0ull;
  __syncthreads();
  for (uint32_t i = tid; i < c; i += kThreads) {
    const float x = fkey_inv(uint32_t(s.list[i] >> 32));
    const uint32_t at = bins.bin(__float_as_uint(x) >> 16);
    atomicAdd(s.counts + at, 1u);
    if (bins.is_odd(at)) atomicAdd(&s.odd_mass, mass_q(x, M, scale));
  }
  __syncthreads();
  return threshold_in_counts(s, bins, s.counts, s.odd_mass, q, M, scale, S, tau);
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
__device__ Drawn draw_pairs(Shared& s, uint32_t c, const RowSettings& q, float M, float scale, float S, const float* u) {
  const uint32_t tid = threadIdx.x;
  const unsigned long long e = tid < c ? s.list[tid] : 0ull;
  const float x = fkey_inv(uint32_t(e >> 32)), ut = tid < c ? u[best_id(e)] : 0.5f;
  bool stays = tid < c;
  if (q.k || q.p < 1.f) {
    s.masses[tid] = 0ull;
    place_entries<false>(s, c);
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

// Draws from this block's part, tokens >= tau, when they are too many to list:
// from -log u >= 1 - u, a score is at most z - log(1 - u), which costs one
// logarithm in the multi-function unit.  Every thread finds its two best bounds
// and scores the first exactly; a thread whose second bound reaches the block's
// best exact score scores its whole part.
template <bool BF16, int NV>
__device__ unsigned long long draw_screened(Shared& s, const Held<BF16, NV>& h, const RowSettings& q, float tau, float M,
                                            float c, const float* u) {
  constexpr uint32_t E = Fmt<BF16>::E;
  const bool wide = ((reinterpret_cast<uintptr_t>(u) / 4 - h.r.a) & 3u) == 0;
  float first = -INFINITY, second = -INFINITY, fx = 0.f;
  uint32_t ft = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int t0 = h.first_token(j);
    if (t0 >= int(h.r.V)) continue;
    float un[E];
    if (wide && t0 >= 0 && uint32_t(t0) + E <= h.r.V) {
#pragma unroll
      for (uint32_t i = 0; i < E / 4; ++i) {
        const uint4 w = ld_group(u + t0 + 4 * i);
        un[4 * i] = __uint_as_float(w.x);
        un[4 * i + 1] = __uint_as_float(w.y);
        un[4 * i + 2] = __uint_as_float(w.z);
        un[4 * i + 3] = __uint_as_float(w.w);
      }
    } else {
#pragma unroll
      for (uint32_t e = 0; e < E; ++e) un[e] = t0 + int(e) >= 0 && t0 + int(e) < int(h.r.V) ? u[t0 + int(e)] : 0.5f;
    }
#pragma unroll
    for (uint32_t e = 0; e < E; ++e) {
      const float x = elem<BF16>(h.v[j], e);
      float lg;
      asm("lg2.approx.f32 %0, %1;" : "=f"(lg) : "f"(1.f - clamp_u(un[e])));
      const float ub = x >= tau ? (x - M) * c - lg : -INFINITY;
      second = fmaxf(second, fminf(first, ub));
      if (ub > first) {
        first = ub;
        fx = x;
        ft = uint32_t(t0) + e;
      }
    }
  }
  unsigned long long best = 0ull;
  float score;
  if (first > -INFINITY && score_of(q, fx - M, u[ft], score)) best = pack_best(score, ft);
  best = block_max(best, s.red64);
  // 1e-3 covers the roundings of the bound (bounds in bits, scores in nats)
  if (second > -INFINITY && (best == 0ull || second * 0.6931472f + 1e-3f >= fkey_inv(uint32_t(best >> 32)))) {
    h.each(tau, [&](uint32_t t, float x) {
      float sc;
      if (score_of(q, x - M, u[t], sc)) best = max(best, pack_best(sc, t));
    });
  }
  return block_max(best, s.red64b);
}

template <bool BF16, int NV>
__global__ void __launch_bounds__(kThreads, NV <= 8 ? 4 : 2) draw_kernel(const DrawArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  griddep_launch_dependents();
  const uint32_t n = cluster_size(), rank = cluster_rank(), b = blockIdx.x / n, tid = threadIdx.x;
  begin(s);
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
  if (q.k >= a.V || q.greedy) q.k = 0;
  const float c = exp_scale(q.Ts);
  const uint32_t per_warp = q.k ? bounds_per_warp(q.k, n) : 0u;
  h.find_max();
  h.sum_exps(c);
  ready_others();
  h.publish(s, c, per_warp);
  if (tid < 32) {
    const bool ok = wait_sent(&s.bar_rec);
    float M, S;
    merge(s, n, c, M, S);
    // a lower bound of the threshold, and how to settle it.  Without top-k the
    // mass that top-p refers to is known, so min-p bounds what matters as well.
    const bool bad = !(q.T >= 0.f && q.T <= FLT_MAX) || p != p || mp != mp || (!q.greedy && !a.u);
    const float floor_z = logf(fminf(fmaxf(mp, 0.f), 1.f));  // -inf for min_p = 0
    float cut = -FLT_MAX, guess = 0.f;
    Mode mode = kSpread;
    if (bad || !ok || M == -INFINITY) {
      mode = kNothing;
    } else if (q.greedy) {
      cut = M;
    } else if (q.k) {
      const uint32_t key = per_warp ? bound_key(s, n * kWarps * per_warp, q.k) : 0u;
      if (key >= kKeyLowest) cut = fkey_inv(key);
      if (per_warp) mode = kGather;
    } else {
      // a little below M + T log(min_p), for the roundings
      if (floor_z > -INFINITY) {
        cut = fmaxf(M + floor_z * q.T * 1.000001f - 1e-6f * fabsf(M), -FLT_MAX);
        if (S <= kGatherCount * mp) mode = kGather;  // every kept token has at least min_p of the maximum's mass
      }
      if (q.p < 1.f) {
        const float D = logf(float(a.V) / ((1.f - q.p) * S)) + 1e-3f;
        cut = fmaxf(cut, M - D * q.T);
        if (mode != kGather && q.p * S < float(kListCap)) {
          guess = fmaxf(cut, M - fmaxf(D - kGuess, 0.f) * q.T);
          mode = kGuessFirst;
        }
      }
    }
    if (tid == 0) {
      s.M = M;
      s.S = S;
      s.cut = cut;
      s.guess = guess;
      s.floor_z = floor_z;
      s.mode = mode;
      s.late = !ok;
      if (rank == 0 && mode == kNothing) {
        if (!ok) record_error(a.status, CG_DEV_TIMEOUT);
        else if (bad) record_error(a.status, CG_DEV_BAD_PARAM);
        a.out_tok[b] = CG_NO_TOKEN;
        if (a.out_lp) a.out_lp[b] = -INFINITY;
      }
    }
  }
  __syncthreads();
  const float M = s.M, S = s.S, cut = s.cut;
  uint32_t mode = s.mode;
  if (mode == kNothing) return;
  q.floor_z = s.floor_z;
  const float* u = a.u + size_t(b) * a.ld_u;

  Drawn d;
  float list_cut = cut;
  uint32_t total = 0;
  if (mode == kGather) {
    h.gather(s, cut, false, [](float) { return 0ull; });
    if (rank != 0) return;  // its entries are with rank 0
    unsigned long long none;
    if (!h.tallied(s, total, none)) mode = kNothing;
  } else if (mode == kGuessFirst) {
    list_cut = s.guess;
    h.gather(s, list_cut, true, [&](float x) { return mass_q(x, M, c); });
    unsigned long long mass;
    const bool ok = h.tallied(s, total, mass);
    mode = !ok ? kNothing : total <= kListCap && mass >= mass_target(q.p, mass_total(S)) ? kGather : kSpread;
    if (rank != 0 && mode != kSpread) return;
  }
  // the entries are on their way to rank 0, which settles them or, after a wrong
  // guess, uses the list's memory again
  if (s.mode != kSpread && rank == 0 && (mode == kNothing || !h.listed(s, total))) {
    if (tid == 0) {
      record_error(a.status, CG_DEV_TIMEOUT);
      a.out_tok[b] = CG_NO_TOKEN;
      if (a.out_lp) a.out_lp[b] = -INFINITY;
    }
    return;
  }
  const bool gather = mode == kGather;
  if (gather) {
    if (total <= kPairCap) {
      d = draw_pairs(s, total, q, M, c, S, u);
    } else {
      // from the list, or from the row when ties have made it overflow
      const bool fits = total <= kListCap;
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
        if (!(BF16 && fits && threshold_in_list(s, total, q, list_cut, M, c, S, tau))) {
          __syncthreads();
          tau = fkey_inv(threshold_by_levels(
              s, 1, 0, [&](auto f) { entries([&](uint32_t, float x) { f(fkey(x)); }); }, q, list_cut, M, c, S));
        }
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
      if (a.out_lp) a.out_lp[b] = __fdiv_rn(d.x - M, q.Ts) - logf(S);
    }
    return;
  }

  unsigned long long best = 0ull;
  {
    float tau = cut;
    if (!q.greedy && (q.k || q.p < 1.f)) {
      bool settled = false;
      if constexpr (BF16) {
        settled = threshold_by_counts<NV>(s, h, q, cut, M, c, S, tau);
        if (!settled) cluster_sync(n);  // everybody has read the counts: the histograms take their place
      }
      if (!settled)
        tau = fkey_inv(threshold_by_levels(
            s, n, rank, [&](auto f) { h.each(cut, [&](uint32_t, float x) { f(fkey(x)); }); }, q, cut, M, c, S));
    }
    bool listed = false;
    if (q.greedy) {
      if (h.tm == M) h.each(M, [&](uint32_t t, float) { best = max(best, pack_best(0.f, t)); });
      best = block_max(best, s.red64);
    } else {
      if (tau > -FLT_MAX) {
        __syncthreads();  // s.merged has been read
        unsigned long long none;
        h.collect(s, tau, false, [](float) { return 0ull; }, none);
        __syncthreads();
        listed = s.n_local <= kListCap;
      }
      if (listed) {
        for (uint32_t i = tid; i < s.n_local; i += kThreads) {
          const unsigned long long e = s.local[i];
          float score;
          if (score_of(q, fkey_inv(uint32_t(e >> 32)) - M, u[best_id(e)], score)) best = max(best, pack_best(score, best_id(e)));
        }
        best = block_max(best, s.red64);
      } else {
        best = draw_screened<BF16, NV>(s, h, q, tau, M, c, u);
      }
    }
    if (tid == 0) send(at_rank(&s.best[rank], 0), best, at_rank(&s.bar_best, 0));
    if (!q.greedy && (q.k || q.p < 1.f)) {  // the others may still be reading this block's counts
      cluster_arrive_relaxed();
      cluster_wait();
    }
    if (rank != 0) return;
    if (tid == 0) mbar_expect_tx(&s.bar_best, n * 8u);
    if (!wait_sent(&s.bar_best)) {
      if (tid == 0) record_error(a.status, CG_DEV_TIMEOUT);
      best = 0ull;
    } else {
      for (uint32_t i = 0; i < n; ++i) best = max(best, s.best[i]);
    }
  }
  if (tid == 0) {
    const uint32_t tok = best ? best_id(best) : CG_NO_TOKEN;
    a.out_tok[b] = tok;
    if (a.out_lp) a.out_lp[b] = best ? __fdiv_rn(h.r.value(tok) - M, q.Ts) - logf(S) : -INFINITY;
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
