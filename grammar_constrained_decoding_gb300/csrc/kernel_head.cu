// The output layer's cross entropy over the allowed tokens, and its gradients, with no
// logits kept (cg_head_loss, cg_head_grad).
//
//   x_bv = h_b . w_v,  m = max x,  S = sum exp((x - m) / T)  over the allowed tokens,
//   loss = log S - (x_t - m) / T = log1p(sum_{v != t} exp((x_v - x_t) / T)),
//   d_bv = g / T * exp((x_bv - m) / T) / S,  d_bt = g / T * expm1(-loss),
//   dH = d W,  dW = d^T H.
//
// All four are matrix products, and one persistent kernel runs them: tiles of 128 (or, a
// pair of blocks, 256) x 256 on the tensor cores, operands by tensor copies through a ring
// of stages, two accumulators in tensor memory so that a tile is read out while the next
// is multiplied.  What is done to a tile as it is read out makes the difference:
//   kLoss  each row's maximum and sum of exponentials over a reader's columns (target apart);
//   kTerms d, rounded to bf16, for a piece of the vocabulary: it bounds the memory;
//   kOut   a gradient's elements.
// d is rounded to bf16 because the tensor cores multiply bf16: its relative error of at most 2^-8
// is the size of the gradients' own rounding.  Float inputs, and d then, are split into
// three bf16 parts of 8 bits each, and the six products of parts that are not below 2^-24
// are summed, the five small ones apart from the large one.  Up to 8 rows of them, which wait
// for the weight alone, are multiplied without the tensor cores.
//
// Bound by the tensor cores where rows are many: 4096 x 128256 x 2048, loss and gradients, 8.6
// TFLOP with the logits twice in 5.2 ms, 1.65 PFLOP/s (a plain library product sustains 1.73 at the
// card's power limit; runs of a few hundred ms, before that is reached, take 5.1); the gradients'
// launch keeps the tensor pipe 92 % busy (2048 rows, K = 2048).  Few rows wait for the weight: 256 x
// 128256 x 4096 masked 215 us, 4.9 TB/s, the loads alone 186.  That is not the memory's limit
// (few_kernel below reads as many bytes in 153) but how they are asked for: boxes of 128 bytes out of
// each of 128 rows.  Between those, what stands in the way: an accumulator's 256 x 256 tile takes as
// many bytes a cycle from L2 as an SM can get (64), and a stage 560 to 600 cycles instead of 512.
// Figures beside the choices below are of short runs, both sides in turn.
#include <algorithm>

#include "head_jobs.h"
#include "logit_row.cuh"
#include "matrix_args.h"
#include "tensor_core.cuh"

namespace cgk {
namespace {

using namespace row;

constexpr uint32_t kTileN = 256;          // most columns of a tile
constexpr uint32_t kBlockM = 128;         // a block's rows of it
constexpr uint32_t kBlockK = 64;          // k of a stage: 128 bytes of bf16
constexpr uint32_t kReaders = 8;          // warps that read tiles out: four row quarters x two column halves
constexpr uint32_t kFirstReader = 4;      // after the copying, the multiplying and the allocating warp, and a spare
constexpr uint32_t kHeadThreads = (kFirstReader + kReaders) * 32;
constexpr uint32_t kStore = 4096;         // bytes of a box that a reader writes out: 32 rows of 128 bytes
constexpr uint32_t kBand = 16;            // row tiles that are taken together over all columns (4096 x 151936 x 1024: 714 us; 4: 758, 32: 713)
constexpr uint32_t kBoxesEach = 1;        // a reader's boxes under way (two, with a stage less, of bf16: 192 x 32000 x 2048 gradients 110.9 -> 112.5 us, the tied step 367 -> 372)
constexpr uint32_t kReadBoxes = 13, kReadElements = 32;   // stages' time that reading a gradient's tile out takes, at least
constexpr uint32_t kHeadSms = 152;

enum Readout { kLoss, kTerms, kOut };
// How a tile's stages are summed: bf16 products in one accumulator (and the next tile's in
// the other); in chains of 16 stages, added up in registers; or float matrices' six products a
// stage, in chains, the five small ones in an accumulator of their own (in the large one's they
// would each cost a step that is not rounded to nearest).  kTwo is kOne with terms of two parts:
// up to 128 rows, whose products wait for the weight, the terms keep 16 bits (rounded to 8, the one
// term that makes up a row's gradient would double its error).  Pairs of blocks would take it
// worse: 192 x 32000 x 2048 108 -> 127 us.
enum Sums { kOne, kChains, kParts, kTwo };
constexpr uint32_t products_of(Sums sums) { return sums == kParts ? 6 : sums == kTwo ? 2 : 1; }  // of a stage
// Stages of a chain.  A chain of sums in tensor memory drifts, as its steps are not rounded to
// nearest: over 16 stages (1024 k) losses are 2e-7 to 7e-7 off (in one chain of 4096 k 2.2e-6).
// 4 for float matrices (their gradients 4e-7 off against 1.1e-6, for 3 % of the time) and for few
// rows, which wait for memory: 1.0e-7 to 1.5e-7 off there on the whole (of 2, 0.7e-7 to 1.2e-7 for 1
// to 3 % of the time up to 128 rows and 14 to 17 % of 300's; of 1 no better), a lone small loss up to
// 3e-6 of itself with any of them.  16 for many (4096 x 151936 x 1024 in chains of 4: 1000 us where
// 16 take 714).
constexpr uint32_t chain_of(Sums sums, int ctas) { return sums == kParts || ctas == 1 ? 4 : 16; }

// A block's share of a stage, and how many fit beside the readers' boxes.  Float matrices' stages
// hold all three parts of both operands, and a single block's tile then has 128 columns.
template <int CTAS, Readout READ, Sums SUMS>
struct Stage {
  static constexpr uint32_t kPartsA = SUMS == kParts ? 3 : SUMS == kTwo && READ == kOut ? 2 : 1;   // the terms are A
  static constexpr uint32_t kPartsB = SUMS == kParts ? 3 : 1;
  static constexpr uint32_t kWidth = SUMS == kParts && CTAS == 1 ? 128 : kTileN;   // most columns of a tile
  static constexpr uint32_t kA = kBlockM * kBlockK * 2;                             // one part's
  static constexpr uint32_t kB = kWidth / CTAS * kBlockK * 2;
  static constexpr uint32_t kBytes = kPartsA * kA + kPartsB * kB;
  static constexpr uint32_t kBoxes = READ == kLoss ? 0 : SUMS == kTwo && READ == kTerms ? 2 : kBoxesEach;
  static constexpr uint32_t kCount = (kMaxSmem - 2048 - kReaders * kBoxes * kStore) / kBytes;
};

struct Ends {
  uint64_t full[7], empty[7], tile_full[2], tile_empty[2], drain;
  uint32_t tmem;
};

template <typename S, bool NARROW>
__device__ __forceinline__ uint32_t width(const Product& p) { return NARROW ? p.tile_n : S::kWidth; }
// Bands of row tiles over all columns: what runs at one time shares both operands in L2
template <int CTAS, typename S, bool NARROW>
__device__ __forceinline__ Work work_of(const Product& p, uint32_t t) {
  Work w;
  stages_of(p, t, w);
  t -= w.split * p.n_m * p.n_n;
  const uint32_t band = t / (kBand * p.n_n), in = t - band * kBand * p.n_n;
  const uint32_t rows = min(kBand, p.n_m - band * kBand);
  w.n0 = in / rows;
  w.m0 = (band * kBand + in - w.n0 * rows) * kBlockM * CTAS;
  w.n0 *= width<S, NARROW>(p);
  return w;
}
// the parts of the i-th of the six products of a stage; the last is the large one
__device__ __forceinline__ uint32_t part_a(uint32_t i) { return (0x001012u >> (4 * i)) & 15u; }
__device__ __forceinline__ uint32_t part_b(uint32_t i) { return (0x010210u >> (4 * i)) & 15u; }

// ---- reading a tile out ----------------------------------------------------------------------

__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// the rows' conventions: NaN is not allowed, +inf is the largest finite value
__device__ __forceinline__ float logit(float x, bool allowed) {
  return allowed ? fminf(fmaxf(x, -INFINITY), FLT_MAX) : -INFINITY;
}

// The allowed tokens of 128 columns from `col` on of row r of the piece, a word each 32
__device__ __forceinline__ void mask_words(const Job& job, uint32_t r, uint32_t col, uint32_t (&words)[4]) {
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j) {
    const uint32_t c = col + 32 * j;
    uint32_t w = c + 32 <= job.p[0].n ? 0xFFFFFFFFu : c < job.p[0].n ? (1u << (job.p[0].n - c)) - 1u : 0u;
    if (r >= job.p[0].m) w = 0;
    if (w && job.bitmask) w &= job.bitmask[size_t(r) * job.W + ((job.v0 + c) >> 5)];
    words[j] = w;
  }
}

// exp((x - m) / T) of a row as 2^(x c - r) 2^(r - m c), r the integer next to m c: one
// instruction an element in place of two, and no rounding that m shares among them.  Where
// m c is too large for that (+inf among the logits, a temperature near 0) as (x - m) c.
struct Scale {
  float c, m, r, rest;       // rest = 2^(r - m c)
  bool fast;
  __device__ __forceinline__ Scale(float c_, float m_) : c(c_), m(m_), r(rintf(m_ * c_)), rest(1.f) {
    fast = fabsf(m * c) < 1048576.f;
    if (fast) rest = ex2(-fmaf(m, c, -r));
  }
  __device__ __forceinline__ float2 at(float x, float y) const {
    return ex2_pair(__ffma2_rn(make_float2(x, y), make_float2(c, c), make_float2(-r, -r)));
  }
  __device__ __forceinline__ float2 far(float x, float y) const {
    return ex2_pair(__fmul2_rn(__fadd2_rn(make_float2(x, y), make_float2(-m, -m)), make_float2(c, c)));
  }
};

// the convention for values that are not finite, and what the mask forbids, over 32 columns
__device__ __forceinline__ void set_allowed(float* x, uint32_t word) {
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = logit(x[i], (word >> i) & 1u);
}

struct RowSum {
  float m = -INFINITY, s = 0.f;   // maximum, sum of exp((x - m) / T)
  // 32 columns; first as they are where the whole warp's are allowed, again where that met an
  // infinity or a NaN
  __device__ __forceinline__ void add(float* x, uint32_t word, float c) {
    bool plain = __all_sync(0xFFFFFFFFu, word == 0xFFFFFFFFu);
#pragma unroll 1
    for (;; plain = false) {
      if (!plain) set_allowed(x, word);
      float top = x[0], top2 = x[1];
#pragma unroll
      for (int i = 2; i < 32; i += 2) {
        top = fmaxf(top, x[i]);
        top2 = fmaxf(top2, x[i + 1]);
      }
      top = fmaxf(fmaxf(top, top2), m);
      const Scale t(c, top);
      float2 sum[2] = {};
      const bool fast = __all_sync(0xFFFFFFFFu, t.fast);
      if (fast) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) sum[(i >> 1) & 1] = __fadd2_rn(sum[(i >> 1) & 1], t.at(x[i], x[i + 1]));
      } else if (top > -INFINITY) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) sum[(i >> 1) & 1] = __fadd2_rn(sum[(i >> 1) & 1], t.far(x[i], x[i + 1]));
      }
      const float2 all = __fadd2_rn(sum[0], sum[1]);
      const float add = (all.x + all.y) * (fast ? t.rest : 1.f);
      if (plain && __any_sync(0xFFFFFFFFu, !(add <= FLT_MAX) || !(top <= FLT_MAX))) continue;
      if (top > -INFINITY) {
        s = s * (m > -INFINITY ? ex2((m - top) * c) : 0.f) + add;
        m = top;
      }
      return;
    }
  }
};

// 32 columns of a row's logits, from column `col` of the piece on
__device__ __forceinline__ void read_loss(const Job& job, float* x, uint32_t r, uint32_t col, uint32_t target, uint32_t word,
                                          float c, RowSum& sum) {
  const uint32_t at = target - (job.v0 + col);
  if (at < 32) {   // the target is apart from the others
    float xt = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (uint32_t(i) == at) {
        xt = x[i];
        x[i] = -INFINITY;
      }
    if (r < job.p[0].m) job.loss.target_logit[r] = logit(xt, (word >> at) & 1u);
  }
  __syncwarp();
  sum.add(x, word, c);
}

// A reader's box in shared memory as the copies store it: 32 rows of 128 bytes, the 16-byte
// pieces of row i exchanged by i mod 8
__device__ __forceinline__ uint32_t box_piece(uint32_t box, uint32_t row, uint32_t piece) {
  return box + row * 128 + ((piece ^ (row & 7)) << 4);
}
__device__ __forceinline__ void box_write(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// The boxes of a reader, taken in turn: a box is written again once its last copy has read it
template <uint32_t BOXES>
struct Boxes {
  uint32_t at, turn = 0;
  __device__ __forceinline__ explicit Boxes(uint32_t first) : at(first) {}
  __device__ __forceinline__ void next() {
    if ((threadIdx.x & 31) == 0) tc::stores_read<BOXES - 1>();
    __syncwarp();
    turn = turn + 1 == BOXES ? 0 : turn + 1;
  }
  __device__ __forceinline__ void all_free() const {
    if ((threadIdx.x & 31) == 0) tc::stores_read<0>();
    __syncwarp();
  }
  __device__ __forceinline__ uint32_t now() const { return at + turn * kStore; }
  template <bool ADD>
  __device__ __forceinline__ void send(const CUtensorMap* map, uint32_t x, uint32_t y, uint32_t z) const {
    tc::fence_shared();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      if (ADD) tc::add_box(map, now(), int(x), int(y), int(z));
      else tc::store_box(map, now(), int(x), int(y), int(z));
      tc::stores_commit();
    }
  }
};

// The significand of g / T of the first row that counts (its loss is above 0) and whose g / T is a
// normal number.  Terms rounded to bf16 are rounded in units of it, and the gradients multiplied by it:
// where all rows that count have one g, as under a mean, whether or not others are weighted with 0, a
// target's term -g / T (1 - p) is then near a power of two and all but exact, where g / T itself may be
// rounded by up to 2^-8, the same way in every row.  256 rows at a time; mostly the first has it.
__device__ __forceinline__ float common_scale(const Job& job) {
  constexpr uint32_t kAhead = 8;
  const uint32_t lane = threadIdx.x & 31;
#pragma unroll 1
  for (uint32_t r0 = 0; r0 < job.rows; r0 += 32 * kAhead) {
    float g[kAhead];
#pragma unroll
    for (uint32_t u = 0; u < kAhead; ++u) {
      const uint32_t r = r0 + 32 * u + lane;
      g[u] = r < job.rows && job.terms.loss[r] > 0.f ? job.terms.up ? job.terms.up[r] : 1.f : 0.f;
    }
#pragma unroll
    for (uint32_t u = 0; u < kAhead; ++u) {
      const float x = __fdiv_rn(g[u], job.temp);
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, fabsf(x) >= FLT_MIN && fabsf(x) <= FLT_MAX);
      if (who) return __uint_as_float((__shfl_sync(0xFFFFFFFFu, __float_as_uint(x), __ffs(who) - 1) & 0x007FFFFFu) | 0x3F800000u);
    }
  }
  return 1.f;
}

// d = k * exp((x - m) / T), at the target as it stands
struct RowTerms {
  Scale scale;
  float k, at_target;
  uint32_t target;           // CG_NO_TOKEN in a row that does not count
};
__device__ __forceinline__ RowTerms row_terms(const TermsOut& terms, float temp, uint32_t rows, uint32_t r, uint32_t target,
                                              float scale = 1.f) {
  const float c = exp_scale(temp);
  if (r < rows && target != CG_NO_TOKEN) {
    const float loss = terms.loss[r], m = terms.norm[2 * size_t(r)], s = terms.norm[2 * size_t(r) + 1];
    if (loss > 0.f) {   // a loss of 0: no target that counts, or nothing beside it
      Scale t(c, m);
      if (m == FLT_MAX) {   // a logit of +inf, which counts as this: not as it is, however high T
        t.fast = false;
        t.rest = 1.f;
      }
      const float g = __fdiv_rn(__fdiv_rn(terms.up ? terms.up[r] : 1.f, temp), scale);
      float k = __fdiv_rn(g, s) * t.rest;
      if (!(fabsf(k) <= FLT_MAX)) {
        // an infinite or NaN g, whose terms are not finite, but 0 for the tokens that are not allowed: as
        // exponentials that overflow, as 0 times g is NaN
        t.fast = false;
        t.m -= fmaxf(fminf(__fdiv_rn(300.f, c), 1e38f), fabsf(m) * 1e-3f);
        k = copysignf(1.f, k);
      }
      return {t, k, g * expm1f(-loss), target};
    }
  }
  return {Scale(0.f, 0.f), 0.f, 0.f, CG_NO_TOKEN};   // c = 0, k = 0: every term is 0
}
// turns 32 columns of a row's logits into its terms
__device__ __forceinline__ void set_terms(const Job& job, float* x, uint32_t col, uint32_t word, const RowTerms& t) {
  const float2 k2 = make_float2(t.k, t.k);
  const bool none = t.target == CG_NO_TOKEN;
  // as they are: all allowed, no row with a maximum out of the ordinary
  if (__all_sync(0xFFFFFFFFu, (word == 0xFFFFFFFFu || none) && t.scale.fast)) {
    float2 check = {};
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 d = __fmul2_rn(t.scale.at(x[i], x[i + 1]), k2);
      check = __fadd2_rn(check, d);
      x[i] = d.x;
      x[i + 1] = d.y;
    }
    if (!(fabsf(check.x + check.y) <= FLT_MAX)) {   // NaN among them (a row with +inf is not here: its maximum is out of the ordinary)
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = fabsf(x[i]) <= FLT_MAX ? x[i] : 0.f;
    }
  } else {
    set_allowed(x, word);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 d = __fmul2_rn(t.scale.fast ? t.scale.at(x[i], x[i + 1]) : t.scale.far(x[i], x[i + 1]), k2);
      x[i] = none ? 0.f : d.x;
      x[i + 1] = none ? 0.f : d.y;
    }
  }
  const uint32_t at = t.target - (job.v0 + col);
  if (at < 32 && !none) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (uint32_t(i) == at) x[i] = t.at_target;
  }
  __syncwarp();
}
// 32 columns as bf16: the first or the second half of a box
__device__ __forceinline__ void write_bf16(uint32_t box, uint32_t half, const float* x) {
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i)
    box_write(box_piece(box, threadIdx.x & 31, 4 * half + i), pack2(x[8 * i], x[8 * i + 1]), pack2(x[8 * i + 2], x[8 * i + 3]),
              pack2(x[8 * i + 4], x[8 * i + 5]), pack2(x[8 * i + 6], x[8 * i + 7]));
}
// 32 rows of 32 columns (chunk j of the reader's 128) on their way: bf16 boxes hold two chunks
template <uint32_t BOXES>
__device__ __forceinline__ void send_bf16(const Product& p, uint32_t whole, const float* x, uint32_t z, uint32_t row0, uint32_t col,
                                          uint32_t j, Boxes<BOXES>& boxes) {
  if (row0 >= p.m || (col & ~63u) >= p.n) return;
  if (!(j & 1u)) boxes.next();
  write_bf16(boxes.now(), j & 1u, x);
  if ((j & 1u) && (col & ~63u) < whole) boxes.template send<false>(&p.out, col & ~63u, row0, z);
}
// ... of terms in two parts: two boxes hold two chunks
template <uint32_t BOXES>
__device__ __forceinline__ void send_two(const Product& p, float* x, uint32_t row0, uint32_t col, uint32_t j,
                                         Boxes<BOXES>& boxes) {
  if (BOXES != 2 || row0 >= p.m || (col & ~63u) >= p.n) return;
  if (!(j & 1u)) boxes.all_free();
  write_bf16(boxes.at, j & 1u, x);
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] -= __bfloat162float(__float2bfloat16_rn(x[i]));
  write_bf16(boxes.at + kStore, j & 1u, x);
  if (j & 1u) {
#pragma unroll
    for (uint32_t part = 0; part < 2; ++part) {
      boxes.turn = part;
      boxes.template send<false>(&p.out, col & ~63u, row0, part);
    }
  }
}
// 64 columns of float matrices' terms: the three parts one after the other
template <uint32_t BOXES>
__device__ __forceinline__ void send_parts(const Product& p, float* x, uint32_t row0, uint32_t col, Boxes<BOXES>& boxes) {
  if (row0 >= p.m || col >= p.n) return;
#pragma unroll 1
  for (uint32_t part = 0; part < 3; ++part) {
    boxes.next();
    write_bf16(boxes.now(), 0, x);
    write_bf16(boxes.now(), 1, x + 32);
#pragma unroll
    for (int i = 0; i < 64; ++i) x[i] -= __bfloat162float(__float2bfloat16_rn(x[i]));
    boxes.template send<false>(&p.out, col, row0, part);
  }
}

// 32 x 32 elements of a gradient, as boxes; rows off the 16-byte grid element by element, a
// warp along a row
template <uint32_t BOXES>
__device__ __forceinline__ void send_grad(const Product& p, const float* x, uint32_t split, uint32_t row0, uint32_t col, uint32_t j,
                                          Boxes<BOXES>& boxes) {
  const uint32_t lane = threadIdx.x & 31;
  const GradOut& g = p.grad;
  if (g.boxes && !g.f32) {
    send_bf16(p, g.whole, x, split, row0, col, j, boxes);
    return;
  }
  if (row0 >= p.m || col >= p.n) return;
  boxes.next();
  const uint32_t box = boxes.now();
#pragma unroll
  for (uint32_t i = 0; i < 8; ++i)
    box_write(box_piece(box, lane, i), __float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
              __float_as_uint(x[4 * i + 3]));
  if (g.boxes) {
    if (g.add) boxes.template send<true>(&p.out, col, row0, split);
    else if (col < g.whole) boxes.template send<false>(&p.out, col, row0, split);
    return;
  }
  __syncwarp();
  const uint32_t rows = min(32u, p.m - row0);
  if (col + lane < p.n) {
    const uint32_t from = 4 * (lane & 3);
    size_t at = size_t(row0) * g.ld + col + lane;
#pragma unroll 1
    for (uint32_t i = 0; i < rows; i += 8) {   // eight rows' elements on their way together
      float e[8];
#pragma unroll
      for (uint32_t u = 0; u < 8; ++u)
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(e[u]) : "r"(box_piece(box, i + u, lane >> 2) + from) : "memory");
#pragma unroll
      for (uint32_t u = 0; u < 8; ++u, at += g.ld) {
        if (i + u >= rows) break;
        if (g.f32) static_cast<float*>(g.at)[at] = e[u];
        else static_cast<__nv_bfloat16*>(g.at)[at] = __float2bfloat16_rn(e[u]);
      }
    }
  }
  __syncwarp();
}

// What rounding to bf16 left of row r's term at its target, or 0 where that is not in the piece.  It is
// the row's largest term, and added times the target's row of the weight as the row's gradient is read
// out: with a g for each row 1.0 times one rounding's error in place of 1.4 to 1.5, for a read of B
// rows.  (In the gradient by the weight each reader would have to look for its tokens' rows: 192 x
// 32000 x 2048 108 -> 166 us.)
__device__ __forceinline__ float target_rest(const Job& job, uint32_t r, uint32_t target, float scale) {
  if (target - job.v0 >= job.tokens) return 0.f;
  const float loss = job.terms.loss[r];
  if (!(loss > 0.f)) return 0.f;
  const float d = __fdiv_rn(__fdiv_rn(job.terms.up ? job.terms.up[r] : 1.f, job.temp), scale) * expm1f(-loss);
  return d - __bfloat162float(__float2bfloat16_rn(d));
}
// x += e * 32 columns of a row from `col` on
__device__ __forceinline__ void add_row(float* x, float e, const __nv_bfloat16* row, uint32_t col, uint32_t columns) {
#pragma unroll
  for (uint32_t q = 0; q < 4; ++q) {
    if (col + 8 * q + 8 <= columns) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + col + 8 * q);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        x[8 * q + 2 * i] = fmaf(e, __uint_as_float(w[i] << 16), x[8 * q + 2 * i]);
        x[8 * q + 2 * i + 1] = fmaf(e, __uint_as_float(w[i] & 0xFFFF0000u), x[8 * q + 2 * i + 1]);
      }
    } else {
#pragma unroll
      for (uint32_t i = 0; i < 8; ++i)
        if (col + 8 * q + i < columns) x[8 * q + i] = fmaf(e, __bfloat162float(row[col + 8 * q + i]), x[8 * q + i]);
    }
  }
}
// What boxes leave of a gradient's rows, at most 15 bytes of each: a lane's row as it lies in the
// box that a reader of `columns` from `col` on wrote last, if that is the rows' last
__device__ __forceinline__ void send_rest(const Product& p, uint32_t box, uint32_t row0, uint32_t col, uint32_t columns) {
  const GradOut& g = p.grad;
  const uint32_t lane = threadIdx.x & 31, first = (p.n - 1) & ~(g.f32 ? 31u : 63u);
  if (first < col || first >= col + columns || row0 + lane >= p.m) return;
#pragma unroll 1
  for (uint32_t c = g.whole; c < p.n; ++c) {
    const uint32_t off = (c - first) * (g.f32 ? 4 : 2), from = box_piece(box, lane, off >> 4) + (off & 15);
    const size_t at = size_t(row0 + lane) * g.ld + c;
    uint32_t x = 0;
    if (g.f32) {
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(from) : "memory");
      static_cast<uint32_t*>(g.at)[at] = x;
    } else {
      asm volatile("ld.shared.u16 %0, [%1];" : "=r"(x) : "r"(from) : "memory");
      static_cast<uint16_t*>(g.at)[at] = uint16_t(x);
    }
  }
}

// ---- the product kernel ----------------------------------------------------------------------

// where the copying or the multiplying thread is in the ring
struct Place {
  uint32_t s = 0, phase = 0;
  template <uint32_t COUNT>
  __device__ __forceinline__ void step() {
    if (++s == COUNT) s = 0, phase ^= 1;
  }
};

// An item's stages into the ring: a block brings its 128 rows of A and its share of B's, all
// their parts.  With a pair the leader's barrier counts the bytes of both.
template <int CTAS, typename S, bool NARROW, bool A_MN, bool B_MN>
__device__ __forceinline__ bool copy_item(const Product& p, const Work& w, uint32_t rank, uint32_t ring, Ends& ends, Place& at,
                                          uint32_t& issued) {
  const uint32_t share = width<S, NARROW>(p) / CTAS;
  const uint32_t bytes = (S::kPartsA * (A_MN ? kBlockM * p.k_rows : p.a_rows * kBlockK) +
                          S::kPartsB * share * (B_MN ? p.k_rows : kBlockK)) * (2 * CTAS);
  const int am = p.a_mn + int(w.m0 + rank * kBlockM), bn = p.b_mn + int(w.n0 + rank * share);
  for (uint32_t k = w.k0; k < w.k1; ++k) {
    const int ak = p.a_k + int(k * kBlockK), bk = p.b_k + int(k * kBlockK);
    if (!mbar_wait(&ends.empty[at.s], at.phase ^ 1)) return false;
    const uint32_t full = CTAS == 2 ? tc::in_block(smem_addr(&ends.full[at.s]), 0) : smem_addr(&ends.full[at.s]);
    if (rank == 0) mbar_expect_tx(&ends.full[at.s], bytes);
    const uint32_t a = ring + at.s * S::kBytes, b = a + S::kPartsA * S::kA;
#pragma unroll
    for (uint32_t part = 0; part < S::kPartsA; ++part) {
      if (A_MN)
        for (uint32_t q = 0; q < kBlockM / 64; ++q)
          tc::copy_box<CTAS>(a + part * S::kA + q * 8192, &p.a, am + int(64 * q), ak, int(part), full);
      else tc::copy_box<CTAS>(a + part * S::kA, &p.a, ak, am, int(part), full);
    }
#pragma unroll
    for (uint32_t part = 0; part < S::kPartsB; ++part) {
      if (B_MN)
        for (uint32_t q = 0; q < share / 64; ++q)
          tc::copy_box<CTAS>(b + part * S::kB + q * 8192, &p.b, bn + int(64 * q), bk, int(part), full);
      else
        for (uint32_t q = 0; q < (share + 127) / 128; ++q)   // boxes of 128 rows, or of all where they are fewer
          tc::copy_box<CTAS>(b + part * S::kB + q * 16384, &p.b, bk, bn + int(128 * q), int(part), full);
    }
    ++issued;
    at.template step<S::kCount>();
  }
  return true;
}

// An item's products, chain after chain; n counts the chains.  Chains take the two accumulators
// in turn; the six products of a float matrices' stage take both.  FEW: where k runs over few rows,
// fewer than a stage's 64.
template <int CTAS, typename S, Sums SUMS, bool A_MN, bool B_MN, bool FEW = false>
__device__ __forceinline__ bool multiply_item(uint32_t tile_n, uint32_t k_rows, uint32_t blocks, uint32_t ring, uint32_t tmem, Ends& ends, Place& at, bool& ready,
                                              uint32_t& n) {
  const uint32_t instr = tc::instruction<A_MN, B_MN>(kBlockM * CTAS, tile_n);
  auto multiply = [&](uint32_t to, uint64_t a, uint64_t b, bool more) {
#pragma unroll
    for (uint32_t q = 0; q < kBlockK / 16; ++q)
      if (!FEW || q < k_rows / 16) tc::mma<CTAS>(to, a + q * tc::kStep16<A_MN>, b + q * tc::kStep16<B_MN>, instr, more || q != 0);
  };
  for (uint32_t k = 0; k < blocks; ++n) {
    const uint32_t end = SUMS == kOne || SUMS == kTwo ? blocks : min(blocks, k + chain_of(SUMS, CTAS));
    const uint32_t acc = SUMS == kParts ? 0u : n & 1u, round = SUMS == kParts ? n : n >> 1;
    if (!mbar_wait(&ends.tile_empty[acc], (round & 1u) ^ 1u)) return false;
    tc::fence_after_sync();
    for (bool add = false; k < end; ++k, add = true) {
      if (!ready && !mbar_wait(&ends.full[at.s], at.phase)) return false;
      tc::fence_after_sync();
      const uint64_t a = tc::operand<A_MN>(ring + at.s * S::kBytes), b = tc::operand<B_MN>(ring + at.s * S::kBytes + S::kPartsA * S::kA);
      if (SUMS == kParts) {
#pragma unroll 1
        for (uint32_t i = 0; i < 6; ++i)   // the large product last, in an accumulator of its own
          multiply(tmem + (i < 5 ? kTileN : 0u), a + part_a(i) * (S::kA >> 4), b + part_b(i) * (S::kB >> 4), add || (i != 0 && i != 5));
      } else {
        if (S::kPartsA == 2) multiply(tmem + acc * kTileN, a + (S::kA >> 4), b, add);   // the terms' second parts
        multiply(tmem + acc * kTileN, a, b, add || S::kPartsA == 2);
      }
      tc::commit<CTAS>(&ends.empty[at.s]);
      at.template step<S::kCount>();
      ready = tc::mbar_test(&ends.full[at.s], at.phase);
    }
    tc::commit<CTAS>(&ends.tile_full[acc]);
  }
  return true;
}

template <int CTAS, Readout READ, Sums SUMS, bool NARROW>
__global__ void __launch_bounds__(kHeadThreads, 1) product_kernel(const __grid_constant__ Job job) {
  using S = Stage<CTAS, READ, SUMS>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t ring = (smem_addr(smem) + 1023u) & ~1023u;   // the swizzle's pattern repeats every 1024 bytes
  const uint32_t boxes_at = ring + S::kCount * S::kBytes;
  Ends& ends = *reinterpret_cast<Ends*>(smem + (boxes_at - smem_addr(smem)) + kReaders * S::kBoxes * kStore);
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CTAS == 2 ? tc::cta_rank() : 0u;
  Turns<READ == kOut> turns(job, blockIdx.x / CTAS, gridDim.x / CTAS);
  bool second;
  uint32_t t;
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S::kCount; ++s) {
      mbar_init(&ends.full[s], 1);
      mbar_init(&ends.empty[s], 1);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(&ends.tile_full[i], 1);
      mbar_init(&ends.tile_empty[i], CTAS * kReaders);
    }
    mbar_init(&ends.drain, 1);
    tc::fence_barrier_init();
  }
  if (warp == 2) tc::tmem_alloc<CTAS>(&ends.tmem);
  tc::fence_before_sync();
  __syncthreads();
  if (CTAS == 2) tc::cluster_barrier();
  tc::fence_after_sync();
  const uint32_t tmem = ends.tmem;
  griddep_wait();

  if (warp == 0) {
    if (lane == 0) {
      // what the kernel before wrote, as the copies see it
      asm volatile("fence.proxy.async;" ::: "memory");
      Place at;
      uint32_t issued = 0;
      bool ok = true;
      while (ok && turns.next(second, t)) {
        if (READ == kOut && second) {
          ok = copy_item<CTAS, S, false, true, true>(job.p[1], work_of<CTAS, S, false>(job.p[1], t), rank, ring, ends, at, issued);
        } else {
          ok = copy_item<CTAS, S, NARROW, false, READ == kOut>(job.p[0], work_of<CTAS, S, NARROW>(job.p[0], t), rank, ring, ends, at, issued);
        }
      }
      if (!ok) {
        record_error(job.status, CG_DEV_TIMEOUT);
        // what is still in flight lands before the block leaves
        for (uint32_t i = 0; rank == 0 && i < min(issued, S::kCount); ++i) {
          if (at.s-- == 0) at.s = S::kCount - 1, at.phase ^= 1;
          if (!mbar_wait(&ends.full[at.s], at.phase)) break;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      Place at;
      uint32_t n = 0;
      bool ok = true, ready = false;   // ready: the next stage is known to have arrived
      while (ok && turns.next(second, t)) {
        Work w;
        if (READ == kOut && second) {
          stages_of(job.p[1], t, w);
          const uint32_t k_rows = job.p[1].k_rows;
          // (one loop for both: 333 x 32003 x 509 f32 296 us in place of 292)
          if (CTAS == 1 && k_rows < kBlockK)
            ok = multiply_item<CTAS, S, SUMS, true, true, CTAS == 1>(S::kWidth, k_rows, w.k1 - w.k0, ring, tmem, ends, at, ready, n);
          else
            ok = multiply_item<CTAS, S, SUMS, true, true>(S::kWidth, kBlockK, w.k1 - w.k0, ring, tmem, ends, at, ready, n);
        } else {
          stages_of(job.p[0], t, w);
          ok = multiply_item<CTAS, S, SUMS, false, READ == kOut>(width<S, NARROW>(job.p[0]), kBlockK, w.k1 - w.k0, ring, tmem, ends, at, ready, n);
        }
      }
      if (!ok) {
        record_error(job.status, CG_DEV_TIMEOUT);
        tc::commit<CTAS>(&ends.drain);   // the instructions in flight end before tensor memory is given back
        mbar_wait(&ends.drain, 0);
      }
    }
  } else if (warp >= kFirstReader) {
    const uint32_t quarter = warp & 3u, half = (warp - kFirstReader) >> 2;
    Boxes<S::kBoxes ? S::kBoxes : 1> boxes(boxes_at + (warp - kFirstReader) * S::kBoxes * kStore);
    uint32_t n = 0;
    const float c = exp_scale(job.temp);
    const float scale = READ != kLoss && SUMS == kOne ? common_scale(job) : 1.f;
    // frees the accumulator that has been read
    auto done = [&](uint32_t acc) {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (CTAS == 2) tc::arrive_at(tc::in_block(smem_addr(&ends.tile_empty[acc]), 0));
        else mbar_arrive(&ends.tile_empty[acc]);
      }
    };
    // (whether a wait ran out is the warp's to say: lanes that went on alone would read tensor memory without the others)
    auto full = [&](uint32_t i) {
      const bool there = mbar_wait(&ends.tile_full[SUMS == kParts ? 0 : i & 1u], (SUMS == kParts ? i : i >> 1) & 1u);
      if (!__all_sync(0xFFFFFFFFu, there)) {
        if (lane == 0) record_error(job.status, CG_DEV_TIMEOUT);
        return false;
      }
      tc::fence_after_sync();
      return true;
    };
    auto read_item = [&](const Product& p, bool second) {
      const Work w = work_of<CTAS, S, NARROW>(p, t);
      // the reader's columns: half of the tile's, at least 64 (the second half's readers then have none)
      const uint32_t wide = NARROW ? max(64u, p.tile_n / 2) : S::kWidth / 2;
      const uint32_t chunks = !NARROW ? S::kWidth / 64 : half * wide < p.tile_n ? wide / 32 : 0;
      const uint32_t row0 = w.m0 + rank * kBlockM + quarter * 32, r = row0 + lane, col = w.n0 + half * wide;
      const uint32_t blocks = w.k1 - w.k0;
      uint32_t words[4], target = CG_NO_TOKEN;
      const bool rows = row0 < p.m;   // the warp has rows at all
      if (READ != kOut) {
        mask_words(job, r, col, words);
        if (r < p.m) target = job.target[r];
      }
      RowSum sum;
      const RowTerms terms = READ == kTerms ? row_terms(job.terms, job.temp, job.p[0].m, r, target, scale) : RowTerms{Scale(0.f, 0.f), 0.f, 0.f, CG_NO_TOKEN};
      auto read = [&](float* x, uint32_t j, uint32_t word) {
        if (READ == kLoss) {
          read_loss(job, x, r, col + 32 * j, target, word, c, sum);
        } else if (READ == kTerms) {
          set_terms(job, x, col + 32 * j, word, terms);
          if (SUMS == kTwo) send_two(p, x, row0, col + 32 * j, j, boxes);
          else if (SUMS != kParts) send_bf16(p, p.n, x, 0, row0, col + 32 * j, j, boxes);
          else if (j & 1u) send_parts(p, x - 32, row0, col + 32 * j - 32, boxes);   // with the 32 before
        } else {
          send_grad(p, x, w.split, row0, col + 32 * j, j, boxes);
        }
      };
      const uint32_t at = tmem + half * wide + ((quarter * 32) << 16);
      if (SUMS == kChains || SUMS == kParts) {
        // the chains' sums, added up in registers; none in a split without stages
        float v[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) v[i] = 0.f;
        bool ok = true;
        for (uint32_t k = 0; k < blocks; k += chain_of(SUMS, CTAS), ++n) {
          if (!(ok = full(n))) break;
          const uint32_t acc = SUMS == kParts ? 0u : n & 1u;
#pragma unroll
          for (uint32_t q = 0; q < 4; ++q) {
            if (q >= chunks || !rows) break;
            uint32_t x[32];
            if (SUMS == kParts) {   // the small ones first
              tc::tmem_load(at + kTileN + 32 * q, x);
              tc::tmem_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[32 * q + i] += __uint_as_float(x[i]);
            }
            tc::tmem_load(at + acc * kTileN + 32 * q, x);
            tc::tmem_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[32 * q + i] += __uint_as_float(x[i]);
          }
          done(acc);
        }
        if (!ok) return false;
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
          if (j < chunks && rows) read(v + 32 * j, j, words[j]);
      } else {
        float rest = 0.f;
        const __nv_bfloat16* target_row = nullptr;
        if (READ == kOut && SUMS == kOne && !second) {
          if (w.split == 0 && r < p.m) {
            const uint32_t t = job.target[r];
            rest = target_rest(job, r, t, scale);
            target_row = static_cast<const __nv_bfloat16*>(job.w) + uint64_t(t - job.v0) * job.ld_w;
          }
          __syncwarp();
        }
        if (blocks && !full(n)) return false;
        const uint32_t acc = n & 1u;
        n += blocks != 0;
        if ((chunks == 0 || !rows) && blocks) done(acc);
#pragma unroll 1
        for (uint32_t j = 0; rows && j < chunks; ++j) {
          uint32_t x[32];
          float v[32];
          tc::tmem_load(at + acc * kTileN + 32 * j, x);
          tc::tmem_wait();
          if (j + 1 == chunks && blocks) done(acc);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(x[i]);
          if (READ == kOut && SUMS == kOne && !second) {
            if (rest != 0.f) add_row(v, rest, target_row, col + 32 * j, p.n);
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] *= READ == kOut ? scale : 1.f;
          if (!blocks) {   // a split without stages: nothing was multiplied
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
          }
          read(v, j, j == 0 ? words[0] : j == 1 ? words[1] : j == 2 ? words[2] : words[3]);
        }
      }
      if (READ == kOut && p.grad.boxes && p.grad.whole < p.n) send_rest(p, boxes.now(), row0, col, 32 * chunks);
      if (READ == kLoss && chunks && r < p.m && col < p.n)
        job.loss.part[size_t((job.v0 + col) / wide) * p.m + r] = make_float2(sum.m, sum.s);
      return true;
    };
    // (each product read where it lies: through a pointer to either the gradients' tiles took a fifth longer)
    bool ok = true;
    while (ok && turns.next(second, t)) ok = READ == kOut && second ? read_item(job.p[1], true) : read_item(job.p[0], false);
    if (READ != kLoss && lane == 0) tc::stores_done();
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (CTAS == 2) tc::cluster_barrier();   // the other block's instructions read this one's shared memory
  tc::fence_after_sync();
  if (warp == 2) tc::tmem_free<CTAS>(tmem);
}

template <int CTAS, Readout READ, Sums SUMS>
constexpr size_t product_smem() {
  using S = Stage<CTAS, READ, SUMS>;
  static_assert(S::kCount <= 7 && S::kCount >= 2, "barriers for the stages");
  return 1024 + size_t(S::kCount) * S::kBytes + size_t(kReaders) * S::kBoxes * kStore + sizeof(Ends);
}
static_assert(sizeof(Ends) <= 1024, "the ring, the boxes and the barriers fit a block's shared memory");

// ---- joining the parts of a row --------------------------------------------------------------

// 32 rows a block; its 32 warps take the column groups in turn
__global__ void __launch_bounds__(1024) join_loss_kernel(const float2* part, const float* target_logit,
                                                         const uint32_t* target, uint32_t groups, uint32_t B, uint32_t V,
                                                         float T, float* loss, float* lse, float* norm,
                                                         uint32_t* status) {
  __shared__ float2 mine[32][33];
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.x * 32 + lane;
  const float c = exp_scale(T);
  float m = -INFINITY, s = 0.f;
  if (b < B) {
    constexpr uint32_t kAhead = 8;
    for (uint32_t g0 = warp; g0 < groups; g0 += 32 * kAhead) {
      float2 x[kAhead];
      float top = m;
#pragma unroll
      for (uint32_t u = 0; u < kAhead; ++u) {
        const uint32_t g = g0 + 32 * u;
        x[u] = g < groups ? part[size_t(g) * B + b] : make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (uint32_t u = 0; u < kAhead; ++u) top = fmaxf(top, x[u].x);
      if (!(top > -INFINITY)) continue;
      float add = 0.f;
#pragma unroll
      for (uint32_t u = 0; u < kAhead; ++u) add += x[u].y * ex2((x[u].x - top) * c);   // 0 times 0 for an empty group
      s = s * (m > -INFINITY ? ex2((m - top) * c) : 0.f) + add;
      m = top;
    }
  }
  mine[warp][lane] = make_float2(m, s);
  __syncthreads();
  // each warp joins a row's 32 entries, then the first thread of each finishes its row
  const uint32_t row = blockIdx.x * 32 + warp;
  const float2 part_of_row = mine[lane][warp];
  m = warp_reduce(part_of_row.x, MaxOp());
  s = warp_reduce(m > -INFINITY ? part_of_row.y * ex2((part_of_row.x - m) * c) : 0.f, SumOp());
  if (lane != 0 || row >= B) return;
  // m, s: the others' maximum and sum; x: the target's logit
  const uint32_t t = target[row];
  if (t >= V && t != CG_NO_TOKEN) record_error(status, CG_DEV_BAD_TOKEN);
  const float x = t < V ? target_logit[row] : -INFINITY;
  float l = 0.f, M = m, rest = s;   // S = 1 + rest where the target is the maximum
  bool first = false;
  if (x > -INFINITY) {
    if (!(m > -INFINITY)) {
      M = x;
      rest = 0.f;
      first = true;
    } else if (x >= m) {
      M = x;
      rest = s * ex2((m - x) * c);
      first = true;
      l = log1pf(rest);
    } else {
      rest = s + ex2((x - m) * c);
      l = __fdiv_rn(m - x, T) + logf(rest);
    }
  }
  loss[row] = l;
  if (norm) {
    norm[2 * size_t(row)] = M;
    norm[2 * size_t(row) + 1] = first ? 1.f + rest : rest;
  }
  if (lse) lse[row] = M > -INFINITY ? __fdiv_rn(M, T) + (first ? log1pf(rest) : logf(rest)) : -INFINITY;
}

// 4 columns of a gradient's row, `left` of them in the row
__device__ __forceinline__ void put4(void* out, size_t at, uint32_t left, bool bf16, bool wide, float4 s) {
  if (wide && left >= 4) {
    if (bf16) *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) = make_uint2(pack2(s.x, s.y), pack2(s.z, s.w));
    else *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = s;
    return;
  }
  const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (uint32_t e = 0; e < 4; ++e) {
    if (e >= left) break;
    if (bf16) static_cast<__nv_bfloat16*>(out)[at + e] = __float2bfloat16_rn(v[e]);
    else static_cast<float*>(out)[at + e] = v[e];
  }
}
// The splits' sums of a gradient, added in their order.  A few splits: a thread takes 4 columns
// of all of them.
constexpr uint32_t kFewSplits = 8;
__global__ void __launch_bounds__(256) join_few_kernel(const float* sums, uint32_t ld_sums, uint32_t splits, uint32_t m,
                                                       uint32_t n, void* out, uint64_t ld, bool bf16, bool wide) {
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t groups = ld_sums / 4;
  const uint64_t i = uint64_t(blockIdx.x) * 256 + threadIdx.x;
  const uint32_t r = uint32_t(i / groups), col = 4 * uint32_t(i - uint64_t(r) * groups);
  if (r >= m || col >= n) return;
  float4 s = *reinterpret_cast<const float4*>(sums + size_t(r) * ld_sums + col);
#pragma unroll 4
  for (uint32_t k = 1; k < splits; ++k) {
    const float4 x = *reinterpret_cast<const float4*>(sums + (size_t(k) * m + r) * ld_sums + col);
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  }
  put4(out, size_t(r) * ld + col, n - col, bf16, wide, s);
}
// Many (few rows, which leave few threads): 32 groups of 4 columns to a block, whose warps take
// the splits in turn; the warps' sums are added in their order (152 splits of 127 x 192: 26 us
// the way above).
__global__ void __launch_bounds__(256) join_many_kernel(const float* sums, uint32_t ld_sums, uint32_t splits, uint32_t m,
                                                        uint32_t n, void* out, uint64_t ld, bool bf16, bool wide) {
  __shared__ float4 mine[8][32];
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t groups = ld_sums / 4, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t i = uint64_t(blockIdx.x) * 32 + lane;
  const uint32_t r = uint32_t(i / groups), col = 4 * uint32_t(i - uint64_t(r) * groups);
  const bool there = r < m && col < n;
  float4 s = {};
  if (there)
#pragma unroll 4
    for (uint32_t k = warp; k < splits; k += 8) {
      const float4 x = *reinterpret_cast<const float4*>(sums + (size_t(k) * m + r) * ld_sums + col);
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
  mine[warp][lane] = s;
  __syncthreads();
  if (warp || !there) return;
#pragma unroll
  for (uint32_t w = 1; w < 8; ++w) {
    const float4 x = mine[w][lane];
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  }
  put4(out, size_t(r) * ld + col, n - col, bf16, wide, s);
}

// ---- float matrices of few rows ----------------------------------------------------------------

// Up to 8 rows of float matrices are multiplied on the ordinary pipes as they are: reading the
// weight bounds that, and laying it out as three bf16 parts takes 16 bytes an element where this
// takes 4.  60000 x 2003, this way and by the tensor cores: loss of 1 row 92 and 442 us, of 8 127
// and 442, of 16 390 and 442 (the hidden rows no longer fit); gradients of 1 row 366 and 819, of
// 8 352 and 819, of 16 872 and 821.  128256 x 2048, 1 row: 153 us, 6.9 TB/s.
constexpr uint32_t kFewRows = 8, kFewThreads = 256, kFewBytes = 96 << 10;   // of the hidden rows at once
constexpr uint32_t few_tokens(uint32_t rows) { return rows <= 2 ? 8 : 4; }  // of a warp at once

struct FewArgs {
  const float* hidden;
  const float* weight;
  uint64_t ld_h, ld_w;
  uint32_t B, V, D, chunk;   // columns at once: a multiple of 128 unless it is all of them
  const uint32_t* bitmask;
  uint32_t W;
  const uint32_t* target;
  float temp;
  LossOut loss;              // parts by block
  TermsOut terms;
  float* d;                  // [V][ROWS]
};

// Sums N values of every lane over the lanes; lane i ends with those from i * N / 32 on (several
// lanes with the same one where N < 32)
template <uint32_t N>
__device__ __forceinline__ void sum_lanes(float (&v)[N]) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t n = N;
#pragma unroll
  for (uint32_t o = 16; o > 0; o >>= 1) {
    if (n > 1) {
      n /= 2;
      const bool upper = lane & o;
#pragma unroll
      for (uint32_t i = 0; i < N / 2; ++i)
        if (i < n) {
          const float send = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
          v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
        }
    } else {
      v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
    }
  }
}

// A warp takes a few tokens at a time, its lanes the columns; the hidden rows lie in shared
// memory.  WIDE: the weight's rows lie on the 16-byte grid.
template <uint32_t ROWS, bool WIDE, Readout READ>
__global__ void __launch_bounds__(kFewThreads, 2) few_kernel(const FewArgs a) {
  constexpr uint32_t T = few_tokens(ROWS), N = T * ROWS, kWarps = kFewThreads / 32;
  static_assert(N >= 8 && N <= 32, "a value for each lane");
  extern __shared__ __align__(16) float hidden[];   // [ROWS][chunk]
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  griddep_wait();
  // the value that a lane ends with
  const uint32_t slot = lane / (32 / N), token = slot / ROWS, r = slot % ROWS;
  const uint32_t target = r < a.B ? a.target[r] : CG_NO_TOKEN;
  const float c = exp_scale(a.temp);
  const RowTerms terms = READ == kTerms ? row_terms(a.terms, a.temp, a.B, r, target) : RowTerms{Scale(0.f, 0.f), 0.f, 0.f, CG_NO_TOKEN};
  float m = -INFINITY, s = 0.f;
  const uint32_t tiles = (a.V + kWarps * T - 1) / (kWarps * T);
  bool loaded = false;
  for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const uint32_t v0 = (tile * kWarps + warp) * T;
    const float* w[T];   // past the vocabulary its last row, whose values nobody takes
#pragma unroll
    for (uint32_t t = 0; t < T; ++t) w[t] = a.weight + min(v0 + t, a.V - 1) * a.ld_w;
    float2 acc[N];
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) acc[i] = float2{};
    for (uint32_t k0 = 0; k0 < a.D; k0 += a.chunk) {
      const uint32_t n = min(a.chunk, a.D - k0);
      if (!loaded || a.chunk < a.D) {
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < ROWS * n; i += kFewThreads) {
          const uint32_t row = i / n, k = i - row * n;
          hidden[row * a.chunk + k] = row < a.B ? a.hidden[row * a.ld_h + k0 + k] : 0.f;
        }
        loaded = true;
        __syncthreads();
      }
      const uint32_t whole = WIDE ? n & ~3u : 0u;
      if constexpr (WIDE) {
#pragma unroll 2
        for (uint32_t k = 4 * lane; k < whole; k += 128) {
          float4 x[T];
#pragma unroll
          for (uint32_t t = 0; t < T; ++t) x[t] = __ldg(reinterpret_cast<const float4*>(w[t] + k0 + k));
#pragma unroll
          for (uint32_t b = 0; b < ROWS; ++b) {
            const float4 h = *reinterpret_cast<const float4*>(hidden + b * a.chunk + k);
#pragma unroll
            for (uint32_t t = 0; t < T; ++t) {
              float2& y = acc[t * ROWS + b];
              y = __ffma2_rn(make_float2(x[t].x, x[t].y), make_float2(h.x, h.y), y);
              y = __ffma2_rn(make_float2(x[t].z, x[t].w), make_float2(h.z, h.w), y);
            }
          }
        }
      }
#pragma unroll 4
      for (uint32_t k = whole + lane; k < n; k += 32) {
        float x[T];
#pragma unroll
        for (uint32_t t = 0; t < T; ++t) x[t] = __ldg(w[t] + k0 + k);
#pragma unroll
        for (uint32_t b = 0; b < ROWS; ++b) {
          const float h = hidden[b * a.chunk + k];
#pragma unroll
          for (uint32_t t = 0; t < T; ++t) acc[t * ROWS + b].x = fmaf(x[t], h, acc[t * ROWS + b].x);
        }
      }
    }
    float x[N];
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) x[i] = acc[i].x + acc[i].y;
    sum_lanes<N>(x);
    const uint32_t v = v0 + token;
    bool allowed = v < a.V && r < a.B;
    if (allowed && a.bitmask) allowed = (a.bitmask[size_t(r) * a.W + (v >> 5)] >> (v & 31)) & 1u;
    float y = logit(x[0], allowed);
    if (READ == kLoss) {
      if (v == target && v < a.V) {   // the target is apart from the others
        a.loss.target_logit[r] = y;   // (from all lanes that hold it)
        y = -INFINITY;
      }
      if (y > -INFINITY) {
        const float top = fmaxf(m, y);
        s = s * (m > -INFINITY ? ex2((m - top) * c) : 0.f) + ex2((y - top) * c);
        m = top;
      }
    } else if (v < a.V && lane % (32 / N) == 0) {
      const float2 e = terms.scale.fast ? terms.scale.at(y, y) : terms.scale.far(y, y);
      float d = terms.target == CG_NO_TOKEN ? 0.f : e.x * terms.k;
      if (v == terms.target) d = terms.at_target;
      a.d[size_t(v) * ROWS + r] = d;
    }
  }
  if constexpr (READ == kLoss) {
    // the tokens' lanes of a row, then the warps
#pragma unroll
    for (uint32_t o = 32 / T; o < 32; o <<= 1) {
      const float m2 = __shfl_xor_sync(0xFFFFFFFFu, m, o), s2 = __shfl_xor_sync(0xFFFFFFFFu, s, o), top = fmaxf(m, m2);
      if (top > -INFINITY) s = s * ex2((m - top) * c) + s2 * ex2((m2 - top) * c);   // 0 times 0 for an empty one
      m = top;
    }
    float2(*mine)[ROWS] = reinterpret_cast<float2(*)[ROWS]>(hidden);   // the rows are done with
    __syncthreads();
    if (lane < 32 / T && lane % (32 / N) == 0) mine[warp][r] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x < a.B) {
      float top = -INFINITY, sum = 0.f;
      for (uint32_t i = 0; i < kWarps; ++i) top = fmaxf(top, mine[i][threadIdx.x].x);
      if (top > -INFINITY)
        for (uint32_t i = 0; i < kWarps; ++i) sum += mine[i][threadIdx.x].y * ex2((mine[i][threadIdx.x].x - top) * c);
      a.loss.part[size_t(blockIdx.x) * a.B + threadIdx.x] = make_float2(top, sum);
    }
  }
}

constexpr uint32_t kFewGradThreads = 128, kFewAhead = 4;
struct FewGradArgs {
  const float* hidden;
  const float* weight;
  const float* d;            // [V][ROWS]
  uint64_t ld_h, ld_w;
  uint32_t B, V, D, slabs, each;   // tokens of a block
  float* dw;                 // or none
  uint64_t ld_dw;
  float* sums;               // [blocks of tokens][B][ld_sums], or none
  uint32_t ld_sums;
};
// A thread takes 4 columns (WIDE: side by side, in one vector) over a block's tokens: grad_weight's
// elements, and its part of grad_hidden's sums
template <uint32_t ROWS, bool WIDE>
__global__ void __launch_bounds__(kFewGradThreads) few_grad_kernel(const FewGradArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t split = blockIdx.x / a.slabs, base = (blockIdx.x - split * a.slabs) * (4 * kFewGradThreads);
  const uint32_t from = split * a.each, to = min(a.V, from + a.each);
  uint32_t col[4];
  bool there[4];
#pragma unroll
  for (uint32_t q = 0; q < 4; ++q) {
    col[q] = base + (WIDE ? 4 * threadIdx.x + q : threadIdx.x + q * kFewGradThreads);
    there[q] = col[q] < a.D;
  }
  if (!there[0]) return;
  const bool wide = WIDE && there[3];
  float2 h[ROWS][2], acc[ROWS][2];
#pragma unroll
  for (uint32_t b = 0; b < ROWS; ++b)
#pragma unroll
    for (uint32_t q = 0; q < 2; ++q) {
      const float* x = a.hidden + b * a.ld_h;
      h[b][q] = make_float2(b < a.B && there[2 * q] ? x[col[2 * q]] : 0.f, b < a.B && there[2 * q + 1] ? x[col[2 * q + 1]] : 0.f);
      acc[b][q] = float2{};
    }
  for (uint32_t v0 = from; v0 < to; v0 += kFewAhead) {
    float4 w[kFewAhead];
    if (a.sums)
#pragma unroll
      for (uint32_t u = 0; u < kFewAhead; ++u) {
        if (v0 + u >= to) break;
        const float* x = a.weight + (v0 + u) * a.ld_w;
        if (wide) w[u] = __ldg(reinterpret_cast<const float4*>(x + col[0]));
        else w[u] = make_float4(x[col[0]], there[1] ? x[col[1]] : 0.f, there[2] ? x[col[2]] : 0.f, there[3] ? x[col[3]] : 0.f);
      }
#pragma unroll
    for (uint32_t u = 0; u < kFewAhead; ++u) {
      if (v0 + u >= to) break;
      float2 y[2] = {};
      const float* at = a.d + size_t(v0 + u) * ROWS;
#pragma unroll
      for (uint32_t b = 0; b < ROWS; ++b) {
        const float d = at[b];
        const float2 d2 = make_float2(d, d);
        if (a.dw) {
          y[0] = __ffma2_rn(d2, h[b][0], y[0]);
          y[1] = __ffma2_rn(d2, h[b][1], y[1]);
        }
        if (a.sums) {
          acc[b][0] = __ffma2_rn(d2, make_float2(w[u].x, w[u].y), acc[b][0]);
          acc[b][1] = __ffma2_rn(d2, make_float2(w[u].z, w[u].w), acc[b][1]);
        }
      }
      if (a.dw) {
        float* out = a.dw + (v0 + u) * a.ld_dw;
        if (wide) {
          *reinterpret_cast<float4*>(out + col[0]) = make_float4(y[0].x, y[0].y, y[1].x, y[1].y);
        } else {
          out[col[0]] = y[0].x;
          if (there[1]) out[col[1]] = y[0].y;
          if (there[2]) out[col[2]] = y[1].x;
          if (there[3]) out[col[3]] = y[1].y;
        }
      }
    }
  }
  if (a.sums)
#pragma unroll
    for (uint32_t b = 0; b < ROWS; ++b)
      if (b < a.B) {
        float* out = a.sums + (size_t(split) * a.B + b) * a.ld_sums;
        out[col[0]] = acc[b][0].x;
        if (there[1]) out[col[1]] = acc[b][0].y;
        if (there[2]) out[col[2]] = acc[b][1].x;
        if (there[3]) out[col[3]] = acc[b][1].y;
      }
}

// bf16 rows off the 16-byte grid are copied onto it; float rows are split into three parts
// that add up to the value (8 bits each; a value that is not finite is its first part).  A
// thread writes 8 columns at once.
struct Layout {
  const void* from;
  uint64_t ld;
  uint32_t rows;             // 0: not this one
  bool wide;                 // the rows lie on the 16-byte grid
  __nv_bfloat16* to;         // [parts][rows][Dp]
};
struct Layouts {
  Layout hidden, weight;
};
template <bool F32>
__global__ void __launch_bounds__(256) lay_out_kernel(const Layouts both, uint32_t D, uint32_t Dp) {
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t groups = Dp / 8;
  const uint64_t all = uint64_t(both.hidden.rows + both.weight.rows) * groups, step = uint64_t(gridDim.x) * 256;
  for (uint64_t i = uint64_t(blockIdx.x) * 256 + threadIdx.x; i < all; i += step) {
    uint64_t r = all >> 32 ? i / groups : uint32_t(i) / groups;
    const uint32_t d = uint32_t(i - r * groups) * 8;
    const bool first = r < both.hidden.rows;
    const Layout& a = first ? both.hidden : both.weight;
    if (!first) r -= both.hidden.rows;
    const uint64_t n = uint64_t(a.rows) * Dp;
    if (!F32) {
      const uint16_t* x = static_cast<const uint16_t*>(a.from) + r * a.ld + d;
      uint32_t w[4];
      if (d + 8 <= D) {
        // whole words, shifted where the row begins in the middle of one (the halves beside it
        // share a word with the row's own first or last element)
        const uint32_t* at = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(x) & ~uintptr_t(3));
        const uint32_t shift = (reinterpret_cast<uintptr_t>(x) & 2u) * 8;
        uint32_t word[5];
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) word[q] = at[q];
        word[4] = shift ? at[4] : 0u;
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) w[q] = __funnelshift_r(word[q], word[q + 1], shift);
      } else {
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q)
          w[q] = (d + 2 * q < D ? x[2 * q] : 0u) | (d + 2 * q + 1 < D ? uint32_t(x[2 * q + 1]) << 16 : 0u);
      }
      *reinterpret_cast<uint4*>(a.to + r * Dp + d) = make_uint4(w[0], w[1], w[2], w[3]);
      continue;
    }
    const float* x = static_cast<const float*>(a.from) + r * a.ld + d;
    float v[8];
    if (a.wide && d + 8 <= D) {
      const float4 lo = *reinterpret_cast<const float4*>(x), hi = *reinterpret_cast<const float4*>(x + 4);
      v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
    } else {
#pragma unroll
      for (uint32_t q = 0; q < 8; ++q) v[q] = d + q < D ? x[q] : 0.f;
    }
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      uint32_t w[4];
#pragma unroll
      for (uint32_t q = 0; q < 4; ++q) w[q] = pack2(v[2 * q], v[2 * q + 1]);
      *reinterpret_cast<uint4*>(a.to + uint64_t(part) * n + r * Dp + d) = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
      for (uint32_t q = 0; q < 8; ++q) {
        const float h = __uint_as_float(q & 1u ? w[q / 2] & 0xFFFF0000u : w[q / 2] << 16);
        v[q] = fabsf(v[q]) <= FLT_MAX && fabsf(h) <= FLT_MAX ? v[q] - h : 0.f;
      }
    }
  }
}

// ---- host ------------------------------------------------------------------------------------

// of a piece's weight laid out, and of its terms: 4096 x 128256 x 2048 in pieces of 64 MB 5.45 ms, of
// 128 5.25, of 256 5.17, of 512 0.3 % less
constexpr size_t kPieceBytes = size_t(256) << 20;

// What a call works on, and where its workspace's parts lie
struct HeadPlan {
  uint32_t B, V, D, Dp, parts, term_parts;
  bool lay_h, lay_w;
  uint32_t piece;            // tokens of a piece: a multiple of 256 unless it is all of them
  uint32_t out_n;            // columns of the gradients' tiles
  uint32_t tile_n, groups;   // columns of the logits' tiles; column groups of their readers
  uint64_t ld_terms, ld_sums;
  uint32_t splits;           // of the product that sums over tokens
  bool pair;                 // rows in pairs of blocks
  uint32_t few;              // or none of all this: few rows of float matrices, as many as this at most
  size_t at_h, at_w, at_part, at_target, at_terms, at_sums, bytes;
};

// Columns of the logits' tiles: halved, and halved again, where that takes a third of the time
// off what the tiles' rounds over all blocks take (few tiles: 95 rows of 18944 tokens in 74 tiles
// of 256 on 152 blocks).  Narrow tiles read the rows' operand more often: 4 x 48675 x 3520 in two
// rounds of 256 80 us, in three of 128 121.
uint32_t tile_width(uint32_t row_tiles, uint32_t columns, uint32_t slots, uint32_t w) {
  auto rounds = [&](uint32_t width) { return (uint64_t(row_tiles) * tiles_of(columns, width) + slots - 1) / slots; };
  while (w > 64 && 3 * rounds(w / 2) < 4 * rounds(w)) w /= 2;
  return w;
}

HeadPlan plan_head(const void* hidden, uint64_t ld_h, const void* weight, uint64_t ld_w, int dtype, uint32_t B, uint32_t V,
                   uint32_t D, bool grad) {
  HeadPlan p = {};
  p.B = B;
  p.V = V;
  p.D = D;
  p.Dp = uint32_t(up_to(D, 8));
  const bool f32 = dtype == CG_F32;
  p.few = f32 && B <= kFewRows ? B <= 2 ? std::max(B, 1u) : B <= 4 ? 4 : 8 : 0;
  if (p.few) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
      const size_t here = at;
      at += up_to(bytes, 256);
      return here;
    };
    p.groups = std::min(tiles_of(V, kFewThreads / 32 * few_tokens(p.few)), 2 * kHeadSms);
    p.ld_sums = up_to(D, 4);
    // four blocks an SM
    p.splits = std::min(std::max(1u, 4 * kHeadSms / tiles_of(D, 4 * kFewGradThreads)), tiles_of(V, 16));
    p.splits = tiles_of(V, tiles_of(V, p.splits));
    if (!grad) {
      p.at_part = take(size_t(p.groups) * B * 8);
      p.at_target = take(size_t(B) * 4);
    } else {
      p.at_terms = take(size_t(V) * p.few * 4);
      p.at_sums = take(size_t(p.splits) * B * p.ld_sums * 4);
    }
    p.bytes = at;
    return p;
  }
  p.parts = f32 ? 3 : 1;
  p.term_parts = f32 ? 3 : B <= kBlockM ? 2 : 1;
  p.lay_h = f32 || !rows_on_grid(hidden, dtype, ld_h);
  p.lay_w = f32 || !rows_on_grid(weight, dtype, ld_w);
  // rows in pairs of blocks, but not 257 to 384: three blocks pad them to 384, two pairs to 512
  // (steps in blocks and in pairs, us: 333 x 32000 x 1024 bf16 112 and 114, 300 x 32003 x 509 bf16 114 and
  // 126, 300 x 128256 x 2048 bf16 645 and 667; float matrices, 333 x 32003 x 509 301 and 370, 257 x
  // 128256 x 2048 4140 and 4970)
  p.pair = B > kBlockM && !(B > 2 * kBlockM && B <= 3 * kBlockM);
  uint64_t most = V;
  if (p.lay_w) most = std::min<uint64_t>(most, kPieceBytes / (uint64_t(p.parts) * p.Dp * 2));
  if (grad) most = std::min<uint64_t>(most, kPieceBytes / (uint64_t(p.term_parts) * std::max(B, 1u) * 2));
  if (most < V) most = std::max<uint64_t>(most / 256 * 256, 256);
  const uint64_t pieces = (V + most - 1) / most;
  p.piece = uint32_t(std::min<uint64_t>(up_to((V + pieces - 1) / pieces, 256), V));
  const uint32_t slots = kHeadSms / (p.pair ? 2 : 1);
  p.out_n = p.parts > 1 && !p.pair ? 128 : kTileN;
  p.tile_n = tile_width(tiles_of(B, kBlockM * (p.pair ? 2 : 1)), p.piece, slots, p.out_n);
  p.groups = tiles_of(V, std::max(64u, p.tile_n / 2));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up_to(bytes, 256);
    return here;
  };
  if (p.lay_h) p.at_h = take(size_t(p.parts) * B * p.Dp * 2);
  if (p.lay_w) p.at_w = take(size_t(p.parts) * p.piece * p.Dp * 2);
  if (!grad) {
    p.at_part = take(size_t(p.groups) * B * 8);
    p.at_target = take(size_t(B) * 4);
  } else {
    p.ld_terms = up_to(p.piece, 8);
    p.at_terms = take(size_t(p.term_parts) * B * p.ld_terms * 2);
    p.ld_sums = up_to(D, 4);
    const uint32_t tiles = tiles_of(B, kBlockM * (p.pair ? 2 : 1)) * tiles_of(D, p.out_n);
    const uint32_t blocks = tiles_of(p.piece, kBlockK);
    p.splits = std::max(1u, std::min(slots / std::max(tiles, 1u), blocks / 8));
    if (p.splits > 1 || p.piece < V) p.at_sums = take(size_t(p.splits) * B * p.ld_sums * 4);
  }
  p.bytes = at;
  return p;
}

template <int CTAS, Readout READ, Sums SUMS, bool NARROW>
cudaError_t launch_job(int device, Job& j, cudaStream_t stream) {
  if (!j.status) return cudaErrorInvalidValue;   // where a wait that runs out writes
  uint32_t items[2] = {0, 0}, longest[2] = {0, 0};
  for (int i = 0; i < (READ == kOut ? 2 : 1); ++i) {
    Product& p = j.p[i];
    if (!p.splits) continue;   // not wanted
    p.n_m = tiles_of(p.m, kBlockM * CTAS);
    p.n_n = tiles_of(p.n, p.tile_n);
    items[i] = p.n_m * p.n_n * p.splits;
    // in stages; a tile of few is as long as it takes to read out and write
    if (items[i]) longest[i] = std::max(tiles_of(p.blocks, p.splits) * products_of(SUMS), p.grad.boxes ? kReadBoxes : kReadElements);
  }
  // what one item of the first product is worth in items of the second
  j.early = longest[1] ? (longest[0] + longest[1] / 2) / longest[1] : 0;
  return launch_clusters<product_kernel<CTAS, READ, SUMS, NARROW>>(device, std::min(items[0] + items[1], kHeadSms / CTAS), CTAS,
                                                             kHeadThreads, product_smem<CTAS, READ, SUMS>(), stream, j);
}
// Results in 32 bits are summed in chains: losses, and all that float matrices give.
template <int CTAS, Readout READ, bool NARROW>
cudaError_t launch_job(int device, const HeadPlan& p, Job& j, cudaStream_t stream) {
  if (p.parts > 1) return launch_job<CTAS, READ, kParts, NARROW>(device, j, stream);
  if (READ == kLoss)
    return j.p[0].blocks > chain_of(kChains, CTAS) ? launch_job<CTAS, READ, READ == kLoss ? kChains : kOne, NARROW>(device, j, stream)
                                                   : launch_job<CTAS, READ, kOne, NARROW>(device, j, stream);
  if (CTAS == 1 && p.term_parts == 2)
    return launch_job<CTAS, READ, CTAS == 1 && READ != kLoss ? kTwo : kOne, NARROW>(device, j, stream);
  return launch_job<CTAS, READ, kOne, NARROW>(device, j, stream);
}
template <Readout READ>
cudaError_t launch_job(int device, const HeadPlan& p, Job& j, cudaStream_t stream) {
  if (READ != kOut && p.tile_n < p.out_n)
    return p.pair ? launch_job<2, READ, READ != kOut>(device, p, j, stream) : launch_job<1, READ, READ != kOut>(device, p, j, stream);
  return p.pair ? launch_job<2, READ, false>(device, p, j, stream) : launch_job<1, READ, false>(device, p, j, stream);
}

// the operands as the tensor copies read them: the caller's, or laid out in the workspace
struct Operands {
  const void* h;
  const void* w;
  uint64_t ld_h, ld_w;
};
// The hidden rows (with the first piece) and a piece's n rows of the weight from v0 on, laid out
// where that is needed
cudaError_t lay_out(const HeadArgs& a, const HeadPlan& p, uint32_t v0, uint32_t n, unsigned char* ws, Operands& o,
                    cudaStream_t stream) {
  const bool f32 = a.dtype == CG_F32;
  Layouts both = {};
  uint32_t rows = 0;
  if (p.lay_h && v0 == 0) {
    both.hidden = Layout{a.hidden, a.ld_h, p.B, rows_on_grid(a.hidden, a.dtype, a.ld_h),
                       reinterpret_cast<__nv_bfloat16*>(ws + p.at_h)};
    o.h = ws + p.at_h;
    o.ld_h = p.Dp;
    rows += p.B;
  }
  if (p.lay_w) {
    both.weight = Layout{static_cast<const char*>(a.weight) + uint64_t(v0) * a.ld_w * dtype_size(a.dtype), a.ld_w, n,
                       rows_on_grid(a.weight, a.dtype, a.ld_w), reinterpret_cast<__nv_bfloat16*>(ws + p.at_w)};
    o.w = ws + p.at_w;
    o.ld_w = p.Dp;
    rows += n;
  }
  if (!rows) return cudaSuccess;
  const dim3 grid(uint32_t(std::min<uint64_t>((uint64_t(rows) * (p.Dp / 8) + 255) / 256, 1u << 30)));
  return launch_dependent(f32 ? lay_out_kernel<true> : lay_out_kernel<false>, grid, dim3(256), 0, stream, both, p.D, p.Dp);
}
bool map_h(CUtensorMap* map, const HeadPlan& p, const Operands& o, uint32_t box) {
  return tc::make_map(map, o.h, p.D, p.B, p.parts, o.ld_h, p.lay_h ? uint64_t(p.B) * p.Dp : o.ld_h, box);
}
bool map_w(CUtensorMap* map, const HeadPlan& p, const Operands& o, uint32_t rows, uint32_t box) {
  return tc::make_map(map, o.w, p.D, rows, p.parts, o.ld_w, p.lay_w ? uint64_t(rows) * p.Dp : o.ld_w, box);
}

// rows of the weight's boxes: a block's share of a tile's, at most 128
uint32_t b_rows(const HeadPlan& p) { return std::min(128u, p.tile_n / (p.pair ? 2 : 1)); }
// and of the hidden rows', or the terms': where they are few, what lies past them in the tile stays
// as it is (it reaches only rows that are not there).  Copies that fill whole boxes with zeros held
// up 152 blocks that all read the same few rows: 1 x 128256 x 4096 221 -> 178 us, 16 rows alike
uint32_t h_rows(const HeadPlan& p) { return std::min<uint32_t>(kBlockM, uint32_t(up_to(p.B, 8))); }
// x = H W^T of a piece, read out one way or the other
Job logits_of(const HeadArgs& a, const HeadPlan& p, const CtxView& v, uint32_t v0, uint32_t n) {
  Job j(a, v.t.W, v.t.status, v0, n);
  Product& q = j.p[0];
  q.m = p.B;
  q.n = n;
  q.blocks = tiles_of(p.D, kBlockK);
  q.splits = 1;
  q.tile_n = p.tile_n;
  q.a_rows = h_rows(p);
  q.b_mn = p.lay_w ? 0 : int(v0);
  return j;
}

template <uint32_t ROWS, Readout READ>
cudaError_t launch_few(int device, const HeadPlan& p, FewArgs& f, cudaStream_t stream) {
  f.chunk = uint32_t(std::min<uint64_t>(up_to(f.D, 4), kFewBytes / (ROWS * 4) / 128 * 128));
  const size_t smem = size_t(ROWS) * std::max(f.chunk * 4, kFewThreads / 32 * 8);
  return rows_on_grid(f.weight, CG_F32, f.ld_w)
             ? launch_clusters<few_kernel<ROWS, true, READ>>(device, p.groups, 1, kFewThreads, smem, stream, f)
             : launch_clusters<few_kernel<ROWS, false, READ>>(device, p.groups, 1, kFewThreads, smem, stream, f);
}
template <uint32_t ROWS>
cudaError_t launch_few_grad(const HeadPlan& p, const FewGradArgs& f, cudaStream_t stream) {
  const bool wide = (!f.sums || rows_on_grid(f.weight, CG_F32, f.ld_w)) && (!f.dw || rows_on_grid(f.dw, CG_F32, f.ld_dw));
  return launch_dependent(wide ? few_grad_kernel<ROWS, true> : few_grad_kernel<ROWS, false>, dim3(f.slabs * p.splits),
                          dim3(kFewGradThreads), 0, stream, f);
}
template <Readout READ>
cudaError_t launch_few(int device, const HeadPlan& p, FewArgs& f, cudaStream_t stream) {
  switch (p.few) {
    case 1: return launch_few<1, READ>(device, p, f, stream);
    case 2: return launch_few<2, READ>(device, p, f, stream);
    case 4: return launch_few<4, READ>(device, p, f, stream);
    default: return launch_few<8, READ>(device, p, f, stream);
  }
}
cudaError_t launch_few_grad(const HeadPlan& p, const FewGradArgs& f, cudaStream_t stream) {
  switch (p.few) {
    case 1: return launch_few_grad<1>(p, f, stream);
    case 2: return launch_few_grad<2>(p, f, stream);
    case 4: return launch_few_grad<4>(p, f, stream);
    default: return launch_few_grad<8>(p, f, stream);
  }
}
FewArgs few_args(const HeadArgs& a, const CtxView& v) {
  FewArgs f = {};
  f.hidden = static_cast<const float*>(a.hidden);
  f.weight = static_cast<const float*>(a.weight);
  f.ld_h = a.ld_h;
  f.ld_w = a.ld_w;
  f.B = a.B;
  f.V = a.V;
  f.D = a.D;
  f.bitmask = a.bitmask;
  f.W = v.t.W;
  f.target = a.target;
  f.temp = a.temp;
  return f;
}

int head_loss(cg_ctx* c, const HeadArgs& a, const HeadPlan& p, float* loss, float* lse, float* norm, unsigned char* ws) {
  DeviceGuard dg(ctx_device(c), "cg_head_loss");
  if (!dg.ok) return CG_E_CUDA;
  const CtxView v = ctx_view(c);
  const int dev = ctx_device(c);
  const LossOut out{reinterpret_cast<float2*>(ws + p.at_part), reinterpret_cast<float*>(ws + p.at_target)};
  Operands o{a.hidden, a.weight, a.ld_h, a.ld_w};
  if (p.few) {
    FewArgs f = few_args(a, v);
    f.loss = out;
    if (launch_few<kLoss>(dev, p, f, v.stream) != cudaSuccess) return CG_E_CUDA;
  }
  for (uint32_t v0 = 0; !p.few && v0 < p.V; v0 += p.piece) {
    const uint32_t n = std::min(p.piece, p.V - v0);
    if (lay_out(a, p, v0, n, ws, o, v.stream) != cudaSuccess) return CG_E_CUDA;
    Job j = logits_of(a, p, v, v0, n);
    j.loss = out;
    if (!map_h(&j.p[0].a, p, o, h_rows(p)) || !map_w(&j.p[0].b, p, o, p.lay_w ? n : p.V, b_rows(p))) return CG_E_CUDA;
    if (launch_job<kLoss>(dev, p, j, v.stream) != cudaSuccess) return CG_E_CUDA;
  }
  return launch_dependent(join_loss_kernel, dim3(tiles_of(p.B, 32)), dim3(1024), 0, v.stream,
                          static_cast<const float2*>(out.part), static_cast<const float*>(out.target_logit), a.target,
                          p.groups, p.B, p.V, a.temp, loss, lse, norm, v.t.status) == cudaSuccess
             ? CG_OK
             : CG_E_CUDA;
}

// where a product's elements go: [rows][ld] at `to`
bool grad_out(Product& g, void* to, uint32_t rows, uint64_t ld, int dtype) {
  g.grad.f32 = dtype == CG_F32;
  g.grad.whole = g.n & ~(g.grad.f32 ? 3u : 7u);
  g.grad.boxes = rows_on_grid(to, dtype, ld) && g.grad.whole;
  g.grad.at = to;
  g.grad.ld = ld;
  return !g.grad.boxes || tc::make_map(&g.out, to, g.grad.whole, rows, 1, ld, ld, 32, g.grad.f32);
}

int head_grad(cg_ctx* c, const HeadArgs& a, const HeadPlan& p, const float* loss, const float* norm, const float* up, void* dh, uint64_t ld_dh,
              void* dw, uint64_t ld_dw, unsigned char* ws) {
  DeviceGuard dg(ctx_device(c), "cg_head_grad");
  if (!dg.ok) return CG_E_CUDA;
  const CtxView v = ctx_view(c);
  const int dev = ctx_device(c);
  const bool f32 = a.dtype == CG_F32;
  const size_t size = f32 ? 4 : 2;
  if (a.B == 0)  // no rows: the weight's gradient is zero
    return !dw || cudaMemset2DAsync(dw, ld_dw * size, 0, size_t(a.D) * size, a.V, v.stream) == cudaSuccess ? CG_OK
                                                                                                            : CG_E_CUDA;
  Operands o{a.hidden, a.weight, a.ld_h, a.ld_w};
  __nv_bfloat16* terms = reinterpret_cast<__nv_bfloat16*>(ws + p.at_terms);
  const uint64_t part_stride = uint64_t(p.B) * p.ld_terms;
  // the hidden rows' gradient is summed over pieces and splits in 32 bits where there are several
  const bool summed = p.few || p.splits > 1 || p.piece < p.V;
  float* sums = reinterpret_cast<float*>(ws + p.at_sums);
  if (p.few) {
    FewArgs f = few_args(a, v);
    f.terms = TermsOut{loss, norm, up};
    f.d = reinterpret_cast<float*>(ws + p.at_terms);
    if (launch_few<kTerms>(dev, p, f, v.stream) != cudaSuccess) return CG_E_CUDA;
    FewGradArgs g = {};
    g.hidden = f.hidden;
    g.weight = f.weight;
    g.d = f.d;
    g.ld_h = a.ld_h;
    g.ld_w = a.ld_w;
    g.B = a.B;
    g.V = a.V;
    g.D = a.D;
    g.slabs = tiles_of(a.D, 4 * kFewGradThreads);
    g.each = tiles_of(a.V, p.splits);
    g.dw = static_cast<float*>(dw);
    g.ld_dw = ld_dw;
    g.sums = dh ? sums : nullptr;
    g.ld_sums = uint32_t(p.ld_sums);
    if (launch_few_grad(p, g, v.stream) != cudaSuccess) return CG_E_CUDA;
  }
  for (uint32_t v0 = 0; !p.few && v0 < p.V; v0 += p.piece) {
    const uint32_t n = std::min(p.piece, p.V - v0);
    if (lay_out(a, p, v0, n, ws, o, v.stream) != cudaSuccess) return CG_E_CUDA;
    const uint32_t w_rows = p.lay_w ? n : p.V;
    Job j = logits_of(a, p, v, v0, n);
    j.terms = TermsOut{loss, norm, up};
    if (!map_h(&j.p[0].a, p, o, h_rows(p)) || !map_w(&j.p[0].b, p, o, w_rows, b_rows(p)) ||
        !tc::make_map(&j.p[0].out, terms, n, p.B, p.term_parts, p.ld_terms, part_stride, 32))
      return CG_E_CUDA;
    if (launch_job<kTerms>(dev, p, j, v.stream) != cudaSuccess) return CG_E_CUDA;

    Job g(a, v.t.W, v.t.status, v0, n);
    g.terms = j.terms;
    g.w = static_cast<const __nv_bfloat16*>(o.w) + (p.lay_w ? 0 : uint64_t(v0) * o.ld_w);   // (float matrices' is not read)
    g.ld_w = o.ld_w;
    if (dh) {  // terms [B][n] x W [n][D], summed over the pieces
      Product& q = g.p[0];
      q.m = p.B;
      q.n = p.D;
      q.blocks = tiles_of(n, kBlockK);
      q.splits = p.splits;
      q.tile_n = p.out_n;
      q.a_rows = h_rows(p);
      q.k_rows = kBlockK;
      q.b_k = p.lay_w ? 0 : int(v0);
      if (summed) {
        q.grad.boxes = q.grad.f32 = true;
        q.grad.add = v0 != 0;
        q.grad.whole = p.D;   // the workspace's rows end on the grid
        if (!tc::make_map(&q.out, sums, p.D, p.B, p.splits, p.ld_sums, uint64_t(p.B) * p.ld_sums, 32, true)) return CG_E_CUDA;
      } else if (!grad_out(q, dh, p.B, ld_dh, a.dtype)) {
        return CG_E_CUDA;
      }
      if (!tc::make_map(&q.a, terms, n, p.B, p.term_parts, p.ld_terms, part_stride, h_rows(p)) || !map_w(&q.b, p, o, w_rows, 64))
        return CG_E_CUDA;
    }
    if (dw) {  // terms^T [n][B] x H [B][D]
      Product& q = g.p[1];
      q.m = n;
      q.n = p.D;
      q.blocks = tiles_of(p.B, kBlockK);
      q.splits = 1;
      q.tile_n = p.out_n;
      q.k_rows = std::min<uint32_t>(kBlockK, uint32_t(up_to(p.B, 16)));   // zeros past the rows, to a whole step of k
      if (!grad_out(q, static_cast<char*>(dw) + uint64_t(v0) * ld_dw * size, n, ld_dw, a.dtype)) return CG_E_CUDA;
      if (!tc::make_map(&q.a, terms, n, p.B, p.term_parts, p.ld_terms, part_stride, q.k_rows) || !map_h(&q.b, p, o, q.k_rows)) return CG_E_CUDA;
    }
    if (launch_job<kOut>(dev, p, g, v.stream) != cudaSuccess) return CG_E_CUDA;
  }
  if (!dh || !summed) return CG_OK;
  const uint64_t groups = p.B * (p.ld_sums / 4);
  const bool wide = rows_on_grid(dh, a.dtype, ld_dh);
  const bool few = p.splits <= kFewSplits;
  const cudaError_t e = launch_dependent(few ? join_few_kernel : join_many_kernel, dim3(tiles_of(groups, few ? 256 : 32)),
                                         dim3(256), 0, v.stream, static_cast<const float*>(sums), uint32_t(p.ld_sums), p.splits,
                                         p.B, p.D, dh, ld_dh, !f32, wide);
  return e == cudaSuccess ? CG_OK : CG_E_CUDA;
}

int head_args(const cg_ctx* c, const HeadArgs& a) {
  if (!c || (a.dtype != CG_F32 && a.dtype != CG_BF16) || a.V != ctx_view(c).t.V || a.D == 0) return CG_E_ARG;
  if (!matrix_ok(a.hidden, a.dtype, a.B, a.D, a.ld_h) || !matrix_ok(a.weight, a.dtype, a.V, a.D, a.ld_w)) return CG_E_ARG;
  if ((a.B && !a.target) || !aligned4(a.target) || !aligned4(a.bitmask)) return CG_E_ARG;
  if (!(a.temp > 0.f) || a.temp > FLT_MAX) return CG_E_ARG;
  return a.B > kMaxMatrixRows || a.D > kMaxMatrixWidth ? CG_E_LIMIT : CG_OK;
}
}  // namespace
}  // namespace cgk

extern "C" int cg_head_workspace(const cg_ctx* c, const void* d_hidden, const void* d_weight, int dtype, uint32_t B,
                                 uint32_t V, uint32_t D, uint64_t ld_hidden, uint64_t ld_weight, int grad, size_t* bytes) {
  using namespace cgk;
  if (!c || !bytes || (dtype != CG_F32 && dtype != CG_BF16) || V != ctx_view(c).t.V || D == 0) return CG_E_ARG;
  if (!matrix_ok(d_hidden, dtype, B, D, ld_hidden) || !matrix_ok(d_weight, dtype, V, D, ld_weight)) return CG_E_ARG;
  if (B > kMaxMatrixRows || D > kMaxMatrixWidth) return CG_E_LIMIT;
  *bytes = B == 0 ? 0 : plan_head(d_hidden, ld_hidden, d_weight, ld_weight, dtype, B, V, D, grad != 0).bytes;
  return CG_OK;
}

extern "C" int cg_head_loss(cg_ctx* c, const void* d_hidden, const void* d_weight, int dtype, uint32_t B, uint32_t V,
                            uint32_t D, uint64_t ld_hidden, uint64_t ld_weight, const uint32_t* d_bitmask,
                            const uint32_t* d_target, float temp, float* d_out_loss, float* d_out_lse, float* d_out_norm,
                            void* d_workspace, size_t workspace_bytes) {
  using namespace cgk;
  const HeadArgs a{d_hidden, d_weight, dtype, B, V, D, ld_hidden, ld_weight, d_bitmask, d_target, temp};
  const int rc = head_args(c, a);
  if (rc != CG_OK) return rc;
  if (B == 0) return CG_OK;
  if (!d_out_loss || !aligned4(d_out_loss) || !aligned4(d_out_lse) || !aligned4(d_out_norm)) return CG_E_ARG;
  const HeadPlan p = plan_head(d_hidden, ld_hidden, d_weight, ld_weight, dtype, B, V, D, false);
  if (!d_workspace || reinterpret_cast<uintptr_t>(d_workspace) % 256) return CG_E_ARG;
  if (workspace_bytes < p.bytes) return CG_E_NOMEM;
  return head_loss(c, a, p, d_out_loss, d_out_lse, d_out_norm, static_cast<unsigned char*>(d_workspace));
}

extern "C" int cg_head_grad(cg_ctx* c, const void* d_hidden, const void* d_weight, int dtype, uint32_t B, uint32_t V,
                            uint32_t D, uint64_t ld_hidden, uint64_t ld_weight, const uint32_t* d_bitmask,
                            const uint32_t* d_target, float temp, const float* d_loss, const float* d_norm,
                            const float* d_grad_loss, void* d_out_grad_hidden, uint64_t ld_grad_hidden,
                            void* d_out_grad_weight, uint64_t ld_grad_weight, void* d_workspace, size_t workspace_bytes) {
  using namespace cgk;
  const HeadArgs a{d_hidden, d_weight, dtype, B, V, D, ld_hidden, ld_weight, d_bitmask, d_target, temp};
  const int rc = head_args(c, a);
  if (rc != CG_OK) return rc;
  if (!d_out_grad_hidden && !d_out_grad_weight) return CG_E_ARG;
  if (B && (!d_loss || !d_norm)) return CG_E_ARG;
  if (!aligned4(d_loss) || !aligned4(d_norm) || !aligned4(d_grad_loss)) return CG_E_ARG;
  const uint64_t size = dtype == CG_BF16 ? 2 : 4;
  const void* out[2] = {d_out_grad_hidden, d_out_grad_weight};
  const uint64_t rows[2] = {B, V}, ld[2] = {ld_grad_hidden, ld_grad_weight};
  for (int i = 0; i < 2; ++i) {
    if (!out[i]) continue;
    if (!matrix_ok(out[i], dtype, rows[i], D, ld[i]) || matrices_meet(out[i], rows[i], ld[i], d_hidden, B, ld_hidden, D, size) ||
        matrices_meet(out[i], rows[i], ld[i], d_weight, V, ld_weight, D, size))
      return CG_E_ARG;
  }
  if (out[0] && out[1] && matrices_meet(out[0], rows[0], ld[0], out[1], rows[1], ld[1], D, size)) return CG_E_ARG;
  const HeadPlan p = plan_head(d_hidden, ld_hidden, d_weight, ld_weight, dtype, B, V, D, true);
  if (B && (!d_workspace || reinterpret_cast<uintptr_t>(d_workspace) % 256)) return CG_E_ARG;
  if (B && workspace_bytes < p.bytes) return CG_E_NOMEM;
  return head_grad(c, a, p, d_loss, d_norm, d_grad_loss, d_out_grad_hidden, ld_grad_hidden, d_out_grad_weight,
                   ld_grad_weight, static_cast<unsigned char*>(d_workspace));
}
