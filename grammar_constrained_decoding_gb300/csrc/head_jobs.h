// What a launch of the output layer's product kernel computes, and how its items are dealt out
// (kernel_head.cu).  Compiles on the host alone, where it is tested.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <vector_types.h>

#ifdef __CUDACC__
#define CG_BOTH __host__ __device__ __forceinline__
#else
#define CG_BOTH inline
#endif

namespace cgk {

// a call's arguments that all its launches read
struct HeadArgs {
  const void* hidden;
  const void* weight;
  int dtype;
  uint32_t B, V, D;
  uint64_t ld_h, ld_w;
  const uint32_t* bitmask;
  const uint32_t* target;
  float temp;
};

// What is read out of the tiles
struct LossOut {
  float2* part;              // [readers' column groups over all pieces][B]: maximum and sum without the target
  float* target_logit;       // [B], written by the tile that holds the row's target
};
struct TermsOut {
  const float* loss;
  const float* norm;
  const float* up;
};
struct GradOut {
  bool boxes;                // written (added, with `add`) as boxes of `out`; else element by element to `at`
  bool add, f32;
  uint32_t whole;            // columns that boxes write: a box ends on the 16-byte grid, whatever lies there
  void* at;                  // [m][ld]
  uint64_t ld;
};

struct Product {
  CUtensorMap a, b, out;     // operands; the terms or the gradient as they are written
  uint32_t m, n, n_m, n_n;   // extent, and in tiles
  uint32_t tile_n;           // columns of a tile: 256, or 128 or 64 where tiles are few
  uint32_t a_rows, k_rows;   // rows of a box of A where k is its width, of A and B where k is their rows
  uint32_t blocks, splits;   // stages of one product; splits of them
  int a_mn, a_k, b_mn, b_k;  // where the product begins in the maps
  GradOut grad;
};
// What a launch computes: one product, or the gradient by the hidden rows and the one by the
// weight.  Made by its constructor alone, which fills in what every launch reads: a wait that runs
// out in any of them writes to the status.
struct Job {
  Product p[2] = {};
  uint32_t early = 0;        // items of the second product that a pair without a last item of the first takes meanwhile
  // the rows' vocabulary side, and the piece
  const uint32_t* bitmask;
  uint32_t W, v0, tokens;    // words a row; the piece's first token and its tokens
  const uint32_t* target;
  float temp;
  uint32_t rows;             // of the batch
  uint32_t* status;
  LossOut loss = {};
  TermsOut terms = {};
  // the gradients: the weight from the piece's first token on
  const void* w = nullptr;
  uint64_t ld_w = 0;

  Job(const HeadArgs& a, uint32_t words, uint32_t* status_, uint32_t first, uint32_t count)
      : bitmask(a.bitmask), W(words), v0(first), tokens(count), target(a.target), temp(a.temp), rows(a.B), status(status_) {}
};

// The items of a launch, dealt out to `pairs` takers (blocks, or pairs of them) beforehand.  The
// first product's (a tile, or a split of one) go round in turn; a taker without one in the last
// round takes items of the second in that time, and from then on they go round.
template <bool TWO>
struct Turns {
  uint32_t pair, pairs, extra, mine, items, early, nth = 0;
  CG_BOTH Turns(const Job& j, uint32_t pair_, uint32_t pairs_) : pair(pair_), pairs(pairs_) {
    const uint32_t first = j.p[0].n_m * j.p[0].n_n * j.p[0].splits;
    mine = first / pairs;
    extra = first - mine * pairs;
    items = TWO ? j.p[1].n_m * j.p[1].n_n * j.p[1].splits : 0;
    early = pair < extra ? 0 : j.early;
    mine += pair < extra;
    if (TWO) head = j.early * (pairs - extra);
  }
  uint32_t head = 0;
  CG_BOTH bool next(bool& second, uint32_t& t) {
    const uint32_t i = nth++;
    second = i >= mine;
    if (!second) {
      t = pair + i * pairs;
      return true;
    }
    if (!TWO) return false;
    const uint32_t k = i - mine;
    t = k < early ? k * (pairs - extra) + pair - extra : head + (k - early) * pairs + pair;
    return t < items;
  }
};

struct Work {
  uint32_t m0, n0, split, k0, k1;
};
// An item's stages: all of them, or its split's (blocks * splits fits 32 bits)
CG_BOTH void stages_of(const Product& p, uint32_t t, Work& w) {
  w.split = 0;
  w.k0 = 0;
  w.k1 = p.blocks;
  if (p.splits > 1) {
    w.split = t / (p.n_m * p.n_n);
    w.k0 = p.blocks * w.split / p.splits;
    w.k1 = p.blocks * (w.split + 1) / p.splits;
  }
}

}  // namespace cgk
