// What a launch of the output layer's product kernel computes (kernel_head.cu).  No device
// code: compiles on the host alone.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <vector_types.h>

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

}  // namespace cgk
