// Host checks and sizes shared by the calls that take matrices (rows at any pitch).
#pragma once

#include <cstdint>

#include "../../include/cg.h"

namespace cgk {

constexpr uint32_t kMaxMatrixRows = 1u << 22, kMaxMatrixWidth = 1u << 16;  // numbers of tiles and of a row's elements fit 32 bits

inline uint64_t up_to(uint64_t x, uint64_t n) { return (x + n - 1) / n * n; }
inline uint32_t tiles_of(uint64_t x, uint32_t n) { return uint32_t((x + n - 1) / n); }
inline uint64_t dtype_size(int dtype) { return dtype == CG_BF16 ? 2 : 4; }

inline bool matrix_ok(const void* at, int dtype, uint64_t rows, uint32_t D, uint64_t ld) {
  return ld >= D && ld <= (uint64_t(1) << 32) && (rows == 0 || at) &&
         reinterpret_cast<uintptr_t>(at) % dtype_size(dtype) == 0;
}
// Whether two matrices of D columns share memory: their byte ranges meet, and they are not
// columns of one buffer side by side.
inline bool matrices_meet(const void* x, uint64_t nx, uint64_t ldx, const void* y, uint64_t ny, uint64_t ldy, uint32_t D,
                          uint64_t size) {
  if (!nx || !ny) return false;
  if (nx == 1) ldx = ldy;   // the pitch of one row is nobody's
  if (ny == 1) ldy = ldx;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  const uint64_t width = D * size;
  if (a + (nx - 1) * ldx * size + width <= b || b + (ny - 1) * ldy * size + width <= a) return false;
  if (ldx != ldy) return true;
  const uint64_t pitch = ldx * size, off = (b > a ? b - a : pitch - (a - b) % pitch) % pitch;
  return off < width || pitch - off < width;
}

}  // namespace cgk
