// What the tiled products of the operators share: compile-time loops, scalar base
// addresses, LDS swizzles and the order of tiles over the XCDs.
#pragma once

#include "common.h"

namespace beam {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// source of what a tile loads past an operand's end
static __device__ __align__(16) const uint8_t kZeros[16] = {};

// A pointer that is the same in every lane, kept in scalar registers: loads
// from it plus a 32-bit lane offset then need one vector register each.
__device__ __forceinline__ const uint8_t* scalar(const uint8_t* p) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm("" : "+s"(p));
#endif
  return p;
}

// f(0), f(1), ..., f(N - 1) with compile-time arguments.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void for_each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    for_each<N, I + 1>(f);
  }
}

// LDS rows of a reduction step of 128: E4M3 128 bytes, 16-byte chunk c of row r
// at position c ^ ((r >> 1) & 7); E2M1 64 bytes, chunk c at c ^ ((r >> 2) & 3).
// A 16-byte read is served 16 lanes at a time, 0-3, 12-15 and 20-27 of the first
// 32 and then the rest of them: with these keys each such group covers all 64
// banks (c ^ (r & 7) and c ^ ((r >> 1) & 3) conflicted on every read). Operands have no
// conflicts by the counters; the tiles' scale dwords, 32 rows at a pitch of 16 bytes,
// have 6 cycles each, up to 36 a wave and stage.
template <int ROW>
__device__ __forceinline__ int swizzle(int row) {
  return ROW == 64 ? (row >> 2) & 3 : (row >> 1) & 7;
}

// Tiles that run together on one XCD (32 consecutive, dealt to the XCDs in
// turn) cover 4 token tiles x 8 weight tiles, which share operands in its L2.
__device__ __forceinline__ void tile_of(int b, int n_tiles, int mt, int nt, int& m, int& n) {
  constexpr int R = 256, GM = 4;
  if (b < n_tiles / R * R) {
    const int q = b >> 3;
    b = ((q / 32) * 8 + (b & 7)) * 32 + q % 32;
  } else {
    // the last, partial round: each XCD takes consecutive tiles too
    const int b0 = n_tiles / R * R, n = n_tiles - b0, x = (b - b0) & 7, q = (b - b0) >> 3;
    b = b0 + x * (n / 8) + min(x, n % 8) + q;
  }
  const int mb = b / (GM * nt), rem = b - mb * GM * nt;
  const int gm = min(GM, mt - mb * GM);
  n = rem / gm;
  m = mb * GM + rem % gm;
}

}  // namespace beam
