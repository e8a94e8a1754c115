// Sums and maxima over the 64 lanes of a wave with DPP moves (no LDS traffic, as
// lane exchanges by address have): neighbours and quads, then the mirrored quad
// and half of a row of 16, then rows 0-1 and 0-3 through the row broadcasts of
// lanes 15 and 31; lane 63 ends with the result, which every lane gets.
#pragma once

#include "common.h"

namespace beam {

// The 32-bit words of v moved by CTRL; a lane of a row outside ROWS gets `old`'s.
template <int CTRL, int ROWS = 0xF, typename F>
__device__ __forceinline__ F dpp_move(F old, F v) {
  if constexpr (sizeof(F) == 8) {
    const uint64_t o = __builtin_bit_cast(uint64_t, old), b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)o, (int)(uint32_t)b, CTRL,
                                                              ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)(o >> 32),
                                                              (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF,
                                                              false);
    return __builtin_bit_cast(F, (uint64_t)hi << 32 | lo);
  } else {
    return __builtin_bit_cast(F, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old),
                                                             __builtin_bit_cast(int, v), CTRL, ROWS, 0xF,
                                                             false));
  }
}

// v of one lane (the same lane for the whole wave), in every lane.
template <typename F>
__device__ __forceinline__ F lane_value(F v, int lane) {
  if constexpr (sizeof(F) == 8) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(F, (uint64_t)hi << 32 | lo);
  } else {
    return __builtin_bit_cast(F, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
  }
}

// op over the 16 lanes of a row, in every lane of it.
template <typename F, typename Op>
__device__ __forceinline__ F row_reduce(F v, Op op) {
  v = op(v, dpp_move<0xB1>(v, v));
  v = op(v, dpp_move<0x4E>(v, v));
  v = op(v, dpp_move<0x141>(v, v));
  return op(v, dpp_move<0x140>(v, v));
}

template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
  v = row_reduce(v, [](F a, F b) { return a + b; });
  v += dpp_move<0x142, 0xA>(F(0), v);
  v += dpp_move<0x143, 0xC>(F(0), v);
  return lane_value(v, 63);
}

// NaN lanes are passed over.
template <typename F>
__device__ __forceinline__ F wave_max(F v) {
  auto op = [](F a, F b) { return fmax(a, b); };
  v = row_reduce(v, op);
  v = op(v, dpp_move<0x142, 0xA>(v, v));
  v = op(v, dpp_move<0x143, 0xC>(v, v));
  return lane_value(v, 63);
}

}  // namespace beam
