// Dropout whose mask is never stored: element i of the flattened rows is kept by
// 16 bits of a counter-based generator at (seed, offset, i), so the backward pass
// draws the same bits again.
//
// Generator: Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011), counter (i / 8 as 64 bits, offset as 64
// bits), key seed. A call gives four words, 16 bits for each of 8 elements: element
// i takes half i % 2 of word (i % 8) / 2.
#include "common.h"
#include "operators.h"

#include <algorithm>

namespace beam {
namespace {

__device__ __forceinline__ u32x4 philox4x32(uint64_t j, uint64_t offset, uint64_t seed) {
  uint32_t c0 = (uint32_t)j, c1 = (uint32_t)(j >> 32);
  uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
    c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)q;
    c3 = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

__device__ __forceinline__ float value(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float value(const uint16_t* p, int64_t i) { return bf16_bits_to_f32(p[i]); }
__device__ __forceinline__ void put(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void put(uint16_t* p, int64_t i, float v) { p[i] = (uint16_t)f32_to_bf16_bits(v); }

template <typename T>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs a) {
  const uint64_t offset = a.offset + (a.offset_dev ? (uint64_t)*a.offset_dev : 0);
  const int64_t n8 = (a.n + 7) / 8, stride = (int64_t)gridDim.x * 256;
  for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < n8; j += stride) {
    const u32x4 bits = philox4x32((uint64_t)j, offset, a.seed);
    for (int e = 0; e < 8 && j * 8 + e < a.n; ++e) {
      const int64_t i = j * 8 + e;
      const uint32_t u = (bits[e >> 1] >> (16 * (e & 1))) & 0xffffu;
      const float x = value((const T*)a.x, i);
      // a dropped value reaches nothing, an infinity or NaN neither
      float v = u >= a.border ? a.add * (x * a.scale) : 0.f;
      if (a.stream_in) v += a.keep * value((const T*)a.stream_in, i);
      put((T*)a.out, i, v);
      if (a.kept_grad) put((T*)a.kept_grad, i, a.keep * x);
    }
  }
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, int f32, hipStream_t st) {
  const unsigned grid = (unsigned)std::min<int64_t>((a.n + 2047) / 2048, 1 << 20);
  if (f32)
    dropout_kernel<float><<<grid, 256, 0, st>>>(a);
  else
    dropout_kernel<uint16_t><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace beam
