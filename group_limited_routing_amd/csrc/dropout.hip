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

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const u32x4 a = ld16(p), b = ld16(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  } else {
    const u32x4 a = ld16(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    st16(p, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
    st16(p + 4, u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])});
  } else {
    st16(p, u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                  pack_bf16x2(v[6], v[7])});
  }
}
template <typename T>
__device__ __forceinline__ float load1(const T* p) {
  if constexpr (sizeof(T) == 4)
    return *p;
  else
    return bf16_bits_to_f32(*p);
}
template <typename T>
__device__ __forceinline__ void store1(T* p, float v) {
  if constexpr (sizeof(T) == 4)
    *p = v;
  else
    *p = (uint16_t)f32_to_bf16_bits(v);
}

// 8 elements a thread and step, one call of the generator. A lane's random words, and so
// the mask, depend on the place in the tensor alone, not on the launch. Bound by memory:
// 16384 x 5120 in bf16 58 us (x to out), 87 us with the stream, 86 us with its gradient, in fp32
// 119, 168 and 185: 5.7 to 6 TB/s, so the ten rounds of the generator cost nothing. 16 bits an
// element halve them as against 32, and put p within 2^-17.
enum Rest { kNothing, kStream, kGrad };  // what stands beside x: nothing, stream_in, keep * x

template <typename T, Rest REST>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs a) {
  const uint64_t offset = a.offset + (a.offset_dev ? (uint64_t)*a.offset_dev : 0);
  const T *px = (const T*)a.x, *ps = (const T*)a.stream_in;
  T *po = (T*)a.out, *pg = (T*)a.kept_grad;
  // a dropped value reaches nothing, an infinity or NaN neither
  auto one = [&](const u32x4& bits, int e, float x) {
    const uint32_t u = e & 1 ? bits[e >> 1] >> 16 : bits[e >> 1] & 0xffffu;
    return u >= a.border ? a.add * (x * a.scale) : 0.f;
  };
  const int64_t n8 = a.n / 8, stride = (int64_t)gridDim.x * 256;
  for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < n8; j += stride) {
    float x[8], s[8], v[8];
    load8(px + j * 8, x);
    if constexpr (REST == kStream) load8(ps + j * 8, s);
    const u32x4 bits = philox4x32((uint64_t)j, offset, a.seed);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = one(bits, e, x[e]);
      if constexpr (REST == kStream) v[e] += a.keep * s[e];
      if constexpr (REST == kGrad) s[e] = a.keep * x[e];
    }
    store8(po + j * 8, v);
    if constexpr (REST == kGrad) store8(pg + j * 8, s);
  }
  // the last n % 8, one a thread
  const int64_t i = n8 * 8 + threadIdx.x;
  if (blockIdx.x == 0 && i < a.n) {
    const float x = load1(px + i);
    float v = one(philox4x32((uint64_t)n8, offset, a.seed), threadIdx.x, x);
    if constexpr (REST == kStream) v += a.keep * load1(ps + i);
    store1(po + i, v);
    if constexpr (REST == kGrad) store1(pg + i, a.keep * x);
  }
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, int f32, hipStream_t st) {
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>((a.n / 8 + 255) / 256, 1 << 20));
  auto go = [&](auto rest) {
    constexpr Rest R = decltype(rest)::value;
    if (f32)
      dropout_kernel<float, R><<<grid, 256, 0, st>>>(a);
    else
      dropout_kernel<uint16_t, R><<<grid, 256, 0, st>>>(a);
  };
  if (a.stream_in)
    go(std::integral_constant<Rest, kStream>{});
  else if (a.kept_grad)
    go(std::integral_constant<Rest, kGrad>{});
  else
    go(std::integral_constant<Rest, kNothing>{});
  return hipGetLastError();
}

}  // namespace beam
