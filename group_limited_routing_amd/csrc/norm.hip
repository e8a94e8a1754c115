// RMS norm of the residual stream, with the stream's own update and an E4M3
// output, and its gradient.
//
// Beam launch post ("Introducing Beam"), section "Residual Stream", and the
// transformers model doc "Beam", section "Overview": every sublayer reads the
// RMS norm of the stream (sandwich norm), the stream is depth scaled, and the
// norm is computed in fp32 or better. Per row of H values:
//   s = keep * stream_in + add * x        r = 1 / sqrt(mean(s^2) + eps)
//   y = s r w
// One pass over memory: a row stays in the registers of the threads that
// loaded it from its load to its last use.
#include "common.h"
#include "operators.h"
#include "wave.h"

#include <algorithm>

namespace beam {
namespace {

// ------------------------------------------------------------------ rows
// A row is held by NT threads, V units of 8 values each: unit j of thread i is the
// chunk i + j NT, read and written whole. kVec (H a multiple of 8): every row, so
// every chunk, is 16-byte aligned. Else a chunk starts at any element, which the
// memory unit allows, and the row's last one is taken value by value; of fp32 rows
// a unit is then 8 / CH chunks of CH values, NT chunks apart, so that neighbouring
// lanes read neighbouring bytes. Odd rows, us, value by value and in chunks:
//   bf16, 8192 x 5001: row scales 293 and 83, without 162 and 76, gradient 263 and 142
//   fp32, 4096 x 5001: row scales 169 and 71 (chunks of 4); the gradient, which
//   also writes fp32 partials, 90 and 96 (chunks of 8: 107), so it takes single values
enum Form { kVec, kAny, kFour, kOne };
template <Form F>
constexpr int kChunk = F == kFour ? 4 : F == kOne ? 1 : 8;
// The element that value u of a unit is; u a multiple of the chunk.
template <Form F>
__device__ __forceinline__ int elem(int tid, int nt, int j, int u = 0) {
  constexpr int CH = kChunk<F>;
  return (tid + (j * (8 / CH) + u / CH) * nt) * CH;
}

// 8 raw values of a row: bf16 pairs or fp32.
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
  u32x4 v;
  __device__ __forceinline__ float get(int u) const {
    return (u & 1) ? __uint_as_float(v[u >> 1] & 0xffff0000u) : __uint_as_float(v[u >> 1] << 16);
  }
  __device__ __forceinline__ void set(int u, uint16_t b) {
    if (u & 1)
      v[u >> 1] |= (uint32_t)b << 16;
    else
      v[u >> 1] = b;
  }
  __device__ __forceinline__ void load(const uint16_t* p) { v = ld16(p); }
  __device__ __forceinline__ void load_any(const uint16_t* p) { __builtin_memcpy(&v, p, 16); }
  // From here on the values are unpacked again from the packed form: their fp32
  // forms are not kept in registers across the row's reduction.
  __device__ __forceinline__ void repack() {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+v"(v));
#endif
  }
};
template <>
struct Raw<float> {
  u32x4 lo, hi;
  __device__ __forceinline__ float get(int u) const {
    return __uint_as_float(u < 4 ? lo[u & 3] : hi[u & 3]);
  }
  __device__ __forceinline__ void set(int u, float f) {
    if (u < 4)
      lo[u & 3] = __float_as_uint(f);
    else
      hi[u & 3] = __float_as_uint(f);
  }
  __device__ __forceinline__ void load(const float* p) {
    lo = ld16(p);
    hi = ld16(p + 4);
  }
  __device__ __forceinline__ void load_any(const float* p) {
    __builtin_memcpy(&lo, p, 16);
    __builtin_memcpy(&hi, p + 4, 16);
  }
  __device__ __forceinline__ void repack() {}
};

// Unit j of the row at p; values past the row read as 0.
template <Form F, typename T>
__device__ __forceinline__ Raw<T> load_unit(const T* p, int tid, int nt, int j, int H) {
  Raw<T> r;
  if constexpr (F == kFour) {
#pragma unroll
    for (int h = 0; h < 8; h += 4) {
      const int e = elem<F>(tid, nt, j, h);
      u32x4 v{};
      if (e + 4 <= H) {
        __builtin_memcpy(&v, p + e, 16);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = e + u < H ? __float_as_uint(p[e + u]) : 0u;
      }
      (h ? r.hi : r.lo) = v;
    }
  } else if constexpr (F == kOne) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int e = elem<F>(tid, nt, j, u);
      r.set(u, e < H ? p[e] : T(0));
    }
  } else {
    const int e = elem<F>(tid, nt, j);
    if (F == kVec ? e < H : e + 8 <= H) {
      if constexpr (F == kVec)
        r.load(p + e);
      else
        r.load_any(p + e);
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u) r.set(u, F != kVec && e + u < H ? p[e + u] : T(0));
    }
  }
  return r;
}

__device__ __forceinline__ float load_value(const float* p) { return *p; }
__device__ __forceinline__ float load_value(const uint16_t* p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ void store_value(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_value(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16_bits(v); }

template <Form F>
__device__ __forceinline__ void store16(void* p, u32x4 v) {
  if constexpr (F == kVec)
    st16(p, v);
  else
    __builtin_memcpy(p, &v, 16);
}

template <Form F, typename T>
__device__ __forceinline__ void store_unit(T* p, int tid, int nt, int j, int H, const float (&v)[8]) {
  constexpr int CH = kChunk<F>;
#pragma unroll
  for (int h = 0; h < 8; h += CH) {
    const int e = elem<F>(tid, nt, j, h);
    if constexpr (CH == 1) {
      if (e < H) store_value(p + e, v[h]);
    } else if (F == kVec ? e < H : e + CH <= H) {
      if constexpr (sizeof(T) == 2) {
        store16<F>(p + e, u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])});
      } else {
#pragma unroll
        for (int u = h; u < h + CH; u += 4)
          store16<F>(p + e + u - h, u32x4{__float_as_uint(v[u]), __float_as_uint(v[u + 1]),
                                          __float_as_uint(v[u + 2]), __float_as_uint(v[u + 3])});
      }
    } else if (F != kVec) {
#pragma unroll
      for (int u = 0; u < CH; ++u)
        if (e + u < H) store_value(p + e + u, v[h + u]);
    }
  }
}

// ------------------------------------------------------------------ sums
// Sum / maximum over the row's waves, in every thread: wave results through
// LDS in wave order (the same order for every thread and every run).
template <bool MAX, typename F>
__device__ __forceinline__ F block_reduce(F v, F* lds, int nwaves) {
  v = MAX ? wave_max(v) : wave_sum(v);
  if (nwaves == 1) return v;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  F s = lds[0];
  for (int i = 1; i < nwaves; ++i) s = MAX ? (lds[i] > s ? lds[i] : s) : s + lds[i];
  return s;
}

// Rows whose mean square, with eps, lies outside of [2^-40, 2^100]: there fp32 sums of
// squares may have overflowed or vanished (rows of 1e20, of 1e-25 with eps = 0), and
// 1 / rms may not be a normal number. Such a row's sums are done over in fp64, and it
// goes on as s p, with p a power of two that brings it near 1, and f = 1 / (p rms); 0,
// infinity and NaN come out as they are. (fp64 sums of every row cost the gradient of
// 16384 x 5120 bf16 168 -> 181 us, of 65536 x 256 39 -> 47 us; so they stay at 168.5
// and 39. Rows of more than 16384 values, which spill, pay 1 to 13%.)
__device__ __forceinline__ bool fp32_range(float mean_sq) { return mean_sq > 0x1p-40f && mean_sq < 0x1p100f; }
struct InvRms {
  float p, f;
};
// 2^e as a double, |e| < 1022
__device__ __forceinline__ double power2(int e) { return __builtin_bit_cast(double, (uint64_t)(1023 + e) << 52); }
__device__ __forceinline__ InvRms inv_rms(double mean_sq) {
  // mean_sq = 4^k m with m in [1, 4); p = 2^-k as far as fp32 has normal numbers
  const int e = (int)(__builtin_bit_cast(uint64_t, mean_sq) >> 52 & 0x7ff) - 1023;
  const int k = min(max(e >> 1, -160), 160), c = min(max(-k, -126), 127);
  return {(float)power2(c), (float)power2(-k - c) / sqrtf((float)(mean_sq * power2(-2 * k)))};
}

// ------------------------------------------------------------------ E4M3
// fp64 -> fp32 rounded to odd: the value cut after 24 bits, its last bit set
// if anything was cut, so that a later rounding to few bits decides as from
// the fp64 value itself. Below 2^-126 the result is 0 (far under half of the
// smallest E4M3 value).
__device__ __forceinline__ float round_to_odd(double d) {
  const uint64_t b = __builtin_bit_cast(uint64_t, d);
  const uint32_t hi = (uint32_t)(b >> 32), lo = (uint32_t)b, mag = hi & 0x7fffffffu;
  if (mag < (897u << 20)) return 0.0f;
  const uint32_t sticky = (lo & 0x1fffffffu) ? 1u : 0u;
  return __uint_as_float((hi & 0x80000000u) | ((mag - (896u << 20)) << 3) | (lo >> 29) | sticky);
}

// Eight values, each at most 448 in magnitude after the clamp, to E4M3 codes
// (round to nearest even, one instruction per pair).
__device__ __forceinline__ u32x2 e4m3x8(const float (&v)[8]) {
  u32x2 out;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = fminf(fmaxf(v[4 * h + i], -448.0f), 448.0f);
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w, true);
    out[h] = (uint32_t)w;
  }
  return out;
}

// ------------------------------------------------------------------ forward
// The 8-bit outputs are decided in fp64 (QUANT != 0): a code is the nearest
// to the exact quotient, not to one with an fp32 rounding on either side of a
// border. fp64 runs at the unpacked fp32 rate here and the kernel is bound by
// memory. Without an 8-bit output everything is fp32 (see fp32_range).
// Bound by memory where there are many rows: 8192 x 5120 bf16 with the stream's
// update, E4M3 blocks and no bf16 output 58-61 us on warm inputs, 66 on cold ones (295
// MB, 4.5-5.0 TB/s; a large copy reaches 5.2; what follows is warm). Few rows wait for one row's chain of loads and two reductions:
// 64 x 5120 with row scales and a bf16 output 5.6 us, one row 3.2 us. Narrow rows
// with an 8-bit output are bound by fp64: 65536 x 256 45 us, 22 us without. Odd
// rows: 8192 x 5001 83 us with row scales, 76 us without an 8-bit output.
template <typename T, bool VEC, int V, int QUANT>
__global__ __launch_bounds__(V == 8 ? 1024 : 512) void add_rms_norm_kernel(NormArgs p, int nt) {
  using A = typename std::conditional<QUANT != 0, double, float>::type;
  constexpr Form F = VEC ? kVec : sizeof(T) == 2 ? kAny : kFour;
  __shared__ A lds[2][16];
  const int nwaves = nt >> 6;
  // rows of one wave: four of them in a workgroup
  const int row = nt == 64 ? blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6) : blockIdx.x;
  if (row >= p.T) return;
  const int tid = nt == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int H = p.H;
  const size_t off = (size_t)row * H;

  Raw<T> xr[V], sr[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    xr[j] = load_unit<F, T>((const T*)p.x + off, tid, nt, j, H);
    if (p.stream_in) sr[j] = load_unit<F, T>((const T*)p.stream_in + off, tid, nt, j, H);
  }
  A s[V][8], sq = 0;
  const A keep = p.keep, add = p.add;
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      A h = add * (A)xr[j].get(u);
      if (p.stream_in) h += keep * (A)sr[j].get(u);
      s[j][u] = h;
      sq += h * h;
    }
  if (p.stream_out) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = (float)s[j][u];
      store_unit<F>((T*)p.stream_out + off, tid, nt, j, H, v);
    }
  }
  sq = block_reduce<false>(sq, lds[0], nwaves);
  A r;
  if constexpr (QUANT) {
    r = 1.0 / sqrt(sq / H + (double)p.eps);
  } else {
    const float v = sq / H + p.eps;
    r = 1.0f / sqrtf(v);
    if (!fp32_range(v)) {  // the same for the whole row
      double sq2 = 0;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int u = 0; u < 8; ++u) sq2 += (double)s[j][u] * s[j][u];
      __shared__ double lds2[16];
      const InvRms ir = inv_rms(block_reduce<false>(sq2, lds2, nwaves) / H + p.eps);
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int u = 0; u < 8; ++u) s[j][u] *= ir.p;
      r = ir.f;
    }
  }

  // s becomes s w; y = r (s w)
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const Raw<float> w = load_unit<F, float>(p.w, tid, nt, j, H);
#pragma unroll
    for (int u = 0; u < 8; ++u) s[j][u] *= (A)w.get(u);
    if (p.y) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = (float)(s[j][u] * r);
      store_unit<F>((T*)p.y + off, tid, nt, j, H, v);
    }
  }
  if constexpr (QUANT == 1) {
    // one scale per row, amax / 448; r is common to all of a row's values, so
    // y 448 / amax|y| = (s w) 448 / amax|s w|. An infinity or NaN among them makes
    // the scale a NaN: no code stands for one, and the maximum passes over a NaN.
    double m = 0;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const double a = fabs(s[j][u]);
        m = a > m ? a : m;
        bad |= a != a;
      }
    if (bad) m = INFINITY;
    m = block_reduce<true>(m, lds[1], nwaves);
    const double ym = m * r;
    const bool zero = m == 0;
    const double inv = zero ? 0.0 : 448.0 / m;
    if (tid == 0)
      ((float*)p.q_scale)[row] = !(m < INFINITY) ? NAN : zero && ym == ym ? 1.0f : (float)(ym / 448.0);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = round_to_odd(s[j][u] * inv);
      const u32x2 c = e4m3x8(v);
      constexpr int CH = kChunk<F>;
#pragma unroll
      for (int h = 0; h < 8; h += CH) {
        const int e = elem<F>(tid, nt, j, h);
        if (F == kVec ? e < H : e + CH <= H) {
          if constexpr (F == kVec)
            *reinterpret_cast<u32x2*>(p.q + off + e) = c;
          else
            __builtin_memcpy(p.q + off + e, (const char*)&c + h, CH);
        } else if (F != kVec) {
#pragma unroll
          for (int u = h; u < h + CH; ++u)
            if (e + u - h < H) p.q[off + e + u - h] = (uint8_t)(c[u >> 2] >> (8 * (u & 3)));
        }
      }
    }
  }
  if constexpr (QUANT == 2) {
    // One E8M0 scale per 32 values (four neighbouring lanes): the power of two
    // that brings the block's largest binade to E4M3's own, 2^8; values that
    // still pass 448 become 448. The exponent of the maximum is the maximum of
    // the exponents, so only the high words are compared.
#pragma unroll
    for (int j = 0; j < V; ++j) {
      double y[8];
      uint32_t top = 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        y[u] = s[j][u] * r;
        const uint32_t hi = (uint32_t)(__builtin_bit_cast(uint64_t, y[u]) >> 32) & 0x7fffffffu;
        top = hi > top ? hi : top;
      }
      top = max(top, dpp_move<0xB1>(top, top));
      top = max(top, dpp_move<0x4E>(top, top));
      const int be = (int)(top >> 20);  // biased exponent; 0x7ff: infinity or NaN in the block
      const int e = min(max(be - 1023 - 8, -127), 127);
      const double inv = __builtin_bit_cast(double, (uint64_t)(1023 - e) << 52);
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = round_to_odd(y[u] * inv);
      u32x2 c = e4m3x8(v);
      if (be == 0x7ff) c = u32x2{0x7f7f7f7fu, 0x7f7f7f7fu};
      const int at = elem<F>(tid, nt, j);
      if (at < H) {
        *reinterpret_cast<u32x2*>(p.q + off + at) = c;
        if ((tid & 3) == 0)
          ((uint8_t*)p.q_scale)[(size_t)row * (H / 32) + at / 32] =
              be == 0x7ff ? (uint8_t)255 : (uint8_t)(e + 127);
      }
    }
  }
}

// ------------------------------------------------------------------ backward
// With g = dy w and n = s r:
//   ds = d_stream_out + r (g - n mean(g n)),  dx = add ds,  d_stream_in = keep ds,
//   dw = sum over rows of dy n.
// A workgroup walks the rows b, b + gridDim.x, ...; it keeps its partial dw in
// registers over all of them and writes it once (norm_dw_kernel adds the
// partials in order: no atomics). The rows stay packed across the reduction
// (repack), so that three of them and the partial fit in registers.
// Bound by memory: 16384 x 5120 bf16, five arrays of 168 MB, 154-172 us with the
// weight gradient (4.9-5.4 TB/s, one card and another) and 141-149 us without; odd
// rows, 8192 x 5001 bf16, 142-155 us.
// Rows over 16384 values need more registers than their threads have and spill: 512
// x 65536 373 us (five arrays of 67 MB; 343 before rare rows had sums of their own).
// bf16 rows of two units are held to five waves a SIMD (96 registers), which the sums
// over again of rare rows would take them from: 16384 x 5120 168.5 us so and 172.5
// without, 64 x 5120 7.3 and 7.0.
template <typename T, bool VEC, int V>
constexpr int kBwdWaves = VEC && V == 2 && sizeof(T) == 2 ? 5 : V == 8 ? 4 : 2;
template <typename T, bool VEC, int V, bool DW>
__global__ __launch_bounds__(V == 8 ? 1024 : 512)
__attribute__((amdgpu_waves_per_eu(kBwdWaves<T, VEC, V>)))
void add_rms_norm_bwd_kernel(NormBwdArgs p, int nt) {
  constexpr Form F = VEC ? kVec : sizeof(T) == 2 ? kAny : kOne;
  __shared__ float lds[2][2][16];  // double buffered over rows: one barrier per row
  __shared__ double lds2[2][2][16];
  const int nwaves = nt >> 6;
  const int per = nt == 64 ? (blockDim.x >> 6) : 1;  // rows side by side in the workgroup
  const int tid = nt == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int first = nt == 64 ? blockIdx.x * per + (threadIdx.x >> 6) : blockIdx.x;
  const int H = p.H;

  Raw<float> w[V];
  float dw[DW ? V : 1][8];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    w[j] = load_unit<F, float>(p.w, tid, nt, j, H);
    if (DW)
#pragma unroll
      for (int u = 0; u < 8; ++u) dw[DW ? j : 0][u] = 0.f;
  }
  int buf = 0;
  for (int row = first; row < p.T; row += gridDim.x * per, buf ^= 1) {
    const size_t off = (size_t)row * H;
    Raw<T> s[V], dy[V], d[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s[j] = load_unit<F, T>((const T*)p.s + off, tid, nt, j, H);
      dy[j] = load_unit<F, T>((const T*)p.dy + off, tid, nt, j, H);
      if (p.d_stream_out)
        d[j] = load_unit<F, T>((const T*)p.d_stream_out + off, tid, nt, j, H);
      else
        d[j] = Raw<T>{};
    }
    float sq = 0.f, gs = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float sv = s[j].get(u);
        sq += sv * sv;
        gs += dy[j].get(u) * w[j].get(u) * sv;
      }
    sq = wave_sum(sq);
    gs = wave_sum(gs);
    if (nwaves > 1) {
      if ((threadIdx.x & 63) == 0) {
        lds[buf][0][threadIdx.x >> 6] = sq;
        lds[buf][1][threadIdx.x >> 6] = gs;
      }
      __syncthreads();
      sq = lds[buf][0][0];
      gs = lds[buf][1][0];
      for (int i = 1; i < nwaves; ++i) {
        sq += lds[buf][0][i];
        gs += lds[buf][1][i];
      }
    }
    const float v = sq / H + p.eps;
    float r = 1.0f / sqrtf(v), scale = 1.f;
    float c = gs * r / H;  // mean(g n)
    if (!fp32_range(v) || !(fabsf(gs) < 0x1p120f)) {  // the same for the whole row
      // read again value by value: units would need registers that every row pays for.
      // (All of the row's reads are behind the barrier before its first store.)
      double sq2 = 0, gs2 = 0;
#pragma unroll 1
      for (int e = tid; e < H; e += nt) {
        const double sv = load_value((const T*)p.s + off + e);
        sq2 += sv * sv;
        gs2 += (double)(load_value((const T*)p.dy + off + e) * p.w[e]) * sv;
      }
      sq2 = wave_sum(sq2);
      gs2 = wave_sum(gs2);
      if (nwaves > 1) {
        if ((threadIdx.x & 63) == 0) {
          lds2[buf][0][threadIdx.x >> 6] = sq2;
          lds2[buf][1][threadIdx.x >> 6] = gs2;
        }
        __syncthreads();
        sq2 = lds2[buf][0][0];
        gs2 = lds2[buf][1][0];
#pragma unroll 1
        for (int i = 1; i < nwaves; ++i) {
          sq2 += lds2[buf][0][i];
          gs2 += lds2[buf][1][i];
        }
      }
      const InvRms ir = inv_rms(sq2 / H + p.eps);
      scale = ir.p;
      r = ir.f;
      c = (float)(gs2 * scale * r / H);
    }
    scale = lane_value(scale, 0);
    r = lane_value(r, 0);
    c = lane_value(c, 0);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s[j].repack();
      dy[j].repack();
      d[j].repack();
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float a[8], b[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float n = s[j].get(u) * scale * r, g = dy[j].get(u);
        float ds = r * (g * w[j].get(u) - n * c) * scale;
        ds += d[j].get(u);
        if (DW) dw[DW ? j : 0][u] += g * n;
        a[u] = p.add * ds;
        b[u] = p.keep * ds;
      }
      store_unit<F>((T*)p.dx + off, tid, nt, j, H, a);
      if (p.d_stream_in) store_unit<F>((T*)p.d_stream_in + off, tid, nt, j, H, b);
    }
  }
  if (DW) {
    float* out = p.part + (size_t)blockIdx.x * H;
    if constexpr (V == 1) {  // rows of one wave have one unit: the waves' sums are added
      __shared__ float side[4][8][64];
      if (nt == 64) {
        const int wave = threadIdx.x >> 6;
#pragma unroll
        for (int u = 0; u < 8; ++u) side[wave][u][tid] = dw[0][u];
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int u = 0; u < 8; ++u)
          for (int i = 1; i < per; ++i) dw[0][u] += side[i][u][tid];
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) store_unit<F>(out, tid, nt, j, H, dw[DW ? j : 0]);
  }
}

// dw[c] = sum over the groups of part[group, c]: 32 columns per workgroup, 32
// shares of the groups side by side, added in order. 768 partials of 5120 values
// (16 MB, from L2 and the last-level cache) 4.5 us.
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* __restrict__ part, int groups,
                                                       int H, float* __restrict__ dw) {
  __shared__ float lds[32][33];
  const int cl = threadIdx.x & 31, q = threadIdx.x >> 5, c = blockIdx.x * 32 + cl;
  float s = 0.f;
  if (c < H) {
    int g = q;
    for (; g + 96 < groups; g += 128) {  // four loads in flight
      const float a = part[(size_t)g * H + c], b = part[(size_t)(g + 32) * H + c];
      const float d = part[(size_t)(g + 64) * H + c], e = part[(size_t)(g + 96) * H + c];
      s += a;
      s += b;
      s += d;
      s += e;
    }
    for (; g < groups; g += 32) s += part[(size_t)g * H + c];
  }
  lds[q][cl] = s;
  __syncthreads();
  if (q == 0 && c < H) {
    for (int i = 1; i < 32; ++i) s += lds[i][cl];
    dw[c] = s;
  }
}

// ------------------------------------------------------------------ launch shape
// Threads of a row and units of 8 values per thread: the fewest units (1, 2,
// 4, 8) whose threads, a whole number of waves, are at most `most`.
struct RowShape {
  int nt, v;
};
RowShape row_shape(int H, int most) {
  const int units = (H + 7) / 8;
  int v = 1;
  while (v < 8 && (units + v - 1) / v > most) v *= 2;
  const int nt = ((units + v - 1) / v + 63) / 64 * 64;
  return {nt, v};
}

template <typename T, bool VEC, int V>
void norm_launch(const NormArgs& a, int quant, int nt, hipStream_t st) {
  const int threads = nt == 64 ? 256 : nt;
  const int grid = nt == 64 ? (a.T + 3) / 4 : a.T;
  if (quant == 0)
    add_rms_norm_kernel<T, VEC, V, 0><<<grid, threads, 0, st>>>(a, nt);
  else if (quant == 1)
    add_rms_norm_kernel<T, VEC, V, 1><<<grid, threads, 0, st>>>(a, nt);
  else if constexpr (VEC)
    add_rms_norm_kernel<T, true, V, 2><<<grid, threads, 0, st>>>(a, nt);
}

template <typename T, bool VEC>
void norm_units(const NormArgs& a, int quant, RowShape rs, hipStream_t st) {
  if (rs.v == 1)
    norm_launch<T, VEC, 1>(a, quant, rs.nt, st);
  else if (rs.v == 2)
    norm_launch<T, VEC, 2>(a, quant, rs.nt, st);
  else if (rs.v == 4)
    norm_launch<T, VEC, 4>(a, quant, rs.nt, st);
  else
    norm_launch<T, VEC, 8>(a, quant, rs.nt, st);
}

template <typename T, bool VEC, int V>
void bwd_launch(const NormBwdArgs& a, int nt, int grid, hipStream_t st) {
  const int threads = nt == 64 ? 256 : nt;
  if (a.part)
    add_rms_norm_bwd_kernel<T, VEC, V, true><<<grid, threads, 0, st>>>(a, nt);
  else
    add_rms_norm_bwd_kernel<T, VEC, V, false><<<grid, threads, 0, st>>>(a, nt);
}

template <typename T, bool VEC>
void bwd_units(const NormBwdArgs& a, RowShape rs, int grid, hipStream_t st) {
  if (rs.v == 1)
    bwd_launch<T, VEC, 1>(a, rs.nt, grid, st);
  else if (rs.v == 2)
    bwd_launch<T, VEC, 2>(a, rs.nt, grid, st);
  else if (rs.v == 4)
    bwd_launch<T, VEC, 4>(a, rs.nt, grid, st);
  else
    bwd_launch<T, VEC, 8>(a, rs.nt, grid, st);
}

// Threads of a row before it takes more units. Less threads with more units each
// leave a row longer on its way where there are few rows, and nothing is gained
// with many: 512 and 256 threads at 5120 values, forward 64 rows 5.6 and 6.5 us,
// 8192 rows 58 and 63; backward 64 rows 6.9 and 7.2, 16384 rows 154 and 155.
constexpr int kNormThreads = 512;

// Workgroups of the backward pass with a weight gradient, each with a partial of H
// values that is written and read again. bf16, us, 512 / 768 / 1024 workgroups:
// 65536 x 256 44 / 40 / 38, 65536 x 512 65 / 65 / 67, 8192 x 512 13.2 / 12.9 / 13.7;
// 16384 x 5120 was 219 / 176 / 180 when the reductions still cost more.
constexpr int kNormBwdGroups = 768;

}  // namespace

hipError_t launch_add_rms_norm(const NormArgs& a, int f32, int quant, hipStream_t st) {
  RowShape rs = row_shape(a.H, kNormThreads);
  if (rs.nt > 1024) return hipErrorInvalidValue;
  const bool vec = a.H % 8 == 0;
  if (f32)
    vec ? norm_units<float, true>(a, quant, rs, st) : norm_units<float, false>(a, quant, rs, st);
  else
    vec ? norm_units<uint16_t, true>(a, quant, rs, st) : norm_units<uint16_t, false>(a, quant, rs, st);
  return hipGetLastError();
}

int norm_bwd_groups(int T, int H) {
  const RowShape rs = row_shape(H, kNormThreads);
  const int per = rs.nt == 64 ? 4 : 1;
  return std::min((T + per - 1) / per, kNormBwdGroups);
}

hipError_t launch_add_rms_norm_backward(const NormBwdArgs& a, int f32, hipStream_t st) {
  RowShape rs = row_shape(a.H, kNormThreads);
  if (rs.nt > 1024) return hipErrorInvalidValue;
  const int per = rs.nt == 64 ? 4 : 1;
  const int groups = norm_bwd_groups(a.T, a.H);
  const int grid = a.part ? groups : (a.T + per - 1) / per;
  const bool vec = a.H % 8 == 0;
  if (f32)
    vec ? bwd_units<float, true>(a, rs, grid, st) : bwd_units<float, false>(a, rs, grid, st);
  else
    vec ? bwd_units<uint16_t, true>(a, rs, grid, st) : bwd_units<uint16_t, false>(a, rs, grid, st);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.part) return e;
  norm_dw_kernel<<<(a.H + 31) / 32, 1024, 0, st>>>(a.part, groups, a.H, a.dw);
  return hipGetLastError();
}

}  // namespace beam
