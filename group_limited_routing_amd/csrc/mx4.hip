// OCP MXFP4: quantisation of rows, the values of codes, and the dense product
// with MXFP4 weights.
//
// Beam launch post ("Introducing Beam"), sections "Mixture of Experts" and
// "Hardware requirements": a 4-bit expert checkpoint serves the model on one
// node; the matrix cores here take the OCP microscaling formats natively.
// An element is an E2M1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign); 32
// consecutive elements of a row share an E8M0 scale 2^(byte - 127).
#include "common.h"
#include "operators.h"
#include "wave.h"

#include <algorithm>

namespace beam {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Eight values, at most 8 in magnitude, to E2M1 codes: nearest, ties to the
// even code, magnitudes beyond 6 to 6; value i in bits 4 i .. 4 i + 3.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t c = 0;
#if defined(__HIP_DEVICE_COMPILE__)
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], 1.0f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], 1.0f, 3);
#endif
  return c;
}

__device__ __forceinline__ void e2m1_values(uint32_t c, float (&v)[8]) {
#if defined(__HIP_DEVICE_COMPILE__)
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
  const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  v[4] = d.x; v[5] = d.y; v[6] = e.x; v[7] = e.y;
#endif
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const u32x4 a = ld16(p), b = ld16(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = __uint_as_float(a[i]);
    v[4 + i] = __uint_as_float(b[i]);
  }
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const u32x4 a = ld16(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(a[i] << 16);
    v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
}

// One thread per 8 consecutive values, four neighbouring lanes per block.
// With amax the block's largest magnitude, the scale is 2^e, e = floor(log2
// amax) - 2 (at least -127): the largest value lands in [4, 8). The exponent
// is read from amax's bits and the product with 2^-e is exact, so the codes
// are those of the exact quotients. A block that holds an infinity or a NaN
// takes the NaN scale (255) and zero codes. Bound by memory: 20480 x 5120 bf16 (268
// MB) 50 us from memory, 40 us where the last-level cache holds part of it; 1003 x
// 5120 3.4 us. Packed 8192 x 5120 28 us (its 4-byte stores scatter over 1 KB blocks;
// done once, at load time).
template <typename T, bool PACKED>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(const T* __restrict__ x, int64_t n8,
                                                           int C, uint8_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
  // n8 and the stride are multiples of 4: the four lanes of a block stay together
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += stride) {
    float v[8];
    load8(x + i * 8, v);
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t a = __float_as_uint(v[u]) & 0x7fffffffu;
      m = a > m ? a : m;
    }
    m = max(m, dpp_move<0xB1>(m, m));
    m = max(m, dpp_move<0x4E>(m, m));
    const bool bad = m >= 0x7f800000u;
    const uint32_t byte = bad ? 255u : (uint32_t)max((int)(m >> 23) - 2, 0);
    const float inv = __uint_as_float((254u - (bad ? 127u : byte)) << 23);
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = bad ? 0.f : v[u] * inv;
    const uint32_t c = e2m1x8(v);
    if constexpr (PACKED) {
      // the matrix-core fragment order of packed weights: block (16 rows, 128
      // columns) of 1 KB, lane (row % 16) + 16 (column % 128 / 32) holding its
      // 32 codes; scales in 4-byte groups of four consecutive steps
      const int u8 = C / 8;
      const int64_t row = i / u8;
      const int c0 = (int)(i - row * u8) * 8;
      const int64_t rb = row >> 4;
      const int rl = (int)(row & 15), b = c0 >> 5;
      const int64_t at = (rb * (C / 128) + (c0 >> 7)) * 1024 + (rl + 16 * (b & 3)) * 16 + ((c0 & 31) >> 1);
      *reinterpret_cast<uint32_t*>(codes + at) = c;
      if ((i & 3) == 0)
        scales[(rb * (C / 512) + (b >> 4)) * 256 + (rl + 16 * (b & 3)) * 4 + ((b & 15) >> 2)] =
            (uint8_t)byte;
    } else {
      *reinterpret_cast<uint32_t*>(codes + i * 4) = c;
      if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
    }
  }
}

// One thread per 8 codes of row-major rows. Bound by the stores: 20480 x 5120 bf16
// 38 us, 1003 x 5120 4.1 us.
template <typename T>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales,
                                                             int64_t n8, T* __restrict__ out) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += stride) {
    const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + i * 4);
    const uint32_t b = scales[i >> 2];
    // 2^(b - 127): b = 0 is the fp32 subnormal 2^-127, b = 255 is NaN
    const float s = __uint_as_float(b == 255 ? 0x7fc00000u : b == 0 ? 0x00400000u : b << 23);
    float v[8];
    e2m1_values(c, v);
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] *= s;
    if constexpr (sizeof(T) == 4) {
      st16(out + i * 8, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                              __float_as_uint(v[3])});
      st16(out + i * 8 + 4, u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]),
                                  __float_as_uint(v[6]), __float_as_uint(v[7])});
    } else {
      st16(out + i * 8, u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])});
    }
  }
}

// ------------------------------------------------------------------ product
// out[t, n] = xs[t] * sum over k of x[t, k] 2^.. w[n, k] 2^.. on the scaled
// matrix cores: the E8M0 scales of both operands go into the instruction,
// products are exact and sums are fp32 (E4M3 rows in two parts, see Parts).
//
// Operand order of the scaled instructions (measured with one-hot operands):
// the reduction block b of 32 values takes the scale byte that lane group b
// supplies, for either operand. E2M1: lane group b holds block b's 16 bytes.
// E4M3: lane group a holds values 16 a .. + 15 of the step's first half and
// the same of its second half.

__device__ __align__(16) const uint8_t kZeros[16] = {};

// A pointer that is the same in every lane, kept in scalar registers: loads
// from it plus a 32-bit lane offset then need one vector register each.
__device__ __forceinline__ const uint8_t* scalar(const uint8_t* p) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm("" : "+s"(p));
#endif
  return p;
}

// The instruction adds the products of 8 consecutive reduction values on one grid, 13
// bits below the largest sum of their exponents, and cuts what lies under it; the
// groups of 8 and the accumulator are added in fp32. Products of E4M3 (2^-9 .. 448)
// and E2M1 span 21 bits, so an E4M3 fragment is multiplied in two parts, which the top
// exponent bit separates: `hi` has the values of 2 and more (their products are
// multiples of 2^-3 and have exponents up to 8 + 2), `lo` the others (multiples of
// 2^-10, exponents up to 0 + 2), and a zero of the same sign stands where the other
// part has the value. Neither part loses a bit (checked on every pair of codes in a
// group and on sums of 512), and sums are fp32. E2M1 products span 8 bits and need
// one part. Whole E4M3 fragments, off by up to 3e-4 of a sum's magnitudes at K = 32 and
// 4e-5 at K = 512, took half the matrix instructions: N = K = 5120, us, whole and in
// parts, 1 token 4.9 and 5.9, 64 tokens 7.7 and 8.2, 512 tokens 21 and 36, 8192 tokens
// with block scales 175 and 292.
struct Parts {
  i32x8 hi, lo;
};
__device__ __forceinline__ Parts split_e4m3(const i32x8& x) {
  Parts p;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t v = (uint32_t)x[q], top = v & 0x40404040u;
    const uint32_t low = top - (top >> 6);  // 0x3f in every byte of 2 and more
    p.hi[q] = (int)(v & (low | 0xc0c0c0c0u));
    p.lo[q] = (int)(v & ~(low | 0x40404040u));
  }
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

// K not a multiple of 128: a row's K / 32 scale bytes start anywhere in a dword. The
// aligned dwords that hold them are loaded, and a step's four bytes are cut out of
// two neighbours; the bytes past the row's end count as 127 (2^0: their codes are
// 0, and a 255 would make them NaN). Rows that are multiples of 4 apart start at the
// same byte, so one count of bytes serves all of a lane's rows. Behind the last
// scale of all up to 3 bytes of its own dword are read. (Loaded byte by byte where
// they are needed, which waits for every load before them, the scales more than
// doubled the time: 512 tokens, N = 5120, row scales, E4M3 rows in one part, K = 5120
// 21 us, K = 5152 56 us by bytes and 26 us so. In two parts, 36 and 41 us.)
struct ScaleCut {
  uint32_t first, keep, fill;  // first byte of lane row r; the last step's bytes of the row
  int last;
  __device__ __forceinline__ ScaleCut(int r, int nb, int nk)
      : first((r * nb) & 3), last(nk - 1) {
    const int bytes = nb - 4 * (nk - 1);
    keep = bytes == 4 ? ~0u : (1u << (8 * bytes)) - 1;
    fill = 0x7f7f7f7fu & ~keep;
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t lo, uint32_t hi, int kt) const {
    const uint32_t v = __builtin_amdgcn_alignbyte(hi, lo, first);
    return kt == last ? (v & keep) | fill : v;
  }
};
// Offset of the last dword that holds scales of rows 0 .. row, from row 0's first.
__device__ __forceinline__ uint32_t last_dword(int row, int nb) {
  return (uint32_t)min(((uint64_t)row + 1) * nb - 1, (uint64_t)UINT32_MAX) & ~3u;
}

// ------------------------------------------------------------------ few tokens
// Few tokens: the weights are read once and bound the time. A workgroup takes
// 32 FN weight rows; its waves split the reduction, and each loads its own
// share of the weights and of the TR token rows into a ring of its own in LDS,
// NS steps of 128 values ahead, with no barrier until the partial tiles are
// added through LDS in wave order. (The same loads into registers, 16 bytes of 32
// rows a lane pair, took 17 us for 64 tokens at N = K = 5120: each touches 32
// lines. Through LDS a load is whole lines of 8 rows.) N = K = 5120, E4M3 rows: 1
// token 5.9 us, 64 tokens 8.2 us (13.9 MB of weights) by 32 x 64 workgroups, bound by
// the token rows, which every workgroup reads from L2, and by taking them apart and
// multiplying them twice; 1 token at N = K = 10240 15.8 us, 3.5 TB/s of weights. (All
// figures with warm inputs: replays of a graph.)
template <int XMODE, int TR, int FN, bool RAGGED>
struct StreamShape {
  static constexpr int FM = TR > 32 ? TR / 32 : 1, WAVES = TR > 32 ? 4 : 8;
  static constexpr int XROW = XMODE == 2 ? 64 : 128;
  static constexpr int XU = TR * XROW / 1024;             // loads of token rows
  static constexpr int BN = 32 * FN, WU = 2 * FN;          // weight rows and their loads
  static constexpr int SROWS = XMODE == 0 ? BN : BN + TR;  // rows with block scales
  static constexpr int SU = (SROWS + 63) / 64;
  static constexpr int SD = RAGGED ? 2 : 1;                // scale dwords of a row in a step
  static constexpr int STAGE = (XU + WU) * 1024 + SD * SU * 256;
  static constexpr int NS0 = 158 * 1024 / WAVES / STAGE, NS = NS0 > 4 ? 4 : NS0;
  static constexpr int PITCH = BN + 4;  // floats of a staged output row, padded
  static constexpr int OUT = WAVES * FM * 32 * PITCH * 4;
  static constexpr int LDS = WAVES * NS * STAGE > OUT ? WAVES * NS * STAGE : OUT;
  static_assert(NS >= 2, "ring too small");
};

template <int XMODE, int TR, int FN, bool RAGGED, bool OUT_F32>
__global__ __launch_bounds__(TR > 32 ? 256 : 512)
void mx4_linear_stream_kernel(Mx4LinearArgs p) {
  using S = StreamShape<XMODE, TR, FN, RAGGED>;
  constexpr int FM = S::FM, XROW = S::XROW, XU = S::XU, WU = S::WU, SU = S::SU, NS = S::NS;
  constexpr int WAVES = S::WAVES, BN = S::BN, SOFF = (XU + WU) * 1024;
  constexpr int PER = XU + WU + S::SD * SU;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::LDS];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 31, h = lane >> 5;
  const int K = p.K, nb = K / 32, nk = (K + 127) / 128;
  const int ntn = (p.N + BN - 1) / BN;
  const int n0 = blockIdx.x % ntn * BN, t0 = blockIdx.x / ntn * TR;
  const int k0 = nk * wave / WAVES, k1 = nk * (wave + 1) / WAVES;
  uint8_t* ring = smem + wave * (NS * S::STAGE);

  const uint8_t* xbase = p.x + (size_t)t0 * (XMODE == 2 ? K / 2 : K);
  const uint8_t* wbase = p.w + (size_t)n0 * (K / 2);
  const uint8_t* wsbase = p.ws + (size_t)n0 * nb;
  const uint8_t* xsbase = (const uint8_t*)p.xs + (size_t)t0 * nb;
  const int nlast = p.N - 1 - n0, tlast = p.T - 1 - t0;
  uint32_t xsrc[XU], wsrc[WU], ssrc[SU];
  int xk[XU], wk[WU];
#pragma unroll
  for (int i = 0; i < XU; ++i) {
    constexpr int L = XROW / 16;
    const int row = i * (64 / L) + lane / L, c = (lane % L) ^ swizzle<XROW>(row);
    xsrc[i] = min(row, tlast) * (XMODE == 2 ? K / 2 : K) + c * 16;
    xk[i] = c * (XMODE == 2 ? 32 : 16);
  }
#pragma unroll
  for (int i = 0; i < WU; ++i) {
    const int row = i * 16 + (lane >> 2), c = (lane & 3) ^ swizzle<64>(row);
    wsrc[i] = min(row, nlast) * (K / 2) + c * 16;
    wk[i] = c * 32;
  }
  // scale rows: the weights', then the tokens'; what is past them repeats a row.
  // Of ragged rows the aligned dwords are loaded (see below), the last of all at slast.
  const uint8_t* sbase[SU];
  uint32_t slast[RAGGED ? SU : 1];
#pragma unroll
  for (int i = 0; i < SU; ++i) {
    const int row = i * 64 + lane;
    const bool of_w = row < BN || XMODE == 0;
    sbase[i] = of_w ? wsbase : xsbase;
    ssrc[i] = (of_w ? min(row % BN, nlast) : min(row - BN, tlast)) * nb;
    if (RAGGED) {
      ssrc[i] &= ~3u;
      slast[RAGGED ? i : 0] = last_dword(of_w ? nlast : tlast, nb);
    }
  }
  auto issue = [&](int kt, uint8_t* st) {
#pragma unroll
    for (int i = 0; i < XU; ++i) {
      const uint8_t* src = scalar(xbase + (size_t)kt * XROW) + xsrc[i];
      if (RAGGED && kt * 128 + xk[i] >= K) src = kZeros;
      dma16(src, st + i * 1024);
    }
#pragma unroll
    for (int i = 0; i < WU; ++i) {
      const uint8_t* src = scalar(wbase + (size_t)kt * 64) + wsrc[i];
      if (RAGGED && kt * 128 + wk[i] >= K) src = kZeros;
      dma16(src, st + XU * 1024 + i * 1024);
    }
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int i = 0; i < SU; ++i)
#pragma unroll
      for (int d = 0; d < S::SD; ++d) {
        const uint32_t at = ssrc[i] + (kt + d) * 4;
        __builtin_amdgcn_global_load_lds(sbase[i] + (RAGGED ? min(at, slast[RAGGED ? i : 0]) : at),
                                         st + SOFF + (i * S::SD + d) * 256, 4, 0, 0);
      }
#endif
  };
  const ScaleCut cut(r, nb, nk);
  auto scale = [&](const uint8_t* st, int row, int kt) {
    const uint32_t* sc = reinterpret_cast<const uint32_t*>(st + SOFF);
    if constexpr (!RAGGED) return sc[row];
    const uint32_t* at = sc + (row >> 6) * 128 + (row & 63);
    return cut(at[0], at[64], kt);
  };

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][n][q] = 0.f;
  const int rx = TR < 32 ? r & (TR - 1) : r;  // fewer than 32 rows stand twice
  const int xsw = swizzle<XROW>(rx), wsw = swizzle<64>(r);
  auto multiply = [&](const uint8_t* st, int kt) {
    int ws[FN];
    u32x4 w[FN][2];
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      ws[n] = (int)(scale(st, n * 32 + r, kt) >> (8 * h));
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w[n][j] = ld16(st + XU * 1024 + (n * 32 + r) * 64 + (((2 * j + h) ^ wsw) << 4));
    }
    for_each<FM>([&](auto ic) {
      constexpr int I = decltype(ic)::value;
      const int xs = XMODE == 0 ? 0x7f7f7f7f : (int)(scale(st, BN + I * 32 + rx, kt) >> (8 * h));
      const uint8_t* xr = st + (I * 32 + rx) * XROW;
      for_each<2>([&](auto jc) {
        constexpr int J = decltype(jc)::value;
        i32x8 xf{};
        const u32x4 lo = ld16(xr + ((((XMODE == 2 ? 2 : 4) * J + h) ^ xsw) << 4));
        u32x4 hi = lo;
        if constexpr (XMODE != 2) hi = ld16(xr + (((4 * J + 2 + h) ^ xsw) << 4));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          xf[q] = (int)lo[q];
          if constexpr (XMODE != 2) xf[4 + q] = (int)hi[q];
        }
        auto products = [&](const i32x8& part) {
          for_each<FN>([&](auto nc) {
            constexpr int N = decltype(nc)::value;
            i32x8 wf{};
#pragma unroll
            for (int q = 0; q < 4; ++q) wf[q] = (int)w[N][J][q];
            acc[I][N] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                wf, part, acc[I][N], 4, XMODE == 2 ? 4 : 0, 2 * J, ws[N], 2 * J, xs);
          });
        };
        if constexpr (XMODE == 2) {
          products(xf);
        } else {
          const Parts parts = split_e4m3(xf);
          products(parts.lo);
          products(parts.hi);
        }
      });
    });
  };
#pragma unroll
  for (int s = 0; s < NS; ++s)
    if (k0 + s < k1) issue(k0 + s, ring + s * S::STAGE);
  int slot = 0;
  for (int kt = k0; kt < k1; ++kt) {
    uint8_t* st = ring + slot;
    if (kt + NS - 1 < k1)
      wait_vmcnt<(NS - 1) * PER>();
    else
      wait_vmcnt<0>();
    asm volatile("" ::: "memory");
    multiply(st, kt);
    if (kt + NS < k1) {
      wait_lgkmcnt0();  // the step has been read
      asm volatile("" ::: "memory");
      issue(kt + NS, st);
    }
    slot = slot == (NS - 1) * S::STAGE ? 0 : slot + S::STAGE;
  }

  __syncthreads();  // the rings become the staging of the partial tiles
  float* part = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        st16(part + ((wave * FM + i) * 32 + r) * S::PITCH + n * 32 + 8 * q + 4 * h,
             u32x4{__float_as_uint(acc[i][n][4 * q]), __float_as_uint(acc[i][n][4 * q + 1]),
                   __float_as_uint(acc[i][n][4 * q + 2]), __float_as_uint(acc[i][n][4 * q + 3])});
  __syncthreads();
  const int c = threadIdx.x % BN;
  for (int t = threadIdx.x / BN; t < TR; t += WAVES * 64 / BN) {
    float v = part[t * S::PITCH + c];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += part[(w * FM * 32 + t) * S::PITCH + c];
    if (t <= tlast && n0 + c < p.N) {
      if (XMODE == 0) v *= ((const float*)p.xs)[t0 + t];
      const size_t at = (size_t)(t0 + t) * p.N + n0 + c;
      if (OUT_F32)
        ((float*)p.out)[at] = v;
      else
        ((uint16_t*)p.out)[at] = (uint16_t)f32_to_bf16_bits(v);
    }
  }
}

template <int XMODE, int TR, int FN>
void stream_launch(const Mx4LinearArgs& a, hipStream_t st) {
  using S = StreamShape<XMODE, TR, FN, false>;
  const int grid = (a.N + S::BN - 1) / S::BN * ((a.T + TR - 1) / TR), threads = 64 * S::WAVES;
  const bool ragged = a.K % 128 != 0;
  if (ragged && a.out_f32)
    mx4_linear_stream_kernel<XMODE, TR, FN, true, true><<<grid, threads, 0, st>>>(a);
  else if (ragged)
    mx4_linear_stream_kernel<XMODE, TR, FN, true, false><<<grid, threads, 0, st>>>(a);
  else if (a.out_f32)
    mx4_linear_stream_kernel<XMODE, TR, FN, false, true><<<grid, threads, 0, st>>>(a);
  else
    mx4_linear_stream_kernel<XMODE, TR, FN, false, false><<<grid, threads, 0, st>>>(a);
}

// ------------------------------------------------------------------ tiles
// Waves as WM x WN, each FM x FN fragments of 32 tokens x 32 weight rows on
// 32x32x64 scaled MFMAs (weights first, so a lane ends with runs of 4
// consecutive output columns of one token). Operands go from memory straight
// into LDS (16 bytes a lane) through a ring of NS stages of 128 reduction
// values, filled NS - 1 stages ahead; waits leave only the later stages'
// loads outstanding and raw barriers publish a stage.
//
// LDS of a stage: the token rows and the weight rows, swizzled as above. The block
// scales of four stages are 16 bytes of a row and are loaded together, into one of
// two buffers, while the four stages before them are multiplied (a load per stage,
// 4 bytes of each row, was half of all requests to L2).
// N = K = 5120, 8192 tokens: E4M3 rows 292 us (1.5 PF/s, 2.9 of instructions, matrix
// cores busy 59% of the time), 4-bit rows 121-129 us (3.3-3.5 PF/s); each round of
// tiles starts and ends with 9 us outside its loop. Tiles of 128 with 4-bit rows fill
// LDS at 50 GB/s per CU, which bounds them; rings of 160 KB and 8 waves a tile did not
// help (1111 x 2560 x 5120: 17.3, 17.6 and 18.4 us).
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

template <int XMODE, int FM, int FN, int WM, int WN>
struct TileShape {
  static constexpr int WAVES = WM * WN;
  static constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN;
  static constexpr int XROW = XMODE == 2 ? 64 : 128;  // bytes of a row in a stage
  static constexpr int X_BYTES = BM * XROW, W_BYTES = BN * 64, STAGE = X_BYTES + W_BYTES;
  static constexpr int SROWS = XMODE == 0 ? BN : BM + BN;  // rows with block scales
  static constexpr int SCALES = SROWS * 16;                // of four stages
  static constexpr int PITCH = FN * 32 * 4 + 16;           // staged output row (fp32)
  // 8 waves have a CU's LDS for themselves, fewer share it with another workgroup
  static constexpr int ROOM = (WAVES == 8 ? 160 : 80) * 1024 - 2 * SCALES;
  static constexpr int NS = ROOM / STAGE > 4 ? 4 : ROOM / STAGE;
  static constexpr int OUT = WAVES * 32 * PITCH;
  static constexpr int LDS = NS * STAGE + 2 * SCALES > OUT ? NS * STAGE + 2 * SCALES : OUT;
  static_assert(NS >= 3 && BN % 64 == 0 && BM % 64 == 0, "tile");
};

// How the scales come: four stages at a time, cut out of unaligned rows, or (fewer
// than four stages) byte by byte.
enum Scales { kAligned, kCut, kShort };

template <int XMODE, int FM, int FN, int WM, int WN, Scales SC, bool OUT_F32>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2)))
void mx4_linear_tile_kernel(Mx4LinearArgs p) {
  using S = TileShape<XMODE, FM, FN, WM, WN>;
  constexpr bool RAGGED = SC != kAligned;  // the last stage may end within the row
  constexpr int BM = S::BM, BN = S::BN, XROW = S::XROW, NS = S::NS, WAVES = S::WAVES;
  // Loads of a stage: 1 KB of rows each, the tokens', then the weights'; and every
  // four stages 64 rows' scales each, the weights', then the tokens'. They are
  // dealt to the waves in turn; what is left over repeats the last one, so that
  // every wave waits for the same count.
  constexpr int XU = S::X_BYTES / 1024, WU = S::W_BYTES / 1024, SU = S::SROWS / 64;
  constexpr int PER = (XU + WU + WAVES - 1) / WAVES, SI = (SU + WAVES - 1) / WAVES;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::LDS];
  uint8_t* scales = smem + NS * S::STAGE;

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave / WN, wn = wave % WN, r = lane & 31, h = lane >> 5;
  const int K = p.K, nb = K / 32, nk = (K + 127) / 128;
  const int ntt = (p.N + BN - 1) / BN, mtt = (p.T + BM - 1) / BM;
  int mi, ni;
  tile_of(blockIdx.x, ntt * mtt, mtt, ntt, mi, ni);
  const int t0 = mi * BM, n0 = ni * BN;

  // Sources of this lane's loads, as offsets from the tile's first row (at most
  // 256 rows of 65536 bytes); rows past the end repeat the last one.
  const uint8_t* xbase = p.x + (size_t)t0 * (XMODE == 2 ? K / 2 : K);
  const uint8_t* wbase = p.w + (size_t)n0 * (K / 2);
  const uint8_t* wsbase = p.ws + (size_t)n0 * nb;
  const uint8_t* xsbase = XMODE == 0 ? wsbase : (const uint8_t*)p.xs + (size_t)t0 * nb;
  const int tlast = p.T - 1 - t0, nlast = p.N - 1 - n0;
  uint32_t dsrc[PER], ssrc[SI];
  int dk[RAGGED ? PER : 1];  // first reduction value of the lane's chunk in a stage
  auto unit = [&](int q) { return min(q * WAVES + wave, XU + WU - 1); };
  auto sunit = [&](int q) { return min(q * WAVES + wave, SU - 1); };
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int u = unit(q);
    if (XMODE != 2 && u < XU) {
      const int row = u * 8 + (lane >> 3), c = (lane & 7) ^ swizzle<128>(row);
      dsrc[q] = min(row, tlast) * K + c * 16;
      if (RAGGED) dk[q] = c * 16;
    } else {
      const int row = (u < XU ? u : u - XU) * 16 + (lane >> 2), c = (lane & 3) ^ swizzle<64>(row);
      dsrc[q] = min(row, u < XU ? tlast : nlast) * (K / 2) + c * 16;
      if (RAGGED) dk[q] = c * 32;
    }
  }
#pragma unroll
  for (int q = 0; q < SI; ++q) {
    const int row = sunit(q) * 64 + lane;
    ssrc[q] = (sunit(q) < BN / 64 ? min(row, nlast) : min(row - BN, tlast)) * nb;
    if (SC == kCut) ssrc[q] &= ~3u;
  }
  auto sbase = [&](int q) { return sunit(q) < BN / 64 ? wsbase : xsbase; };
  // Load q of stage kt, into the slot at byte `slot`. Addresses are a scalar
  // base and a lane offset.
  auto issue_one = [&](int kt, int slot, auto qc, bool end) {  // end: it is the last stage
    constexpr int Q = decltype(qc)::value;
    if constexpr (Q < PER) {
      const int u = unit(Q);
      const uint8_t* src = scalar(u < XU ? xbase + (size_t)kt * XROW : wbase + (size_t)kt * 64) + dsrc[Q];
      if (RAGGED && end && kt * 128 + dk[RAGGED ? Q : 0] >= K) src = kZeros;
      dma16(src, smem + slot + u * 1024);
    }
  };
  // Scales of stages 4 g .. 4 g + 3: 16 bytes of every row. The last group ends
  // with the last stage, so that nothing is read past a row (kCut: past the dword
  // of its last stage; the one after it is loaded by itself, into the slot `tail`,
  // when no stage needs that any more).
  auto first_of = [&](int g) { return SC == kShort ? 4 * g : min(4 * g, nk - 4); };
  auto issue_scales = [&](int g) {
#pragma unroll
    for (int q = 0; q < SI; ++q)
      dma16(scalar(sbase(q) + first_of(g) * 4) + ssrc[q], scales + (g & 1) * S::SCALES + sunit(q) * 1024);
  };
  int tail = 0;
  auto issue_tail = [&](int slot) {
    tail = slot;
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int q = 0; q < SI; ++q)
      __builtin_amdgcn_global_load_lds(
          sbase(q) + min(ssrc[q] + nk * 4, last_dword(sunit(q) < BN / 64 ? nlast : tlast, nb)),
          smem + slot + sunit(q) * 256, 4, 0, 0);
#endif
  };
  // fewer than four stages: the bytes of a stage go through registers
  auto short_scales = [&](int kt) {
    uint8_t* at = scales + (kt & 3) * 4 + lane * 16;
#pragma unroll
    for (int q = 0; q < SI; ++q) {
      uint32_t v = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        v |= (uint32_t)(kt * 4 + b < nb ? sbase(q)[ssrc[q] + kt * 4 + b] : 127) << (8 * b);
      *reinterpret_cast<uint32_t*>(at + sunit(q) * 1024) = v;
    }
  };

  // Operand offsets in a stage: fragments are 32 rows apart, which leaves the
  // swizzle as it is. Chunks of half J: E4M3 4 J + h and 4 J + 2 + h, E2M1 2 J + h.
  const int xrow = wm * FM * 32 + r, wrow = wn * FN * 32 + r;
  const int xsw = swizzle<XROW>(r), wsw = swizzle<64>(r);
  int xo[2][2], wo[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    xo[j][0] = xrow * XROW + ((((XMODE == 2 ? 2 : 4) * j + h) ^ xsw) << 4);
    xo[j][1] = xrow * XROW + (((4 * j + 2 + h) ^ xsw) << 4);
    wo[j] = S::X_BYTES + wrow * 64 + (((2 * j + h) ^ wsw) << 4);
  }
  const int xso = (BN + xrow) * 16, wso = wrow * 16;
  // bytes h and 2 + h (this lane half's blocks) of two rows' scale dwords
  const uint32_t pick = h ? 0x07030501u : 0x06020400u;

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;

  // A stage is 2 FM steps: step i multiplies token fragment i % FM of half i / FM
  // (64 values; lane half h holds block h of them) with the FN weight fragments.
  // A token fragment is read from LDS three steps before its products, into one
  // of four register sets, and the weights' of a half some steps before it, so
  // the matrix core has work while reads and loads issue. The reads of stage
  // kt + 1 begin at step 2 FM - 3 of stage kt: a barrier there says that every
  // wave has read all of stage kt, whose slot the next stage refills, and that
  // stage kt + 1 has landed.
  constexpr int STEPS = 2 * FM, AHEAD = 3, TURN = STEPS - AHEAD;
  static_assert(FM >= 2 && STEPS % 4 == 0, "four register sets");
  struct Frag {
    u32x4 lo, hi;
  };
  Frag xr[4];
  u32x4 wr[2][FN];
  auto read_x = [&](const uint8_t* st, auto sc) {
    constexpr int I = decltype(sc)::value, J = I / FM;
    xr[I % 4].lo = ld16(st + xo[J][0] + I % FM * 32 * XROW);
    if constexpr (XMODE != 2) xr[I % 4].hi = ld16(st + xo[J][1] + I % FM * 32 * XROW);
  };
  auto read_w = [&](const uint8_t* st, auto jc) {
    constexpr int J = decltype(jc)::value;
#pragma unroll
    for (int j = 0; j < FN; ++j) wr[J][j] = ld16(st + wo[J] + j * 32 * 64);
  };
  // The scale dwords as stored (read ahead), and the bytes that this lane half
  // needs of two fragments in a register: fragment f's of half J in byte 2 J + f % 2
  uint32_t wraw[FN], xraw[FM];
  int wsc[(FN + 1) / 2], xsc[(FM + 1) / 2];
  const ScaleCut cut(r, nb, nk);
  auto read_scales = [&](int kt) {
    const int g = kt >> 2;
    const uint8_t* at = scales + (g & 1) * S::SCALES + (kt - first_of(g)) * 4;
    const auto dword = [](const uint8_t* q) { return *reinterpret_cast<const uint32_t*>(q); };
#pragma unroll
    for (int j = 0; j < FN; ++j) wraw[j] = dword(at + wso + j * 512);
    if constexpr (XMODE != 0) {
#pragma unroll
      for (int i = 0; i < FM; ++i) xraw[i] = dword(at + xso + i * 512);
    }
    if constexpr (SC == kCut) {
      // the dwords after them: the next group's first one has landed
      const int g1 = (kt + 1) >> 2, pitch = kt + 1 < nk ? 16 : 4;
      const uint8_t* next = kt + 1 < nk ? scales + (g1 & 1) * S::SCALES + (kt + 1 - first_of(g1)) * 4
                                        : smem + tail;
#pragma unroll
      for (int j = 0; j < FN; ++j)
        wraw[j] = cut(wraw[j], dword(next + (wrow + j * 32) * pitch), kt);
      if constexpr (XMODE != 0) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
          xraw[i] = cut(xraw[i], dword(next + (BN + xrow + i * 32) * pitch), kt);
      }
    }
  };
  auto pick_scales = [&]() {
#pragma unroll
    for (int j = 0; j < FN; j += 2)
      wsc[j / 2] = (int)__builtin_amdgcn_perm(wraw[j + 1 < FN ? j + 1 : j], wraw[j], pick);
#pragma unroll
    for (int i = 0; i < FM; i += 2)
      xsc[i / 2] = XMODE == 0 ? 0x7f7f7f7f : (int)__builtin_amdgcn_perm(xraw[i + 1], xraw[i], pick);
  };
  auto multiply = [&](auto sc) {
    constexpr int I = decltype(sc)::value % FM, J = decltype(sc)::value / FM, R = decltype(sc)::value % 4;
    i32x8 xf{};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      xf[q] = (int)xr[R].lo[q];
      if constexpr (XMODE != 2) xf[4 + q] = (int)xr[R].hi[q];
    }
    auto products = [&](const i32x8& part) {
      for_each<FN>([&](auto nc) {
        constexpr int N = decltype(nc)::value;
        i32x8 wf{};
#pragma unroll
        for (int q = 0; q < 4; ++q) wf[q] = (int)wr[J][N][q];
        acc[I][N] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            wf, part, acc[I][N], 4, XMODE == 2 ? 4 : 0, 2 * J + N % 2, wsc[N / 2], 2 * J + I % 2, xsc[I / 2]);
      });
    };
    if constexpr (XMODE == 2) {
      products(xf);
    } else {
      const Parts parts = split_e4m3(xf);
      products(parts.lo);
      products(parts.hi);
    }
  };

  if (SC != kShort) issue_scales(0);
#pragma unroll
  for (int s = 0; s < NS - 1; ++s)
    if (s < nk) for_each<PER>([&](auto q) { issue_one(s, s * S::STAGE, q, s + 1 == nk); });
  if (SC == kShort) short_scales(0);
  if (NS - 1 <= nk)
    wait_vmcnt<(NS - 2) * PER>();
  else
    wait_vmcnt<0>();
  if (SC == kShort) wait_lgkmcnt0();
  barrier_only();
  asm volatile("" ::: "memory");
  std::integral_constant<int, 0> j0;
  std::integral_constant<int, 1> j1;
  for_each<AHEAD>([&](auto q) { read_x(smem, q); });
  read_w(smem, j0);
  read_scales(0);
  pick_scales();
  int slot = 0, last = (NS - 1) * S::STAGE;  // of stage kt, and of the stage before it
  auto stage = [&](int kt, auto loads_c) {
    // stage kt + NS - 1: 0 there is none, 2 it is the last one
    constexpr int LOADS = decltype(loads_c)::value;
    constexpr int LP = (PER + TURN - 1) / TURN;       // loads of a step, all before the barrier
    const int next = slot == (NS - 1) * S::STAGE ? 0 : slot + S::STAGE;
    // The scales of the next four stages: their buffer was last read before the
    // barrier of stage kt - 1; they are read three stages on, when the loads of
    // these three (more than any wait leaves outstanding) are behind them.
    if (SC != kShort && (kt & 3) == 0 && kt + 4 < nk) issue_scales((kt >> 2) + 1);
    if (SC == kCut && !LOADS && kt + NS - 1 == nk) issue_tail(last);
    for_each<STEPS>([&](auto sc) {
      constexpr int I = decltype(sc)::value;
      if constexpr (I == TURN) {
        if (SC == kShort && kt + 1 < nk) short_scales(kt + 1);
        wait_vmcnt<LOADS ? (NS - 2) * PER : 0>();
        wait_lgkmcnt0();
        barrier_only();
        asm volatile("" ::: "memory");
      }
      // past the last stage these read what nothing uses
      if constexpr (I < TURN)
        read_x(smem + slot, std::integral_constant<int, I + AHEAD>{});
      else
        read_x(smem + next, std::integral_constant<int, I - TURN>{});
      if constexpr (I == (FM > 3 ? FM - 3 : 0)) read_w(smem + slot, j1);
      if constexpr (I == (TURN > FM ? TURN : FM)) read_w(smem + next, j0);  // half 0 is done
      if constexpr (I == TURN) read_scales(min(kt + 1, nk - 1));
      multiply(sc);
      if constexpr (LOADS && I < TURN)
        for_each<LP>([&](auto e) {
          issue_one(kt + NS - 1, last, std::integral_constant<int, I * LP + decltype(e)::value>{},
                    LOADS == 2);
        });
      __builtin_amdgcn_sched_barrier(0);
    });
    pick_scales();
    last = slot;
    slot = next;
  };
  int kt = 0;
  for (; kt + NS - 1 < nk - (RAGGED ? 1 : 0); ++kt) stage(kt, j1);
  if (RAGGED && kt + NS - 1 < nk) stage(kt++, std::integral_constant<int, 2>{});
  for (; kt < nk; ++kt) stage(kt, j0);

  // Output: lane (r, h) of a fragment holds token r, columns 8 q + 4 h .. + 3.
  // 32 tokens of the wave at a time go through its own piece of the ring (rows
  // padded by 16 bytes), so that a store writes whole 128-byte runs of a row.
  // Stored straight from the registers, 8 bytes a lane, the tile's output took
  // as long as a quarter of its reduction at K = 5120.
  asm volatile("" ::: "memory");
  barrier_only();  // every wave has read the last stage
  asm volatile("" ::: "memory");
  constexpr int OB = OUT_F32 ? 4 : 2, COLS = FN * 32, PITCH = COLS * OB + 16;
  static_assert(WAVES * 32 * PITCH <= S::LDS, "output staging");
  uint8_t* mine = smem + wave * (32 * PITCH);
  const int c0 = n0 + wn * COLS, cols = min(COLS, p.N - c0);
  const bool whole = p.N % (16 / OB) == 0 && cols == COLS;
  for_each<FM>([&](auto ic) {
    constexpr int I = decltype(ic)::value;
    const int tb = t0 + (wm * FM + I) * 32;
    const float scale = XMODE == 0 ? ((const float*)p.xs)[min(tb + r, p.T - 1)] : 1.0f;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[I][j][4 * q + e] * scale;
        uint8_t* at = mine + r * PITCH + (j * 32 + 8 * q + 4 * h) * OB;
        if constexpr (OUT_F32)
          st16(at, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                         __float_as_uint(v[3])});
        else
          *reinterpret_cast<u32x2*>(at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
    wait_lgkmcnt0();
    asm volatile("" ::: "memory");
    uint8_t* out = (uint8_t*)p.out + ((size_t)tb * p.N + c0) * OB;
    if (whole) {
      constexpr int L = COLS * OB / 16, RS = 64 / L;  // lanes of a row, rows of a store
#pragma unroll
      for (int g = 0; g < 32 / RS; ++g) {
        const int row = g * RS + lane / L;
        if (tb + row < p.T)
          st16(out + (size_t)row * p.N * OB + (lane % L) * 16,
               ld16(mine + row * PITCH + (lane % L) * 16));
      }
    } else {
      for (int row = 0; row < 32 && tb + row < p.T; ++row)
        for (int c = lane; c < cols; c += 64) {
          if constexpr (OUT_F32)
            ((float*)(out + (size_t)row * p.N * OB))[c] = ((const float*)(mine + row * PITCH))[c];
          else
            ((uint16_t*)(out + (size_t)row * p.N * OB))[c] = ((const uint16_t*)(mine + row * PITCH))[c];
        }
    }
    wait_lgkmcnt0();
    asm volatile("" ::: "memory");
  });
}

template <int XMODE, int FM, int FN, int WM, int WN>
void tile_launch(const Mx4LinearArgs& a, hipStream_t st) {
  using S = TileShape<XMODE, FM, FN, WM, WN>;
  const int grid = (a.T + S::BM - 1) / S::BM * ((a.N + S::BN - 1) / S::BN);
  auto go = [&](auto sc) {
    constexpr Scales SC = decltype(sc)::value;
    if (a.out_f32)
      mx4_linear_tile_kernel<XMODE, FM, FN, WM, WN, SC, true><<<grid, 64 * S::WAVES, 0, st>>>(a);
    else
      mx4_linear_tile_kernel<XMODE, FM, FN, WM, WN, SC, false><<<grid, 64 * S::WAVES, 0, st>>>(a);
  };
  if (a.K <= 384)
    go(std::integral_constant<Scales, kShort>{});
  else if (a.K % 128 != 0)
    go(std::integral_constant<Scales, kCut>{});
  else
    go(std::integral_constant<Scales, kAligned>{});
}

constexpr int64_t kMaxGrid = 1 << 23;  // workgroups of 256: a launch has fewer than 2^32 threads

}  // namespace

hipError_t launch_mx4_quantize(const void* x, int f32, int64_t rows, int C, int packed,
                               uint8_t* codes, uint8_t* scales, hipStream_t st) {
  const int64_t n8 = rows * (C / 8);
  const unsigned grid = (unsigned)std::min<int64_t>((n8 + 255) / 256, kMaxGrid);
  if (f32 && packed)
    mx4_quantize_kernel<float, true><<<grid, 256, 0, st>>>((const float*)x, n8, C, codes, scales);
  else if (f32)
    mx4_quantize_kernel<float, false><<<grid, 256, 0, st>>>((const float*)x, n8, C, codes, scales);
  else if (packed)
    mx4_quantize_kernel<uint16_t, true><<<grid, 256, 0, st>>>((const uint16_t*)x, n8, C, codes, scales);
  else
    mx4_quantize_kernel<uint16_t, false><<<grid, 256, 0, st>>>((const uint16_t*)x, n8, C, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int C,
                                 int f32, void* out, hipStream_t st) {
  const int64_t n8 = rows * (C / 8);
  const unsigned grid = (unsigned)std::min<int64_t>((n8 + 255) / 256, kMaxGrid);
  if (f32)
    mx4_dequantize_kernel<float><<<grid, 256, 0, st>>>(codes, scales, n8, (float*)out);
  else
    mx4_dequantize_kernel<uint16_t><<<grid, 256, 0, st>>>(codes, scales, n8, (uint16_t*)out);
  return hipGetLastError();
}

// Which kernel takes a product: the one whose rounds of 256 workgroups cost least. The
// first round pays for the start and the first loads, a later one overlaps with the
// one before it (of 64 and 128 token tiles two share a CU). Tenths of a us, first and
// later rounds, at K = 5120 (at other K taken to be in the same proportion):
//                            E4M3 rows   4-bit rows
//   stream, 16 x  32          60   45     45   33
//           16 x  64          85   70     72   60
//           32 x  32          66   52     50   43
//           32 x  64          95   72     72   66
//           64 x  32           -         70   65
//           64 x  64         145  125    105  100
//   tile,   64 x 128         250  200    132  103
//          128 x 128         355  290    155  155
//          256 x 256         950  960    345  420
// (64 x 32 takes as many workgroups as 32 x 64 and is slower with E4M3 rows, 10.2 and
// 9.5 a round; with 4-bit rows 33 tokens of N = 5120 take 6.2 and 6.9.)
// Measured around the borders, N = 5120, us, the kernel taken and the next best one.
// E4M3 rows: T = 64, 32 x 64 9.0 and 64 x 32 10.3; 128, 64 x 64 14.0 and 32 x 64 16.5;
// 256, 32 x 64 24.7 and 64 x 64 26.4; 384, 64 x 128 27.5 and 64 x 64 28.4; 512, 128 x
// 128 36.7 and 64 x 128 39.9; 2048, 128 x 128 91.5 and 256 x 256 93.2; 3000, 256 x 256
// 102 and 128 x 128 124; 4096, 128 x 128 161 and 256 x 256 189; 8192, 256 x 256 292 and
// 128 x 128 314. 4-bit rows: T = 128, 64 x 64 10.4 and 64 x 128 12.9; 512, 128 x 128
// 15.5 and 64 x 128 21.4; 2048, 256 x 256 36.3 and 128 x 128 46.3; 4096, 256 x 256 77.4
// and 128 x 128 84.2.
enum class Variant { kStream16, kStream16Wide, kStream32, kStream32Wide, kStream64, kStream64Wide,
                     kTile64, kTile128, kTile256 };
struct Cost {
  int first, later;
};
Variant variant_of(int T, int N, bool mx4_rows) {
  struct {
    Variant v;
    int bm, bn;
    Cost e4m3, mx4;
  } const all[] = {{Variant::kStream16, 16, 32, {60, 45}, {45, 33}},
                   {Variant::kStream16Wide, 16, 64, {85, 70}, {72, 60}},
                   {Variant::kStream32, 32, 32, {66, 52}, {50, 43}},
                   {Variant::kStream32Wide, 32, 64, {95, 72}, {72, 66}},
                   {Variant::kStream64, 64, 32, {0, 0}, {70, 65}},
                   {Variant::kStream64Wide, 64, 64, {145, 125}, {105, 100}},
                   {Variant::kTile64, 64, 128, {250, 200}, {132, 103}},
                   {Variant::kTile128, 128, 128, {355, 290}, {155, 155}},
                   {Variant::kTile256, 256, 256, {950, 960}, {345, 420}}};
  Variant best = Variant::kTile256;
  int64_t least = INT64_MAX;
  for (const auto& c : all) {
    const int64_t wgs = (int64_t)((T + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
    const Cost& us = mx4_rows ? c.mx4 : c.e4m3;
    if (us.first == 0) continue;  // not for this format
    const int64_t cost = us.first + ((wgs + 255) / 256 - 1) * us.later;
    if (cost < least) {
      least = cost;
      best = c.v;
    }
  }
  return best;
}

hipError_t launch_mx4_linear(const Mx4LinearArgs& a, int x_mode, hipStream_t st) {
  auto go = [&](auto m) {
    constexpr int XMODE = decltype(m)::value;
    switch (variant_of(a.T, a.N, XMODE == 2)) {
      case Variant::kStream16: stream_launch<XMODE, 16, 1>(a, st); break;
      case Variant::kStream16Wide: stream_launch<XMODE, 16, 2>(a, st); break;
      case Variant::kStream32: stream_launch<XMODE, 32, 1>(a, st); break;
      case Variant::kStream32Wide: stream_launch<XMODE, 32, 2>(a, st); break;
      case Variant::kStream64:
        if constexpr (XMODE == 2) stream_launch<XMODE, 64, 1>(a, st);
        break;
      case Variant::kStream64Wide: stream_launch<XMODE, 64, 2>(a, st); break;
      case Variant::kTile64: tile_launch<XMODE, 2, 1, 1, 4>(a, st); break;
      case Variant::kTile128: tile_launch<XMODE, 2, 2, 2, 2>(a, st); break;
      case Variant::kTile256:
        // E4M3 rows: two fragments of tokens a wave, so that half as much is taken apart
        // (8192 tokens, N = K = 5120: 293 us, as 4 x 2 fragments 310, which spills)
        if constexpr (XMODE == 2)
          tile_launch<XMODE, 4, 2, 2, 4>(a, st);
        else
          tile_launch<XMODE, 2, 4, 4, 2>(a, st);
        break;
    }
  };
  if (x_mode == 0)
    go(std::integral_constant<int, 0>{});
  else if (x_mode == 1)
    go(std::integral_constant<int, 1>{});
  else
    go(std::integral_constant<int, 2>{});
  return hipGetLastError();
}

}  // namespace beam
