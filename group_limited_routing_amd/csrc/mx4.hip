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

#include <algorithm>

namespace beam {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

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
// takes the NaN scale (255) and zero codes.
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
    uint32_t o = __shfl_xor(m, 1);
    m = o > m ? o : m;
    o = __shfl_xor(m, 2);
    m = o > m ? o : m;
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

// One thread per 8 codes of row-major rows.
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
// products are exact and sums are fp32.
//
// Operand order of the scaled instructions (measured with one-hot operands):
// the reduction block b of 32 values takes the scale byte that lane group b
// supplies, for either operand. E2M1: lane group b holds block b's 16 bytes.
// E4M3: lane group a holds values 16 a .. + 15 of the step's first half and
// the same of its second half.

// One 16 x 16 tile per wave, straight from memory.
template <int XMODE, bool OUT_F32>
__global__ __launch_bounds__(256) void mx4_linear_kernel(Mx4LinearArgs p) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int nbn = (p.N + 63) / 64;
  const int n0 = (blockIdx.x % nbn * 4 + wave) * 16, t0 = blockIdx.x / nbn * 16;
  const int K = p.K, nb = K / 32;
  const int n = min(n0 + r, p.N - 1), t = min(t0 + r, p.T - 1);
  const uint8_t* wr = p.w + (size_t)n * (K / 2);
  const uint8_t* wsr = p.ws + (size_t)n * nb;
  const uint8_t* xr = p.x + (size_t)t * (XMODE == 2 ? K / 2 : K);
  const uint8_t* xsr = (const uint8_t*)p.xs + (size_t)t * nb;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int b0 = 0; b0 < nb; b0 += 4) {
    const int b = b0 + g;
    i32x8 a{}, x{};
    int sa = 127, sx = 127;
    if (b < nb) {
      const u32x4 v = ld16(wr + b * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = (int)v[i];
      sa = wsr[b];
      if (XMODE != 0) sx = xsr[b];
    }
    if constexpr (XMODE == 2) {
      if (b < nb) {
        const u32x4 v = ld16(xr + b * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (int)v[i];
      }
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, x, acc, 4, 4, 0, sa, 0, sx);
    } else {
      const int k = b0 * 32 + 16 * g;
      if (k < K) {
        const u32x4 v = ld16(xr + k);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (int)v[i];
      }
      if (k + 64 < K) {
        const u32x4 v = ld16(xr + k + 64);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 + i] = (int)v[i];
      }
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, x, acc, 4, 0, 0, sa, 0, sx);
    }
  }
  if (t0 + r >= p.T) return;
  const float s = XMODE == 0 ? ((const float*)p.xs)[t] : 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = n0 + 4 * g + i;
    if (c < p.N) {
      if (OUT_F32)
        ((float*)p.out)[(size_t)t * p.N + c] = acc[i] * s;
      else
        ((uint16_t*)p.out)[(size_t)t * p.N + c] = (uint16_t)f32_to_bf16_bits(acc[i] * s);
    }
  }
}

constexpr int64_t kMaxGrid = 1 << 23;  // workgroups of 256: a launch has fewer than 2^32 threads

// ------------------------------------------------------------------ tiles
// 8 waves as WM x WN, each FM x FN fragments of 32 tokens x 32 weight rows on
// 32x32x64 scaled MFMAs (weights first, so a lane ends with runs of 4
// consecutive output columns of one token). Operands go from memory straight
// into LDS (16 bytes a lane) through a ring of NS stages of 128 reduction
// values, filled NS - 1 stages ahead; waits leave only the later stages'
// loads outstanding and raw barriers publish a stage.
//
// LDS of a stage: E4M3 rows 128 bytes, 16-byte chunk c of row r at position
// c ^ (r & 7); E2M1 rows 64 bytes, chunk c at c ^ ((r >> 1) & 3): the rows of
// a fragment read spread over all banks. Then one dword per row with the
// scale bytes of the stage's four blocks.
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __align__(16) const uint8_t kZeros[16] = {};

// Tiles that run together on one XCD (32 consecutive, dealt to the XCDs in
// turn) cover 4 token tiles x 8 weight tiles, which share operands in its L2.
__device__ __forceinline__ void tile_of(int b, int n_tiles, int mt, int nt, int& m, int& n) {
  constexpr int R = 256, GM = 4;
  if (b < n_tiles / R * R) {
    const int q = b >> 3;
    b = ((q / 32) * 8 + (b & 7)) * 32 + q % 32;
  }
  const int mb = b / (GM * nt), rem = b - mb * GM * nt;
  const int gm = min(GM, mt - mb * GM);
  n = rem / gm;
  m = mb * GM + rem % gm;
}

template <int XMODE, int FM, int FN, int WM, int WN, bool RAGGED>
struct TileShape {
  static constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN;
  static constexpr int XROW = XMODE == 2 ? 64 : 128;  // bytes of a row in a stage
  static constexpr int X_BYTES = BM * XROW, W_BYTES = BN * 64;
  static constexpr int S_BYTES = (BM + BN) * 4;
  static constexpr int STAGE = X_BYTES + W_BYTES + S_BYTES;
  static constexpr int NS = 158 * 1024 / STAGE > 4 ? 4 : 158 * 1024 / STAGE;
  static_assert(NS >= 2, "ring too small");
};

template <int XMODE, int FM, int FN, int WM, int WN, bool RAGGED, bool OUT_F32>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
void mx4_linear_tile_kernel(Mx4LinearArgs p) {
  using S = TileShape<XMODE, FM, FN, WM, WN, RAGGED>;
  constexpr int BM = S::BM, BN = S::BN, XROW = S::XROW, NS = S::NS;
  constexpr int XI = S::X_BYTES / 8192, WI = S::W_BYTES / 8192;  // loads of a wave per stage
  constexpr int SI = (BM + BN) / 512;                            // scale loads of a wave
  static_assert(S::X_BYTES % 8192 == 0 && S::W_BYTES % 8192 == 0 && (BM + BN) % 512 == 0, "tile");
  constexpr int PER = XI + WI + (RAGGED ? 0 : SI);
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * S::STAGE];

  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int wm = wave / WN, wn = wave % WN, r = lane & 31, h = lane >> 5;
  const int K = p.K, nb = K / 32, nk = (K + 127) / 128;
  const int ntt = (p.N + BN - 1) / BN, mtt = (p.T + BM - 1) / BM;
  int mi, ni;
  tile_of(blockIdx.x, ntt * mtt, mtt, ntt, mi, ni);
  const int t0 = mi * BM, n0 = ni * BN;

  // sources of this lane's loads: rows past the end repeat the last one
  const uint8_t* xsrc[XI];
  int xk[XI];
#pragma unroll
  for (int i = 0; i < XI; ++i) {
    constexpr int L = XROW / 16;  // lanes per row
    const int row = (wave * XI + i) * (64 / L) + lane / L;
    const int c = XMODE == 2 ? (lane & 3) ^ ((row >> 1) & 3) : (lane & 7) ^ (row & 7);
    xsrc[i] = p.x + (size_t)min(t0 + row, p.T - 1) * (XMODE == 2 ? K / 2 : K) + c * 16;
    xk[i] = c * (XMODE == 2 ? 32 : 16);
  }
  const uint8_t* wsrc[WI];
  int wk[WI];
#pragma unroll
  for (int i = 0; i < WI; ++i) {
    const int row = (wave * WI + i) * 16 + (lane >> 2);
    const int c = (lane & 3) ^ ((row >> 1) & 3);
    wsrc[i] = p.w + (size_t)min(n0 + row, p.N - 1) * (K / 2) + c * 16;
    wk[i] = c * 32;
  }
  // scale rows: the BN weight rows, then the BM token rows (with row scales
  // there is nothing to load for these: the weights' own are loaded again and
  // not read)
  const uint8_t* ssrc[SI];
#pragma unroll
  for (int i = 0; i < SI; ++i) {
    const int row = (wave * SI + i) * 64 + lane;
    if (row < BN || XMODE == 0)
      ssrc[i] = p.ws + (size_t)min(n0 + row % BN, p.N - 1) * nb;
    else
      ssrc[i] = (const uint8_t*)p.xs + (size_t)min(t0 + row - BN, p.T - 1) * nb;
  }
  auto issue = [&](int kt) {
    uint8_t* st = smem + (kt % NS) * S::STAGE;
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const uint8_t* src = xsrc[i] + (size_t)kt * XROW;
      if (RAGGED && kt * 128 + xk[i] >= K) src = kZeros;
      dma16(src, st + (wave * XI + i) * 1024);
    }
#pragma unroll
    for (int i = 0; i < WI; ++i) {
      const uint8_t* src = wsrc[i] + (size_t)kt * 64;
      if (RAGGED && kt * 128 + wk[i] >= K) src = kZeros;
      dma16(src, st + S::X_BYTES + (wave * WI + i) * 1024);
    }
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (!RAGGED) {
#pragma unroll
      for (int i = 0; i < SI; ++i)
        __builtin_amdgcn_global_load_lds(ssrc[i] + (size_t)kt * 4,
                                         st + S::X_BYTES + S::W_BYTES + (wave * SI + i) * 256, 4, 0, 0);
    }
#endif
  };
  // K not a multiple of 128: rows of scales are not 4-byte aligned; their bytes
  // go through registers, 127 (2^0) past the end
  auto ragged_scales = [&](int kt) {
    uint8_t* st = smem + (kt % NS) * S::STAGE + S::X_BYTES + S::W_BYTES;
#pragma unroll
    for (int i = 0; i < SI; ++i) {
      uint32_t v = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        v |= (uint32_t)(kt * 4 + b < nb ? ssrc[i][kt * 4 + b] : 127) << (8 * b);
      *reinterpret_cast<uint32_t*>(st + ((wave * SI + i) * 64 + lane) * 4) = v;
    }
  };

  // operand offsets in a stage
  int xo[FM], wo[FN], xso[FM], wso[FN], xsw[FM], wsw[FN];
#pragma unroll
  for (int f = 0; f < FM; ++f) {
    const int row = (wm * FM + f) * 32 + r;
    xo[f] = row * XROW;
    xsw[f] = XMODE == 2 ? (row >> 1) & 3 : row & 7;
    xso[f] = S::X_BYTES + S::W_BYTES + (BN + row) * 4;
  }
#pragma unroll
  for (int f = 0; f < FN; ++f) {
    const int row = (wn * FN + f) * 32 + r;
    wo[f] = S::X_BYTES + row * 64;
    wsw[f] = (row >> 1) & 3;
    wso[f] = S::X_BYTES + S::W_BYTES + row * 4;
  }

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;

#pragma unroll
  for (int s = 0; s < NS - 1; ++s)
    if (s < nk) issue(s);
  for (int kt = 0; kt < nk; ++kt) {
    if (RAGGED) ragged_scales(kt);
    if (kt + NS - 2 < nk)
      wait_vmcnt<(NS - 2) * PER>();
    else
      wait_vmcnt<0>();
    if (RAGGED) wait_lgkmcnt0();
    barrier_only();
    asm volatile("" ::: "memory");
    if (kt + NS - 1 < nk) issue(kt + NS - 1);
    const uint8_t* st = smem + (kt % NS) * S::STAGE;
    int wsc[FN], xsc[FM];
#pragma unroll
    for (int f = 0; f < FN; ++f)
      wsc[f] = (int)(*reinterpret_cast<const uint32_t*>(st + wso[f]) >> (8 * h));
#pragma unroll
    for (int f = 0; f < FM; ++f)
      xsc[f] = XMODE == 0 ? 0x7f7f7f7f
                          : (int)(*reinterpret_cast<const uint32_t*>(st + xso[f]) >> (8 * h));
    // two halves of 64 values; lane half h holds block h of each
    auto half = [&](auto jc) {
      constexpr int J = decltype(jc)::value;
      i32x8 wf[FN];
#pragma unroll
      for (int f = 0; f < FN; ++f) {
        const u32x4 v = ld16(st + wo[f] + (((2 * J + h) ^ wsw[f]) << 4));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          wf[f][q] = (int)v[q];
          wf[f][4 + q] = 0;
        }
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        i32x8 xf;
        if constexpr (XMODE == 2) {
          const u32x4 v = ld16(st + xo[i] + (((2 * J + h) ^ xsw[i]) << 4));
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            xf[q] = (int)v[q];
            xf[4 + q] = 0;
          }
        } else {
          const u32x4 v = ld16(st + xo[i] + (((4 * J + h) ^ xsw[i]) << 4));
          const u32x4 u = ld16(st + xo[i] + (((4 * J + 2 + h) ^ xsw[i]) << 4));
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            xf[q] = (int)v[q];
            xf[4 + q] = (int)u[q];
          }
        }
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              wf[j], xf, acc[i][j], 4, XMODE == 2 ? 4 : 0, 2 * J, wsc[j], 2 * J, xsc[i]);
      }
    };
    half(std::integral_constant<int, 0>{});
    half(std::integral_constant<int, 1>{});
    wait_lgkmcnt0();
    asm volatile("" ::: "memory");
  }

  // lane (r, h): token r of the fragment, columns 8 q + 4 h .. + 3
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int t = t0 + (wm * FM + i) * 32 + r;
    if (t >= p.T) continue;
    const float sc = XMODE == 0 ? ((const float*)p.xs)[t] : 1.0f;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + (wn * FN + j) * 32 + 8 * q + 4 * h;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e] * sc;
        const size_t at = (size_t)t * p.N + n;
        if (n + 4 <= p.N && p.N % 4 == 0) {
          if (OUT_F32)
            st16((float*)p.out + at, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]),
                                           __float_as_uint(v[2]), __float_as_uint(v[3])});
          else
            *reinterpret_cast<u32x2*>((uint16_t*)p.out + at) =
                u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < p.N) {
              if (OUT_F32)
                ((float*)p.out)[at + e] = v[e];
              else
                ((uint16_t*)p.out)[at + e] = (uint16_t)f32_to_bf16_bits(v[e]);
            }
        }
      }
  }
}

template <int XMODE, int FM, int FN, int WM, int WN>
void tile_launch(const Mx4LinearArgs& a, hipStream_t st) {
  using S = TileShape<XMODE, FM, FN, WM, WN, false>;
  const int grid = (a.T + S::BM - 1) / S::BM * ((a.N + S::BN - 1) / S::BN);
  const bool ragged = a.K % 128 != 0;
  if (ragged && a.out_f32)
    mx4_linear_tile_kernel<XMODE, FM, FN, WM, WN, true, true><<<grid, 512, 0, st>>>(a);
  else if (ragged)
    mx4_linear_tile_kernel<XMODE, FM, FN, WM, WN, true, false><<<grid, 512, 0, st>>>(a);
  else if (a.out_f32)
    mx4_linear_tile_kernel<XMODE, FM, FN, WM, WN, false, true><<<grid, 512, 0, st>>>(a);
  else
    mx4_linear_tile_kernel<XMODE, FM, FN, WM, WN, false, false><<<grid, 512, 0, st>>>(a);
}

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

size_t mx4_linear_workspace(int T, int N, int K, int x_mode) { return 0; }

hipError_t launch_mx4_linear(const Mx4LinearArgs& a, int x_mode, hipStream_t st) {
  const int grid = (a.N + 63) / 64 * ((a.T + 15) / 16);
  auto go = [&](auto m) {
    if (a.T > 64)
      tile_launch<decltype(m)::value, 4, 2, 2, 4>(a, st);
    else if (a.out_f32)
      mx4_linear_kernel<decltype(m)::value, true><<<grid, 256, 0, st>>>(a);
    else
      mx4_linear_kernel<decltype(m)::value, false><<<grid, 256, 0, st>>>(a);
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
