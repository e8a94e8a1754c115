// The dense MLP's gated product: h = act(x Wg^T) * (x Wu^T) in one kernel, and its
// gradient.
//
// Beam launch post ("Introducing Beam"), section "Mixture of Experts": the first
// three layers have a dense SwiGLU MLP in place of the experts.
#include "common.h"
#include "operators.h"

namespace beam {
namespace {

// act(g), and its derivative in d. gelu by erfc, which keeps its relative accuracy
// where 1 + erf cancels (g below -3).
template <bool GELU>
__device__ __forceinline__ float activation(float g) {
  if constexpr (GELU)
    return 0.5f * g * erfcf(g * -0.70710678118654752f);
  else
    return silu_f32(g);
}
template <bool GELU>
__device__ __forceinline__ float activation(float g, float& d) {
  if constexpr (GELU) {
    const float p = 0.5f * erfcf(g * -0.70710678118654752f);
    d = p + g * 0.39894228040143268f * __builtin_amdgcn_exp2f(g * g * -0.72134752044448170f);
    return g * p;
  } else {
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f));
    d = s * (1.0f + g * (1.0f - s));
    return g * s;
  }
}

// ------------------------------------------------------------------ simple product
// element (row, k) at p[row * rs + k * ks]
struct Operand {
  const uint16_t* p;
  int64_t rs, ks;
};

__device__ __forceinline__ void stage64(const Operand& o, int row0, int rows, int k0, int K,
                                        uint16_t (*tile)[40]) {
  const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 8;
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + r, k = k0 + c + i;
    tile[r][c + i] = row < rows && k < K ? o.p[row * o.rs + k * o.ks] : 0;
  }
}

// acc += A B^T of a 64 x 64 tile; wave w has rows 16 w .. + 15.
__device__ __forceinline__ void product64(const Operand& a, const Operand& b, int m0, int M, int n0, int N,
                                          int K, uint16_t (*at)[40], uint16_t (*bt)[40], f32x4 (&acc)[4]) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int k0 = 0; k0 < K; k0 += 32) {
    __syncthreads();
    stage64(a, m0, M, k0, K, at);
    stage64(b, n0, N, k0, K, bt);
    __syncthreads();
    const bf16x8 af = as_bf16x8(ld16(&at[wave * 16 + lane % 16][lane / 16 * 8]));
    for (int j = 0; j < 4; ++j)
      acc[j] = mfma_bf16(af, as_bf16x8(ld16(&bt[j * 16 + lane % 16][lane / 16 * 8])), acc[j]);
  }
}

template <bool GELU>
__global__ __launch_bounds__(256) void gated_kernel(GatedArgs p) {
  __shared__ __attribute__((aligned(16))) uint16_t at[64][40], bt[64][40];
  const int n0 = blockIdx.x * 64, m0 = blockIdx.y * 64;
  f32x4 g[4] = {}, u[4] = {};
  const Operand x{p.x, p.H, 1};
  product64(x, Operand{p.wg, p.H, 1}, m0, p.T, n0, p.F, p.H, at, bt, g);
  product64(x, Operand{p.wu, p.H, 1}, m0, p.T, n0, p.F, p.H, at, bt, u);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int j = 0; j < 4; ++j)
    for (int q = 0; q < 4; ++q) {
      const int m = m0 + wave * 16 + lane / 16 * 4 + q, n = n0 + j * 16 + lane % 16;
      if (m >= p.T || n >= p.F) continue;
      const size_t i = (size_t)m * p.F + n;
      float gv = g[j][q], uv = u[j][q];
      if (p.add_gate) gv += bf16_bits_to_f32(p.add_gate[i]);
      if (p.add_up) uv += bf16_bits_to_f32(p.add_up[i]);
      p.h[i] = (uint16_t)f32_to_bf16_bits(activation<GELU>(gv) * uv);
      if (p.gate) p.gate[i] = (uint16_t)f32_to_bf16_bits(gv);
      if (p.up) p.up[i] = (uint16_t)f32_to_bf16_bits(uv);
    }
}

// out [M, N] = A0 B0^T + A1 B1^T
__global__ __launch_bounds__(256) void sum_kernel(Operand a0, Operand b0, Operand a1, Operand b1, int M,
                                                  int N, int K, uint16_t* out) {
  __shared__ __attribute__((aligned(16))) uint16_t at[64][40], bt[64][40];
  const int n0 = blockIdx.x * 64, m0 = blockIdx.y * 64;
  f32x4 acc[4] = {};
  product64(a0, b0, m0, M, n0, N, K, at, bt, acc);
  if (a1.p) product64(a1, b1, m0, M, n0, N, K, at, bt, acc);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int j = 0; j < 4; ++j)
    for (int q = 0; q < 4; ++q) {
      const int m = m0 + wave * 16 + lane / 16 * 4 + q, n = n0 + j * 16 + lane % 16;
      if (m < M && n < N) out[(size_t)m * N + n] = (uint16_t)f32_to_bf16_bits(acc[j][q]);
    }
}

// d_up = dh act(gate), d_gate = dh up act'(gate), 8 values a thread. Rounded to bf16,
// which is their type as outputs and as operands of the products.
template <bool GELU>
__global__ __launch_bounds__(256) void gated_grad_kernel(GatedBwdArgs p) {
  const int64_t n8 = (int64_t)p.T * p.F / 8, stride = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += stride) {
    const u32x4 dh = ld16(p.dh + i * 8), g = ld16(p.gate + i * 8), u = ld16(p.up + i * 8);
    u32x4 dg, du;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float a[2], b[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        auto half = [&](uint32_t v) { return __uint_as_float(e ? v & 0xffff0000u : v << 16); };
        float d;
        const float f = activation<GELU>(half(g[q]), d), dhv = half(dh[q]);
        a[e] = dhv * half(u[q]) * d;
        b[e] = dhv * f;
      }
      dg[q] = pack_bf16x2(a[0], a[1]);
      du[q] = pack_bf16x2(b[0], b[1]);
    }
    st16(p.d_gate + i * 8, dg);
    st16(p.d_up + i * 8, du);
  }
}

}  // namespace

hipError_t launch_gated_linear(const GatedArgs& a, int gelu, hipStream_t st) {
  const dim3 grid((a.F + 63) / 64, (a.T + 63) / 64);
  if (gelu)
    gated_kernel<true><<<grid, 256, 0, st>>>(a);
  else
    gated_kernel<false><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

size_t gated_bwd_workspace_bytes(int T, int H, int F) { return 0; }

hipError_t launch_gated_linear_backward(const GatedBwdArgs& a, int gelu, hipStream_t st) {
  const int64_t n8 = (int64_t)a.T * a.F / 8;
  const unsigned grid = (unsigned)((n8 + 255) / 256 < (1 << 20) ? (n8 + 255) / 256 : 1 << 20);
  if (gelu)
    gated_grad_kernel<true><<<grid, 256, 0, st>>>(a);
  else
    gated_grad_kernel<false><<<grid, 256, 0, st>>>(a);
  const Operand none{nullptr, 0, 0}, xt{a.x, 1, a.H};
  if (a.dx)
    sum_kernel<<<dim3((a.H + 63) / 64, (a.T + 63) / 64), 256, 0, st>>>(
        Operand{a.d_gate, a.F, 1}, Operand{a.wg, 1, a.H}, Operand{a.d_up, a.F, 1}, Operand{a.wu, 1, a.H},
        a.T, a.H, a.F, a.dx);
  if (a.d_wg) {
    const dim3 g((a.H + 63) / 64, (a.F + 63) / 64);
    sum_kernel<<<g, 256, 0, st>>>(Operand{a.d_gate, 1, a.F}, xt, none, none, a.F, a.H, a.T, a.d_wg);
    sum_kernel<<<g, 256, 0, st>>>(Operand{a.d_up, 1, a.F}, xt, none, none, a.F, a.H, a.T, a.d_wu);
  }
  return hipGetLastError();
}

}  // namespace beam
