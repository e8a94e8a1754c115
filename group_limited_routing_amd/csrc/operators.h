// Launchers of the operators around the MoE block: RMS norm with the
// residual's addition, routing of given logits, MXFP4 quantisation and product.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.h"

namespace beam {

// ---------------------------------------------------------------- norm.hip
constexpr int kNormMaxH = 65536;

struct NormArgs {
  const void* x;          // [T, H]
  const void* stream_in;  // [T, H] or null
  const float* w;         // [H]
  void* stream_out;       // [T, H] or null
  void* y;                // [T, H] or null
  uint8_t* q;             // [T, H] E4M3 codes or null
  void* q_scale;          // [T] fp32 (row) or [T, H / 32] E8M0 (block)
  int T, H;
  float keep, add, eps;
};
// f32: x, stream and y are fp32 (else bf16); quant: 0 none, 1 row, 2 block
hipError_t launch_add_rms_norm(const NormArgs& a, int f32, int quant, hipStream_t st);

struct NormBwdArgs {
  const void* dy;            // [T, H]
  const void* s;             // [T, H], the forward's stream_out
  const float* w;            // [H]
  const void* d_stream_out;  // [T, H] or null
  void* dx;                  // [T, H]
  void* d_stream_in;         // [T, H] or null
  float* part;               // [groups, H] partial weight gradients or null
  float* dw;                 // [H] or null
  int T, H;
  float keep, add, eps;
};
// Workgroups of the backward pass with a weight gradient (rows of `part`).
int norm_bwd_groups(int T, int H);
hipError_t launch_add_rms_norm_backward(const NormBwdArgs& a, int f32, hipStream_t st);

// ---------------------------------------------------------------- gate.hip
constexpr int kGateMaxE = 1024;
constexpr int kGateMaxK = 32;

struct GateArgs {
  const void* z;         // [T, E] logits
  const float* bias;     // [E] or null
  const uint8_t* valid;  // [T] or null
  int32_t* idx;          // [T, k]
  float* w;              // [T, k]
  int32_t* counts;       // [E] or null
  int T, E, n_group, topk_group, k;
  int softmax, top2, renorm;
  float rsf;
};
hipError_t launch_gate(const GateArgs& a, int f32, hipStream_t st);

struct GateBwdArgs {
  const float* dw;     // [T, k]
  const void* z;       // [T, E]
  const int32_t* idx;  // [T, k]
  void* dz;            // [T, E]
  int T, E, k;
  int softmax, renorm;
  float rsf;
};
hipError_t launch_gate_backward(const GateBwdArgs& a, int f32, hipStream_t st);

// ---------------------------------------------------------------- mx4.hip
hipError_t launch_mx4_quantize(const void* x, int f32, int64_t rows, int C, int packed,
                               uint8_t* codes, uint8_t* scales, hipStream_t st);
hipError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int C,
                                 int f32, void* out, hipStream_t st);

struct Mx4LinearArgs {
  const uint8_t* x;    // [T, K] E4M3 codes or [T, K / 2] E2M1 codes
  const void* xs;      // [T] fp32 or [T, K / 32] E8M0
  const uint8_t* w;    // [N, K / 2] E2M1 codes
  const uint8_t* ws;   // [N, K / 32] E8M0
  void* out;           // [T, N]
  int T, N, K;
  int out_f32;
};
// x_mode: 0 E4M3 with row scales, 1 E4M3 with block scales, 2 MXFP4
hipError_t launch_mx4_linear(const Mx4LinearArgs& a, int x_mode, hipStream_t st);

}  // namespace beam
