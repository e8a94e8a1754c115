// Launchers of the operators around the MoE block: RMS norm with the
// residual's addition, routing of given logits, MXFP4 quantisation and product,
// and the dense MLP's gated product, its adapters and dropout.
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

// ---------------------------------------------------------------- mlp.hip
constexpr int kMlpMaxH = 65536;    // hidden
constexpr int kMlpMaxF = 262144;   // intermediate

struct GatedArgs {
  const uint16_t* x;         // [T, H] bf16
  const uint16_t* wg;        // [F, H]
  const uint16_t* wu;        // [F, H]
  const uint16_t* add_gate;  // [T, F] or null
  const uint16_t* add_up;    // [T, F] or null
  uint16_t* h;               // [T, F]
  void* gate;                // [T, F] bf16, or fp32, or null
  void* up;                  // as gate
  float* part;               // workspace: sums over parts of H
  int T, H, F;
  bool pre_f32;              // gate and up are fp32
};
size_t gated_workspace_bytes(int T, int H, int F);
// gelu: the activation is gelu (else silu)
hipError_t launch_gated_linear(const GatedArgs& a, int gelu, hipStream_t st);

struct GatedBwdArgs {
  const uint16_t* dh;    // [T, F] bf16
  const uint16_t* x;     // [T, H]
  const uint16_t* wg;    // [F, H]
  const uint16_t* wu;    // [F, H]
  const void* gate;      // [T, F] bf16 or fp32
  const void* up;        // as gate
  uint16_t* d_gate;      // [T, F]
  uint16_t* d_up;        // [T, F]
  uint16_t* dx;          // [T, H] or null
  uint16_t* d_wg;        // [F, H] or null (both or none)
  uint16_t* d_wu;        // [F, H]
  float* part;           // workspace: sums over parts of a product's reduction
  int T, H, F;
  bool pre_f32;          // gate and up are fp32
};
size_t gated_bwd_workspace_bytes(int T, int H, int F);
hipError_t launch_gated_linear_backward(const GatedBwdArgs& a, int gelu, hipStream_t st);

// ---------------------------------------------------------------- lora.hip
constexpr int kLoraMaxR = 128;
constexpr int kLoraMaxE = 1024;

// A plan: int32 words. The tokens in order of their adapter, those without one
// last (stable), cut into tiles of one adapter's tokens and, for the gradients
// of the adapters, into longer chunks.
constexpr int kLoraTile = 64;
struct LoraPlanLayout {
  int chunk;          // tokens of a chunk: 1024, or so many that T tokens make at most 65
  int tiles, chunks;  // at most
  int slots;          // chunks, at most, of adapters that have more than one
  int padded;         // tokens, at most, with every adapter's rounded up to 32
  size_t o_order, o_tiles, o_tokens, o_chunks, o_first, o_slot, words;
  __host__ __device__ LoraPlanLayout(int T, int E) {
    const int used = E < T ? E : T;
    chunk = T <= 64 * 1024 ? 1024 : (T / 64 + 511) & ~511;
    tiles = T / kLoraTile + (E + 1 < T ? E + 1 : T);
    chunks = T / chunk + used;
    slots = 2 * (T / chunk);  // n > chunk tokens make at most 2 n / chunk chunks
    padded = (T + 31 * used + 31) & ~31;
    auto up4 = [](size_t n) { return (n + 3) & ~(size_t)3; };
    o_order = 16;                           // [0] tiles, [1] chunks
    o_tiles = o_order + up4(T);             // {adapter or -1, first, count, first of the padded order}
    o_tokens = o_tiles + 4 * (size_t)tiles; // [tiles, 64], the last one repeated
    o_chunks = o_tokens + kLoraTile * (size_t)tiles;  // as the tiles
    o_first = o_chunks + 4 * (size_t)chunks;  // [E + 1] first chunk of an adapter
    o_slot = o_first + up4((size_t)E + 1);    // [E] first slot of an adapter with several chunks
    words = o_slot + up4(E);
  }
};
hipError_t launch_lora_plan(const int32_t* index, int T, int E, int32_t* plan, hipStream_t st);

struct LoraArgs {
  const uint16_t* x;     // [T, K] bf16
  const uint16_t* a;     // [E, R, K]
  const uint16_t* b;     // [E, N, R]
  const float* scale;    // [E] or null
  const int32_t* plan;
  const uint16_t* base;  // [T, N] or null
  uint16_t* out;         // [T, N]
  float* v;              // [T, R] or null
  float* part;           // workspace
  int T, K, N, R, E;
};
size_t lora_workspace_bytes(int T, int K, int N, int R, int E);
hipError_t launch_lora(const LoraArgs& a, hipStream_t st);

struct LoraBwdArgs {
  const uint16_t* dy;    // [T, N] bf16
  const uint16_t* x;     // [T, K]
  const float* v;        // [T, R]
  const uint16_t* a;     // [E, R, K]
  const uint16_t* b;     // [E, N, R]
  const float* scale;    // [E] or null
  const int32_t* plan;
  const uint16_t* base;  // [T, K] or null
  uint16_t* dx;          // [T, K] or null
  uint16_t* da;          // [E, R, K] or null (both or none)
  uint16_t* db;          // [E, N, R]
  void* workspace;
  int T, K, N, R, E;
};
size_t lora_bwd_workspace_bytes(int T, int K, int N, int R, int E);
hipError_t launch_lora_backward(const LoraBwdArgs& a, hipStream_t st);

// ---------------------------------------------------------------- dropout.hip
struct DropoutArgs {
  const void* x;              // [n]
  const void* stream_in;      // [n] or null
  void* out;                  // [n]
  void* kept_grad;            // [n] or null: keep * x
  const int64_t* offset_dev;  // [1] or null, added to offset
  uint64_t seed, offset;
  int64_t n;
  uint32_t border;            // of 65536: elements whose 16 random bits are below it are 0
  float scale, keep, add;     // scale = 1 / (1 - border / 65536)
};
hipError_t launch_dropout(const DropoutArgs& a, int f32, hipStream_t st);

}  // namespace beam
