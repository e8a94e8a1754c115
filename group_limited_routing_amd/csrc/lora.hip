// Low-rank adapters of many requests beside a shared projection: out = base + s_i B_i
// A_i x for the adapter i of each token, and the gradients.
//
// Beam launch post ("Introducing Beam"), section "Post-training": rank-16 adapters on
// the dense MLP and the experts.
#include "common.h"
#include "operators.h"
#include "wave.h"

#include <algorithm>

namespace beam {
namespace {

constexpr int kPlanWaves = 16;

// One workgroup: counts of each wave's part of the tokens, offsets by a scan over
// the adapters, then each wave places its part in order, so the order is stable.
__global__ __launch_bounds__(64 * kPlanWaves) void lora_plan_kernel(const int32_t* __restrict__ index, int T,
                                                                    int E, int32_t* __restrict__ plan) {
  __shared__ int32_t part[kPlanWaves][kLoraMaxE + 1];
  __shared__ int32_t start[kLoraMaxE + 2], tile0[kLoraMaxE + 2], chunk0[kLoraMaxE + 2];
  const LoraPlanLayout at(T, E);
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, G = E + 1;
  const int per = ((T + kPlanWaves - 1) / kPlanWaves + 63) & ~63;
  const int t0 = min(wave * per, T), t1 = min(t0 + per, T);
  for (int i = lane; i < G; i += 64) part[wave][i] = 0;
  __syncthreads();
  auto group = [&](int t) {
    const int e = index[t];
    return e >= 0 && e < E ? e : E;
  };
  for (int t = t0 + lane; t < t1; t += 64) atomicAdd(&part[wave][group(t)], 1);
  __syncthreads();
  if (wave == 0) {  // exclusive scans of the groups' tokens, tiles and chunks
    int s = 0, ts = 0, cs = 0;
    for (int g0 = 0; g0 < G; g0 += 64) {
      const int g = g0 + lane;
      int n = 0;
      if (g < G)
        for (int w = 0; w < kPlanWaves; ++w) n += part[w][g];
      const int nt = (n + kLoraTile - 1) / kLoraTile, nc = g < E ? (n + kLoraChunk - 1) / kLoraChunk : 0;
      int a = n, b = nt, c = nc;
      for (int d = 1; d < 64; d <<= 1) {
        const int oa = __shfl_up(a, d), ob = __shfl_up(b, d), oc = __shfl_up(c, d);
        if (lane >= d) a += oa, b += ob, c += oc;
      }
      if (g < G) {
        start[g] = s + a - n;
        tile0[g] = ts + b - nt;
        chunk0[g] = cs + c - nc;
      }
      s += __shfl(a, 63);
      ts += __shfl(b, 63);
      cs += __shfl(c, 63);
    }
    if (lane == 0) {
      start[G] = s;
      tile0[G] = ts;
      chunk0[G] = cs;
      plan[0] = ts;
      plan[1] = cs;
    }
  }
  __syncthreads();
  for (int g = tid; g < G; g += 64 * kPlanWaves) {
    int s = start[g];
    for (int w = 0; w < kPlanWaves; ++w) {
      const int n = part[w][g];
      part[w][g] = s;
      s += n;
    }
    plan[at.o_first + g] = chunk0[g];  // chunk0[E]: all of them
  }
  int4* tiles = reinterpret_cast<int4*>(plan + at.o_tiles);
  int4* chunks = reinterpret_cast<int4*>(plan + at.o_chunks);
  for (int g = 0; g < G; ++g) {
    const int s = start[g], n = start[g + 1] - s, e = g < E ? g : -1;
    for (int j = tid; j * kLoraTile < n; j += 64 * kPlanWaves)
      tiles[tile0[g] + j] = make_int4(e, s + j * kLoraTile, min(kLoraTile, n - j * kLoraTile), 0);
    if (g < E)
      for (int j = tid; j * kLoraChunk < n; j += 64 * kPlanWaves)
        chunks[chunk0[g] + j] = make_int4(e, s + j * kLoraChunk, min(kLoraChunk, n - j * kLoraChunk), 0);
  }
  __syncthreads();
  int32_t* order = plan + at.o_order;
  for (int t = t0; t < t1; t += 64) {
    const bool live = t + lane < t1;
    const int g = live ? group(t + lane) : -1;
    uint64_t left = __ballot(live);
    while (left) {
      const int lead = __ffsll((unsigned long long)left) - 1, lg = __shfl(g, lead);
      const uint64_t same = __ballot(live && g == lg);
      int base = 0;
      if (lane == lead) base = atomicAdd(&part[wave][lg], __popcll(same));
      base = __shfl(base, lead);
      if (live && g == lg) order[base + __popcll(same & ((1ull << lane) - 1))] = t + lane;
      left &= ~same;
    }
  }
}

__device__ __forceinline__ float bf(const uint16_t* p, size_t i) { return bf16_bits_to_f32(p[i]); }

// ------------------------------------------------------------------ simple kernels
// v[t, r] = f sum over k of x[t, k] m[e][r * rs + k * ks]; a workgroup per token tile
// and r, a wave per token in turn.
__global__ __launch_bounds__(256) void lora_in_kernel(const uint16_t* x, const uint16_t* m, const float* scale,
                                                      const int32_t* plan, int T, int E, int R, int K,
                                                      int rs, int ks, float* v) {
  const LoraPlanLayout at(T, E);
  if ((int)blockIdx.x >= plan[0]) return;
  const int4 tile = reinterpret_cast<const int4*>(plan + at.o_tiles)[blockIdx.x];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = blockIdx.y;
  for (int i = wave; i < tile.z; i += 4) {
    const int t = plan[at.o_order + tile.y + i];
    float s = 0.f;
    if (tile.x >= 0)
      for (int k = lane; k < K; k += 64)
        s += bf(x, (size_t)t * K + k) * bf(m, (size_t)tile.x * R * K + (size_t)r * rs + (size_t)k * ks);
    s = wave_sum(s);
    if (lane == 0) v[(size_t)t * R + r] = tile.x >= 0 && scale ? s * scale[tile.x] : s;
  }
}

// out[t, n] = base[t, n] + f sum over r of v[t, r] m[e][n * ns + r * rs]
__global__ __launch_bounds__(256) void lora_out_kernel(const float* v, const uint16_t* m, const float* scale,
                                                       const int32_t* plan, int T, int E, int R, int N, int ns,
                                                       int rs, const uint16_t* base, uint16_t* out) {
  const LoraPlanLayout at(T, E);
  if ((int)blockIdx.x >= plan[0]) return;
  const int4 tile = reinterpret_cast<const int4*>(plan + at.o_tiles)[blockIdx.x];
  const int n = blockIdx.y * 256 + threadIdx.x;
  if (n >= N) return;
  for (int i = 0; i < tile.z; ++i) {
    const int t = plan[at.o_order + tile.y + i];
    float s = 0.f;
    if (tile.x >= 0) {
      for (int r = 0; r < R; ++r)
        s += v[(size_t)t * R + r] * bf(m, (size_t)tile.x * R * N + (size_t)n * ns + (size_t)r * rs);
      if (scale) s *= scale[tile.x];
    }
    const size_t o = (size_t)t * N + n;
    out[o] = (uint16_t)f32_to_bf16_bits(base ? s + bf(base, o) : s);
  }
}

// d[e][r * rs + c * cs] = f sum over the adapter's tokens of v[t, r] x[t, c]
__global__ __launch_bounds__(256) void lora_grad_kernel(const float* v, const uint16_t* x, const float* scale,
                                                        const int32_t* plan, int T, int E, int R, int C, int rs,
                                                        int cs, uint16_t* d) {
  const LoraPlanLayout at(T, E);
  const int e = blockIdx.z, r = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
  if (c >= C) return;
  float s = 0.f;
  for (int j = plan[at.o_first + e]; j < plan[at.o_first + e + 1]; ++j) {
    const int4 ch = reinterpret_cast<const int4*>(plan + at.o_chunks)[j];
    for (int i = 0; i < ch.z; ++i) {
      const int t = plan[at.o_order + ch.y + i];
      s += v[(size_t)t * R + r] * bf(x, (size_t)t * C + c);
    }
  }
  if (scale) s *= scale[e];
  d[(size_t)e * R * C + (size_t)r * rs + (size_t)c * cs] = (uint16_t)f32_to_bf16_bits(s);
}

}  // namespace

hipError_t launch_lora_plan(const int32_t* index, int T, int E, int32_t* plan, hipStream_t st) {
  lora_plan_kernel<<<1, 64 * kPlanWaves, 0, st>>>(index, T, E, plan);
  return hipGetLastError();
}

size_t lora_workspace_bytes(int T, int K, int N, int R, int E) { return (size_t)T * R * sizeof(float); }

hipError_t launch_lora(const LoraArgs& p, hipStream_t st) {
  const LoraPlanLayout at(p.T, p.E);
  float* v = p.v ? p.v : p.part;
  lora_in_kernel<<<dim3(at.tiles, p.R), 256, 0, st>>>(p.x, p.a, nullptr, p.plan, p.T, p.E, p.R, p.K, p.K, 1, v);
  lora_out_kernel<<<dim3(at.tiles, (p.N + 255) / 256), 256, 0, st>>>(v, p.b, p.scale, p.plan, p.T, p.E, p.R,
                                                                     p.N, p.R, 1, p.base, p.out);
  return hipGetLastError();
}

size_t lora_bwd_workspace_bytes(int T, int K, int N, int R, int E) { return (size_t)T * R * sizeof(float); }

hipError_t launch_lora_backward(const LoraBwdArgs& p, hipStream_t st) {
  const LoraPlanLayout at(p.T, p.E);
  float* dv = (float*)p.workspace;
  lora_in_kernel<<<dim3(at.tiles, p.R), 256, 0, st>>>(p.dy, p.b, p.scale, p.plan, p.T, p.E, p.R, p.N, 1, p.R,
                                                      dv);
  if (p.dx)
    lora_out_kernel<<<dim3(at.tiles, (p.K + 255) / 256), 256, 0, st>>>(dv, p.a, nullptr, p.plan, p.T, p.E, p.R,
                                                                       p.K, 1, p.K, p.base, p.dx);
  if (p.da) {
    lora_grad_kernel<<<dim3((p.K + 255) / 256, p.R, p.E), 256, 0, st>>>(dv, p.x, nullptr, p.plan, p.T, p.E, p.R,
                                                                        p.K, p.K, 1, p.da);
    lora_grad_kernel<<<dim3((p.N + 255) / 256, p.R, p.E), 256, 0, st>>>(p.v, p.dy, p.scale, p.plan, p.T, p.E,
                                                                        p.R, p.N, 1, p.R, p.db);
  }
  return hipGetLastError();
}

}  // namespace beam
