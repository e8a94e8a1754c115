// Low-rank adapters of many requests beside a shared projection: out = base + s_i B_i
// A_i x for the adapter i of each token, and the gradients.
//
// Beam launch post ("Introducing Beam"), section "Post-training": rank-16 adapters on
// the dense MLP and the experts.
#include "common.h"
#include "operators.h"
#include "tile.h"
#include "wave.h"

#include <algorithm>

namespace beam {
namespace {

constexpr int kPlanWaves = 16;
constexpr int kMaxParts = 8;  // of a reduction over k

// One workgroup: counts of each wave's part of the tokens, offsets by a scan over
// the adapters, then each wave places its part in order, so the order is stable. Bound by latency:
// a turn for each different adapter among 64 tokens, and the last tile's repeated tokens one by
// one. 515 tokens in any order of 5 adapters 8 us, 64 of 32 18, 8192 of 8 26 (one after the
// other 19), 4096 of 64 57, 16384 of 256 265.
__global__ __launch_bounds__(64 * kPlanWaves) void lora_plan_kernel(const int32_t* __restrict__ index, int T,
                                                                    int E, int32_t* plan) {
  __shared__ int32_t part[kPlanWaves][kLoraMaxE + 1];
  __shared__ int32_t start[kLoraMaxE + 2], tile0[kLoraMaxE + 2], chunk0[kLoraMaxE + 2], padded0[kLoraMaxE + 2];
  const LoraPlanLayout at(T, E);
  const int chunk = at.chunk;
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
  if (wave == 0) {  // exclusive scans of the groups' tokens, tiles, chunks, slots and padded tokens
    int total[5] = {};
    for (int g0 = 0; g0 < G; g0 += 64) {
      const int g = g0 + lane;
      int n = 0;
      if (g < G)
        for (int w = 0; w < kPlanWaves; ++w) n += part[w][g];
      const int nc = g < E ? (n + chunk - 1) / chunk : 0;
      const int own[5] = {n, (n + kLoraTile - 1) / kLoraTile, nc, nc > 1 ? nc : 0, g < E ? (n + 31) & ~31 : 0};
      int before[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        int v = own[i];
        for (int d = 1; d < 64; d <<= 1) {
          const int o = __shfl_up(v, d);
          if (lane >= d) v += o;
        }
        before[i] = total[i] + v - own[i];
        total[i] += __shfl(v, 63);
      }
      if (g < G) {
        start[g] = before[0];
        tile0[g] = before[1];
        chunk0[g] = before[2];
        padded0[g] = before[4];
        if (g < E) plan[at.o_slot + g] = nc > 1 ? before[3] : -1;
      }
    }
    if (lane == 0) {
      start[G] = total[0];
      plan[0] = total[1];
      plan[1] = total[2];
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
      tiles[tile0[g] + j] = make_int4(e, s + j * kLoraTile, min(kLoraTile, n - j * kLoraTile), padded0[g] + j * kLoraTile);
    if (g < E)
      for (int j = tid; j * chunk < n; j += 64 * kPlanWaves)
        chunks[chunk0[g] + j] = make_int4(e, s + j * chunk, min(chunk, n - j * chunk), padded0[g] + j * chunk);
  }
  __syncthreads();
  int32_t *order = plan + at.o_order, *tokens = plan + at.o_tokens;
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
      if (live && g == lg) {
        const int pos = base + __popcll(same & ((1ull << lane) - 1));
        order[pos] = t + lane;
        tokens[(size_t)tile0[lg] * kLoraTile + pos - start[lg]] = t + lane;
      }
      left &= ~same;
    }
  }
  __syncthreads();
  for (int g = tid; g < G; g += 64 * kPlanWaves) {
    const int n = start[g + 1] - start[g];
    int32_t* end = tokens + (size_t)tile0[g] * kLoraTile + n;
    for (int i = n; i % kLoraTile != 0; ++i) *end++ = tokens[(size_t)tile0[g] * kLoraTile + n - 1];
  }
}

__device__ __forceinline__ int4 tile_at(const int32_t* plan, const LoraPlanLayout& at, int i) {
  return reinterpret_cast<const int4*>(plan + at.o_tiles)[i];
}
__device__ __forceinline__ int4 chunk_at(const int32_t* plan, const LoraPlanLayout& at, int i) {
  return reinterpret_cast<const int4*>(plan + at.o_chunks)[i];
}

// A launch of `parts` workgroups for each of `tiles` tiles, dealt so that a tile's are on one
// XCD (workgroups go to the 8 XCDs in turn) and run one after the other: each XCD then
// works on rows of its own, whose pages its address translation holds. (With a tile's parts on
// several XCDs, 8192 x 5120 in 2 parts took 36 us, so 23.)
int grid_of(int tiles, int parts) { return (tiles + 7) / 8 * 8 * parts; }
__device__ __forceinline__ void place(int parts, int& tile, int& part) {
  const int q = blockIdx.x >> 3;
  part = q % parts;
  tile = q / parts * 8 + (blockIdx.x & 7);
}

// The tokens of a tile that are this lane's MFMA columns. What a tile's work
// begins with, its record and its tokens, stands at places that the workgroup's number
// gives, and is read at once: each read after another costs a microsecond.
__device__ __forceinline__ void tile_tokens(const int32_t* plan, const LoraPlanLayout& at, int tile,
                                            int (&tokens)[4]) {
#pragma unroll
  for (int b = 0; b < 4; ++b)
    tokens[b] = plan[at.o_tokens + (size_t)tile * kLoraTile + b * 16 + (threadIdx.x & 15)];
}

// f(i, sum over the parts, in their order, of the 4 values at from(i)) for this thread's i of
// `count`; parts is 1, 2, 4 or 8, all of an i's loads go out together.
template <typename From, typename F>
__device__ __forceinline__ void each_sum(int count, int parts, size_t pitch, From from, F f) {
  auto go = [&](auto pc) {
    constexpr int P = decltype(pc)::value;
    for (int i = threadIdx.x; i < count; i += 256) {
      const float* at = from(i);
      f32x4 w[P];
#pragma unroll
      for (int q = 0; q < P; ++q) w[q] = *reinterpret_cast<const f32x4*>(at + q * pitch);
      f32x4 s = w[0];
#pragma unroll
      for (int q = 1; q < P; ++q) s += w[q];
      f(i, s);
    }
  };
  if (parts == 1)
    go(std::integral_constant<int, 1>{});
  else if (parts == 2)
    go(std::integral_constant<int, 2>{});
  else if (parts == 4)
    go(std::integral_constant<int, 4>{});
  else
    go(std::integral_constant<int, kMaxParts>{});
}

// v as the sum of two bf16 values, 16 significant bits (a finite v that would round beyond the
// largest bf16 number is that number and the rest); an infinity or a NaN is the first alone.
__device__ __forceinline__ void split(float v, uint32_t& hi, uint32_t& lo) {
  hi = f32_to_bf16_bits(v);
  if ((hi & 0x7fffu) == 0x7f80u && (__float_as_uint(v) & 0x7fffffffu) != 0x7f800000u) --hi;
  const float rest = v - bf16_bits_to_f32(hi);
  lo = (hi & 0x7f80u) == 0x7f80u ? 0u : f32_to_bf16_bits(rest);
}

// Eight bf16 values with zeros for infinities and NaN. The second part of a v is 0 or of either
// sign, so its product with an infinity would turn the first part's into a NaN: it gets these.
// lora_out_kernel looks for them among the adapter's values before it multiplies, at 4 RB products
// with zeros for 64 columns (8192 x 5120 x 10240 of rank 16: 120 us, without 119; gradient of rank
// 64, 8191 x 5120 x 5120: 167, without 164; smallest calls 0.3 us). lora_grad_kernel, which holds no operand for long, makes a sum again that came
// out as a NaN.
__device__ __forceinline__ u32x4 finite(u32x4 m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t low = (m[i] & 0x7f80u) == 0x7f80u ? 0u : m[i] & 0xffffu;
    const uint32_t high = (m[i] & 0x7f800000u) == 0x7f800000u ? 0u : m[i] & 0xffff0000u;
    m[i] = low | high;
  }
  return m;
}

// ------------------------------------------------------------------ into the rank
// part[ks][position][r] = sum over a part of k of x[t, k] m[e][r, k]: a workgroup per
// tile of tokens and part of k, its waves take 128 values of k in turn, and the four
// sums are added through LDS. MFMA rows are r, columns tokens; both operands go from
// memory into registers, 64 bytes of a row at a time. Bound by reading x: 8192 x 5120 (84 MB)
// 23 us warm and 30 to 39 us from memory (2.2 to 2.8 TB/s), of ranks 16 and 64; a kernel that only
// reads x in this order takes 15 us warm.
template <int RB, int TB>
__device__ __forceinline__ void rank_sums(const uint16_t* x, const uint16_t* m, const int (&tokens)[4], int R, int K, int first, int step, f32x4 (&acc)[TB][RB]) {
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const uint16_t* xr[TB];
  const uint16_t* mr[RB];
#pragma unroll
  for (int b = 0; b < TB; ++b) xr[b] = x + (size_t)tokens[b] * K + g * 8;
#pragma unroll
  for (int b = 0; b < RB; ++b) mr[b] = m + (size_t)min(b * 16 + l, R - 1) * K + g * 8;
  constexpr int S = TB * RB > 8 ? 2 : 4;  // steps of 32 whose loads go out together
  auto group = [&](int k0, auto end) {
    u32x4 xf[S][TB], mf[S][RB];
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int k = k0 + s * 32;
      // past the end (K is a multiple of 8) zeros, from an address: a load that some lanes
      // leave out would be a branch of its own
      const bool in = !decltype(end)::value || k + g * 8 < K;
#pragma unroll
      for (int b = 0; b < TB; ++b) xf[s][b] = ld16(in ? (const void*)(xr[b] + k) : (const void*)kZeros);
#pragma unroll
      for (int b = 0; b < RB; ++b) mf[s][b] = ld16(in ? (const void*)(mr[b] + k) : (const void*)kZeros);
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int b = 0; b < TB; ++b)
#pragma unroll
        for (int q = 0; q < RB; ++q)
          acc[b][q] = mfma_bf16(as_bf16x8(mf[s][q]), as_bf16x8(xf[s][b]), acc[b][q]);
  };
  int k0 = first * S * 32;
  for (; k0 + S * 32 <= K; k0 += step * S * 32) group(k0, std::false_type{});
  if (k0 < K) group(k0, std::true_type{});
}

template <int RB>
__global__ __launch_bounds__(256, RB <= 2 ? 4 : RB <= 4 ? 2 : 1) void lora_in_kernel(const uint16_t* __restrict__ x,
                                                      const uint16_t* __restrict__ m,
                                                      const int32_t* __restrict__ plan, int parts, int T,
                                                      int E, int R, int K, float* __restrict__ part) {
  __shared__ f32x4 sums[4][4][RB][64];
  const LoraPlanLayout at(T, E);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int number, mine;
  place(parts, number, mine);
  if (number >= at.tiles) return;
  const int4 tile = tile_at(plan, at, number);
  int tokens[4];
  tile_tokens(plan, at, number, tokens);
  if (number >= plan[0] || tile.x < 0) return;  // no adapter: nothing reads these sums
  const uint16_t* me = m + (size_t)tile.x * R * K;
  const int step = parts * 4, first = mine * 4 + wave, tb = (tile.z + 15) / 16;
  auto run = [&](auto n) {
    constexpr int TB = decltype(n)::value;
    f32x4 acc[TB][RB] = {};
    rank_sums<RB, TB>(x, me, tokens, R, K, first, step, acc);
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int q = 0; q < RB; ++q) sums[wave][b][q][lane] = acc[b][q];
  };
  if (tb == 1)
    run(std::integral_constant<int, 1>{});
  else if (tb == 2)
    run(std::integral_constant<int, 2>{});
  else
    run(std::integral_constant<int, 4>{});
  __syncthreads();
  // lane (token l, rows 4 g ..): 4 consecutive values of r
  for (int i = wave; i < tb * RB; i += 4) {
    const int b = i / RB, q = i % RB, t = b * 16 + (lane & 15), r = q * 16 + (lane >> 4) * 4;
    f32x4 s = sums[0][b][q][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) s += sums[w][b][q][lane];
    if (t < tile.z && r < R)
      *reinterpret_cast<f32x4*>(part + ((size_t)mine * T + tile.y + t) * R + r) = s;
  }
}

// ------------------------------------------------------------------ out of the rank
// out[t, n] = base[t, n] + sum over r of f v[t, r] m[e][n, r], v the sum of `parts` rows in
// their order. MFMA rows are n, columns tokens, and the reduction runs over the first
// and then the second parts of f v. Fragments (i, j) of a wave's 64 columns take rows n =
// 32 i + 8 (m / 4) + 4 j + m % 4, so that a lane ends with two runs of 8 columns of a token,
// and four lanes have 64 bytes of a row. Bound by base and out: 8192 x 10240 80 us, 335 MB at
// 4.1 TB/s; a kernel that only copies them in this order takes 70. Of rank 64, 8191 x 5120:
// 61 us (2.7 TB/s), where every tile also reads b, from L2, as many bytes as base.
struct LoraOutArgs {
  const float* part;     // [parts, T, R]
  const uint16_t* m;     // [E, N, R]
  const float* scale;    // [E] or null
  const int32_t* plan;
  const uint16_t* base;  // [T, N] or null
  uint16_t* out;         // [T, N]
  float* v;              // [T, R] or null
  int parts, T, E, R, N, width;
};

template <int RB, int TB, bool BASE>
__device__ __forceinline__ void rank_out(const LoraOutArgs& p, const int4& tile, const int (&tokens)[4],
                                         const int32_t* all_tokens, int n0, uint16_t* vs) {
  constexpr int PITCH = RB * 32 + 8;  // values of a token in LDS: hi, lo, zeros, padding
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, l = lane & 15, g = lane >> 4;
  const int R = p.R, N = p.N, count = tile.z, n1 = min(N, n0 + p.width);
  const uint16_t* m = p.m + (size_t)tile.x * R * N;
  size_t row[TB];
#pragma unroll
  for (int b = 0; b < TB; ++b) row[b] = (size_t)tokens[b] * N;
  // Every load is made, of what is there: columns past the end and tokens past the tile's
  // last one repeat others and are not stored. The next columns' loads go out before the
  // stores, so that waiting for them is not waiting for the stores.
  u32x4 mf[RB][2][2], d[TB][2];
  auto load = [&](int nb) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (BASE)
#pragma unroll
        for (int b = 0; b < TB; ++b) d[b][i] = ld16(p.base + row[b] + min(nb + 32 * i + 8 * g, N - 8));
#pragma unroll
      for (int s = 0; s < RB; ++s) {
        const int kk = s * 32 + g * 8, r = kk < R ? kk : kk - R;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint16_t* from = m + (size_t)min(nb + 32 * i + 8 * (l / 4) + 4 * j + l % 4, N - 1) * R + r;
          mf[s][i][j] = ld16(kk < 2 * R ? (const void*)from : (const void*)kZeros);
        }
      }
    }
  };
  int nb = n0 + wave * 64;
  load(min(nb, N - 8));
  const float f = p.scale ? p.scale[tile.x] : 1.f;
  const int r4 = R / 4;
  each_sum(
      count * r4, p.parts, (size_t)p.T * R,
      [&](int i) { return p.part + (size_t)(tile.y + i / r4) * R + i % r4 * 4; },
      [&](int i, const f32x4& s) {
        const int t = i / r4, r = i % r4 * 4;
        if (p.v && n0 == 0) *reinterpret_cast<f32x4*>(p.v + (size_t)all_tokens[t] * R + r) = s;
        u32x2 hi, lo;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t h0, h1, l0, l1;
          split(s[2 * q] * f, h0, l0);
          split(s[2 * q + 1] * f, h1, l1);
          hi[q] = h0 | h1 << 16;
          lo[q] = l0 | l1 << 16;
        }
        *reinterpret_cast<u32x2*>(vs + t * PITCH + r) = hi;
        *reinterpret_cast<u32x2*>(vs + t * PITCH + R + r) = lo;
      });
  const int rest = RB * 32 - 2 * R;  // of a token's row
  for (int i = tid; i < count * rest; i += 256) vs[i / rest * PITCH + 2 * R + i % rest] = 0;
  __syncthreads();
  for (; nb < n1; nb += 256) {
    u32x4 w[TB][2];
    // products with zeros tell whether an infinity or a NaN is among the adapter's values
    f32x4 zero[2][2] = {};
#pragma unroll
    for (int s = 0; s < RB; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) zero[i][j] = mfma_bf16(as_bf16x8(mf[s][i][j]), as_bf16x8(u32x4{}), zero[i][j]);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) bad |= __builtin_isunordered(zero[i][0][q], zero[i][1][q]);
    if (__builtin_expect(__ballot(bad) != 0, 0))
#pragma unroll
      for (int s = 0; s < RB; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (s * 32 + g * 8 >= R) mf[s][i][j] = finite(mf[s][i][j]);
#pragma unroll
    for (int b = 0; b < TB; ++b) {
      f32x4 acc[2][2] = {};
#pragma unroll
      for (int s = 0; s < RB; ++s) {  // behind the 2 R values of a token its row of vs holds zeros
        const u32x4 vf = ld16(vs + min(b * 16 + l, count - 1) * PITCH + s * 32 + g * 8);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = mfma_bf16(as_bf16x8(mf[s][i][j]), as_bf16x8(vf), acc[i][j]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float lo = acc[i][q / 2][q % 2 * 2], hi = acc[i][q / 2][q % 2 * 2 + 1];
          if constexpr (BASE) {
            lo += __uint_as_float(d[b][i][q] << 16);
            hi += __uint_as_float(d[b][i][q] & 0xffff0000u);
          }
          w[b][i][q] = pack_bf16x2(lo, hi);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (nb + 256 < n1) load(nb + 256);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int n = nb + 32 * i + 8 * g;
        if (b * 16 + l < count && n < N) st16(p.out + row[b] + n, w[b][i]);
      }
  }
}

template <int RB>
__global__ __launch_bounds__(256, RB <= 4 ? 2 : 1) void lora_out_kernel(LoraOutArgs p) {
  __shared__ __attribute__((aligned(16))) uint16_t vs[64 * (RB * 32 + 8)];
  const LoraPlanLayout at(p.T, p.E);
  int number, n0;
  place((p.N + p.width - 1) / p.width, number, n0);
  n0 *= p.width;
  if (number >= at.tiles) return;
  const int4 tile = tile_at(p.plan, at, number);
  int tokens[4];
  tile_tokens(p.plan, at, number, tokens);
  if (number >= p.plan[0]) return;
  const int32_t* all = p.plan + at.o_tokens + (size_t)number * kLoraTile;
  if (tile.x < 0) {  // these keep their base
    if (p.v && n0 == 0)
      for (int i = threadIdx.x; i < tile.z * p.R; i += 256) p.v[(size_t)all[i / p.R] * p.R + i % p.R] = 0.f;
    if (p.base == p.out) return;
    const int chunks = (min(p.N, n0 + p.width) - n0) / 8;
    for (int i = threadIdx.x; i < tile.z * chunks; i += 256) {
      const size_t o = (size_t)all[i / chunks] * p.N + n0 + i % chunks * 8;
      st16(p.out + o, p.base ? ld16(p.base + o) : u32x4{0, 0, 0, 0});
    }
    return;
  }
  auto run = [&](auto tb) {
    constexpr int TB = decltype(tb)::value;
    if (p.base)
      rank_out<RB, TB, true>(p, tile, tokens, all, n0, vs);
    else
      rank_out<RB, TB, false>(p, tile, tokens, all, n0, vs);
  };
  if (tile.z <= 16)
    run(std::integral_constant<int, 1>{});
  else if (tile.z <= 32)
    run(std::integral_constant<int, 2>{});
  else
    run(std::integral_constant<int, 4>{});
}

// ------------------------------------------------------------------ gradients
// a [E, R, K] -> [E, K, R] and b [E, N, R] -> [E, R, N], 64 x 64 blocks through LDS, of
// the adapters that have tokens; zeros in the gradients of the others.
__global__ __launch_bounds__(256) void lora_transpose_kernel(const uint16_t* __restrict__ a,
                                                             const uint16_t* __restrict__ b,
                                                             const int32_t* __restrict__ plan, int T, int E, int R,
                                                             int K, int N, uint16_t* __restrict__ at,
                                                             uint16_t* __restrict__ bt, uint16_t* __restrict__ da,
                                                             uint16_t* __restrict__ db) {
  __shared__ uint16_t tile[64][72];
  const LoraPlanLayout l(T, E);
  const int32_t* chunks = plan + l.o_first + blockIdx.y;
  const bool used = chunks[0] != chunks[1];
  if (!used && !da) return;
  const int rb = (R + 63) / 64, kb = (K + 63) / 64, nb = (N + 63) / 64;
  int i = blockIdx.x;
  const bool of_a = i < rb * kb;
  if (!of_a) i -= rb * kb;
  const int rows = of_a ? R : N, cols = of_a ? K : R, cb = of_a ? kb : rb;
  const uint16_t* src = (of_a ? a : b) + (size_t)blockIdx.y * rows * cols;
  uint16_t* dst = (of_a ? at : bt) + (size_t)blockIdx.y * rows * cols;
  const int r0 = i / cb * 64, c0 = i % cb * 64;
  if (!used) {
    uint16_t* grad = (of_a ? da : db) + (size_t)blockIdx.y * rows * cols;
    for (int q = threadIdx.x; q < 512; q += 256) {
      const int r = r0 + q / 8, c = c0 + q % 8 * 8;
      if (r < rows && c < cols) st16(grad + (size_t)r * cols + c, u32x4{0, 0, 0, 0});
    }
    return;
  }
  for (int q = threadIdx.x; q < 512; q += 256) {
    const int r = r0 + q / 8, c = c0 + q % 8 * 8;
    if (r < rows && c < cols) {
      const u32x4 v = ld16(src + (size_t)r * cols + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        tile[q % 8 * 8 + 2 * e][q / 8] = (uint16_t)v[e];
        tile[q % 8 * 8 + 2 * e + 1][q / 8] = (uint16_t)(v[e] >> 16);
      }
    }
  }
  __syncthreads();
  for (int q = threadIdx.x; q < 512; q += 256) {
    const int c = c0 + q / 8, r = r0 + q % 8 * 8;
    if (c < cols && r < rows) st16(dst + (size_t)c * rows + r, ld16(&tile[q / 8][q % 8 * 8]));
  }
}

// dv = f times the sum of its parts, in the tokens' order, and, for the adapters'
// gradients, dv and f v as operands: two bf16 parts, a row of padded positions for each
// r. A workgroup per tile (positions past its last token: zeros). 8 us at 8191 tokens of rank
// 64, 129 workgroups: latency.
__global__ __launch_bounds__(256) void lora_operands_kernel(const float* part, int parts, const float* v,
                                                            const float* scale, const int32_t* __restrict__ plan,
                                                            int T, int E, int R, float* dv, uint16_t* dvt,
                                                            uint16_t* vt) {
  extern __shared__ uint32_t pairs[];  // [R][66]: hi in the low half, lo
  const LoraPlanLayout at(T, E);
  if ((int)blockIdx.x >= plan[0]) return;
  const int4 tile = tile_at(plan, at, blockIdx.x);
  if (tile.x < 0) return;
  const int count = tile.z, padded = (count + 31) & ~31;
  const float f = scale ? scale[tile.x] : 1.f;
  const int which = blockIdx.y;  // 0: dv, 1: v
  const int r4 = R / 4;
  auto pair = [&](int t, int r, const f32x4& s) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t hi, lo;
      split(s[q], hi, lo);
      pairs[(r + q) * 66 + t] = hi | lo << 16;
    }
  };
  if (which == 0)
    each_sum(
        count * r4, parts, (size_t)T * R, [&](int i) { return part + (size_t)(tile.y + i / r4) * R + i % r4 * 4; },
        [&](int i, const f32x4& s) {
          *reinterpret_cast<f32x4*>(dv + (size_t)(tile.y + i / r4) * R + i % r4 * 4) = s * f;
          pair(i / r4, i % r4 * 4, s * f);
        });
  else
    for (int i = threadIdx.x; i < count * r4; i += 256)
      pair(i / r4, i % r4 * 4,
           f * *reinterpret_cast<const f32x4*>(
                   v + (size_t)plan[at.o_tokens + (size_t)blockIdx.x * kLoraTile + i / r4] * R + i % r4 * 4));
  for (int i = count * R + threadIdx.x; i < padded * R; i += 256) pairs[i % R * 66 + i / R] = 0;
  __syncthreads();
  uint16_t* to = which == 0 ? dvt : vt;
  if (!to) return;
  for (int i = threadIdx.x; i < R * 8; i += 256) {
    const int r = i / 8, t = i % 8 * 8;
    if (t >= padded) continue;
    u32x4 hi, lo;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t x = pairs[r * 66 + t + 2 * q], y = pairs[r * 66 + t + 2 * q + 1];
      hi[q] = (x & 0xffffu) | y << 16;
      lo[q] = x >> 16 | (y & 0xffff0000u);
    }
    uint16_t* row = to + (size_t)r * at.padded + tile.w + t;
    st16(row, hi);
    st16(row + (size_t)R * at.padded, lo);
  }
}

struct LoraGradArgs {
  const uint16_t* op[2];  // operands [2, R, padded]: dv for d_a, f v for d_b
  const uint16_t* rows[2];  // x [T, K], dy [T, N]
  uint16_t* out[2];       // d_a [E, R, K], d_b [E, N, R]
  float* part[2];         // [slots, R, C]
  const int32_t* plan;
  int T, E, R, C[2];
};

// sum over a chunk's tokens of op[t, r] rows[t, c] for 16 RB values of r and 128 columns:
// the four waves take 32 tokens in turn, and their sums are added through LDS. MFMA rows
// are r, columns c, the reduction runs over 32 tokens. Lane (l, g) loads columns 8 l .. + 7
// of tokens 8 g .. + 7, whole 256-byte runs of a row, and turns them in its registers into
// fragment j of column 8 l + j, whose reduction values are its 8 tokens. Rank 64, 8191 tokens,
// 5120 + 5120 columns: 57 us. The rows (168 MB) come twice, for two blocks of 32 ranks (one block
// of 64 spilled registers); the second time from the XCD's L2 (70% of its reads hit).
template <int RB>
__global__ __launch_bounds__(256, 2) void lora_grad_kernel(LoraGradArgs p) {
  __shared__ __attribute__((aligned(16))) int32_t tokens[512];
  __shared__ f32x4 sums[2][RB][8][64];
  const LoraPlanLayout at(p.T, p.E);
  const int wgs0 = (p.C[0] + 127) / 128;
  int number, block;
  const int ranks = (p.R + RB * 16 - 1) / (RB * 16);
  place((wgs0 + (p.C[1] + 127) / 128) * ranks, number, block);
  const int r0 = block % ranks * (RB * 16);
  block /= ranks;
  const int which = block >= wgs0;
  if (number >= at.chunks || number >= p.plan[1]) return;
  const int4 chunk = chunk_at(p.plan, at, number);
  const int C = which ? p.C[1] : p.C[0], R = p.R;
  const uint16_t* rows = which ? p.rows[1] : p.rows[0];
  const uint16_t* op = which ? p.op[1] : p.op[0];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int c0 = (block - (which ? wgs0 : 0)) * 128 + l * 8, c = min(c0, C - 8);
  const size_t lo = (size_t)R * at.padded;
  const uint16_t* ops[RB];
#pragma unroll
  for (int q = 0; q < RB; ++q)
    ops[q] = op + (size_t)min(r0 + q * 16 + l, R - 1) * at.padded + chunk.w + g * 8;
  auto turn = [](const u32x4 (&x)[8], u32x4 (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[j][i] = __builtin_amdgcn_perm(x[2 * i + 1][j / 2], x[2 * i][j / 2], j % 2 ? 0x07060302u : 0x05040100u);
  };
  f32x4 acc[RB][8] = {};
  for (int p0 = 0; p0 < chunk.z; p0 += 512) {
    __syncthreads();
    for (int i = threadIdx.x; i < 512; i += 256)
      tokens[i] = p.plan[at.o_order + chunk.y + min(p0 + i, chunk.z - 1)];
    __syncthreads();
    const int n = min(512, chunk.z - p0);
    // the next rows are loaded while these are multiplied, the next operands behind the
    // last product that reads these
    u32x4 x[8], a[RB][2];
    auto load_x = [&](int s) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = ld16(rows + (size_t)tokens[s + g * 8 + i] * C + c);
    };
    auto load_a = [&](int s) {
#pragma unroll
      for (int q = 0; q < RB; ++q) {
        a[q][0] = ld16(ops[q] + p0 + s);
        a[q][1] = ld16(ops[q] + lo + p0 + s);
      }
    };
    if (wave * 32 < n) {
      load_x(wave * 32);
      load_a(wave * 32);
    }
    for (int s = wave * 32; s < n; s += 128) {
      if (s + 32 > n) {  // tokens past the chunk's last one: zeros on both sides
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (s + g * 8 + i >= n) x[i] = u32x4{0, 0, 0, 0};
      }
      u32x4 f[8];
      turn(x, f);
      __builtin_amdgcn_sched_barrier(0);
      if (s + 128 < n) load_x(s + 128);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int q = 0; q < RB; ++q) {
          acc[q][j] = mfma_bf16(as_bf16x8(a[q][0]), as_bf16x8(f[j]), acc[q][j]);
          acc[q][j] = mfma_bf16(as_bf16x8(a[q][1]), as_bf16x8(f[j]), acc[q][j]);
        }
      __builtin_amdgcn_sched_barrier(0);
      if (s + 128 < n) load_a(s + 128);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  bool nan = false;
#pragma unroll
  for (int q = 0; q < RB; ++q)
#pragma unroll
    for (int j = 0; j < 8; j += 2)
#pragma unroll
      for (int i = 0; i < 4; ++i) nan |= __builtin_isunordered(acc[q][j][i], acc[q][j + 1][i]);
  if (__builtin_expect(__ballot(nan) != 0, 0)) {
    // this wave's sum again, a step after the other, by a lane that no loop knows: the pass
    // above holds nothing for it in registers
    int lane = threadIdx.x & 63;
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+v"(lane));
#endif
    const int l = lane & 15, g = lane >> 4;
    const uint16_t* from = rows + min((block - (which ? wgs0 : 0)) * 128 + l * 8, C - 8);
#pragma unroll
    for (int q = 0; q < RB; ++q)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[q][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int s = wave * 32; s < chunk.z; s += 128) {
      u32x4 x[8], f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = s + g * 8 + i;
        const int token = p.plan[at.o_order + chunk.y + min(t, chunk.z - 1)];
        x[i] = t < chunk.z ? ld16(from + (size_t)token * C) : u32x4{0, 0, 0, 0};
      }
      turn(x, f);
#pragma unroll
      for (int q = 0; q < RB; ++q) {
        const uint16_t* o = op + (size_t)min(r0 + q * 16 + l, R - 1) * at.padded + chunk.w + g * 8 + s;
        const u32x4 first = ld16(o), second = ld16(o + lo);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc[q][j] = mfma_bf16(as_bf16x8(first), as_bf16x8(f[j]), acc[q][j]);
          acc[q][j] = mfma_bf16(as_bf16x8(second), as_bf16x8(finite(f[j])), acc[q][j]);
        }
      }
    }
  }
  // waves 2 and 3 onto 0 and 1, then 1 onto 0
#pragma unroll
  for (int half = 2; half >= 1; half /= 2) {
    __syncthreads();
    if (wave >= half && wave < 2 * half)
#pragma unroll
      for (int q = 0; q < RB; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[wave - half][q][j][lane] = acc[q][j];
    __syncthreads();
    if (wave < half)
#pragma unroll
      for (int q = 0; q < RB; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[q][j] += sums[wave][q][j][lane];
  }
  if (wave > 0) return;
  if (c0 >= C) return;
  const int slot = p.plan[at.o_slot + chunk.x];
#pragma unroll
  for (int q = 0; q < RB; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + q * 16 + g * 4 + i;
      if (r >= R) continue;
      if (slot >= 0) {  // one of several chunks: added by lora_grad_sum_kernel
        float* to = (which ? p.part[1] : p.part[0]) +
                    ((size_t)(slot + number - p.plan[at.o_first + chunk.x]) * R + r) * C + c0;
        *reinterpret_cast<f32x4*>(to) = f32x4{acc[q][0][i], acc[q][1][i], acc[q][2][i], acc[q][3][i]};
        *reinterpret_cast<f32x4*>(to + 4) = f32x4{acc[q][4][i], acc[q][5][i], acc[q][6][i], acc[q][7][i]};
      } else if (!which) {
        st16(p.out[0] + ((size_t)chunk.x * R + r) * C + c0,
             u32x4{pack_bf16x2(acc[q][0][i], acc[q][1][i]), pack_bf16x2(acc[q][2][i], acc[q][3][i]),
                   pack_bf16x2(acc[q][4][i], acc[q][5][i]), pack_bf16x2(acc[q][6][i], acc[q][7][i])});
      }
    }
  if (slot < 0 && which) {  // [N, R]: 4 consecutive values of r of a column
#pragma unroll
    for (int q = 0; q < RB; ++q)
      if (r0 + q * 16 + g * 4 < R)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<u32x2*>(p.out[1] + ((size_t)chunk.x * C + c0 + j) * R + r0 + q * 16 + g * 4) =
              u32x2{pack_bf16x2(acc[q][j][0], acc[q][j][1]), pack_bf16x2(acc[q][j][2], acc[q][j][3])};
  }
}

// The sums of adapters with several chunks, in their order: 8 values a thread. 6 to 8 us for 21 MB (8 chunks of rank 64, 5120 + 5120 columns).
__global__ __launch_bounds__(256) void lora_grad_sum_kernel(LoraGradArgs p) {
  const LoraPlanLayout at(p.T, p.E);
  const int e = blockIdx.y;
  const int first = p.plan[at.o_first + e], n = p.plan[at.o_first + e + 1] - first;
  if (n <= 1) return;
  const int slot = p.plan[at.o_slot + e], R = p.R;
  int i = blockIdx.x * 256 + threadIdx.x;
  const int n0 = R * (p.C[0] / 8), n1 = (R / 8) * p.C[1];
  if (i >= n0 + n1) return;
  const bool which = i >= n0;
  if (which) i -= n0;
  const int C = which ? p.C[1] : p.C[0];
  float s[8] = {};
  for (int j = 0; j < n; ++j) {
    const float* from = (which ? p.part[1] : p.part[0]) + (size_t)(slot + j) * R * C;
    if (which) {  // column i % C, rows 8 (i / C) ..
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] += from[(size_t)(i / C * 8 + q) * C + i % C];
    } else {
      const f32x4 a = *reinterpret_cast<const f32x4*>(from + (size_t)i * 8),
                  b = *reinterpret_cast<const f32x4*>(from + (size_t)i * 8 + 4);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        s[q] += a[q];
        s[4 + q] += b[q];
      }
    }
  }
  uint16_t* to = which ? p.out[1] + ((size_t)e * C + i % C) * R + i / C * 8 : p.out[0] + (size_t)e * R * C + (size_t)i * 8;
  st16(to, u32x4{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]), pack_bf16x2(s[4], s[5]), pack_bf16x2(s[6], s[7])});
}

// Parts of a reduction over k: a power of two (5 parts of 8192 x 5120 took 25 us, 4 took
// 22), as long as the chip holds all workgroups at once and every wave has 128 values of k.
int parts_of(int tiles, int K) {
  int p = 1;
  while (2 * p <= kMaxParts && 2 * p * tiles <= 700 && 2 * p * 512 <= K + 511) p *= 2;
  return p;
}

template <typename F>
void with_rank(int R, F f) {
  if (R <= 16)
    f(std::integral_constant<int, 1>{});
  else if (R <= 32)
    f(std::integral_constant<int, 2>{});
  else if (R <= 64)
    f(std::integral_constant<int, 4>{});
  else
    f(std::integral_constant<int, 8>{});
}

void into_rank(const uint16_t* x, const uint16_t* m, const int32_t* plan, int T, int E, int R, int K, float* part,
               hipStream_t st) {
  const int tiles = LoraPlanLayout(T, E).tiles;
  with_rank(R, [&](auto rb) {
    const int parts = parts_of(tiles, K);
    lora_in_kernel<decltype(rb)::value><<<grid_of(tiles, parts), 256, 0, st>>>(x, m, plan, parts, T, E, R, K, part);
  });
}

void out_of_rank(LoraOutArgs a, hipStream_t st) {
  const int tiles = LoraPlanLayout(a.T, a.E).tiles;
  // columns of a workgroup: the more, the less often the tile's parts are added
  a.width = 256;
  while (a.width < 1024 && tiles * ((a.N + 2 * a.width - 1) / (2 * a.width)) >= 1100) a.width *= 2;
  with_rank(a.R, [&](auto rb) {
    lora_out_kernel<decltype(rb)::value><<<grid_of(tiles, (a.N + a.width - 1) / a.width), 256, 0, st>>>(a);
  });
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Workspace of the backward pass
struct LoraBwdSpace {
  size_t at, bt, part, dv, dvt, vt, part_a, part_b, bytes;
  LoraBwdSpace(int T, int K, int N, int R, int E) {
    const LoraPlanLayout l(T, E);
    size_t o = 0;
    auto take = [&](size_t n) {
      const size_t was = o;
      o += up256(n);
      return was;
    };
    at = take((size_t)E * R * K * 2);
    bt = take((size_t)E * R * N * 2);
    part = take((size_t)parts_of(l.tiles, N) * T * R * 4);
    dv = take((size_t)T * R * 4);
    dvt = take((size_t)l.padded * R * 4);
    vt = take((size_t)l.padded * R * 4);
    part_a = take((size_t)l.slots * R * K * 4);
    part_b = take((size_t)l.slots * R * N * 4);
    bytes = o;
  }
};

}  // namespace

hipError_t launch_lora_plan(const int32_t* index, int T, int E, int32_t* plan, hipStream_t st) {
  lora_plan_kernel<<<1, 64 * kPlanWaves, 0, st>>>(index, T, E, plan);
  return hipGetLastError();
}

size_t lora_workspace_bytes(int T, int K, int N, int R, int E) {
  return (size_t)parts_of(LoraPlanLayout(T, E).tiles, K) * T * R * sizeof(float);
}

hipError_t launch_lora(const LoraArgs& p, hipStream_t st) {
  into_rank(p.x, p.a, p.plan, p.T, p.E, p.R, p.K, p.part, st);
  out_of_rank({p.part, p.b, p.scale, p.plan, p.base, p.out, p.v, parts_of(LoraPlanLayout(p.T, p.E).tiles, p.K), p.T, p.E,
               p.R, p.N, 0},
              st);
  return hipGetLastError();
}

size_t lora_bwd_workspace_bytes(int T, int K, int N, int R, int E) { return LoraBwdSpace(T, K, N, R, E).bytes; }

hipError_t launch_lora_backward(const LoraBwdArgs& p, hipStream_t st) {
  const LoraPlanLayout l(p.T, p.E);
  const LoraBwdSpace w(p.T, p.K, p.N, p.R, p.E);
  uint8_t* ws = (uint8_t*)p.workspace;
  uint16_t *at = (uint16_t*)(ws + w.at), *bt = (uint16_t*)(ws + w.bt);
  float *part = (float*)(ws + w.part), *dv = (float*)(ws + w.dv);
  uint16_t *dvt = (uint16_t*)(ws + w.dvt), *vt = (uint16_t*)(ws + w.vt);
  const int blocks = (p.R + 63) / 64 * ((p.K + 63) / 64 + (p.N + 63) / 64);
  lora_transpose_kernel<<<dim3(blocks, p.E), 256, 0, st>>>(p.a, p.b, p.plan, p.T, p.E, p.R, p.K, p.N, at, bt, p.da,
                                                               p.db);
  into_rank(p.dy, bt, p.plan, p.T, p.E, p.R, p.N, part, st);
  lora_operands_kernel<<<dim3(l.tiles, p.da ? 2 : 1), 256, p.R * 66 * 4, st>>>(
      part, parts_of(l.tiles, p.N), p.v, p.scale, p.plan, p.T, p.E, p.R, dv, p.da ? dvt : nullptr, vt);
  if (p.da) {
    const LoraGradArgs a{{dvt, vt}, {p.x, p.dy}, {p.da, p.db},
                         {(float*)(ws + w.part_a), (float*)(ws + w.part_b)}, p.plan, p.T, p.E, p.R, {p.K, p.N}};
    const int wgs = (p.K + 127) / 128 + (p.N + 127) / 128;
    if (p.R <= 16)
      lora_grad_kernel<1><<<grid_of(l.chunks, wgs), 256, 0, st>>>(a);
    else
      lora_grad_kernel<2><<<grid_of(l.chunks, wgs * ((p.R + 31) / 32)), 256, 0, st>>>(a);
    if (l.slots > 0)
      lora_grad_sum_kernel<<<dim3((p.R * (p.K + p.N) / 8 + 255) / 256, p.E), 256, 0, st>>>(a);
  }
  // last: dx may be the memory of dy or x
  if (p.dx) out_of_rank({dv, at, nullptr, p.plan, p.base, p.dx, nullptr, 1, p.T, p.E, p.R, p.K, 0}, st);
  return hipGetLastError();
}

}  // namespace beam
