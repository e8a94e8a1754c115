// Routing of given logits and its gradient: scores (sigmoid or softmax), a
// selection bias, groups of experts, top-k, normalised weights.
//
// Beam launch post ("Introducing Beam"), section "Mixture of Experts":
// sigmoid scores, 8 groups of 32 experts, the 4 groups with the best sum of
// their two top scores, top 8, normalised weights; transformers model doc
// "Beam", section "Overview": the bias shifts the selection key only.
//
// One wave per token; lane l holds the experts KPL l .. KPL l + KPL - 1.
// Scores and keys are fp64: which of two experts a token goes to is decided
// by the values themselves, not by an fp32 rounding of them. 37 tokens x 160 experts
// 6.2 us, bound by top_k rounds of a maximum over the wave, each waiting for the last.
#include "common.h"
#include "operators.h"
#include "wave.h"

namespace beam {
namespace {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_bits_to_f32(v); }

// Keeps the two largest of (t1 >= t2) and v.
__device__ __forceinline__ void top2_add(double& t1, double& t2, double v) {
  t2 = fmax(t2, fmin(t1, v));
  t1 = fmax(t1, v);
}

template <typename T, int KPL>
__device__ __forceinline__ void load_logits(const T* z, int lane, int E, float (&v)[KPL]) {
  // whole vectors where every row starts on one
  if (KPL * sizeof(T) >= 4 && KPL * sizeof(T) <= 16 && E % KPL == 0) {
    struct alignas(KPL * sizeof(T)) Vec {
      T e[KPL];
    };
    Vec q;
    if (lane * KPL < E) q = *reinterpret_cast<const Vec*>(z + lane * KPL);
#pragma unroll
    for (int i = 0; i < KPL; ++i) v[i] = lane * KPL < E ? to_f32(q.e[i]) : -INFINITY;
  } else {
#pragma unroll
    for (int i = 0; i < KPL; ++i) v[i] = lane * KPL + i < E ? to_f32(z[lane * KPL + i]) : -INFINITY;
  }
}

// Tokens per expert from the chosen indices. A workgroup counts its share in LDS;
// alone, it writes the counts, else it adds them to zeroed ones (whole numbers:
// any order gives the same). Adding every slot to memory from the routing itself
// took 100 us at 16384 tokens x 8, all on 256 addresses; this takes 6.
constexpr int kCountShare = 16384;  // slots of a workgroup

// The routing's first workgroup zeroes them.
__device__ __forceinline__ void zero_counts(const GateArgs& p) {
  if (p.counts && blockIdx.x == 0)
    for (int e = threadIdx.x; e < p.E; e += 256) p.counts[e] = 0;
}

__global__ __launch_bounds__(1024) void gate_count_kernel(const int32_t* __restrict__ idx, int64_t n,
                                                          int E, int32_t* __restrict__ counts) {
  __shared__ int32_t hist[kGateMaxE];
  for (int e = threadIdx.x; e < E; e += 1024) hist[e] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * kCountShare, i1 = min(n, i0 + kCountShare);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += 1024) {
    const int e = idx[i];
    if (e >= 0) atomicAdd(hist + e, 1);  // padding has -1
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 1024) {
    if (gridDim.x == 1)
      counts[e] = hist[e];
    else if (hist[e])
      atomicAdd(counts + e, hist[e]);
  }
}

// One token by a whole wave, lane l with the experts KPL l .. KPL l + KPL - 1 and
// every key in fp64. lds_keys: E doubles of the wave's own.
template <typename T, int KPL>
__device__ __forceinline__ void gate_token(const GateArgs& p, int t, double* lds_keys) {
  const int lane = threadIdx.x & 63;
  const int E = p.E, k = p.k;
  float z[KPL];
  load_logits<T, KPL>((const T*)p.z + (size_t)t * E, lane, E, z);

  // score f; a logit of -inf or NaN is a masked expert: score 0, key -inf
  double f[KPL], key[KPL];
  bool off[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) off[i] = !(z[i] > -INFINITY);
  if (p.softmax) {
    double m = -INFINITY, sum = 0;
#pragma unroll
    for (int i = 0; i < KPL; ++i) m = off[i] ? m : fmax(m, (double)z[i]);
    m = wave_max(m);
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      // equal logits share the mass, +inf ones too
      f[i] = off[i] ? 0.0 : (double)z[i] == m ? 1.0 : exp((double)z[i] - m);
      sum += f[i];
    }
    sum = wave_sum(sum);
    const double inv = sum > 0 ? 1.0 / sum : 0.0;
#pragma unroll
    for (int i = 0; i < KPL; ++i) f[i] *= inv;
  } else {
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const double e = exp(-fabs((double)z[i]));
      f[i] = off[i] ? 0.0 : (z[i] >= 0.f ? 1.0 : e) / (1.0 + e);
    }
  }
  uint32_t avail = 0;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int e = lane * KPL + i;
    key[i] = f[i];
    if (p.bias && e < E) key[i] += (double)p.bias[e];
    if (off[i] || !(key[i] > -INFINITY)) key[i] = -INFINITY;
    if (e < E) avail |= 1u << i;
  }

  if (p.n_group > 1) {
    const int gs = E / p.n_group;
    const int lpg = gs / KPL;
    const bool by_lane = gs % KPL == 0 && (lpg & (lpg - 1)) == 0;
    double t1 = -INFINITY, t2 = -INFINITY;
    int stride, mine;  // lane gg * stride speaks for group gg; this lane's group
    if (by_lane) {
#pragma unroll
      for (int i = 0; i < KPL; ++i) top2_add(t1, t2, key[i]);
      for (int o = 1; o < lpg; o <<= 1) {
        const double o1 = __shfl_xor(t1, o), o2 = __shfl_xor(t2, o);
        t2 = fmax(fmin(t1, o1), fmax(t2, o2));
        t1 = fmax(t1, o1);
      }
      stride = lpg;
      mine = lane / lpg;
    } else {
      double* keys = lds_keys;
#pragma unroll
      for (int i = 0; i < KPL; ++i)
        if (lane * KPL + i < E) keys[lane * KPL + i] = key[i];
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      if (lane < p.n_group)
        for (int i = 0; i < gs; ++i) top2_add(t1, t2, keys[lane * gs + i]);
      stride = 1;
      mine = lane;
    }
    // a group of one expert has no second: its score is that expert's key
    double score = p.top2 && gs > 1 ? t1 + t2 : t1;
    if (!(score == score)) score = -INFINITY;
    int rank = 0;
    for (int g = 0; g < p.n_group; ++g) {
      const double o = lane_value(score, g * stride);
      rank += (o > score || (o == score && g < mine)) ? 1 : 0;
    }
    const uint64_t kept = __ballot(rank < p.topk_group);
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int e = lane * KPL + i;
      if (e < E && !((kept >> (e / gs * stride)) & 1)) avail &= ~(1u << i);
    }
  }

  double sum = 0, my_f = 0;
  int my_e = 0;
  for (int j = 0; j < k; ++j) {
    double best = -INFINITY;
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if ((avail >> i) & 1) best = fmax(best, key[i]);
    const double m = wave_max(best);
    // the lowest lane, then its lowest slot, that holds the maximum: the
    // lowest expert. At least k experts are available, so there is one.
    const uint64_t hold = __ballot(avail != 0 && best == m);
    const int owner = __ffsll((unsigned long long)hold) - 1;
    int slot = 0;
    double fv = 0;
#pragma unroll
    for (int i = KPL - 1; i >= 0; --i)
      if (((avail >> i) & 1) && key[i] == m) {
        slot = i;
        fv = f[i];
      }
    slot = __builtin_amdgcn_readlane(slot, owner);
    fv = lane_value(fv, owner);
    if (lane == owner) avail &= ~(1u << slot);
    sum += fv;
    if (lane == j) {
      my_e = owner * KPL + slot;
      my_f = fv;
    }
  }
  if (lane < k) {
    const double w = p.renorm ? (sum > 0 ? my_f / sum : 0.0) : my_f;
    p.idx[(size_t)t * k + lane] = my_e;
    p.w[(size_t)t * k + lane] = (float)((double)p.rsf * w);
  }
}

template <typename T, int KPL>
__global__ __launch_bounds__(256) void gate_kernel(GateArgs p) {
  extern __shared__ double lds_keys[];  // [4][E] with groups
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + wave;
  zero_counts(p);
  if (t >= p.T) return;  // no barrier below: a wave works alone
  if (p.valid && !p.valid[t]) {
    if (lane < p.k) {
      p.idx[(size_t)t * p.k + lane] = -1;
      p.w[(size_t)t * p.k + lane] = 0.f;
    }
    return;
  }
  gate_token<T, KPL>(p, t, lds_keys + (size_t)wave * p.E);
}

// ------------------------------------------------------------------ four tokens a wave
// Up to 512 experts in 1, 2, 4, 8 or 16 groups and top_k <= 16: 16 lanes per
// token, a group on whole lanes, at most KPL experts a lane. The order is decided
// on 32-bit keys: the score with its bias, or without a bias the logit itself
// (the score grows with it), in fp32, its 24 leading bits (23 with more than 16
// experts a lane) in the order of unsigned integers, with 255 (511) - expert below
// them. So a maximum is one integer maximum, it says which expert it is, and ties
// go to the lower index. Where two neighbours of
// the first top_k + 1 keys, or the last kept group and the first dropped one, lie
// so near each other that the fp64 keys might stand the other way, the token is
// done over in fp64 by the whole wave (about 1% of tokens with random logits).
// With bf16 logits and no bias the 24 bits are the logit, and equal ones are ties. Of
// these, logits below 2^-20 other than 0 may share one fp64 score with any number of
// others, 0 among them: where one is chosen, or may be hidden behind a 0 that is the
// first not to be chosen, the token is done over too. Larger logits are 2^-29 apart or
// more, which their scores show. (Looking for such logits in every token took bf16
// softmax routing of 16384 x 256 from 8.7 to 12.6 us; so it takes 9.1.)
// Weights are fp64 from the chosen logits in either case. 16384 tokens x 256
// experts, 8 groups, top 8: 8 rounds of the fp64 maximum over a wave per token
// took 33 us.
// Up to here a wave per token is faster: a wave of four tokens has four times as
// much to do before the first is done (16384 x 256, us, wave per token and this:
// 64 tokens 6.3 and 7.0, 4096 11.1 and 11.9, 8192 18.5 and 15.7, 16384 33 and 16;
// 5000 x 512 17.3 and 16.4, 16384 x 512 51 and 28), with random logits. Where every
// token is near, sigmoids of 16 and more without a bias or fp32 logits that are all
// equal, 16384 x 256 takes 46 us: each wave does its four tokens over in turn.
constexpr int kWaveTokens = 4096;
__device__ __forceinline__ uint32_t key_bits(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k);
}

// A lane's cnt of at most c values at q, `fill` behind them; `whole`: cnt is c or 0
// for every lane, and q a multiple of c values from an aligned row.
template <int KPL, typename T>
__device__ __forceinline__ void load_share(const T* q, int c, int cnt, bool whole, float fill,
                                           float (&v)[KPL]) {
  constexpr int VE = 16 / sizeof(T);
  if (KPL % VE == 0 && whole && c % VE == 0) {  // 16 bytes at a time
#pragma unroll
    for (int i = 0; i < KPL; i += VE) {
      T w[VE];
      if (i < cnt) __builtin_memcpy(w, __builtin_assume_aligned(q + i, 16), 16);
#pragma unroll
      for (int j = 0; j < VE; ++j)
        if (i + j < KPL) v[i + j] = i < cnt ? to_f32(w[j]) : fill;
    }
  } else {
#pragma unroll
    for (int i = 0; i < KPL; ++i) v[i] = i < cnt ? to_f32(q[i]) : fill;
  }
}

template <typename T, int KPL>
__global__ __launch_bounds__(256) void gate_rows_kernel(GateArgs p) {
  constexpr uint32_t kLow = 16 * KPL > 256 ? 511 : 255;  // the expert's bits of a key
  constexpr uint32_t kMasked = kLow + 1;  // leading bits of a masked expert; a free slot is 0
  extern __shared__ double lds_keys[];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, l = lane & 15;
  zero_counts(p);
  const int E = p.E, k = p.k, G = p.n_group;
  const int t0 = (blockIdx.x * 4 + wave) * 4, t = t0 + (lane >> 4);
  const bool live = t < p.T && !(p.valid && !p.valid[t]);
  const T* zr = (const T*)p.z + (size_t)min(t, p.T - 1) * E;

  // this lane's experts: c of its group's gs
  const int gs = E / G, lpg = 16 / G, c = (gs + lpg - 1) / lpg;
  const int grp = l / lpg, at = (l % lpg) * c;
  const int e0 = grp * gs + at, cnt = min(c, max(0, gs - at));
  float z[KPL];
  load_share<KPL>(zr + e0, c, cnt, gs % c == 0, -INFINITY, z);

  float m = -INFINITY;
  if (p.softmax) {
#pragma unroll
    for (int i = 0; i < KPL; ++i) m = fmaxf(m, z[i]);
    m = row_reduce(m, [](float a, float b) { return fmaxf(a, b); });
  }
  // scores in fp32, where they are compared: with a bias, or summed for groups
  const bool scored = p.bias || (G > 1 && p.top2);
  float v[KPL];
  if (scored) {
    float inv = 1.f;
    if (p.softmax) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        v[i] = z[i] > -INFINITY ? __expf(z[i] - m) : 0.f;
        sum += v[i];
      }
      sum = row_reduce(sum, [](float a, float b) { return a + b; });
      inv = 1.f / sum;
    }
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      if (p.softmax) {
        v[i] *= inv;
      } else {
        const float e = __expf(-fabsf(z[i]));
        v[i] = (z[i] >= 0.f ? 1.f : e) * __builtin_amdgcn_rcpf(1.f + e);
      }
    }
    if (p.bias) {
      float b[KPL];
      load_share<KPL>(p.bias + e0, c, cnt, gs % c == 0, 0.f, b);
#pragma unroll
      for (int i = 0; i < KPL; ++i) v[i] += b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < KPL; ++i) v[i] = z[i];
  }
  // Logits stand for their scores, but not where fp64 scores saturate or vanish.
  auto saturated = [&](float lower) {
    return p.softmax ? !(m - lower < 600.f) : !(lower < 16.f && lower > -600.f);
  };
  const bool exact = sizeof(T) == 2 && !p.bias;
  bool near = false;
  uint32_t key[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const bool off = !(z[i] > -INFINITY) || !(v[i] > -INFINITY);
    if (off) v[i] = -INFINITY;
    const uint32_t low = kLow - (uint32_t)(e0 + i);
    const float order = p.bias ? v[i] : z[i];
    key[i] = i >= cnt ? 0u : (off ? kMasked : key_bits(order) & ~kLow) | low;
  }

  if (G > 1 && p.topk_group < G) {
    float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      t2 = fmaxf(t2, fminf(t1, v[i]));
      t1 = fmaxf(t1, v[i]);
    }
    auto merge = [&](float o1, float o2) {
      t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
      t1 = fmaxf(t1, o1);
    };
    if (lpg > 1) merge(dpp_move<0xB1>(t1, t1), dpp_move<0xB1>(t2, t2));
    if (lpg > 2) merge(dpp_move<0x4E>(t1, t1), dpp_move<0x4E>(t2, t2));
    if (lpg > 4) merge(dpp_move<0x141>(t1, t1), dpp_move<0x141>(t2, t2));
    float score = p.top2 && gs > 1 ? t1 + t2 : t1;
    if (!(score == score)) score = -INFINITY;  // +inf by its bias and a masked second
    int rank = 0;
    for (int g = 0; g < G; ++g) {
      const float o = __shfl(score, (lane & 48) + g * lpg);
      rank += (o > score || (o == score && g < grp)) ? 1 : 0;
    }
    const bool kept = rank < p.topk_group;
    const float lo = row_reduce(kept ? score : INFINITY, [](float a, float b) { return fminf(a, b); });
    const float hi = row_reduce(kept ? -INFINITY : score, [](float a, float b) { return fmaxf(a, b); });
    if (!scored) {
      near |= !(lo - hi > 0x1p-28f) || saturated(hi);
    } else {
      // a score is within 2^-21, and relative to itself within 2^-16 down to 1e-30
      // (its exponential's argument is rounded)
      near |= !(lo - hi > (p.bias ? 0x1p-18f * (fabsf(lo) + fabsf(hi) + 1.f) : 0x1p-15f * (lo + hi)));
      near |= !p.bias && !(lo > 1e-30f);
    }
    if (!kept) {
#pragma unroll
      for (int i = 0; i < KPL; ++i) key[i] = 0u;
    }
  }

  // the k largest keys, lane j of the row keeps the j-th; `next`: the one after
  uint32_t mine = 0, next = 0;
  for (int j = 0; j <= k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < KPL; ++i) best = max(best, key[i]);
    best = row_reduce(best, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
    if (l == j) mine = best;
    if (j == k) next = best;
#pragma unroll
    for (int i = 0; i < KPL; ++i) key[i] = key[i] == best ? 0u : key[i];
  }
  uint32_t after = __shfl(mine, lane + 1);
  if (l == k - 1) after = next;
  int e = (int)(kLow - (mine & kLow));
  const float zc = l < k && live ? to_f32(zr[e]) : -INFINITY;
  bool close = false;    // to the one after
  bool behind0 = false;  // the first key that is not chosen is 0, with others behind it
  if (l < k && after >= 2 * kMasked) {  // neither is masked
    const float lo = key_value(mine & ~kLow), hi = key_value(exact ? after & ~kLow : after | kLow);
    // with a bias both keys are within 2^-20, and their sums' rounding; logits are
    // exact, but fp64 scores of logits this near could be equal
    const float tol = p.bias ? 0x1p-18f + 0x1p-21f * (fabsf(lo) + fabsf(hi)) : 0x1p-28f;
    close = !(lo - hi > tol || (exact && lo == hi));
    if (!p.bias) near |= saturated(hi);
    // (-0, whose key lies below that of 0, shows as a tiny value too)
    auto tiny = [](float x) { return x != 0.f && fabsf(x) < 0x1p-20f; };
    if (exact) near |= tiny(lo) || tiny(hi);
    behind0 = exact && l == k - 1 && hi == 0.f;
  }
  const uint64_t zeros = __ballot(behind0);
  if ((zeros >> (lane & 48)) & 0xffff) {
#pragma unroll
    for (int i = 0; i < KPL; ++i) near |= z[i] <= 0.f && z[i] > -0x1p-20f && __float_as_uint(z[i]) != 0u;
  }

  double f = 0;
  const bool on = zc > -INFINITY;
  if (p.softmax) {
    // renormalised weights are the softmax over the chosen alone
    if (on) f = zc == m ? 1.0 : exp((double)zc - (double)m);
    if (!p.renorm) {
      double sum = 0;
#pragma unroll
      for (int i = 0; i < KPL; ++i)
        if (i < c) sum += z[i] > -INFINITY ? exp((double)z[i] - (double)m) : 0.0;
      sum = row_reduce(sum, [](double a, double b) { return a + b; });
      if (sum > 0) f /= sum;
    }
    if (!(m < INFINITY)) near = true;
  } else if (on) {
    const double x = exp(-fabs((double)zc));
    f = (zc >= 0.f ? 1.0 : x) / (1.0 + x);
  }
  // Two of the chosen that are close, apart from the others: their fp64 scores say
  // which comes first. (Softmax scores with a bias have no fp64 form here.)
  if (__any(close)) {
    // (lane exchanges outside of any condition: every lane has to take part)
    const int cb = __shfl((int)close, lane - 1), ca = __shfl((int)close, lane + 1);
    const bool before = cb && l > 0, behind = ca && l < 15;
    const bool pair = close && l < k - 1 && !before && !behind && !(p.softmax && p.bias);
    near |= close && !pair;
    const int pb = __shfl((int)pair, lane - 1);
    const bool second = pb && l > 0;
    double key64 = f;
    if (p.bias && l < k) key64 += (double)p.bias[e];
    const int other = pair ? lane + 1 : second ? lane - 1 : lane;
    const double okey = __shfl(key64, other), of = __shfl(f, other);
    const int oe = __shfl(e, other);
    const bool wins = key64 > okey || (key64 == okey && e < oe);  // comes before the other
    if ((pair && !wins) || (second && wins)) {
      e = oe;
      f = of;
    }
  }
  if (p.renorm) {
    const double sum = row_reduce(f, [](double a, double b) { return a + b; });
    f = sum > 0 ? f / sum : 0.0;
    if (p.softmax && m > -INFINITY && !(sum > 0)) near = true;  // all chosen far below the maximum
  }
  if (l < k && t < p.T) {
    p.idx[(size_t)t * k + l] = live ? e : -1;
    p.w[(size_t)t * k + l] = live ? (float)((double)p.rsf * f) : 0.f;
  }
  // tokens to do over, one after the other
  uint64_t again = __ballot(near && live);
  while (again) {
    const int row = (__ffsll((unsigned long long)again) - 1) >> 4;
    gate_token<T, (KPL + 3) / 4>(p, t0 + row, lds_keys + (size_t)wave * E);
    again &= ~(0xffffull << (16 * row));
  }
}

// ------------------------------------------------------------------ backward
// With the chosen scores f_j, S their sum, and the gradient dw of the weights:
//   renormalised:     df_j = rsf / S (dw_j - sum_i dw_i f_i / S)
//   as they are:      df_j = rsf dw_j
//   sigmoid:          dz_j = df_j f_j (1 - f_j), 0 for the others
//   softmax:          dz_e = f_e (df_e - sum_j df_j f_j)
// Renormalised softmax weights are the softmax over the chosen logits alone:
// their inner sum is 0, nothing flows to the others, and neither the other
// logits nor the whole row's sum are needed. Only the softmax as it is reads
// the whole row. A wave per token; 16384 x 256 fp32: softmax as it is 11.9 us (34.6
// MB, 2.9 TB/s: exponentials and reductions), renormalised sigmoid 10.9 us (17.9 MB, the
// stores of whole rows of zeros), 9.0 us as it is; warm inputs.
template <typename T, int KPL>
__global__ __launch_bounds__(256) void gate_backward_kernel(GateBwdArgs p) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + wave;
  if (t >= p.T) return;
  const int E = p.E, k = p.k;
  const T* zr = (const T*)p.z + (size_t)t * E;

  int e = -1;
  float dw = 0.f, zc = -INFINITY;
  if (lane < k) {
    e = p.idx[(size_t)t * k + lane];
    if (e < 0 || e >= E) e = -1;  // no slot: nothing flows through it
    if (e >= 0) {
      dw = p.dw[(size_t)t * k + lane];
      zc = to_f32(zr[e]);
    }
  }
  // a masked expert has score 0 and gradient 0, whatever arrives at its slot
  const bool on = zc > -INFINITY;
  if (!on) dw = 0.f;

  float f[KPL];
  const bool full = p.softmax && !p.renorm;
  float fj = 0.f;
  if (p.softmax) {
    float m = -INFINITY, sum = 0.f;
    if (full) {
      load_logits<T, KPL>(zr, lane, E, f);
#pragma unroll
      for (int i = 0; i < KPL; ++i) m = fmaxf(m, f[i]);
    } else {
      m = on ? zc : -INFINITY;
    }
    m = wave_max(m);
    if (full) {
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        f[i] = !(f[i] > -INFINITY) ? 0.f : f[i] == m ? 1.f : expf(f[i] - m);
        sum += f[i];
      }
    }
    fj = !on ? 0.f : zc == m ? 1.f : expf(zc - m);
    if (full) {
      sum = wave_sum(sum);
      const float inv = sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
      for (int i = 0; i < KPL; ++i) f[i] *= inv;
      fj *= inv;
    }
  } else {
    // f = exp(min(z, 0)) / (1 + exp(-|z|)). Renormalised scores are taken over exp(top),
    // a factor that their sum has too: scores below 2^-126 would leave fp32's range.
    const float x = expf(-fabsf(zc));
    float num = zc >= 0.f ? 1.f : x;
    if (p.renorm) {
      const float least = fminf(zc, 0.f), top = wave_max(on ? least : -INFINITY);
      num = expf(least - top);
    }
    fj = on ? num / (1.f + x) : 0.f;
  }
  float df = p.rsf * dw;
  if (p.renorm) {
    const float S = wave_sum(fj);
    const float c = wave_sum(dw * fj);
    df = S > 0.f ? p.rsf / S * (dw - c / S) : 0.f;
  }
  // what each chosen slot adds to its logit, and the sum that every logit takes off
  float own = df * fj, common = 0.f;
  if (!p.softmax) {
    const float x = expf(-fabsf(zc));
    own = on ? own * ((zc >= 0.f ? x : 1.f) / (1.f + x)) : 0.f;  // 1 - f without cancellation
  } else if (full) {
    common = wave_sum(own);
  }
  float dz[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) dz[i] = full ? -f[i] * common : 0.f;
  for (int j = 0; j < k; ++j) {
    const int ej = __builtin_amdgcn_readlane(e, j);
    const float oj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(own), j));
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if (ej == lane * KPL + i) dz[i] += oj;
  }
  T* out = (T*)p.dz + (size_t)t * E;
  T o[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    if constexpr (sizeof(T) == 4)
      o[i] = dz[i];
    else
      o[i] = (T)f32_to_bf16_bits(dz[i]);
  }
  constexpr int BYTES = KPL * sizeof(T);
  if (BYTES >= 4 && BYTES <= 16 && E % KPL == 0) {  // as the logits are read
    if (lane * KPL < E)
      __builtin_memcpy(__builtin_assume_aligned(out + lane * KPL, BYTES <= 16 ? BYTES : 4), o, BYTES);
  } else {
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if (lane * KPL + i < E) out[lane * KPL + i] = o[i];
  }
}

template <typename F>
void by_keys(int E, F&& f) {
  const int per = (E + 63) / 64;
  if (per <= 1)
    f(std::integral_constant<int, 1>{});
  else if (per <= 2)
    f(std::integral_constant<int, 2>{});
  else if (per <= 4)
    f(std::integral_constant<int, 4>{});
  else if (per <= 8)
    f(std::integral_constant<int, 8>{});
  else
    f(std::integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_gate(const GateArgs& args, int f32, hipStream_t st) {
  GateArgs a = args;
  const int64_t slots = (int64_t)a.T * a.k;
  const int shares = (int)((slots + kCountShare - 1) / kCountShare);
  if (shares == 1) a.counts = nullptr;  // the count kernel writes them itself
  const size_t lds = a.n_group > 1 ? (size_t)4 * a.E * sizeof(double) : 0;
  const int G = a.n_group;
  if (a.T > kWaveTokens && a.E <= 512 && G <= 16 && (G & (G - 1)) == 0 && a.k <= 16) {
    const int lpg = 16 / G, c = (a.E / G + lpg - 1) / lpg;  // experts of a lane
    const int grid = (a.T + 15) / 16;
    auto go = [&](auto kpl) {
      if (f32)
        gate_rows_kernel<float, decltype(kpl)::value><<<grid, 256, lds, st>>>(a);
      else
        gate_rows_kernel<uint16_t, decltype(kpl)::value><<<grid, 256, lds, st>>>(a);
    };
    if (c <= 4)
      go(std::integral_constant<int, 4>{});
    else if (c <= 8)
      go(std::integral_constant<int, 8>{});
    else if (c <= 16)
      go(std::integral_constant<int, 16>{});
    else
      go(std::integral_constant<int, 32>{});
  } else {
    const int grid = (a.T + 3) / 4;
    by_keys(a.E, [&](auto c) {
      if (f32)
        gate_kernel<float, decltype(c)::value><<<grid, 256, lds, st>>>(a);
      else
        gate_kernel<uint16_t, decltype(c)::value><<<grid, 256, lds, st>>>(a);
    });
  }
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || !args.counts) return err;
  gate_count_kernel<<<shares, 1024, 0, st>>>(a.idx, slots, a.E, args.counts);
  return hipGetLastError();
}

hipError_t launch_gate_backward(const GateBwdArgs& a, int f32, hipStream_t st) {
  const int grid = (a.T + 3) / 4;
  by_keys(a.E, [&](auto c) {
    if (f32)
      gate_backward_kernel<float, decltype(c)::value><<<grid, 256, 0, st>>>(a);
    else
      gate_backward_kernel<uint16_t, decltype(c)::value><<<grid, 256, 0, st>>>(a);
  });
  return hipGetLastError();
}

}  // namespace beam
