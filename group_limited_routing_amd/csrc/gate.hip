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
// by the values themselves, not by an fp32 rounding of them.
#include "common.h"
#include "operators.h"

namespace beam {
namespace {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_bits_to_f32(v); }

// Maximum over the wave, in every lane: the moves of wave_max in the router,
// on both words of a double.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp_max(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const int lo = (int)(uint32_t)b, hi = (int)(uint32_t)(b >> 32);
  const uint32_t olo = (uint32_t)__builtin_amdgcn_update_dpp(lo, lo, CTRL, ROWS, 0xF, false);
  const uint32_t ohi = (uint32_t)__builtin_amdgcn_update_dpp(hi, hi, CTRL, ROWS, 0xF, false);
  return fmax(v, __builtin_bit_cast(double, (uint64_t)ohi << 32 | olo));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_max(double v) {
  v = dpp_max<0xB1>(v);
  v = dpp_max<0x4E>(v);
  v = dpp_max<0x141>(v);
  v = dpp_max<0x140>(v);
  v = dpp_max<0x142, 0xA>(v);
  v = dpp_max<0x143, 0xC>(v);
  return lane_value(v, 63);
}
template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

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
// took 100 us at 16384 tokens x 8, all on 256 addresses.
constexpr int kCountShare = 16384;  // slots of a workgroup

__global__ __launch_bounds__(256) void gate_zero_kernel(int32_t* counts, int E) {
  const int e = blockIdx.x * 256 + threadIdx.x;
  if (e < E) counts[e] = 0;
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

template <typename T, int KPL>
__global__ __launch_bounds__(256) void gate_kernel(GateArgs p) {
  extern __shared__ double lds_keys[];  // [4][E], groups that are not whole powers of two of lanes
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + wave;
  if (t >= p.T) return;  // no barrier below: a wave works alone
  const int E = p.E, k = p.k;
  if (p.valid && !p.valid[t]) {
    if (lane < k) {
      p.idx[(size_t)t * k + lane] = -1;
      p.w[(size_t)t * k + lane] = 0.f;
    }
    return;
  }
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
      double* keys = lds_keys + (size_t)wave * E;
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

// ------------------------------------------------------------------ backward
// With the chosen scores f_j, S their sum, and the gradient dw of the weights:
//   renormalised:     df_j = rsf / S (dw_j - sum_i dw_i f_i / S)
//   as they are:      df_j = rsf dw_j
//   sigmoid:          dz_j = df_j f_j (1 - f_j), 0 for the others
//   softmax:          dz_e = f_e (df_e - sum_j df_j f_j)
// Renormalised softmax weights are the softmax over the chosen logits alone:
// their inner sum is 0, nothing flows to the others, and neither the other
// logits nor the whole row's sum are needed. Only the softmax as it is reads
// the whole row.
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
  const bool on = zc > -INFINITY;  // a masked expert has score 0 and gradient 0

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
#pragma unroll
    for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
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
    const float x = expf(-fabsf(zc));
    fj = on ? (zc >= 0.f ? 1.f : x) / (1.f + x) : 0.f;
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
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int c = lane * KPL + i;
    if (c < E) {
      if constexpr (sizeof(T) == 4)
        out[c] = dz[i];
      else
        out[c] = (T)f32_to_bf16_bits(dz[i]);
    }
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

hipError_t launch_gate(const GateArgs& a, int f32, hipStream_t st) {
  const size_t lds = a.n_group > 1 ? (size_t)4 * a.E * sizeof(double) : 0;
  const int grid = (a.T + 3) / 4;
  by_keys(a.E, [&](auto c) {
    if (f32)
      gate_kernel<float, decltype(c)::value><<<grid, 256, lds, st>>>(a);
    else
      gate_kernel<uint16_t, decltype(c)::value><<<grid, 256, lds, st>>>(a);
  });
  if (a.counts) {
    const int64_t n = (int64_t)a.T * a.k;
    const int shares = (int)((n + kCountShare - 1) / kCountShare);
    if (shares > 1) gate_zero_kernel<<<(a.E + 255) / 256, 256, 0, st>>>(a.counts, a.E);
    gate_count_kernel<<<shares, 1024, 0, st>>>(a.idx, n, a.E, a.counts);
  }
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
