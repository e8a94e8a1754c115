// The dense MLP's gated product: h = act(x Wg^T) * (x Wu^T) in one kernel, and its
// gradient.
//
// Beam launch post ("Introducing Beam"), section "Mixture of Experts": the first
// three layers have a dense SwiGLU MLP in place of the experts.
#include "common.h"
#include "operators.h"
#include "tile.h"

#include <algorithm>

namespace beam {
namespace {

// The normal distribution Phi(g) = erfc(-g / sqrt 2) / 2, and e^(-g^2 / 2) in e, with a
// relative accuracy of 4 (g^2 + 16) 2^-24, also where Phi is small. e^(x^2) erfc(x) = t P(t)
// with t = 1 / (1 + 0.35 x); P of degree 9 is a Chebyshev fit over all x >= 0, within 5e-8 of the
// quotient. About 20 instructions; erfcf, whose ranges are branches, took 150, and 15 us of
// an output of 1111 x 5000.
__device__ __forceinline__ float normal_cdf(float g, float& e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(g), 0.35f * 0.70710678118654752f, 1.0f));
  e = __builtin_amdgcn_exp2f(g * g * -0.72134752044448170f);
  float p = 0.0393733224f;
  p = fmaf(p, t, -0.167890257f);
  p = fmaf(p, t, 0.210833749f);
  p = fmaf(p, t, -0.0772500421f);
  p = fmaf(p, t, 0.136077123f);
  p = fmaf(p, t, 0.116022718f);
  p = fmaf(p, t, 0.162620229f);
  p = fmaf(p, t, 0.185278087f);
  p = fmaf(p, t, 0.197468678f);
  p = fmaf(p, t, 0.197466345f);
  const float tail = 0.5f * e * (p * t);
  return g < 0.f ? tail : 1.0f - tail;
}

// act(g), and its derivative in d.
template <bool GELU>
__device__ __forceinline__ float activation(float g) {
  float e;
  if constexpr (GELU)
    return g * normal_cdf(g, e);
  else
    return silu_f32(g);
}
template <bool GELU>
__device__ __forceinline__ float activation(float g, float& d) {
  if constexpr (GELU) {
    float e;
    const float p = normal_cdf(g, e);
    d = p + g * 0.39894228040143268f * e;
    return g * p;
  } else {
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f));
    d = s * (1.0f + g * (1.0f - s));
    return g * s;
  }
}

// ------------------------------------------------------------------ tiles
// One kernel for the three products, out[m, n] = sum over k of x[m, k] w[n, k], whose
// operands lie in memory as rows of k ("along") or with a row for each k ("across"):
//   kGated    x [T, H] along, the rows of w_gate and w_up along, 32 of each in turn, so
//             that a wave holds gate and up of the same columns: the activation and the
//             product are its epilogue.
//   kInput    d_gate along and w_gate across, then d_up and w_up: one sum over 2 F.
//   kWeights  d_gate (or d_up) across, x across: a sum over the tokens.
//
// Large products are bound by the matrix cores under the chip's power limit: 8192 x 5120 x
// 10240 (kGated, 1.72e12 operations) takes 1.26 to 1.31 ms a call in a row of them (1.3 to 1.4 each
// under the profiler), 1.31 to 1.36 PF/s, with the matrix cores
// busy 76% of the time at 1.45 to 1.65 GHz. The same loop without its loads from memory takes
// 1.14 ms, without reads of LDS 1.19, without both 0.85 (the instructions alone). The
// gradient's two products at 4096 tokens: 1.32 to 1.41 ms, profiled.
enum Mode { kGated, kInput, kWeights };

struct TileArgs {
  const uint8_t* x[2];
  const uint8_t* w[2];
  int64_t ldx, ldw;  // bytes of a row in memory
  int M, N, K;       // N: columns of the output; K: of one of the two sums of kInput
  const uint16_t* add_gate;
  const uint16_t* add_up;
  uint16_t* out[2];  // h; or the output of each of two products
  void* pre[2];      // gate and up, bf16 or fp32, or null
  bool pre_f32;
  // The first `whole` tiles are one item of work each; the others are cut into `splits`
  // ranges of k, whose sums go to part[item - whole], a tile each.
  int whole, items, splits;
  float* part;
};

typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// 4 values of one column from each of 4 rows: lanes 4 i .. 4 i + 3 of 16 give the
// addresses of 4 values each of row i, and lane c gets column c.
__device__ __forceinline__ u32x2 read_across(const uint8_t* p) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
#else
  return {};
#endif
}

// dma16 as the instruction itself. Behind the builtin, the compiler has a transposing read
// wait for all loads in flight, whatever they write, and another read of LDS for all reads
// before it (8192 x 5120 x 5120, kWeights: 1647 us and 761 us so). The kernel's own
// waits and barriers say when a stage has landed.
__device__ __forceinline__ void dma16_unseen(const uint8_t* src, const uint8_t* lds_base) {
#if defined(__HIP_DEVICE_COMPILE__)
  const uint32_t at = (uint32_t)(uintptr_t)(lds_s16x4*)lds_base;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(at), "v"(src)
               : "memory", "m0");
#endif
}

__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
#else
  return c;
#endif
}

// Waves as WM x WN, each FM x FN fragments of 32 x 32 on 32x32x16 MFMAs (w first, so
// that a lane ends with runs of 4 consecutive output columns). Operands go from memory
// straight into LDS (16 bytes a lane) through a ring of NS stages of 64 values of k (four
// stages of 32, twice the barriers: 1386 us where two of 64 take 1290; 8192 x 5120 x 10240). A
// workgroup stays for many items of work, and its loads run ahead into the next one, so
// that neither the first loads of an item nor its output stop the ring.
//
// LDS of a stage. Along: 128 bytes a row, swizzled as tile.h says. Across: a row of the
// tile's width for each k; the 64-byte chunk c (32 columns, one fragment) of row k
// stands at c ^ (k & 3), so that the 4 rows of a transposing read cover all banks.
template <Mode MODE, int FM, int FN, int WM, int WN>
struct Tile {
  static constexpr int WAVES = WM * WN, BM = 32 * FM * WM, BN = 32 * FN * WN;
  static constexpr int KS = 64;  // values of k in a stage
  static constexpr int X_BYTES = BM * 2 * KS, STAGE = (BM + BN) * 2 * KS;
  static constexpr int NS = BM == 64 && MODE == kGated ? 3 : 2;  // stages: what LDS holds
  static constexpr int COLS = MODE == kGated ? FN * 16 : FN * 32;  // of the output, a wave's
  static constexpr int TN = COLS * WN;                             // and the tile's
  static constexpr int STAGING = 32 * COLS * 2;                    // 32 rows of a wave's output
  static constexpr int LDS = NS * STAGE + WAVES * STAGING;
  static constexpr int PER_CU = LDS <= 80 * 1024 ? 2 : 1;          // workgroups
};

// The work of workgroup `block` of `blocks`, in `smem`.
template <Mode MODE, int FM, int FN, int WM, int WN, bool RAGGED, bool GELU>
__device__ __forceinline__ void tile_work(const TileArgs& p, int block, int blocks, uint8_t* smem) {
  using S = Tile<MODE, FM, FN, WM, WN>;
  constexpr bool XA = MODE == kWeights, WA = MODE != kGated;  // across
  constexpr int BM = S::BM, BN = S::BN, NS = S::NS, WAVES = S::WAVES, TN = S::TN;
  constexpr int KS = S::KS, ROW = 2 * KS, HALVES = KS / 16;
  constexpr int XU = S::X_BYTES / 1024, WU = BN * ROW / 1024, PER = (XU + WU) / WAVES;
  static_assert(XU % WAVES == 0 && WU % WAVES == 0, "a load is of one operand for every wave");
  static_assert((!XA || BM >= 128) && (!WA || BN >= 128), "four 64-byte chunks in a row of k");

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave / WN, wn = wave % WN, r = lane & 31, h = lane >> 5;
  const int nk1 = (p.K + KS - 1) / KS, nk_all = MODE == kInput ? 2 * nk1 : nk1;
  const int mtt = (p.M + BM - 1) / BM, ntt = (p.N + TN - 1) / TN;
  constexpr int PROBLEMS = MODE == kWeights ? 2 : 1;
  struct Item {
    int m0, n0, problem, k0, nk, part;
  };
  auto item_of = [&](int i) {
    Item t;
    int tile = i, split = 0, splits = 1;
    t.part = -1;
    if (i >= p.whole) {
      t.part = i - p.whole;
      splits = p.splits;
      tile = p.whole + t.part / splits;
      split = t.part % splits;
    }
    tile_of(tile, PROBLEMS * mtt * ntt, PROBLEMS * mtt, ntt, t.m0, t.n0);
    t.problem = MODE == kWeights && t.m0 >= mtt;
    t.m0 = (t.problem ? t.m0 - mtt : t.m0) * BM;
    t.n0 *= TN;
    t.k0 = (uint32_t)nk_all * split / splits;
    t.nk = (int)((uint32_t)nk_all * (split + 1) / splits) - t.k0;
    return t;
  };

  // Loads: sources of this lane's, as offsets from the tile's first element (at most 256
  // rows of 512 KB); rows and columns past the end repeat the last ones.
  const int64_t xstep = XA ? KS * p.ldx : ROW, wstep = WA ? KS * p.ldw : ROW;
  uint32_t src[PER];
  int srck[RAGGED ? PER : 1];  // first value of k of the lane's chunk in a stage
  const uint8_t *x0, *x1, *w0, *w1;  // the tile's first elements
  int load_item = block, load_k, load_end;  // the stage that the next loads are of
  // The lane anew, as a value that no loop knows: what an item computes from it once is not
  // kept in registers across the stages.
  auto fresh_lane = [&] {
    int l = threadIdx.x & 63;
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+v"(l));
#endif
    return l;
  };
  auto seek = [&]() {
    const Item t = item_of(load_item);
    const int lane = fresh_lane();
    load_k = t.k0;
    load_end = t.k0 + t.nk;
    const int mlast = p.M - 1 - t.m0, nlast = p.N - 1 - t.n0;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const bool of_x = q * WAVES < XU;
      const int v = q * WAVES + wave - (of_x ? 0 : XU);  // unit of its operand
      if (of_x ? XA : WA) {
        const int B = of_x ? BM : BN, at = v * 1024 + lane * 16, k = at / (2 * B);
        const int pos = at % (2 * B), c = ((((pos >> 6) ^ (k & 3)) << 6) | (pos & 63)) / 2;
        const int last = ((of_x ? mlast : nlast) & ~7);
        src[q] = (uint32_t)(k * (of_x ? p.ldx : p.ldw)) + min(c, last) * 2;
        if (RAGGED) srck[q] = k;
      } else {
        constexpr int CH = ROW / 16;  // chunks of a row
        const int row = v * (64 / CH) + lane / CH, c = (lane % CH) ^ swizzle<ROW>(row);
        const int at = of_x || MODE != kGated ? row : (row / 64) * 32 + row % 32;
        src[q] = (uint32_t)(min(at, of_x ? mlast : nlast) * (of_x ? p.ldx : p.ldw)) + c * 16;
        if (RAGGED) srck[q] = c * 8;
      }
    }
    const int64_t xat = XA ? 2 * (int64_t)t.m0 : t.m0 * p.ldx, wat = WA ? 2 * (int64_t)t.n0 : t.n0 * p.ldw;
    x0 = (MODE == kWeights && t.problem ? p.x[1] : p.x[0]) + xat;
    x1 = p.x[1] + xat;
    w0 = p.w[0] + wat;
    w1 = p.w[1] + wat;
  };
  auto advance = [&]() {
    if (++load_k < load_end) return;
    // behind the last item its stages are loaded again, which nothing reads
    if (load_item + blocks < p.items) load_item += blocks;
    seek();
  };
  auto issue_one = [&](int slot, auto qc) {  // load q of the stage into a slot
    constexpr int Q = decltype(qc)::value;
    if constexpr (Q < PER) {
      constexpr bool OF_X = Q * WAVES < XU;
      const int u = Q * WAVES + wave, seg = MODE == kInput && load_k >= nk1, kt = load_k - (seg ? nk1 : 0);
      // kGated: 32 rows of w_gate, then the same of w_up
      const bool second = MODE == kGated ? !OF_X && (u - XU) * (1024 / ROW) / 32 % 2 : seg;
      const uint8_t* b = OF_X ? (second ? x1 : x0) : (second ? w1 : w0);
      const uint8_t* at = scalar(b + kt * (OF_X ? xstep : wstep)) + src[Q];
      if (RAGGED && kt * KS + srck[RAGGED ? Q : 0] >= p.K) at = kZeros;
      dma16_unseen(at, smem + slot + u * 1024);
    }
  };

  // Operand offsets in a stage. Along: fragment i is 32 rows on, chunk 2 j + h in step j.
  // Across: fragment i is 64-byte chunk (first + i) of rows 16 j + 8 h + 4 e + kk.
  const int kk = lane % 16 / 4, ac = (lane / 16 % 2) * 32 + lane % 4 * 8;
  int xo[XA ? FM : HALVES], wo[WA ? FN : HALVES];
  if constexpr (XA) {
#pragma unroll
    for (int i = 0; i < FM; ++i) xo[i] = (8 * h + kk) * (2 * BM) + (((wm * FM + i) ^ kk) << 6) + ac;
  } else {
#pragma unroll
    for (int j = 0; j < HALVES; ++j) xo[j] = (wm * FM * 32 + r) * ROW + (((2 * j + h) ^ swizzle<ROW>(r)) << 4);
  }
  if constexpr (WA) {
#pragma unroll
    for (int i = 0; i < FN; ++i)
      wo[i] = S::X_BYTES + (8 * h + kk) * (2 * BN) + (((wn * FN + i) ^ kk) << 6) + ac;
  } else {
#pragma unroll
    for (int j = 0; j < HALVES; ++j)
      wo[j] = S::X_BYTES + (wn * FN * 32 + r) * ROW + (((2 * j + h) ^ swizzle<ROW>(r)) << 4);
  }
  auto across = [](const uint8_t* at, int pitch) {
    const u32x2 lo = read_across(at), hi = read_across(at + 4 * pitch);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  };

  f32x16 acc[FM][FN];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
  };

  // A stage is HALVES steps of 16 values of k, each FM x FN instructions. Beside every
  // instruction goes at most a read or two of LDS and a load, so that neither queue
  // holds the wave back: the fragments of step j + 1 are read during step j, those of the
  // next stage's step 0 during the last one. The barrier before the last step says that
  // every wave has read all of stage s, whose slot stage s + NS refills from then on, and
  // that stage s + 1 has landed.
  constexpr int SLOTS = FM * FN, READS = FM + FN, WITHIN = SLOTS > 4 ? SLOTS * 3 / 4 : SLOTS;
  u32x4 xr[2][FM], wr[2][FN];
  auto read_one = [&](const uint8_t* st, auto jc, auto qc) {  // x fragment 0, w's, the other x's
    constexpr int J = decltype(jc)::value, Q = decltype(qc)::value;
    if constexpr (Q >= 1 && Q <= FN) {
      constexpr int N = Q - 1;
      if constexpr (WA)
        wr[J % 2][N] = across(st + wo[N] + J * 16 * (2 * BN), 2 * BN);
      else
        wr[J % 2][N] = ld16(st + wo[J] + N * 32 * ROW);
    } else {
      constexpr int I = Q == 0 ? 0 : Q - FN;
      if constexpr (XA)
        xr[J % 2][I] = across(st + xo[I] + J * 16 * (2 * BM), 2 * BM);
      else
        xr[J % 2][I] = ld16(st + xo[J] + I * 32 * ROW);
    }
  };
  // loads of a stage that go beside the last step of the stage NS before it; the others
  // beside the first steps of the next one
  constexpr int TURN = (HALVES - 1) * SLOTS, WINDOW = HALVES * SLOTS * (MODE == kGated ? 3 : 4) / 8;
  constexpr int FIRST = (SLOTS * PER + WINDOW - 1) / WINDOW < PER ? (SLOTS * PER + WINDOW - 1) / WINDOW : PER;
  auto issue_some = [&](int slot, auto from, auto to) {
    constexpr int A = decltype(from)::value, B = decltype(to)::value;
    for_each<(B > A ? B - A : 0)>([&](auto e) {
      issue_one(slot, std::integral_constant<int, A + decltype(e)::value>{});
    });
  };
  std::integral_constant<int, 0> j0;
  std::integral_constant<int, 1> j1;
  std::integral_constant<int, FIRST> first;
  std::integral_constant<int, PER> per;

  seek();
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) {
    issue_some(s * S::STAGE, j0, per);
    advance();
  }
  issue_some((NS - 1) * S::STAGE, j0, first);
  wait_vmcnt<(NS - 2) * PER + FIRST>();
  barrier_only();
  asm volatile("" ::: "memory");
  for_each<READS>([&](auto q) { read_one(smem, j0, q); });
  int slot = 0, before = (NS - 1) * S::STAGE;  // of this stage, and of the one before it
  for (int item = block; item < p.items; item += blocks) {
    const Item t = item_of(item);
    clear();
    for (int s = 0; s < t.nk; ++s) {
      const int next = slot == (NS - 1) * S::STAGE ? 0 : slot + S::STAGE;
      for_each<HALVES * SLOTS>([&](auto tc) {
        constexpr int T = decltype(tc)::value, J = T / SLOTS, M = T % SLOTS, I = M / FN, N = M % FN;
        if constexpr (T == TURN) {
          advance();
          wait_vmcnt<(NS - 2) * PER>();
          wait_lgkmcnt0();
          barrier_only();
          asm volatile("" ::: "memory");
        }
        constexpr int R0 = M < WITHIN ? M * READS / WITHIN : READS;
        constexpr int R1 = M < WITHIN ? (M + 1) * READS / WITHIN : READS;
        for_each<R1 - R0>([&](auto e) {
          std::integral_constant<int, R0 + decltype(e)::value> q;
          if constexpr (J + 1 < HALVES)
            read_one(smem + slot, std::integral_constant<int, J + 1>{}, q);
          else
            read_one(smem + next, j0, q);
        });
        // load q goes beside instruction q WINDOW / PER behind the barrier
        constexpr int O = T >= TURN ? T - TURN : T + SLOTS;
        constexpr int A = (O * PER + WINDOW - 1) / WINDOW, B = ((O + 1) * PER + WINDOW - 1) / WINDOW;
        issue_some(T >= TURN ? slot : before, std::integral_constant<int, A < PER ? A : PER>{},
                   std::integral_constant<int, B < PER ? B : PER>{});
        acc[I][N] = mfma32(wr[J % 2][N], xr[J % 2][I], acc[I][N]);
        __builtin_amdgcn_sched_barrier(0);
      });
      before = slot;
      slot = next;
    }

    // Output: lane (r, h) of a fragment holds row r, columns 8 q + 4 h .. + 3.
    const int lane = fresh_lane(), r = lane & 31, h = lane >> 5;
    if (t.part >= 0) {
      float* to = p.part + (size_t)t.part * (BM * BN) + wn * FN * 32 + 4 * h;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (t.m0 + (wm * FM + i) * 32 + r < p.M) st16(to + ((wm * FM + i) * 32 + r) * BN + j * 32 + 8 * q,
                 u32x4{__float_as_uint(acc[i][j][4 * q]), __float_as_uint(acc[i][j][4 * q + 1]),
                       __float_as_uint(acc[i][j][4 * q + 2]), __float_as_uint(acc[i][j][4 * q + 3])});
      continue;
    }
    // 32 rows of the wave at a time go through its own piece of LDS, so that a store
    // writes whole runs of a row. 16-byte chunk c of row r stands at c ^ key(r): rows that
    // share banks differ in it.
    constexpr int COLS = S::COLS, L = COLS / 8, RS = 64 / L;
    uint8_t* mine = smem + NS * S::STAGE + wave * S::STAGING;
    auto chunk = [&](int row, int c) { return mine + row * (COLS * 2) + ((c ^ (row / (16 / L) % L)) << 4); };
    const int c0 = t.n0 + wn * COLS;
    const int row_l = lane / L, ch_l = lane % L;
    const bool col_in = c0 + ch_l * 8 < p.N;
    // what is added to a fragment is loaded during the one before it (what lies outside: other
    // values, which are not stored)
    constexpr int G = 32 / RS;
    u32x4 gate_add[G], up_add[G];
    auto fetch = [&](int i) {
      const int c = min(c0 + ch_l * 8, p.N - 8);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const size_t at = (size_t)min(t.m0 + (wm * FM + i) * 32 + g * RS + row_l, p.M - 1) * p.N + c;
        if (p.add_gate) gate_add[g] = ld16(p.add_gate + at);
        if (p.add_up) up_add[g] = ld16(p.add_up + at);
      }
    };
    if constexpr (MODE == kGated) fetch(0);
    for_each<FM>([&](auto ic) {
      constexpr int I = decltype(ic)::value;
      const int mb = t.m0 + (wm * FM + I) * 32;
      auto settle = [] {  // this wave's reads and writes of its piece
        wait_lgkmcnt0();
        asm volatile("" ::: "memory");
      };
      auto put = [&](uint16_t* out, auto value) {  // value(j, i): column 32 j + .. in acc's order
#pragma unroll
        for (int j = 0; j < COLS / 32; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<u32x2*>(chunk(r, j * 4 + q) + 8 * h) =
                u32x2{pack_bf16x2(value(j, 4 * q), value(j, 4 * q + 1)),
                      pack_bf16x2(value(j, 4 * q + 2), value(j, 4 * q + 3))};
        settle();
#pragma unroll
        for (int g = 0; g < 32 / RS; ++g) {
          const int row = g * RS + row_l;
          if (mb + row < p.M && col_in)
            st16(out + (size_t)(mb + row) * p.N + c0 + ch_l * 8, ld16(chunk(row, ch_l)));
        }
        settle();
      };
      if constexpr (MODE == kGated) {
        auto add = [&](const u32x4 (&from)[G], auto which) {  // onto gate (0) or up (1)
          constexpr int W = decltype(which)::value;
#pragma unroll
          for (int g = 0; g < G; ++g) st16(chunk(g * RS + row_l, ch_l), from[g]);
          settle();
#pragma unroll
          for (int j = 0; j < COLS / 32; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const u32x2 v = *reinterpret_cast<const u32x2*>(chunk(r, j * 4 + q) + 8 * h);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                acc[I][2 * j + W][4 * q + 2 * e] += __uint_as_float(v[e] << 16);
                acc[I][2 * j + W][4 * q + 2 * e + 1] += __uint_as_float(v[e] & 0xffff0000u);
              }
            }
          settle();
        };
        if (p.add_gate) add(gate_add, j0);
        if (p.add_up) add(up_add, j1);
        if constexpr (I + 1 < FM) fetch(I + 1);
        put(p.out[0], [&](int j, int i) { return activation<GELU>(acc[I][2 * j][i]) * acc[I][2 * j + 1][i]; });
        auto keep = [&](void* out, auto which) {  // gate (0) or up (1)
          constexpr int W = decltype(which)::value;
          if (!p.pre_f32) return put((uint16_t*)out, [&](int j, int i) { return acc[I][2 * j + W][i]; });
          // fp32: 32 bytes of a row from two lanes, straight from the sums (4096 x 5120 x 10240:
          // 760 us, with a bf16 pair 690, without 653)
          if (mb + r < p.M)
#pragma unroll
            for (int j = 0; j < COLS / 32; ++j)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int c = c0 + j * 32 + 8 * q + 4 * h;
                const f32x16& v = acc[I][2 * j + W];
                if (c < p.N)
                  *reinterpret_cast<f32x4*>((float*)out + (size_t)(mb + r) * p.N + c) =
                      f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
              }
        };
        if (p.pre[0]) keep(p.pre[0], j0);
        if (p.pre[1]) keep(p.pre[1], j1);
      } else {
        put(p.out[t.problem], [&](int j, int i) { return acc[I][j][i]; });
      }
    });
  }
  wait_vmcnt<0>();  // no load is in flight when the workgroup's LDS is given away
}

template <Mode MODE, int FM, int FN, int WM, int WN, bool RAGGED, bool GELU>
__global__ __launch_bounds__(64 * WM * WN)
    __attribute__((amdgpu_waves_per_eu(Tile<MODE, FM, FN, WM, WN>::PER_CU * WM * WN / 4)))
void tile_kernel(TileArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[Tile<MODE, FM, FN, WM, WN>::LDS];
  tile_work<MODE, FM, FN, WM, WN, RAGGED, GELU>(p, blockIdx.x, gridDim.x, smem);
}

// Both products of the gradient in one launch, which do not wait for each other: the first
// `first` workgroups have dx, by waves of FM x FN fragments, the others the weights'
// gradients, by waves of GM x FN. (777 x 1288 x 1000: 28 us, so 18 and 13 one after the other;
// 4096 x 5120 x 10240: the second product's tiles fill the end of the first's last round.)
template <int FM, int FN, int GM, int WM, int WN, bool RAGGED>
__global__ __launch_bounds__(64 * WM * WN)
    __attribute__((amdgpu_waves_per_eu(Tile<kWeights, GM, FN, WM, WN>::PER_CU * WM * WN / 4)))
void gradients_kernel(TileArgs in, TileArgs weights, int first) {
  using A = Tile<kInput, FM, FN, WM, WN>;
  using B = Tile<kWeights, GM, FN, WM, WN>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[A::LDS > B::LDS ? A::LDS : B::LDS];
  if ((int)blockIdx.x < first)
    tile_work<kInput, FM, FN, WM, WN, RAGGED, false>(in, blockIdx.x, first, smem);
  else
    tile_work<kWeights, GM, FN, WM, WN, RAGGED, false>(weights, blockIdx.x - first, gridDim.x - first, smem);
}

// The tiles that were cut along k: the sum of a tile's parts, in their order, and what
// tile_kernel does with a sum. 8 columns a thread. Bound by the latency of its loads and its
// start: 4 to 5 us at a few MB of parts, 18 us for 67 MB.
template <Mode MODE, int BM, int BN, bool GELU>
__global__ __launch_bounds__(64) void finish_kernel(TileArgs p) {
  constexpr int TN = MODE == kGated ? BN / 2 : BN, PROBLEMS = MODE == kWeights ? 2 : 1;
  const int mtt = (p.M + BM - 1) / BM, ntt = (p.N + TN - 1) / TN;
  int mi, ni;
  tile_of(p.whole + blockIdx.x, PROBLEMS * mtt * ntt, PROBLEMS * mtt, ntt, mi, ni);
  const bool problem = MODE == kWeights && mi >= mtt;
  const int at = blockIdx.y * 64 + threadIdx.x, row = at / (TN / 8), c = at % (TN / 8) * 8;
  const int m = (problem ? mi - mtt : mi) * BM + row, n = ni * TN + c;
  if (row >= BM || m >= p.M || n >= p.N) return;
  const float* from = p.part + (size_t)blockIdx.x * p.splits * (BM * BN) + row * BN;
  auto sum8 = [&](int col, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    for (int s = 0; s < p.splits; s += 4) {  // four parts' loads at a time
      u32x4 a[4], b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float* at = from + (size_t)min(s + e, p.splits - 1) * (BM * BN) + col;
        a[e] = ld16(at);
        b[e] = ld16(at + 4);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (s + e < p.splits)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] += __uint_as_float(a[e][i]);
            v[4 + i] += __uint_as_float(b[e][i]);
          }
    }
  };
  auto add8 = [](const uint16_t* q, float (&v)[8]) {
    const u32x4 a = ld16(q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] += __uint_as_float(a[i] << 16);
      v[2 * i + 1] += __uint_as_float(a[i] & 0xffff0000u);
    }
  };
  auto put8 = [](uint16_t* q, const float (&v)[8]) {
    st16(q, u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                  pack_bf16x2(v[6], v[7])});
  };
  const size_t to = (size_t)m * p.N + n;
  float g[8];
  if constexpr (MODE == kGated) {
    float u[8], f[8];
    sum8(2 * (c - c % 32) + c % 32, g);
    sum8(2 * (c - c % 32) + 32 + c % 32, u);
    if (p.add_gate) add8(p.add_gate + to, g);
    if (p.add_up) add8(p.add_up + to, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = activation<GELU>(g[i]) * u[i];
    put8(p.out[0] + to, f);
    auto keep = [&](void* out, const float (&v)[8]) {
      if (!p.pre_f32) return put8((uint16_t*)out + to, v);
      f32x4* at = reinterpret_cast<f32x4*>((float*)out + to);
      at[0] = f32x4{v[0], v[1], v[2], v[3]};
      at[1] = f32x4{v[4], v[5], v[6], v[7]};
    };
    if (p.pre[0]) keep(p.pre[0], g);
    if (p.pre[1]) keep(p.pre[1], u);
  } else {
    sum8(c, g);
    put8((problem ? p.out[1] : p.out[0]) + to, g);
  }
}

// How a product is cut. Rounds of 256 PER_CU workgroups take whole tiles; what is left
// would keep a part of the chip busy for a whole round, so it is cut along k into as many
// parts as make it cheapest. Costs in ns: a stage of a full round, the parts' way through
// memory at 2 TB/s, and 5 us for the second kernel. It is a model: a stage of a partial round is
// taken to cost as much as a full round's, and each product to have the chip to itself, also where
// two are launched together. (64 tokens, 5120 x 10240: 160 tiles of
// the 512 that run at once, cut in 3, 48 us and 5 us for the sums; the weights alone are
// 31 us at 6.9 TB/s.)
struct Cut {
  int whole, items, splits;
  int64_t cost;
};
Cut cut_of(int tiles, int stages, int slots, int tile_bytes, int stage_ns) {
  const int rest = tiles % slots;
  Cut c{tiles, tiles, 1, (int64_t)((tiles + slots - 1) / slots) * stages * stage_ns};
  if (rest == 0) return c;
  const int64_t before = (int64_t)(tiles / slots) * stages * stage_ns;
  for (int s = 2; s <= 16 && s * 4 <= stages; ++s) {
    const int64_t rounds = ((int64_t)rest * s + slots - 1) / slots;
    const int64_t cost = before + rounds * ((stages + s - 1) / s) * stage_ns +
                         (int64_t)rest * s * tile_bytes / 2000 + 5000;
    if (cost < c.cost) c = {tiles - rest, tiles - rest + rest * s, s, cost};
  }
  return c;
}

template <Mode MODE, int FM, int FN, int WM, int WN>
Cut cut_for(int M, int N, int K, int stage_ns) {
  using S = Tile<MODE, FM, FN, WM, WN>;
  const int mt = (M + S::BM - 1) / S::BM * (MODE == kWeights ? 2 : 1), nt = (N + S::TN - 1) / S::TN;
  return cut_of(mt * nt, (K + S::KS - 1) / S::KS * (MODE == kInput ? 2 : 1), 256 * S::PER_CU,
                S::BM * S::BN * 4, stage_ns);
}

TileArgs with_cut(TileArgs a, const Cut& c) {
  a.whole = c.whole;
  a.items = c.items;
  a.splits = c.splits;
  return a;
}
template <Mode MODE, int FM, int FN, int WM, int WN>
int grid_of(const Cut& c) {
  return std::min(c.items, 256 * Tile<MODE, FM, FN, WM, WN>::PER_CU);
}
template <Mode MODE, int FM, int FN, int WM, int WN, bool GELU>
void finish(const TileArgs& t, hipStream_t st) {
  using S = Tile<MODE, FM, FN, WM, WN>;
  if (t.splits > 1)
    finish_kernel<MODE, S::BM, S::BN, GELU>
        <<<dim3((t.items - t.whole) / t.splits, (std::min(S::BM, t.M) * S::TN + 511) / 512), 64, 0, st>>>(t);
}

template <Mode MODE, int FM, int FN, int WM, int WN>
void tile_launch(const TileArgs& a, const Cut& c, int gelu, hipStream_t st) {
  using S = Tile<MODE, FM, FN, WM, WN>;
  const TileArgs t = with_cut(a, c);
  auto go = [&](auto rc, auto gc) {
    constexpr bool R = decltype(rc)::value, G = decltype(gc)::value;
    tile_kernel<MODE, FM, FN, WM, WN, R, G><<<grid_of<MODE, FM, FN, WM, WN>(c), 64 * S::WAVES, 0, st>>>(t);
    finish<MODE, FM, FN, WM, WN, G>(t, st);
  };
  auto with = [&](auto rc) {
    if constexpr (MODE == kGated) {
      if (gelu) return go(rc, std::true_type{});
    }
    go(rc, std::false_type{});
  };
  if (a.K % S::KS != 0)
    with(std::true_type{});
  else
    with(std::false_type{});
}

// Tiles of 256 x 256, 128 x 128 and 64 x 128 (columns of w): the one whose cut costs least.
// A stage of a full round (256, 512 and 512 tiles) takes 1.6, 1.1 and 0.75 us (8192 x 5120 x
// 10240 by one tile alone: 1.29, 1.76 and 2.37 ms; the gradient's products are given the same).
constexpr size_t kTileFloats[3] = {256 * 256, 128 * 128, 64 * 128};
struct Choice {
  int tile;
  Cut cut;
  size_t part_bytes() const {
    return cut.splits > 1 ? (cut.items - cut.whole) * kTileFloats[tile] * sizeof(float) : 0;
  }
};
template <Mode MODE>
Choice choose(int M, int N, int K) {
  Choice best{0, cut_for<MODE, 4, 2, 2, 4>(M, N, K, 1600)};
  const Cut c = cut_for<MODE, 2, 2, 2, 2>(M, N, K, 1100);
  if (c.cost < best.cut.cost) best = {1, c};
  if constexpr (MODE != kWeights) {  // a row of k has at least 128 columns
    const Cut d = cut_for<MODE, 1, 2, 2, 2>(M, N, K, 750);
    if (d.cost < best.cut.cost) best = {2, d};
  }
  return best;
}
template <Mode MODE>
void product(const TileArgs& a, int gelu, hipStream_t st) {
  const Choice c = choose<MODE>(a.M, a.N, a.K);
  if (c.tile == 0)
    tile_launch<MODE, 4, 2, 2, 4>(a, c.cut, gelu, st);
  else if (c.tile == 1)
    tile_launch<MODE, 2, 2, 2, 2>(a, c.cut, gelu, st);
  else if constexpr (MODE != kWeights)
    tile_launch<MODE, 1, 2, 2, 2>(a, c.cut, gelu, st);
}

template <int FM, int GM, int WM, int WN>
void gradients_launch(const TileArgs& in, const Cut& ci, const TileArgs& weights, const Cut& cw, hipStream_t st) {
  const TileArgs a = with_cut(in, ci), b = with_cut(weights, cw);
  const int first = grid_of<kInput, FM, 2, WM, WN>(ci), grid = first + grid_of<kWeights, GM, 2, WM, WN>(cw);
  if (a.K % 64 != 0 || b.K % 64 != 0)
    gradients_kernel<FM, 2, GM, WM, WN, true><<<grid, 64 * WM * WN, 0, st>>>(a, b, first);
  else
    gradients_kernel<FM, 2, GM, WM, WN, false><<<grid, 64 * WM * WN, 0, st>>>(a, b, first);
  finish<kInput, FM, 2, WM, WN, false>(a, st);
  finish<kWeights, GM, 2, WM, WN, false>(b, st);
}
// Both products in one launch where their tiles have as many waves, else one after the other.
void gradients(const TileArgs& in, const TileArgs& weights, hipStream_t st) {
  const Choice i = choose<kInput>(in.M, in.N, in.K), w = choose<kWeights>(weights.M, weights.N, weights.K);
  if (i.tile == 0 && w.tile == 0)
    gradients_launch<4, 4, 2, 4>(in, i.cut, weights, w.cut, st);
  else if (i.tile == 1 && w.tile == 1)
    gradients_launch<2, 2, 2, 2>(in, i.cut, weights, w.cut, st);
  else if (i.tile == 2 && w.tile == 1)
    gradients_launch<1, 2, 2, 2>(in, i.cut, weights, w.cut, st);
  else {
    product<kInput>(in, 0, st);
    product<kWeights>(weights, 0, st);
  }
}

// ------------------------------------------------------------------ few tokens
// Up to 16 tokens: the weights' stream is all there is. A workgroup takes 16 columns of h,
// its 8 waves 128 values of k in turn, straight into registers (16 rows of w_gate, of
// w_up and the tokens, 256 bytes of a row at a time), and the waves' sums are added
// through LDS in their order: no second kernel. MFMA rows are the weights', columns the
// tokens.
// 5120 x 2560, 1 token 13 us (52 MB of weights; by tiles, whose cut needs a second kernel, 20),
// 16 tokens 16 us. Every workgroup reads all tokens, so wide outputs of many tokens go to
// the tiles: 5120 x 10240, 1 token 37 us (39), 16 tokens 44 us (39).
constexpr int kFewTokens = 16, kFewWaves = 8;
bool few_tokens(int T, int F) { return T <= kFewTokens && (int64_t)T * F <= 81920; }

template <bool GELU>
__global__ __launch_bounds__(64 * kFewWaves) void gated_few_kernel(GatedArgs p) {
  __shared__ f32x4 sums[kFewWaves][2][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int f0 = blockIdx.x * 16;
  const size_t row = (size_t)min(f0 + l, p.F - 1) * p.H + g * 8;
  const uint16_t *gr = p.wg + row, *ur = p.wu + row, *xr = p.x + (size_t)min(l, p.T - 1) * p.H + g * 8;
  f32x4 gate{}, up{};
  auto group = [&](int k0, auto end) {
    u32x4 x[4], a[4], b[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = k0 + s * 32;
      const bool in = !decltype(end)::value || k + g * 8 < p.H;  // H is a multiple of 8
      a[s] = ld16(in ? (const void*)(gr + k) : (const void*)kZeros);
      b[s] = ld16(in ? (const void*)(ur + k) : (const void*)kZeros);
      x[s] = ld16(in ? (const void*)(xr + k) : (const void*)kZeros);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      gate = mfma_bf16(as_bf16x8(a[s]), as_bf16x8(x[s]), gate);
      up = mfma_bf16(as_bf16x8(b[s]), as_bf16x8(x[s]), up);
    }
  };
  int k0 = wave * 128;
  for (; k0 + 128 <= p.H; k0 += kFewWaves * 128) group(k0, std::false_type{});
  if (k0 < p.H) group(k0, std::true_type{});
  sums[wave][0][lane] = gate;
  sums[wave][1][lane] = up;
  __syncthreads();
  // lane (token l, columns 4 g .. + 3)
  if (wave > 0) return;
#pragma unroll
  for (int w = 1; w < kFewWaves; ++w) {
    gate += sums[w][0][lane];
    up += sums[w][1][lane];
  }
  const int f = f0 + 4 * g;
  if (l >= p.T || f >= p.F) return;
  const size_t at = (size_t)l * p.F + f;
  auto add = [&](const uint16_t* from, f32x4& to) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(from + at);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      to[2 * e] += __uint_as_float(v[e] << 16);
      to[2 * e + 1] += __uint_as_float(v[e] & 0xffff0000u);
    }
  };
  auto put = [&](uint16_t* to, const f32x4& v) {
    *reinterpret_cast<u32x2*>(to + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  };
  if (p.add_gate) add(p.add_gate, gate);
  if (p.add_up) add(p.add_up, up);
  f32x4 h;
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = activation<GELU>(gate[e]) * up[e];
  put(p.h, h);
  auto keep = [&](void* to, const f32x4& v) {
    if (p.pre_f32)
      *reinterpret_cast<f32x4*>((float*)to + at) = v;
    else
      put((uint16_t*)to, v);
  };
  if (p.gate) keep(p.gate, gate);
  if (p.up) keep(p.up, up);
}

// d_up = dh act(gate), d_gate = dh up act'(gate), 8 values a thread. Rounded to bf16,
// which is their type as outputs and as operands of the products: dx and the weights' gradients
// are then 0.0023 of their norm off, 0.0017 of it by their own rounding. (Two bf16 parts of each
// would double the products' 1.3 ms.) Bound by memory: 4096 x 10240 64 to 78 us, 420 MB at 5.4 to
// 6.5 TB/s; from fp32 gate and up 104 us, 587 MB. As the products' own operands,
// each of their tiles would compute its part again: 20 times with 5120 columns of x.
// F32: gate and up are fp32. In bf16 they are 2^-8 off, and with them d by 2^-8 |gate act''|, which near
// a zero of d is all of it.
template <bool GELU, bool F32>
__global__ __launch_bounds__(256) void gated_grad_kernel(GatedBwdArgs p) {
  const int64_t n8 = (int64_t)p.T * p.F / 8, stride = (int64_t)gridDim.x * 256;
  constexpr int B = F32 ? 4 : 2, L = F32 ? 2 : 1;  // bytes of a value, loads of 8 of them
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += stride) {
    const u32x4 dh = ld16(p.dh + i * 8);
    u32x4 g[L], u[L];
#pragma unroll
    for (int k = 0; k < L; ++k) {
      g[k] = ld16((const uint8_t*)p.gate + i * (8 * B) + k * 16);
      u[k] = ld16((const uint8_t*)p.up + i * (8 * B) + k * 16);
    }
    u32x4 dg, du;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float a[2], b[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        auto half = [&](uint32_t v) { return __uint_as_float(e ? v & 0xffff0000u : v << 16); };
        auto pre = [&](const u32x4 (&v)[L]) {
          return F32 ? __uint_as_float(v[q / 2 * (L - 1)][q % 2 * 2 + e]) : half(v[0][q]);
        };
        float d;
        const float f = activation<GELU>(pre(g), d), dhv = half(dh[q]);
        a[e] = dhv * pre(u) * d;
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

size_t gated_workspace_bytes(int T, int H, int F) {
  return few_tokens(T, F) ? 0 : choose<kGated>(T, F, H).part_bytes();
}

hipError_t launch_gated_linear(const GatedArgs& a, int gelu, hipStream_t st) {
  if (few_tokens(a.T, a.F)) {
    const int grid = (a.F + 15) / 16;
    if (gelu)
      gated_few_kernel<true><<<grid, 64 * kFewWaves, 0, st>>>(a);
    else
      gated_few_kernel<false><<<grid, 64 * kFewWaves, 0, st>>>(a);
    return hipGetLastError();
  }
  TileArgs t{};
  t.x[0] = (const uint8_t*)a.x;
  t.w[0] = (const uint8_t*)a.wg;
  t.w[1] = (const uint8_t*)a.wu;
  t.ldx = t.ldw = 2 * (int64_t)a.H;
  t.M = a.T;
  t.N = a.F;
  t.K = a.H;
  t.add_gate = a.add_gate;
  t.add_up = a.add_up;
  t.out[0] = a.h;
  t.pre[0] = a.gate;
  t.pre[1] = a.up;
  t.pre_f32 = a.pre_f32;
  t.part = a.part;
  product<kGated>(t, gelu, st);
  return hipGetLastError();
}

// dx's parts, then the weights'
size_t gated_bwd_workspace_bytes(int T, int H, int F) {
  return choose<kInput>(T, H, F).part_bytes() + choose<kWeights>(F, H, T).part_bytes();
}

hipError_t launch_gated_linear_backward(const GatedBwdArgs& a, int gelu, hipStream_t st) {
  const int64_t n8 = (int64_t)a.T * a.F / 8;
  const unsigned grid = (unsigned)std::min<int64_t>((n8 + 255) / 256, 1 << 20);
  auto go = [&](auto gc) {
    constexpr bool G = decltype(gc)::value;
    if (a.pre_f32)
      gated_grad_kernel<G, true><<<grid, 256, 0, st>>>(a);
    else
      gated_grad_kernel<G, false><<<grid, 256, 0, st>>>(a);
  };
  if (gelu)
    go(std::true_type{});
  else
    go(std::false_type{});
  TileArgs in{};
  in.x[0] = (const uint8_t*)a.d_gate;
  in.x[1] = (const uint8_t*)a.d_up;
  in.ldx = 2 * (int64_t)a.F;
  in.ldw = 2 * (int64_t)a.H;
  in.N = a.H;
  TileArgs weights = in;
  in.w[0] = (const uint8_t*)a.wg;
  in.w[1] = (const uint8_t*)a.wu;
  in.M = a.T;
  in.K = a.F;
  in.out[0] = a.dx;
  in.part = a.part;
  weights.w[0] = weights.w[1] = (const uint8_t*)a.x;
  weights.M = a.F;
  weights.K = a.T;
  weights.out[0] = a.d_wg;
  weights.out[1] = a.d_wu;
  weights.part = a.part + choose<kInput>(a.T, a.H, a.F).part_bytes() / sizeof(float);
  if (a.dx && a.d_wg)
    gradients(in, weights, st);
  else if (a.dx)
    product<kInput>(in, 0, st);
  else if (a.d_wg)
    product<kWeights>(weights, 0, st);
  return hipGetLastError();
}

}  // namespace beam
