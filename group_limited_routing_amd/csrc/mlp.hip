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

// ------------------------------------------------------------------ tiles
// One kernel for the three products, out[m, n] = sum over k of x[m, k] w[n, k], whose
// operands lie in memory as rows of k ("along") or with a row for each k ("across"):
//   kGated    x [T, H] along, the rows of w_gate and w_up along, 32 of each in turn, so
//             that a wave holds gate and up of the same columns: the activation and the
//             product are its epilogue.
//   kInput    d_gate along and w_gate across, then d_up and w_up: one sum over 2 F.
//   kWeights  d_gate (or d_up) across, x across: a sum over the tokens.
enum Mode { kGated, kInput, kWeights };

struct TileArgs {
  const uint8_t* x[2];
  const uint8_t* w[2];
  int64_t ldx, ldw;  // bytes of a row in memory
  int M, N, K;       // N: columns of the output; K: of one of the two sums of kInput
  const uint16_t* add_gate;
  const uint16_t* add_up;
  uint16_t* out[3];  // h, gate, up; or the output of each of two products
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
// straight into LDS (16 bytes a lane) through a ring of NS stages of 32 values of k. A
// workgroup stays for many items of work, and its loads run ahead into the next one, so
// that neither the first loads of an item nor its output stop the ring.
//
// LDS of a stage. Along: 64 bytes a row, swizzled as tile.h says. Across: a row of the
// tile's width for each k; the 64-byte chunk c (32 columns, one fragment) of row k
// stands at c ^ (k & 3), so that the 4 rows of a transposing read cover all banks.
template <Mode MODE, int FM, int FN, int WM, int WN>
struct Tile {
  static constexpr int WAVES = WM * WN, BM = 32 * FM * WM, BN = 32 * FN * WN;
  static constexpr int KS = 64;  // values of k in a stage
  static constexpr int X_BYTES = BM * 2 * KS, STAGE = (BM + BN) * 2 * KS;
  static constexpr int NS = BM == 64 ? 3 : 2;  // stages: what 160 KB hold
  static constexpr int COLS = MODE == kGated ? FN * 16 : FN * 32;  // of the output, a wave's
  static constexpr int TN = COLS * WN;                             // and the tile's
  static constexpr int STAGING = 32 * COLS * 2;                    // 32 rows of a wave's output
  static constexpr int LDS = NS * STAGE + WAVES * STAGING;
  static constexpr int PER_CU = LDS <= 80 * 1024 ? 2 : 1;          // workgroups
};

template <Mode MODE, int FM, int FN, int WM, int WN, bool RAGGED, bool GELU>
__global__ __launch_bounds__(64 * WM * WN)
    __attribute__((amdgpu_waves_per_eu(Tile<MODE, FM, FN, WM, WN>::PER_CU * WM * WN / 4)))
void tile_kernel(TileArgs p) {
  using S = Tile<MODE, FM, FN, WM, WN>;
  constexpr bool XA = MODE == kWeights, WA = MODE != kGated;  // across
  constexpr int BM = S::BM, BN = S::BN, NS = S::NS, WAVES = S::WAVES, TN = S::TN;
  constexpr int KS = S::KS, ROW = 2 * KS, HALVES = KS / 16;
  constexpr int XU = S::X_BYTES / 1024, WU = BN * ROW / 1024, PER = (XU + WU) / WAVES;
  static_assert(XU % WAVES == 0 && WU % WAVES == 0, "a load is of one operand for every wave");
  static_assert((!XA || BM >= 128) && (!WA || BN >= 128), "four 64-byte chunks in a row of k");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::LDS];

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
  int load_item = blockIdx.x, load_k, load_end;  // the stage that the next loads are of
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
    if (load_item + (int)gridDim.x < p.items) load_item += gridDim.x;
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

  // Operand offsets in a stage. Along: fragment i is 32 rows on, chunk 2 j + h of half j.
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

  // A stage is two halves of 16 values of k, each FM x FN instructions. Beside every
  // instruction goes at most a read or two of LDS and a load, so that neither queue
  // holds the wave back: the fragments of half 1 are read during half 0, those of the next
  // stage's half 0 during half 1. The barrier between the halves says that every wave has
  // read all of stage s, whose slot stage s + NS refills from then on, and that stage s + 1
  // has landed.
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
  // loads of a stage that go beside half 1 of the stage NS before it; the others beside
  // half 0 of the next one
  constexpr int TURN = (HALVES - 1) * SLOTS, WINDOW = HALVES * SLOTS * (MODE == kWeights ? 5 : 3) / 8;
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
  for (int item = blockIdx.x; item < p.items; item += gridDim.x) {
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
        acc[I][N] = mfma32(wr[J % 2][N], xr[J % 2][I], acc[I][N]);
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
        auto add = [&](const uint16_t* from, auto which) {  // onto gate (0) or up (1)
          constexpr int W = decltype(which)::value;
#pragma unroll
          for (int g = 0; g < 32 / RS; ++g) {
            const int row = g * RS + row_l;
            if (mb + row < p.M && col_in)
              st16(chunk(row, ch_l), ld16(from + (size_t)(mb + row) * p.N + c0 + ch_l * 8));
          }
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
        if (p.add_gate) add(p.add_gate, j0);
        if (p.add_up) add(p.add_up, j1);
        put(p.out[0], [&](int j, int i) { return activation<GELU>(acc[I][2 * j][i]) * acc[I][2 * j + 1][i]; });
        if (p.out[1]) put(p.out[1], [&](int j, int i) { return acc[I][2 * j][i]; });
        if (p.out[2]) put(p.out[2], [&](int j, int i) { return acc[I][2 * j + 1][i]; });
      } else {
        put(p.out[t.problem], [&](int j, int i) { return acc[I][j][i]; });
      }
    });
  }
  wait_vmcnt<0>();  // no load is in flight when the workgroup's LDS is given away
}

// The tiles that were cut along k: the sum of a tile's parts, in their order, and what
// tile_kernel does with a sum. 8 columns a thread.
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
    if (p.out[1]) put8(p.out[1] + to, g);
    if (p.out[2]) put8(p.out[2] + to, u);
  } else {
    sum8(c, g);
    put8((problem ? p.out[1] : p.out[0]) + to, g);
  }
}

// How a product is cut. Rounds of 256 PER_CU workgroups take whole tiles; what is left
// would keep a part of the chip busy for a whole round, so it is cut along k into as many
// parts as make it cheapest. Costs in ns: a stage of a full round, the parts' way through memory, and
// the second kernel.
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

template <Mode MODE, int FM, int FN, int WM, int WN>
void tile_launch(const TileArgs& a, const Cut& c, int gelu, hipStream_t st) {
  using S = Tile<MODE, FM, FN, WM, WN>;
  TileArgs t = a;
  t.whole = c.whole;
  t.items = c.items;
  t.splits = c.splits;
  const int grid = c.items < 256 * S::PER_CU ? c.items : 256 * S::PER_CU;
  auto go = [&](auto rc, auto gc) {
    constexpr bool R = decltype(rc)::value, G = decltype(gc)::value;
    tile_kernel<MODE, FM, FN, WM, WN, R, G><<<grid, 64 * S::WAVES, 0, st>>>(t);
    if (c.splits > 1)
      finish_kernel<MODE, S::BM, S::BN, G>
          <<<dim3((c.items - c.whole) / c.splits, (std::min(S::BM, a.M) * S::TN + 511) / 512), 64, 0, st>>>(t);
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
template <Mode MODE>
size_t product(const TileArgs* a, int M, int N, int K, int gelu, hipStream_t st) {
  Cut c[3] = {cut_for<MODE, 4, 2, 2, 4>(M, N, K, 1650), cut_for<MODE, 2, 2, 2, 2>(M, N, K, 1000), {}};
  c[2].cost = INT64_MAX;
  if constexpr (MODE != kWeights) c[2] = cut_for<MODE, 1, 2, 2, 2>(M, N, K, 800);
  int best = 0;
  for (int i = 1; i < 3; ++i)
    if (c[i].cost < c[best].cost) best = i;
  if (!a) {
    const int floats[3] = {256 * 256, 128 * 128, 64 * 128};
    return c[best].splits > 1 ? (size_t)(c[best].items - c[best].whole) * floats[best] * sizeof(float) : 0;
  }
  if (best == 0)
    tile_launch<MODE, 4, 2, 2, 4>(*a, c[0], gelu, st);
  else if (best == 1)
    tile_launch<MODE, 2, 2, 2, 2>(*a, c[1], gelu, st);
  else if constexpr (MODE != kWeights)
    tile_launch<MODE, 1, 2, 2, 2>(*a, c[2], gelu, st);
  return 0;
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

size_t gated_workspace_bytes(int T, int H, int F) { return product<kGated>(nullptr, T, F, H, 0, nullptr); }

hipError_t launch_gated_linear(const GatedArgs& a, int gelu, hipStream_t st) {
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
  t.out[1] = a.gate;
  t.out[2] = a.up;
  t.part = a.part;
  product<kGated>(&t, a.T, a.F, a.H, gelu, st);
  return hipGetLastError();
}

size_t gated_bwd_workspace_bytes(int T, int H, int F) {
  const size_t in = product<kInput>(nullptr, T, H, F, 0, nullptr), w = product<kWeights>(nullptr, F, H, T, 0, nullptr);
  return in > w ? in : w;
}

hipError_t launch_gated_linear_backward(const GatedBwdArgs& a, int gelu, hipStream_t st) {
  const int64_t n8 = (int64_t)a.T * a.F / 8;
  const unsigned grid = (unsigned)((n8 + 255) / 256 < (1 << 20) ? (n8 + 255) / 256 : 1 << 20);
  if (gelu)
    gated_grad_kernel<true><<<grid, 256, 0, st>>>(a);
  else
    gated_grad_kernel<false><<<grid, 256, 0, st>>>(a);
  TileArgs t{};
  t.x[0] = (const uint8_t*)a.d_gate;
  t.x[1] = (const uint8_t*)a.d_up;
  t.ldx = 2 * (int64_t)a.F;
  t.ldw = 2 * (int64_t)a.H;
  t.N = a.H;
  t.part = a.part;
  if (a.dx) {
    t.w[0] = (const uint8_t*)a.wg;
    t.w[1] = (const uint8_t*)a.wu;
    t.M = a.T;
    t.K = a.F;
    t.out[0] = a.dx;
    product<kInput>(&t, a.T, a.H, a.F, 0, st);
  }
  if (a.d_wg) {
    t.w[0] = t.w[1] = (const uint8_t*)a.x;
    t.M = a.F;
    t.K = a.T;
    t.out[0] = a.d_wg;
    t.out[1] = a.d_wu;
    product<kWeights>(&t, a.F, a.H, a.T, 0, st);
  }
  return hipGetLastError();
}

}  // namespace beam
