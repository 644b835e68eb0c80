// Products of bf16 or int8 operands for many rows: 256- and 128-wide tiles of eight waves that
// take turns at the matrix cores, fed straight into LDS (int8.hip, ffn.hip).
//
// One step is 128 bytes of K: 64 bf16 values or 128 codes. Both types' MFMAs (16 x 16 x 32 bf16,
// 16 x 16 x 64 int8) take 16 bytes a lane of either operand, so a step is two of them on each pair
// of blocks, whatever the type. An operand lies in LDS as
//  * K-contiguous rows of 128 bytes (frag_at): lane l takes chunks l / 16 and 4 + l / 16 of row
//    l % 16, the first in the step's first MFMA and the other in the second; or
//  * K-major (bf16: 64 rows of K as they lie in memory, column groups permuted by kmajor_swz), read
//    with the transposing LDS read, which gives the same k in the same places.
//
// Waves w and w + 4 share a SIMD and run a phase apart: the one multiplies while the other reads its
// fragments and sends out loads, and a barrier ends each phase. A step is one turn of reading and one
// of multiplying (phase 2k reads, 2k + 1 multiplies for waves 0..3, one later for waves 4..7), or in
// the 256 x 256 tiles two:
//     phase        4k        4k + 1    4k + 2    4k + 3    4k + 4
//     waves 0..3   read k.0  mfma k.0  read k.1  mfma k.1  read (k+1).0
//     waves 4..7   mfma ..   read k.0  mfma k.0  read k.1  mfma k.1
// Loads go out as early as their place is free; half stages refilled one by one instead of whole stages
// took the forward of 2048 x 7168 x 2048 from 223 us to 157:
//  * With NS = 3 stages and more, step k - 1's stage is read for the last time in phase 2k - 1, and a
//    wave fills it with step k + NS - 1 in its phase read k.
//  * The 256 x 256 tiles have two stages, each in two parts. Part 0 is what read k.0 reads: all of the
//    columns and half of the rows' blocks, or (rows K-major) the first half of K of both. Once
//    everyone has read it, it takes step k + 2's, in phase read k.1; part 1 takes step k + 1's in
//    read k.0. So every load has a whole step to arrive, with 64 KB on their way throughout.
// At the end of a reading phase a wave waits for its own loads of what the next one reads, a barrier
// or more before anyone reads it; those issued since stay on their way. Loads past the last step
// read that one again into a place that nobody reads.
//
// LDS: ten units of 16 KB, 128 rows of 128 bytes or 32 rows of K of 256 values. A 256-wide operand
// takes two: K-contiguous, the first half of each wave's blocks and the second; K-major, the halves
// of the step. The units are distinct arrays and the loop is unrolled over the stages, so that the
// compiler sees which loads and reads meet, and does not wait for every load before each read.
//
// A step takes 1.35 us in 256 x 256 tiles, 0.95 in 256 x 128 and 0.67 in 128 x 128 with the card full
// of them, each some 12.5 TB/s of loads. Over 128 steps and more of the first the MFMAs are busy 86 to
// 91% of the time, and the clock, 2.4 GHz at first, falls as the card's power allows: 2.0 GHz after 0.1
// ms of 256 int8 tiles, 1.8 after 0.2, 1.45 after 0.45. Four waves of 128 x 128, which read a third less
// from LDS, took 1.34 us, panels that all lie in L2 1.32, and a step without its loads, at a higher
// clock, 0.9 to 0.98. No change: K begun elsewhere in each tile, a later start of every second CU.
#pragma once

#include "dma.h"
#include "tiles8.h"

namespace moe {
namespace {

typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;

// Two values rounded to nearest even, NaN kept.
MOE_DEV uint32_t to_bf2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

struct Bf16 {
  using Acc = f32x4;
  static constexpr int kStepK = 64;  // values of K a step
  static MOE_DEV Acc zero() { return f32x4{0.f, 0.f, 0.f, 0.f}; }
  // columns first: lane l gets row l % 16, columns 4 (l / 16) .. + 3
  static MOE_DEV Acc mma(const i32x4& b, const i32x4& a, const Acc& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b),
                                                   __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
  }
};
struct Int8 {
  using Acc = i32x4;
  static constexpr int kStepK = 128;
  static MOE_DEV Acc zero() { return i32x4{0, 0, 0, 0}; }
  static MOE_DEV Acc mma(const i32x4& b, const i32x4& a, const Acc& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(b, a, c, 0, 0, 0);
  }
};

__shared__ __align__(1024) uint8_t prod_u0[16384];
__shared__ __align__(1024) uint8_t prod_u1[16384];
__shared__ __align__(1024) uint8_t prod_u2[16384];
__shared__ __align__(1024) uint8_t prod_u3[16384];
__shared__ __align__(1024) uint8_t prod_u4[16384];
__shared__ __align__(1024) uint8_t prod_u5[16384];
__shared__ __align__(1024) uint8_t prod_u6[16384];
__shared__ __align__(1024) uint8_t prod_u7[16384];
__shared__ __align__(1024) uint8_t prod_u8[16384];
__shared__ __align__(1024) uint8_t prod_u9[16384];
template <int U>
MOE_DEV uint8_t* prod_unit() {
  if constexpr (U == 0) return prod_u0;
  else if constexpr (U == 1) return prod_u1;
  else if constexpr (U == 2) return prod_u2;
  else if constexpr (U == 3) return prod_u3;
  else if constexpr (U == 4) return prod_u4;
  else if constexpr (U == 5) return prod_u5;
  else if constexpr (U == 6) return prod_u6;
  else if constexpr (U == 7) return prod_u7;
  else if constexpr (U == 8) return prod_u8;
  else return prod_u9;
}

template <int I>
struct Int {
  static constexpr int value = I;
};
// fn(Int<0>) .. fn(Int<N - 1>)
template <int N, int I = 0, class Fn>
MOE_DEV void each(Fn fn) {
  if constexpr (I < N) {
    fn(Int<I>());
    each<N, I + 1>(fn);
  }
}

MOE_DEV i32x4 lds_chunk(const uint8_t* p) { return *reinterpret_cast<const i32x4*>(p); }
// kmajor_frag_dma for stages W values wide
template <int W>
MOE_DEV i32x4 kmajor_chunk(const uint8_t* st, int base, int kb, int lane) {
  const uint16_t* s = reinterpret_cast<const uint16_t*>(st);
  const int g = lane / 16, q = lane % 16, kr = 8 * g + q / 4;
  const int n = (base ^ kmajor_swz(kr)) + 4 * (q % 4);
  const s16x4 a = lds_read_tr16_scoped(s + (kb + kr) * W + n);
  const s16x4 b = lds_read_tr16_scoped(s + (kb + kr + 4) * W + n);
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  const s16x8 v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(i32x4, v);
}

// AKM, BKM: that operand is K-major. GATED: columns 0 .. BN / 2 - 1 of the tile are the gate's, the
// rest the matching ones of the up projection, and a wave's blocks half of each.
template <class El, int BM_, int BN_, bool AKM = false, bool BKM = false, bool GATED = false>
struct Tile8 {
  using Acc = typename El::Acc;
  static constexpr int BM = BM_, BN = BN_;
  static constexpr int WM = BM == 256 && BN == 128 ? 4 : 2, WN = 8 / WM;  // waves
  static constexpr int MB = BM / 16 / WM, NB = BN / 16 / WN;              // blocks a wave
  static constexpr int AU = BM / 128, BU = BN / 128, NS = 10 / (AU + BU);  // units, stages
  static constexpr bool kTwo = NS == 2;            // two turns a step
  static constexpr bool kByK = AKM;                // which split K, not the rows
  static constexpr int AJ = 2 * AU, BJ = 2 * BU;   // loads a wave and step
  static constexpr int kBehind = kTwo ? AJ + BJ : (NS - 2) * (AJ + BJ);  // loads not waited for
  static constexpr int kWait = 0x0070 | kBehind;   // lgkmcnt(0) too
  static_assert(kBehind < 16, "the low bits of vmcnt");
  static_assert(El::kStepK == 64 || (!AKM && !BKM), "transposing reads are 16-bit");
  static_assert(!AKM || BKM, "parts by K need both K-major");

  struct Src {  // a tile's operands, from its first row (column) on
    __amdgpu_buffer_rsrc_t a, b;
  };
  Src cur, nxt;
  uint32_t ao[AJ], bo[BJ], astep, bstep;  // a lane's places in any tile, and a step's bytes
  int nK, lane, wave, wm, wn;
  FragAt f;
  Acc acc[MB][NB];

  MOE_DEV void begin() {
    lane = threadIdx.x % kWave;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    wm = wave / WN;
    wn = wave % WN;
    f = frag_at(lane);
  }
  // The KB of an operand's units that a wave's load j fills: load j goes to unit j / 2.
  MOE_DEV int kb_of(int j) const { return 16 * (j / 2) + 2 * wave + j % 2; }
  // Where row L of an operand's units lies in the tile: a unit has the first (second) half of each
  // wave's B blocks.
  template <int U, int B>
  static MOE_DEV int tile_row(int L) {
    return U == 1 ? L : L % 128 / (B * 8) * (B * 16) + L / 128 * (B * 8) + L % (B * 8);
  }
  // Where a tile's rows lie, `pitch` bytes apart; B's (columns of the product) i-th in row row(i)
  // behind the first. K-major: `pitch` bytes from one row of K to the next. What lies past the end of
  // an operand reads as zeros, and what lies past a tile's own rows or columns goes into sums that are
  // not stored.
  MOE_DEV void a_rows(uint32_t pitch) {
    astep = 128;
#pragma unroll
    for (int j = 0; j < AJ; ++j)
      ao[j] = (uint32_t)tile_row<AU, MB>(kb_of(j) * 8 + lane / 8) * pitch + lds_piece(lane);
  }
  template <class Row>
  MOE_DEV void b_rows(uint32_t pitch, Row row) {
    bstep = 128;
#pragma unroll
    for (int j = 0; j < BJ; ++j) {
      const int L = kb_of(j) * 8 + lane / 8;  // a gated tile's: gate rows, then up rows
      bo[j] = (uint32_t)row(GATED ? L : tile_row<BU, NB>(L)) * pitch + lds_piece(lane);
    }
  }
  template <int W, int J>
  MOE_DEV void k_major(uint32_t (&off)[J], uint32_t pitch) {
    constexpr int R = 512 / W;  // rows of K a load
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int kr = kb_of(j) * R + lane / (W / 8);
      off[j] = (uint32_t)kr * pitch + 2u * ((lane % (W / 8) * 8) ^ kmajor_swz(kr));
    }
  }
  MOE_DEV void a_cols(uint32_t pitch) {
    astep = 64 * pitch;
    k_major<BM>(ao, pitch);
  }
  MOE_DEV void b_cols(uint32_t pitch) {
    bstep = 64 * pitch;
    k_major<BN>(bo, pitch);
  }
  // The next tile: its first row and column, and the bytes of each operand from there on that may be
  // read (rows of A past the last one's end are another tile's, or nobody's).
  MOE_DEV void next(const void* a, uint32_t a_bytes, const void* b, uint32_t b_bytes) {
    nxt = {raw_rsrc(a, a_bytes), raw_rsrc(b, b_bytes)};
  }

  // Part P of step kb into stage S (P = 2: all of it). Past the tile's end FLOW goes on with the
  // next tile's steps; else the last one is read again, into a place that nobody reads.
  template <bool FLOW, int S, int P>
  MOE_DEV void issue(int kb) {
    if (!FLOW || kb < nK) issue_from<S, P>(cur, min(kb, nK - 1));
    else issue_from<S, P>(nxt, kb - nK);
  }
  template <int S, int P>
  MOE_DEV void issue_from(const Src& o, int kb) {
    // the range of a resource is checked against the lane's offset alone
    const uint32_t sa = AKM ? 0u : (uint32_t)kb * 128, va = AKM ? (uint32_t)kb * astep : 0u;
    const uint32_t sb = BKM ? 0u : (uint32_t)kb * 128, vb = BKM ? (uint32_t)kb * bstep : 0u;
    constexpr int U = S * (AU + BU);
    auto load_a = [&](auto j) {
      constexpr int J = decltype(j)::value;
      if constexpr (P == 2 || P == J / 2)
        load_lds16(o.a, ao[J] + va, sa, prod_unit<U + J / 2>() + (2 * wave + J % 2) * 1024);
    };
    auto load_b = [&](auto j) {
      constexpr int J = decltype(j)::value;
      if constexpr (P == 2 || (kByK ? P == J / 2 : P == 0))
        load_lds16(o.b, bo[J] + vb, sb, prod_unit<U + AU + J / 2>() + (2 * wave + J % 2) * 1024);
    };
    load_b(Int<0>());
    load_b(Int<1>());
    if constexpr (BJ == 4) {
      load_b(Int<2>());
      load_b(Int<3>());
    }
    load_a(Int<0>());
    load_a(Int<1>());
    if constexpr (AJ == 4) {
      load_a(Int<2>());
      load_a(Int<3>());
    }
  }
  // half h of row block mb, of column block nb
  template <int S, int M, int Hh>
  MOE_DEV i32x4 a_frag() const {
    constexpr int U = S * (AU + BU);
    if constexpr (AKM && AU == 2)
      return kmajor_chunk<256>(prod_unit<U + Hh>(), (wm * MB + M) * 16, 0, lane);
    else if constexpr (AKM)
      return kmajor_chunk<128>(prod_unit<U>(), (wm * MB + M) * 16, 32 * Hh, lane);
    else if constexpr (AU == 2)
      return lds_chunk(prod_unit<U + M / (MB / 2)>() + (wm * MB * 8 + M % (MB / 2) * 16) * 128 +
                       (Hh ? f.hi : f.lo));
    else
      return lds_chunk(prod_unit<U>() + (wm * MB + M) * 2048 + (Hh ? f.hi : f.lo));
  }
  template <int S, int N, int Hh>
  MOE_DEV i32x4 b_frag() const {
    constexpr int U = S * (AU + BU) + AU;
    if constexpr (BKM && BU == 2)
      return kmajor_chunk<256>(prod_unit<U + Hh>(), (wn * NB + N) * 16, 0, lane);
    else if constexpr (BKM)
      return kmajor_chunk<128>(prod_unit<U>(), (wn * NB + N) * 16, 32 * Hh, lane);
    else if constexpr (BU == 2)
      return lds_chunk(prod_unit<U + N / (NB / 2)>() + (wn * NB * 8 + N % (NB / 2) * 16) * 128 +
                       (Hh ? f.hi : f.lo));
    else if constexpr (GATED)
      return lds_chunk(prod_unit<U>() + (N / (NB / 2) * 64 + wn * NB * 8 + N % (NB / 2) * 16) * 128 +
                       (Hh ? f.hi : f.lo));
    else
      return lds_chunk(prod_unit<U>() + (wn * NB + N) * 2048 + (Hh ? f.hi : f.lo));
  }
  MOE_DEV void phase_end() const {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  }
  // halves H0 .. H0 + HN - 1 of row blocks M0 .. M0 + MN - 1, and of all column blocks
  template <int S, int M0, int MN, int H0, int HN>
  MOE_DEV void read_a(i32x4 (&af)[HN][MN]) const {
    each<HN * MN>([&](auto i) {
      constexpr int I = decltype(i)::value;
      af[I / MN][I % MN] = a_frag<S, M0 + I % MN, H0 + I / MN>();
    });
  }
  template <int S, int H0, int HN>
  MOE_DEV void read_b(i32x4 (&bf)[HN][NB]) const {
    each<HN * NB>([&](auto i) {
      constexpr int I = decltype(i)::value;
      bf[I / NB][I % NB] = b_frag<S, I % NB, H0 + I / NB>();
    });
  }
  // the end of a reading phase, the multiplication, and its end
  template <int M0, int MN, int HN>
  MOE_DEV void multiply(const i32x4 (&bf)[HN][NB], const i32x4 (&af)[HN][MN]) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(kWait);
    phase_end();
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int h = 0; h < HN; ++h)
#pragma unroll
      for (int mb = 0; mb < MN; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          acc[M0 + mb][nb] = El::mma(bf[h][nb], af[h][mb], acc[M0 + mb][nb]);
    __builtin_amdgcn_s_setprio(0);
    phase_end();
  }
  template <bool FLOW, int S>
  MOE_DEV void step(int kb) {
    if constexpr (!kTwo) {
      i32x4 bf[2][NB], af[2][MB];
      issue<FLOW, (S + NS - 1) % NS, 2>(kb + NS - 1);
      read_b<S, 0, 2>(bf);
      read_a<S, 0, MB, 0, 2>(af);
      multiply<0, MB, 2>(bf, af);
    } else if constexpr (kByK) {
      i32x4 bf[1][NB], af[1][MB];
      issue<FLOW, S ^ 1, 1>(kb + 1);
      read_b<S, 0, 1>(bf);
      read_a<S, 0, MB, 0, 1>(af);
      multiply<0, MB, 1>(bf, af);
      issue<FLOW, S, 0>(kb + 2);
      read_b<S, 1, 1>(bf);
      read_a<S, 0, MB, 1, 1>(af);
      multiply<0, MB, 1>(bf, af);
    } else {
      i32x4 bf[2][NB], af[2][MB / 2];
      issue<FLOW, S ^ 1, 1>(kb + 1);
      read_b<S, 0, 2>(bf);
      read_a<S, 0, MB / 2, 0, 2>(af);
      multiply<0, MB / 2, 2>(bf, af);
      issue<FLOW, S, 0>(kb + 2);
      read_a<S, MB / 2, MB / 2, 0, 2>(af);
      multiply<MB / 2, MB / 2, 2>(bf, af);
    }
  }
  template <bool FLOW, int S, int C>  // steps kb + S, .. while fewer than C and n
  MOE_DEV void steps(int kb, int n) {
    if constexpr (S < C) {
      if (S < n) {
        step<FLOW, S>(kb + S);
        steps<FLOW, S + 1, C>(kb, n);
      }
    }
  }
  template <int S>
  MOE_DEV void fill() {
    if constexpr (S < NS - 1) {
      issue<false, S, 2>(S);
      loads_in_order();
      fill<S + 1>();
    }
  }
  // The next tile becomes the current one, and its first loads go out.
  MOE_DEV void start(int steps_of_k) {
    nK = steps_of_k;
    cur = nxt;
    if constexpr (kTwo) {
      issue<false, 0, 0>(0);
      loads_in_order();
      issue<false, 0, 1>(0);
      loads_in_order();
      issue<false, 1, 0>(1);
    } else {
      fill<0>();
    }
    __builtin_amdgcn_s_waitcnt(kWait);  // what step 0 reads first
    phase_end();
  }
  // The sums over the current tile's steps (one at least). FLOW, for numbers of steps that are a
  // multiple of NS: the next tile's first loads are on their way at the end, as start leaves them.
  template <bool FLOW>
  MOE_DEV void sum() {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = El::zero();
    const bool late = wave >= 4;
    if (late) phase_end();
    int kb = 0;
    if constexpr (FLOW) {
      do {  // at least once: so the compiler knows that what went out before has landed
        steps<true, 0, NS>(kb, NS);
        kb += NS;
      } while (kb < nK);
    } else {
      for (; kb + NS <= nK; kb += NS) steps<false, 0, NS>(kb, NS);
      steps<false, 0, NS - 1>(kb, nK - kb);
    }
    if (!late) phase_end();  // as many barriers for the early waves as for the late ones
    if constexpr (!FLOW) {
      // the loads past the end land before the units are filled again or given back
      __builtin_amdgcn_s_waitcnt(kVm0Lgkm0);
      phase_end();
    } else {
      cur = nxt;
    }
  }
  MOE_DEV void run(int steps_of_k) {
    start(steps_of_k);
    sum<false>();
  }

  MOE_DEV int row_of(int mb) const { return (wm * MB + mb) * 16 + lane % 16; }
};

// Few rows a weight: the weights' stream is what takes the time. Tiles of up to 128 rows and 128 of
// the weights' rows, four waves of 32 of them each; 128 bytes of K a step go straight into LDS, the
// weights SB - 1 steps ahead and the rows one.
//  * 128 rows, three weight stages: 80 KB, two workgroups a CU, 64 KB of weights on their way.
//  * 32 rows, two weight stages: 40 KB, four workgroups a CU with as much on their way.
// A tile's K loop is compiled for 2, 4, 6 and 8 blocks of 16 rows and runs the least that hold its
// rows. Weights that one row tile reads go past the caches (nt) up to 64 rows.
// A wave's loads complete in order; a step issues rows, then weights, so at its top the weight loads
// issued last may be missing if they are a step further ahead. Loads past the last step read it
// again into a stage nobody reads, so the counts hold.
template <int SB>
struct StreamStages {
  uint8_t *a0, *a1, *b0, *b1, *b2;
  template <int S>
  MOE_DEV uint8_t* a() const {
    if constexpr (S == 0) return a0;
    else return a1;
  }
  template <int S>
  MOE_DEV uint8_t* b() const {
    if constexpr (S == 0) return b0;
    else if constexpr (S == 1) return b1;
    else return b2;
  }
};
template <class El, int NMB, int SB, bool GATED>
struct StreamProduct {
  static constexpr int MB = NMB, NB = 2, BN = 128;
  static constexpr int AJ = NMB / 2;  // row loads a wave: 8 rows each
  __amdgpu_buffer_rsrc_t ra, rb;
  uint32_t ao[AJ], bo[4];
  int nK, lane, wn;  // wn: the wave
  FragAt f;
  typename El::Acc acc[NMB][2];

  MOE_DEV void begin() {
    lane = threadIdx.x % kWave;
    wn = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    f = frag_at(lane);
  }
  MOE_DEV void a_rows(const void* base, uint32_t pitch, int rows) {
    ra = buf_rsrc(base);
#pragma unroll
    for (int j = 0; j < AJ; ++j)  // rows past the count read the last one again
      ao[j] = (uint32_t)min(8 * (wn * AJ + j) + lane / 8, rows - 1) * pitch + lds_piece(lane);
  }
  // row(i): where the i-th of the tile's weight rows lies; a gated tile's first half are the gate's
  template <class Row>
  MOE_DEV void b_rows(const void* base, uint32_t pitch, Row row) {
    rb = buf_rsrc(base);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = 8 * (wn * 4 + j) + lane / 8;  // a wave's 32: its own two blocks
      bo[j] = (uint32_t)row(GATED ? j / 2 * 64 + wn * 16 + i % 16 : i) * pitch + lds_piece(lane);
    }
  }
  template <int S>
  MOE_DEV void issue_a(const StreamStages<SB>& L, int kb) {
    const uint32_t step = (uint32_t)min(kb, nK - 1) * 128;
#pragma unroll
    for (int j = 0; j < AJ; ++j)
      load_lds16(ra, ao[j], step, L.template a<S>() + (wn * AJ + j) * 1024);
  }
  template <int S>
  MOE_DEV void issue_b(const StreamStages<SB>& L, int kb) {
    const uint32_t step = (uint32_t)min(kb, nK - 1) * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      load_lds16<NMB <= 4 ? 2 : 0>(rb, bo[j], step, L.template b<S>() + (wn * 4 + j) * 1024);
  }
  template <int S>  // S: the step's number modulo the stages' common cycle
  MOE_DEV void step(const StreamStages<SB>& L, int kb) {
    __builtin_amdgcn_s_waitcnt(SB == 3 ? kVm4Lgkm0 : kVm0Lgkm0);
    __builtin_amdgcn_s_barrier();
    issue_a<(S + 1) % 2>(L, kb + 1);
    loads_in_order();
    issue_b<(S + SB - 1) % SB>(L, kb + SB - 1);
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* A = L.template a<S % 2>();
    const uint8_t* B = L.template b<S % SB>() + wn * 4096;
    const i32x4 b0l = lds_chunk(B + f.lo), b0h = lds_chunk(B + f.hi);
    const i32x4 b1l = lds_chunk(B + 2048 + f.lo), b1h = lds_chunk(B + 2048 + f.hi);
#pragma unroll
    for (int mb = 0; mb < NMB; ++mb) {
      const i32x4 al = lds_chunk(A + mb * 2048 + f.lo), ah = lds_chunk(A + mb * 2048 + f.hi);
      acc[mb][0] = El::mma(b0l, al, acc[mb][0]);
      acc[mb][1] = El::mma(b1l, al, acc[mb][1]);
      acc[mb][0] = El::mma(b0h, ah, acc[mb][0]);
      acc[mb][1] = El::mma(b1h, ah, acc[mb][1]);
    }
  }
  template <int S, int C>  // steps kb + S, .. while fewer than C and n
  MOE_DEV void steps(const StreamStages<SB>& L, int kb, int n) {
    if constexpr (S < C) {
      if (S < n) {
        step<S>(L, kb + S);
        steps<S + 1, C>(L, kb, n);
      }
    }
  }
  MOE_DEV void run(const StreamStages<SB>& L, int steps_of_k) {
    nK = steps_of_k;
#pragma unroll
    for (int i = 0; i < NMB; ++i) acc[i][0] = acc[i][1] = El::zero();
    issue_b<0>(L, 0);
    issue_a<0>(L, 0);
    loads_in_order();
    if constexpr (SB == 3) issue_b<1>(L, 1);
    // whole cycles of the stages, then the rest: a loop left from its middle would hold two sets
    // of accumulators
    constexpr int C = SB == 3 ? 6 : 2;
    int kb = 0;
    for (; kb + C <= nK; kb += C) steps<0, C>(L, kb, C);
    steps<0, C - 1>(L, kb, nK - kb);
    // the loads past the end land before the workgroup gives its LDS back
    __builtin_amdgcn_s_waitcnt(kVm0Lgkm0);
  }
  MOE_DEV int row_of(int mb) const { return mb * 16 + lane % 16; }
};

// A handful of rows and few tiles: a product that reads its weights once, with every CU at it. A
// workgroup takes 16 NNB of the weights' rows and up to 64 rows; its eight waves take the steps of
// K in turn, each straight from memory into registers, U steps on their way, and add up their sums
// through LDS in the waves' order. (One wave a tile, the other kernels' chain of steps, leaves a
// CU with little on its way.) A gated tile's blocks hold 8 gate rows and the 8 up rows that match.
template <class El, int NMB, int NNB, int U>
struct SkinnyProduct {
  using Acc = typename El::Acc;
  __amdgpu_buffer_rsrc_t ra, rb;
  uint32_t ao[NMB], bo[NNB];
  int lane, wave;
  i32x4 a[U][NMB][2], b[U][NNB][2];
  Acc acc[NMB][NNB];

  MOE_DEV void begin() {
    lane = threadIdx.x % kWave;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  }
  MOE_DEV void a_rows(const void* base, uint32_t pitch, int rows) {
    ra = buf_rsrc(base);
#pragma unroll
    for (int mb = 0; mb < NMB; ++mb)  // rows past the count read the last one again
      ao[mb] = (uint32_t)min(mb * 16 + lane % 16, rows - 1) * pitch + 16 * (lane / 16);
  }
  // row(i): where the tile's i-th weight row lies
  template <class Row>
  MOE_DEV void b_rows(const void* base, uint32_t pitch, Row row) {
    rb = buf_rsrc(base);
#pragma unroll
    for (int nb = 0; nb < NNB; ++nb)
      bo[nb] = (uint32_t)row(nb * 16 + lane % 16) * pitch + 16 * (lane / 16);
  }
  template <int AUX>
  static MOE_DEV i32x4 load(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, AUX));
  }
  template <int S>
  MOE_DEV void fetch(int step) {
    const uint32_t at = (uint32_t)step * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int nb = 0; nb < NNB; ++nb)
        b[S][nb][h] = load<2>(rb, bo[nb] + 64 * h, at);  // read once: past the caches
#pragma unroll
      for (int mb = 0; mb < NMB; ++mb) a[S][mb][h] = load<0>(ra, ao[mb] + 64 * h, at);
    }
  }
  template <int S>
  MOE_DEV void multiply() {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int mb = 0; mb < NMB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NNB; ++nb) acc[mb][nb] = El::mma(b[S][nb][h], a[S][mb][h], acc[mb][nb]);
  }
  template <int V>
  MOE_DEV void sum(int nK) {
    const int n = (nK - wave + 7) / 8;  // steps wave, wave + 8, ..
    if (n <= 0) return;
    each<V>([&](auto s) {
      constexpr int S = decltype(s)::value;
      fetch<S>(wave + 8 * min(S, n - 1));
    });
    int i = 0;
    for (; i + 2 * V <= n; i += V)
      each<V>([&](auto s) {
        constexpr int S = decltype(s)::value;
        multiply<S>();
        fetch<S>(wave + 8 * (i + V + S));
      });
    if (i + V <= n) {
      each<V>([&](auto s) {
        constexpr int S = decltype(s)::value;
        multiply<S>();
        if (i + V + S < n) fetch<S>(wave + 8 * (i + V + S));
      });
      i += V;
    }
    each<V - 1>([&](auto s) {
      constexpr int S = decltype(s)::value;
      if (i + S < n) multiply<S>();
    });
  }
  // The sums over nK steps: block (mb, nb)'s in wave mb NNB + nb's acc[0][0], for the waves that have
  // one. red: 8 NMB NNB KB.
  MOE_DEV void run(int nK, Acc* red) {
#pragma unroll
    for (int mb = 0; mb < NMB; ++mb)
#pragma unroll
      for (int nb = 0; nb < NNB; ++nb) acc[mb][nb] = El::zero();
    if (U > 2 && nK < 8 * U) sum<2>(nK);  // a wave has fewer steps than U
    else sum<U>(nK);
    constexpr int NB = NMB * NNB;
    static_assert(NB <= 8, "a wave for each block");
#pragma unroll
    for (int mb = 0; mb < NMB; ++mb)
#pragma unroll
      for (int nb = 0; nb < NNB; ++nb)
        red[(wave * NB + mb * NNB + nb) * kWave + lane] = acc[mb][nb];
    __syncthreads();
    if (wave < NB) {
      acc[0][0] = red[wave * kWave + lane];
#pragma unroll
      for (int w = 1; w < 8; ++w) acc[0][0] += red[(w * NB + wave) * kWave + lane];
    }
  }
};

// Two side-by-side 16 x 16 blocks of bf16 results stored (with add, added in fp32 to what is
// there). Lanes 16..31 of lo and 0..15 of hi change places, and 48..63 and 32..47, so that each lane
// stores eight consecutive columns and a row's 64 bytes leave together. row: this lane's row at the
// blocks' first column.
MOE_DEV void swap16(uint32_t& lo, uint32_t& hi) {
  const auto v = __builtin_amdgcn_permlane16_swap(lo, hi, false, false);
  lo = v[0];
  hi = v[1];
}
MOE_DEV void store_pair(uint16_t* row, const f32x4& lo, const f32x4& hi, int lane, bool on,
                        bool add) {
  const int g = lane / 16;
  uint4* p = reinterpret_cast<uint4*>(row + ((g & 1) == 0 ? 4 * g : 12 + 4 * g));
  if (!add) {
    uint32_t l0 = to_bf2(lo[0], lo[1]), l1 = to_bf2(lo[2], lo[3]);
    uint32_t h0 = to_bf2(hi[0], hi[1]), h1 = to_bf2(hi[2], hi[3]);
    swap16(l0, h0);
    swap16(l1, h1);
    if (on) *p = make_uint4(l0, l1, h0, h1);
    return;
  }
  uint32_t o[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    o[q] = __float_as_uint(lo[q]);
    o[4 + q] = __float_as_uint(hi[q]);
    swap16(o[q], o[4 + q]);
  }
  if (!on) return;
  const uint4 v = *p;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t r[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    r[q] = to_bf2(__uint_as_float(o[2 * q]) + bf2f_lo(w[q]),
                  __uint_as_float(o[2 * q + 1]) + bf2f_hi(w[q]));
  *p = make_uint4(r[0], r[1], r[2], r[3]);
}
// NB blocks of a row, 16 columns each
template <int NB>
MOE_DEV void store_blocks(uint16_t* row, const f32x4 (&v)[NB], int lane, bool on, bool add) {
  if constexpr (NB == 1) {
    if (!on) return;
    uint2* p = reinterpret_cast<uint2*>(row + 4 * (lane / 16));
    f32x4 o = v[0];
    if (add) {
      const uint2 w = *p;
      o[0] += bf2f_lo(w.x);
      o[1] += bf2f_hi(w.x);
      o[2] += bf2f_lo(w.y);
      o[3] += bf2f_hi(w.y);
    }
    *p = make_uint2(to_bf2(o[0], o[1]), to_bf2(o[2], o[3]));
  } else {
#pragma unroll
    for (int nb = 0; nb < NB; nb += 2)
      store_pair(row + nb * 16, v[nb], v[nb + 1], lane, on, add);
  }
}

// The activations of the gated products and their derivatives, in fp32.
constexpr int kSilu = 0, kGelu = 1, kGeluTanh = 2, kRelu = 3;
constexpr float kGeluC = 0.7978845608028654f, kGeluK = 0.044715f;  // sqrt(2 / pi), the cubic's
// 1 / (1 + exp(-x)) by the reciprocal instruction, off by two half steps where a division is by one,
// for a third of its instructions: the epilogue of a gated 256 x 256 tile is 64 of these a lane.
MOE_DEV float fast_sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + __expf(-x)); }
template <int ACT>
MOE_DEV float act_of(float g) {
  if constexpr (ACT == kSilu) return g * fast_sigmoid(g);
  else if constexpr (ACT == kGelu) return 0.5f * g * erfcf(g * -0.70710678f);
  else if constexpr (ACT == kGeluTanh)  // 0.5 (1 + tanh z) = sigmoid(2 z)
    return g * fast_sigmoid(2.f * kGeluC * (g + kGeluK * g * g * g));
  else return g < 0.f ? 0.f : g;  // NaN stays
}
// act(g) and act'(g)
template <int ACT>
MOE_DEV float2 act_grad(float g) {
  if constexpr (ACT == kSilu) {
    const float s = fast_sigmoid(g);
    return make_float2(g * s, s * (1.f + g * (1.f - s)));
  } else if constexpr (ACT == kGelu) {
    const float p = 0.5f * erfcf(g * -0.70710678f);  // 1 + erf would cancel
    return make_float2(g * p, p + g * 0.3989422804f * __expf(-0.5f * g * g));
  } else if constexpr (ACT == kGeluTanh) {
    const float s = fast_sigmoid(2.f * kGeluC * (g + kGeluK * g * g * g));
    const float t = fminf(g * g, 256.f);  // from there on s (1 - s) is 0, and 0 inf would be NaN
    return make_float2(g * s,
                       s + g * s * (1.f - s) * (2.f * kGeluC) * (1.f + 3.f * kGeluK * t));
  } else {
    return g < 0.f ? make_float2(0.f, 0.f) : make_float2(g, g > 0.f ? 1.f : g);
  }
}
template <int A>
struct ActTag {
  static constexpr int value = A;
};
// fn(ActTag<act>)
template <class Fn>
MOE_DEV void with_act(int act, Fn fn) {
  switch (act) {
    case kSilu: fn(ActTag<kSilu>()); break;
    case kGelu: fn(ActTag<kGelu>()); break;
    case kGeluTanh: fn(ActTag<kGeluTanh>()); break;
    default: fn(ActTag<kRelu>()); break;
  }
}

}  // namespace
}  // namespace moe
