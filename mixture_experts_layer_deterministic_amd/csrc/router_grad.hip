// Gradients of the router's linear map l = x Wr^T from any gradient dl of its logits:
//   dx[t]  (+)= sum_e dl[t, e] Wr[e]      T x d, reduced over the experts
//   dWr[e] (+)= sum_t dl[t, e] x[t]       E x d, reduced over the tokens
//
// dl is fp32 and x, Wr are bf16. Each dl value is split into bf16 parts whose products with bf16
// values are exact in fp32, so bf16 MFMAs do an fp32 product's work at a rate that fp32 MFMAs
// (1/16 of bf16's) do not reach. Cutting a value's upper 8 bits off, then the next 8 of what is
// left, gives three parts that add up to all its 24 bits: dWr, an fp32 sum, takes the three. dx
// is rounded to bf16 (2^-8) at the end and takes two, both rounded to nearest: of x in [1, 2) the
// first leaves at most 2^-8 and the second at most 2^-17 of that. Those 2^-17 of a term stay below
// the output's own rounding unless the terms cancel to 2^-9 of their size, and Wr, itself bf16,
// does not hold values that agree so far and differ: a dense softmax's gradients, whose rows sum to
// 0, against weights whose common part is 100 (300) times their spread give dx an error of 1.68e-3
// (1.81e-3), an fp32 product rounded to bf16 1.66e-3. Three parts for dx, both gradients of 2048 x
// 7168 x 256 with the copies around them: 57 -> 66 us; of 1777 x 4096 x 509: 41 -> 56.
#include "common.h"
#include "kernels.h"
#include "ops.h"

namespace moe {
namespace {

constexpr int kRgN = 128;  // tile columns
constexpr int kRgK = 64;   // reduction depth of a step

typedef __attribute__((ext_vector_type(2))) float rg_f2;
typedef __attribute__((ext_vector_type(2))) __bf16 rg_bf2;

MOE_DEV uint32_t upper2(float lo, float hi) {  // the upper halves of two floats: cut-off bf16
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
MOE_DEV uint32_t round2(float lo, float hi) {  // two floats rounded to bf16
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(rg_f2{lo, hi}, rg_bf2));
}
MOE_DEV float cut(float x) {  // what is left of x below its upper 8 bits (exact)
  return x - __uint_as_float(__float_as_uint(x) & 0xffff0000u);
}
template <int P>
MOE_DEV void split4(const f32x4& x, uint2 (&part)[P]) {
  if constexpr (P == 2) {
    part[0] = make_uint2(round2(x[0], x[1]), round2(x[2], x[3]));
    part[1] = make_uint2(round2(x[0] - bf2f_lo(part[0].x), x[1] - bf2f_hi(part[0].x)),
                         round2(x[2] - bf2f_lo(part[0].y), x[3] - bf2f_hi(part[0].y)));
  } else {
    const float r0 = cut(x[0]), r1 = cut(x[1]), r2 = cut(x[2]), r3 = cut(x[3]);
    part[0] = make_uint2(upper2(x[0], x[1]), upper2(x[2], x[3]));
    part[1] = make_uint2(upper2(r0, r1), upper2(r2, r3));
    part[2] = make_uint2(upper2(cut(r0), cut(r1)), upper2(cut(r2), cut(r3)));
  }
}

MOE_DEV __amdgpu_buffer_rsrc_t rg_rsrc(const void* base, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0,
                                           (int)(bytes < 0xffffffffu ? bytes : 0xffffffffu),
                                           0x00020000);
}

// kmajor_swz for rows of 64 values: four groups of 16 to permute.
MOE_DEV int swz64(int k) { return 16 * (k & 3); }
// kmajor_frag on such rows.
MOE_DEV uint4 kmajor_frag64(const uint16_t* s, int base, int kb, int lane) {
  const int g = lane / 16, q = lane % 16, kr = 8 * g + q / 4;
  const int n = (base ^ swz64(kr)) + 4 * (q % 4);
  const uint16_t* p = s + (kb + kr) * 64 + n;
  const uint2 a = __builtin_bit_cast(uint2, lds_read_tr16(p));
  const uint2 b = __builtin_bit_cast(uint2, lds_read_tr16(p + 4 * 64));
  return make_uint4(a.x, a.y, b.x, b.y);
}

// One tile a workgroup of eight waves. DW: 64 experts x 128 columns of dWr, reduced over the
// tokens; waves 0..3 take the even steps of 64 tokens and waves 4..7 the odd ones, and the second
// sum is added to the first at the end: the tokens are many and these tiles few, and two chains
// of steps fill a CU better than one (dWr alone at 1792 x 4096 x 512: 36 -> 30 us). Else 128
// tokens x 128 columns of dx, reduced over the experts by all eight waves. A wave holds 32 x 64
// outputs.
// A step's dl tile is split once for its waves, on its way from registers to LDS; the loads of
// the next step are out by then. The bf16 operand lies in LDS as it does in memory and reaches
// the MFMAs through the transposing read; so does dl for dWr, whose reduction axis is the slow
// one of both.
//
// Both gradients of 2048 x 7168 x 256, five bf16 products of 7.5 GFLOP: 44.5 us, 0.84 PFLOP/s, of
// 1.2 that a large library product reaches. A step's fragment reads (20 KB a wave for 48 MFMAs of
// dWr, 16 KB for 32 of dx) and its split tile's writes keep LDS as busy as the MFMAs, and dx's
// tiles end in a part round. 256 x 128 tiles of dx, 64 x 64 outputs a wave, would read less and fit
// the same LDS, but take 156 registers of the 128 that two workgroups a CU leave a wave.
constexpr int kRgLdsW = 3 * 64 * kRgK + kRgK * kRgN;   // values of one half's stage
constexpr int kRgLdsX = 2 * 128 * kRgK + kRgK * kRgN;
constexpr int kRgLds = 2 * kRgLdsW;
static_assert(kRgLdsX <= kRgLds && 64 * kRgN * 2 <= kRgLds, "dx's stage and a half's sums fit");

template <bool DW>
struct RouterTile {
  static constexpr int P = DW ? 3 : 2, BM = DW ? 64 : 128, MB = 2, AJ = 4;
  static constexpr int kThr = DW ? 256 : 512;   // threads that share a stage
  static constexpr int kRows = kThr / 16, BJ = kRgK / kRows;
  static constexpr int kPlane = BM * kRgK;      // values of one part
  static constexpr int kStride = DW ? 2 * kRgK : kRgK;
  int tid, wm, wn, lane;
  f32x4 av[AJ];
  uint4 bv[BJ];
  f32x4 acc[MB][4];

  // dl rows: DW, tokens k0 + i (reduction), experts r0 ..; else tokens r0 + i, experts k0 ..
  // Buffer loads that end with their tensor, so rows past its end read as zeros without a branch.
  // A dl row's columns past E belong to the next row: for dx they are cleared on their way to
  // LDS (the weight rows they meet are zeros, but NaN times zero is not), for dWr they lead to
  // rows that are not stored.
  MOE_DEV void load(const RouterGradArgs& a, int r0, int c0, int k0) {
    const int i = tid / 16, c = tid % 16, K = DW ? a.T : a.E;
    const size_t t0 = DW ? k0 : r0, e0 = DW ? r0 : k0;
    const size_t left = k0 < K ? 1 : 0;  // a half may have no step where the other has one
    const __amdgpu_buffer_rsrc_t ra =
        rg_rsrc(a.dl + t0 * a.E + e0, left * ((a.T - t0) * a.E - e0) * 4);
#pragma unroll
    for (int j = 0; j < AJ; ++j)
      av[j] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                            ra, ((i + kRows * j) * a.E + c * 4) * 4, 0, 0));
    const uint16_t* src = DW ? a.x : a.wr;
    const __amdgpu_buffer_rsrc_t rb =
        rg_rsrc(src + (size_t)k0 * a.d + c0, left * ((size_t)(K - k0) * a.d - c0) * 2);
#pragma unroll
    for (int j = 0; j < BJ; ++j)
      bv[j] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                            rb, ((i + kRows * j) * a.d + c * 8) * 2, 0, 0));
  }
  MOE_DEV void store(uint16_t* lds, int left) {  // left: what remains of the reduction
    if (!DW && left < kRgK) {
#pragma unroll
      for (int j = 0; j < AJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (tid % 16 * 4 + q >= left) av[j][q] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < AJ; ++j) {
      const int i = tid / 16 + kRows * j, c = tid % 16 * 4;
      uint2 part[P];
      split4<P>(av[j], part);
      const int at = DW ? i * 64 + (c ^ swz64(i)) : rowswz(i, c / 8) + c % 8;
#pragma unroll
      for (int p = 0; p < P; ++p) *reinterpret_cast<uint2*>(lds + p * kPlane + at) = part[p];
    }
#pragma unroll
    for (int j = 0; j < BJ; ++j) {
      const int k = tid / 16 + kRows * j;
      *reinterpret_cast<uint4*>(lds + P * kPlane + k * kRgN + ((tid % 16 * 8) ^ kmajor_swz(k))) =
          bv[j];
    }
  }
  MOE_DEV void run(const RouterGradArgs& a, int r0, int c0, uint16_t* all) {
    const int wave = threadIdx.x / kWave, half = DW ? wave / 4 : 0;
    lane = threadIdx.x % kWave;
    tid = threadIdx.x % kThr;
    wm = wave % (kThr / kWave) / 2;
    wn = wave % 2;
    uint16_t* lds = all + half * kRgLdsW;
    const int R = DW ? a.E : a.T, K = DW ? a.T : a.E;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int first = __builtin_amdgcn_readfirstlane(half) * kRgK;
    load(a, r0, c0, first);
    for (int k0 = 0; k0 < K; k0 += kStride) {
      __syncthreads();
      store(lds, K - k0);
      __syncthreads();
      if (k0 + kStride < K) load(a, r0, c0, k0 + kStride + first);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        uint4 bf[4];
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
          bf[nb] = kmajor_frag<kRgN>(lds + P * kPlane, wn * 64 + nb * 16, ks * 32, lane);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          const int m = (wm * MB + mb) * 16;
#pragma unroll
          for (int p = P - 1; p >= 0; --p) {  // the small parts first
            const uint16_t* pl = lds + p * kPlane;
            const uint4 af = DW ? kmajor_frag64(pl, m, ks * 32, lane)
                                : *reinterpret_cast<const uint4*>(
                                      pl + rowswz(m + lane % 16, ks * 4 + lane / 16));
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) acc[mb][nb] = mfma16(bf[nb], af, acc[mb][nb]);
          }
        }
      }
    }
    if constexpr (DW) {  // the odd steps' sums, lane by lane
      f32x4* sum = reinterpret_cast<f32x4*>(all) + tid;
      __syncthreads();
      if (half == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i * 256] = acc[i / 4][i % 4];
      }
      __syncthreads();
      if (half == 1) return;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i / 4][i % 4] += sum[i * 256];
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const int r = r0 + (wm * MB + mb) * 16 + lane % 16;
      if (r >= R) continue;
      if constexpr (DW) {
        float* p = a.dwr + (size_t)r * a.d + c0 + wn * 64 + 4 * (lane / 16);
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          if (a.acc_dwr) store_dw4<true>(p + nb * 16, acc[mb][nb]);
          else store_dw4<false>(p + nb * 16, acc[mb][nb]);
        }
      } else {
        // one rounding to bf16, of the fp32 sum with what dx held
        uint16_t* p = a.dx + (size_t)r * a.d + c0 + wn * 64;
#pragma unroll
        for (int nb = 0; nb < 4; nb += 2) {
          if (a.acc_dx) store_dw8_bf16<true>(p + nb * 16, acc[mb][nb], acc[mb][nb + 1], lane);
          else store_dw8_bf16<false>(p + nb * 16, acc[mb][nb], acc[mb][nb + 1], lane);
        }
      }
    }
  }
};

// The dWr tiles come first: their reductions are the long ones.
__global__ void __launch_bounds__(512, 4) router_backward_kernel(const RouterGradArgs a, int nw) {
  __shared__ __align__(16) uint16_t lds[kRgLds];
  const int nc = a.d / kRgN;
  const int b = blockIdx.x;
  if (b < nw) {
    RouterTile<true> t;
    t.run(a, b / nc * 64, b % nc * kRgN, lds);
  } else {
    RouterTile<false> t;
    t.run(a, (b - nw) / nc * 128, (b - nw) % nc * kRgN, lds);
  }
}

// dWr where experts x columns are few and tokens many: tiles of 16 MB experts x 16 NB columns,
// whose 16 waves split the tokens, steps of 32 in turn. Operands go from memory to registers in
// whole pieces and never through LDS, and no wave waits for another: lane l = 16 g + r loads, i =
// 0 .. 7,
//  * of x token 8 g + i, columns NB r .. NB r + NB - 1: those 8 x NB values are the lane's parts of
//    NB fragments once pairs of tokens are woven (one byte permutation a register), fragment n's
//    column r standing for column NB r + n of the tile;
//  * of dl token 8 g + i, experts MB r .. MB r + MB - 1: likewise MB fragments.
// The waves' sums are added in LDS in a fixed order.
// 8 experts, 16384 x 4096: 48 us, 2.8 TB/s of x, bound by the latency of a wave's one step ahead;
// 128 experts, 8192 x 4096: 46 us, 0.56 PFLOP/s in three products, bound by the vector work of
// splitting and weaving. (The 64 x 128 tiles: 233 and 121, on 32 and 64 CUs.)
constexpr int kFewWaves = 16;
// A number the compiler has to take as new: sums with it are made where they are used, since kept
// over the loop they cost more registers than a wave has.
MOE_DEV uint32_t here(uint32_t x) {
  asm volatile("" : "+s"(x));
  return x;
}
template <int WORDS>
MOE_DEV void get_words(__amdgpu_buffer_rsrc_t rows, uint32_t at, uint32_t (&w)[WORDS]) {
  if constexpr (WORDS == 1) {
    w[0] = __builtin_amdgcn_raw_buffer_load_b32(rows, at, 0, 0);
  } else {
    static_assert(WORDS == 2, "one or two words");
    const uint2 v = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rows, at, 0, 0));
    w[0] = v.x;
    w[1] = v.y;
  }
}
template <int MB, int NB>
__global__ void __launch_bounds__(kFewWaves* kWave) router_dw_few_kernel(const RouterGradArgs a) {
  constexpr int kStep = 32, kStride = kFewWaves * kStep;
  __shared__ float sums[kFewWaves][MB * NB][4][kWave];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x % kWave, r = lane % 16, g = lane / 16;
  const int nc = a.d / (16 * NB), r0 = blockIdx.x / nc * 16 * MB, c0 = blockIdx.x % nc * 16 * NB;
  uint32_t dv[8][MB], xv[8][NB / 2];
  // buffer loads that end with their step's rows: tokens past the end read as zeros without a
  // branch. dl's columns past E, the next token's, lead to rows that are not stored.
  auto load = [&](int k0) {
    const int left = min(a.T - k0, kStep);
    const __amdgpu_buffer_rsrc_t dl =
        rg_rsrc(a.dl + (size_t)k0 * a.E + r0, left > 0 ? 4u * (left * a.E - r0) : 0u);
    const __amdgpu_buffer_rsrc_t x =
        rg_rsrc(a.x + (size_t)k0 * a.d + c0, left > 0 ? 2u * (left * a.d - c0) : 0u);
    const uint32_t dl_row = here(a.E * 4), x_row = here(a.d * 2);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      get_words<MB>(dl, (8 * g + i) * dl_row + 4 * MB * r, dv[i]);
      get_words<NB / 2>(x, (8 * g + i) * x_row + 2 * NB * r, xv[i]);
    }
  };
  f32x4 acc[MB][NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  load(wave * kStep);
  for (int k0 = wave * kStep; k0 < a.T; k0 += kStride) {
    uint4 bf[NB], af[MB][3];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = __builtin_amdgcn_perm(xv[2 * q + 1][n / 2], xv[2 * q][n / 2],
                                     n % 2 ? 0x07060302u : 0x05040100u);
      bf[n] = make_uint4(w[0], w[1], w[2], w[3]);
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      f32x4 v[2];
      uint2 lo[3], hi[3];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i / 4][i % 4] = __uint_as_float(dv[i][m]);
      split4<3>(v[0], lo);
      split4<3>(v[1], hi);
#pragma unroll
      for (int p = 0; p < 3; ++p) af[m][p] = make_uint4(lo[p].x, lo[p].y, hi[p].x, hi[p].y);
    }
    __builtin_amdgcn_sched_barrier(0);  // the next loads go out into the registers just read
    load(k0 + kStride);
#pragma unroll
    for (int p = 2; p >= 0; --p)  // the small parts first
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n) acc[m][n] = mfma16(bf[n], af[m][p], acc[m][n]);
  }
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) sums[wave][m * NB + n][j][lane] = acc[m][n][j];
  __syncthreads();
  // a thread an output: column c of row e of the tile, tile columns side by side
  for (int o = threadIdx.x; o < 16 * MB * 16 * NB; o += kFewWaves * kWave) {
    const int e = o / (16 * NB), c = o % (16 * NB);
    const int m = e % MB, n = c % NB, j = c / NB % 4, l = c / NB / 4 * 16 + e / MB;
    float s = sums[0][m * NB + n][j][l];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) s += sums[w][m * NB + n][j][l];
    if (r0 + e < a.E) {
      float* p = a.dwr + (size_t)(r0 + e) * a.d + c0 + c;
      *p = a.acc_dwr ? *p + s : s;
    }
  }
}

}  // namespace

hipError_t launch_router_backward(const RouterGradArgs& a, hipStream_t s) {
  const int nc = a.d / kRgN;
  int nw = a.dwr ? (a.E + 63) / 64 * nc : 0;
  const int nx = a.dx ? (a.T + 127) / 128 * nc : 0;
  // Which kernel sums dWr (by T, d and E alone, so that asking for dx changes no bit of it). Both
  // gradients in us, 64 x 128 tiles in dx's launch against small tiles in a launch of their own:
  //  * up to 64 tiles of 64 x 128 and 32 tokens a tile, 1024 at least: small. 16 tiles (64 experts,
  //    2048 columns) 1024 tokens 19 against 14, 16384 243 against 83; 64 tiles (128 experts, 4096
  //    columns) 2048 tokens 36 against 31. Fewer tokens: 16 tiles, 512 tokens 11 against 13; 64
  //    tiles, 1024 tokens 20 against 22. More tiles: 80, 4096 tokens 68 against 76.
  //  * of them tiles of 16 experts while they are one a CU at most, else of 32. 256 of 16 (64
  //    experts, 4096 columns), 4096 tokens: 37 against 42; 512 (128 experts, 4096 columns): 53
  //    against 47.
  if (nw && nw <= 64 && a.T >= 1024 && a.T >= 32 * nw) {
    const int n16 = (a.E + 15) / 16 * (a.d / 64), n32 = (a.E + 31) / 32 * (a.d / 64);
    TraceScope trace("router_dwr", s);
    if (n16 <= 256)
      hipLaunchKernelGGL((router_dw_few_kernel<1, 4>), dim3(n16), dim3(kFewWaves * kWave), 0, s, a);
    else
      hipLaunchKernelGGL((router_dw_few_kernel<2, 4>), dim3(n32), dim3(kFewWaves * kWave), 0, s, a);
    nw = 0;
  }
  if (nw + nx) {
    TraceScope trace("router_backward", s);
    hipLaunchKernelGGL(router_backward_kernel, dim3(nw + nx), dim3(512), 0, s, a, nw);
  }
  return hipGetLastError();
}

}  // namespace moe
