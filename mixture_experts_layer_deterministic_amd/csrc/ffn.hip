// The dense gated feed-forward block in bf16, forward and backward: the layer's shared expert.
//   [g | u] = x W1^T    A = act(g) u    y (+)= A W2^T
//   dA = dy W2    dH = bf16([dA u act'(g) | dA act(g)])
//   dx (+)= dH W1    dW1 (+)= dH^T x    dW2 (+)= dy^T A
// 2048 tokens x 7168 x 2048: forward 108 + 50 us (1.14e15 operations a second; library products of
// these sizes, without activation or H, take 111 to 114 + 54), backward 121 to 124 + 198 to 200 us in
// two launches, with fp32 gradients up to 9% more. What bounds the tiles stands in products.h.
// Adding to what is there: y of 1777 x 4096 x 1408 22.7 -> 24.8 us, the backward's kernels of 333 x
// 4096 x 1024 46 -> 50 us with bf16 gradients, 51 -> 70 with fp32 ones (50 MB more to read; each lane
// loads, adds and stores in turn).
//
// Sums are fp32 in a fixed order. A is formed from the fp32 g and u, dH from the bf16 H that the
// forward stored, and both are rounded once, as the next product reads them.
#include "common.h"
#include "ffn_plan.h"
#include "kernels.h"
#include "ops.h"
#include "products.h"

#define MOE_BOTH static __host__ __device__ __forceinline__

namespace moe {
namespace {

// The five products. Each has rows m x columns n (a gated one: of its weights) over steps of K, the
// layouts of its operands, where a tile reads them from step k0 on, and what becomes of its sums:
// store(w) for the rows row0 .. row0 + rows - 1 and columns n0 .. of the result, `cols` of the tile's
// columns being there. w.acc holds the sums, for rows w.row_of(mb) and column blocks of wave w.wn.

// A and, if it is wanted, H = [g | u].
struct GateUp {
  using Args = FfnArgs;
  static constexpr bool kAKM = false, kBKM = false, kGated = true;
  static constexpr const char* kName = "ffn_gate_up";
  MOE_BOTH long long m(const Args& a) { return a.T; }
  MOE_BOTH long long n(const Args& a) { return 2LL * a.I; }
  MOE_BOTH int steps(const Args& a) { return a.d / 64; }
  template <class W>
  static MOE_DEV void setup(const Args& a, W& w, int row0, int rows, int n0, int k0) {
    w.a_rows(2 * a.d);
    const int I = a.I;
    w.b_rows(2 * a.d, [&](int i) { return i < W::BN / 2 ? i : I + i - W::BN / 2; });
    w.next(a.x + (size_t)row0 * a.d + 64 * k0, 2u * rows * a.d - 128 * k0,
           a.w1 + (size_t)n0 * a.d + 64 * k0, 2u * (2 * I - n0) * a.d - 128 * k0);
  }
  template <class W>
  static MOE_DEV void store(const Args& a, const W& w, int row0, int rows, int n0, int) {
    constexpr int NG = W::NB / 2;
    const int c0 = n0 + w.wn * NG * 16, I = a.I;
    with_act(a.act, [&](auto tag) {
#pragma unroll
      for (int mb = 0; mb < W::MB; ++mb) {
        const int m = w.row_of(mb);
        const bool on = m < rows;
        f32x4 g[NG], u[NG], v[NG];
#pragma unroll
        for (int nb = 0; nb < NG; ++nb) {
          g[nb] = w.acc[mb][nb];
          u[nb] = w.acc[mb][nb + NG];
#pragma unroll
          for (int r = 0; r < 4; ++r) v[nb][r] = act_of<decltype(tag)::value>(g[nb][r]) * u[nb][r];
        }
        const size_t row = row0 + m;
        store_blocks<NG>(a.A + row * I + c0, v, w.lane, on, false);
        if (a.H) {
          store_blocks<NG>(a.H + row * 2 * I + c0, g, w.lane, on, false);
          store_blocks<NG>(a.H + row * 2 * I + I + c0, u, w.lane, on, false);
        }
      }
    });
  }
};

template <class W>
MOE_DEV void store_rows(uint16_t* out, int ld, bool add, const W& w, int row0, int rows, int n0,
                        int cols) {
  const int c0 = w.wn * W::NB * 16;
  if (c0 >= cols) return;
#pragma unroll
  for (int mb = 0; mb < W::MB; ++mb) {
    const int m = w.row_of(mb);
    store_blocks<W::NB>(out + (size_t)(row0 + m) * ld + n0 + c0, w.acc[mb], w.lane, m < rows, add);
  }
}

// y (+)= A W2^T
struct Down {
  using Args = FfnArgs;
  static constexpr bool kAKM = false, kBKM = false, kGated = false;
  static constexpr const char* kName = "ffn_down";
  MOE_BOTH long long m(const Args& a) { return a.T; }
  MOE_BOTH long long n(const Args& a) { return a.d; }
  MOE_BOTH int steps(const Args& a) { return a.I / 64; }
  template <class W>
  static MOE_DEV void setup(const Args& a, W& w, int row0, int rows, int n0, int k0) {
    w.a_rows(2 * a.I);
    w.b_rows(2 * a.I, [](int i) { return i; });
    w.next(a.A + (size_t)row0 * a.I + 64 * k0, 2u * rows * a.I - 128 * k0,
           a.w2 + (size_t)n0 * a.I + 64 * k0, 2u * (a.d - n0) * a.I - 128 * k0);
  }
  template <class W>
  static MOE_DEV void store(const Args& a, const W& w, int row0, int rows, int n0, int cols) {
    store_rows(a.y, a.d, a.acc_y, w, row0, rows, n0, cols);
  }
};

// dH from dA = dy W2 and H. W2 is [d, I]: K-major.
struct Dh {
  using Args = FfnArgs;
  static constexpr bool kAKM = false, kBKM = true, kGated = false;
  static constexpr bool kWideDw = true;  // whether its dW is ever in 128 x 256 tiles
  MOE_BOTH long long m(const Args& a) { return a.T; }
  MOE_BOTH long long n(const Args& a) { return a.I; }
  MOE_BOTH int steps(const Args& a) { return a.d / 64; }
  template <class W>
  static MOE_DEV void setup(const Args& a, W& w, int row0, int rows, int n0, int k0) {
    w.a_rows(2 * a.d);
    w.b_cols(2 * a.I);
    w.next(a.dy + (size_t)row0 * a.d + 64 * k0, 2u * rows * a.d - 128 * k0,
           a.w2 + (size_t)64 * k0 * a.I + n0, 2u * (a.d - 64 * k0) * a.I - 2 * n0);
  }
  template <class W>
  static MOE_DEV void store(const Args& a, const W& w, int row0, int rows, int n0, int cols) {
    const int c0 = w.wn * W::NB * 16, I = a.I;
    if (c0 >= cols) return;
    with_act(a.act, [&](auto tag) {
#pragma unroll
      for (int mb = 0; mb < W::MB; ++mb) {
        const int m = w.row_of(mb);
        const bool on = m < rows;
        const size_t at = (size_t)(row0 + min(m, rows - 1)) * 2 * I + n0 + c0;
        f32x4 dg[W::NB], du[W::NB];
#pragma unroll
        for (int nb = 0; nb < W::NB; ++nb) {
          const int c = nb * 16 + 4 * (w.lane / 16);
          const uint2 gv = *reinterpret_cast<const uint2*>(a.H + at + c);
          const uint2 uv = *reinterpret_cast<const uint2*>(a.H + at + I + c);
          const float g4[4] = {bf2f_lo(gv.x), bf2f_hi(gv.x), bf2f_lo(gv.y), bf2f_hi(gv.y)};
          const float u4[4] = {bf2f_lo(uv.x), bf2f_hi(uv.x), bf2f_lo(uv.y), bf2f_hi(uv.y)};
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float da = w.acc[mb][nb][r];
            const float2 f = act_grad<decltype(tag)::value>(g4[r]);
            dg[nb][r] = da * u4[r] * f.y;
            du[nb][r] = da * f.x;
          }
        }
        store_blocks<W::NB>(a.dH + at, dg, w.lane, on, false);
        store_blocks<W::NB>(a.dH + at + I, du, w.lane, on, false);
      }
    });
  }
};

// dx (+)= dH W1. W1 is [2I, d]: K-major.
struct Dx {
  using Args = FfnArgs;
  static constexpr bool kAKM = false, kBKM = true, kGated = false;
  // dW1 has 2I rows, whole 256s: 256 x 128 tiles are as few as 128 x 256 ones, and come first
  static constexpr bool kWideDw = false;
  MOE_BOTH long long m(const Args& a) { return a.T; }
  MOE_BOTH long long n(const Args& a) { return a.d; }
  MOE_BOTH int steps(const Args& a) { return 2 * a.I / 64; }
  template <class W>
  static MOE_DEV void setup(const Args& a, W& w, int row0, int rows, int n0, int k0) {
    w.a_rows(4 * a.I);
    w.b_cols(2 * a.d);
    w.next(a.dH + (size_t)row0 * 2 * a.I + 64 * k0, 4u * rows * a.I - 128 * k0,
           a.w1 + (size_t)64 * k0 * a.d + n0, 2u * (2 * a.I - 64 * k0) * a.d - 2 * n0);
  }
  template <class W>
  static MOE_DEV void store(const Args& a, const W& w, int row0, int rows, int n0, int cols) {
    store_rows(a.dx, a.d, a.acc_dx, w, row0, rows, n0, cols);
  }
};

// dW [Md, Nd] (+)= L^T R over the tokens, both operands K-major; rows past the last are zeros.
struct Dw {
  using Args = FfnDwArgs;
  static constexpr bool kAKM = true, kBKM = true, kGated = false;
  MOE_BOTH long long m(const Args& a) { return a.Md; }
  MOE_BOTH long long n(const Args& a) { return a.Nd; }
  MOE_BOTH int steps(const Args& a) { return (a.T + 63) / 64; }
  template <class W>
  static MOE_DEV void setup(const Args& a, W& w, int row0, int, int n0, int k0) {
    w.a_cols(2 * a.Md);
    w.b_cols(2 * a.Nd);
    w.next(a.L + (size_t)64 * k0 * a.Md + row0, 2u * (a.T - 64 * k0) * a.Md - 2 * row0,
           a.R + (size_t)64 * k0 * a.Nd + n0, 2u * (a.T - 64 * k0) * a.Nd - 2 * n0);
  }
  template <class W>
  static MOE_DEV void store(const Args& a, const W& w, int row0, int rows, int n0, int cols) {
    if (a.bf16_dw) {
      store_rows(static_cast<uint16_t*>(a.dw), a.Nd, a.acc, w, row0, rows, n0, cols);
      return;
    }
    const int c0 = w.wn * W::NB * 16;
    if (c0 >= cols) return;
#pragma unroll
    for (int mb = 0; mb < W::MB; ++mb) {
      const int m = w.row_of(mb);
      if (m >= rows) continue;
      float* p = static_cast<float*>(a.dw) + (size_t)(row0 + m) * a.Nd + n0 + c0 +
                 4 * (w.lane / 16);
#pragma unroll
      for (int nb = 0; nb < W::NB; ++nb) {
        if (a.acc) store_dw4<true>(p + nb * 16, w.acc[mb][nb]);
        else store_dw4<false>(p + nb * 16, w.acc[mb][nb]);
      }
    }
  }
};

// ------------------------------------------------------------------------------------------
// Where tile lt of P lies
struct Place {
  int row0, rows, n0, cols;
};
template <class P, int BM, int BN>
MOE_DEV Place place_of(const typename P::Args& a, int lt) {
  const int m = (int)P::m(a), n = (int)P::n(a);
  const int2 mn = big_order(lt, (m + BM - 1) / BM, (n + BN - 1) / BN);
  return {mn.x * BM, min(m - mn.x * BM, BM), mn.y * (P::kGated ? BN / 2 : BN),
          min(n - mn.y * BN, BN)};
}
template <class P, int BM, int BN>
MOE_BOTH long long tiles_of(const typename P::Args& a) {
  return (P::m(a) + BM - 1) / BM * ((P::n(a) + BN - 1) / BN);
}

template <class P, int BM, int BN>
MOE_DEV void whole_tile(const typename P::Args& a, int lt) {
  const Place t = place_of<P, BM, BN>(a, lt);
  Tile8<Bf16, BM, BN, P::kAKM, P::kBKM, P::kGated> w;
  w.begin();
  P::setup(a, w, t.row0, t.rows, t.n0, 0);
  w.run(P::steps(a));
  P::store(a, w, t.row0, t.rows, t.n0, t.cols);
}
// A tile a workgroup, an XCD's share contiguous.
template <class P, int BM, int BN>
__global__ void __launch_bounds__(512, 2) ffn_kernel(const typename P::Args a) {
  const int lt = xcd_contiguous(blockIdx.x, gridDim.x);
  if (lt < tiles_of<P, BM, BN>(a)) whole_tile<P, BM, BN>(a, lt);
}

// Few tiles: the steps of K in S shares, as even as they come, and a workgroup for each share of
// each 128 x 128 tile. Its sums go to memory as the lanes hold them (a.part), and a second kernel, a
// wave for 16 rows of a wave's columns, adds the shares in order and stores. A short chain of steps on
// every CU takes the place of a long one on few.
template <class P>
MOE_DEV void share_of_tile(const typename P::Args& a, int j) {
  const int S = a.shares, tiles = (int)tiles_of<P, 128, 128>(a);
  // one share of every tile, then the next: an XCD's tiles share their steps of K
  const int share = j / tiles, lt = j % tiles;
  const Place t = place_of<P, 128, 128>(a, lt);
  const int nk = P::steps(a), k0 = (int)((long long)nk * share / S);
  const int k1 = (int)((long long)nk * (share + 1) / S);
  using W = Tile8<Bf16, 128, 128, P::kAKM, P::kBKM, P::kGated>;
  W w;
  w.begin();
  P::setup(a, w, t.row0, t.rows, t.n0, k0);
  w.run(k1 - k0);
  f32x4* p = reinterpret_cast<f32x4*>(a.part) +
             ((size_t)(lt * S + share) * 8 + w.wave) * (W::MB * W::NB * kWave) + w.lane;
#pragma unroll
  for (int mb = 0; mb < W::MB; ++mb) {
    if ((w.wm * W::MB + mb) * 16 >= t.rows) continue;
#pragma unroll
    for (int nb = 0; nb < W::NB; ++nb) p[(mb * W::NB + nb) * kWave] = w.acc[mb][nb];
  }
}
template <class P>
__global__ void __launch_bounds__(512, 2) ffn_split_kernel(const typename P::Args a) {
  const int j = xcd_contiguous(blockIdx.x, gridDim.x);
  if (j < tiles_of<P, 128, 128>(a) * a.shares) share_of_tile<P>(a, j);
}

// A gradient of rows and one of weights that do not wait for each other, in one launch: the
// rows' tiles (or shares) first, `first` workgroups, then the weights'. One's last round runs beside
// the other's first: 333 x 4096 x 1024 73 -> 66 us.
using ffn::Shape;
using ffn::kBig;
using ffn::kTall;
using ffn::kWide;
using ffn::kSmall;
using ffn::kShares;
template <class P>
struct Pair {
  typename P::Args rows;
  FfnDwArgs dw;
  int rows_shape, dw_shape, first;
};
template <class P>
__global__ void __launch_bounds__(512, 2) ffn_pair_kernel(const Pair<P> p) {
  const int b = blockIdx.x;
  if (b < p.first) {
    const int lt = xcd_contiguous(b, p.first);
    switch (p.rows_shape) {
      case kBig:
        if (lt < tiles_of<P, 256, 256>(p.rows)) whole_tile<P, 256, 256>(p.rows, lt);
        break;
      case kTall:
        if (lt < tiles_of<P, 256, 128>(p.rows)) whole_tile<P, 256, 128>(p.rows, lt);
        break;
      case kWide:
        if (lt < tiles_of<P, 128, 256>(p.rows)) whole_tile<P, 128, 256>(p.rows, lt);
        break;
      case kSmall:
        if (lt < tiles_of<P, 128, 128>(p.rows)) whole_tile<P, 128, 128>(p.rows, lt);
        break;
      default:
        if (lt < tiles_of<P, 128, 128>(p.rows) * p.rows.shares) share_of_tile<P>(p.rows, lt);
    }
    return;
  }
  const int lt = xcd_contiguous(b - p.first, gridDim.x - p.first);
  switch (p.dw_shape) {
    case kBig:
      if (lt < tiles_of<Dw, 256, 256>(p.dw)) whole_tile<Dw, 256, 256>(p.dw, lt);
      break;
    case kTall:
      if (lt < tiles_of<Dw, 256, 128>(p.dw)) whole_tile<Dw, 256, 128>(p.dw, lt);
      break;
    case kWide:
      if constexpr (P::kWideDw)
        if (lt < tiles_of<Dw, 128, 256>(p.dw)) whole_tile<Dw, 128, 256>(p.dw, lt);
      break;
    case kSmall:
      if (lt < tiles_of<Dw, 128, 128>(p.dw)) whole_tile<Dw, 128, 128>(p.dw, lt);
      break;
    default:
      if (lt < tiles_of<Dw, 128, 128>(p.dw) * p.dw.shares) share_of_tile<Dw>(p.dw, lt);
  }
}

template <class T>
struct JoinedRows {  // one row block of a wave of tile T
  static constexpr int MB = 1, NB = T::NB, BN = T::BN;
  int lane, wn, row0;
  f32x4 acc[1][NB];
  MOE_DEV int row_of(int) const { return row0 + lane % 16; }
};
// Workgroup b of eight a tile.
template <class P>
MOE_DEV void join_rows(const typename P::Args& a, int block) {
  using T = Tile8<Bf16, 128, 128, P::kAKM, P::kBKM, P::kGated>;
  const int S = a.shares, lt = block / (2 * T::MB);
  const int b = block % (2 * T::MB) * 4 + threadIdx.x / kWave;  // row block of the tile's waves
  const int wave = b / T::MB, mb = b % T::MB;
  const Place t = place_of<P, 128, 128>(a, lt);
  JoinedRows<T> w;
  w.lane = threadIdx.x % kWave;
  w.wn = wave % T::WN;
  w.row0 = (wave / T::WN * T::MB + mb) * 16;
  if (w.row0 >= t.rows) return;  // a whole wave
  const f32x4* p = reinterpret_cast<const f32x4*>(a.part) +
                   ((size_t)lt * S * 8 + wave) * (T::MB * T::NB * kWave) + mb * T::NB * kWave +
                   w.lane;
#pragma unroll
  for (int nb = 0; nb < T::NB; ++nb) w.acc[0][nb] = p[nb * kWave];
#pragma unroll 8
  for (int s = 1; s < S; ++s) {
    p += 8 * T::MB * T::NB * kWave;
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb) w.acc[0][nb] += p[nb * kWave];
  }
  P::store(a, w, t.row0, t.rows, t.n0, t.cols);
}
template <class P>
__global__ void __launch_bounds__(256) ffn_join_kernel(const typename P::Args a) {
  join_rows<P>(a, blockIdx.x);
}
// Of a pair: the first `rows` workgroups for the rows' gradient, the others for the weights'.
template <class P>
__global__ void __launch_bounds__(256) ffn_join_pair_kernel(const Pair<P> p, int rows) {
  const int b = blockIdx.x;
  if (b < rows) join_rows<P>(p.rows, b);
  else join_rows<Dw>(p.dw, b - rows);
}

// A handful of tokens, up to 16 NMB: a workgroup for 8 columns of A. Its 34 MB of weights
// for 8 x 4096 x 2048, and y's 17, take 15.5 us.
template <int NMB, int U>
__global__ void __launch_bounds__(512, NMB == 1 ? 4 : 2) ffn_skinny_gate_up_kernel(const FfnArgs a) {
  __shared__ f32x4 red[8 * NMB * kWave];
  const int n0 = blockIdx.x * 8, I = a.I;
  SkinnyProduct<Bf16, NMB, 1, U> w;
  w.begin();
  w.a_rows(a.x, 2 * a.d, a.T);
  w.b_rows(a.w1, 2 * a.d, [&](int i) { return n0 + (i < 8 ? i : I + i - 8); });
  w.run(a.d / 64, red);
  if (w.wave >= NMB) return;
  // lanes 0..31 hold four gate columns of a row, lanes 32..63 the matching ups
  const int m = w.wave * 16 + w.lane % 16, c = n0 + 4 * (w.lane / 16 % 2);
  const f32x4 v = w.acc[0][0];
  f32x4 u;
#pragma unroll
  for (int r = 0; r < 4; ++r) u[r] = __shfl_xor(v[r], 32);
  if (m >= a.T) return;
  if (a.H)
    *reinterpret_cast<uint2*>(a.H + (size_t)m * 2 * I + (w.lane < 32 ? 0 : I) + c) =
        make_uint2(to_bf2(v[0], v[1]), to_bf2(v[2], v[3]));
  if (w.lane >= 32) return;
  with_act(a.act, [&](auto tag) {
    constexpr int A = decltype(tag)::value;
    *reinterpret_cast<uint2*>(a.A + (size_t)m * I + c) =
        make_uint2(to_bf2(act_of<A>(v[0]) * u[0], act_of<A>(v[1]) * u[1]),
                   to_bf2(act_of<A>(v[2]) * u[2], act_of<A>(v[3]) * u[3]));
  });
}
// Up to 16 NMB, a workgroup for 16 NNB columns of y. 16 x 2048 into 7168 columns in 9 us.
template <int NMB, int NNB, int U>
__global__ void __launch_bounds__(512, 2) ffn_skinny_down_kernel(const FfnArgs a) {
  __shared__ f32x4 red[8 * NMB * NNB * kWave];
  const int n0 = blockIdx.x * 16 * NNB;
  SkinnyProduct<Bf16, NMB, NNB, U> w;
  w.begin();
  w.a_rows(a.A, 2 * a.I, a.T);
  w.b_rows(a.w2, 2 * a.I, [&](int i) { return n0 + i; });
  w.run(a.I / 64, red);
  if (w.wave >= NMB * NNB) return;
  const int m = w.wave / NNB * 16 + w.lane % 16;
  const f32x4 v[1] = {w.acc[0][0]};
  store_blocks<1>(a.y + (size_t)m * a.d + n0 + w.wave % NNB * 16, v, w.lane, m < a.T, a.acc_y);
}

static_assert(ffn::kPlanCus == kCus, "one card");
template <class P>
ffn::Size size_of(const typename P::Args& a) {
  return {P::m(a), P::n(a), P::steps(a)};
}

template <class K, class A>
hipError_t launch_kernel(const char* name, K kernel, const A& a, long long grid, int threads,
                         hipStream_t s) {
  {
    TraceScope trace(name, s);
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(threads), 0, s, a);
  }
  return hipGetLastError();
}
long long grid8(long long tiles) { return (tiles + kXcds - 1) / kXcds * kXcds; }

template <class P>
hipError_t launch_whole(Shape shape, const char* name, const typename P::Args& a, hipStream_t s) {
  switch (shape) {
    case kBig:
      return launch_kernel(name, ffn_kernel<P, 256, 256>, a, grid8(tiles_of<P, 256, 256>(a)), 512, s);
    case kTall:
      return launch_kernel(name, ffn_kernel<P, 256, 128>, a, grid8(tiles_of<P, 256, 128>(a)), 512, s);
    case kWide:
      return launch_kernel(name, ffn_kernel<P, 128, 256>, a, grid8(tiles_of<P, 128, 256>(a)), 512, s);
    default:
      return launch_kernel(name, ffn_kernel<P, 128, 128>, a, grid8(tiles_of<P, 128, 128>(a)), 512, s);
  }
}
template <class P>
hipError_t launch_pair(const char* name, const FfnArgs& rows, const FfnDwArgs& dw, hipStream_t s) {
  const ffn::Size szr = size_of<P>(rows), szw = size_of<Dw>(dw);
  const ffn::PairPlan plan = ffn::plan_of_pair(szr, szw);
  if (!P::kWideDw && plan.dw.shape == kWide) return hipErrorInvalidValue;  // has no such tiles
  Pair<P> p{rows, dw, plan.rows.shape, plan.dw.shape, 0};
  p.rows.shares = plan.rows.shares;
  p.dw.shares = plan.dw.shares;
  const bool split_rows = plan.rows.shape == kShares, split_dw = plan.dw.shape == kShares;
  const long long nr = ffn::shape_tiles(szr, split_rows ? kSmall : plan.rows.shape);
  const long long nw = ffn::shape_tiles(szw, split_dw ? kSmall : plan.dw.shape);
  p.first = (int)grid8(nr * p.rows.shares);
  hipError_t e = launch_kernel(name, ffn_pair_kernel<P>, p, p.first + grid8(nw * p.dw.shares), 512, s);
  if (e != hipSuccess || (!split_rows && !split_dw)) return e;
  const long long jr = split_rows ? 8 * nr : 0, jw = split_dw ? 8 * nw : 0;
  {
    TraceScope trace(name, s);
    hipLaunchKernelGGL(ffn_join_pair_kernel<P>, dim3((unsigned)(jr + jw)), dim3(256), 0, s, p,
                       (int)jr);
  }
  return hipGetLastError();
}
template <class P>
hipError_t launch_product(FfnArgs a, hipStream_t s) {
  const ffn::Plan plan = ffn::plan_of(size_of<P>(a));
  a.shares = plan.shares;
  if (plan.shape != kShares) return launch_whole<P>(plan.shape, P::kName, a, s);
  const long long tiles = tiles_of<P, 128, 128>(a);
  const hipError_t e =
      launch_kernel(P::kName, ffn_split_kernel<P>, a, grid8(tiles * a.shares), 512, s);
  if (e != hipSuccess) return e;
  return launch_kernel(P::kName, ffn_join_kernel<P>, a, tiles * 8, 256, s);
}

}  // namespace

hipError_t launch_ffn_gate_up(const FfnArgs& a, hipStream_t s) {
  if (!ffn::few_gate_up(a.T, a.d, a.I)) return launch_product<GateUp>(a, s);
  const auto kernel = a.T <= 16   ? ffn_skinny_gate_up_kernel<1, 4>
                      : a.T <= 32 ? ffn_skinny_gate_up_kernel<2, 4>
                                  : ffn_skinny_gate_up_kernel<4, 2>;
  return launch_kernel("ffn_gate_up", kernel, a, a.I / 8, 512, s);
}
hipError_t launch_ffn_down(const FfnArgs& a, hipStream_t s) {
  if (!ffn::few_down(a.T, a.d, a.I)) return launch_product<Down>(a, s);
  const int cols = ffn::few_down_cols(a.d);
  const auto narrow = a.T <= 16   ? ffn_skinny_down_kernel<1, 1, 4>
                      : a.T <= 32 ? ffn_skinny_down_kernel<2, 1, 4>
                                  : ffn_skinny_down_kernel<4, 1, 2>;
  const auto broad = a.T <= 16   ? ffn_skinny_down_kernel<1, 2, 4>
                     : a.T <= 32 ? ffn_skinny_down_kernel<2, 2, 4>
                                 : ffn_skinny_down_kernel<4, 2, 2>;
  return launch_kernel("ffn_down", cols == 32 ? broad : narrow, a, a.d / cols, 512, s);
}
hipError_t launch_ffn_dh_dw2(const FfnArgs& a, const FfnDwArgs& dw, hipStream_t s) {
  return launch_pair<Dh>("ffn_dh_dw2", a, dw, s);
}
hipError_t launch_ffn_dx_dw1(const FfnArgs& a, const FfnDwArgs& dw, hipStream_t s) {
  return launch_pair<Dx>("ffn_dx_dw1", a, dw, s);
}

}  // namespace moe
