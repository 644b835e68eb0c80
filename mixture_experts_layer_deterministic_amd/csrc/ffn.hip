// The dense gated feed-forward block in bf16, forward and backward: the layer's shared expert.
//   [g | u] = x W1^T    A = act(g) u    y (+)= A W2^T
//   dA = dy W2    dH = bf16([dA u act'(g) | dA act(g)])
//   dx (+)= dH W1    dW1 (+)= dH^T x    dW2 (+)= dy^T A
// Sums are fp32 in ascending order of K. A is formed from the fp32 g and u, dH from the bf16 H that
// the forward stored, and both are rounded once, as the next product reads them.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "ops.h"
#include "products.h"

namespace moe {
namespace {

// Tile b of a grid of nm x nN tiles, dealt so that an XCD's share is contiguous; x < 0: none.
MOE_DEV int2 dense_tile(int b, int grid, int nm, int nN) {
  const int lt = xcd_contiguous(b, grid);
  return lt < nm * nN ? big_order(lt, nm, nN) : make_int2(-1, 0);
}
MOE_DEV int tiles_of(int n, int t) { return (n + t - 1) / t; }

// A and, if it is wanted, H = [g | u].
template <int BM, int BN>
__global__ void __launch_bounds__(512, 2) ffn_gate_up_kernel(const FfnArgs a) {
  constexpr int kCols = BN / 2;
  const int2 mn = dense_tile(blockIdx.x, gridDim.x, tiles_of(a.T, BM), a.I / kCols);
  if (mn.x < 0) return;
  const int row0 = mn.x * BM, rows = min(a.T - row0, BM), n0 = mn.y * kCols;
  Tile8<Bf16, BM, BN, false, false, true> w;
  w.begin();
  w.a_rows(a.x + (size_t)row0 * a.d, 2 * a.d, rows);
  const int I = a.I;
  w.b_rows(a.w1, 2 * a.d, [&](int i) { return i < kCols ? n0 + i : I + n0 + i - kCols; });
  w.run(a.d / 64);
  constexpr int NG = w.NB / 2;
  const int c0 = n0 + w.wn * NG * 16;
  with_act(a.act, [&](auto tag) {
#pragma unroll
    for (int mb = 0; mb < w.MB; ++mb) {
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

// out (+)= L R^T with both K-contiguous: y from A and W2.
template <int BM, int BN>
__global__ void __launch_bounds__(512, 2) ffn_down_kernel(const FfnArgs a) {
  const int2 mn = dense_tile(blockIdx.x, gridDim.x, tiles_of(a.T, BM), tiles_of(a.d, BN));
  if (mn.x < 0) return;
  const int row0 = mn.x * BM, rows = min(a.T - row0, BM), n0 = mn.y * BN;
  const int cols = min(BN, a.d - n0);
  Tile8<Bf16, BM, BN> w;
  w.begin();
  w.a_rows(a.A + (size_t)row0 * a.I, 2 * a.I, rows);
  w.b_rows(a.w2 + (size_t)n0 * a.I, 2 * a.I, [&](int i) { return min(i, cols - 1); });
  w.run(a.I / 64);
  const int c0 = w.wn * w.NB * 16;
  if (c0 >= cols) return;
#pragma unroll
  for (int mb = 0; mb < w.MB; ++mb) {
    const int m = w.row_of(mb);
    store_blocks<w.NB>(a.y + (size_t)(row0 + m) * a.d + n0 + c0, w.acc[mb], w.lane, m < rows,
                       a.acc_y);
  }
}

// dH from dA = dy W2 and H. W2 is [d, I]: K-major.
template <int BM, int BN>
__global__ void __launch_bounds__(512, 2) ffn_dh_kernel(const FfnArgs a) {
  const int2 mn = dense_tile(blockIdx.x, gridDim.x, tiles_of(a.T, BM), tiles_of(a.I, BN));
  if (mn.x < 0) return;
  const int row0 = mn.x * BM, rows = min(a.T - row0, BM), n0 = mn.y * BN;
  const int cols = min(BN, a.I - n0), I = a.I;
  Tile8<Bf16, BM, BN, false, true> w;
  w.begin();
  w.a_rows(a.dy + (size_t)row0 * a.d, 2 * a.d, rows);
  w.b_cols(a.w2 + n0, 2 * I, 2u * a.d * I, cols);
  w.run(a.d / 64);
  const int c0 = w.wn * w.NB * 16;
  if (c0 >= cols) return;
  with_act(a.act, [&](auto tag) {
#pragma unroll
    for (int mb = 0; mb < w.MB; ++mb) {
      const int m = w.row_of(mb);
      const bool on = m < rows;
      const size_t at = (size_t)(row0 + min(m, rows - 1)) * 2 * I + n0 + c0;
      f32x4 dg[w.NB], du[w.NB];
#pragma unroll
      for (int nb = 0; nb < w.NB; ++nb) {
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
      store_blocks<w.NB>(a.dH + at, dg, w.lane, on, false);
      store_blocks<w.NB>(a.dH + at + I, du, w.lane, on, false);
    }
  });
}

// dx (+)= dH W1. W1 is [2I, d]: K-major.
template <int BM, int BN>
__global__ void __launch_bounds__(512, 2) ffn_dx_kernel(const FfnArgs a) {
  const int2 mn = dense_tile(blockIdx.x, gridDim.x, tiles_of(a.T, BM), tiles_of(a.d, BN));
  if (mn.x < 0) return;
  const int row0 = mn.x * BM, rows = min(a.T - row0, BM), n0 = mn.y * BN;
  const int cols = min(BN, a.d - n0);
  Tile8<Bf16, BM, BN, false, true> w;
  w.begin();
  w.a_rows(a.dH + (size_t)row0 * 2 * a.I, 4 * a.I, rows);
  w.b_cols(a.w1 + n0, 2 * a.d, 4u * a.I * a.d, cols);
  w.run(2 * a.I / 64);
  const int c0 = w.wn * w.NB * 16;
  if (c0 >= cols) return;
#pragma unroll
  for (int mb = 0; mb < w.MB; ++mb) {
    const int m = w.row_of(mb);
    store_blocks<w.NB>(a.dx + (size_t)(row0 + m) * a.d + n0 + c0, w.acc[mb], w.lane, m < rows,
                       a.acc_dx);
  }
}

// dW [Md, Nd] (+)= L^T R over the tokens, both operands K-major; rows past the last are zeros.
template <int BM, int BN>
__global__ void __launch_bounds__(512, 2) ffn_dw_kernel(const FfnDwArgs a) {
  const int2 mn = dense_tile(blockIdx.x, gridDim.x, tiles_of(a.Md, BM), tiles_of(a.Nd, BN));
  if (mn.x < 0) return;
  const int m0 = mn.x * BM, n0 = mn.y * BN;
  const int rows = min(BM, a.Md - m0), cols = min(BN, a.Nd - n0);
  Tile8<Bf16, BM, BN, true, true> w;
  w.begin();
  w.a_cols(a.L + m0, 2 * a.Md, 2u * a.T * a.Md, rows);
  w.b_cols(a.R + n0, 2 * a.Nd, 2u * a.T * a.Nd, cols);
  w.run((a.T + 63) / 64);
  const int c0 = w.wn * w.NB * 16;
  if (c0 >= cols) return;
#pragma unroll
  for (int mb = 0; mb < w.MB; ++mb) {
    const int m = w.row_of(mb);
    const size_t at = (size_t)(m0 + m) * a.Nd + n0 + c0;
    if (a.bf16_dw) {
      store_blocks<w.NB>(static_cast<uint16_t*>(a.dw) + at, w.acc[mb], w.lane, m < rows, a.acc);
    } else if (m < rows) {
      float* p = static_cast<float*>(a.dw) + at + 4 * (w.lane / 16);
#pragma unroll
      for (int nb = 0; nb < w.NB; ++nb) {
        if (a.acc) store_dw4<true>(p + nb * 16, w.acc[mb][nb]);
        else store_dw4<false>(p + nb * 16, w.acc[mb][nb]);
      }
    }
  }
}

long long ceil_div(long long n, int t) { return (n + t - 1) / t; }

// The tile shape for a product of m rows and n columns: that of the fewest rounds of one tile a CU,
// each at what a step of it takes when the card is full, in us: 256 x 256 1.35, 256 x 128 0.95,
// 128 x 128 0.67 (bytes a step 64, 48 and 32 KB). Measured, the whole call in us, 256 x 256 / 256 x
// 128 / 128 x 128: [g | u] of 2048 x 7168 x 2048 141 / 107 / 142 (128, 256, 512 tiles), its y
// 51 / 64 / 88 (224, 448, 896), dH 155 / 107 / 80 (64, 128, 256); [g | u] of 1777 x 4096 x 1408
// 80 / 53 / 72 (77, 154, 308).
enum Shape { kBig, kTall, kWide, kSmall };
Shape tile_shape(long long m, long long n) {
  static const struct {
    int bm, bn;
    float us;
  } shapes[4] = {{256, 256, 1.35f}, {256, 128, 0.95f}, {128, 256, 0.95f}, {128, 128, 0.67f}};
  int best = 0;
  float least = 0.f;
  long long fewest = 0;
  for (int i = 0; i < 4; ++i) {
    const long long tiles = ceil_div(m, shapes[i].bm) * ceil_div(n, shapes[i].bn);
    const float us = (float)ceil_div(tiles, kCus) * shapes[i].us;
    if (i == 0 || us < least || (us == least && tiles < fewest)) {
      best = i;
      least = us;
      fewest = tiles;
    }
  }
  return (Shape)best;
}

template <class K, class A>
hipError_t launch_tiles(const char* name, K kernel, const A& a, long long tiles, hipStream_t s) {
  {
    TraceScope trace(name, s);
    hipLaunchKernelGGL(kernel, dim3((unsigned)((tiles + kXcds - 1) / kXcds * kXcds)), dim3(512), 0,
                       s, a);
  }
  return hipGetLastError();
}
// Kernel K<BM, BN> of the shape that fits m rows and n columns.
#define MOE_LAUNCH_SHAPE(name, K, a, m, n, s)                                                   \
  switch (tile_shape(m, n)) {                                                                   \
    case kBig:                                                                                  \
      return launch_tiles(name, K<256, 256>, a, ceil_div(m, 256) * ceil_div(n, 256), s);         \
    case kTall:                                                                                 \
      return launch_tiles(name, K<256, 128>, a, ceil_div(m, 256) * ceil_div(n, 128), s);         \
    case kWide:                                                                                 \
      return launch_tiles(name, K<128, 256>, a, ceil_div(m, 128) * ceil_div(n, 256), s);         \
    default:                                                                                    \
      return launch_tiles(name, K<128, 128>, a, ceil_div(m, 128) * ceil_div(n, 128), s);         \
  }

}  // namespace

hipError_t launch_ffn_gate_up(const FfnArgs& a, hipStream_t s) {
  MOE_LAUNCH_SHAPE("ffn_gate_up", ffn_gate_up_kernel, a, a.T, 2LL * a.I, s)
}
hipError_t launch_ffn_down(const FfnArgs& a, hipStream_t s) {
  MOE_LAUNCH_SHAPE("ffn_down", ffn_down_kernel, a, a.T, a.d, s)
}
hipError_t launch_ffn_dh(const FfnArgs& a, hipStream_t s) {
  MOE_LAUNCH_SHAPE("ffn_dh", ffn_dh_kernel, a, a.T, a.I, s)
}
hipError_t launch_ffn_dx(const FfnArgs& a, hipStream_t s) {
  MOE_LAUNCH_SHAPE("ffn_dx", ffn_dx_kernel, a, a.T, a.d, s)
}
hipError_t launch_ffn_dw(const FfnDwArgs& a, hipStream_t s) {
  MOE_LAUNCH_SHAPE(a.name, ffn_dw_kernel, a, a.Md, a.Nd, s)
}

}  // namespace moe
