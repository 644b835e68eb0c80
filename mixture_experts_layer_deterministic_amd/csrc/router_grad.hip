// Gradients of the router's linear map l = x Wr^T from any gradient dl of its logits:
//   dx[t]  (+)= sum_e dl[t, e] Wr[e]      T x d, reduced over the experts
//   dWr[e] (+)= sum_t dl[t, e] x[t]       E x d, reduced over the tokens
//
// dl is fp32 and x, Wr are bf16. Each dl value is split into three bf16 parts, the rounding of
// what the parts before left over: h + m + l keeps 24 bits, the products of the parts with bf16
// values are exact in fp32, and three bf16 MFMAs do an fp32 product's work at a rate that
// fp32 MFMAs (1/16 of bf16's) do not reach.
#include "common.h"
#include "kernels.h"
#include "ops.h"

namespace moe {
namespace {

constexpr int kRgB = 128;     // tile rows and columns
constexpr int kRgK = 32;      // reduction depth of a step
constexpr int kRgPlane = kRgB * kRgK;  // uint16 of one part of a step's dl tile
constexpr int kRgStage = 4 * kRgPlane;  // three parts, then the bf16 operand

// Element offset of 16-byte chunk c of row r in a tile of 32-value rows, chunks permuted so that
// the 16 rows a fragment read touches spread over the banks.
MOE_DEV int rg_row(int r, int c) { return r * kRgK + ((c ^ ((r >> 1) & 3)) << 3); }

MOE_DEV void split3(float x, uint32_t& h, uint32_t& m, uint32_t& l) {
  h = f2bf(x);
  const float r = x - bf2f((uint16_t)h);
  m = f2bf(r);
  l = f2bf(r - bf2f((uint16_t)m));
}

// Workgroup tiles: first the dWr tiles (the longer reductions), then the dx tiles, so that the
// long ones start first. Four waves of 64 x 64.
__global__ void __launch_bounds__(256, 2) router_backward_kernel(const RouterGradArgs a) {
  __shared__ __align__(16) uint16_t lds[kRgStage];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int wm = wave / 2, wn = wave % 2;
  const int nc = a.d / kRgB;
  const int nw = a.dwr ? (a.E + kRgB - 1) / kRgB * nc : 0;
  const bool dw = (int)blockIdx.x < nw;
  const int b = dw ? blockIdx.x : blockIdx.x - nw;
  const int r0 = b / nc * kRgB, c0 = b % nc * kRgB;  // output rows (experts or tokens), columns
  const int R = dw ? a.E : a.T, K = dw ? a.T : a.E;
  const uint16_t* bsrc = dw ? a.x : a.wr;
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // this thread's 16 dl values of a step: dx, row tid / 2 and 16 experts; dWr, token tid / 8 and
  // 16 experts
  const int ar = dw ? tid / 8 : tid / 2, ac = dw ? tid % 8 * 16 : tid % 2 * 16;
  float av[16];
  uint4 bv[2];
  auto load = [&](int k0) {
    const int t = dw ? k0 + ar : r0 + ar, e0 = dw ? r0 + ac : k0 + ac;
    const float* p = a.dl + (size_t)t * a.E + e0;
#pragma unroll
    for (int i = 0; i < 16; ++i) av[i] = t < a.T && e0 + i < a.E ? p[i] : 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int v = tid + 256 * j, kr = k0 + v / 16;
      bv[j] = kr < K ? *reinterpret_cast<const uint4*>(bsrc + (size_t)kr * a.d + c0 + v % 16 * 8)
                     : make_uint4(0, 0, 0, 0);
    }
  };
  auto store = [&] {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t w[3][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t h0, m0, l0, h1, m1, l1;
        split3(av[8 * q + 2 * i], h0, m0, l0);
        split3(av[8 * q + 2 * i + 1], h1, m1, l1);
        w[0][i] = h0 | (h1 << 16);
        w[1][i] = m0 | (m1 << 16);
        w[2][i] = l0 | (l1 << 16);
      }
      const int at = dw ? ar * kRgB + ((ac + 8 * q) ^ kmajor_swz(ar)) : rg_row(ar, ac / 8 + q);
#pragma unroll
      for (int s = 0; s < 3; ++s)
        *reinterpret_cast<uint4*>(lds + s * kRgPlane + at) =
            make_uint4(w[s][0], w[s][1], w[s][2], w[s][3]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int v = tid + 256 * j, kr = v / 16;
      *reinterpret_cast<uint4*>(lds + 3 * kRgPlane + kr * kRgB + ((v % 16 * 8) ^ kmajor_swz(kr))) =
          bv[j];
    }
  };
  load(0);
  for (int k0 = 0; k0 < K; k0 += kRgK) {
    __syncthreads();
    store();
    __syncthreads();
    if (k0 + kRgK < K) load(k0 + kRgK);
    uint4 bf[4];
#pragma unroll
    for (int nb = 0; nb < 4; ++nb)
      bf[nb] = kmajor_frag<kRgB>(lds + 3 * kRgPlane, wn * 64 + nb * 16, 0, lane);
#pragma unroll
    for (int mb = 0; mb < 4; ++mb) {
      const int m = wm * 64 + mb * 16;
#pragma unroll
      for (int s = 2; s >= 0; --s) {  // the small parts first
        const uint16_t* pl = lds + s * kRgPlane;
        const uint4 af = dw ? kmajor_frag<kRgB>(pl, m, 0, lane)
                            : *reinterpret_cast<const uint4*>(pl + rg_row(m + lane % 16, lane / 16));
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) acc[mb][nb] = mfma16(bf[nb], af, acc[mb][nb]);
      }
    }
  }
#pragma unroll
  for (int mb = 0; mb < 4; ++mb) {
    const int r = r0 + wm * 64 + mb * 16 + lane % 16;
    if (r >= R) continue;
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      const int c = c0 + wn * 64 + nb * 16 + 4 * (lane / 16);
      f32x4 v = acc[mb][nb];
      if (dw) {
        float* p = a.dwr + (size_t)r * a.d + c;
        if (a.acc_dwr) store_dw4<true>(p, v);
        else store_dw4<false>(p, v);
      } else {
        // one rounding to bf16, of the fp32 sum with what dx held
        uint2* p = reinterpret_cast<uint2*>(a.dx + (size_t)r * a.d + c);
        if (a.acc_dx) {
          const uint2 o = *p;
          v[0] += bf2f_lo(o.x);
          v[1] += bf2f_hi(o.x);
          v[2] += bf2f_lo(o.y);
          v[3] += bf2f_hi(o.y);
        }
        *p = make_uint2(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]));
      }
    }
  }
}

}  // namespace

hipError_t launch_router_backward(const RouterGradArgs& a, hipStream_t s) {
  const int nc = a.d / kRgB;
  const int grid = ((a.dwr ? (a.E + kRgB - 1) / kRgB : 0) +
                    (a.dx ? (a.T + kRgB - 1) / kRgB : 0)) * nc;
  {
    TraceScope trace("router_backward", s);
    hipLaunchKernelGGL(router_backward_kernel, dim3(grid), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace moe
