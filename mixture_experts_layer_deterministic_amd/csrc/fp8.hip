// Block-scaled FP8: E4M3 codes with one fp32 scale per block of 128 along the reduction axis
// (activations: 1 x 128; weights: 128 x 128), the quantisers and the expert-grouped product.
//
// A block's scale is amax / 448 (1 for a block of zeros) and its codes are the values times
// 448 / amax, rounded to nearest even: the largest magnitude lands on E4M3's largest, 448.
// The product takes each 128-deep block from one MFMA in fp32, then adds it, times the two scales,
// to the fp32 sum: out[p, n] = sum_kb sa[p, kb] sb[n / 128, kb] sum_k a[p, k] b[n, k].
//
// What the FP8 MFMAs keep (every one of gfx950's, measured with pairs of powers of two and with
// random codes): the products of eight consecutive k are added on a grid of about 2^-13 of the
// largest, the groups' sums then in fp32. On quantised Gaussian operands that is 1.3e-5 of the
// result in rms, 300 times less than the bf16 rounding of the output; bf16 MFMAs of the widened
// codes would keep 1e-8 at half the rate.
#include "common.h"
#include "kernels.h"
#include "ops.h"

namespace moe {
namespace {

constexpr int kQB = 128;  // quantisation block

struct BlockScale {
  float scale, inv;
};
MOE_DEV BlockScale block_scale(float amax) {
  return amax > 0.f ? BlockScale{amax / 448.f, 448.f / amax} : BlockScale{1.f, 1.f};
}
MOE_DEV void widen8(const uint4& x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = bf2f_lo(w[q]);
    f[2 * q + 1] = bf2f_hi(w[q]);
  }
}
MOE_DEV float amax8(const float (&f)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  return m;
}
MOE_DEV uint2 codes8(const float (&f)[8], float inv) {
  return make_uint2(e4m3x2(f[0] * inv, f[1] * inv) | (e4m3x2(f[2] * inv, f[3] * inv) << 16),
                    e4m3x2(f[4] * inv, f[5] * inv) | (e4m3x2(f[6] * inv, f[7] * inv) << 16));
}

// Sixteen lanes of eight values make one block.
__global__ void __launch_bounds__(256) fp8_quant_rows_kernel(const uint16_t* __restrict__ src,
                                                             int rows, int cols,
                                                             uint8_t* __restrict__ codes,
                                                             float* __restrict__ scales) {
  const long long v = (long long)blockIdx.x * 256 + threadIdx.x;
  const bool live = v < (long long)rows * cols / 8;
  const uint4 x = live ? reinterpret_cast<const uint4*>(src)[v] : make_uint4(0, 0, 0, 0);
  float f[8];
  widen8(x, f);
  float amax = amax8(f);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
  const BlockScale b = block_scale(amax);
  if (live) {
    reinterpret_cast<uint2*>(codes)[v] = codes8(f, b.inv);
    if (v % 16 == 0) {
      const long long blk = v / 16;
      const int nkb = cols / kQB;
      scales[(size_t)(blk % nkb) * rows + blk / nkb] = b.scale;
    }
  }
}

// One workgroup per 128 x 128 block, which it reads once; the transposed copy goes through LDS.
__global__ void __launch_bounds__(256) fp8_quant_weights_kernel(
    const uint16_t* __restrict__ src, int N, int K, uint8_t* __restrict__ codes,
    float* __restrict__ scales, uint8_t* __restrict__ codes_t, float* __restrict__ scales_t) {
  constexpr int P = kQB + 4;  // LDS row pitch in bytes
  __shared__ __align__(16) uint8_t tile[kQB * P];
  __shared__ float red[4];
  const int t = threadIdx.x, cv = t % 16;
  const int kb = blockIdx.x, nb = blockIdx.y;
  const size_t e = blockIdx.z;
  const uint16_t* s = src + (e * N + (size_t)nb * kQB) * K + (size_t)kb * kQB;
  uint4 x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    x[j] = *reinterpret_cast<const uint4*>(s + (size_t)(t / 16 + 16 * j) * K + cv * 8);
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float f[8];
    widen8(x[j], f);
    amax = fmaxf(amax, amax8(f));
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
  if (t % 64 == 0) red[t / 64] = amax;
  __syncthreads();
  const BlockScale b = block_scale(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
  const int nN = N / kQB, nK = K / kQB;
  if (t == 0) {
    scales[(e * nN + nb) * nK + kb] = b.scale;
    if (scales_t) scales_t[(e * nK + kb) * nN + nb] = b.scale;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float f[8];
    widen8(x[j], f);
    const uint2 c = codes8(f, b.inv);
    const int r = t / 16 + 16 * j;
    *reinterpret_cast<uint2*>(codes + (e * N + (size_t)nb * kQB + r) * K + (size_t)kb * kQB +
                              cv * 8) = c;
    *reinterpret_cast<uint32_t*>(tile + r * P + cv * 8) = c.x;
    *reinterpret_cast<uint32_t*>(tile + r * P + cv * 8 + 4) = c.y;
  }
  if (!codes_t) return;
  __syncthreads();
  // column c's 128 codes leave as 16-byte pieces
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int v = t + 256 * j, c = v / 8, r0 = v % 8 * 16;
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i / 4] |= (uint32_t)tile[(r0 + i) * P + c] << (8 * (i % 4));
    *reinterpret_cast<uint4*>(codes_t + (e * K + (size_t)kb * kQB + c) * N + (size_t)nb * kQB +
                              r0) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ------------------------------------------------------------------------------------------
// The product

// Row tiles without a table. Expert e's tiles take the slots from offsets[e] / BM + e on: the
// next expert's first slot is at least that plus ceil(rows / BM), since floor((o + c) / BM) + 1
// >= floor(o / BM) + ceil(c / BM). M / BM + E slots hold every tile, whatever the load; a slot
// finds its expert from the offsets alone, and the ones between two experts' tiles do nothing.
struct RowTile {
  int e, row0, rows;  // rows <= 0: nothing to do
};
template <int BM>
MOE_DEV RowTile find_rows(const int32_t* __restrict__ offsets, int M, int E, int slot) {
  // the last expert whose first slot is at most this one: starts ascend, so it is a count
  const int lane = threadIdx.x % kWave;
  int n = 0;
  for (int e0 = 0; e0 < E; e0 += kWave) {
    const int e = e0 + lane;
    const bool le = e < E && min(max(offsets[e], 0), M) / BM + e <= slot;
    const int c = __popcll(__ballot(le));
    n += c;
    if (c < kWave) break;
  }
  RowTile t{0, 0, 0};
  n = __builtin_amdgcn_readfirstlane(n);
  if (n == 0) return t;  // offsets[0] > 0, and no expert starts this early
  t.e = n - 1;
  const int o = min(max(offsets[t.e], 0), M), end = min(max(offsets[t.e + 1], 0), M);
  const int i = slot - (o / BM + t.e);
  t.row0 = o + i * BM;
  t.rows = i < 0 ? 0 : min(end - t.row0, BM);  // i < 0: the offsets do not ascend
  return t;
}

typedef __attribute__((ext_vector_type(4))) int i32x4;
MOE_DEV int fp8_swz(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }
MOE_DEV i32x8 fp8_frag(const uint8_t* tile, int row, int g) {
  const i32x4 lo = *reinterpret_cast<const i32x4*>(tile + fp8_swz(row, g));
  const i32x4 hi = *reinterpret_cast<const i32x4*>(tile + fp8_swz(row, 4 + g));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// 128 x 128 tiles, four waves of 64 x 64, a step per 128-deep block.
__global__ void __launch_bounds__(256, 2) fp8_gemm_kernel(const Fp8GemmArgs a) {
  __shared__ __align__(16) uint8_t lds[2 * kQB * 128];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int wm = wave / 2, wn = wave % 2, r16 = lane % 16, g = lane / 16;
  const int nN = a.N / kQB, nK = a.K / kQB;
  const int n0 = blockIdx.x % nN;
  const RowTile t = find_rows<128>(a.offsets, a.M, a.E, blockIdx.x / nN);
  if (t.rows <= 0) return;
  const uint8_t* ap[4];
  const uint8_t* bp[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int v = tid + 256 * j, r = v / 8;
    ap[j] = a.a + (size_t)(t.row0 + min(r, t.rows - 1)) * a.K + v % 8 * 16;
    bp[j] = a.b + ((size_t)t.e * a.N + (size_t)n0 * kQB + r) * a.K + v % 8 * 16;
  }
  const float* sb = a.sb + ((size_t)t.e * nN + n0) * nK;
  int srow[4];
#pragma unroll
  for (int mb = 0; mb < 4; ++mb) srow[mb] = t.row0 + min(wm * 64 + mb * 16 + r16, t.rows - 1);
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  i32x4 av[4], bv[4];
  auto load = [&](int kb) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bv[j] = *reinterpret_cast<const i32x4*>(bp[j] + (size_t)kb * 128);
      av[j] = *reinterpret_cast<const i32x4*>(ap[j] + (size_t)kb * 128);
    }
  };
  load(0);
  for (int kb = 0; kb < nK; ++kb) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = tid + 256 * j;
      *reinterpret_cast<i32x4*>(lds + fp8_swz(v / 8, v % 8)) = av[j];
      *reinterpret_cast<i32x4*>(lds + kQB * 128 + fp8_swz(v / 8, v % 8)) = bv[j];
    }
    __syncthreads();
    if (kb + 1 < nK) load(kb + 1);
    float s[4];
#pragma unroll
    for (int mb = 0; mb < 4; ++mb) s[mb] = a.sa[(size_t)kb * a.M + srow[mb]] * sb[kb];
    i32x8 bf[4];
#pragma unroll
    for (int nb = 0; nb < 4; ++nb)
      bf[nb] = fp8_frag(lds + kQB * 128, wn * 64 + nb * 16 + r16, g);
#pragma unroll
    for (int mb = 0; mb < 4; ++mb) {
      const i32x8 af = fp8_frag(lds, wm * 64 + mb * 16 + r16, g);
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        const f32x4 blk = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            bf[nb], af, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[mb][nb][r] = __builtin_fmaf(s[mb], blk[r], acc[mb][nb][r]);
      }
    }
  }
#pragma unroll
  for (int mb = 0; mb < 4; ++mb) {
    const int m = wm * 64 + mb * 16 + r16;
    if (m >= t.rows) continue;
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      const size_t at = (size_t)(t.row0 + m) * a.N + n0 * kQB + wn * 64 + nb * 16 + 4 * g;
      const f32x4 v = acc[mb][nb];
      *reinterpret_cast<uint2*>(a.out + at) =
          make_uint2(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]));
    }
  }
}

}  // namespace

hipError_t launch_fp8_quant_rows(const uint16_t* src, int rows, int cols, uint8_t* codes,
                                 float* scales, hipStream_t s) {
  const long long nv = (long long)rows * cols / 8;
  {
    TraceScope trace("fp8_quant_rows", s);
    hipLaunchKernelGGL(fp8_quant_rows_kernel, dim3((unsigned)((nv + 255) / 256)), dim3(256), 0, s,
                       src, rows, cols, codes, scales);
  }
  return hipGetLastError();
}

hipError_t launch_fp8_quant_weights(const uint16_t* src, int E, int N, int K, uint8_t* codes,
                                    float* scales, uint8_t* codes_t, float* scales_t,
                                    hipStream_t s) {
  {
    TraceScope trace("fp8_quant_weights", s);
    hipLaunchKernelGGL(fp8_quant_weights_kernel, dim3(K / kQB, N / kQB, E), dim3(256), 0, s, src,
                       N, K, codes, scales, codes_t, scales_t);
  }
  return hipGetLastError();
}

hipError_t launch_fp8_gemm(const Fp8GemmArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)(a.M / 128 + a.E) * (unsigned)(a.N / kQB);
  {
    TraceScope trace("fp8_gemm", s);
    hipLaunchKernelGGL(fp8_gemm_kernel, dim3(grid), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace moe
