// Block-scaled FP8: E4M3 codes with one fp32 scale per block of 128 along the reduction axis
// (activations: 1 x 128; weights: 128 x 128), the quantisers and the expert-grouped product.
//
// A block's scale is amax / 448 (1 for a block of zeros) and its codes are the values times
// 448 / amax, rounded to nearest even: the largest magnitude lands on E4M3's largest, 448. An
// amax below 2^-110 counts as 2^-110, so that neither quotient leaves fp32's normal numbers.
// A value that is not finite gets the NaN code (E4M3 has no infinity) and takes no part in amax:
// it spoils the sums it is in, and the codes beside it are as without it.
// The product takes each 128-deep block from one MFMA in fp32, then adds it, times the two scales,
// to the fp32 sum: out[p, n] = sum_kb sa[p, kb] sb[n / 128, kb] sum_k a[p, k] b[n, k].
//
// What the FP8 MFMAs keep (every one of gfx950's, measured with pairs of powers of two and with
// random codes): the products of eight consecutive k are added on a grid of about 2^-13 of the
// largest, the groups' sums then in fp32. On quantised Gaussian operands that is 1.3e-5 of the
// result in rms, 300 times less than the bf16 rounding of the output; bf16 MFMAs of the widened
// codes would keep 1e-8 at half the rate.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "ops.h"
#include "tiles8.h"

namespace moe {
namespace {

constexpr int kQB = 128;  // quantisation block

struct BlockScale {
  float scale, inv;
};
MOE_DEV BlockScale block_scale(float amax) {
  if (amax > 0.f) amax = fmaxf(amax, 0x1p-110f);
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
// The largest finite magnitude of eight bf16 values. Magnitudes order as their bits; with 0x80
// added those that are not finite (0x7f80 and above) become the negative 16-bit numbers.
MOE_DEV float amax8(const uint4& x) {
  typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
  typedef __attribute__((ext_vector_type(2))) short s16x2;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  s16x2 m = {0x80, 0x80};
#pragma unroll
  for (int q = 0; q < 4; ++q)
    m = __builtin_elementwise_max(
        m, __builtin_bit_cast(s16x2, __builtin_bit_cast(u16x2, w[q] & 0x7fff7fffu) +
                                         u16x2{0x80, 0x80}));
  return __uint_as_float((uint32_t)(max(m[0], m[1]) - 0x80) << 16);
}
// Two codes. No finite value of a block leaves E4M3's range: amax times 448 / amax, each rounded,
// is at most 448 and a step, which rounds to 448. The conversion makes NaN of what is not finite.
MOE_DEV uint32_t code2(float a, float b) {
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false)) & 0xffffu;
}
MOE_DEV uint2 codes8(const float (&f)[8], float inv) {
  return make_uint2(code2(f[0] * inv, f[1] * inv) | (code2(f[2] * inv, f[3] * inv) << 16),
                    code2(f[4] * inv, f[5] * inv) | (code2(f[6] * inv, f[7] * inv) << 16));
}

// A workgroup quantises 32 rows x 512 columns: a wave takes a row's 512 columns at a time, eight
// values a lane and sixteen lanes a block, eight rows one after the other with all their loads
// out at once. The scales of 32 consecutive rows leave as one 128-byte line: with one row a
// wave, each scale was a 4-byte store of its own to a line that workgroups on other XCDs wrote
// too. HBM bounds it: 16384 x 7168 in 58 us, 6.1 TB/s, two thirds of it reads.
// GATHER, in the layer: row pos of dY in position order, dy[row_src[pos] / k], for the rows
// before `placed` (skipped bad-index rows leave some; those are neither read nor written).
constexpr int kQRows = 32, kQCols = 512;
template <bool GATHER>
__global__ void __launch_bounds__(256) fp8_quant_rows_kernel(
    const uint16_t* __restrict__ src, const int32_t* __restrict__ row_src, int k,
    const int32_t* __restrict__ placed, int rows, int cols, uint8_t* __restrict__ codes,
    float* __restrict__ scales) {
  __shared__ float sc[kQCols / kQB][kQRows];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int nx = (cols + kQCols - 1) / kQCols;
  const int r0 = blockIdx.x / nx * kQRows, c = blockIdx.x % nx * kQCols + lane * 8;
  const int end = GATHER ? min(*placed, rows) : rows;
  if (r0 >= end) return;  // whole workgroup
  const bool on = c < cols;  // the same for the sixteen lanes of a block
  uint4 x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + wave * 8 + i;
    const bool live = on && r < end;
    const size_t at = GATHER ? (size_t)((live ? row_src[r] : 0) / k) : (size_t)r;
    const uint16_t* p = src + at * cols + c;
    // rows are read once: past the caches (66 -> 57 us a call); dY's rows k times
    x[i] = !live    ? make_uint4(0, 0, 0, 0)
           : GATHER ? *reinterpret_cast<const uint4*>(p)
                    : nt_load16(p);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + wave * 8 + i;
    float f[8];
    widen8(x[i], f);
    float amax = amax8(x[i]);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
    const BlockScale b = block_scale(amax);
    if (on && r < end) *reinterpret_cast<uint2*>(codes + (size_t)r * cols + c) = codes8(f, b.inv);
    if (lane % 16 == 0) sc[lane / 16][wave * 8 + i] = b.scale;
  }
  __syncthreads();
  const int kb = blockIdx.x % nx * (kQCols / kQB) + threadIdx.x / kQRows;
  const int r = r0 + threadIdx.x % kQRows;
  if (threadIdx.x < kQRows * (kQCols / kQB) && kb < cols / kQB && r < end)
    scales[(size_t)kb * rows + r] = sc[threadIdx.x / kQRows][threadIdx.x % kQRows];
}

// The layer's own operands, in position order: rows at and past offsets[E] (skipped bad-index
// rows leave some) are neither read nor written.
//
// A = silu(g) u from the stored H = [g | u], rounded to bf16 and quantised from that. A thread
// takes eight columns and sixteen threads a block, all in registers, so HBM bounds it: 16384 x
// 2048 (2048 tokens, k = 8) in 42 us, 5.6 TB/s with the codes.
__global__ void __launch_bounds__(256) fp8_swiglu_kernel(const uint16_t* __restrict__ H,
                                                         const int32_t* __restrict__ placed, int M,
                                                         int I, uint16_t* __restrict__ A,
                                                         uint8_t* __restrict__ codes,
                                                         float* __restrict__ scales) {
  const long long v = (long long)blockIdx.x * 256 + threadIdx.x;
  const int vpr = I / 8;
  const long long pos = v / vpr;
  if (pos >= min(*placed, M)) return;
  const int c = (int)(v - pos * vpr);
  const uint16_t* h = H + pos * 2 * I + c * 8;
  float g[8], u[8], f[8];
  widen8(*reinterpret_cast<const uint4*>(h), g);
  widen8(*reinterpret_cast<const uint4*>(h + I), u);
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    w[q] = pack_bf2(silu(g[2 * q]) * u[2 * q], silu(g[2 * q + 1]) * u[2 * q + 1]);
  const uint4 a = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(A)[v] = a;
  widen8(a, f);
  float amax = amax8(a);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
  const BlockScale b = block_scale(amax);
  reinterpret_cast<uint2*>(codes)[v] = codes8(f, b.inv);
  if (c % 16 == 0) scales[(size_t)(c / 16) * M + pos] = b.scale;
}

// The SwiGLU backward: dH = [dg | du] from dA' (bf16), H, A and the row's weight, rounded to bf16
// and quantised from that; and the router-weight gradient's partial <dA', A> of each 128 columns.
// In one pass, as above: 16384 x 2048 in 83 us, 5.6 TB/s.
__global__ void __launch_bounds__(256) fp8_swiglu_bwd_kernel(
    const uint16_t* __restrict__ dAp, const uint16_t* __restrict__ H,
    const uint16_t* __restrict__ A, const int32_t* __restrict__ row_src,
    const float* __restrict__ topk_w, const int32_t* __restrict__ placed, int M, int I,
    uint16_t* __restrict__ dH, uint8_t* __restrict__ codes, float* __restrict__ scales,
    float* __restrict__ dwpart) {
  const long long v = (long long)blockIdx.x * 256 + threadIdx.x;
  const int vpr = I / 8;
  const long long pos = v / vpr;
  if (pos >= min(*placed, M)) return;
  const int c = (int)(v - pos * vpr);
  const float wt = topk_w[row_src[pos]];
  const uint16_t* h = H + pos * 2 * I + c * 8;
  float dap[8], a[8], g[8], u[8];
  widen8(reinterpret_cast<const uint4*>(dAp)[v], dap);
  widen8(reinterpret_cast<const uint4*>(A)[v], a);
  widen8(*reinterpret_cast<const uint4*>(h), g);
  widen8(*reinterpret_cast<const uint4*>(h + I), u);
  float dg[8], du[8], part = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    part = __builtin_fmaf(dap[i], a[i], part);
    const float da = wt * dap[i], s = sigmoid(g[i]);
    dg[i] = da * u[i] * s * (1.0f + g[i] * (1.0f - s));
    du[i] = da * (g[i] * s);
  }
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) part += __shfl_xor(part, o);
  const int blk = c / 16, nb = I / kQB;
  if (c % 16 == 0) dwpart[pos * nb + blk] = part;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const float* d = half ? du : dg;
    const uint4 o = make_uint4(pack_bf2(d[0], d[1]), pack_bf2(d[2], d[3]), pack_bf2(d[4], d[5]),
                               pack_bf2(d[6], d[7]));
    const size_t at = pos * 2 * I + half * I + c * 8;
    *reinterpret_cast<uint4*>(dH + at) = o;
    float f[8];
    widen8(o, f);
    float amax = amax8(o);
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) amax = fmaxf(amax, __shfl_xor(amax, x));
    const BlockScale b = block_scale(amax);
    *reinterpret_cast<uint2*>(codes + at) = codes8(f, b.inv);
    if (c % 16 == 0) scales[(size_t)(half * nb + blk) * M + pos] = b.scale;
  }
}

// One workgroup per 128 x 128 block, which it reads once; the transposed copy goes through LDS.
// HBM bounds it: 8 x 4096 x 7168 with both copies in 180 us, 5.2 TB/s, half reads. (Transposes
// of 8 x 8 in registers instead of byte reads: 178.6 a call where these took 177.)
__global__ void __launch_bounds__(256) fp8_quant_weights_kernel(
    const uint16_t* __restrict__ src, int N, int K, uint8_t* __restrict__ codes,
    float* __restrict__ scales, uint8_t* __restrict__ codes_t, float* __restrict__ scales_t) {
  constexpr int P = kQB + 4;  // LDS row pitch in bytes
  __shared__ __align__(16) uint8_t tile[kQB * P];
  __shared__ float red[4];
  const int t = threadIdx.x, cv = t % 16;
  const int nN = N / kQB, nK = K / kQB;
  const int kb = blockIdx.x % nK, nb = blockIdx.x / nK;  // N / 128 may pass a grid's 65535 in y
  const size_t e = blockIdx.y;
  const uint16_t* s = src + (e * N + (size_t)nb * kQB) * K + (size_t)kb * kQB;
  uint4 x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    x[j] = *reinterpret_cast<const uint4*>(s + (size_t)(t / 16 + 16 * j) * K + cv * 8);
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, amax8(x[j]));
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
  if (t % 64 == 0) red[t / 64] = amax;
  __syncthreads();
  const BlockScale b = block_scale(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
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

MOE_DEV i32x8 fp8_frag(const uint8_t* rows16, const FragAt& f) {
  const i32x4 lo = *reinterpret_cast<const i32x4*>(rows16 + f.lo);
  const i32x4 hi = *reinterpret_cast<const i32x4*>(rows16 + f.hi);
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
// One block's product of 16 rows and 16 columns; with the columns first, lane l gets row l % 16,
// columns 4 (l / 16) .. + 3. (Both scale operands 0: the unscaled instruction.)
MOE_DEV f32x4 fp8_mfma(const i32x8& b, const i32x8& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0,
                                                          0, 0, 0, 0);
}

// Few rows an expert: the weights' stream is what takes the time. BM x 128 tiles, four waves of
// BM x 32; 128 bytes of K a step go from memory straight into LDS, the weights SB - 1 steps ahead
// and the rows one. The rows' scales ride in registers, one row a lane, and reach the lanes that
// need them through the LDS crossbar.
//  * BM = 128, three weight stages: 80 KB, two workgroups a CU to the last byte of its LDS, with
//    64 KB of weights on their way.
//  * BM = 32, two weight stages: 40 KB, four workgroups a CU with as much on their way.
// Tiles are dealt to the XCDs one by one: the column tiles of one expert run side by side on
// different XCDs (one XCD's consecutive tiles at a time: 1483 us against 1453 at 256 experts of 64
// rows). HBM bounds it: 256 experts of 64 rows, 4096 x 7168, in 1.39 ms, 5.6 TB/s.
// Weights that one row tile reads go past the caches (nt) up to 64 rows, where it pays
// (32 rows an expert 1274 -> 1207 us; 96 rows 1503 -> 1556).
// A tile's K loop is compiled for 2, 4, 6 and 8 blocks of 16 rows and runs the least that hold its
// rows: no MFMA, LDS read or load for the rest. (A test per block inside the loop made the
// compiler keep both sides' accumulators, 1 KB a lane of them in memory.)
// A wave's loads complete in order; a step issues rows, scales, then weights, so at its top the
// weight loads issued last may be missing if they are a step further ahead. Loads past the last
// block read it again into a stage nobody reads, so the counts hold.
template <int SB>
struct StreamLds {
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
template <int NMB, int SB>
struct StreamTile {
  static constexpr int AJ = NMB / 2;          // row loads a wave: 8 rows each
  static constexpr int SJ = (NMB + 3) / 4;    // scale registers: 64 rows each
  __amdgpu_buffer_rsrc_t ra, rb;
  uint32_t ao[AJ], bo[4];
  const float* sp[SJ];
  const float* sb;
  size_t M;
  float sv[SJ];
  int nK, wave, r16;
  FragAt f;
  f32x4 acc[NMB][2];

  template <int S>
  MOE_DEV void issue_a(const StreamLds<SB>& L, int kb) {
    const uint32_t step = (uint32_t)min(kb, nK - 1) * 128;
#pragma unroll
    for (int j = 0; j < AJ; ++j)
      load_lds16(ra, ao[j], step, L.template a<S>() + (wave * AJ + j) * 1024);
  }
  template <int S>
  MOE_DEV void issue_b(const StreamLds<SB>& L, int kb) {
    const uint32_t step = (uint32_t)min(kb, nK - 1) * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      load_lds16<NMB <= 4 ? 2 : 0>(rb, bo[j], step, L.template b<S>() + (wave * 4 + j) * 1024);
  }
  MOE_DEV void issue_s(int kb) {
    const size_t at = (size_t)min(kb, nK - 1) * M;
#pragma unroll
    for (int j = 0; j < SJ; ++j) sv[j] = sp[j][at];
  }
  template <int S>  // S: the step's number modulo the stages' common cycle
  MOE_DEV void step(const StreamLds<SB>& L, int kb) {
    __builtin_amdgcn_s_waitcnt(SB == 3 ? kVm4Lgkm0 : kVm0Lgkm0);
    __builtin_amdgcn_s_barrier();
    // the weights' scale does not change under the kernel: a scalar load
    const float sbk = ((const __attribute__((address_space(4))) float*)sb)[kb];
    float s[NMB];
#pragma unroll
    for (int mb = 0; mb < NMB; ++mb) s[mb] = __shfl(sv[mb / 4], mb % 4 * 16 + r16) * sbk;
    issue_a<(S + 1) % 2>(L, kb + 1);
    issue_s(kb + 1);
    loads_in_order();
    issue_b<(S + SB - 1) % SB>(L, kb + SB - 1);
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* A = L.template a<S % 2>();
    const uint8_t* B = L.template b<S % SB>() + wave * 4096;
    const i32x8 bf0 = fp8_frag(B, f), bf1 = fp8_frag(B + 2048, f);
#pragma unroll
    for (int mb = 0; mb < NMB; ++mb) {
      const i32x8 af = fp8_frag(A + mb * 2048, f);
      const f32x4 p0 = fp8_mfma(bf0, af), p1 = fp8_mfma(bf1, af);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        acc[mb][0][r] = __builtin_fmaf(s[mb], p0[r], acc[mb][0][r]);
        acc[mb][1][r] = __builtin_fmaf(s[mb], p1[r], acc[mb][1][r]);
      }
    }
  }
  template <int S, int C>  // steps kb + S, .. while fewer than C and n
  MOE_DEV void steps(const StreamLds<SB>& L, int kb, int n) {
    if constexpr (S < C) {
      if (S < n) {
        step<S>(L, kb + S);
        steps<S + 1, C>(L, kb, n);
      }
    }
  }
  MOE_DEV void run(const Fp8GemmArgs& a, const RowTile& t, int n0, const StreamLds<SB>& L) {
    const int lane = threadIdx.x % kWave;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    r16 = lane % 16;
    f = frag_at(lane);
    nK = a.K / kQB;
    M = a.M;
    ra = buf_rsrc(a.a + (size_t)t.row0 * a.K);
    rb = buf_rsrc(a.b + ((size_t)t.e * a.N + (size_t)n0 * kQB) * a.K);
    sb = a.sb + ((size_t)t.e * (a.N / kQB) + n0) * nK;
#pragma unroll
    for (int j = 0; j < AJ; ++j)  // rows past the count read the last one again
      ao[j] = (uint32_t)min(8 * (wave * AJ + j) + lane / 8, t.rows - 1) * a.K + lds_piece(lane);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      bo[j] = (uint32_t)(8 * (wave * 4 + j) + lane / 8) * a.K + lds_piece(lane);
#pragma unroll
    for (int j = 0; j < SJ; ++j) sp[j] = a.sa + t.row0 + min(64 * j + lane, t.rows - 1);
#pragma unroll
    for (int i = 0; i < NMB; ++i) acc[i][0] = acc[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    issue_b<0>(L, 0);
    issue_a<0>(L, 0);
    issue_s(0);
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
#pragma unroll
    for (int mb = 0; mb < NMB; ++mb) {
      const int m = mb * 16 + r16;
      if (m >= t.rows) continue;
      store_dw8_bf16<false>(
          a.out + (size_t)(t.row0 + m) * a.N + (size_t)n0 * kQB + wave * 32, acc[mb][0], acc[mb][1],
          lane);
    }
  }
};

template <int BM>
__global__ void __launch_bounds__(256, BM == 128 ? 2 : 4) fp8_stream_kernel(const Fp8GemmArgs a) {
  constexpr int SB = BM == 128 ? 3 : 2;
  __shared__ __align__(1024) uint8_t a0[BM * 128];
  __shared__ __align__(1024) uint8_t a1[BM * 128];
  __shared__ __align__(1024) uint8_t b0[kQB * 128];
  __shared__ __align__(1024) uint8_t b1[kQB * 128];
  __shared__ __align__(1024) uint8_t b2[SB == 3 ? kQB * 128 : 16];
  const StreamLds<SB> L{a0, a1, b0, b1, b2};
  const int nN = a.N / kQB;
  const int lt = blockIdx.x;
  const RowTile t = find_rows<BM>(a.offsets, a.M, a.E, lt / nN);
  if (t.rows <= 0) return;  // whole workgroup
  const int n0 = lt % nN;
  if (BM == 32 || t.rows <= 32) {
    StreamTile<2, SB> s;
    s.run(a, t, n0, L);
  } else if (t.rows <= 64) {
    StreamTile<4, SB> s;
    s.run(a, t, n0, L);
  } else if (t.rows <= 96) {
    StreamTile<6, SB> s;
    s.run(a, t, n0, L);
  } else {
    StreamTile<8, SB> s;
    s.run(a, t, n0, L);
  }
}

// Few column tiles: with a handful of experts the 128-column tiles leave most CUs without work,
// and a step's latency is what takes the time. One wave a workgroup takes 32 columns of 32 rows
// (eight stages) or 64 (five), about 64 KB on their way, two workgroups a CU, and no barrier: its
// loads complete in order and only it reads them. One expert of 32 rows, 4096 x 7168: 17 us, 1.7
// TB/s of weights, a wave's chain of 56 steps. Every value is summed in the other kernels'
// order. Loads past the last block read it again into a stage that is not read.
template <int NMB, int NS>
struct NarrowTile {
  static constexpr int AJ = 2 * NMB, G = AJ + 5;    // row loads, all loads of a step
  static constexpr int kA = NMB * 2048, kB = 4096, kStage = kA + kB + 256;
  static constexpr int kAhead = (NS - 1) * G;       // loads that may be missing at a step's top
  static_assert(kAhead < 64, "a wait counts 63 loads");
  static constexpr int kWait = 0x0f70 | (kAhead & 15) | (kAhead >> 4 << 14);  // vmcnt alone
  __amdgpu_buffer_rsrc_t ra, rb;
  uint32_t ao[AJ], bo[4], so;
  const float *sa, *sb;
  size_t M;
  int nK, lane;
  FragAt f;
  f32x4 acc[NMB][2];

  MOE_DEV void issue(uint8_t* st, int kb) {
    kb = min(kb, nK - 1);
    const uint32_t step = (uint32_t)kb * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j) load_lds16<2>(rb, bo[j], step, st + kA + j * 1024);
#pragma unroll
    for (int j = 0; j < AJ; ++j) load_lds16(ra, ao[j], step, st + j * 1024);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        buf_rsrc(sa + kb * M), (__attribute__((address_space(3))) void*)(st + kA + kB), 4, so, 0, 0,
        0);
  }
  MOE_DEV void step(uint8_t* st, int kb) {
    __builtin_amdgcn_s_waitcnt(kWait);
    __builtin_amdgcn_sched_barrier(0);
    const float sbk = ((const __attribute__((address_space(4))) float*)sb)[kb];
    const float* sc = reinterpret_cast<const float*>(st + kA + kB) + lane % 16;
    const i32x8 bf0 = fp8_frag(st + kA, f), bf1 = fp8_frag(st + kA + 2048, f);
    i32x8 af[NMB];
    float s[NMB];
#pragma unroll
    for (int mb = 0; mb < NMB; ++mb) {
      af[mb] = fp8_frag(st + mb * 2048, f);
      s[mb] = sc[mb * 16] * sbk;
    }
    __builtin_amdgcn_s_waitcnt(kLgkm0);  // read, so that the stage may be filled again
    __builtin_amdgcn_sched_barrier(0);
    issue(st, kb + NS);
#pragma unroll
    for (int mb = 0; mb < NMB; ++mb) {
      const f32x4 p0 = fp8_mfma(bf0, af[mb]), p1 = fp8_mfma(bf1, af[mb]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        acc[mb][0][r] = __builtin_fmaf(s[mb], p0[r], acc[mb][0][r]);
        acc[mb][1][r] = __builtin_fmaf(s[mb], p1[r], acc[mb][1][r]);
      }
    }
  }
  template <int S, int C>
  MOE_DEV void steps(uint8_t* const (&st)[NS], int kb, int n) {
    if constexpr (S < C) {
      if (S < n) {
        step(st[S], kb + S);
        steps<S + 1, C>(st, kb, n);
      }
    }
  }
  MOE_DEV void run(const Fp8GemmArgs& a, const RowTile& t, int n0,
                   uint8_t* const (&st)[NS]) {
    lane = threadIdx.x;
    f = frag_at(lane);
    nK = a.K / kQB;
    M = a.M;
    ra = buf_rsrc(a.a + (size_t)t.row0 * a.K);
    rb = buf_rsrc(a.b + ((size_t)t.e * a.N + n0) * a.K);
    sa = a.sa + t.row0;
    sb = a.sb + ((size_t)t.e * (a.N / kQB) + n0 / kQB) * nK;
#pragma unroll
    for (int j = 0; j < AJ; ++j)  // rows past the count read the last one again
      ao[j] = (uint32_t)min(8 * j + lane / 8, t.rows - 1) * a.K + lds_piece(lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) bo[j] = (uint32_t)(8 * j + lane / 8) * a.K + lds_piece(lane);
    so = (uint32_t)min(lane, t.rows - 1) * 4;
#pragma unroll
    for (int i = 0; i < NMB; ++i) acc[i][0] = acc[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      issue(st[i], i);
      loads_in_order();
    }
    int kb = 0;
    for (; kb + NS <= nK; kb += NS) steps<0, NS>(st, kb, NS);
    steps<0, NS - 1>(st, kb, nK - kb);
    __builtin_amdgcn_s_waitcnt(kVm0Lgkm0);  // before the workgroup gives its LDS back
#pragma unroll
    for (int mb = 0; mb < NMB; ++mb) {
      const int m = mb * 16 + lane % 16;
      if (m >= t.rows) continue;
      store_dw8_bf16<false>(a.out + (size_t)(t.row0 + m) * a.N + n0, acc[mb][0], acc[mb][1], lane);
    }
  }
};

template <int NMB>
__global__ void __launch_bounds__(64, 1) fp8_narrow_kernel(const Fp8GemmArgs a) {
  constexpr int kStage = NarrowTile<NMB, 5>::kStage, kMore = NMB == 2 ? kStage : 16;
  __shared__ __align__(1024) uint8_t s0[kStage];
  __shared__ __align__(1024) uint8_t s1[kStage];
  __shared__ __align__(1024) uint8_t s2[kStage];
  __shared__ __align__(1024) uint8_t s3[kStage];
  __shared__ __align__(1024) uint8_t s4[kStage];
  __shared__ __align__(1024) uint8_t s5[kMore];
  __shared__ __align__(1024) uint8_t s6[kMore];
  __shared__ __align__(1024) uint8_t s7[kMore];
  const int nN = a.N / 32;
  const RowTile t = find_rows<16 * NMB>(a.offsets, a.M, a.E, blockIdx.x / nN);
  if (t.rows <= 0) return;
  const int n0 = blockIdx.x % nN * 32;
  if constexpr (NMB == 2) {
    uint8_t* const st[8] = {s0, s1, s2, s3, s4, s5, s6, s7};
    NarrowTile<2, 8> w;
    w.run(a, t, n0, st);
  } else {
    uint8_t* const st[5] = {s0, s1, s2, s3, s4};
    if (t.rows <= 32) {
      NarrowTile<2, 5> w;
      w.run(a, t, n0, st);
    } else {
      NarrowTile<4, 5> w;
      w.run(a, t, n0, st);
    }
  }
}

// Many rows an expert: the MFMAs are what takes the time. 256 x 256 tiles, eight waves of 128 x 64,
// two stages of 64 KB filled straight from memory; one workgroup a CU, two waves a SIMD.
//
// The two waves of a SIMD take turns: while the one runs 16 MFMAs (half its row blocks by its
// columns, about 515 cycles) with the scaling of their results in the gaps, the other reads its
// next fragments from LDS. Waves w and w + 4 share a SIMD, so waves 4..7 run one phase behind,
// and a barrier ends each phase:
//     phase        4k        4k + 1    4k + 2    4k + 3    4k + 4
//     waves 0..3   read k.0  mfma k.0  read k.1  mfma k.1  read (k+1).0
//     waves 4..7   mfma ..   read k.0  mfma k.0  read k.1  mfma k.1
// Step k - 1's stage is read for the last time in phase 4k - 1 (a read phase ends with its reads
// returned), so a wave refills it for step k + 1 in its phase read k.0, and waits for its own
// loads at the end of read k.1, in phase 4k + 2 or 4k + 3; it is read from 4k + 4 on. Every wave
// runs the same code, the late ones behind one more barrier.
//
// 16384 rows over 5 of 8 experts, 4096 x 7168: 456 us, 2.11 PFLOP/s (128-row tiles above: 682).
// A library product of that size with one scale an operand takes 375; without the block scales
// this kernel took 422 a call where it took 445. The MFMAs are busy 59% of the time that tiles run;
// the rest is the phases' ends, a tile's first loads and its epilogue, and the last round.
constexpr int kBigCodes = kBigT * 128;                // one operand's codes of a step
constexpr int kBigStage = 2 * kBigCodes + kBigT * 4;  // rows, weights, the rows' scales
__shared__ __align__(1024) uint8_t fp8_big0[kBigStage];
__shared__ __align__(1024) uint8_t fp8_big1[kBigStage];
template <int S>
MOE_DEV uint8_t* fp8_big() {
  if constexpr (S == 0) return fp8_big0;
  else return fp8_big1;
}

// MB x NB blocks of 16 x 16 a wave: 8 x 4 (256 x 256 tiles), 8 x 2 (256 x 128), 4 x 2 (128 x 128).
template <int MB, int NB>
struct BigTile {
  static constexpr int BM = 32 * MB, BN = 64 * NB, HB = MB / 2;
  __amdgpu_buffer_rsrc_t ra, rb;
  uint32_t ao[HB], bo[NB], so;
  const float *sa, *sb;
  size_t M;
  int nK, wave, wm, wn;
  FragAt f;
  f32x4 acc[MB][NB];
  f32x4 last[3];  // the last products of a phase, and their scales
  float last_s[3];

  template <int S>
  MOE_DEV void issue(int kb) {
    uint8_t* st = fp8_big<S>();
    const uint32_t step = (uint32_t)kb * 128;
#pragma unroll
    for (int j = 0; j < NB; ++j)
      load_lds16(rb, bo[j], step, st + kBigCodes + (wave * NB + j) * 1024);
#pragma unroll
    for (int j = 0; j < HB; ++j) load_lds16(ra, ao[j], step, st + (wave * HB + j) * 1024);
    // 64 rows' scales a wave; several waves write the same
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        buf_rsrc(sa + kb * M),  // K / 128 rows of M may pass 32 bits
        (__attribute__((address_space(3))) void*)(st + 2 * kBigCodes + wave % (BM / 64) * 256), 4,
        so, 0, 0, 0);
  }
  MOE_DEV void phase_end() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  }
  // row blocks HB H .. of the step
  template <int S, int H>
  MOE_DEV void read(i32x8 (&af)[HB]) {
    const uint8_t* A = fp8_big<S>() + (wm * MB + H * HB) * 2048;
#pragma unroll
    for (int mb = 0; mb < HB; ++mb) af[mb] = fp8_frag(A + mb * 2048, f);
  }
  // The four FMAs that scale an MFMA's result go out while the third MFMA after it runs (left
  // alone, the compiler waits out each pair's latency before its FMAs); those of the last three
  // go out in the next phase, when the other waves have the MFMAs (finish).
  template <int H>
  MOE_DEV void multiply(const i32x8 (&bf)[NB], const i32x8 (&af)[HB], const float (&s)[MB],
                        float sbk) {
    constexpr int n = HB * NB;
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int mb = 0; mb < HB; ++mb) {
      const float sk = s[HB * H + mb] * sbk;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const f32x4 p = fp8_mfma(bf[nb], af[mb]);
        const int i = mb * NB + nb - (n - 3);
        if (i >= 0) {
          last[i] = p;
          last_s[i] = sk;
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[HB * H + mb][nb][r] = __builtin_fmaf(sk, p[r], acc[HB * H + mb][nb][r]);
        }
      }
    }
    // masks: 0x2 VALU, 0x8 MFMA
    __builtin_amdgcn_sched_group_barrier(0x2, HB, 0);
    __builtin_amdgcn_sched_group_barrier(0x8, 3, 0);
#pragma unroll
    for (int i = 3; i < n; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    }
    __builtin_amdgcn_s_setprio(0);
  }
  template <int H>
  MOE_DEV void finish() {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int at = HB * NB - 3 + i, mb = HB * H + at / NB, nb = at % NB;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[mb][nb][r] = __builtin_fmaf(last_s[i], last[i][r], acc[mb][nb][r]);
    }
  }
  template <int S>
  MOE_DEV void step(int kb) {
    i32x8 bf[NB], af[HB];
    float s[MB];
    issue<S ^ 1>(min(kb + 1, nK - 1));  // past the end: the last again, into a stage nobody reads
    // the weights' scale does not change under the kernel: a scalar load
    const float sbk = ((const __attribute__((address_space(4))) float*)sb)[kb];
    const uint8_t* B = fp8_big<S>() + kBigCodes + wn * NB * 2048;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) bf[nb] = fp8_frag(B + nb * 2048, f);
    const float* sc = reinterpret_cast<const float*>(fp8_big<S>() + 2 * kBigCodes) + wm * MB * 16 +
                      threadIdx.x % 16;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) s[mb] = sc[mb * 16];
    read<S, 0>(af);
    finish<1>();
    __builtin_amdgcn_s_waitcnt(kLgkm0);
    phase_end();
    multiply<0>(bf, af, s, sbk);
    phase_end();
    read<S, 1>(af);
    finish<0>();
    __builtin_amdgcn_s_waitcnt(kVm0Lgkm0);
    phase_end();
    multiply<1>(bf, af, s, sbk);
    phase_end();
  }
  // rows row0 .. of expert e and columns n0 .. of its weights (n0 a multiple of 128)
  MOE_DEV void run(const Fp8GemmArgs& a, int e, int row0, int rows, int n0) {
    const int lane = threadIdx.x % kWave;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    wm = wave / 4;
    wn = wave % 4;
    f = frag_at(lane);
    nK = a.K / kQB;
    M = a.M;
    ra = buf_rsrc(a.a + (size_t)row0 * a.K);
    rb = buf_rsrc(a.b + ((size_t)e * a.N + n0) * a.K);
    sa = a.sa + row0;
    const int cols = min(BN, a.N - n0);  // BN, or 128 at an odd end
    sb = a.sb + ((size_t)e * (a.N / kQB) + n0 / kQB + min(wn * NB * 16, cols - 1) / kQB) * nK;
    // rows past the end read the last one again
#pragma unroll
    for (int j = 0; j < HB; ++j)
      ao[j] = (uint32_t)min((wave * HB + j) * 8 + lane / 8, rows - 1) * a.K + lds_piece(lane);
#pragma unroll
    for (int j = 0; j < NB; ++j)
      bo[j] = (uint32_t)min((wave * NB + j) * 8 + lane / 8, cols - 1) * a.K + lds_piece(lane);
    so = (uint32_t)min(wave % (BM / 64) * 64 + lane, rows - 1) * 4;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      last[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      last_s[i] = 0.f;
    }
    issue<0>(0);
    __builtin_amdgcn_s_waitcnt(kVm0Lgkm0);
    phase_end();
    if (wm) phase_end();
    int kb = 0;
    for (; kb + 2 <= nK; kb += 2) {
      step<0>(kb);
      step<1>(kb + 1);
    }
    if (kb < nK) step<0>(kb);
    finish<1>();
    if (!wm) phase_end();  // as many barriers for the early waves as for the late ones
    const int c0 = wn * NB * 16;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const int m = (wm * MB + mb) * 16 + lane % 16;
      if (m >= rows || c0 >= cols) continue;
      uint16_t* row = a.out + (size_t)(row0 + m) * a.N + n0 + c0;
#pragma unroll
      for (int nb = 0; nb < NB; nb += 2)
        store_dw8_bf16<false>(row + nb * 16, acc[mb][nb], acc[mb][nb + 1], lane);
    }
  }
};

// Whole rounds of one tile a CU, then what is left: its tiles cut in two (256 x 128) or four
// (128 x 128) where the parts still fit one round, so that the last round takes half or a quarter
// of a tile's time. A tile's values do not depend on how it is cut.
__global__ void __launch_bounds__(512, 2) fp8_big_kernel(const Fp8GemmArgs a) {
  const int nN = (a.N + kBigT - 1) / kBigT;
  const int nm = big_count(a), tiles = nm * nN;
  const int whole = tiles / kCus * kCus, left = tiles - whole;
  const int cut = left * 4 <= kCus ? 4 : left * 2 <= kCus ? 2 : 1;
  const int b = blockIdx.x;
  int lt, part = 0;
  if (b < whole) {
    lt = xcd_contiguous(b, whole);
  } else {
    const int n8 = (left * cut + kXcds - 1) / kXcds * kXcds;
    if (b - whole >= n8) return;  // whole workgroups leave
    const int j = xcd_contiguous(b - whole, n8);
    if (j >= left * cut) return;
    lt = whole + j / cut;
    part = j % cut;
  }
  const int2 mn = big_order(lt, nm, nN);
  const RowTile t = big_rows(a, mn.x);
  const int n0 = mn.y * kBigT;
  if (t.rows <= 0) return;
  if (b < whole || cut == 1) {
    BigTile<8, 4> w;
    w.run(a, t.e, t.row0, t.rows, n0);
    return;
  }
  const int c = n0 + part % 2 * 128;
  if (c >= a.N) return;
  if (cut == 2) {
    BigTile<8, 2> w;
    w.run(a, t.e, t.row0, t.rows, c);
  } else {
    const int r = part / 2 * 128;
    if (r >= t.rows) return;
    BigTile<4, 2> w;
    w.run(a, t.e, t.row0 + r, min(t.rows - r, 128), c);
  }
}

}  // namespace

static dim3 quant_grid(int rows, int cols) {
  return dim3((unsigned)((rows + kQRows - 1) / kQRows) * (unsigned)((cols + kQCols - 1) / kQCols));
}
hipError_t launch_fp8_quant_rows(const uint16_t* src, int rows, int cols, uint8_t* codes,
                                 float* scales, hipStream_t s) {
  {
    TraceScope trace("fp8_quant_rows", s);
    hipLaunchKernelGGL(fp8_quant_rows_kernel<false>, quant_grid(rows, cols), dim3(256), 0, s, src,
                       nullptr, 1, nullptr, rows, cols, codes, scales);
  }
  return hipGetLastError();
}
static dim3 grid8(long long rows, int cols) {  // a thread for eight values
  return dim3((unsigned)((rows * cols / 8 + 255) / 256));
}
hipError_t launch_fp8_quant_gather(const uint16_t* src, const int32_t* row_src, int k,
                                   const int32_t* placed, int M, int cols, uint8_t* codes,
                                   float* scales, hipStream_t s) {
  {
    TraceScope trace("fp8_quant_dy", s);
    hipLaunchKernelGGL(fp8_quant_rows_kernel<true>, quant_grid(M, cols), dim3(256), 0, s, src,
                       row_src, k, placed, M, cols, codes, scales);
  }
  return hipGetLastError();
}
hipError_t launch_fp8_swiglu(const uint16_t* H, const int32_t* placed, int M, int I, uint16_t* A,
                             uint8_t* codes, float* scales, hipStream_t s) {
  {
    TraceScope trace("fp8_swiglu", s);
    hipLaunchKernelGGL(fp8_swiglu_kernel, grid8(M, I), dim3(256), 0, s, H, placed, M, I, A, codes,
                       scales);
  }
  return hipGetLastError();
}
hipError_t launch_fp8_swiglu_bwd(const Fp8SwigluBwdArgs& a, hipStream_t s) {
  {
    TraceScope trace("fp8_swiglu_bwd", s);
    hipLaunchKernelGGL(fp8_swiglu_bwd_kernel, grid8(a.M, a.I), dim3(256), 0, s, a.dAp, a.H, a.A,
                       a.row_src, a.topk_w, a.placed, a.M, a.I, a.dH, a.codes, a.scales, a.dwpart);
  }
  return hipGetLastError();
}

hipError_t launch_fp8_quant_weights(const uint16_t* src, int E, int N, int K, uint8_t* codes,
                                    float* scales, uint8_t* codes_t, float* scales_t,
                                    hipStream_t s) {
  {
    TraceScope trace("fp8_quant_weights", s);
    hipLaunchKernelGGL(fp8_quant_weights_kernel, dim3((unsigned)(K / kQB) * (N / kQB), E),
                       dim3(256), 0, s, src, N, K, codes, scales, codes_t, scales_t);
  }
  return hipGetLastError();
}

// Which kernel, by the rows an expert has on average and the 128-column tiles there may be (M, E
// and N are all the host knows of the load; every kernel is right for every load). Measured in us,
// rows spread evenly, N x K = 4096 x 7168 where not said:
//  * up to 128 tiles, rows few: narrow. E = 1, 32 rows 17 (128-row tiles 34); E = 4, 16 rows an
//    expert 20 (36). At 256 tiles level: E = 8, 16 rows 39 (42), 64 rows 66 (62).
//  * up to 16 rows an expert and 513 to 704 tiles with rows in them: 32-row tiles. 128-row tiles
//    run two a CU, and their second round is then nearly empty. All with rows, 2 or 16 an expert:
//    512 tiles level (69 and 70 both), 520 81 (128-row tiles 99 and 100), 640 90 and 93 (107 and
//    111); 768 102 and 127 (112 and 118), 896 132 and 137 (120 and 131), 1024 141 and 147 (135 and
//    145). The host counts the experts that have rows as if M rows were dealt at random: 7168 x
//    2048, 24 rows on 11 of 16 experts 30.7 (33.5); 6144 x 7168, 32 on 13 of 16 86 (106), 64 on all
//    16 123 (112). A load less even than that is not seen: 64 of those rows on 13 experts take 105
//    (32-row tiles 86).
//  * up to 112 rows an expert: 128-row tiles. E = 64, 96 rows 369 (256 x 256 tiles 463). Above, an
//    expert's rows begin to need a second tile and its weights a second read: 160 rows 710 (482).
hipError_t launch_fp8_gemm(const Fp8GemmArgs& a, hipStream_t s) {
  auto grid = [&](int bm, int bn) {
    const unsigned n = (unsigned)(a.M / bm + a.E) * (unsigned)((a.N + bn - 1) / bn);
    return dim3((n + kXcds - 1) / kXcds * kXcds);
  };
  const long long M = a.M, E = a.E, tiles = E * (a.N / kQB);
  const double busy = (double)tiles * -std::expm1(-(double)M / (double)E);
  TraceScope trace("fp8_gemm", s);
  if (tiles <= kCus / 2 && M <= 32)
    hipLaunchKernelGGL(fp8_narrow_kernel<2>, grid(32, 32), dim3(64), 0, s, a);
  else if (tiles <= kCus / 2 && M <= 64 * E)
    hipLaunchKernelGGL(fp8_narrow_kernel<4>, grid(64, 32), dim3(64), 0, s, a);
  else if (busy > 2 * kCus && busy <= 2.75 * kCus && M <= 16 * E)
    hipLaunchKernelGGL(fp8_stream_kernel<32>, grid(32, kQB), dim3(256), 0, s, a);
  else if (M <= 112 * E)
    hipLaunchKernelGGL(fp8_stream_kernel<128>, grid(128, kQB), dim3(256), 0, s, a);
  else  // room for every tile, and for a last round's parts
    hipLaunchKernelGGL(fp8_big_kernel, dim3(grid(kBigT, kBigT).x + kCus), dim3(512), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
